"""PyTorch plumbing around the C ABI of the standalone operators (include/flint_ops.h).

As in `layer`, PyTorch supplies device memory and streams only; every step runs in the library's CUDA
kernels. Shapes, types and strides are checked here (ValueError) or by the C entry points (FlintError).
Outputs that are not given are allocated. Work goes to `stream` (default: the current stream of the
inputs' device); an input written on another stream must have been ordered before it by the caller.
"""

from __future__ import annotations

import torch

from . import binding as B

_TYPES = {torch.bfloat16: B.FLINT_T_BF16, torch.float16: B.FLINT_T_F16}
_FORMATS = {"int4": B.FLINT_W_INT4_G128_FWHT128, "nvfp4": B.FLINT_W_NVFP4}
_ACTS = {None: B.FLINT_ACT_NONE, "none": B.FLINT_ACT_NONE, "swiglu": B.FLINT_ACT_SWIGLU}
_GATES = {None: B.FLINT_GATE_NONE, "none": B.FLINT_GATE_NONE, "sigmoid": B.FLINT_GATE_SIGMOID}


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _check_cuda(device, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")


def _rows(t: torch.Tensor, name: str) -> int:
    """Elements between the rows of a matrix whose columns are neighbours."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _on_stream(fn, device, stream, *args, **kw):
    """Runs fn with `stream` current (its device too), or with the tensors' device current."""
    if device.type != "cuda":
        raise ValueError("the operators run on CUDA tensors only")
    if stream is not None:
        _need(stream.device == device, "the stream belongs to another device than the tensors")
        with torch.cuda.stream(stream):
            return fn(stream.cuda_stream, *args, **kw)
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            return fn(torch.cuda.current_stream(device).cuda_stream, *args, **kw)
    return fn(torch.cuda.current_stream(device).cuda_stream, *args, **kw)


def _ptr(t) -> int:
    return 0 if t is None else t.data_ptr()


def q4_linear(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, tscale: torch.Tensor | None = None, *,
              fmt: str = "int4", rotated: bool = True, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T][N] = x [T][K] W^T with W in a 4-bit storage format (flint_q4_linear).

    codes u8 [N][K/2]; scales bf16 [N][K/128] ("int4") or float8_e4m3fn / uint8 [N][K/16] ("nvfp4", which is
    never rotated); tscale f32 [1]. x may be rows of a wider matrix (row stride a multiple of 8 elements)."""
    return _on_stream(_q4_linear, x.device, stream, x, codes, scales, tscale, fmt, rotated, y)


def _q4_linear(stream, x, codes, scales, tscale, fmt, rotated, y):
    if fmt not in _FORMATS or x.dtype not in _TYPES:
        raise ValueError(f"format {fmt!r} with {x.dtype} activations")
    ldx = _rows(x, "x")
    T, K = x.shape
    N = codes.shape[0]
    _need(codes.dtype == torch.uint8 and codes.shape == (N, K // 2) and K % 2 == 0 and codes.is_contiguous(),
          "codes must be contiguous u8 [N][K/2]")
    if fmt == "int4":
        _need(scales.dtype in (torch.bfloat16, torch.int16) and scales.shape == (N, K // 128), "scales must be bf16 [N][K/128]")
    else:
        rotated = False
        _need(scales.element_size() == 1 and scales.shape == (N, K // 16), "scales must be E4M3 [N][K/16]")
    _need(scales.is_contiguous(), "scales must be contiguous")
    _need(tscale is None or (tscale.dtype == torch.float32 and tscale.numel() == 1), "tscale must be f32 [1]")
    _check_cuda(x.device, codes=codes, scales=scales, tscale=tscale, y=y)
    if y is None:
        y = torch.empty((T, N), dtype=x.dtype, device=x.device)
    else:
        _need(y.shape == (T, N) and y.dtype == x.dtype, "y must be [T][N] of x's type")
    need = B.flint_q4_linear_workspace_size(K, T)
    ws = torch.empty((need,), dtype=torch.uint8, device=x.device) if need else None
    B.flint_q4_linear(_FORMATS[fmt], N, K, 1 if rotated else 0, codes.data_ptr(), scales.data_ptr(), _ptr(tscale),
                      x.data_ptr(), ldx, T, _TYPES[x.dtype], y.data_ptr(), _rows(y, "y"), _ptr(ws), need, stream)
    return y


def quantize_linear(w: torch.Tensor, *, fmt: str = "int4", rotate: bool = True, stream=None) -> tuple:
    """bf16 w [N][K] -> (codes, scales, tscale) for q4_linear, by the library's quantisers (flint_quant.h);
    tscale is None for int4."""
    _need(fmt in _FORMATS and w.dtype == torch.bfloat16 and w.dim() == 2 and w.is_contiguous(),
          "w must be contiguous bf16 [N][K]")
    _need(w.shape[0] > 0 and w.shape[1] % (128 if fmt == "int4" else 16) == 0, "K must be a multiple of the scale group")
    return _on_stream(_quantize_linear, w.device, stream, w, fmt, rotate)


def _quantize_linear(stream, w, fmt, rotate):
    N, K = w.shape
    codes = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    if fmt == "int4":
        scales = torch.empty((N, K // 128), dtype=torch.bfloat16, device=w.device)
        B.flint_quantize_int4_g128(w.data_ptr(), N, K, rotate, codes.data_ptr(), scales.data_ptr(), stream)
        return codes, scales, None
    scales = torch.empty((N, K // 16), dtype=torch.float8_e4m3fn, device=w.device)
    tscale = torch.empty((1,), dtype=torch.float32, device=w.device)
    B.flint_quantize_nvfp4(w.data_ptr(), 1, N, K, codes.data_ptr(), scales.data_ptr(), tscale.data_ptr(), stream)
    return codes, scales, tscale


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *, rows: torch.Tensor | None = None,
                   row_div: int = 1, act: str | None = None, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Row p of y, offsets[e] <= p < offsets[e+1], is W[e] x[rows[p] // row_div] (x[p] without rows), with
    act="swiglu" silu(gate) * up of W's two halves (flint_grouped_linear).

    x [x_rows][K], w [E][N][K] contiguous, offsets int32 [E+1], rows int32 [P]. Rows of y at or behind
    offsets[E] are left as they were (uninitialised when y is allocated here)."""
    return _on_stream(_grouped_linear, x.device, stream, x, w, offsets, rows, row_div, act, y)


def _grouped_linear(stream, x, w, offsets, rows, row_div, act, y):
    if act not in _ACTS or x.dtype not in _TYPES or w.dtype != x.dtype:
        raise ValueError(f"act {act!r} with {x.dtype} activations and {w.dtype} weights")
    ldx = _rows(x, "x")
    _need(w.dim() == 3 and w.is_contiguous() and w.shape[2] == x.shape[1], "w must be contiguous [E][N][K]")
    E, N, K = w.shape
    _need(offsets.dtype == torch.int32 and offsets.shape == (E + 1,) and offsets.is_contiguous(),
          "offsets must be int32 [E+1]")
    _need(rows is None or (rows.dtype == torch.int32 and rows.dim() == 1 and rows.is_contiguous()), "rows must be int32 [P]")
    _check_cuda(x.device, w=w, offsets=offsets, rows=rows, y=y)
    P = x.shape[0] if rows is None else rows.shape[0]
    a = _ACTS[act]
    nout = N // 2 if a else N
    if y is None:
        y = torch.empty((P, nout), dtype=x.dtype, device=x.device)
    else:
        _need(y.shape == (P, nout) and y.dtype == x.dtype, "y must be [P][N], [P][N/2] with swiglu, of x's type")
    B.flint_grouped_linear(E, N, K, a, _TYPES[x.dtype], w.data_ptr(), x.data_ptr(), ldx, x.shape[0], _ptr(rows), row_div,
                           offsets.data_ptr(), P, y.data_ptr(), _rows(y, "y"), stream)
    return y


def expert_permute(ids: torch.Tensor, n_experts: int, *, stream=None) -> tuple:
    """ids int32 [T][top_k] -> (offsets [E+1], perm [T*top_k], inv [T][top_k]), all int32: the expert-major
    order of the (token, slot) pairs. Ids outside [0, E) are dropped (flint_expert_permute)."""
    return _on_stream(_expert_permute, ids.device, stream, ids, n_experts)


def _expert_permute(stream, ids, E):
    _need(ids.dtype == torch.int32 and ids.dim() == 2 and ids.is_contiguous(), "ids must be contiguous int32 [T][top_k]")
    T, K = ids.shape
    offsets = torch.empty((max(int(E), 0) + 1,), dtype=torch.int32, device=ids.device)
    perm = torch.empty((T * K,), dtype=torch.int32, device=ids.device)
    inv = torch.empty((T, K), dtype=torch.int32, device=ids.device)
    B.flint_expert_permute(ids.data_ptr(), T, K, int(E), offsets.data_ptr(), perm.data_ptr(), inv.data_ptr(), stream)
    return offsets, perm, inv


def expert_combine(o: torch.Tensor, inv: torch.Tensor, w: torch.Tensor, *, addend: torch.Tensor | None = None,
                   scale: float = 1.0, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = scale * sum_k w[t][k] o[inv[t][k]] + addend[t]; slots with inv < 0 are skipped
    (flint_expert_combine). o [P][H], inv int32 and w f32 [T][top_k], addend [T][H] (may be y)."""
    return _on_stream(_expert_combine, o.device, stream, o, inv, w, addend, scale, y)


def _expert_combine(stream, o, inv, w, addend, scale, y):
    if o.dtype not in _TYPES:
        raise ValueError(f"expert rows of {o.dtype}")
    ldo = _rows(o, "o")
    _need(inv.dtype == torch.int32 and inv.dim() == 2 and inv.is_contiguous(), "inv must be contiguous int32 [T][top_k]")
    _need(w.dtype == torch.float32 and w.shape == inv.shape and w.is_contiguous(), "w must be contiguous f32 [T][top_k]")
    T, K = inv.shape
    P, H = o.shape
    _need(addend is None or (addend.shape == (T, H) and addend.dtype == o.dtype), "addend must be [T][H] of o's type")
    _check_cuda(o.device, inv=inv, w=w, addend=addend, y=y)
    if y is None:
        y = torch.empty((T, H), dtype=o.dtype, device=o.device)
    else:
        _need(y.shape == (T, H) and y.dtype == o.dtype, "y must be [T][H] of o's type")
    B.flint_expert_combine(o.data_ptr(), ldo, P, inv.data_ptr(), w.data_ptr(), T, K, H, scale, _ptr(addend),
                           0 if addend is None else _rows(addend, "addend"), _TYPES[o.dtype], y.data_ptr(),
                           _rows(y, "y"), stream)
    return y


def block_norm(x: torch.Tensor, y: torch.Tensor | None = None, *, post_norm: bool = False,
               post_weight: torch.Tensor | None = None, gate: torch.Tensor | None = None, gate_act: str | None = None,
               res_scale: float = 1.0, branch_scale: float = 1.0, pre_weight: torch.Tensor | None = None,
               eps: float = 1e-6, x_out: torch.Tensor | None = None, z: torch.Tensor | None = None,
               z_dtype: torch.dtype | None = None, stream=None) -> tuple:
    """The residual step around a block (flint_block_norm): b = post-norm of the branch y (or y itself),
    x' = res_scale x + branch_scale act(gate) b, z = pre-norm of x'. Returns (x', z).

    x [T][H] fp32 or the branch's type; y [T][H]; gate [T][H], [1][H] or [H]; weights [H], fp32 or the branch's
    type (both the same). x_out may be x (in place). z has the branch's type (z_dtype without a branch)."""
    return _on_stream(_block_norm, x.device, stream, x, y, post_norm, post_weight, gate, gate_act, res_scale,
                      branch_scale, pre_weight, eps, x_out, z, z_dtype)


def _block_norm(stream, x, y, post_norm, post_weight, gate, gate_act, res_scale, branch_scale, pre_weight, eps, x_out, z,
                z_dtype):
    ldx = _rows(x, "x")
    T, H = x.shape
    dt = y.dtype if y is not None else z.dtype if z is not None else z_dtype or (
        x.dtype if x.dtype in _TYPES else torch.bfloat16)
    if dt not in _TYPES or x.dtype not in (torch.float32, dt) or gate_act not in _GATES:
        raise ValueError(f"a {x.dtype} residual with a {dt} branch, gate_act {gate_act!r}")
    _need(y is None or y.shape == (T, H), "y must be [T][H]")
    ldg = 0
    if gate is not None:
        _need(gate.dtype == dt and tuple(gate.shape) in ((T, H), (1, H), (H,)), "gate must be [T][H] or [H] of the branch's type")
        ldg = _rows(gate, "gate") if gate.dim() == 2 and gate.shape[0] == T and T > 1 else 0
        _need(H == 1 or gate.stride(-1) == 1, "gate must have contiguous rows")
    wt = torch.float32
    for name, v in (("post_weight", post_weight), ("pre_weight", pre_weight)):
        if v is not None:
            _need(v.shape == (H,) and v.dtype in (torch.float32, dt) and v.is_contiguous(),
                  f"{name} must be contiguous [H], fp32 or the branch's type")
            wt = v.dtype
    _need(post_weight is None or pre_weight is None or post_weight.dtype == pre_weight.dtype, "both weights have one type")
    _check_cuda(x.device, y=y, gate=gate, post_weight=post_weight, pre_weight=pre_weight, x_out=x_out, z=z)
    if x_out is None:
        x_out = torch.empty((T, H), dtype=x.dtype, device=x.device)
    if z is None:
        z = torch.empty((T, H), dtype=dt, device=x.device)
    _need(x_out.shape == (T, H) and x_out.dtype == x.dtype, "x_out must be [T][H] of x's type")
    _need(z.shape == (T, H) and z.dtype == dt, "z must be [T][H] of the branch's type")
    a = B.flint_norm_args(x.data_ptr(), x_out.data_ptr(), _ptr(y), _ptr(gate), _ptr(post_weight), _ptr(pre_weight),
                          z.data_ptr(), ldx, _rows(x_out, "x_out"), 0 if y is None else _rows(y, "y"), ldg, _rows(z, "z"),
                          T, H, _TYPES[dt], B.FLINT_T_F32 if x.dtype == torch.float32 else _TYPES[dt],
                          B.FLINT_T_F32 if wt == torch.float32 else _TYPES[dt], 1 if post_norm else 0, _GATES[gate_act],
                          res_scale, branch_scale, eps)
    B.flint_block_norm(a, stream)
    return x_out, z


class FlintExperts16:
    """The layer's routed experts kept in 16 bits (the type their checkpoint has them in, before
    flint_quantize_*), run on a routing the caller gives, as FlintMoELayer.forward_routed runs the 4-bit ones.

    gate_up [E][2I][H] (gate rows, then up rows) and down [E][H][I], bf16 or fp16, on one device; any widths that
    flint_grouped_linear takes. Holds references to the weights and no other device memory."""

    def __init__(self, gate_up: torch.Tensor, down: torch.Tensor):
        E, two_i, H = gate_up.shape
        _need(two_i % 2 == 0 and tuple(down.shape) == (E, H, two_i // 2) and down.dtype == gate_up.dtype,
              "gate_up must be [E][2I][H] and down [E][H][I] of one type")
        self.gate_up, self.down = gate_up, down
        self.E, self.H, self.I = E, H, two_i // 2

    def forward(self, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, *, addend: torch.Tensor | None = None,
                scale: float = 1.0, stream=None) -> torch.Tensor:
        """y[t] = scale * sum_k w[t][k] E_ids[t][k](x[t]) + addend[t]: ids int32 [T][top_k] (outside [0, E):
        no expert), w f32 [T][top_k], addend [T][H] (a shared expert's output)."""
        _need(x.dim() == 2 and ids.dim() == 2 and x.shape[0] == ids.shape[0], "x [T][H] and ids [T][top_k]")
        offsets, perm, inv = expert_permute(ids, self.E, stream=stream)
        h = grouped_linear(x, self.gate_up, offsets, rows=perm, row_div=ids.shape[1], act="swiglu", stream=stream)
        o = grouped_linear(h, self.down, offsets, stream=stream)
        return expert_combine(o, inv, w, addend=addend, scale=scale, stream=stream)
