"""PyTorch plumbing around the C ABI of the standalone operators (include/flint_ops.h).

As in `layer`, PyTorch supplies device memory and streams only; every step runs in the library's CUDA
kernels. Shapes, types and strides are checked here (ValueError) or by the C entry points (FlintError).
Outputs that are not given are allocated; no gradients are recorded. Work goes to `stream` (default: the current stream of
the inputs' device); an input written on another stream must have been ordered before it by the caller. With `stream`, the
call's tensors are recorded on it, so that they may be dropped as soon as the call returns. Allocated outputs belong to it,
and are recorded on the caller's stream, which reads them when it has been ordered behind the call.

Waits inside the kernels are bounded. Should one give up, its call's output is incomplete and `error_word` says so.

The smallest calls take a few microseconds on the device, so the common path (tensors of the current
device, its current stream) goes straight to the entry point.
"""

from __future__ import annotations

import torch

from . import binding as B

_TYPES = {torch.bfloat16: B.FLINT_T_BF16, torch.float16: B.FLINT_T_F16}
_FORMATS = {"int4": B.FLINT_W_INT4_G128_FWHT128, "nvfp4": B.FLINT_W_NVFP4}
_ACTS = {None: B.FLINT_ACT_NONE, "none": B.FLINT_ACT_NONE, "swiglu": B.FLINT_ACT_SWIGLU}
_SCALES = {"int4": (torch.bfloat16,), "nvfp4": (torch.float8_e4m3fn, torch.uint8)}
_GATES = {None: B.FLINT_GATE_NONE, "none": B.FLINT_GATE_NONE, "sigmoid": B.FLINT_GATE_SIGMOID}

_current_device = torch.cuda.current_device


def _current_stream(index: int) -> int:
    return torch.cuda.current_stream(index).cuda_stream


# the same handle without building a Stream object around it, where torch offers that
_stream_of = getattr(torch._C, "_cuda_getCurrentRawStream", _current_stream)


def _elsewhere(device, stream) -> bool:
    """Whether a call must switch device or stream first."""
    return stream is not None or device.type != "cuda" or device.index != _current_device()


def _used_on(stream, *values) -> None:
    """The memory of the tensors among `values` is not handed out again before the work that `stream` then holds is done."""
    for v in values:
        if isinstance(v, torch.Tensor) and v.device == stream.device:
            v.record_stream(stream)


def _switched(fn, device, stream, *args, **kw):
    """fn with `stream` current (its device too), or with the tensors' device current."""
    if device.type != "cuda":
        raise ValueError("the operators run on CUDA tensors only")
    if stream is None:
        with torch.cuda.device(device):
            return fn(*args, **kw)
    _need(stream.device == device, "the stream belongs to another device than the tensors")
    caller = torch.cuda.current_stream(device)
    try:
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
        _used_on(caller, *(out if isinstance(out, tuple) else (out,)))
        return out
    finally:
        _used_on(stream, *args, *kw.values())


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


# Sizes cross the C boundary as 32-bit integers, which ctypes would cut without a word. Checked all at once: their OR has a
# high bit, or the sign, where one of them has it.
_INT_MAX = 2 ** 31 - 1


def _refuse_size() -> None:
    raise ValueError("a negative size, or one of 2^31 or more: the operators take at most 2^31 - 1")


def _together(device, *tensors) -> None:
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError(f"a tensor is on {t.device}, not on {device}")


def _rows(t: torch.Tensor, name: str) -> int:
    """Elements between the rows of a matrix whose columns are neighbours."""
    if t.is_contiguous() and t.dim() == 2:
        return t.shape[1]
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a matrix with contiguous rows")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def q4_linear(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, tscale: torch.Tensor | None = None, *,
              fmt: str = "int4", rotated: bool = True, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T][N] = x [T][K] W^T with W in a 4-bit storage format (flint_q4_linear).

    codes u8 [N][K/2]; scales bf16 [N][K/128] ("int4") or float8_e4m3fn / uint8 [N][K/16] ("nvfp4", which is
    never rotated); tscale f32 [1]. x may be rows of a wider matrix (row stride a multiple of 8 elements)."""
    dev = x.device
    if _elsewhere(dev, stream):
        return _switched(q4_linear, dev, stream, x, codes, scales, tscale, fmt=fmt, rotated=rotated, y=y)
    f, dt = _FORMATS.get(fmt), _TYPES.get(x.dtype)
    if f is None or dt is None:
        raise ValueError(f"format {fmt!r} with {x.dtype} activations")
    ldx = _rows(x, "x")
    T, K = x.shape
    N = codes.shape[0]
    if not 0 <= (T | K | N) <= _INT_MAX:
        _refuse_size()
    group = 128 if fmt == "int4" else 16
    if codes.dtype != torch.uint8 or codes.shape != (N, K // 2) or K % 2 or not codes.is_contiguous():
        raise ValueError("codes must be contiguous u8 [N][K/2]")
    if scales.shape != (N, K // group) or scales.dtype not in _SCALES[fmt] or not scales.is_contiguous():
        raise ValueError("scales must be contiguous bf16 [N][K/128] (int4) or E4M3 [N][K/16] (nvfp4)")
    if tscale is not None and (tscale.dtype != torch.float32 or tscale.numel() != 1):
        raise ValueError("tscale must be f32 [1]")
    _together(dev, codes, scales, tscale, y)
    if y is None:
        y, ldy = x.new_empty((T, N)), N
    else:
        _need(y.shape == (T, N) and y.dtype == x.dtype, "y must be [T][N] of x's type")
        ldy = _rows(y, "y")
    need = B.flint_q4_linear_workspace_size(K, T)
    ws = x.new_empty((need,), dtype=torch.uint8) if need else None
    B.flint_q4_linear(f, N, K, 1 if rotated and group == 128 else 0, codes.data_ptr(), scales.data_ptr(),
                      0 if tscale is None else tscale.data_ptr(), x.data_ptr(), ldx, T, dt, y.data_ptr(), ldy,
                      ws.data_ptr() if need else 0, need, _stream_of(dev.index))
    return y


def quantize_linear(w: torch.Tensor, *, fmt: str = "int4", rotate: bool = True, stream=None) -> tuple:
    """bf16 w [N][K] -> (codes, scales, tscale) for q4_linear, by the library's quantisers (flint_quant.h);
    tscale is None for int4."""
    if _elsewhere(w.device, stream):
        return _switched(quantize_linear, w.device, stream, w, fmt=fmt, rotate=rotate)
    _need(fmt in _FORMATS and w.dtype == torch.bfloat16 and w.dim() == 2 and w.is_contiguous(),
          "w must be contiguous bf16 [N][K]")
    N, K = w.shape
    if not 0 <= (N | K) <= _INT_MAX:
        _refuse_size()
    _need(N > 0 and K % (128 if fmt == "int4" else 16) == 0, "K must be a multiple of the scale group")
    s = _stream_of(w.device.index)
    codes = w.new_empty((N, K // 2), dtype=torch.uint8)
    if fmt == "int4":
        scales = w.new_empty((N, K // 128))
        B.flint_quantize_int4_g128(w.data_ptr(), N, K, rotate, codes.data_ptr(), scales.data_ptr(), s)
        return codes, scales, None
    scales = w.new_empty((N, K // 16), dtype=torch.float8_e4m3fn)
    tscale = w.new_empty((1,), dtype=torch.float32)
    B.flint_quantize_nvfp4(w.data_ptr(), 1, N, K, codes.data_ptr(), scales.data_ptr(), tscale.data_ptr(), s)
    return codes, scales, tscale


def grouped_linear(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, *, rows: torch.Tensor | None = None,
                   row_div: int = 1, act: str | None = None, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Row p of y, offsets[e] <= p < offsets[e+1], is W[e] x[rows[p] // row_div] (x[p] without rows), with
    act="swiglu" silu(gate) * up of W's two halves (flint_grouped_linear).

    x [x_rows][K], w [E][N][K] contiguous, offsets int32 [E+1], rows int32 [P]. Rows of y at or behind
    offsets[E] are left as they were (uninitialised when y is allocated here)."""
    dev = x.device
    if _elsewhere(dev, stream):
        return _switched(grouped_linear, dev, stream, x, w, offsets, rows=rows, row_div=row_div, act=act, y=y)
    a, dt = _ACTS.get(act), _TYPES.get(x.dtype)
    if a is None or dt is None or w.dtype != x.dtype:
        raise ValueError(f"act {act!r} with {x.dtype} activations and {w.dtype} weights")
    ldx = _rows(x, "x")
    if w.dim() != 3 or not w.is_contiguous() or w.shape[2] != x.shape[1]:
        raise ValueError("w must be contiguous [E][N][K]")
    E, N, K = w.shape
    if offsets.dtype != torch.int32 or offsets.shape != (E + 1,) or not offsets.is_contiguous():
        raise ValueError("offsets must be contiguous int32 [E+1]")
    if rows is None:
        P = x.shape[0]
    else:
        if rows.dtype != torch.int32 or rows.dim() != 1 or not rows.is_contiguous():
            raise ValueError("rows must be contiguous int32 [P]")
        P = rows.shape[0]
    if not 0 <= (E | N | K | x.shape[0] | P | row_div) <= _INT_MAX:
        _refuse_size()
    _together(dev, w, offsets, rows, y)
    nout = N // 2 if a else N
    if y is None:
        y, ldy = x.new_empty((P, nout)), nout
    else:
        _need(y.shape == (P, nout) and y.dtype == x.dtype, "y must be [P][N], [P][N/2] with swiglu, of x's type")
        ldy = _rows(y, "y")
    B.flint_grouped_linear(E, N, K, a, dt, w.data_ptr(), x.data_ptr(), ldx, x.shape[0],
                           0 if rows is None else rows.data_ptr(), row_div, offsets.data_ptr(), P, y.data_ptr(), ldy,
                           _stream_of(dev.index))
    return y


def expert_permute(ids: torch.Tensor, n_experts: int, *, stream=None) -> tuple:
    """ids int32 [T][top_k] -> (offsets [E+1], perm [T*top_k], inv [T][top_k]), all int32: the expert-major
    order of the (token, slot) pairs. Ids outside [0, E) are dropped (flint_expert_permute)."""
    dev = ids.device
    if _elsewhere(dev, stream):
        return _switched(expert_permute, dev, stream, ids, n_experts)
    if ids.dtype != torch.int32 or ids.dim() != 2 or not ids.is_contiguous() or n_experts < 1:
        raise ValueError("ids must be contiguous int32 [T][top_k], and at least one expert")
    T, K = ids.shape
    if not 0 <= (T | K | n_experts) <= _INT_MAX:
        _refuse_size()
    offsets, perm, inv = ids.new_empty((n_experts + 1,)), ids.new_empty((T * K,)), ids.new_empty((T, K))
    B.flint_expert_permute(ids.data_ptr(), T, K, n_experts, offsets.data_ptr(), perm.data_ptr(), inv.data_ptr(),
                           _stream_of(dev.index))
    return offsets, perm, inv


def expert_combine(o: torch.Tensor, inv: torch.Tensor, w: torch.Tensor, *, addend: torch.Tensor | None = None,
                   scale: float = 1.0, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y[t] = scale * sum_k w[t][k] o[inv[t][k]] + addend[t]; slots with inv < 0 are skipped
    (flint_expert_combine). o [P][H], inv int32 and w f32 [T][top_k], addend [T][H] (may be y)."""
    dev = o.device
    if _elsewhere(dev, stream):
        return _switched(expert_combine, dev, stream, o, inv, w, addend=addend, scale=scale, y=y)
    dt = _TYPES.get(o.dtype)
    if dt is None:
        raise ValueError(f"expert rows of {o.dtype}")
    ldo = _rows(o, "o")
    if inv.dtype != torch.int32 or inv.dim() != 2 or not inv.is_contiguous():
        raise ValueError("inv must be contiguous int32 [T][top_k]")
    if w.dtype != torch.float32 or w.shape != inv.shape or not w.is_contiguous():
        raise ValueError("w must be contiguous f32 [T][top_k]")
    T, K = inv.shape
    P, H = o.shape
    if not 0 <= (T | K | P | H) <= _INT_MAX:
        _refuse_size()
    add = lda = 0
    if addend is not None:
        _need(addend.shape == (T, H) and addend.dtype == o.dtype, "addend must be [T][H] of o's type")
        add, lda = addend.data_ptr(), _rows(addend, "addend")
    _together(dev, inv, w, addend, y)
    if y is None:
        y, ldy = o.new_empty((T, H)), H
    else:
        _need(y.shape == (T, H) and y.dtype == o.dtype, "y must be [T][H] of o's type")
        ldy = _rows(y, "y")
    B.flint_expert_combine(o.data_ptr(), ldo, P, inv.data_ptr(), w.data_ptr(), T, K, H, scale, add, lda, dt, y.data_ptr(),
                           ldy, _stream_of(dev.index))
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
    dev = x.device
    if _elsewhere(dev, stream):
        return _switched(block_norm, dev, stream, x, y, post_norm=post_norm, post_weight=post_weight, gate=gate,
                         gate_act=gate_act, res_scale=res_scale, branch_scale=branch_scale, pre_weight=pre_weight, eps=eps,
                         x_out=x_out, z=z, z_dtype=z_dtype)
    ldx = _rows(x, "x")
    shape = x.shape
    T, H = shape
    if not 0 <= (T | H) <= _INT_MAX:
        _refuse_size()
    xt = x.dtype
    dt = y.dtype if y is not None else z.dtype if z is not None else z_dtype or (
        xt if xt in _TYPES else torch.bfloat16)
    t, act = _TYPES.get(dt), _GATES.get(gate_act)
    if z_dtype is not None and z_dtype != dt:
        raise ValueError(f"z_dtype {z_dtype} where the branch or z is {dt}")
    if t is None or act is None or (xt != torch.float32 and xt != dt):
        raise ValueError(f"a {xt} residual with a {dt} branch, gate_act {gate_act!r}")
    py = ldy = pg = ldg = 0
    if y is not None:
        _need(y.shape == shape, "y must be [T][H]")
        py, ldy = y.data_ptr(), _rows(y, "y")
    if gate is not None:
        _need(gate.dtype == dt and tuple(gate.shape) in ((T, H), (1, H), (H,)) and (H == 1 or gate.stride(-1) == 1),
              "gate must be [T][H] or [H] of the branch's type, with contiguous rows")
        pg, ldg = gate.data_ptr(), _rows(gate, "gate") if gate.dim() == 2 and gate.shape[0] == T and T > 1 else 0
    wt, pp, pq = B.FLINT_T_F32, 0, 0
    if post_weight is not None or pre_weight is not None:
        both = post_weight if post_weight is not None else pre_weight
        for v in (post_weight, pre_weight):
            if v is not None and (v.shape != (H,) or v.dtype != both.dtype or not v.is_contiguous()):
                raise ValueError("the weights must be contiguous [H] of one type")
        if both.dtype != torch.float32:
            _need(both.dtype == dt, "the weights must be fp32 or of the branch's type")
            wt = t
        pp = 0 if post_weight is None else post_weight.data_ptr()
        pq = 0 if pre_weight is None else pre_weight.data_ptr()
    _together(dev, y, gate, post_weight, pre_weight, x_out, z)
    if x_out is None:
        x_out, ldxo = x.new_empty(shape), H
    else:
        _need(x_out.shape == shape and x_out.dtype == xt, "x_out must be [T][H] of x's type")
        ldxo = _rows(x_out, "x_out")
    if z is None:
        z, ldz = x.new_empty(shape, dtype=dt), H
    else:
        _need(z.shape == shape and z.dtype == dt, "z must be [T][H] of the branch's type")
        ldz = _rows(z, "z")
    B.flint_block_norm(B.pack_norm_args(x.data_ptr(), x_out.data_ptr(), py, pg, pp, pq, z.data_ptr(), ldx, ldxo, ldy, ldg, ldz,
                                        T, H, t, B.FLINT_T_F32 if xt == torch.float32 else t, wt, 1 if post_norm else 0, act,
                                        res_scale, branch_scale, eps), _stream_of(dev.index))
    return x_out, z


def error_word(device=None) -> int:
    """0, or the timeout bit (4) when a wait inside a kernel of q4_linear or grouped_linear gave up on this device (default:
    the current one) since the last call: what that kernel wrote is incomplete. Waits for the device and clears the word
    (flint_ops_error_word)."""
    with torch.cuda.device(device):
        return B.flint_ops_error_word()


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

    def error_word(self) -> int:
        """The operators' error word of the weights' device (ops.error_word)."""
        return error_word(self.gate_up.device)

    def forward(self, x: torch.Tensor, ids: torch.Tensor, w: torch.Tensor, *, addend: torch.Tensor | None = None,
                scale: float = 1.0, stream=None) -> torch.Tensor:
        """y[t] = scale * sum_k w[t][k] E_ids[t][k](x[t]) + addend[t]: ids int32 [T][top_k] (outside [0, E):
        no expert), w f32 [T][top_k], addend [T][H] (a shared expert's output)."""
        if _elsewhere(x.device, stream):
            if stream is not None:
                _used_on(stream, self.gate_up, self.down)
            return _switched(self.forward, x.device, stream, x, ids, w, addend=addend, scale=scale)
        _need(x.dim() == 2 and ids.dim() == 2 and x.shape[0] == ids.shape[0], "x [T][H] and ids [T][top_k]")
        offsets, perm, inv = expert_permute(ids, self.E)
        h = grouped_linear(x, self.gate_up, offsets, rows=perm, row_div=ids.shape[1], act="swiglu")
        o = grouped_linear(h, self.down, offsets)
        return expert_combine(o, inv, w, addend=addend, scale=scale)
