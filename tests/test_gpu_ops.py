"""The standalone operators on the GPU against their fp64 oracle (oracle/ops_ref.py).

Tolerances. An output of type t carries one rounding: u_t |ref| with u_t half a step (bf16 2^-8, fp16 2^-11),
plus half the smallest subnormal step of fp16. Before it, an fp32 sum of n products taken in any order with
intermediate rounding is within n 2^-23 of sum |w x| (2^-24 per addition, doubled because the tensor cores may
truncate); the kernels add 16 products per step at least and join at most 64 partial sums, so n = K/16 + 80.
Rotated activations are rounded once to 16 bits of at least fp16's precision per element: 2^-11 of sum |w' x'|
more. Over a whole output the roundings are independent, so the error's norm stays below (u_t + 2^-11 if rotated)
times the result's norm, a bound that a wrong element or group breaks at once."""

import os
import subprocess
import sys

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # collected on CPU-only machines, skipped there
    pytest.skip("no CUDA device", allow_module_level=True)

from bit_routed_expert_sigmoid_b200 import binding as B  # noqa: E402
from bit_routed_expert_sigmoid_b200 import ops  # noqa: E402
from oracle import flint_moe_ref as R  # noqa: E402
from oracle import ops_ref as O  # noqa: E402

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
TYPES = [torch.bfloat16, torch.float16]


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def close(got, ref, dtype, slack=0.0, norm_extra=0.0, rows=None):
    got, ref = f64(got), np.asarray(ref)
    if rows is not None:
        got, ref, slack = got[rows], ref[rows], (slack[rows] if isinstance(slack, np.ndarray) else slack)
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    tol = U[dtype] * (np.abs(ref) + slack) + slack + (2.0 ** -25 if dtype == torch.float16 else 0.0)
    assert np.all(err <= tol), float((err / np.maximum(tol, 1e-300)).max())
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(err) <= (U[dtype] + norm_extra + 2.0 ** -20) * norm + 2.0 ** -25 * np.sqrt(ref.size)


# ------------------------------------------------------------------------------------------ 4-bit linear

def q4_case(fmt, N, K, T, dtype, seed, pad=0, hot=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((T, K + pad), generator=g) * 1.26
    if hot:
        x[:, torch.randint(0, K, (1 + K // 512,), generator=g)] *= 50.0
    x = x.to(dtype).cuda()[:, :K]
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    if fmt == "int4":
        scales = (torch.randn((N, K // 128), generator=g) * 0.01).to(torch.bfloat16)
        ts = None
    else:
        scales = (torch.randn((N, K // 16), generator=g).abs() * 4).to(torch.float8_e4m3fn)
        ts = torch.tensor([0.013])
    return x, codes.cuda(), scales.cuda(), ts.cuda() if ts is not None else None


def q4_reference(x, codes, scales, ts, fmt, rotated):
    bits = scales.cpu().view(torch.int16 if fmt == "int4" else torch.uint8).numpy()
    bits = bits.view(np.uint16) if fmt == "int4" else bits
    tsv = None if ts is None else ts.item()
    xd = f64(x)
    ref = O.q4_linear(xd, fmt, codes.cpu().numpy(), bits, tsv, rotated)
    xa = np.abs(R.rotate_segments(xd) if rotated else xd)
    mass = xa @ np.abs(O.q4_weight(fmt, codes.cpu().numpy(), bits, tsv)).T
    n = x.shape[1] / 16 + 80
    return ref, mass * (n * 2.0 ** -23 + (2.0 ** -11 if rotated else 0.0))


Q4_SHAPES = [(1, 128, 1), (2048, 512, 1), (17, 128, 3), (300, 256, 8), (2048, 1024, 9), (129, 1152, 16), (515, 2048, 33),
             (64, 16384, 2), (1000, 640, 64), (40, 8320, 5), (2049, 384, 70), (10000, 256, 40), (700, 1024, 129), (130, 896, 300)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rotated", [True, False])
@pytest.mark.parametrize("N,K,T", Q4_SHAPES)
def test_q4_int4(N, K, T, rotated, dtype):
    x, codes, scales, ts = q4_case("int4", N, K, T, dtype, N + K + T, pad=8 if N % 2 else 0)
    y = ops.q4_linear(x, codes, scales, ts, fmt="int4", rotated=rotated)
    ref, slack = q4_reference(x, codes, scales, ts, "int4", rotated)
    close(y, ref, dtype, slack, 2.0 ** -11 if rotated else 0.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,K,T", [(1, 16, 1), (5, 32, 2), (300, 48, 7), (77, 4112, 3), (2048, 512, 8), (130, 2064, 17), (513, 1040, 37),
                                   (2049, 144, 65), (16, 16400, 1)])
def test_q4_nvfp4(N, K, T, dtype):
    x, codes, scales, ts = q4_case("nvfp4", N, K, T, dtype, N + K + T, pad=16 if T % 2 else 0)
    y = ops.q4_linear(x, codes, scales, ts, fmt="nvfp4")
    ref, slack = q4_reference(x, codes, scales, ts, "nvfp4", False)
    close(y, ref, dtype, slack)


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
def test_q4_every_code_and_scale_is_exact(fmt):
    # x = one-hot rows: y is the stored weight itself, rounded once
    K = 128
    codes = torch.arange(256, dtype=torch.uint8).repeat(K // 2, 1).t().contiguous().cuda()           # row b: byte b everywhere
    if fmt == "int4":
        vals = [2.0 ** -20, 2.0 ** -130, 1.0, 255.0, -3.0, 1.5 * 2.0 ** 100, 0.0, 0.0039]
        scales = torch.tensor(vals, dtype=torch.float32).to(torch.bfloat16).repeat(32)[:, None].contiguous().cuda()
        ts = None
    else:
        scales = torch.arange(256 * 8, dtype=torch.int64).remainder(256).to(torch.uint8)
        scales[(scales & 0x7F) == 0x7F] = 0x38                                                       # no NaN scale
        scales = scales.reshape(256, 8).view(torch.float8_e4m3fn).cuda()
        ts = torch.ones(1).cuda()
    x = torch.eye(K)[::9].contiguous().to(torch.bfloat16).cuda()
    y = ops.q4_linear(x, codes, scales, ts, fmt=fmt, rotated=False)
    ref, _ = q4_reference(x, codes, scales, ts, fmt, False)
    np.testing.assert_array_equal(f64(y), f64(torch.from_numpy(ref).to(torch.bfloat16)))


def test_q4_extreme_activations_stay_in_their_row():
    # bf16 values fp16 cannot hold, tiny ones, an all-zero row, an infinity and a NaN: each token on its own
    x, codes, scales, _ = q4_case("int4", 96, 256, 6, torch.bfloat16, 5, hot=False)
    x = x.clone()
    x[0] *= 1e30
    x[1] *= 1e-30
    x[2] = 0
    x[3, 7] = float("inf")
    x[4, 200] = float("nan")
    codes = codes.clone()
    codes[:, 3] = (codes[:, 3] & 0x0F) | 0x30                                                        # code 3 against the infinity
    for rotated in (False, True):
        y = ops.q4_linear(x, codes, scales, None, fmt="int4", rotated=rotated)
        keep = [0, 1, 2, 5]
        ref, slack = q4_reference(x[keep], codes, scales, None, "int4", rotated)
        close(y[keep], ref, torch.bfloat16, slack, 2.0 ** -11)
        assert not torch.isfinite(y[3]).any() and torch.isnan(y[4]).all()
        assert torch.all(y[2] == 0)
        if not rotated:
            assert torch.equal(torch.isinf(y[3]), torch.ones_like(y[3], dtype=torch.bool))
            assert torch.equal(y[3] > 0, (scales[:, 0] > 0))


@pytest.mark.parametrize("fmt,N,K,T", [("int4", 20001, 128, 3), ("int4", 20001, 256, 11), ("nvfp4", 40003, 32, 8), ("nvfp4", 19001, 64, 17),
                                       ("int4", 3, 65536, 1), ("int4", 24, 65536, 8), ("int4", 9, 65536, 12), ("nvfp4", 5, 65536, 70),
                                       ("nvfp4", 6, 65520, 5), ("nvfp4", 6, 65520, 9), ("int4", 7, 128, 700)])
def test_q4_at_the_ends_of_its_range(fmt, N, K, T):
    # more rows than one wave of full tiles, the longest K on few rows, many chunks of tokens
    x, codes, scales, ts = q4_case(fmt, N, K, T, torch.bfloat16, N + K + T)
    y = ops.q4_linear(x, codes, scales, ts, fmt=fmt, rotated=fmt == "int4")
    ref, slack = q4_reference(x, codes, scales, ts, fmt, fmt == "int4")
    close(y, ref, torch.bfloat16, slack, 2.0 ** -11 if fmt == "int4" else 0.0)


@pytest.mark.parametrize("T", [1, 5, 8, 20])
@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
def test_q4_scales_at_any_address(fmt, T):
    # scales that start inside a buffer, one element behind a 16-byte boundary: the same bits as aligned ones
    x, codes, scales, ts = q4_case(fmt, 130, 1024, T, torch.bfloat16, T)
    raw = torch.empty(scales.numel() + 1, dtype=scales.dtype, device="cuda")
    moved = raw[1:].view(scales.shape)
    moved.copy_(scales)
    assert moved.data_ptr() % 16 != 0
    want = ops.q4_linear(x, codes, scales, ts, fmt=fmt, rotated=False)
    assert torch.equal(ops.q4_linear(x, codes, moved, ts, fmt=fmt, rotated=False), want)


@pytest.mark.parametrize("T", [2, 8, 24])
def test_q4_reads_weights_written_just_before(T):
    # codes, scales and activations rewritten on the stream before every call, in a graph as well: each call sees its own
    N, K = 2048, 1024
    cases = [q4_case("int4", N, K, T, torch.bfloat16, s) for s in range(4)]
    want = [ops.q4_linear(x, c, s) for x, c, s, _ in cases]
    torch.cuda.synchronize()
    x, c, s = (torch.empty_like(t) for t in cases[0][:3])

    def steps():
        out = []
        for a, b, d, _ in cases:
            s.copy_(d), c.copy_(b), x.copy_(a)
            out.append(ops.q4_linear(x, c, s))
        return out
    for got in (steps(), steps()):
        for u, v in zip(got, want):
            assert torch.equal(u, v)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = steps()
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for u, v in zip(out, want):
            assert torch.equal(u, v)


def test_q4_writes_only_its_columns_and_repeats_bit_for_bit():
    x, codes, scales, _ = q4_case("int4", 77, 384, 11, torch.float16, 6)
    buf = torch.full((11, 100), 7.0, dtype=torch.float16, device="cuda")
    ops.q4_linear(x, codes, scales, fmt="int4", y=buf[:, 3:80])
    assert torch.all(buf[:, :3] == 7) and torch.all(buf[:, 80:] == 7)
    assert torch.equal(buf[:, 3:80], ops.q4_linear(x, codes, scales, fmt="int4"))
    # up to 8 tokens, a token's result does not depend on its batch
    one = torch.cat([ops.q4_linear(x[t:t + 1].contiguous(), codes, scales, fmt="int4") for t in range(8)])
    assert torch.equal(one, ops.q4_linear(x[:8], codes, scales, fmt="int4"))


def test_q4_takes_the_quantisers_output():
    g = torch.Generator().manual_seed(3)
    w = (torch.randn((192, 512), generator=g) * 0.05).to(torch.bfloat16).cuda()
    x = (torch.randn((5, 512), generator=g)).to(torch.bfloat16).cuda()
    want = f64(x) @ f64(w).T
    for fmt, rotate in (("int4", True), ("int4", False), ("nvfp4", False)):
        codes, scales, ts = ops.quantize_linear(w, fmt=fmt, rotate=rotate)
        y = f64(ops.q4_linear(x, codes, scales, ts, fmt=fmt, rotated=rotate))
        # 4-bit rounding of normal weights: ~11% of each weight's rms at most, independent over K
        assert np.linalg.norm(y - want) <= 0.15 * np.linalg.norm(want)


@pytest.mark.parametrize("T", [1, 3, 8, 12, 33])
def test_q4_rotation_near_the_top_of_bf16(T):
    # x' = Hn x is a sum of 128 activations over sqrt(128): the sum passes fp32's range before x' does, and x' (of a segment
    # of one sign) before the product with small scales does. Ordinary tokens and infinities stand beside such ones.
    x, codes, scales, _ = q4_case("int4", 200, 384, T, torch.bfloat16, 40 + T, hot=False)
    big = [0.0, 1e37, 3.3e38, 3.2e36][:T]
    x = x.clone()
    for t, v in enumerate(big):
        if v:
            x[t] = x[t].sign() * v
            x[t, 128:256] = v if t % 2 else -v
            x[t, 300] = 1e-30
    if T > 5:
        x[5, 7] = float("inf")
        x[6] = -3.3e38
    scales = (scales.float() * 2.0 ** -12).to(torch.bfloat16)
    y = ops.q4_linear(x, codes, scales, None, fmt="int4", rotated=True)
    keep = [t for t in range(T) if t != 5]
    ref, slack = q4_reference(x[keep], codes, scales, None, "int4", True)
    close(y[keep], ref, torch.bfloat16, slack, 2.0 ** -11)
    if T > 5:
        assert not torch.isfinite(y[5]).any()
    # a power of two taken out of the whole input comes out of the whole output, bit for bit
    small = ops.q4_linear((x.float() * 2.0 ** -40).to(torch.bfloat16), codes, (scales.float() * 2.0 ** 40).to(torch.bfloat16), None,
                          fmt="int4", rotated=True)
    assert torch.equal(small[keep], y[keep])


@pytest.mark.parametrize("N,K,T", [(515, 2048, 9), (515, 2048, 24), (1000, 1152, 37), (300, 4096, 64), (260, 640, 129), (4096, 128, 70)])
def test_q4_rotated_fp16_keeps_the_outputs_rounding(N, K, T):
    # y = round(v), v off the exact value by e: the rounding and e are independent, so |y - ref|^2 is |round(ref) - ref|^2 +
    # |e|^2 up to its scatter. x' = hi + lo, two fp16 numbers, leaves |e| below 2^-20 of the norm; x' as one fp16 number is
    # 2^-12.3 off and breaks the bound of 2^-13. The scatter: squares of n roundings, each in [0, (1/2 step)^2], add up to
    # their mean within 4 / sqrt(n) of it.
    x, codes, scales, _ = q4_case("int4", N, K, T, torch.float16, N + K + T, hot=False)
    scales = (scales.float() * 64).to(torch.bfloat16)            # outputs far above fp16's smallest normal
    y = f64(ops.q4_linear(x, codes, scales, None, fmt="int4", rotated=True))
    ref, _ = q4_reference(x, codes, scales, None, "int4", True)
    r = ref.astype(np.float16).astype(np.float64)
    assert np.isfinite(r).all()
    got, least = np.sum((y - ref) ** 2), np.sum((r - ref) ** 2)
    assert got <= (1 + 4 / np.sqrt(ref.size)) * least + (2.0 ** -13 * np.linalg.norm(ref)) ** 2, (got, least)


def ring_form(fmt, N, K, T, sms):
    """(blocks a team takes at a time, rounds, whether x comes through the ring, whether the scales stay in shared memory) of
    the product for up to 8 tokens (csrc/q4_linear.cu)."""
    segs, per = -(-K // 128), -(-N // sms)
    b16 = -(-per // 16)
    kw = 1
    while kw < segs and kw < (16 if b16 == 1 else 8):
        kw *= 2
    teams = 16 // kw
    rb = 1 if b16 <= teams else 2
    blocks = -(-b16 // (teams * rb)) * teams * rb
    scale_row = K // 64 if fmt == "int4" else K // 16
    rows = -(-per // blocks) * blocks
    tma = K % 32 == 0
    return rb, blocks // (teams * rb), tma and T * segs > 64, tma and scale_row % 16 == 0 and rows * scale_row <= 72 * 1024


LARGE = [("int4", True, 5001, 1024, 8, (2, 1, False, True)), ("int4", True, 5001, 4096, 8, (2, 1, True, True)),
         ("int4", False, 8192, 1152, 8, (2, 1, True, False)), ("int4", True, 20001, 1024, 3, (2, 3, False, True)),
         ("int4", True, 20001, 1152, 8, (2, 3, True, False)), ("int4", False, 20001, 2048, 5, (2, 3, True, True)),
         ("nvfp4", False, 5001, 1152, 8, (2, 1, True, False)), ("nvfp4", False, 9600, 4112, 2, (2, 2, False, False)),
         ("nvfp4", False, 8192, 4112, 8, (2, 1, False, False)), ("nvfp4", False, 20001, 1280, 8, (2, 3, True, True)),
         ("nvfp4", False, 10001, 1040, 7, (2, 2, False, False)), ("nvfp4", False, 12001, 2048, 8, (2, 2, True, True)),
         ("int4", True, 2368, 16384, 1, (1, 1, True, True)), ("int4", True, 9600, 8192, 8, (2, 2, True, True))]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("i", range(len(LARGE)))
def test_q4_few_tokens_many_rows(i, dtype):
    # two blocks of rows per team, one to three rounds that end inside the last, the operand built by every CTA or brought
    # through the ring, scales kept in shared memory or read when needed
    fmt, rotated, N, K, T, form = LARGE[i]
    if torch.cuda.get_device_properties(0).multi_processor_count == 148:
        assert ring_form(fmt, N, K, T, 148) == form
    x, codes, scales, ts = q4_case(fmt, N, K, T, dtype, N + K + T, pad=8 * (i % 2))
    y = ops.q4_linear(x, codes, scales, ts, fmt=fmt, rotated=rotated)
    ref, slack = q4_reference(x, codes, scales, ts, fmt, rotated)
    close(y, ref, dtype, slack, 2.0 ** -11 if rotated else 0.0)


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
@pytest.mark.parametrize("T,N,K", [(2, 96, 256), (8, 5001, 1024), (12, 96, 256), (40, 515, 1152)])
def test_q4_extreme_activations_at_any_token_count(fmt, T, N, K):
    # as above, for both formats and on both sides of eight tokens
    x, codes, scales, ts = q4_case(fmt, N, K, T, torch.bfloat16, T, hot=False)
    x = x.clone()
    x[0] *= 1e30
    x[1] *= 1e-30
    kinds = {"zero": 2, "inf": 3, "nan": 4} if T > 4 else {}
    if kinds:
        x[2] = 0
        x[3, K - 7] = float("-inf")
        x[4, 200] = float("nan")
        codes = codes.clone()
        at = (K - 7) // 2                                    # K - 7 is odd: the high nibble, code 3 against the infinity
        codes[:, at] = (codes[:, at] & 0x0F) | 0x30
        if fmt == "nvfp4":                                       # and no scale of zero against it
            b = scales.view(torch.uint8).clone()
            b[:, (K - 7) // 16] = b[:, (K - 7) // 16].clamp(min=0x20)
            scales = b.view(torch.float8_e4m3fn)
    keep = [t for t in range(T) if t not in (kinds.get("inf"), kinds.get("nan"))]
    for rotated in ((False, True) if fmt == "int4" else (False,)):
        y = ops.q4_linear(x, codes, scales, ts, fmt=fmt, rotated=rotated)
        ref, slack = q4_reference(x[keep], codes, scales, ts, fmt, rotated)
        got = y[keep]
        order = np.argsort([0 if t == 0 else 1 if t == 1 else 2 for t in keep], kind="stable")
        for part in (order[:1], order[1:2], order[2:]):          # a norm bound for each magnitude
            if len(part):
                close(got[part.tolist()], ref[part], torch.bfloat16, slack[part], 2.0 ** -11)
        if kinds:
            assert torch.all(y[2] == 0) and torch.isnan(y[4]).all() and not torch.isfinite(y[3]).any()
            if not rotated:
                sign = scales.float()[:, 0 if fmt != "int4" else (K - 7) // 128] if fmt == "int4" else torch.ones(N, device="cuda")
                assert torch.equal(y[3] < 0, sign > 0) and torch.isinf(y[3]).all()


@pytest.mark.parametrize("fmt", ["int4", "nvfp4"])
def test_q4_every_code_and_scale_is_exact_in_small_batches(fmt):
    # the test of 15 one-hot rows above, through the kernel for up to 8 tokens
    K = 128
    codes = torch.arange(256, dtype=torch.uint8).repeat(K // 2, 1).t().contiguous().cuda()
    if fmt == "int4":
        vals = [2.0 ** -20, 2.0 ** -130, 1.0, 255.0, -3.0, 1.5 * 2.0 ** 100, 0.0, 0.0039]
        scales = torch.tensor(vals, dtype=torch.float32).to(torch.bfloat16).repeat(32)[:, None].contiguous().cuda()
        ts = None
    else:
        scales = torch.arange(256 * 8, dtype=torch.int64).remainder(256).to(torch.uint8)
        scales[(scales & 0x7F) == 0x7F] = 0x38
        scales = scales.reshape(256, 8).view(torch.float8_e4m3fn).cuda()
        ts = torch.ones(1).cuda()
    for rows in (torch.arange(0, 8), torch.arange(60, 68), torch.arange(3, 128, 25)):
        x = torch.eye(K)[rows].contiguous().to(torch.bfloat16).cuda()
        y = ops.q4_linear(x, codes, scales, ts, fmt=fmt, rotated=False)
        ref, _ = q4_reference(x, codes, scales, ts, fmt, False)
        np.testing.assert_array_equal(f64(y), f64(torch.from_numpy(ref).to(torch.bfloat16)))


# ------------------------------------------------------------------------------------------ grouped linear

def counts_to_offsets(counts):
    return torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32).cuda()


def grouped_check(counts, N, K, dtype, act, seed, gather, pad=0, tail=0, row_div=1, x_rows=None):
    g = torch.Generator().manual_seed(seed)
    E, P = len(counts), int(sum(counts)) + tail
    w = (torch.randn((E, N, K), generator=g) * 0.05).to(dtype).cuda()
    P = max(P, 1)                                    # at least one row, of no group if need be
    n_x = x_rows or (P if not gather else max(1, P // 2))
    x = torch.randn((n_x, K + pad), generator=g).to(dtype).cuda()[:, :K]
    rows = torch.randint(0, n_x * row_div, (P,), generator=g).to(torch.int32).cuda() if gather else None
    off = counts_to_offsets(counts)
    nout = N // 2 if act == "swiglu" else N
    buf = torch.full((P, nout + 5), 9.0, dtype=dtype, device="cuda")
    y = ops.grouped_linear(x, w, off, rows=rows, row_div=row_div, act=act, y=buf[:, 2:2 + nout])
    ref, live = O.grouped_linear(f64(x), f64(w), off.cpu().numpy(), None if rows is None else rows.cpu().numpy(), row_div,
                                 act == "swiglu")
    wa, xa = np.abs(f64(w)), np.abs(f64(x))
    n = (K / 16 + 80) * 2.0 ** -23
    if act == "swiglu":
        # silu has slope below 1.1 and |silu(g)| <= |g|: the halves' errors da, db give 1.1 da |u| + |g| db, and silu
        # itself (exponential, division) a few 2^-22
        lin, _ = O.grouped_linear(f64(x), f64(w), off.cpu().numpy(), None if rows is None else rows.cpu().numpy(), row_div)
        mass, _ = O.grouped_linear(xa, wa, off.cpu().numpy(), None if rows is None else rows.cpu().numpy(), row_div)
        ga, u = np.abs(lin[:, :nout]), np.abs(lin[:, nout:])
        slack = 1.1 * n * mass[:, :nout] * u + ga * n * mass[:, nout:] + 2.0 ** -20 * ga * u
    else:
        mass, _ = O.grouped_linear(xa, wa, off.cpu().numpy(), None if rows is None else rows.cpu().numpy(), row_div)
        slack = mass * n
    if live.any():
        close(y, ref, dtype, slack, 2.0 ** -14, rows=live)
    assert torch.all(buf[:, :2] == 9) and torch.all(buf[:, 2 + nout:] == 9)
    assert torch.all(y[torch.from_numpy(~live).cuda()] == 9)
    return y


FEW = [[1], [0, 1, 0], [3, 0, 5, 0], [1] * 6, [0, 0, 0], [17, 1, 0, 2], [64], [0] * 200 + [2, 0, 1], [8, 9, 7, 16]]
MANY = [[65], [100, 0, 1, 27], [0, 300, 5], [128, 129, 127, 0, 1], [40] * 9, [0, 0, 513], [1, 2, 3, 4, 5] * 20, [256, 257]]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("i", range(len(FEW)))
def test_grouped_few_rows(i, act, dtype):
    N, K = [(64, 64), (128, 520), (30, 8), (256, 2048), (34, 72), (200, 136), (16, 1024), (70, 256), (130, 640)][i]
    grouped_check(FEW[i], N, K, dtype, act, i, gather=i % 2 == 1, pad=8 * (i % 3), tail=i % 2, row_div=1 + i % 3)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("i", range(len(MANY)))
def test_grouped_many_rows(i, act, dtype):
    N, K = [(64, 64), (128, 520), (30, 8), (256, 1024), (34, 72), (1000, 200), (16, 128), (390, 264)][i]
    grouped_check(MANY[i], N, K, dtype, act, 50 + i, gather=i % 2 == 0, pad=8 * (i % 3), tail=3 * (i % 2), row_div=1 + i % 4)


@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("gather", [True, False])
def test_grouped_large_groups(act, gather):
    # several hundred rows per group and enough weight tiles that two blocks of them share the rows
    grouped_check([700, 0, 300, 513, 40], 5000 if act else 4900, 136, torch.bfloat16, act, 11, gather=gather, tail=5, row_div=2)
    grouped_check([1030], 6000, 72, torch.float16, act, 12, gather=gather)


def two_blocks(counts, N, act, sms):
    """Whether gathered rows in these groups go to the kernel with two blocks of weights per tile (csrc/grouped.cu)."""
    P, E, nout = sum(counts), len(counts), N // 2 if act else N
    wide = -(-nout // (128 if act else 256))
    return P // E > 128 and 2 * wide * max(P // 256, E) >= 3 * sms


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("act", [None, "swiglu"])
@pytest.mark.parametrize("over", [1, 100, 127, 128, 129, 200, 256])
def test_grouped_two_blocks_of_weights(over, act, dtype):
    # uneven groups (an empty one, one that ends inside a tile) and outputs that end `over` behind a tile's start: inside its
    # first block, on the blocks' border, inside the second one
    counts = [300, 0, 257, 513, 40, 129]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    step = 128 if act else 256                       # outputs of a tile
    tiles = -(-3 * sms // (2 * len(counts)))
    nout = (tiles - 1) * step + (over + 1) // (2 if act else 1)
    N = 2 * nout if act else nout
    assert two_blocks(counts, N, act, sms)
    grouped_check(counts, N, 72 if over % 2 else 136, dtype, act, over, gather=True, pad=8, row_div=1 + over % 3)


def test_grouped_many_experts_and_odd_widths():
    rng = np.random.default_rng(0)
    counts = rng.integers(0, 4, 1024)
    grouped_check(list(counts), 19, 40, torch.bfloat16, None, 7, gather=True, row_div=6)
    grouped_check([70, 0, 3], 1, 64, torch.float16, None, 8, gather=False)
    grouped_check([70, 0, 3], 2, 64, torch.float16, "swiglu", 9, gather=False)


def test_grouped_offsets_and_rows_outside_are_clamped():
    for P in (10, 200):
        g = torch.Generator().manual_seed(P)
        x = torch.randn((P, 64), generator=g).to(torch.bfloat16).cuda()
        w = (torch.randn((4, 32, 64), generator=g) * 0.1).to(torch.bfloat16).cuda()
        off = torch.tensor([-7, 4, 4, 2, P + 1000], dtype=torch.int32).cuda()       # group 2 ends before it begins
        rows = torch.arange(P, dtype=torch.int32).cuda()
        rows[0], rows[P - 1] = -5, 1 << 30
        y = torch.full((P, 32), 9.0, dtype=torch.bfloat16, device="cuda")
        off_ok = torch.tensor([0, 4, 4, 4, P], dtype=torch.int32).cuda()
        off_ok[3] = 4
        ops.grouped_linear(x, w, torch.tensor([-7, 4, 4, 4, P + 1000], dtype=torch.int32).cuda(), rows=rows, y=y)
        ref, live = O.grouped_linear(f64(x), f64(w), off_ok.cpu().numpy(), rows.cpu().numpy())
        assert live.all()
        close(y, ref, torch.bfloat16, 1e-4)
        ops.grouped_linear(x, w, off, rows=rows, y=y)                               # overlapping groups: no fault
        torch.cuda.synchronize()


def test_grouped_nan_rows_stay_in_their_row():
    for counts in ([5, 3], [70, 130]):
        P = sum(counts)
        g = torch.Generator().manual_seed(P)
        x = torch.randn((P, 136), generator=g).to(torch.bfloat16).cuda()
        w = (torch.randn((2, 48, 136), generator=g) * 0.1).to(torch.bfloat16).cuda()
        off = counts_to_offsets(counts)
        want = ops.grouped_linear(x, w, off)
        x2 = x.clone()
        x2[counts[0] - 1, 5] = float("nan")
        x2[counts[0], 100] = float("inf")
        got = ops.grouped_linear(x2, w, off)
        keep = torch.ones(P, dtype=torch.bool, device="cuda")
        keep[counts[0] - 1:counts[0] + 1] = False
        assert torch.equal(got[keep], want[keep])
        assert torch.isnan(got[counts[0] - 1]).all() and not torch.isfinite(got[counts[0]]).any()


def test_grouped_is_deterministic():
    g = torch.Generator().manual_seed(1)
    x = torch.randn((700, 512), generator=g).to(torch.bfloat16).cuda()
    w = (torch.randn((8, 256, 512), generator=g) * 0.1).to(torch.bfloat16).cuda()
    for counts in ([100, 0, 200, 1, 99, 50, 50, 200], [3, 0, 1, 1, 0, 7, 2, 0]):
        P = sum(counts)
        off = counts_to_offsets(counts)
        first = ops.grouped_linear(x[:P], w, off, act="swiglu")
        for _ in range(5):
            assert torch.equal(ops.grouped_linear(x[:P], w, off, act="swiglu"), first)


# ------------------------------------------------------------------------------------- permute and combine

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 6, 256), (5, 6, 256), (33, 2, 7), (64, 64, 64), (700, 6, 256), (2048, 6, 256), (4099, 1, 3),
                                   (1500, 8, 1024), (20001, 3, 129), (1, 8, 1000)])
@pytest.mark.parametrize("kind", ["all", "dropped", "one", "none"])
def test_permute(T, k, E, kind):
    g = torch.Generator().manual_seed(T + k + E)
    ids = torch.randint(0, E, (T, k), generator=g)
    if kind == "dropped":
        ids = torch.randint(-3, E + 3, (T, k), generator=g)
    elif kind == "one":
        ids[:] = E - 1
    elif kind == "none":
        ids[:] = -1
    ids = ids.to(torch.int32)
    off, perm, inv = ops.expert_permute(ids.cuda(), E)
    flat = ids.reshape(-1).long().numpy()
    key = np.where((flat < 0) | (flat >= E), E, flat)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=E + 1)[:E]
    kept = int(counts.sum())
    np.testing.assert_array_equal(off.cpu().numpy(), np.concatenate([[0], np.cumsum(counts)]))
    want = np.where(np.arange(T * k) < kept, order, -1)
    np.testing.assert_array_equal(perm.cpu().numpy(), want)
    pos = np.empty(T * k, dtype=np.int64)
    pos[order] = np.arange(T * k)
    np.testing.assert_array_equal(inv.cpu().numpy().reshape(-1), np.where(key < E, pos, -1))


def test_permute_of_no_tokens():
    off, perm, inv = ops.expert_permute(torch.empty((0, 6), dtype=torch.int32, device="cuda"), 9)
    assert torch.all(off == 0) and off.numel() == 10 and perm.numel() == 0 and inv.shape == (0, 6)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (3, 6, 2048), (7, 2, 513), (50, 9, 64), (129, 64, 40), (300, 8, 4096), (2, 3, 8200)])
def test_combine(T, k, H, dtype):
    g = torch.Generator().manual_seed(T + k + H)
    P = T * k
    o = torch.randn((P, H + 8), generator=g).to(dtype).cuda()[:, :H]
    inv = torch.randperm(P, generator=g).to(torch.int32).reshape(T, k)
    inv[torch.rand((T, k), generator=g) < 0.2] = -1
    if T > 2:
        inv[1] = -1                                  # a token with no expert left
        inv[2, 0] = P + 3                            # outside: skipped
    w = torch.rand((T, k), generator=g)
    add = torch.randn((T, H), generator=g).to(dtype).cuda()
    o = o.clone() if H % 8 else o
    for addend in (None, add):
        y = ops.expert_combine(o, inv.cuda(), w.cuda(), addend=addend, scale=0.75)
        ref = O.expert_combine(f64(o), inv.numpy(), w.double().numpy(), None if addend is None else f64(addend), 0.75)
        mass = O.expert_combine(np.abs(f64(o)), inv.numpy(), w.double().numpy(), None if addend is None else np.abs(f64(addend)), 0.75)
        close(y, ref, dtype, mass * (k + 4) * 2.0 ** -24)
    inplace = add.clone()
    assert ops.expert_combine(o, inv.cuda(), w.cuda(), addend=inplace, scale=0.75, y=inplace) is inplace
    assert torch.equal(inplace, ops.expert_combine(o, inv.cuda(), w.cuda(), addend=add, scale=0.75))


def test_combine_skips_dropped_rows_whatever_they_hold():
    o = torch.ones((4, 64), dtype=torch.bfloat16, device="cuda")
    o[1] = float("nan")
    inv = torch.tensor([[0, -1], [2, 3]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[2.0, float("inf")], [1.0, 0.5]], device="cuda")
    y = ops.expert_combine(o, inv, w)
    assert torch.all(y[0] == 2) and torch.all(y[1] == 1.5)


# -------------------------------------------------------------------------------------------- block norm

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("res32", [True, False])
@pytest.mark.parametrize("T,H", [(1, 1), (4, 2048), (3, 65), (17, 512), (2, 8192), (5, 8200), (2, 20000), (9, 4095), (1, 32768), (1030, 2056), (1025, 4095)])
@pytest.mark.parametrize("mode", ["plain", "branch", "post", "gate_row", "gate_token"])
def test_block_norm(T, H, mode, res32, dtype):
    g = torch.Generator().manual_seed(T + H)
    rt = torch.float32 if res32 else dtype
    x = (torch.randn((T, H + 8), generator=g) * torch.exp2(torch.randint(-6, 6, (T, 1), generator=g).float())).to(rt).cuda()[:, :H]
    y = torch.randn((T, H), generator=g).to(dtype).cuda() if mode != "plain" else None
    gate = None
    if mode.startswith("gate"):
        gate = (2 * torch.randn((1 if mode == "gate_row" else T, H), generator=g)).to(dtype).cuda()
    post = mode in ("post", "gate_token")
    wt = torch.float32 if T % 2 else dtype
    pw = (1 + 0.1 * torch.randn(H, generator=g)).to(wt).cuda() if post else None
    qw = (1 + 0.1 * torch.randn(H, generator=g)).to(wt).cuda() if mode != "branch" else None
    kw = dict(res_scale=0.875, branch_scale=1.5, eps=1e-5)
    xo, z = ops.block_norm(x, y, post_norm=post, post_weight=pw, gate=gate, gate_act="sigmoid", pre_weight=qw, z_dtype=dtype, **kw)
    rx, rz = O.block_norm(f64(x), None if y is None else f64(y), post_norm=post, post_weight=None if pw is None else f64(pw),
                          gate=None if gate is None else f64(gate), sigmoid=True, pre_weight=None if qw is None else f64(qw), **kw)
    # fp32 arithmetic: a dozen roundings per element on |res x| + |branch b|; a norm adds its sum's error, at most
    # (32 + log2 terms per thread...) 64 roundings of positive terms, halved by the square root
    parts = 0.875 * np.abs(f64(x)) + (0 if y is None else np.abs(rx - 0.875 * f64(x)))
    sx = parts * 64 * 2.0 ** -24
    rms = np.sqrt((rx * rx).mean(1, keepdims=True) + 1e-5)
    qa = 1.0 if qw is None else np.abs(f64(qw))
    sz = (sx + np.abs(rx) * 64 * 2.0 ** -24) / rms * qa + np.abs(rz) * (np.linalg.norm(sx, axis=1, keepdims=True) / np.maximum(np.linalg.norm(rx, axis=1, keepdims=True), 1e-30))
    if rt == torch.float32:
        assert np.all(np.abs(f64(xo) - rx) <= sx + 2.0 ** -149)
    else:
        close(xo, rx, rt, sx, 2.0 ** -14)
    close(z, rz, dtype, sz, 2.0 ** -14)
    # in place, and without one of the outputs' buffers shared
    x2 = x.clone()
    xo2, z2 = ops.block_norm(x2, y, post_norm=post, post_weight=pw, gate=gate, gate_act="sigmoid", pre_weight=qw, z_dtype=dtype,
                             x_out=x2, **kw)
    assert xo2 is x2 and torch.equal(x2, xo) and torch.equal(z2, z)


def test_block_norm_agrees_with_the_stack_glue():
    g = torch.Generator().manual_seed(0)
    x = torch.randn((37, 2048), generator=g).cuda()
    y = torch.randn((37, 2048), generator=g).to(torch.bfloat16).cuda()
    xs, zs = x.clone(), torch.empty((37, 2048), dtype=torch.bfloat16, device="cuda")
    B.flint_residual_rmsnorm(xs.data_ptr(), y.data_ptr(), 37, 1e-6, zs.data_ptr(), torch.cuda.current_stream().cuda_stream)
    xo, z = ops.block_norm(x, y, eps=1e-6)
    assert torch.equal(xo, xs) and torch.equal(z, zs)


def test_block_norm_rows_are_independent_and_padding_is_kept():
    x = torch.ones((4, 100), dtype=torch.bfloat16, device="cuda")
    x[1] = float("nan")
    x[2] = 0
    z = torch.full((4, 112), 5.0, dtype=torch.bfloat16, device="cuda")
    ops.block_norm(x, z=z[:, :100])
    assert torch.all(z[0, :100] == 1) and torch.isnan(z[1, :100]).all() and torch.all(z[2, :100] == 0) and torch.all(z[:, 100:] == 5)


@pytest.mark.parametrize("H", [40, 2048, 4100, 8200, 32768])
@pytest.mark.parametrize("T", [3, 1030])
def test_block_norm_of_values_whose_squares_pass_fp32(T, H):
    # rows of ordinary size, of 1e25 and of nearly the largest bf16 value: the mean square does not fit fp32, the norm does
    g = torch.Generator().manual_seed(H + T)
    if T * H > 1 << 23:
        T = 7
    mag = torch.tensor([1.0, 1e25, 1e38])[torch.arange(T) % 3][:, None]
    y = ((0.5 + torch.rand((T, H), generator=g)) * mag).to(torch.bfloat16).cuda()
    x = (torch.randn((T, H), generator=g) * mag * 0.5).cuda()
    pw = (1 + 0.1 * torch.randn(H, generator=g)).cuda()
    fits = x.clamp(-1.5e38, 1.5e38)                  # some of x's largest values are infinite: those rows are looked at by themselves
    for res in (x, x.to(torch.bfloat16), fits, fits.to(torch.bfloat16)):
        rows = torch.isfinite(res).all(1).cpu().numpy()
        assert rows[1] and (res is x or res.dtype != torch.float32 or rows.all())
        for kw in (dict(post_norm=True, post_weight=pw), dict(branch_scale=0.5)):
            xo, z = ops.block_norm(res, y, pre_weight=pw, **kw)
            assert torch.all((z == 0) | torch.isnan(z) | torch.from_numpy(rows).cuda()[:, None])
            xo, z, rs = xo[rows], z[rows], f64(res)[rows]
            rx, rz = O.block_norm(rs, f64(y)[rows], pre_weight=f64(pw), **{k: f64(v) if k == "post_weight" else v for k, v in kw.items()})
            sx = (np.abs(rs) + np.abs(rx - rs)) * 64 * 2.0 ** -24
            if res.dtype == torch.float32:
                assert np.all(np.abs(f64(xo) - rx) <= sx)
            else:
                close(xo, rx, torch.bfloat16, sx, 2.0 ** -14)
            rms = np.sqrt((rx * rx).mean(1, keepdims=True) + 1e-6)
            sz = (sx + np.abs(rx) * 64 * 2.0 ** -24) / rms * np.abs(f64(pw)) + np.abs(rz) * (
                np.linalg.norm(sx, axis=1, keepdims=True) / np.linalg.norm(rx, axis=1, keepdims=True))
            close(z, rz, torch.bfloat16, sz, 2.0 ** -14)
    # infinities and NaN are no such rows: they go through as before
    y[0, 0], y[1, 1] = float("inf"), float("nan")
    _, z = ops.block_norm(torch.zeros_like(x), y)
    assert torch.isnan(z[0, 0]) and torch.all(z[0, 1:] == 0) and torch.isnan(z[1]).all() and torch.isfinite(z[2]).all()


def test_block_norm_gate_at_any_size():
    # sigmoid of every bf16 gate value, seen through an fp32 residual: x' = sigmoid(g) b with b = 1. The bound is the one
    # stated at the kernel's sigmoid, (1.3 |g| + 7) 2^-24 of the value, plus half a step of the fp32 product; values below
    # fp32's normal range may be flushed to zero.
    bits = torch.arange(65536, dtype=torch.int32).to(torch.uint16).view(torch.bfloat16)
    g = bits[torch.isfinite(bits.float())]
    g = torch.cat((g, g[:(-g.numel()) % 8])).reshape(1, -1)[:, :32768]
    rest = bits[torch.isfinite(bits.float())][32768:].reshape(1, -1)
    for gate in (g, rest):
        H = gate.shape[1]
        xo, _ = ops.block_norm(torch.zeros((1, H), device="cuda"), torch.ones((1, H), dtype=torch.bfloat16, device="cuda"),
                               gate=gate.cuda(), gate_act="sigmoid")
        gd = f64(gate)
        with np.errstate(over="ignore"):
            ref = 1 / (1 + np.exp(-gd))
        tol = ref * ((1.3 * np.abs(gd) + 7) * 2.0 ** -24 + 2.0 ** -24) + 2.0 ** -126
        err = np.abs(f64(xo) - ref)
        assert np.all(err <= np.where(np.isfinite(tol), tol, 2.0 ** -126)), float((err / tol).max())


# ---------------------------------------------------------------------------------- the ends of the ranges

def test_q4_of_the_largest_token_count_and_of_many_rows():
    for fmt, N, K, T in (("int4", 5, 128, 65536), ("nvfp4", 3, 48, 65536), ("int4", 400003, 128, 2), ("int4", 400003, 128, 9),
                         ("nvfp4", 400003, 32, 8)):
        x, codes, scales, ts = q4_case(fmt, N, K, T, torch.bfloat16, N + T)
        y = ops.q4_linear(x, codes, scales, ts, fmt=fmt, rotated=fmt == "int4")
        ref, slack = q4_reference(x, codes, scales, ts, fmt, fmt == "int4")
        close(y, ref, torch.bfloat16, slack, 2.0 ** -11 if fmt == "int4" else 0.0)


@pytest.mark.parametrize("T", [3, 20])
@pytest.mark.parametrize("dtype", TYPES)
def test_q4_int4_with_a_tensor_scale(dtype, T):
    x, codes, scales, _ = q4_case("int4", 130, 512, T, dtype, T, hot=False)
    ts = torch.tensor([-0.37]).cuda()
    for rotated in (True, False):
        y = ops.q4_linear(x, codes, scales, ts, fmt="int4", rotated=rotated)
        ref, slack = q4_reference(x, codes, scales, ts, "int4", rotated)
        close(y, ref, dtype, np.abs(slack), 2.0 ** -11 if rotated else 0.0)


@pytest.mark.parametrize("gather", [True, False])
def test_grouped_of_several_hundred_thousand_rows(gather):
    grouped_check([100001, 0, 200003, 7], 24, 16, torch.bfloat16, "swiglu", 3, gather=gather, tail=9, row_div=3)


def test_permute_of_the_largest_batch():
    T, k, E = 1 << 21, 2, 1024
    g = torch.Generator().manual_seed(0)
    ids = torch.randint(-20, E + 20, (T, k), generator=g, dtype=torch.int32)
    off, perm, inv = ops.expert_permute(ids.cuda(), E)
    flat = ids.reshape(-1).long().numpy()
    key = np.where((flat < 0) | (flat >= E), E, flat)
    order = np.argsort(key, kind="stable")
    counts = np.bincount(key, minlength=E + 1)[:E]
    kept = int(counts.sum())
    np.testing.assert_array_equal(off.cpu().numpy(), np.concatenate([[0], np.cumsum(counts)]))
    np.testing.assert_array_equal(perm.cpu().numpy(), np.where(np.arange(T * k) < kept, order, -1))
    pos = np.empty(T * k, dtype=np.int64)
    pos[order] = np.arange(T * k)
    np.testing.assert_array_equal(inv.cpu().numpy().reshape(-1), np.where(key < E, pos, -1))


def test_rows_behind_2_to_the_31_elements():
    # offsets of rows that pass 32 bits: the last rows of large strided buffers, and the first ones beside them
    bf = torch.bfloat16
    wide = torch.empty((6, 1 << 29), dtype=bf, device="cuda")      # rows 2^29 elements apart, the last from 5 * 2^29 on
    g = torch.Generator().manual_seed(0)
    x = torch.randn((6, 512), generator=g).to(bf).cuda()
    far = wide[:, :512]
    far.copy_(x)
    w = (torch.randn((2, 64, 512), generator=g) * 0.05).to(bf).cuda()
    off = torch.tensor([0, 2, 6], dtype=torch.int32).cuda()
    assert torch.equal(ops.grouped_linear(far, w, off), ops.grouped_linear(x, w, off))
    rows = torch.tensor([5, 0, 4, 5, 3, 1] * 20, dtype=torch.int32).cuda()
    off2 = torch.tensor([0, 50, 120], dtype=torch.int32).cuda()
    assert torch.equal(ops.grouped_linear(far, w, off2, rows=rows), ops.grouped_linear(x, w, off2, rows=rows))
    codes, scales, _ = ops.quantize_linear(w[0].contiguous(), fmt="int4")
    assert torch.equal(ops.q4_linear(far, codes, scales), ops.q4_linear(x, codes, scales))
    inv = torch.tensor([[5, 0], [4, -1], [3, 5]], dtype=torch.int32).cuda()
    cw = torch.rand((3, 2), generator=g).cuda()
    assert torch.equal(ops.expert_combine(far, inv, cw), ops.expert_combine(x, inv, cw))
    want = ops.block_norm(x, x)
    out = wide[:, 1024:1536], wide[:, 2048:2560]
    got = ops.block_norm(far, far, x_out=out[0], z=out[1])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = wide[:, 4096:4160]
    ops.grouped_linear(x, w, off, y=y)
    assert torch.equal(y, ops.grouped_linear(x, w, off))
    del wide, far, out, got, y
    torch.cuda.empty_cache()


FIRST_CALLS = """
import sys
sys.path.insert(0, {root!r})
import torch
from bit_routed_expert_sigmoid_b200 import ops
bf = torch.bfloat16
e = lambda *s, dtype=bf: torch.ones(s, device="cuda").to(dtype)
T = {T}
x, y = e(T, 256, dtype=torch.float32), e(T, 256)
codes, scales = e(64, 128, dtype=torch.uint8), e(64, 2)
n_codes, n_scales, ts = e(64, 128, dtype=torch.uint8), e(64, 16, dtype=torch.uint8), e(1, dtype=torch.float32)
gu, dn, ids, w = e(4, 64, 256), e(4, 256, 32), e(T, 2, dtype=torch.int32), e(T, 2, dtype=torch.float32)
def step():
    x1, z = ops.block_norm(x, y)
    return (z, ops.q4_linear(z, codes, scales), ops.q4_linear(z, n_codes, n_scales, ts, fmt="nvfp4"),
            ops.FlintExperts16(gu, dn).forward(z, ids, w, addend=y))
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = step()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(out, step())) and ops.error_word() == 0
print("captured")
"""


@pytest.mark.parametrize("T", [3, 300])
def test_the_first_call_of_a_process_may_be_captured(T):
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=root, T=T)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


# ------------------------------------------------------------------------------------------- used together

def block_inputs(T, H=256, I=128, E=16, k=4, seed=0):
    g = torch.Generator().manual_seed(seed)
    bf = torch.bfloat16
    d = dict(x=torch.randn((T, H), generator=g).cuda(), y=torch.randn((T, H), generator=g).to(bf).cuda(),
             gu=(torch.randn((E, 2 * I, H), generator=g) / H ** 0.5).to(bf).cuda(),
             dn=(torch.randn((E, H, I), generator=g) / I ** 0.5).to(bf).cuda(),
             ws=(torch.randn((H, H), generator=g) / H ** 0.5).to(bf).cuda(),
             ids=torch.stack([torch.randperm(E, generator=g)[:k].sort().values for _ in range(T)]).to(torch.int32).cuda(),
             w=torch.softmax(torch.randn((T, k), generator=g), 1).cuda())
    if T > 3:
        d["ids"][3] = -1                             # a padded token: no expert
    d["q"] = ops.quantize_linear(d["ws"], fmt="int4")
    return d


def block_step(d, experts, stream=None):
    """One block: norm, 4-bit dense projection beside the routed 16-bit experts, norm after."""
    x1, z = ops.block_norm(d["x"], d["y"], stream=stream)
    shared = ops.q4_linear(z, *d["q"], fmt="int4", stream=stream)
    y = experts.forward(z, d["ids"], d["w"], addend=shared, stream=stream)
    x2, z2 = ops.block_norm(x1, y, post_norm=True, branch_scale=0.5, stream=stream)
    return x2, z2, z, y


@pytest.mark.parametrize("T", [1, 5, 40, 333])
def test_a_block_of_the_operators_against_the_oracle(T):
    d = block_inputs(T)
    ex = ops.FlintExperts16(d["gu"], d["dn"])
    x2, z2, z, y = block_step(d, ex)
    x1, rz = O.block_norm(f64(d["x"]), f64(d["y"]))
    close(z, rz, torch.bfloat16, 1e-5)
    # each later step against the oracle on the device's own z (its rounding is checked above)
    codes, scales, _ = d["q"]
    shared = O.q4_linear(f64(z), "int4", codes.cpu().numpy(), scales.cpu().view(torch.int16).numpy().view(np.uint16), None, True)
    off, perm, inv = O.expert_permute(d["ids"].cpu().numpy(), 16)
    h, live = O.grouped_linear(f64(z), f64(d["gu"]), off, perm, 4, True)
    o, _ = O.grouped_linear(h, f64(d["dn"]), off)
    ry = O.expert_combine(o, inv, f64(d["w"]), shared)
    # three bf16 roundings on the way (h, o, shared) and the output's: each at most 2^-8 of the norm it acts on
    assert np.linalg.norm(f64(y) - ry) <= 4 * 2.0 ** -8 * np.linalg.norm(ry)
    rx2, rz2 = O.block_norm(x1, f64(y), post_norm=True, branch_scale=0.5)
    assert np.abs(f64(x2) - rx2).max() <= 2.0 ** -18 * np.abs(rx2).max()
    close(z2, rz2, torch.bfloat16, 1e-5)


def test_operators_in_a_graph_and_on_another_stream():
    d = block_inputs(9, seed=4)
    ex = ops.FlintExperts16(d["gu"], d["dn"])
    want = [t.clone() for t in block_step(d, ex)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = block_step(d, ex, stream=s)
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block_step(d, ex)
    other = block_inputs(9, seed=5)
    fresh = [t.clone() for t in block_step({**other, "gu": d["gu"], "dn": d["dn"], "q": d["q"]}, ex)]
    for k in ("x", "y", "ids", "w"):
        d[k].copy_(other[k])
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, fresh):
            assert torch.equal(a, b)


def test_two_streams_at_once():
    ds = [block_inputs(70, seed=i) for i in (6, 7)]
    exs = [ops.FlintExperts16(d["gu"], d["dn"]) for d in ds]
    want = [[t.clone() for t in block_step(d, e)] for d, e in zip(ds, exs)]
    streams = [torch.cuda.Stream() for _ in ds]
    torch.cuda.synchronize()
    for _ in range(10):
        got = [block_step(d, e, stream=s) for d, e, s in zip(ds, exs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            for u, v in zip(a, b):
                assert torch.equal(u, v)


def test_inputs_may_be_dropped_while_another_stream_still_reads_them():
    # the stream is busy when each call returns; what the caller then drops, and writes to next, must not reach the call
    s = torch.cuda.Stream()

    def fresh(i):
        d = block_inputs(24, seed=30 + i)
        return d, ops.FlintExperts16(d["gu"], d["dn"])

    def steps(d, ex, stream):
        q = ops.q4_linear(d["y"], *d["q"], fmt="int4", stream=stream)
        off, perm, inv = ops.expert_permute(d["ids"], 16, stream=stream)
        h = ops.grouped_linear(d["y"], d["gu"], off, rows=perm, row_div=4, act="swiglu", stream=stream)
        y = ex.forward(d["y"], d["ids"], d["w"], addend=q, stream=stream)
        c = ops.expert_combine(h, inv, d["w"], stream=stream)
        return q, off, perm, inv, h, y, c, *ops.block_norm(d["x"], d["y"], stream=stream)

    for i in range(2):
        d, ex = fresh(i)
        live = int(steps(d, ex, None)[1][-1])
        want = [t.clone() for t in steps(d, ex, None)]
        s.wait_stream(torch.cuda.current_stream())
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            torch.cuda._sleep(1_000_000_000)         # about 0.5 s
        got = steps(d, ex, s)
        shapes = [(t.shape, t.dtype) for k, v in d.items() for t in (v if isinstance(v, tuple) else (v,)) if t is not None]
        del d, ex
        over = [torch.full(shape, 77, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(2)]
        assert not s.query()                         # the calls had not even begun
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(got, want)):
            if j == 4:                               # rows of no expert are not written
                a, b = a[:live], b[:live]
            assert torch.equal(a, b)
        del over


def test_allocated_outputs_may_be_dropped_while_the_caller_still_reads_them():
    # the output is the given stream's memory: dropped by the caller, it must outlive what the caller's stream still does
    d = block_inputs(24, seed=50)
    want = ops.q4_linear(d["y"], *d["q"], fmt="int4").clone()
    s = torch.cuda.Stream()
    for _ in range(2):
        s.wait_stream(torch.cuda.current_stream())
        y = ops.q4_linear(d["y"], *d["q"], fmt="int4", stream=s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(1_000_000_000)             # about 0.5 s
        got = y.clone()
        shape = y.shape
        del y
        with torch.cuda.stream(s):
            over = [torch.full(shape, 77, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        assert not torch.cuda.current_stream().query()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        del over


def test_a_stream_argument_inside_a_capture():
    d = block_inputs(9, seed=8)
    ex = ops.FlintExperts16(d["gu"], d["dn"])
    want = [t.clone() for t in block_step(d, ex)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        out = block_step(d, ex, stream=side)
        here.wait_stream(side)
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, want):
            assert torch.equal(a, b)


def test_no_rows_are_no_ops():
    e = torch.empty
    bf = torch.bfloat16
    assert ops.q4_linear(e((0, 128), dtype=bf, device="cuda"), e((4, 64), dtype=torch.uint8, device="cuda"),
                         e((4, 1), dtype=bf, device="cuda")).shape == (0, 4)
    assert ops.grouped_linear(e((0, 64), dtype=bf, device="cuda"), e((2, 8, 64), dtype=bf, device="cuda"),
                              torch.zeros(3, dtype=torch.int32, device="cuda")).shape == (0, 8)
    x, z = ops.block_norm(e((0, 64), device="cuda"))
    assert x.shape == z.shape == (0, 64)


def test_no_wait_has_given_up():
    assert B.flint_ops_error_word() == 0


def test_error_word_of_each_way_to_ask():
    d = block_inputs(12, seed=3)
    ex = ops.FlintExperts16(d["gu"], d["dn"])
    block_step(d, ex)
    assert ops.error_word() == ops.error_word("cuda:0") == ops.error_word(torch.device("cuda", 0)) == ex.error_word() == 0
