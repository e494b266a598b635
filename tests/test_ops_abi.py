"""Argument checks of the standalone operators on the host, before any launch. No GPU needed: the pointers
are never dereferenced."""

import contextlib
import ctypes
import types

import pytest
import torch

from bit_routed_expert_sigmoid_b200 import binding as B
from bit_routed_expert_sigmoid_b200 import ops

INVALID, UNSUPPORTED, OK = B.FLINT_ERR_INVALID_ARG, B.FLINT_ERR_UNSUPPORTED, B.FLINT_OK
A, C, D, E_, F = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000        # 16-byte aligned stand-ins


def _status(name, defaults, **kw):
    args = dict(defaults)
    assert set(kw) <= set(args)
    args.update(kw)
    return B.raw_status(name, *args.values())


Q4 = dict(fmt=0, N=64, K=256, rotated=1, codes=A, scales=C, tscale=0, x=D, ldx=256, T=4, type=0, y=E_, ldy=64,
          workspace=0, workspace_bytes=ctypes.c_size_t(0), stream=0)


@pytest.mark.parametrize("kw", [
    dict(fmt=2), dict(N=0), dict(K=0), dict(K=192), dict(K=-128), dict(rotated=2), dict(fmt=1, rotated=1, tscale=F),
    dict(fmt=1, rotated=0, tscale=0), dict(fmt=1, rotated=0, K=248, tscale=F), dict(T=-1), dict(type=2), dict(type=-1),
    dict(ldx=255), dict(ldx=260), dict(ldx=128), dict(ldy=63), dict(codes=0), dict(codes=A + 8), dict(scales=0), dict(scales=C + 1),
    dict(x=0), dict(x=D + 2), dict(y=0), dict(y=E_ + 1), dict(y=D), dict(tscale=F + 2)])
def test_q4_linear_refuses(kw):
    assert _status("flint_q4_linear", Q4, **kw) == INVALID


def test_q4_linear_limits_and_no_op():
    assert _status("flint_q4_linear", Q4, K=65536 + 128, ldx=65536 + 128) == UNSUPPORTED
    assert _status("flint_q4_linear", Q4, T=65537) == UNSUPPORTED
    assert _status("flint_q4_linear", Q4, N=(1 << 30) + 1, ldy=1 << 31, K=128, ldx=128) == UNSUPPORTED
    assert _status("flint_q4_linear", Q4, N=1 << 26, ldy=1 << 26, K=4096, ldx=4096) == UNSUPPORTED
    big = dict(T=64, K=4096, ldx=4096)                     # needs a workspace: missing, misaligned, too small
    need = B.flint_q4_linear_workspace_size(4096, 64)
    assert need > 0 and B.flint_q4_linear_workspace_size(256, 4) == B.flint_q4_linear_workspace_size(0, 64) == 0
    for ws, n in ((0, need), (F + 16, need), (F, need - 1)):
        assert _status("flint_q4_linear", Q4, **big, workspace=ws, workspace_bytes=ctypes.c_size_t(n)) == B.FLINT_ERR_WORKSPACE
    assert _status("flint_q4_linear", Q4, T=0, x=0, y=0, codes=0, scales=0) == OK


GR = dict(E=4, N=64, K=64, act=0, type=0, w=A, x=C, ldx=64, x_rows=10, row_of=0, row_div=1, offsets=D, P=10, y=E_, ldy=64,
          stream=0)


@pytest.mark.parametrize("kw", [
    dict(E=0), dict(N=0), dict(K=0), dict(K=60), dict(P=-1), dict(x_rows=-1), dict(row_div=0), dict(act=2), dict(type=2),
    dict(act=1, N=63), dict(ldx=60), dict(ldx=66), dict(ldy=63), dict(act=1, ldy=31), dict(x_rows=9), dict(row_of=F, x_rows=0),
    dict(w=0), dict(w=A + 8), dict(x=0), dict(x=C + 2), dict(y=0), dict(y=E_ + 1), dict(offsets=0), dict(offsets=D + 2),
    dict(row_of=F + 1), dict(y=C), dict(y=A)])
def test_grouped_linear_refuses(kw):
    assert _status("flint_grouped_linear", GR, **kw) == INVALID


def test_grouped_linear_limits_and_no_op():
    for kw in (dict(E=1025), dict(K=65544, ldx=65544), dict(E=1024, N=1 << 21, ldy=1 << 21),
               dict(E=1, N=1 << 20, ldy=1 << 20, P=1 << 30, x_rows=1 << 30),
               dict(E=1024, N=32768, ldy=32768, P=1 << 20, x_rows=1 << 20)):     # tiles of groups that all overlap
        assert _status("flint_grouped_linear", GR, **kw) == UNSUPPORTED
    assert _status("flint_grouped_linear", GR, P=0, x_rows=0, w=0, x=0, y=0, offsets=0) == OK


PE = dict(ids=A, T=4, top_k=2, E=8, offsets=C, perm=D, inv=E_, stream=0)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(top_k=0), dict(E=0), dict(ids=0), dict(ids=A + 2), dict(offsets=0),
                                dict(perm=0), dict(inv=0), dict(perm=E_), dict(perm=A), dict(inv=A + 1), dict(offsets=A)])
def test_permute_refuses(kw):
    assert _status("flint_expert_permute", PE, **kw) == INVALID


def test_permute_limits():
    for kw in (dict(top_k=65), dict(E=1025), dict(T=1 << 21, top_k=3), dict(T=2 ** 31 - 1, top_k=64)):
        assert _status("flint_expert_permute", PE, **kw) == UNSUPPORTED


CO = dict(o=A, ldo=64, P=8, inv=C, w=D, T=4, top_k=2, H=64, scale=ctypes.c_float(1.0), addend=E_, lda=64, type=0, y=F, ldy=64,
          stream=0)


@pytest.mark.parametrize("kw", [dict(T=-1), dict(P=-1), dict(top_k=0), dict(H=0), dict(type=2), dict(ldo=63), dict(ldy=63),
                                dict(lda=63), dict(o=0), dict(o=A + 1), dict(inv=0), dict(inv=C + 2), dict(w=0), dict(y=0),
                                dict(y=A), dict(y=F + 1), dict(addend=E_ + 1), dict(addend=F, lda=72)])
def test_combine_refuses(kw):
    assert _status("flint_expert_combine", CO, **kw) == INVALID


def test_combine_limits_and_no_op():
    assert _status("flint_expert_combine", CO, top_k=65) == UNSUPPORTED
    big = (1 << 23) + 8
    assert _status("flint_expert_combine", CO, H=big, ldo=big, lda=big, ldy=big) == UNSUPPORTED
    assert _status("flint_expert_combine", CO, T=0, o=0, inv=0, w=0, y=0, addend=0) == OK


def _norm(**kw):
    base = dict(x=A, x_out=A, y=C, gate=0, post_weight=0, pre_weight=0, z=D, ldx=64, ldxo=64, ldy=64, ldg=0, ldz=64, T=4, H=64,
                type=0, res_type=2, w_type=2, post_norm=0, gate_act=0, res_scale=1.0, branch_scale=1.0, eps=1e-6)
    assert set(kw) <= set(base)
    base.update(kw)
    return B.raw_status("flint_block_norm", ctypes.byref(B.flint_norm_args(*base.values())), None)


@pytest.mark.parametrize("kw", [
    dict(T=-1), dict(H=0), dict(eps=0.0), dict(eps=float("nan")), dict(type=2), dict(res_type=1), dict(w_type=1), dict(post_norm=2),
    dict(post_norm=1, y=0), dict(gate_act=2), dict(gate=E_, y=0), dict(post_weight=E_), dict(pre_weight=E_, z=0), dict(ldx=63, ldxo=63),
    dict(ldxo=72), dict(ldy=63), dict(ldz=63), dict(gate=E_, ldg=63), dict(x=0, x_out=0), dict(x=A + 2, x_out=A + 2), dict(y=C + 1),
    dict(z=D + 1), dict(gate=E_ + 1), dict(pre_weight=E_ + 2), dict(z=A), dict(z=C), dict(x_out=C), dict(x_out=D)])
def test_block_norm_refuses(kw):
    assert _norm(**kw) == INVALID


def test_block_norm_limits_and_no_op():
    assert B.raw_status("flint_block_norm", None, None) == INVALID
    assert _norm(H=32776, ldx=32776, ldxo=32776, ldy=32776, ldz=32776) == UNSUPPORTED
    assert _norm(T=0, x=0, x_out=0, y=0, z=0) == OK
    assert _norm(x_out=0, z=0) == OK


def test_packed_norm_arguments_are_the_structure():
    vals = list(range(1, 8)) + [64, 65, 66, 0, 68] + [4, 64, 0, 2, 2, 1, 1] + [0.5, 2.0, 1e-6]
    packed = B.pack_norm_args(*vals)
    assert packed == bytes(B.flint_norm_args(*vals)) and len(packed) == ctypes.sizeof(B.flint_norm_args)


def test_error_word_needs_a_place():
    assert B.raw_status("flint_ops_error_word", None) == INVALID


def test_wrappers_refuse_cpu_tensors_and_bad_shapes():
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    codes, scales = torch.zeros((4, 64), dtype=torch.uint8), torch.zeros((4, 1), dtype=torch.bfloat16)
    for call in (lambda: ops.q4_linear(x, codes, scales),
                 lambda: ops.grouped_linear(x, torch.zeros((1, 4, 128), dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)),
                 lambda: ops.expert_permute(torch.zeros((2, 1), dtype=torch.int32), 4),
                 lambda: ops.expert_combine(x, torch.zeros((2, 1), dtype=torch.int32), torch.zeros((2, 1))),
                 lambda: ops.block_norm(x)):
        with pytest.raises(ValueError):
            call()


def test_wrappers_refuse_other_scale_types(monkeypatch):
    # the checks run before anything touches a device: let CPU tensors through to them
    monkeypatch.setattr(ops, "_elsewhere", lambda device, stream: False)
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    codes = torch.zeros((4, 64), dtype=torch.uint8)
    for fmt, scales in (("int4", torch.zeros((4, 1), dtype=torch.float16)), ("int4", torch.zeros((4, 1), dtype=torch.int16)),
                        ("nvfp4", torch.zeros((4, 8), dtype=torch.float8_e5m2)), ("nvfp4", torch.zeros((4, 8), dtype=torch.int8)),
                        ("int4", torch.zeros((4, 2), dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="scales"):
            ops.q4_linear(x, codes, scales, torch.ones(1), fmt=fmt, rotated=False)


class _OnDevice(torch.Tensor):
    """A host tensor that passes for one of device 0 and notes the streams it is recorded on."""

    device = property(lambda self: torch.device("cuda", 0))

    def record_stream(self, stream):
        self.streams = getattr(self, "streams", []) + [stream]


def test_tensors_of_a_call_on_another_stream_are_recorded_there(monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", lambda stream: contextlib.nullcontext())
    caller = types.SimpleNamespace(device=torch.device("cuda", 0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: caller)
    monkeypatch.setattr(ops, "_current_device", lambda: 0)
    stream = types.SimpleNamespace(device=torch.device("cuda", 0))
    a, b, c, d = (torch.zeros(1).as_subclass(_OnDevice) for _ in range(4))
    out = torch.zeros(1).as_subclass(_OnDevice), torch.zeros(1).as_subclass(_OnDevice)
    assert ops._switched(lambda x, k, z=None, f=0: out, a.device, stream, a, 3, z=b, f=1.5) is out
    assert a.streams == b.streams == [stream]
    # what the call allocated is the stream's own, and the caller's to read
    assert out[0].streams == out[1].streams == [caller]
    assert ops._switched(lambda x: out[0], a.device, stream, a) is out[0] and out[0].streams == [caller, caller]

    def fails(x, y):
        raise ValueError("refused behind a launch")
    with pytest.raises(ValueError, match="refused"):
        ops._switched(fails, a.device, stream, c, torch.zeros(1))
    assert c.streams == [stream]
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext())
    ops._switched(lambda x: x, a.device, None, d)
    assert not hasattr(d, "streams")
    # the experts' weights as well, which are no arguments of the call
    ex = ops.FlintExperts16(torch.zeros((2, 4, 8)).as_subclass(_OnDevice), torch.zeros((2, 8, 2)).as_subclass(_OnDevice))
    with pytest.raises(ValueError):
        ex.forward(a, b, c, stream=stream)
    assert ex.gate_up.streams == ex.down.streams == [stream]


def test_wrappers_refuse_sizes_that_pass_32_bits(monkeypatch):
    # meta tensors stand for the large ones; nothing must reach the library, which would see the sizes modulo 2^32
    monkeypatch.setattr(ops, "_elsewhere", lambda device, stream: False)
    monkeypatch.setattr(ops, "_stream_of", lambda index: 0)
    for name in ("flint_q4_linear", "flint_grouped_linear", "flint_expert_permute", "flint_expert_combine", "flint_block_norm"):
        monkeypatch.setattr(ops.B, name, lambda *a, name=name: pytest.fail(f"{name} was called"))
    bf, i32, u8 = torch.bfloat16, torch.int32, torch.uint8

    def m(*shape, dtype=bf):
        return torch.empty(shape, dtype=dtype, device="meta")

    big = (1 << 32) + 5
    for call in (lambda: ops.q4_linear(m(big, 128), m(4, 64, dtype=u8), m(4, 1)),
                 lambda: ops.q4_linear(m(2, 128), m(big, 64, dtype=u8), m(big, 1)),
                 lambda: ops.grouped_linear(m(big, 8), m(2, 4, 8), m(3, dtype=i32)),
                 lambda: ops.grouped_linear(m(big, 8), m(2, 4, 8), m(3, dtype=i32), rows=m(9, dtype=i32)),
                 lambda: ops.grouped_linear(m(9, 8), m(2, 4, 8), m(3, dtype=i32), rows=m(9, dtype=i32), row_div=big),
                 lambda: ops.grouped_linear(m(9, 8), m(2, 4, 8), m(3, dtype=i32), rows=m(9, dtype=i32), row_div=5 - (1 << 32)),
                 lambda: ops.expert_permute(m(big, 1, dtype=i32), 4),
                 lambda: ops.expert_permute(m(3, 1, dtype=i32), big),
                 lambda: ops.expert_combine(m(4, 8), m(big, 1, dtype=i32), m(big, 1, dtype=torch.float32)),
                 lambda: ops.expert_combine(m(big, 8), m(4, 1, dtype=i32), m(4, 1, dtype=torch.float32)),
                 lambda: ops.block_norm(m(big, 1)), lambda: ops.block_norm(m(1, big))):
        with pytest.raises(ValueError, match="at most 2"):
            call()


def test_error_word_is_the_asked_devices(monkeypatch):
    asked = []
    monkeypatch.setattr(torch.cuda, "device", lambda device: contextlib.nullcontext(asked.append(device)))
    monkeypatch.setattr(ops.B, "flint_ops_error_word", lambda: 4)
    ex = ops.FlintExperts16(torch.zeros((2, 4, 8)).as_subclass(_OnDevice), torch.zeros((2, 8, 2)).as_subclass(_OnDevice))
    assert ops.error_word() == ops.error_word(1) == ex.error_word() == 4
    assert asked == [None, 1, torch.device("cuda", 0)]


@pytest.mark.parametrize("kw", [dict(perm=C), dict(inv=C)])
def test_permute_refuses_offsets_that_are_another_output(kw):
    assert _status("flint_expert_permute", PE, **kw) == INVALID


def test_block_norm_refuses_another_type_for_z_than_the_branchs(monkeypatch):
    monkeypatch.setattr(ops, "_elsewhere", lambda device, stream: False)
    monkeypatch.setattr(ops, "_stream_of", lambda index: 0)
    monkeypatch.setattr(ops.B, "flint_block_norm", lambda *a: None)
    x, b, h = torch.zeros((2, 8)), torch.zeros((2, 8), dtype=torch.bfloat16), torch.zeros((2, 8), dtype=torch.float16)
    with pytest.raises(ValueError, match="z_dtype"):
        ops.block_norm(x, b, z_dtype=torch.float16)
    with pytest.raises(ValueError, match="z_dtype"):
        ops.block_norm(x, z=h, z_dtype=torch.bfloat16)
    assert ops.block_norm(x, b, z_dtype=torch.bfloat16)[1].dtype == torch.bfloat16
    assert ops.block_norm(x, z_dtype=torch.float16)[1].dtype == ops.block_norm(x, z=h)[1].dtype == torch.float16
