"""FlintMoELayer and FlintMoEStack record the tensors of a call with `stream` on that stream. No GPU needed: the library's
calls are left out."""

import contextlib

import pytest
import torch

from bit_routed_expert_sigmoid_b200 import layer as LY


class _Noted(torch.Tensor):
    def record_stream(self, stream):
        self.streams = getattr(self, "streams", []) + [stream]


class _Stream:
    cuda_stream = 7


_CALLER = _Stream()


def _tensor(*shape):
    return torch.zeros(shape or (2, LY.H)).as_subclass(_Noted)


@pytest.fixture
def bare(monkeypatch):
    """A layer without a handle, whose forwards launch nothing."""
    made = []
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext(made.append(s)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: _CALLER)
    for name in ("flint_moe_forward", "flint_moe_forward_routed", "flint_moe_stack_forward"):
        monkeypatch.setattr(LY.B, name, lambda *a: None)
    one = object.__new__(LY.FlintMoELayer)
    one.device, one.top_k, one.cache, one.handle, one._recorded = torch.device("cpu"), 2, None, 0, set()
    one.workspace, one.tensors = _tensor(8), {"a": _tensor(4), "b": None}
    one.allocated_on = made
    yield one
    one.handle = None


def test_a_forward_on_a_stream_records_what_it_uses(bare):
    s = _Stream()
    x, y, ids, w = (_tensor() for _ in range(4))
    assert bare.forward(x, y, stream=s) is y
    bare.forward_routed(x, ids, w, y, stream=s)
    assert x.streams == y.streams == [s, s] and ids.streams == w.streams == [s]
    # the layer's own memory once per stream
    assert bare.workspace.streams == bare.tensors["a"].streams == [s]


def test_an_allocated_output_belongs_to_the_stream(bare, monkeypatch):
    # it is an ordinary host tensor here
    monkeypatch.setattr(torch.Tensor, "record_stream", _Noted.record_stream)
    s = _Stream()
    y = bare.forward(_tensor(), stream=s)
    assert y.shape == (2, LY.H) and bare.allocated_on == [s] and y.streams == [_CALLER, s]
    assert not hasattr(bare.forward(_tensor()), "streams") and bare.allocated_on == [s]


def test_a_stack_on_a_stream_records_all_its_memory(bare):
    s = _Stream()
    st = object.__new__(LY.FlintMoEStack)
    st.device, st.eps, st.layers, st.z, st.y = bare.device, 1e-6, [bare], _tensor(), _tensor()
    x = _tensor()
    st.forward(x, stream=s)
    for t in (x, st.z, st.y, bare.workspace, bare.tensors["a"]):
        assert t.streams == [s]
