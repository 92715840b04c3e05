"""training.py's bookkeeping: what a call keeps, and leaves behind when it
fails.  The library's entries are replaced by ones that record their calls; no
GPU."""
import contextlib

import pytest
import torch

from mixture_experts_layer_56_b200 import _lib as L
from mixture_experts_layer_56_b200 import training as TR

ENTRIES = ("moe_grouped_matmul", "moe_grouped_matmul_dx", "moe_grouped_matmul_dw", "moe_swiglu",
           "moe_swiglu_backward", "moe_layer_norm", "moe_layer_norm_backward", "moe_orthogonalize")
STREAM = 4321


class Calls(list):
    """(entry, arguments, stream) of each call; `fail` names the entry whose
    n-th call from now raises."""
    fail = None

    def entry(self, name):
        def call(*args, stream=None, **kw):
            if self.fail is not None and self.fail[0] == name:
                self.fail = (name, self.fail[1] - 1) if self.fail[1] > 1 else None
                if self.fail is None:
                    raise L.MoeError(name, L.MOE_ERR_CUDA)
            self.append((name, args, stream))
        return call

    def named(self, name):
        return [args for n, args, _ in self if n == name]


@pytest.fixture
def calls(monkeypatch):
    seen = Calls()
    for name in ENTRIES:
        monkeypatch.setattr(L, name, seen.entry(name))
    for name in ("moe_layer_norm_workspace_size", "moe_orthogonalize_workspace_size"):
        monkeypatch.setattr(L, name, lambda shape: 1 << 16)
    monkeypatch.setattr(L, "_stream", lambda stream: STREAM if stream is None else stream)
    monkeypatch.setattr(TR, "_on_current", lambda t, what: t)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: handle)
    monkeypatch.setattr(TR, "_on", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, stream: seen.recorded.setdefault(stream, []).append(t),
                        raising=False)
    seen.recorded = {}
    return seen


def experts():
    return TR.TrainableExperts(torch.ones(2, 128, 16), torch.ones(2, 16, 64))


def flags(calls):
    return [a[0].flags for a in calls.named("moe_grouped_matmul_dw")]


OFF = torch.tensor([0, 2, 4], dtype=torch.int32)
OVER, ADD = L.MOE_GROUPED_DW_F32, L.MOE_GROUPED_DW_F32 | L.MOE_GROUPED_DW_ACCUMULATE


def no_memory(*a, **kw):
    raise torch.OutOfMemoryError("planted")


def test_backward_without_memory_changes_nothing(calls, monkeypatch):
    ex, x = experts(), torch.ones(4, 16)
    ex.forward(x, OFF)
    with monkeypatch.context() as m:
        m.setattr(torch, "empty_like", no_memory)
        with pytest.raises(torch.OutOfMemoryError):
            ex.backward(x)
    assert not calls.named("moe_grouped_matmul_dw")
    ex.backward(x)              # the forward is still there
    assert flags(calls) == [OVER, OVER]
    ex.forward(x, OFF)
    ex.backward(x)
    assert flags(calls)[2:] == [ADD, ADD]


def test_backward_that_fails_before_a_gradient_keeps_the_gradients(calls):
    ex, x = experts(), torch.ones(4, 16)
    ex.forward(x, OFF)
    calls.fail = ("moe_grouped_matmul_dx", 1)
    with pytest.raises(L.MoeError):
        ex.backward(x)
    with pytest.raises(RuntimeError, match="forward"):
        ex.backward(x)
    ex.forward(x, OFF)
    ex.backward(x)
    assert flags(calls) == [OVER, OVER]  # nothing was there to add to


@pytest.mark.parametrize("entry,nth", [("moe_swiglu_backward", 1), ("moe_grouped_matmul_dx", 2),
                                       ("moe_grouped_matmul_dw", 2)])
def test_backward_that_fails_between_the_gradients_asks_for_zero_grad(calls, entry, nth):
    ex, x = experts(), torch.ones(4, 16)
    ex.forward(x, OFF)
    calls.fail = (entry, nth)
    with pytest.raises(L.MoeError):
        ex.backward(x)
    ex.forward(x, OFF)
    with pytest.raises(RuntimeError, match="zero_grad"):
        ex.backward(x)
    ex.zero_grad()
    ex.backward(x)
    assert flags(calls)[-2:] == [OVER, OVER]


def test_gradients_add_up_until_zero_grad(calls):
    ex, x = experts(), torch.ones(4, 16)
    for zero in (False, False, True, False):
        if zero:
            ex.zero_grad()
        ex.forward(x, OFF)
        ex.backward(x)
    assert flags(calls) == [OVER, OVER, ADD, ADD, OVER, OVER, ADD, ADD]


def test_norm_backward_without_memory_changes_nothing(calls, monkeypatch):
    nm, x = TR.LayerNorm(torch.ones(16)), torch.ones(4, 16)
    nm.forward(x)
    with monkeypatch.context() as m:
        m.setattr(torch, "empty_like", no_memory)
        with pytest.raises(torch.OutOfMemoryError):
            nm.backward(x)
    nm.backward(x)
    assert len(calls.named("moe_layer_norm_backward")) == 1
    with pytest.raises(RuntimeError, match="forward"):
        nm.backward(x)


@pytest.mark.parametrize("stream", [None, STREAM, 77])
def test_what_a_call_uses_is_recorded_on_a_stream_of_its_own(calls, stream):
    """Everything passed to the library that was there before the call: the
    caller's inputs and the module's own tensors."""
    ex, nm = experts(), TR.LayerNorm(torch.ones(16), torch.ones(16))
    u, dy, m, ws = torch.ones(4, 16), torch.ones(4, 16), torch.ones(2, 8, 16), torch.zeros(256)
    x = nm.forward(u, stream=stream)
    y = ex.forward(x, OFF, stream=stream)
    dx = ex.backward(dy, stream=stream)
    nm.backward(dx, stream=stream)
    TR.orthogonalize(m, ws=ws, stream=stream)
    assert y.shape == u.shape and all(s == stream for _, _, s in calls)
    there = [u, dy, m, ws, OFF, x, dx, ex.W13, ex.W2, ex.ws, ex.dW13, ex.dW2, nm.gamma, nm.beta,
             nm.dgamma, nm.dbeta]
    used = {id(a) for _, args, _ in calls for a in args if isinstance(a, torch.Tensor)}
    recorded = {id(t) for t in calls.recorded.get(stream, [])}
    assert all(id(t) in used for t in there)
    if stream == 77:
        assert all(id(t) in recorded for t in there)
    else:   # the current one
        assert not calls.recorded


def test_raw_handles_of_the_default_stream(monkeypatch):
    monkeypatch.setattr(torch.cuda, "default_stream", lambda *a: "default")
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle: ("external", handle))
    monkeypatch.setattr(torch.cuda, "stream", lambda s: s)
    assert [TR._on(h) for h in (0, 1, 4096)] == ["default", "default", ("external", 4096)]
    with TR._on(None):
        pass


def test_status_waits_for_the_stream_of_the_last_call(calls, monkeypatch):
    """The word is read once the kernels that may write it are done."""
    order = []

    class Handle:
        def __init__(self, raw):
            self.raw = raw

        def synchronize(self):
            order.append(("wait", self.raw))

    monkeypatch.setattr(torch.cuda, "ExternalStream", Handle)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, stream: None, raising=False)
    monkeypatch.setattr(L, "moe_read_status", lambda ws, stream=None: order.append(("read", stream)) or 0)
    ex, x = experts(), torch.ones(4, 16)
    ex.status()
    ex.forward(x, OFF)
    ex.status()
    assert order == [("read", None)] * 2
    order.clear()
    ex.forward(x, OFF, stream=77)
    ex.status()
    ex.backward(x, stream=77)
    ex.status()
    ex.status(stream=78)
    assert order == [("wait", 77), ("read", None)] * 2 + [("read", 78)]


def test_a_workspace_is_not_zeroed_beyond_its_status_word(calls, monkeypatch):
    """The workspace of a large stack is as large as its matrices."""
    zeroed = []
    real = torch.zeros
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: zeroed.append(a) or real(*a, **kw))
    monkeypatch.setattr(torch.Tensor, "zero_",
                        lambda t: zeroed.append((t.numel() * t.element_size(),)) or t.fill_(0),
                        raising=False)
    m = torch.ones(2, 8, 16)
    TR.orthogonalize(m)
    assert zeroed == []
    ws = TR.orthogonalize_workspace(m)
    assert zeroed == [(4,)] and ws.numel() == 1 << 16 and (ws[:4] == 0).all()
    TR.orthogonalize(m, ws=ws)
    assert zeroed == [(4,)] and [a[3] is ws for a in calls.named("moe_orthogonalize")] == [False, True]


def test_orthogonalize_refuses_a_workspace_that_is_not_memory_of_its_device(calls):
    m = torch.ones(2, 8, 16)
    for ws in (torch.empty(1 << 16, dtype=torch.uint8, device="meta"),
               torch.empty(1 << 17, dtype=torch.uint8)[::2]):
        with pytest.raises(ValueError, match="ws"):
            TR.orthogonalize(m, ws=ws)
    assert not calls
    TR.orthogonalize(m, ws=torch.empty(1 << 14))


def test_pointers_of_subclasses_of_int():
    class Address(int):
        pass

    assert L._ptr(Address(4096)) == 4096 and L._ptr(None) is None
    assert L._ptr(torch.ones(1)) != 0


@pytest.mark.parametrize("beta", [False, True])
def test_norm_gradients_add_up_when_asked_to(calls, monkeypatch, beta):
    """Two micro-batches: without accumulate the second one's gradients alone
    remain, with it their sum; the first one after zero_grad writes."""
    nm = TR.LayerNorm(torch.ones(16), torch.ones(16) if beta else None)
    x, given = torch.ones(4, 16), []

    def backward(shape, dy, x, gamma, mean, rstd, dx, dgamma, dbeta, ws, stream=None):
        given.append((dgamma, dbeta))
        for t in (dgamma, dbeta):
            if t is not None:
                t.fill_(float(dy[0, 0]))

    monkeypatch.setattr(L, "moe_layer_norm_backward", backward)

    def step(value, **kw):
        nm.forward(x)
        nm.backward(torch.full((4, 16), float(value)), **kw)
        for t in (nm.dgamma, nm.dbeta):
            if t is not None:
                assert (t == t[0]).all()
        assert (nm.dbeta is None) is not beta
        return float(nm.dgamma[0] if not beta else nm.dbeta[0])

    assert step(3, accumulate=True) == 3  # nothing was there
    assert given[0][0] is nm.dgamma
    assert step(4, accumulate=True) == 7
    assert step(5) == 5
    assert step(1, accumulate=True) == 6
    nm.zero_grad()
    assert step(2, accumulate=True) == 2
