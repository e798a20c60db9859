"""Helpers called with a stream other than the current one, without a GPU: whose memory they
allocate from, and for which streams the allocator is told to hold it."""
import contextlib

import pytest
import torch

from exact_attention_126_b200 import fa

BF16 = torch.bfloat16
HOME, OTHER = 11, 22


class Stream:
    def __init__(self, handle, device=None):
        self.cuda_stream = handle


class Machine:
    def __init__(self):
        self.current = HOME
        self.allocated = []  # (address, stream whose memory it is)
        self.held = []       # (address, stream)
        self.launched = []   # streams


@pytest.fixture
def machine(monkeypatch):
    m = Machine()

    @contextlib.contextmanager
    def stream(s):
        before, m.current = m.current, s.cuda_stream
        yield
        m.current = before

    def allocating(make):
        def f(*args, **kw):
            t = make(*args, **kw)
            m.allocated.append((t.data_ptr(), m.current))
            return t
        return f

    monkeypatch.setattr(fa, "_elsewhere", lambda t: False)
    monkeypatch.setattr(fa, "_check_inputs", lambda *t: None)
    monkeypatch.setattr(fa, "_stream", lambda s: m.current if s is None else int(s))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: Stream(m.current))
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    monkeypatch.setattr(torch, "empty", allocating(torch.empty))
    monkeypatch.setattr(torch, "empty_like", allocating(torch.empty_like))
    monkeypatch.setattr(torch.Tensor, "new_empty", allocating(torch.Tensor.new_empty))
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: m.held.append((t.data_ptr(), s.cuda_stream)))
    for name, at in (("fa_fwd", 8), ("fa_fwd_ex", 9), ("fa_bwd", 13), ("fa_qk_norm_rope_fwd", 10),
                     ("fa_qk_norm_rope_bwd", 15)):
        monkeypatch.setattr(fa, name, lambda *a, at=at, **kw: m.launched.append(
            fa._stream(a[at] if len(a) > at else kw.get("stream"))))
    monkeypatch.setattr(fa, "fa_bwd_workspace_bytes_ex", lambda *a: 64)
    return m


def calls():
    q, k, v, o, do = (torch.zeros(1, 2, 3, 64, dtype=BF16) for _ in range(5))
    lse = torch.zeros(1, 2, 3)
    w = torch.ones(64)
    out = [torch.zeros(1, 3, 2, 64, dtype=BF16) for _ in range(3)]
    rows = lambda t: t.transpose(1, 2).contiguous()  # noqa
    yield (lambda s: fa.attention_forward(q, k, v, stream=s)), (q, k, v)
    yield (lambda s: fa.attention_forward(q, k, v, stream=s, keep_residual=True)), (q, k, v)
    yield (lambda s: fa.attention_backward(q, k, v, o, lse, do, stream=s)), (q, k, v, o, lse, do)
    x, y, z = rows(q), rows(k), rows(v)
    yield (lambda s: fa.qk_norm_rope_forward(x, y, z, q_weight=w, stream=s)), (x, y, z, w)
    yield (lambda s: fa.qk_norm_rope_backward(q, k, v, q=x, k=y, q_weight=w, stream=s)), (
        q, k, v, x, y, w)
    yield (lambda s: fa.qk_norm_rope_backward(q, k, v, q=x, k=y, q_weight=w, stream=s, out=out)), (
        q, k, v, x, y, w, *out)


@pytest.mark.parametrize("which", range(6))
def test_memory_of_a_call_on_another_stream(machine, which):
    # (inputs made before what the call allocates is noted)
    call, inputs = list(calls())[which]
    del machine.allocated[:]
    res = call(OTHER)
    assert machine.launched == [OTHER] and machine.current == HOME
    assert machine.allocated and all(s == OTHER for _, s in machine.allocated)
    held = set(machine.held)
    assert all((t.data_ptr(), OTHER) in held for t in inputs)
    assert all((t.data_ptr(), HOME) in held for t in res if t is not None)


@pytest.mark.parametrize("which", range(6))
@pytest.mark.parametrize("stream", [None, HOME])
def test_memory_of_a_call_on_the_current_stream(machine, which, stream):
    call, inputs = list(calls())[which]
    del machine.allocated[:]
    call(stream)
    assert machine.launched == [HOME] and not machine.held
    assert all(s == HOME for _, s in machine.allocated)
