"""Helpers called with a stream other than the current one, while calls of the current stream are
pending: the kernels are deterministic, so every result has to be the one of a call by itself, bit
for bit."""
import pytest
import torch

from exact_attention_126_b200 import fa
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def problem(seed, B=4, H=8, N=1500, d=64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(B, N, 3 * H, d, device="cuda", generator=g).to(BF16)
    do = torch.randn(B, H, N, d, device="cuda", generator=g).to(BF16)
    return dict(x=x, do=do, w=1 + 0.3 * torch.randn(d, device="cuda", generator=g),
                f=10000.0 ** -(torch.arange(32, device="cuda") / 32.0), H=H)


def layer(p, stream=None, softcap=0.0):
    """Norm and rotation, attention, and their gradients; whatever lies between is dropped."""
    rope = dict(q_weight=p["w"], k_weight=p["w"], inv_freq=p["f"], stream=stream)
    att = dict(causal=True, softcap=softcap, stream=stream)
    x, y, z = p["x"].split(p["H"], 2)
    q, k, v = fa.qk_norm_rope_forward(x, y, z, **rope)
    o, lse, low = fa.attention_forward(q, k, v, keep_residual=True, **att)
    grads = fa.attention_backward(q, k, v, o, lse, p["do"], o_low=low, **att)
    return (o, lse) + fa.qk_norm_rope_backward(*grads, q=x, k=y, **rope)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_pending_calls_of_the_current_stream(softcap):
    a, b = problem(1), problem(2)
    want = layer(a, softcap=softcap), layer(b, softcap=softcap)
    torch.cuda.synchronize()
    s1 = torch.cuda.Stream()
    s1.wait_stream(torch.cuda.current_stream())
    runs = []
    for i in range(8):  # (kept or dropped at once, so that blocks change hands)
        r = layer(a, softcap=softcap), layer(b, s1 if i % 2 else s1.cuda_stream, softcap)
        if i % 3:
            runs.append(r)
    torch.cuda.synchronize()
    for r in runs:
        assert same(r[0], want[0]) and same(r[1], want[1])


def test_temporary_arguments_on_another_stream():
    """Arguments that nobody holds after the call; the allocator may hand their memory to the next
    call on their stream only behind the kernels that read them."""
    p = problem(3)
    want = layer(p)
    torch.cuda.synchronize()
    s1 = torch.cuda.Stream()
    got = []
    for _ in range(6):
        t = dict(p, x=p["x"].clone(), do=p["do"].clone())
        s1.wait_stream(torch.cuda.current_stream())
        got.append(layer(t, s1))
        del t
        torch.full_like(p["x"], 7.0)
        torch.full_like(p["do"], 7.0)
    torch.cuda.synchronize()
    assert all(same(g, want) for g in got)


def test_the_default_stream_from_another():
    p = problem(4, B=1, N=200)
    want = layer(p)
    torch.cuda.synchronize()
    default = torch.cuda.default_stream()
    with torch.cuda.stream(torch.cuda.Stream()):
        got = [layer(p, s) for s in (default, default.cuda_stream)]
    torch.cuda.synchronize()
    assert all(same(g, want) for g in got)


def test_forked_stream_inside_a_graph():
    a, b = problem(5, B=1, N=300), problem(6, B=1, N=300)
    want = layer(a), layer(b)
    torch.cuda.synchronize()
    s1 = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cur = torch.cuda.current_stream()
        s1.wait_stream(cur)
        got = layer(a), layer(b, s1)
        cur.wait_stream(s1)
    for _ in range(3):
        for r in got:
            for t in r:
                t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(got[0], want[0]) and same(got[1], want[1])


def test_e4m3_forward_on_another_stream():
    q, k, v = (torch.randn(2, 4, 700, 128, device="cuda").to(torch.float8_e4m3fn)
               for _ in range(3))
    want = fa.attention_forward_fp8(q, k, v, causal=True)
    torch.cuda.synchronize()
    s1 = torch.cuda.Stream()
    runs = [fa.attention_forward_fp8(q, k, v, causal=True, stream=s) for s in (None, s1) * 3]
    torch.cuda.synchronize()
    assert all(same(r, want) for r in runs)
