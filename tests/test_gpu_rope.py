"""Per-head norm and rotary positions on the GPU against the 64-bit reference.

Tolerances, from the arithmetic. Outputs are rounded once to bf16: at most half a step, 2^-8 of
the value. Before that everything is fp32: a row's sum of squares has 16 sequential terms per lane
at most and up to four shuffles, the products a handful of roundings and the cosines an absolute error below
2^-22, so a value is off by less than 32 * 2^-24 of its row's largest magnitude, about 2e-6. The
gains' gradients are fp32 sums of the terms g x^: at most (rows + 64) roundings of 2^-24 of the sum
of magnitudes, and each term carries the error of its g = e cos + f sin, a turned value like the
others: where the two members cancel, 2e-6 of the row's largest |dy| (not of g), times |x^|."""
import numpy as np
import pytest
import torch

import rope_ref
from exact_attention_126_b200 import build, fa

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    build.build()


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, scale, what):
    """|got - ref| <= 2^-8 |ref| + 2e-6 of the row's scale."""
    got = f64(got)
    assert np.isfinite(got).all(), what
    bad = np.abs(got - ref) > 2.0 ** -8 * np.abs(ref) + 2e-6 * scale
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3],
                           float(np.abs(got - ref).max()))


def make(tokens, heads, d, rot, axes, seed=0, positions=None, gains=True, spread=False):
    """A fused projection's output and what a call takes beside it."""
    dev = torch.device("cuda:0")
    g = torch.Generator(device=dev).manual_seed(seed)
    x = torch.randn(*tokens, sum(heads), d, device=dev, generator=g)
    if spread:  # rows of very uneven size
        x = x * 10.0 ** torch.randint(-4, 5, x.shape[:-1] + (1,), device=dev, generator=g)
    x = x.to(BF16)
    kw = {}
    if gains:
        kw["q_weight"] = 1 + 0.3 * torch.randn(d, device=dev, generator=g)
        kw["k_weight"] = 1 + 0.3 * torch.randn(d, device=dev, generator=g)
    if rot:
        p = torch.arange(rot // 2, device=dev, dtype=torch.float64)
        kw["inv_freq"] = (10000.0 ** (-2 * p / rot)).float()
        if positions == "far":
            kw["positions"] = torch.randint(-2 ** 31, 2 ** 31, (axes,) + tokens, device=dev,
                                            generator=g).to(torch.int32)
        elif positions is not None or axes > 1:
            kw["positions"] = torch.randint(0, 5000, (axes,) + tokens, device=dev,
                                            generator=g).to(torch.int32)
        if axes > 1:
            kw["pair_axis"] = torch.randint(0, axes, (rot // 2,), device=dev, generator=g).to(
                torch.uint8)
    return x, kw


def flat_angles(tokens, kw, places):
    """(rows, rot/2) angles; places: the place in the sequence of each flat token."""
    if "inv_freq" not in kw:
        return np.zeros((len(places), 0))
    pos = f64(kw["positions"]).reshape(-1, len(places)) if "positions" in kw else places[None]
    axis = kw["pair_axis"].cpu().numpy() if "pair_axis" in kw else None
    return rope_ref.angles(pos, f64(kw["inv_freq"]), axis)


def token_major(t, packed):
    """(B, H, N, d) or (total, H, d) -> (rows, H, d)."""
    return t if packed else t.transpose(1, 2).reshape(-1, t.shape[1], t.shape[3])


def check(x, heads, kw, interleaved=False, norm=True, eps=EPS, live=None, places=None, seed=1,
          **call):
    """Forward and backward of a dense (B, N, heads, d) or packed (total, heads, d) projection;
    live: which flat tokens the call is to work on."""
    packed = x.dim() == 3
    d = x.shape[-1]
    q, k, v = x.split(heads, -2)
    rows = x.shape[0] if packed else x.shape[0] * x.shape[1]
    if places is None:
        places = np.arange(rows) if packed else np.tile(np.arange(x.shape[1]), x.shape[0])
    live = np.ones(rows, bool) if live is None else live
    ang = flat_angles(x.shape[:-2], kw, places)
    outs = fa.qk_norm_rope_forward(q, k, v, eps=eps, norm=norm, interleaved=interleaved, **kw,
                                   **call)
    g = torch.Generator(device=x.device).manual_seed(seed)
    grads_in = [torch.randn(o.shape, device=o.device, generator=g).to(BF16) for o in outs]
    for t in grads_in:  # what lies in rows that take no part must not matter
        token_major(t, packed)  # (shape check)
        if packed:
            t[torch.from_numpy(~live).to(t.device)] = float("nan")
        else:
            m = torch.from_numpy(~live.reshape(x.shape[:2])).to(t.device)
            t.masked_fill_(m[:, None, :, None], float("nan"))
    back = fa.qk_norm_rope_backward(*grads_in, q=q, k=k, eps=eps, norm=norm,
                                    interleaved=interleaved, **kw, **call)
    torch.cuda.synchronize()
    for i, (src, out, dy) in enumerate(zip((q, k, v), outs, grads_in)):
        src = f64(src).reshape(rows, heads[i], d)[live]
        out = token_major(out, packed).reshape(rows, heads[i], d)
        dy = f64(token_major(dy, packed)).reshape(rows, heads[i], d)[live]
        got = back[i].reshape(rows, heads[i], d)
        if not packed:  # rows past a length are zero on either side
            assert (f64(out)[~live] == 0).all() and (f64(got)[~live] == 0).all()
        lv = torch.from_numpy(live)
        out, got = out.cpu()[lv], got.cpu()[lv]
        if i == 2:
            assert np.array_equal(f64(out), src) and np.array_equal(f64(got), dy)
            continue
        gain = kw.get("q_weight" if i == 0 else "k_weight")
        gain = None if gain is None else f64(gain)
        ref = rope_ref.forward(src, gain, ang[live], interleaved, norm, eps)
        u = rope_ref.forward(src, gain, ang[live][:, :0], interleaved, norm, eps)
        close(out, ref, np.abs(u).max(-1, keepdims=True), "output %d" % i)
        dx, dg, mag = rope_ref.backward(dy, src, gain, ang[live], interleaved, norm, eps)
        if norm:
            r = 1.0 / np.sqrt((src * src).mean(-1, keepdims=True) + eps)
            t = np.abs(dy).max(-1, keepdims=True) * (1 if gain is None else np.abs(gain).max())
            scale = 2 * r * t * (1 + np.abs(src * r).max(-1, keepdims=True))
        else:
            scale = 2 * np.abs(dy).max(-1, keepdims=True)
        close(got, dx, scale, "gradient %d" % i)
        if gain is not None:
            n = live.sum() * heads[i]
            assert back[3 + i].dtype == torch.float32
            err = np.abs(f64(back[3 + i]) - dg)
            turned = (np.abs(dy).max(-1, keepdims=True) * np.abs(src * r)).sum((0, 1))
            assert (err <= (n + 64) * 2.0 ** -24 * mag + 2e-6 * turned).all(), (i, err.max())
        else:
            assert back[3 + i] is None
    return outs, back


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,axes", [(0, 1), (8, 1), (16, 1), (40, 2), (64, 3), (None, 1)])
def test_rotations(d, interleaved, rot, axes):
    rot = d if rot is None else rot
    x, kw = make((2, 37), (3, 1, 1), d, rot, axes)
    check(x, (3, 1, 1), kw, interleaved)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("heads", [(1, 1, 1), (8, 8, 8), (9, 3, 3), (33, 1, 1), (5, 17, 2)])
@pytest.mark.parametrize("tokens", [(1, 1), (3, 1), (1, 130)])
def test_heads(d, heads, tokens):
    x, kw = make(tokens, heads, d, d, 1, positions="near")
    check(x, heads, kw)


@pytest.mark.parametrize("norm,gains", [(True, False), (False, False)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_without_gain_and_without_norm(norm, gains, interleaved):
    x, kw = make((3, 50), (4, 2, 2), 64, 32, 2, gains=gains)
    check(x, (4, 2, 2), kw, interleaved, norm=norm)


def test_one_gain():
    x, kw = make((2, 9), (2, 2, 2), 64, 64, 1)
    gain = kw.pop("k_weight")
    check(x, (2, 2, 2), kw)
    kw["k_weight"] = gain
    del kw["q_weight"]
    check(x, (2, 2, 2), kw)


@pytest.mark.parametrize("axes", [1, 3])
def test_far_positions(axes):
    x, kw = make((2, 65), (2, 2, 2), 128, 128, axes, positions="far")
    check(x, (2, 2, 2), kw)
    kw["inv_freq"] = torch.linspace(0.0, 6.5, 64, device=x.device)  # past a turn per position
    kw["positions"] = kw["positions"] // 4096
    check(x, (2, 2, 2), kw, True)


def test_rows_of_uneven_size():
    x, kw = make((2, 40), (4, 4, 1), 128, 128, 1, spread=True)
    check(x, (4, 4, 1), kw)
    check(x, (4, 4, 1), kw, eps=0.0)
    x, kw = make((1, 5), (3, 5, 1), 64, 64, 1)  # rows of a step that hold no head
    check(x, (3, 5, 1), kw, eps=0.0)
    x, kw = make((2, 40), (4, 4, 1), 128, 128, 1, spread=True)
    x[0, 3] = 0  # a row of zeros: 0 / sqrt(eps)
    check(x, (4, 4, 1), kw)


def test_many_tokens():
    # every block takes several tokens
    x, kw = make((3, 2731), (6, 2, 2), 64, 64, 1)
    check(x, (6, 2, 2), kw)
    x, kw = make((1, 9001), (2, 1, 1), 128, 64, 2)
    check(x, (2, 1, 1), kw, True)


# Large problems go through tiles of tokens (32 at d 64, 16 at d 128) by heads (4): odd numbers of
# both, heads that share a tile with none, several tiles per block.
@pytest.mark.parametrize("d,heads", [(64, (9, 3, 3)), (128, (5, 2, 1))])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot,axes,norm", [(None, 1, True), (24, 3, True), (0, 1, True),
                                           (None, 2, False)])
def test_tiles(d, heads, interleaved, rot, axes, norm):
    x, kw = make((5, 3503), heads, d, d if rot is None else rot, axes, gains=norm)
    check(x, heads, kw, interleaved, norm=norm)


# (the forward at d 128 takes tiles from 96 MB on)
@pytest.mark.parametrize("interleaved,rot,axes,norm", [(False, None, 1, True), (True, 24, 3, True),
                                                       (False, None, 2, False)])
def test_tiles_of_a_large_batch(interleaved, rot, axes, norm):
    d, heads = 128, (21, 6, 5)
    x, kw = make((3, 4333), heads, d, d if rot is None else rot, axes, gains=norm)
    assert x.numel() * 2 > 97 << 20
    check(x, heads, kw, interleaved, norm=norm)


@pytest.mark.parametrize("padded", [True, False])
def test_tiles_of_a_large_batch_of_lengths(padded):
    d, heads = 128, (21, 6, 5)
    if padded:
        N, lens = 2111, [2111, 0, 33, 1, 5000, 2048]
        x, kw = make((6, N), heads, d, d, 1)
        live = (np.arange(N) < np.array(lens)[:, None]).reshape(-1)
        x[torch.from_numpy(~live.reshape(6, N))] = float("nan")
        check(x, heads, kw, live=live, eps=0.0,
              seq_lengths=torch.tensor(lens, dtype=torch.int32, device=x.device))
    else:
        lens, first, total, N = [5, 0, 5400, 1, 0, 4900, 2000, 0], 37, 12600, 5000
        cu = first + np.concatenate([[0], np.cumsum(lens)])
        x, kw = make((total,), heads, d, d, 1)
        live, places = np.zeros(total, bool), np.zeros(total)
        for b, n in enumerate(lens):
            live[cu[b]:cu[b] + min(n, N)] = True
            places[cu[b]:cu[b] + n] = np.arange(n)
        x[torch.from_numpy(~live)] = float("inf")
        check(x, heads, kw, live=live, places=places, max_seqlen=N,
              cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=x.device))
    assert x.numel() * 2 > 97 << 20


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [17, 33, 65, 257])
def test_large_batches_of_short_sequences(d, N):
    """Either side of the rule that keeps tiles of few rows out."""
    heads = (9, 4, 3) if d == 64 else (4, 2, 2)
    x, kw = make((33000 // N, N), heads, d, d, 1)
    assert x.numel() * 2 > 33 << 20
    check(x, heads, kw)


@pytest.mark.parametrize("d", [64, 128])
def test_tiles_of_a_padded_batch(d):
    B, N, heads = 7, 2705, (6, 5, 4)
    x, kw = make((B, N), heads, d, d, 1)
    lens = [2705, 0, 33, 1, 5000, 2048, 1000]
    live = (np.arange(N) < np.array(lens)[:, None]).reshape(-1)
    x[torch.from_numpy(~live.reshape(B, N))] = float("nan")
    check(x, heads, kw, live=live, eps=0.0,
          seq_lengths=torch.tensor(lens, dtype=torch.int32, device=x.device))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("given", [False, True])
def test_tiles_of_a_packed_batch(d, given):
    lens, first, total, N = [5, 0, 6400, 1, 0, 9000, 3400, 0], 37, 19000, 8000
    heads = (6, 3, 5)
    cu = first + np.concatenate([[0], np.cumsum(lens)])
    x, kw = make((total,), heads, d, d, 1, positions="near" if given else None)
    live, places = np.zeros(total, bool), np.zeros(total)
    for b, n in enumerate(lens):
        live[cu[b]:cu[b] + min(n, N)] = True
        places[cu[b]:cu[b] + n] = np.arange(n)
    x[torch.from_numpy(~live)] = float("inf")
    call = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=x.device), max_seqlen=N)
    check(x, heads, kw, live=live, places=places, **call)
    # in place, and rows that no sequence covers stay as they were
    q, k, v = x.split(heads, -2)
    ref = fa.qk_norm_rope_forward(q, k, v, **kw, **call)
    y = x.clone()
    B, N, params = fa._norm_rope_params(0, (total,), d, kw["q_weight"], kw["k_weight"],
                                        1e-6, True, kw["inv_freq"], kw.get("positions"), None,
                                        False, None, call["cu_seqlens"], N)
    parts = [fa._rows(t, "x", (total,), d, 0, 1) for t in y.split(heads, 1)]
    fa.fa_qk_norm_rope_fwd(*parts, *parts, B, N, d, params)
    for a, b in zip(y.split(heads, 1), ref):
        assert torch.equal(a.cpu()[torch.from_numpy(live)], b.cpu()[torch.from_numpy(live)])
    assert torch.isinf(y.cpu()[torch.from_numpy(~live)]).all()


def test_tiles_and_rows_agree():
    """A stride of 0 (shared rows) keeps a call out of the tiles: the same values either way; and
    repeats, streams and a graph of the tile kernels."""
    dev = torch.device("cuda:0")
    x, kw = make((4, 4200), (8, 1, 4), 64, 64, 1)
    q, k, v = x.split((8, 1, 4), 2)
    k4 = k.expand(4, 4200, 4, 64)
    a = fa.qk_norm_rope_forward(q, k4, v, **kw)
    b = fa.qk_norm_rope_forward(q, k4.contiguous(), v, **kw)
    for s, t in zip(a, b):
        # (the norm's sum in another order: at most one bf16 step apart)
        assert (s.float() - t.float()).abs().max() <= 2.0 ** -7 * s.float().abs().max()
        assert (s != t).float().mean() < 1e-3
    dy = [torch.randn_like(t) for t in b]
    kc = k4.contiguous()
    ref = fa.qk_norm_rope_backward(*dy, q=q, k=kc, **kw)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for _ in range(4):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                runs.append(fa.qk_norm_rope_backward(*dy, q=q, k=kc, **kw))
    torch.cuda.synchronize()
    for r in runs:
        assert all(torch.equal(m, n) for m, n in zip(r, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.qk_norm_rope_forward(q, kc, v, **kw)
        grads = fa.qk_norm_rope_backward(*dy, q=q, k=kc, **kw)
    for t in out + grads:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(m, n) for m, n in zip(out, b))
    assert all(torch.equal(m, n) for m, n in zip(grads, ref))
    assert fa.fa_debug_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_padded_batch(d):
    B, N = 5, 70
    x, kw = make((B, N), (4, 2, 2), d, d, 1)
    lens = [70, 0, 33, 1, 99]  # (clamped)
    live = (np.arange(N) < np.array(lens)[:, None]).reshape(-1)
    x[torch.from_numpy(~live.reshape(B, N))] = float("nan")
    check(x, (4, 2, 2), kw, live=live,
          seq_lengths=torch.tensor(lens, dtype=torch.int32, device=x.device))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("given", [False, True])
def test_packed_batch(d, given):
    """Offsets that start past 0, empty sequences, one cut at N, tokens behind the last."""
    lens, first, total, N = [5, 0, 64, 1, 0, 90, 0], 3, 170, 80
    cu = first + np.concatenate([[0], np.cumsum(lens)])
    x, kw = make((total,), (4, 2, 2), d, d, 1, positions="near" if given else None)
    live, places = np.zeros(total, bool), np.zeros(total)
    for b, n in enumerate(lens):
        live[cu[b]:cu[b] + min(n, N)] = True
        places[cu[b]:cu[b] + n] = np.arange(n)
    x[torch.from_numpy(~live)] = float("inf")
    call = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=x.device), max_seqlen=N)
    check(x, (4, 2, 2), kw, live=live, places=places, **call)
    # tokens no sequence covers stay as they were, in place too
    y = x.clone()
    q, k, v = y.split((4, 2, 2), -2)
    out = [torch.full_like(t, 7.0) for t in (q, k, v)]
    g = [torch.randn_like(t) for t in (q, k, v)]
    fa.qk_norm_rope_backward(*g, q=q, k=k, out=out, **kw, **call)
    for t in out:
        assert (f64(t)[~live] == 7.0).all() and not (f64(t)[live] == 7.0).all()


@pytest.mark.parametrize("d,total", [(64, 170), (128, 170), (64, 19000), (128, 19000)])
@pytest.mark.parametrize("norm", [True, False])
def test_tokens_no_sequence_covers_are_zero(d, total, norm):
    """In tensors that the call allocates: before the first sequence, behind the last, past N, and
    where no sequence has a token at all; rows and tiles, on memory that held something else."""
    N = total // 4
    x, kw = make((total,), (6, 3, 5), d, d, 1, gains=norm)
    x[:] = torch.randn_like(x)
    q, k, v = x.split((6, 3, 5), 1)
    for cu in ([3, 3 + N // 2, 3 + N // 2, 3 + 3 * N], [7, 7, 7, 7], [0, 1, 1, total - 1]):
        live = np.zeros(total, bool)
        for a, b in zip(cu[:-1], cu[1:]):
            live[a:min(b, a + N)] = True
        dead = torch.from_numpy(~live).to(x.device)
        call = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device=x.device), max_seqlen=N,
                    norm=norm, **kw)
        for _ in range(2):
            junk = [torch.full_like(x, float("nan")), *(torch.full_like(t, float("nan"))
                                                        for t in (q, k, v))]
            torch.cuda.synchronize()
            del junk
            outs = fa.qk_norm_rope_forward(q, k, v, **call)
            back = fa.qk_norm_rope_backward(*outs, q=q, k=k, **call)
            for t in outs + back[:3]:
                assert (t[dead] == 0).all() and torch.isfinite(t.float()).all()
                assert (t[~dead].float().abs().amax((1, 2)) > 0).all()


def test_views_of_any_stride():
    """A projection stored head-major, a slice of wider rows, one tensor of queries and keys, and
    gradients into strided outputs with sentinels around them."""
    dev = torch.device("cuda:0")
    B, N, d = 2, 19, 64
    x, kw = make((B, N), (3, 3, 3), d, d, 1)
    ref, back = check(x, (3, 3, 3), kw)
    wide = torch.randn(B, N, 3, 3, d + 8, device=dev).to(BF16)
    wide[..., :d] = x.view(B, N, 3, 3, d)
    q, k, v = (wide[:, :, i, :, :d] for i in range(3))
    for a, b in zip(fa.qk_norm_rope_forward(q, k, v, eps=EPS, **kw), ref):
        assert torch.equal(a, b)
    hm = x.transpose(1, 2).contiguous().transpose(1, 2)  # (B, N, H, d), heads outermost
    q, k, v = hm.split(3, 2)
    for a, b in zip(fa.qk_norm_rope_forward(q, k, v, eps=EPS, **kw), ref):
        assert torch.equal(a, b)
    g = torch.Generator(device=dev).manual_seed(1)
    dy = [torch.randn(o.shape, device=dev, generator=g).to(BF16) for o in ref]
    hold = torch.full((B, N + 2, 11, d + 16), 3.0, device=dev, dtype=BF16)
    out = [hold[:, 1:-1, 1 + 3 * i:4 + 3 * i, 8:d + 8] for i in range(3)]
    # incoming gradients of another layout than the forward's outputs
    res = fa.qk_norm_rope_backward(*[t.transpose(1, 2).contiguous().transpose(1, 2) for t in dy],
                                   q=q, k=k, eps=EPS, out=out, **kw)
    for a, b in zip(res, back):
        assert torch.equal(a, b)
    mask = torch.ones_like(hold, dtype=torch.bool)
    mask[:, 1:-1, 1:10, 8:d + 8] = False
    assert (hold[mask] == 3.0).all()


@pytest.mark.parametrize("N", [7, 6000])
def test_rows_far_apart(N):
    """Batch entries more than 2^31 elements from each other (views of a large buffer), through the
    row kernels and through tiles."""
    dev = torch.device("cuda:0")
    heads, d, step = (8, 8, 8), 64, 3 << 30
    x, kw = make((2, N), heads, d, d, 1)
    hold = torch.empty(step + N * 24 * d, dtype=BF16, device=dev)
    far = hold.as_strided((2, N, 24, d), (step, 24 * d, d, 1))
    far.copy_(x)
    ref = fa.qk_norm_rope_forward(*x.split(heads, 2), **kw)
    got = fa.qk_norm_rope_forward(*far.split(heads, 2), **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    dy = [torch.randn_like(t) for t in ref]
    q, k, v = x.split(heads, 2)
    ref = fa.qk_norm_rope_backward(*dy, q=q, k=k, **kw)
    q, k, v = far.split(heads, 2)
    got = fa.qk_norm_rope_backward(*dy, q=q, k=k, out=far.split(heads, 2), **kw)  # in place
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_calls_follow_their_tensors_device(monkeypatch):
    """A call on tensors of another device than the current one runs there (here: the one device,
    with the check made to say so once)."""
    x, kw = make((2, 9), (2, 2, 2), 64, 64, 1)
    q, k, v = x.split(2, 2)
    ref = fa.qk_norm_rope_forward(q, k, v, **kw)
    back = fa.qk_norm_rope_backward(*ref, q=q, k=k, **kw)
    att = fa.attention_forward(*ref, causal=True, softcap=5.0)
    grads = fa.attention_backward(*ref, *att, ref[0], causal=True, softcap=5.0)
    entered = []

    def elsewhere(t):
        entered.append(t.device)
        return len(entered) % 2 == 1  # the call itself; then the one under its device

    monkeypatch.setattr(fa, "_elsewhere", elsewhere)
    for f, args, kws, want in ((fa.qk_norm_rope_forward, (q, k, v), kw, ref),
                               (fa.qk_norm_rope_backward, ref, dict(q=q, k=k, **kw), back),
                               (fa.attention_forward, ref, dict(causal=True, softcap=5.0), att),
                               (fa.attention_backward, ref + att + (ref[0],),
                                dict(causal=True, softcap=5.0), grads)):
        n = len(entered)
        got = f(*args, **kws)
        assert len(entered) == n + 2
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_shared_input_rows():
    """One key head read as several (stride 0)."""
    x, kw = make((2, 21), (4, 1, 1), 64, 64, 1)
    q, k, v = x.split((4, 1, 1), 2)
    k4 = k.expand(2, 21, 4, 64)
    a = fa.qk_norm_rope_forward(q, k4, None, **kw)
    b = fa.qk_norm_rope_forward(q, k, None, **kw)
    assert len(a) == 2 and torch.equal(a[0], b[0])
    assert torch.equal(a[1], b[1].expand(2, 4, 21, 64))


@pytest.mark.parametrize("tokens", [(2, 21), (77,), (4, 4100)])
@pytest.mark.parametrize("values", [False, True])
def test_queries_without_keys(tokens, values):
    """A call on queries alone (or with values) gives what the whole call gives for them."""
    heads = (8, 2, 4)
    x, kw = make(tokens, heads, 64, 64, 1)
    call = {}
    if len(tokens) == 1:
        call = dict(cu_seqlens=torch.tensor([0, 30, 77], dtype=torch.int32, device=x.device),
                    max_seqlen=64)
    q, k, v = x.split(heads, -2)
    ref = fa.qk_norm_rope_forward(q, k, v, **kw, **call)
    back = fa.qk_norm_rope_backward(*ref, q=q, k=k, **kw, **call)
    kw["k_weight"] = None
    out = fa.qk_norm_rope_forward(q, None, v if values else None, **kw, **call)
    assert out[1] is None and len(out) == 2 + values
    assert torch.equal(out[0], ref[0]) and (not values or torch.equal(out[2], ref[2]))
    got = fa.qk_norm_rope_backward(out[0], None, out[2] if values else None, q=q, **kw, **call)
    assert got[1] is None and got[4] is None and (got[2] is None) == (not values)
    assert torch.equal(got[0], back[0]) and (not values or torch.equal(got[2], back[2]))
    # The gain's gradient is summed over other blocks than in the whole call, so in another order:
    # both are off by at most rows + 64 roundings of 2^-24 of the sum of the terms' magnitudes, and
    # a term is a turned dy (at most the norm of its two members, here sqrt(2) max |dy|) times x^
    # (at most sqrt(64)).
    rows = ref[0].numel() // 64
    most = rows * 2.0 ** 0.5 * float(ref[0].float().abs().max()) * 8.0
    assert float((got[3] - back[3]).abs().max()) <= 2 * (rows + 64) * 2.0 ** -24 * most
    given = [torch.empty_like(q), None, torch.empty_like(v) if values else None]
    again = fa.qk_norm_rope_backward(out[0], None, out[2] if values else None, q=q, out=given,
                                     **kw, **call)
    if len(tokens) == 2:
        assert again[0] is given[0] and torch.equal(again[0], got[0])
    with pytest.raises(ValueError):
        fa.qk_norm_rope_backward(ref[0], ref[1], q=q, **kw, **call)


def test_in_place():
    x, kw = make((77,), (4, 2, 2), 128, 64, 1)
    cu = torch.tensor([0, 30, 77], dtype=torch.int32, device=x.device)
    call = dict(cu_seqlens=cu, max_seqlen=64)
    q, k, v = x.split((4, 2, 2), 1)
    ref = fa.qk_norm_rope_forward(q, k, v, **kw, **call)
    y = x.clone()
    B, N, params = fa._norm_rope_params(0, (77,), 128, kw["q_weight"], kw["k_weight"],
                                        1e-6, True, kw["inv_freq"], None, None, False, None, cu,
                                        64)
    parts = [fa._rows(t, "x", (77,), 128, 0, 1) for t in y.split((4, 2, 2), 1)]
    fa.fa_qk_norm_rope_fwd(*parts, *parts, B, N, 128, params)
    for a, b in zip(y.split((4, 2, 2), 1), ref):
        assert torch.equal(a, b)


def test_repeats_streams_and_graphs():
    x, kw = make((4, 500), (6, 2, 2), 64, 64, 1)
    q, k, v = x.split((6, 2, 2), 2)
    ref = fa.qk_norm_rope_forward(q, k, v, **kw)
    dy = [torch.randn_like(t) for t in ref]
    back = fa.qk_norm_rope_backward(*dy, q=q, k=k, **kw)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for _ in range(10):
        with torch.cuda.stream(s1):
            runs.append(fa.qk_norm_rope_backward(*dy, q=q, k=k, **kw))
        with torch.cuda.stream(s2):
            runs.append(fa.qk_norm_rope_backward(*dy, q=q, k=k, **kw))
    runs.append(fa.qk_norm_rope_backward(*dy, q=q, k=k, stream=s1, **kw))
    torch.cuda.synchronize()
    for r in runs:
        assert all(torch.equal(a, b) for a, b in zip(r, back))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fa.qk_norm_rope_forward(q, k, v, **kw)
        grads = fa.qk_norm_rope_backward(*dy, q=q, k=k, **kw)
    for t in out + grads:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    assert all(torch.equal(a, b) for a, b in zip(grads, back))


def test_empty_batches():
    dev = torch.device("cuda:0")
    w = torch.ones(64, device=dev)
    x = torch.empty(0, 5, 3, 64, device=dev, dtype=BF16)
    q, k, v = x.split(1, 2)
    out = fa.qk_norm_rope_forward(q, k, v, q_weight=w)
    assert [tuple(t.shape) for t in out] == [(0, 1, 5, 64)] * 3
    back = fa.qk_norm_rope_backward(*out, q=q, k=k, q_weight=w)
    assert (back[3] == 0).all() and back[4] is None
    # a batch whose every row is past its length
    x = torch.full((2, 5, 3, 64), float("nan"), device=dev, dtype=BF16)
    lens = torch.zeros(2, dtype=torch.int32, device=dev)
    q, k, v = x.split(1, 2)
    out = fa.qk_norm_rope_forward(q, k, v, q_weight=w, seq_lengths=lens)
    assert all((t == 0).all() for t in out)
    back = fa.qk_norm_rope_backward(q.transpose(1, 2), k.transpose(1, 2), v.transpose(1, 2), q=q,
                                    k=k, q_weight=w, seq_lengths=lens)
    assert all((t == 0).all() for t in back[:4])


def test_refusals():
    x, kw = make((2, 6), (2, 2, 2), 64, 64, 1)
    q, k, v = x.split(2, 2)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q.float(), k, v)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, k[:, :5], v)
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, k, v, norm=False, q_weight=kw["q_weight"])
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, k, v, positions=torch.zeros(2, 6, device=x.device,
                                                               dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q, k, v, q_weight=kw["q_weight"].double())
    with pytest.raises(ValueError):
        fa.qk_norm_rope_forward(q[0], k[0], v[0])  # packed rows without offsets
    with pytest.raises(ValueError):
        fa.qk_norm_rope_backward(q.transpose(1, 2), k.transpose(1, 2))
    with pytest.raises(fa.FAError):  # rotary_dim 10
        fa.qk_norm_rope_forward(q, k, v, inv_freq=kw["inv_freq"][:5])
    with pytest.raises(fa.FAError):  # written rows that overlap
        fa.qk_norm_rope_backward(q.transpose(1, 2), k.transpose(1, 2), q=q, k=k,
                                 out=[q[:, :1].expand(2, 6, 2, 64), torch.empty_like(k)])
    assert fa.fa_debug_status() == 0
