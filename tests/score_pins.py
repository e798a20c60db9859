"""Pins of the oracle's capped scores and prefixes (each a function of an Oracle)."""
import math

import numpy as np
import torch


def _inputs(seed, *shape, n=4):
    return np.random.default_rng(seed).normal(size=(n,) + shape)


def pin_no_cap_no_prefix_is_identity(orc):
    q, k, v, do = _inputs(0, 2, 2, 7, 3)
    a = orc.fwd(q, k, v, 0.7, True) + orc.bwd(q, k, v, do, 0.7, True)
    kw = dict(softcap=0.0, prefixes=[0, 0])
    b = orc.fwd(q, k, v, 0.7, True, **kw) + orc.bwd(q, k, v, do, 0.7, True, **kw)
    for x, y in zip(a, b):
        assert np.array_equal(x, y)


def pin_cap_two_keys(orc):
    """One query, two keys with known scores: the weights are those of the capped ones."""
    q = np.array([1.0, 0.0]).reshape(1, 1, 2, 1)
    k = np.array([3.0, -1.0]).reshape(1, 1, 2, 1)
    v = np.array([1.0, 0.0]).reshape(1, 1, 2, 1)
    o, lse = orc.fwd(q, k, v, 2.0, softcap=1.5)
    s = [1.5 * math.tanh(6.0 / 1.5), 1.5 * math.tanh(-2.0 / 1.5)]
    np.testing.assert_allclose(o[0, 0, 0, 0], 1 / (1 + math.exp(s[1] - s[0])), rtol=1e-12)
    np.testing.assert_allclose(lse[0, 0, 0], math.log(math.exp(s[0]) + math.exp(s[1])), rtol=1e-12)


def pin_large_cap_is_no_cap(orc):
    q, k, v, do = _inputs(1, 1, 2, 6, 4)
    a = orc.fwd(q, k, v, 0.5) + orc.bwd(q, k, v, do, 0.5)
    b = orc.fwd(q, k, v, 0.5, softcap=1e6) + orc.bwd(q, k, v, do, 0.5, softcap=1e6)
    for x, y in zip(a, b):
        np.testing.assert_allclose(x, y, atol=1e-9)


def pin_prefix_of_all_keys_is_no_mask(orc):
    q, k, v, do = _inputs(2, 2, 1, 6, 3)
    kw = dict(prefixes=[6, 6])
    a = orc.fwd(q, k, v, 0.5) + orc.bwd(q, k, v, do, 0.5)
    b = orc.fwd(q, k, v, 0.5, True, **kw) + orc.bwd(q, k, v, do, 0.5, True, **kw)
    for x, y in zip(a, b):
        np.testing.assert_allclose(x, y, atol=1e-12)


def pin_prefix_rows(orc):
    """Rows inside a prefix see exactly its keys, rows behind it are causal."""
    q, k, v, _ = _inputs(3, 2, 1, 8, 3)
    o, lse = orc.fwd(q, k, v, 0.5, True, prefixes=[5, 2])
    for b, p in enumerate((5, 2)):
        for i in range(8):
            n = max(i + 1, p)
            oi, li = orc.fwd(np.repeat(q[b:b + 1, :, i:i + 1], n, 2), k[b:b + 1, :, :n],
                             v[b:b + 1, :, :n], 0.5)
            np.testing.assert_allclose(o[b, 0, i], oi[0, 0, 0], atol=1e-12)
            np.testing.assert_allclose(lse[b, 0, i], li[0, 0, 0], atol=1e-12)


def pin_prefix_within_lengths(orc):
    q, k, v, do = _inputs(4, 1, 1, 8, 3)
    kw = dict(prefixes=[7], lengths=[5])
    o, lse = orc.fwd(q, k, v, 0.5, True, **kw)
    g = orc.bwd(q, k, v, do, 0.5, True, **kw)
    cut = [x[:, :, :5] for x in (q, k, v, do)]
    o5, lse5 = orc.fwd(*cut[:3], 0.5)
    g5 = orc.bwd(*cut, 0.5)
    np.testing.assert_allclose(o[:, :, :5], o5, atol=1e-12)
    np.testing.assert_allclose(lse[:, :, :5], lse5, atol=1e-12)
    assert (o[:, :, 5:] == 0).all() and np.isneginf(lse[:, :, 5:]).all()
    for x, y in zip(g, g5):
        np.testing.assert_allclose(x[:, :, :5], y, atol=1e-12)
        assert (x[:, :, 5:] == 0).all()


def pin_finite_differences(orc):
    rng = np.random.default_rng(5)
    for N, d, causal, kw in [(3, 2, False, dict(softcap=0.8)), (5, 3, True, dict(softcap=2.0)),
                             (6, 2, True, dict(prefixes=[4])),
                             (6, 2, True, dict(prefixes=[3], softcap=1.1, alibi=[0.3]))]:
        q, k, v, do = rng.normal(size=(4, 1, 1, N, d))
        got = orc.bwd(q, k, v, do, 0.9, causal, **kw)
        for t in range(3):
            for idx in np.ndindex(q.shape):
                def loss(h):
                    x = [a.copy() for a in (q, k, v)]
                    x[t][idx] += h
                    return (orc.fwd(*x, 0.9, causal, **kw)[0] * do).sum()
                fd = (loss(1e-5) - loss(-1e-5)) / 2e-5
                np.testing.assert_allclose(got[t][idx], fd, atol=2e-8)


def pin_library_autograd(orc):
    B, H, N, d = 2, 2, 9, 4
    q, k, v, do = _inputs(6, B, H, N, d)
    pre, cap, slopes = [6, 0], 1.7, [0.2, 0.05]
    kw = dict(softcap=cap, prefixes=pre, alibi=slopes)
    o, lse = orc.fwd(q, k, v, 0.6, True, **kw)
    g = orc.bwd(q, k, v, do, 0.6, True, **kw)
    tq, tk, tv = (torch.tensor(x, requires_grad=True) for x in (q, k, v))
    s = cap * torch.tanh(tq @ tk.transpose(2, 3) * 0.6 / cap)
    n = torch.arange(N)
    s = s - torch.tensor(slopes, dtype=torch.float64)[:, None, None] * (n[:, None] - n[None, :]).abs()
    vis = (n[None, :] <= n[:, None]) | (n < torch.tensor(pre)[:, None])[:, None, None, :]
    s = s.masked_fill(~vis, -math.inf)
    to = torch.softmax(s, -1) @ tv
    (to * torch.tensor(do)).sum().backward()
    np.testing.assert_allclose(o, to.detach(), atol=1e-12)
    np.testing.assert_allclose(lse, torch.logsumexp(s, -1).detach(), atol=1e-12)
    for x, t in zip(g, (tq, tk, tv)):
        np.testing.assert_allclose(x, t.grad, atol=1e-12)


ALL_PINS = [f for n, f in sorted(globals().items()) if n.startswith("pin_")]
