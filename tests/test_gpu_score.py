"""Capped scores and prefixes on the GPU against the fp64 oracle.

Tolerances: those of the plain attention (gpu_helpers), whose arithmetic is the same: P, dS and
the outputs are rounded to bf16 (relative error up to 2^-8 each, 2^-8 / sqrt(3) in the norm), and
the cap adds an fp32 tanh: by polynomials up to |u| = 0.625 (4e-7 relative below 0.25, 1.1e-7
above), and beyond in the form 1 - 2 / (1 + e^2u) with an absolute error below 4e-7, so a score is
off by at most 4e-7 c, LSE by as much: 1e-3 holds up to c = 2500, where no score of these inputs
leaves the polynomials' ranges. Gradients with a cap can
be small where most scores sit on it (1 - tanh^2); the error of 1 - tanh^2 is below 1e-6, far
below the bf16 rounding of what remains unless the factor itself is below 1e-4."""
import ctypes

import numpy as np
import pytest
import torch

import oracle
from exact_attention_126_b200 import fa, synth
from gpu_helpers import (assert_within_bounds, cumulative, ensure_built, pack_rows, rel_frob)

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def inputs(B, H, N, d, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(1000 + seed)
    t = {n: torch.randn(B, H, N, d, generator=g) for n in ("q", "k", "v", "do")}
    t["q"] = t["q"] * spread
    return {n: x.to(BF16) for n, x in t.items()}


def run(inp, scale, causal, window=(-1, -1), softcap=0.0, prefixes=None, lengths=None,
        packed=False, alibi=None, key_padding=None, dropout=None, residual=True):
    dev = torch.device("cuda:0")
    B, H, N, d = inp["q"].shape
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=dev)  # noqa
    kw = dict(scale=scale, causal=causal, window=window, softcap=softcap,
              prefix_lengths=i32(prefixes),
              alibi_slopes=None if alibi is None else torch.tensor(alibi, device=dev),
              key_padding=None if key_padding is None else key_padding.to(dev), dropout=dropout)
    t = {n: (pack_rows(x, lengths) if packed else x).to(dev) for n, x in inp.items()}
    if packed:
        kw.update(cu_seqlens=i32(cumulative(lengths)), max_seqlen=N)
    else:
        kw["seq_lengths"] = i32(lengths)
    res = fa.attention_forward(t["q"], t["k"], t["v"], keep_residual=residual, **kw)
    o, lse = res[:2]
    dq, dk, dv = fa.attention_backward(t["q"], t["k"], t["v"], o, lse, t["do"],
                                       o_low=res[2] if residual else None, **kw)
    torch.cuda.synchronize()
    assert fa.fa_debug_status() == 0
    out = dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)
    if packed:
        c = cumulative(lengths)
        full = {}
        for n, x in out.items():
            y = torch.full((B, H, N), float("-inf")) if n == "lse" else torch.zeros(B, H, N, d)
            for b, L in enumerate(lengths):
                y[b, :, :L] = (x[:, c[b]:c[b] + L] if n == "lse"
                               else x[c[b]:c[b] + L].transpose(0, 1)).float().cpu()
            full[n] = y
        out = full
    return {n: x.float().cpu() for n, x in out.items()}


def errors(inp, out, scale, causal, window=(-1, -1), softcap=0.0, prefixes=None, lengths=None,
           alibi=None, key_padding=None, dropout=None):
    f = {n: synth.to_f64(x) for n, x in inp.items()}
    N = inp["q"].shape[2]
    clip = lambda x: None if x is None else np.clip(x, 0, N)  # noqa
    kp = None if key_padding is None else key_padding.numpy().astype(np.uint8)
    kw = dict(alibi=alibi, key_padding=kp, dropout=dropout, lengths=clip(lengths),
              softcap=softcap, prefixes=clip(prefixes))
    o, lse = oracle.fwd(f["q"], f["k"], f["v"], scale, causal, window, **kw)
    g = oracle.bwd(f["q"], f["k"], f["v"], f["do"], scale, causal, window, **kw)
    got = {n: x.double().numpy() for n, x in out.items()}
    dead = np.isneginf(lse)
    assert np.array_equal(np.isneginf(got["lse"]), dead)
    assert (got["o"][dead] == 0).all() and (got["dq"][dead] == 0).all()
    e = {"o": rel_frob(got["o"], o),
         "lse": float(np.abs(got["lse"][~dead] - lse[~dead]).max()) if (~dead).any() else 0.0}
    for n, r in zip(("dq", "dk", "dv"), g):
        e[n] = rel_frob(got[n], r)
    return e


def check(inp, scale, causal, window=(-1, -1), packed=False, residual=True, **kw):
    out = run(inp, scale, causal, window, packed=packed, residual=residual, **kw)
    assert_within_bounds(errors(inp, out, scale, causal, window, **kw), (causal, window, kw))
    return out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N", [2, 17, 128, 129, 300])
@pytest.mark.parametrize("causal,window", [(False, (-1, -1)), (True, (-1, -1)),
                                           (False, (40, 11)), (True, (33, 0))])
@pytest.mark.parametrize("cap", [50.0, 2.0])
def test_cap(d, N, causal, window, cap):
    check(inputs(2, 2, N, d, N, spread=2.0), 0.125, causal, window, softcap=cap)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.05, 0.5, 7.0, 55.0, 60.0, 300.0, 2000.0])
def test_cap_sizes(d, cap):
    """From caps that hold every score to caps that hold none, rows on either side of the
    polynomial's range in one warp."""
    inp = inputs(1, 2, 200, d, 3, spread=3.0)
    inp["q"][:, :, ::7] *= 5
    check(inp, 0.2, False, softcap=cap)


@pytest.mark.parametrize("d", [64, 128])
def test_saturated_scores(d):
    """Scores far past the cap: finite outputs, and gradients of exactly zero where 1 - tanh^2
    rounds to zero."""
    inp = inputs(1, 1, 130, d, 5)
    inp["q"] = torch.full_like(inp["q"], 64.0)
    inp["k"] = torch.full_like(inp["k"], 64.0)
    inp["k"][:, :, ::2] *= -1
    out = run(inp, 1.0, False, softcap=3.0)
    f = {n: synth.to_f64(x) for n, x in inp.items()}
    o, lse = oracle.fwd(f["q"], f["k"], f["v"], 1.0, softcap=3.0)
    assert rel_frob(out["o"].double().numpy(), o) < 5e-3
    assert np.abs(out["lse"].double().numpy() - lse).max() < 1e-3
    assert (out["dq"] == 0).all() and (out["dk"] == 0).all()


@pytest.mark.parametrize("d", [64, 128])
def test_large_cap_beside_saturated_scores(d):
    """Rows whose scores reach a large cap do not cost the other rows of their warp accuracy:
    scores the polynomials cover keep a relative error of 4e-7, here below 1e-5 in the exponent of
    rows whose scores stay below 25, so for them the bounds of the plain attention hold. (The
    saturated rows have scores near 6e4, where fp32 itself steps by 2^-8: LSE is held to two steps
    there, and their dO is zero, which leaves their weights out of the gradients.)"""
    inp = inputs(1, 2, 300, d, 8)
    even = inp["q"][..., ::2].clone()
    inp["q"][..., 1::2] = -even            # scores of 0 against key 0, but for every 50th row
    inp["k"][:, :, 0] = 96.0
    inp["q"][:, :, ::50] = 96.0 * (64 / d)
    inp["do"][:, :, ::50] = 0.0
    out = run(inp, 0.125, False, softcap=1e5)
    f = {n: synth.to_f64(x) for n, x in inp.items()}
    lse = oracle.fwd(f["q"], f["k"], f["v"], 0.125, softcap=1e5)[1][:, :, ::50]
    assert (lse > 5e4).all()
    assert np.abs(out["lse"][:, :, ::50].double().numpy() - lse).max() <= 2.0 ** -7
    out["lse"][:, :, ::50] = torch.from_numpy(lse).float()
    e = errors(inp, out, 0.125, False, softcap=1e5)
    e["lse"] = float(np.abs(out["lse"].double().numpy() - oracle.fwd(
        f["q"], f["k"], f["v"], 0.125, softcap=1e5)[1])[:, :, np.arange(300) % 50 != 0].max())
    assert_within_bounds(e)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [55.0, 56.0])
def test_bounded_and_unbounded_maxima(d, cap):
    """The forward keeps no running maximum up to a cap of 55 (c log2 e <= 80): rows whose scores
    all lie at -c, all at +c, mixed and ordinary ones, with large and tiny values."""
    g = torch.Generator().manual_seed(6)
    B, H, N = 1, 2, 300
    inp = inputs(B, H, N, d, 17)
    inp["k"][..., 0] = 64.0
    inp["q"][:, :, 0::4, 0] = -640.0   # every score at -c
    inp["q"][:, :, 1::4, 0] = 640.0    # every score at +c
    inp["k"][:, 1, ::2, 0] = -64.0     # the second head: half at either end
    for big in (1e4, 1e-6):
        inp["v"] = (big * torch.randn(B, H, N, d, generator=g)).to(BF16)
        out = run(inp, 1.0 / d ** 0.5, False, softcap=cap)
        f = {n: synth.to_f64(x) for n, x in inp.items()}
        o, lse = oracle.fwd(f["q"], f["k"], f["v"], 1.0 / d ** 0.5, softcap=cap)
        for r in range(4):
            assert rel_frob(out["o"].double().numpy()[:, :, r::4], o[:, :, r::4]) < 5e-3
        assert np.abs(out["lse"].double().numpy() - lse).max() < 1e-3
        assert all(torch.isfinite(out[n]).all() for n in ("dq", "dk", "dv"))


def extreme_rows(B, H, N, d, seed):
    """Queries and keys whose scores reach the cap: rows with every score at -c, every one at +c, and
    ordinary ones; in odd heads half of the keys at either end."""
    inp = inputs(B, H, N, d, seed)
    inp["k"][..., 0] = 64.0
    inp["q"][:, :, 0::4, 0] = -640.0
    inp["q"][:, :, 1::4, 0] = 640.0
    inp["k"][:, 1::2, ::2, 0] = -64.0
    return inp


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [55.0, 50.0, 20.0])
@pytest.mark.parametrize("B,H,N,mode", [(1, 2, 300, m) for m in (
    "full", "causal", "window", "pad", "dropout", "padded", "packed")] + [
        (2, 40, 300, m) for m in ("full", "causal", "packed")])
def test_values_of_any_size(d, cap, B, H, N, mode):
    """Sums of the forward that keeps no maximum leave fp32's range against such V and are formed
    again: query tiles shared by two streams, and one each. The weights of those rows are fp32, so
    with the residual O is exact to fp32: scores of a few units carry 64 roundings of 2^-24, 4e-5
    in a weight, and the residual's own rounding 2^-17: 1e-4 in all, asked of the rows whose
    weights are all 2^(c log2 e) and overflow for certain. Other rows may be of the tensor core's
    bf16 weights: the plain bound."""
    inp = extreme_rows(B, H, N, d, 21)
    dev = torch.device("cuda:0")
    lens = [N, 140][:B] if mode in ("padded", "packed") else None
    if lens and B == 1:
        lens = [211]
    kw = dict(causal=mode != "full", window=(70, 0) if mode == "window" else (-1, -1))
    okw = dict(alibi=None, key_padding=None, dropout=None, lengths=lens, softcap=cap)
    call = dict(softcap=cap, keep_residual=True)
    if mode == "causal":
        pre = [100, 0][:B]
        okw["prefixes"] = pre
        call["prefix_lengths"] = torch.tensor(pre, dtype=torch.int32, device=dev)
    if mode == "pad":
        pad = torch.zeros(B, N, dtype=torch.bool)
        pad[0, :5] = pad[0, 60:130] = True
        okw["key_padding"] = pad.numpy().astype(np.uint8)
        call["key_padding"] = pad.to(dev)
    if mode == "dropout":
        okw["dropout"] = call["dropout"] = (0.3, 11, 5)
    if mode == "padded":
        call["seq_lengths"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if mode == "packed":
        call.update(cu_seqlens=torch.tensor(cumulative(lens), dtype=torch.int32, device=dev),
                    max_seqlen=N)
    put = lambda x: (pack_rows(x, lens) if mode == "packed" else x).to(dev)  # noqa
    g = torch.Generator().manual_seed(9)
    sign = torch.where(torch.rand(B, H, N, d, generator=g) < 0.5, -1.0, 1.0)
    heads = [0, 1] if H <= 2 else [0, 1, H - 1]
    for size in (3e38, 1e25, 1e15, 1e-30):
        v = (size * (0.5 + 0.5 * torch.rand(B, H, N, d, generator=g)) * sign).to(BF16)
        o, lse, low = fa.attention_forward(put(inp["q"]), put(inp["k"]), put(v), 1.0 / d ** 0.5,
                                           **kw, **call)
        torch.cuda.synchronize()
        assert fa.fa_debug_status() == 0
        f = [synth.to_f64(x[:, heads]) if mode != "dropout" else synth.to_f64(x)
             for x in (inp["q"], inp["k"], v)]
        ref, ref_lse = oracle.fwd(*f, 1.0 / d ** 0.5, kw["causal"], kw["window"], **okw)
        got = o.double().cpu() + low.double().cpu()
        o, lse = o.double().cpu(), lse.double().cpu()
        if mode == "packed":
            c = cumulative(lens)
            full = [torch.zeros(B, H, N, d, dtype=torch.float64) for _ in range(2)]
            for b, L in enumerate(lens):
                for t, x in zip(full, (o, got)):
                    t[b, :, :L] = x[c[b]:c[b] + L].transpose(0, 1)
            o, got = full
            t = torch.full((B, H, N), float("-inf"), dtype=torch.float64)
            for b, L in enumerate(lens):
                t[b, :, :L] = lse[:, c[b]:c[b] + L]
            lse = t
        o, got, lse = (x[:, heads].numpy() if mode != "dropout" else x.numpy()
                       for x in (o, got, lse))
        # (dropout scales kept weights up: what lies past bf16's largest value, 3.39e38, is
        # infinite; within 2^-7 of it, the bf16 weights' error and the rounding, it may be either)
        past = np.abs(ref) > 3.39e38 * (1 - 2.0 ** -7)
        sure = np.abs(ref) > 3.39e38 * (1 + 2.0 ** -7)
        assert (o[sure] == np.sign(ref[sure]) * np.inf).all() and not (past.any() and size < 3e38)
        for x in (o, got, ref):
            x[past] = 0.0
        for r in range(4):
            assert rel_frob(o[:, :, r::4] / size, ref[:, :, r::4] / size) < 5e-3, (size, r)
        dead = np.isneginf(ref_lse)
        assert np.array_equal(np.isneginf(lse), dead) and (o[dead] == 0).all()
        assert np.abs(lse[~dead] - ref_lse[~dead]).max() < 1e-3
        if size >= 1e25 and cap >= 50:
            assert rel_frob(got[:, ::2, 1::4] / size, ref[:, ::2, 1::4] / size) < 1e-4, size


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,size", [(98304, 2e38), (98304, 1e30), (98305, 1e30)])
def test_values_of_any_size_in_long_sequences(d, N, size):
    """The longest sequence without a running maximum, its rows' sums past fp32's range, and the
    next one, with a maximum: with V the same for all keys O is V, up to the rounding of O and, with
    a maximum, the 2^-8 of each bf16 weight. (A running maximum lags by up to 2^8, so its sums reach
    2^8 N max|V|: 4e37 here, where values of 2e38 would pass fp32's 3.4e38 in any such kernel.
    Without one they reach 2^72 N max|V|.)"""
    dev = torch.device("cuda:0")
    g = torch.Generator().manual_seed(31)
    q, k = (torch.randn(1, 1, N, d, generator=g).to(dev) for _ in range(2))
    row = (size * (1 + 0.5 * torch.rand(d, generator=g))).to(BF16).to(dev)
    v = row.expand(1, 1, N, d).contiguous()
    o, lse = fa.attention_forward((30 * q).to(BF16), k.to(BF16), v, causal=True, softcap=50.0)
    torch.cuda.synchronize()
    assert fa.fa_debug_status() == 0 and torch.isfinite(lse).all()
    assert ((o.double() / row.double() - 1).abs() <= 2.0 ** -7).all()


@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_in_masked_places(d):
    """A value that is infinite, or not a number, reaches the rows that see its key alone."""
    dev = torch.device("cuda:0")
    inp = inputs(1, 2, 300, d, 23)
    inp["v"][0, 0, 200, 3] = float("inf")
    inp["v"][0, 0, 201, 4] = float("nan")
    o, lse = fa.attention_forward(*(inp[n].to(dev) for n in "qkv"), 0.125, True, softcap=30.0)
    f = {n: synth.to_f64(x) for n, x in inp.items()}
    f["v"][0, 0, 200, 3] = f["v"][0, 0, 201, 4] = 0.0
    ref, ref_lse = oracle.fwd(f["q"], f["k"], f["v"], 0.125, True, softcap=30.0)
    o = o.double().cpu().numpy()
    assert np.abs(lse.double().cpu().numpy() - ref_lse).max() < 1e-3
    assert np.isposinf(o[0, 0, 200:, 3]).all() and np.isnan(o[0, 0, 201:, 4]).all()
    o[0, 0, 200:, 3] = ref[0, 0, 200:, 3]
    o[0, 0, 201:, 4] = ref[0, 0, 201:, 4]
    assert np.isfinite(o).all() and rel_frob(o, ref) < 5e-3
    assert rel_frob(o[0, 0, :200], ref[0, 0, :200]) < 5e-3


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kw", [dict(), dict(softcap=20.0), dict(softcap=60.0), dict(prefix=9),
                                dict(softcap=20.0, dropout=(0.5, 3, 1)), dict(alibi=True)])
def test_rows_that_are_no_numbers(d, kw):
    """A query that is NaN gives an O and an LSE that are, not the LSE of a row without visible
    keys; the other rows do not notice, and a row whose keys are all padded keeps O = 0 and
    LSE = -inf."""
    kw = dict(kw)
    dev = torch.device("cuda:0")
    B, H, N = 2, 2, 300
    q, k, v = (torch.randn(B, H, N, d, device=dev).to(BF16) for _ in range(3))
    bad = q.clone()
    rows = [0, 5, 127, 128, 299]
    bad[1, :, rows] = float("nan")
    call = dict(causal=True)
    if "prefix" in kw:
        call["prefix_lengths"] = torch.tensor([kw.pop("prefix")] * B, dtype=torch.int32, device=dev)
    if kw.pop("alibi", False):
        call["alibi_slopes"] = torch.full((H,), 0.1, device=dev)
    pad = torch.zeros(B, N, dtype=torch.bool, device=dev)
    pad[0, :10] = True
    call.update(key_padding=pad, **kw)
    a, b = (fa.attention_forward(t, k, v, **call) for t in (q, bad))
    assert torch.isnan(b[1][1][:, rows]).all()
    assert torch.isnan(b[0][1][:, rows]).all()
    ok = torch.ones(B, H, N, dtype=torch.bool, device=dev)
    ok[1, :, rows] = False
    assert torch.equal(a[1][ok], b[1][ok]) and torch.equal(a[0][ok], b[0][ok])
    if "prefix_lengths" not in call:
        assert torch.isneginf(b[1][0, :, :10]).all() and (b[0][0, :, :10] == 0).all()
    torch.cuda.synchronize()
    assert fa.fa_debug_status() == 0


def test_e4m3_rows_that_are_no_numbers():
    dev = torch.device("cuda:0")
    q, k, v = (torch.randn(2, 2, 300, 128, device=dev) for _ in range(3))
    bad = q.clone()
    rows = [0, 5, 127, 128, 299]
    bad[1, :, rows] = float("nan")
    q, k, v, bad = (t.to(torch.float8_e4m3fn) for t in (q, k, v, bad))
    a, b = (fa.attention_forward_fp8(t, k, v, causal=True) for t in (q, bad))
    assert torch.isnan(b[1][1][:, rows]).all() and torch.isnan(b[0][1][:, rows]).all()
    ok = torch.ones(2, 2, 300, dtype=torch.bool, device=dev)
    ok[1, :, rows] = False
    assert torch.equal(a[1][ok], b[1][ok]) and torch.equal(a[0][ok], b[0][ok])


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("cap", [0.0, 10.0])
@pytest.mark.parametrize("N", [1, 127, 128, 129, 500])
def test_prefix(d, cap, N):
    pre = [0, 1, N // 2, N - 1, N, N + 50, -3, 128]
    if N == 1:  # one key: its gradients with respect to q and k are zero
        out = run(inputs(8, 1, 1, d), 0.125, True, softcap=cap, prefixes=pre)
        assert np.abs(out["dq"].numpy()).max() < 1e-3
        assert np.abs(out["o"].numpy() - inputs(8, 1, 1, d)["v"].float().numpy()).max() < 1e-6
        return
    check(inputs(8, 1, N, d, N), 0.125, True, softcap=cap, prefixes=pre)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("cap", [0.0, 10.0])
def test_prefix_lengths(d, packed, cap):
    lens = [300, 0, 1, 129, 255, 256]
    pre = [140, 5, 1, 300, 0, 200]
    check(inputs(6, 2, 300, d, 9), 0.125, True, packed=packed, softcap=cap, prefixes=pre,
          lengths=lens)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("packed", [False, True])
def test_every_option_at_once(d, packed):
    B, H, N = 4, 3, 270
    lens = [270, 64, 200, 129]
    g = torch.Generator().manual_seed(3)
    pad = torch.rand(B, N, generator=g) < 0.2
    pad[1] = True  # an entry without a visible key
    kw = dict(prefixes=[100, 64, 0, 129], lengths=lens, key_padding=pad, dropout=(0.2, 1234, 5))
    inp = inputs(B, H, N, d, 11, spread=2.0)
    check(inp, 0.125, True, packed=packed, softcap=5.0, alibi=[0.5, 0.1, 0.02], **kw)
    check(inp, 0.125, True, packed=packed, softcap=5.0, **kw)
    check(inp, 0.125, True, packed=packed, softcap=70.0, **kw)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("opt", ["alibi", "pad", "dropout"])
def test_each_option(d, opt):
    g = torch.Generator().manual_seed(4)
    kw = {"alibi": dict(alibi=[0.3, 0.01]), "pad": dict(key_padding=torch.rand(2, 260,
                                                                              generator=g) < 0.4),
          "dropout": dict(dropout=(0.1, 77, 1))}[opt]
    inp = inputs(2, 2, 260, d, 12, spread=2.0)
    check(inp, 0.125, False, softcap=8.0, **kw)
    check(inp, 0.125, True, softcap=8.0, prefixes=[130, 31], residual=False, **kw)


@pytest.mark.parametrize("d", [64, 128])
def test_many_items_per_sm(d):
    """More tiles than SMs, with even and odd tile counts (the paired and chunked schedules);
    sampled heads against the oracle."""
    for N in (1024, 900):
        B, H = 6, 8
        inp = inputs(B, H, N, d, 13)
        pre = [0, 1000, 129, 512, 700, 3]
        out = run(inp, 0.125, True, softcap=6.0, prefixes=pre)
        for b, h in ((0, 0), (1, 3), (3, 5), (5, 7)):
            one = {n: x[b:b + 1, h:h + 1] for n, x in inp.items()}
            got = {n: x[b:b + 1, h:h + 1] for n, x in out.items()}
            assert_within_bounds(errors(one, got, 0.125, True, softcap=6.0, prefixes=[pre[b]]),
                                 (N, b, h))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,lens", [(129, None), (1000, None), (700, [700, 0, 1, 128, 129, 300])])
@pytest.mark.parametrize("packed", [False, True])
def test_key_tiles_shared_by_two_streams(d, N, lens, packed):
    """Few query tiles: a query tile's key tiles go to the block's two streams in turn, an odd and
    an even number of them, one tile, and items of one and of several tiles on one SM."""
    B = 6 if lens else 2
    if packed and not lens:
        lens = [N] * B
    kw = dict(softcap=12.0, lengths=lens)
    inp = inputs(B, 3, N, d, 31, spread=2.0)
    pre = [(5 * N) // 7 if b % 2 else 3 for b in range(B)]
    check(inp, 0.125, True, packed=packed, prefixes=pre, **kw)
    check(inp, 0.125, False, packed=packed, **kw)
    check(inp, 0.125, False, (150, 60), packed=packed, **kw)


@pytest.mark.parametrize("N", [256, 5000])
def test_timeout_is_reported(N):
    """The capped kernels' waits are bounded too (the hook skips every V tile): two streams on one
    query tile, and on one each."""
    dev = torch.device("cuda:0")
    q = torch.randn(1, 4 if N > 256 else 1, N, 64, device=dev).to(BF16)
    fa.fa_debug_set_fault(1)
    try:
        fa.attention_forward(q, q, q, 0.125, True, softcap=5.0)
        status = fa.fa_debug_status()
    finally:
        fa.fa_debug_set_fault(0)
    assert status == 6 and fa.fa_debug_status() == 0
    a = fa.attention_forward(q, q, q, 0.125, True, softcap=5.0)
    b = fa.attention_forward(q, q, q, 0.125, True, softcap=5.0)
    assert fa.fa_debug_status() == 0 and all(torch.equal(x, y) for x, y in zip(a, b))


def test_no_cap_and_no_prefix_is_the_plain_call():
    dev = torch.device("cuda:0")
    inp = inputs(2, 2, 200, 64)
    q, k, v = (inp[n].to(dev) for n in "qkv")
    a = fa.attention_forward(q, k, v, causal=True)
    b = fa.attention_forward(q, k, v, causal=True, softcap=0.0, prefix_lengths=None)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    # prefixes of no keys: the causal result, through the other kernels
    z = torch.zeros(2, dtype=torch.int32, device=dev)
    c = fa.attention_forward(q, k, v, causal=True, prefix_lengths=z)
    assert all(torch.equal(x, y) for x, y in zip(a, c))


def test_packed_equals_padded():
    lens, pre = [130, 70, 256], [60, 70, 0]
    inp = inputs(3, 2, 256, 128, 14)
    a = run(inp, 0.1, True, softcap=4.0, prefixes=pre, lengths=lens)
    b = run(inp, 0.1, True, softcap=4.0, prefixes=pre, lengths=lens, packed=True)
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_repeats_streams_and_graphs():
    dev = torch.device("cuda:0")
    inp = {n: x.to(dev) for n, x in inputs(2, 4, 700, 64, 15).items()}
    pre = torch.tensor([300, 0], dtype=torch.int32, device=dev)
    kw = dict(causal=True, softcap=9.0, prefix_lengths=pre)

    def step(stream=None):
        o, lse, low = fa.attention_forward(inp["q"], inp["k"], inp["v"], keep_residual=True,
                                           stream=stream, **kw)
        return (o, lse) + fa.attention_backward(inp["q"], inp["k"], inp["v"], o, lse, inp["do"],
                                                o_low=low, stream=stream, **kw)

    ref = step()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for _ in range(6):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                runs.append(step())
    runs.append(step(s1))
    torch.cuda.synchronize()
    for r in runs:
        assert all(torch.equal(a, b) for a, b in zip(r, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_packed_rows_outside_are_left_alone():
    dev = torch.device("cuda:0")
    total, H, d = 400, 2, 64
    cu = torch.tensor([20, 150, 150, 380], dtype=torch.int32, device=dev)
    pre = torch.tensor([40, 9, 500], dtype=torch.int32, device=dev)
    q, k, v, do = (torch.randn(total, H, d, device=dev).to(BF16) for _ in range(4))
    dims = (3, H, 230, d)
    opt = fa.options(cu_seqlens=cu, total_tokens=total)
    score = fa.fa_score_t(pre.data_ptr(), 7.0)
    o, dq, dk, dv = (torch.full_like(q, 5.0) for _ in range(4))
    lse = torch.full((H, total), 5.0, device=dev)
    ws = torch.empty(fa.fa_bwd_workspace_bytes_ex(*dims, opt), dtype=torch.uint8, device=dev)
    fa.fa_fwd_score(q, k, v, o, lse, opt, score, causal=True, dims=dims)
    fa.fa_bwd_score(q, k, v, o, do, lse, dq, dk, dv, ws, opt, score, causal=True, dims=dims)
    torch.cuda.synchronize()
    assert fa.fa_debug_status() == 0
    for t in (o, dq, dk, dv):
        assert (t[:20] == 5.0).all() and (t[380:] == 5.0).all()
        assert torch.isfinite(t.float()).all() and not (t[20:380] == 5.0).all(-1).any()
    assert (lse[:, :20] == 5.0).all() and (lse[:, 380:] == 5.0).all()


def test_refusals():
    dev = torch.device("cuda:0")
    q = torch.randn(2, 2, 130, 64, device=dev).to(BF16)
    pre = torch.zeros(2, dtype=torch.int32, device=dev)
    for bad in (pre.long(), pre.cpu(), pre[:1], torch.zeros(4, dtype=torch.int32,
                                                            device=dev)[::2]):
        with pytest.raises(ValueError):
            fa.attention_forward(q, q, q, causal=True, prefix_lengths=bad)
    for kw in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
               dict(softcap=1e-44), dict(prefix_lengths=pre),
               dict(prefix_lengths=pre, causal=True, window=(5, 0))):
        with pytest.raises(fa.FAError):
            fa.attention_forward(q, q, q, **kw)
    with pytest.raises(fa.FAError):
        fa.attention_backward(q, q, q, q, torch.zeros(2, 2, 130, device=dev), q, softcap=3.0,
                              fused=True)
    assert ctypes.sizeof(fa.fa_score_t) == 16


@pytest.mark.parametrize("d,interleaved", [(64, False), (128, True)])
@pytest.mark.parametrize("packed", [False, True])
def test_layer(d, interleaved, packed):
    """A layer's path as it is trained: projection -> norm and rotation -> capped attention with
    prefixes -> gradients -> projection, against the same in 64 bits."""
    import rope_ref
    dev = torch.device("cuda:0")
    B, N, H, cap, eps = 3, 200, 2, 6.0, 1e-6
    lens = [200, 77, 130]
    pre = [50, 77, 0]
    g = torch.Generator().manual_seed(21)
    qkv = torch.randn(B, N, 3 * H, d, generator=g).to(BF16)
    do = torch.randn(B, H, N, d, generator=g).to(BF16)
    gains = [1 + 0.2 * torch.randn(d, generator=g) for _ in range(2)]
    freq = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa
    if packed:
        x = torch.cat([qkv[b, :n] for b, n in enumerate(lens)]).to(dev)
        dox = pack_rows(do, lens).to(dev)
        lay = dict(cu_seqlens=i32(cumulative(lens)), max_seqlen=N)
    else:
        x, dox, lay = qkv.to(dev), do.to(dev), dict(seq_lengths=i32(lens))
    rope = dict(q_weight=gains[0].to(dev), k_weight=gains[1].to(dev), eps=eps,
                inv_freq=freq.to(dev), interleaved=interleaved, **lay)
    att = dict(causal=True, softcap=cap, prefix_lengths=i32(pre), **lay)
    xq, xk, xv = x.split(H, -2)
    q, k, v = fa.qk_norm_rope_forward(xq, xk, xv, **rope)
    o, lse, low = fa.attention_forward(q, k, v, keep_residual=True, **att)
    dq, dk, dv = fa.attention_backward(q, k, v, o, lse, dox, o_low=low, **att)
    dx = torch.empty_like(x)
    grads = fa.qk_norm_rope_backward(dq, dk, dv, xq, xk, out=dx.split(H, -2), **rope)
    torch.cuda.synchronize()
    # 64 bits, with Q and K rounded to bf16 where the path rounds them
    f = lambda t: t.double().numpy()  # noqa
    ang = rope_ref.angles(np.arange(N)[None], f(freq), None)
    out = [np.zeros((B, N, H, d)) for _ in range(3)]
    dg = [0.0, 0.0]
    scale = 1 / np.sqrt(d)
    for b, n in enumerate(lens):
        src = [f(t) for t in qkv[b, :n].split(H, 1)]
        y = [rope_ref.forward(src[i], f(gains[i]), ang[:n], interleaved, True, eps)
             for i in range(2)]
        y = [f(torch.tensor(t).to(BF16)).transpose(1, 0, 2)[None] for t in y]
        vv = src[2].transpose(1, 0, 2)[None]
        kw = dict(softcap=cap, prefixes=[min(pre[b], n)])
        gr = oracle.bwd(y[0], y[1], vv, f(do[b:b + 1, :, :n]), scale, True, **kw)
        ro, rl = oracle.fwd(y[0], y[1], vv, scale, True, **kw)
        c = cumulative(lens)[b]
        go = o[c:c + n].transpose(0, 1) if packed else o[b, :, :n]
        assert rel_frob(f(go.cpu()), ro[0]) < 5e-3
        for i in range(2):
            gx, gg, _ = rope_ref.backward(gr[i][0].transpose(1, 0, 2), src[i], f(gains[i]),
                                          ang[:n], interleaved, True, eps)
            out[i][b, :n] = gx
            dg[i] = dg[i] + gg
        out[2][b, :n] = gr[2][0].transpose(1, 0, 2)
    for i, t in enumerate(dx.split(H, -2)):
        t = f(t.cpu())
        if packed:
            full = np.zeros((B, N, H, d))
            for b, n in enumerate(lens):
                full[b, :n] = t[cumulative(lens)[b]:cumulative(lens)[b] + n]
            t = full
        # the attention's gradient is within 1e-2; the norm's and the last rounding add 2^-8
        assert rel_frob(t, out[i]) < 1e-2 + 2.0 ** -8, i
    for i in range(2):
        assert rel_frob(f(grads[3 + i].cpu()), dg[i]) < 1e-2 + 2.0 ** -8
