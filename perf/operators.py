"""Measured calls of the capped and prefix-masked attention and of the per-head norm with rotary
positions that prepares its queries and keys.

Four operators, named by a case's "op":

  attn_fwd    O and LSE of softmax(cap(scale Q K^T) + mask) V with cap(s) = c tanh(s / c) (c = 0: no
              cap) and the mask "key j <= query i, or j < prefix of the sequence"
  attn_train  the same forward, then its gradients dQ, dK, dV
  rope_fwd    Q and K of a fused projection normalised per head, rotated by their positions (one to
              three axes) and laid out, with V, as the attention takes them
  rope_bwd    the gradient of that with respect to the projection and to the two gains

Layouts: "dense" (B, H, N, d); "lengths", the same with a real length per batch entry; "packed",
the sequences back to back as (total, H, d).
"""
import itertools
import math

import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one short request: the call's own latency
        dict(name="attn_fwd_short", op="attn_fwd", layout="dense", B=1, H=2, N=128, d=64,
             cap=50.0, prefix=0, causal=True),
        # prompts with an image or instruction prefix that is seen in both directions, no cap,
        # of uneven lengths in one padded batch
        dict(name="attn_fwd_prefix_lengths", op="attn_fwd", layout="lengths", B=8, H=16, N=1024,
             d=64, cap=0.0, prefix=300, causal=True),
        # a long prompt of odd length
        dict(name="attn_fwd_long_odd", op="attn_fwd", layout="dense", B=1, H=16, N=8111, d=128,
             cap=30.0, prefix=0, causal=True),
        # a small training batch, both directions visible, ragged last tile
        dict(name="attn_train_small", op="attn_train", layout="dense", B=2, H=8, N=1000, d=64,
             cap=20.0, prefix=0, causal=False),
        # packed documents, each with a prefix, capped scores
        dict(name="attn_train_packed_prefix", op="attn_train", layout="packed", B=12, H=16,
             N=2048, d=128, cap=50.0, prefix=500, causal=True),
        # the repository's training workload (batch 32, 16 heads, 2048 tokens), capped
        dict(name="attn_train_batch", op="attn_train", layout="dense", B=32, H=16, N=2048, d=64,
             cap=50.0, prefix=0, causal=True),
        # one new token for each of 48 running requests, at far positions, few key heads
        dict(name="rope_fwd_tokens", op="rope_fwd", layout="dense", B=48, N=1, Hq=32, Hk=8, d=128,
             rot=128, axes=1, interleaved=False, norm=True, far=True),
        # a clip of video patches: time, height and width positions
        dict(name="rope_fwd_video", op="rope_fwd", layout="dense", B=1, N=15600, Hq=24, Hk=24,
             d=128, rot=128, axes=3, interleaved=True, norm=True, far=False),
        # the training workload's projection
        dict(name="rope_fwd_batch", op="rope_fwd", layout="dense", B=32, N=2048, Hq=16, Hk=16,
             d=64, rot=64, axes=1, interleaved=False, norm=True, far=False),
        # packed sequences, partly rotated heads, shared key heads
        dict(name="rope_bwd_packed", op="rope_bwd", layout="packed", B=9, N=700, Hq=12, Hk=4,
             d=64, rot=32, axes=1, interleaved=False, norm=True, far=False),
        # images: two axes, a padded batch of uneven lengths
        dict(name="rope_bwd_images", op="rope_bwd", layout="lengths", B=6, N=4097, Hq=16, Hk=16,
             d=128, rot=128, axes=2, interleaved=True, norm=True, far=False),
        # the training workload's projection
        dict(name="rope_bwd_batch", op="rope_bwd", layout="dense", B=32, N=2048, Hq=16, Hk=16,
             d=64, rot=64, axes=1, interleaved=False, norm=True, far=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_train", "rope_fwd", "rope_bwd"])
    layout = rng.choice(["dense", "lengths", "packed"])
    d = rng.choice([64, 128])
    if op.startswith("attn"):
        # up to 1.5e9 scores (the largest listed case has 2.1e9)
        # (a lone token's gradients with respect to its query and key are zero: from 8 on)
        N = _log_int(rng, 1 if op == "attn_fwd" else 8, 8192)
        B = _log_int(rng, 1, max(1, min(32, 1.5e9 / (N * N))))
        H = _log_int(rng, 1, max(1, min(32, 1.5e9 / (N * N * B))))
        kind = rng.choice(["cap", "prefix", "both", "open"])
        cap = 0.0 if kind == "prefix" else round(math.exp(rng.uniform(math.log(4), math.log(100))), 2)
        prefix = rng.randint(1, N) if kind in ("prefix", "both") else 0
        return dict(op=op, layout=layout, B=B, H=H, N=N, d=d, cap=cap, prefix=prefix,
                    causal=kind != "open")
    # up to 1.9e8 values of a projection (the largest listed case has 2.0e8)
    Hk = rng.choice([1, 2, 3, 4, 5, 8, 16])
    Hq = Hk * rng.choice([1, 2, 3, 4])
    room = 1.9e8 / (d * (Hq + 2 * Hk))
    N = _log_int(rng, 1, min(16384, room))
    B = _log_int(rng, 1, max(1, min(256, room / N)))
    rot = rng.choice([16, 32, 48, 64, d, d])
    return dict(op=op, layout=layout, B=B, N=N, Hq=Hq, Hk=Hk, d=d, rot=rot,
                axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.5,
                norm=rng.random() < 0.8, far=rng.random() < 0.3)


# ------------------------------------------------------------------------------ the inputs
def _lengths(case, seed):
    """Each sequence's real length, at most N, one of them N: the case's lengths in the seed's
    order (a packed batch then has the same number of tokens whatever the seed)."""
    B, N = case["B"], case["N"]
    if case["layout"] == "dense":
        return [N] * B
    g = torch.Generator().manual_seed(1000 * B + N)
    lens = torch.randint(max(1, N // 4), N + 1, (B,), generator=g)
    lens[0] = N
    g = torch.Generator().manual_seed(seed * 7919 + 11)
    return lens[torch.randperm(B, generator=g)].tolist()


def _prefixes(case, seed):
    """Each sequence's prefix: up to the case's, and at times past the sequence's end."""
    g = torch.Generator().manual_seed(seed * 7919 + 23)
    return torch.randint(0, case["prefix"] + 1, (case["B"],), generator=g).tolist()


def _cumulative(lens):
    return list(itertools.accumulate(lens, initial=0))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(seed)
    rand = lambda *shape: torch.randn(*shape, device=dev, generator=g)  # noqa: E731
    lens = _lengths(case, seed)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    B, N, d = case["B"], case["N"], case["d"]
    s = dict(case=case, lens=None, cu=None)
    if case["layout"] == "lengths":
        s["lens"] = i32(lens)
    if case["layout"] == "packed":
        s["cu"] = i32(_cumulative(lens))
    total = sum(lens)
    if case["op"].startswith("attn"):
        shape = (total, case["H"], d) if case["layout"] == "packed" else (B, case["H"], N, d)
        # scores of a trained layer: a standard deviation of about two before the cap
        s["q"] = (2.0 * rand(*shape)).to(BF16)
        s["k"] = rand(*shape).to(BF16)
        s["v"] = rand(*shape).to(BF16)
        if case["op"] == "attn_train":
            s["do"] = rand(*shape).to(BF16)
        s["prefix"] = i32(_prefixes(case, seed)) if case["prefix"] else None
        s["scale"] = 1.0 / math.sqrt(d)
        return s
    Hq, Hk, rot, axes = case["Hq"], case["Hk"], case["rot"], case["axes"]
    tokens = (total,) if case["layout"] == "packed" else (B, N)
    # the fused projection's output, its heads of uneven size
    qkv = rand(*tokens, Hq + 2 * Hk, d) * (0.5 + 2.0 * torch.rand(
        Hq + 2 * Hk, 1, device=dev, generator=g))
    s["qkv"] = qkv.to(BF16)
    s["wq"] = 1.0 + 0.2 * rand(d) if case["norm"] else None
    s["wk"] = 1.0 + 0.2 * rand(d) if case["norm"] else None
    half = rot // 2
    pair = torch.arange(half, device=dev, dtype=torch.float64)
    s["inv_freq"] = (10000.0 ** (-pair / half)).float()
    # pairs dealt to the axes in contiguous sections
    s["pair_axis"] = None
    if axes > 1:
        s["pair_axis"] = (torch.arange(half, device=dev) * axes // half).to(torch.uint8)
    s["positions"] = None
    if axes > 1:
        # a grid of patches: time (or row), height, width
        n = torch.arange(tokens[-1], device=dev)
        grid = torch.stack([n // 1560, n // 52 % 30, n % 52][3 - axes:])
        grid = grid if len(tokens) == 1 else grid[:, None].expand(axes, B, N)
        s["positions"] = grid.to(torch.int32).contiguous()
    elif case["far"]:
        # continued sequences: the positions start far from zero
        p = torch.randint(0, 131072, tokens, device=dev, generator=g, dtype=torch.int32)
        s["positions"] = p[None].contiguous()
    if case["op"] == "rope_bwd":
        out = (lambda h: (total, h, d)) if case["layout"] == "packed" else (lambda h: (B, h, N, d))
        s["dq"], s["dk"], s["dv"] = (rand(*out(h)).to(BF16) for h in (Hq, Hk, Hk))
    return s


def work(case):
    d, op = case["d"], case["op"]
    lens = _lengths(case, 0)
    if op.startswith("attn"):
        pre = _prefixes(case, 0) if case["prefix"] else [0] * case["B"]
        pairs = rows = 0
        for n, p in zip(lens, pre):
            rows += n
            p = min(p, n)
            pairs += n * (n + 1) // 2 + p * (p - 1) // 2 if case["causal"] else n * n
        H = case["H"]
        # forward: Q K^T, P V; gradients: Q K^T again, dO V^T, P^T dO, dS K, dS^T Q
        flops = 4 * d * pairs * H
        data = 4 * rows * H * d * 2 + 4 * rows * H
        if op == "attn_train":
            flops += 10 * d * pairs * H
            data += 4 * rows * H * d * 2
        return {"bytes": data, "flops": flops}
    tokens = sum(lens)
    heads = case["Hq"] + 2 * case["Hk"]
    rows = tokens * heads
    # forward: each head read and written once; gradient: the incoming one and the normalised
    # heads' inputs read, the projection's written
    data = 2 * rows * d * 2
    if op == "rope_bwd" and case["norm"]:
        data += tokens * (case["Hq"] + case["Hk"]) * d * 2
    return {"bytes": data, "flops": (8 if op == "rope_fwd" else 16) * rows * d}


# ------------------------------------------------------------------------------ plain forms
def _rows_of(s):
    """(sequence, place) of each token of a packed batch."""
    cu = s["cu"].long()
    total = s["q"].shape[0] if "q" in s else s["qkv"].shape[0]
    tok = torch.arange(total, device=cu.device)
    b = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    return b, tok - cu[b]


def _unpack(t, b, n, B, N):
    """(total, H, d) -> (B, H, N, d) in 32 bits, zero where no token is."""
    out = torch.zeros(B, N, *t.shape[1:], device=t.device)
    out[b, n] = t.float()
    return out.transpose(1, 2)


def _visible(s):
    """(B or 1, 1, N, N): which keys each query sees."""
    case, dev = s["case"], s["q"].device
    N = case["N"]
    n = torch.arange(N, device=dev)
    i, j = n[:, None], n[None, :]
    vis = torch.ones(1, 1, N, N, dtype=torch.bool, device=dev)
    if case["causal"]:
        vis = vis & (j <= i)
        if s["prefix"] is not None:
            vis = vis | (j < s["prefix"][:, None, None, None])
    lens = s["lens"] if s["cu"] is None else s["cu"][1:] - s["cu"][:-1]
    if lens is not None:
        live = n < lens[:, None]
        vis = vis & live[:, None, :, None] & live[:, None, None, :]
    return vis


def _attention(s, train):
    case = s["case"]
    B, N, cap = case["B"], case["N"], case["cap"]
    packed = s["cu"] is not None
    if packed:
        b, n = _rows_of(s)
        load = lambda t: _unpack(t, b, n, B, N)  # noqa: E731
        store = lambda t: t.transpose(1, 2)[b, n].to(BF16)  # noqa: E731
    else:
        load, store = (lambda t: t.float()), (lambda t: t.to(BF16))
    q, k, v = load(s["q"]), load(s["k"]), load(s["v"])
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"])
    if cap:
        x = x.div_(cap).tanh_().mul_(cap)
    vis = _visible(s)
    m = x.masked_fill(~vis, -math.inf).amax(3, keepdim=True)
    m = m.masked_fill(m == -math.inf, 0.0)
    p = torch.exp(x - m).masked_fill_(~vis, 0.0)
    l = p.sum(3, keepdim=True)
    lse = (m + torch.log(l)).squeeze(3)
    p = p.div_(l.masked_fill(l == 0.0, 1.0))
    o = torch.matmul(p, v)
    out = {"o": store(o), "lse": lse.transpose(1, 2)[b, n].t().contiguous() if packed else lse}
    if not train:
        return out
    do = load(s["do"])
    out["dv"] = store(torch.matmul(p.transpose(2, 3), do))
    ds = torch.matmul(do, v.transpose(2, 3)).sub_((do * o).sum(3, keepdim=True)).mul_(p)
    if cap:
        ds = ds.mul_(x.div_(cap).square_().neg_().add_(1.0))
    out["dq"] = store(torch.matmul(ds, k) * s["scale"])
    out["dk"] = store(torch.matmul(ds.transpose(2, 3), q) * s["scale"])
    return out


def _angles(s):
    """cos and sin of every token's pairs, (tokens..., 1, rot / 2) in 32 bits."""
    qkv = s["qkv"]
    if s["positions"] is None:
        if s["cu"] is None:
            pos = torch.arange(qkv.shape[1], device=qkv.device).expand(qkv.shape[:2])
        else:
            pos = _rows_of(s)[1]
        pos = pos[None]
    else:
        pos = s["positions"]
    axis = s["pair_axis"].long() if s["pair_axis"] is not None else torch.zeros_like(
        s["inv_freq"]).long()
    a = pos.double()[axis].movedim(0, -1) * s["inv_freq"].double()
    return torch.cos(a).float().unsqueeze(-2), torch.sin(a).float().unsqueeze(-2)


def _pairs(x, case):
    """The two members of each rotated pair, and what is not rotated."""
    rot = case["rot"]
    r, rest = x[..., :rot], x[..., rot:]
    if case["interleaved"]:
        return r[..., 0::2], r[..., 1::2], rest
    return r[..., :rot // 2], r[..., rot // 2:], rest


def _join(a, b, rest, case):
    r = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([r, rest], -1)


def _dead(s):
    """(B, N) of a padded batch's tokens past their sequence's real length, or None."""
    if s["lens"] is None:
        return None
    return torch.arange(s["case"]["N"], device=s["lens"].device) >= s["lens"][:, None]


EPS = 1e-6


def _rope_forward(s):
    case, qkv = s["case"], s["qkv"]
    Hq, Hk = case["Hq"], case["Hk"]
    cos, sin = _angles(s)
    dead = _dead(s)

    def lay(x):
        if dead is not None:
            x = x.masked_fill(dead[:, :, None, None], 0.0)
        return (x if s["cu"] is not None else x.transpose(1, 2)).to(BF16).contiguous()

    def turn(x, w):
        x = x.float()
        if case["norm"]:
            x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
        a, b, rest = _pairs(x, case)
        return lay(_join(a * cos - b * sin, b * cos + a * sin, rest, case))

    return {"q": turn(qkv[..., :Hq, :], s["wq"]), "k": turn(qkv[..., Hq:Hq + Hk, :], s["wk"]),
            "v": lay(qkv[..., Hq + Hk:, :])}


def _rope_backward(s):
    case, qkv = s["case"], s["qkv"]
    Hq, Hk = case["Hq"], case["Hk"]
    cos, sin = _angles(s)
    dead = _dead(s)

    def token_major(t):
        t = (t if s["cu"] is not None else t.transpose(1, 2)).float()
        return t if dead is None else t.masked_fill(dead[:, :, None, None], 0.0)

    def back(dy, x, w):
        a, b, rest = _pairs(token_major(dy), case)
        g = _join(a * cos + b * sin, b * cos - a * sin, rest, case)
        if not case["norm"]:
            return g, None
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        xh = x * r
        gw = (g * xh).flatten(0, -2).sum(0)
        g = g * w
        return r * (g - xh * (g * xh).mean(-1, keepdim=True)), gw

    gq, gwq = back(s["dq"], qkv[..., :Hq, :], s["wq"])
    gk, gwk = back(s["dk"], qkv[..., Hq:Hq + Hk, :], s["wk"])
    out = {"dqkv": torch.cat([gq, gk, token_major(s["dv"])], -2).to(BF16)}
    if case["norm"]:
        out.update(dwq=gwq, dwk=gwk)
    return out


# ------------------------------------------------------------------------------ one pass
def _run_own(s):
    from exact_attention_126_b200 import fa
    case = s["case"]
    op = case["op"]
    if op.startswith("attn"):
        kw = dict(scale=s["scale"], causal=case["causal"], softcap=case["cap"],
                  prefix_lengths=s["prefix"], seq_lengths=s["lens"], cu_seqlens=s["cu"],
                  max_seqlen=case["N"] if s["cu"] is not None else None)
        if op == "attn_fwd":
            o, lse = fa.attention_forward(s["q"], s["k"], s["v"], **kw)
            return {"o": o, "lse": lse}
        o, lse, low = fa.attention_forward(s["q"], s["k"], s["v"], keep_residual=True, **kw)
        dq, dk, dv = fa.attention_backward(s["q"], s["k"], s["v"], o, lse, s["do"], o_low=low,
                                           **kw)
        return {"o": o, "lse": lse, "dv": dv, "dq": dq, "dk": dk}
    Hq, Hk, qkv = case["Hq"], case["Hk"], s["qkv"]
    q, k, v = qkv[..., :Hq, :], qkv[..., Hq:Hq + Hk, :], qkv[..., Hq + Hk:, :]
    kw = dict(q_weight=s["wq"], k_weight=s["wk"], eps=EPS, norm=case["norm"],
              inv_freq=s["inv_freq"], positions=s["positions"], pair_axis=s["pair_axis"],
              interleaved=case["interleaved"], seq_lengths=s["lens"], cu_seqlens=s["cu"],
              max_seqlen=case["N"] if s["cu"] is not None else None)
    if op == "rope_fwd":
        q, k, v = fa.qk_norm_rope_forward(q, k, v, **kw)
        return {"q": q, "k": k, "v": v}
    # the gradients go straight into the fused projection's
    dqkv = torch.empty_like(qkv)
    out = (dqkv[..., :Hq, :], dqkv[..., Hq:Hq + Hk, :], dqkv[..., Hq + Hk:, :])
    grads = fa.qk_norm_rope_backward(s["dq"], s["dk"], s["dv"], q, k, out=out, **kw)
    res = {"dqkv": dqkv}
    if case["norm"]:
        res.update(dwq=grads[3], dwk=grads[4])
    return res


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "rope_fwd":
        return _rope_forward(state)
    if op == "rope_bwd":
        return _rope_backward(state)
    return _attention(state, op == "attn_train")


# ------------------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    """The definitions, one sequence (and head) at a time."""
    s = prepare(case, seed)
    lens = _lengths(case, seed)
    B, N, d, op = case["B"], case["N"], case["d"], case["op"]
    packed = case["layout"] == "packed"
    start = _cumulative(lens)
    f64 = torch.float64
    dev = torch.device("cuda")
    if op.startswith("attn"):
        pre = _prefixes(case, seed) if case["prefix"] else [0] * B
        H, c = case["H"], case["cap"]
        # the mean cost of a 64-bit score, over all of a pass
        if sum(n * n for n in lens) * H * d * (14 if op == "attn_train" else 4) > 2e14:
            return None
        names = ["o", "lse"] + (["dv", "dq", "dk"] if op == "attn_train" else [])
        out = {n: torch.zeros(s["q"].shape, dtype=f64, device=dev) for n in names if n != "lse"}
        out["lse"] = torch.full((H, s["q"].shape[0]) if packed else (B, H, N), -math.inf,
                                dtype=f64, device=dev)
        out = {n: out[n] for n in names}
        for b in range(B):
            n = lens[b]
            at = slice(start[b], start[b] + n)
            place = torch.arange(n, device=dev)
            see = place[None, :] <= place[:, None]
            see |= (place < pre[b])[None, :]
            for h in range(H):
                # (index of the rows, index of their LSE)
                ix, il = ((at, h), (h, at)) if packed else ((b, h, slice(n)), (b, h, slice(n)))
                q, k, v = s["q"][ix].to(f64), s["k"][ix].to(f64), s["v"][ix].to(f64)
                y = (q @ k.T) * s["scale"]
                slope = None
                if c:
                    t = torch.tanh(y / c)
                    y, slope = c * t, 1 - t * t
                if case["causal"]:
                    y = torch.where(see, y, -math.inf)
                lse = torch.logsumexp(y, 1)
                p = torch.exp(y - lse[:, None])
                out["lse"][il] = lse
                o = p @ v
                out["o"][ix] = o
                if op == "attn_train":
                    do = s["do"][ix].to(f64)
                    out["dv"][ix] = p.T @ do
                    g = p * (do @ v.T - (do * o).sum(1)[:, None])
                    if slope is not None:
                        g = g * slope
                    out["dq"][ix] = g @ k * s["scale"]
                    out["dk"][ix] = g.T @ q * s["scale"]
        return out
    # the rotation as a complex product: z e^(i angle)
    Hq, Hk, rot = case["Hq"], case["Hk"], case["rot"]
    axis = [0] * (rot // 2) if s["pair_axis"] is None else s["pair_axis"].tolist()
    freq = s["inv_freq"].to(f64)
    names = {"rope_fwd": ("q", "k", "v"), "rope_bwd": ("dqkv", "dwq", "dwk")}[op]
    ends = (0, Hq, Hq + Hk, Hq + 2 * Hk)
    gains = (s["wq"], s["wk"])
    even = torch.arange(0, rot, 2, device=dev)
    first, second = (even, even + 1) if case["interleaved"] else (even // 2, even // 2 + rot // 2)
    if op == "rope_fwd":
        shape = (lambda h: (start[-1], h, d)) if packed else (lambda h: (B, h, N, d))
        out = {n: torch.zeros(shape(ends[i + 1] - ends[i]), dtype=f64, device=dev)
               for i, n in enumerate(names)}
    else:
        out = {"dqkv": torch.zeros(s["qkv"].shape, dtype=f64, device=dev)}
        if case["norm"]:
            out["dwq"] = torch.zeros(d, dtype=f64, device=dev)
            out["dwk"] = torch.zeros(d, dtype=f64, device=dev)
    for b in range(B):
        n = lens[b]
        at = slice(start[b], start[b] + n)
        x = (s["qkv"][at] if packed else s["qkv"][b, :n]).to(f64)  # (n, heads, d)
        if s["positions"] is None:
            place = torch.arange(n, device=dev, dtype=f64)[None]
        else:
            place = (s["positions"][:, at] if packed else s["positions"][:, b, :n]).to(f64)
        e = torch.exp(1j * (place[axis].T * freq))[:, None, :]  # (n, 1, rot / 2)
        for i in range(3):
            part = x[:, ends[i]:ends[i + 1]]
            if op == "rope_fwd":
                y = part.clone()
                if i < 2:
                    if case["norm"]:
                        y = y / torch.sqrt((y * y).mean(2, keepdim=True) + EPS) * gains[i].to(f64)
                    z = torch.complex(y[..., first], y[..., second]) * e
                    y[..., first], y[..., second] = z.real, z.imag
                if packed:
                    out[names[i]][at] = y
                else:
                    out[names[i]][b, :, :n] = y.transpose(0, 1)
                continue
            dy = s[("dq", "dk", "dv")[i]]
            dy = (dy[at] if packed else dy[b, :, :n].transpose(0, 1)).to(f64).clone()
            if i < 2:
                z = torch.complex(dy[..., first], dy[..., second]) * e.conj()
                dy[..., first], dy[..., second] = z.real, z.imag
                if case["norm"]:
                    rms = torch.sqrt((part * part).mean(2, keepdim=True) + EPS)
                    unit = part / rms
                    out[names[1 + i]] += (dy * unit).sum((0, 1))
                    dy = dy * gains[i].to(f64)
                    dy = (dy - unit * (dy * unit).mean(2, keepdim=True)) / rms
            if packed:
                out["dqkv"][at, ends[i]:ends[i + 1]] = dy
            else:
                out["dqkv"][b, :n, ends[i]:ends[i + 1]] = dy
    return out
