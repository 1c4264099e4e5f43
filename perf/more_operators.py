"""Measured cases of the operators that fill a paged KV cache and attend to it
with many tokens a request: norms and rotation of queries and keys, the append
of rotated tokens, and the attention of a chunk of tokens (causal, or to an
encoder's states).

`run` computes an operator in its plain form (elementary torch operations in
fp32, angles in fp64) or, with `own` set, through
sparse_long_context_page_gb300's calls.  The cache is paged as the package
lays it out: pages of 16 tokens, head dimension 128, 4 query heads per KV
head.  Queries, keys and values are slices of one projection's rows.
"""
import math
import random

import numpy as np
import torch

own = False

D, S, G = 128, 16, 4
EPS = 1e-6
THETA = 500000.0


# ---------------------------------------------------------------- cases
def listed():
    return [
        # queries and keys of one decode step of four requests: the smallest call, where latency counts
        dict(name="rotate_decode", op="rotate", hkv=8, tokens=4, axes=1, pairs=64, interleaved=False, norm=True,
             far=131072),
        # the tokens of a long video: time, height and width positions
        dict(name="rotate_video", op="rotate", hkv=8, tokens=32768, axes=3, pairs=64, interleaved=False, norm=True,
             far=4096),
        # one new token for each request of a serving batch
        dict(name="append_decode", op="append", hkv=8, batch=64, new_lo=1, new_hi=1, old_lo=100, old_hi=8000, axes=1,
             pairs=64, interleaved=False, norm=False, far=0),
        # one prompt of 16k tokens
        dict(name="append_prompt", op="append", hkv=8, batch=1, new_lo=16384, new_hi=16384, old_lo=0, old_hi=0, axes=1,
             pairs=64, interleaved=False, norm=True, far=0),
        # a ragged batch with images in its prompts: every length odd, half of each head rotated, pairs side by side
        dict(name="append_ragged", op="append", hkv=4, batch=37, new_lo=1, new_hi=1531, old_lo=1, old_hi=3001, axes=3,
             pairs=32, interleaved=True, norm=True, far=200000),
        # the second turn of one short chat: latency
        dict(name="chunk_small", op="chunk", hkv=2, batch=1, new_lo=7, new_hi=7, old_lo=519, old_hi=519, causal=True),
        # one prompt of 8k tokens, from an empty cache
        dict(name="chunk_prompt", op="chunk", hkv=8, batch=1, new_lo=8192, new_hi=8192, old_lo=0, old_hi=0,
             causal=True),
        # a piece of a prompt behind 128k cached tokens
        dict(name="chunk_long", op="chunk", hkv=8, batch=1, new_lo=512, new_hi=512, old_lo=131000, old_hi=131000,
             causal=True),
        # a serving batch: new prompts and later turns, every request at its own length
        dict(name="chunk_ragged", op="chunk", hkv=8, batch=24, new_lo=3, new_hi=701, old_lo=1, old_hi=6011,
             causal=True),
        # five proposed tokens of each of sixteen requests are checked at once
        dict(name="chunk_verify", op="chunk", hkv=8, batch=16, new_lo=5, new_hi=5, old_lo=4000, old_hi=32000,
             causal=True),
        # decoders of a few hundred tokens and an encoder's 1500 states
        dict(name="cross_prompt", op="chunk", hkv=4, batch=16, new_lo=224, new_hi=448, old_lo=1500, old_hi=1500,
             causal=False),
        # a decode step of a batch whose encoder states differ in length
        dict(name="cross_decode", op="chunk", hkv=8, batch=48, new_lo=1, new_hi=1, old_lo=90, old_hi=4097,
             causal=False),
    ]


def _log(rng, lo, hi):
    return lo if lo == hi else int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _between(rng, lo, hi):
    """A length of [lo, hi], spread over its logarithm; lo may be 0."""
    return _log(rng, lo + 1, hi + 1) - 1


def draw(rng):
    most_b = max(work(c)["bytes"] for c in listed())
    most_f = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(("rotate", "append", "chunk", "chunk", "chunk"))
        c = dict(op=op, hkv=rng.choice((1, 2, 4, 8)))
        turn = dict(axes=rng.choice((1, 1, 2, 3)), pairs=rng.choice((64, 64, 32, 24)),
                    interleaved=rng.random() < 0.3, norm=rng.random() < 0.6, far=rng.choice((0, 4096, 200000)))
        if op == "rotate":
            c |= dict(tokens=_log(rng, 1, 65536), **turn)
        else:
            new = _log(rng, 1, 32768 if op == "append" else 8192)
            old = _between(rng, 0, 131072 if op == "chunk" else 16384)
            c |= dict(batch=_log(rng, 1, 64), new_lo=_log(rng, 1, new), new_hi=new, old_lo=_between(rng, 0, old),
                      old_hi=old)
            c |= dict(causal=rng.random() < 0.7) if op == "chunk" else turn
        w = work(c)
        # the plain form's padded scores and keys, and the pools, stay below 9 GB each
        big = 0
        if op != "rotate":
            total = old + new if op == "append" or c["causal"] else max(1, old)
            big = 4 * c["batch"] * c["hkv"] * total * max(D, G * new if op == "chunk" else 0)
        if w["bytes"] <= most_b and w["flops"] <= most_f and big <= 8.8e9:
            return c


def _sizes(c):
    """New tokens and cached tokens (an encoder's states, where it is not causal) of every request."""
    rng = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    new = [_log(rng, c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
    old = [_between(rng, c["old_lo"], c["old_hi"]) for _ in range(c["batch"])]
    new[rng.randrange(c["batch"])] = c["new_hi"]
    old[rng.randrange(c["batch"])] = c["old_hi"]
    if c["op"] == "chunk" and not c["causal"]:
        old = [max(1, n) for n in old]
    return new, old


def _total(c, new, old):
    """Tokens in the cache when the call reads it."""
    return old if c["op"] == "chunk" and not c["causal"] else [a + b for a, b in zip(new, old)]


def _pages(n):
    return -(-n // S)


def work(c):
    H = c["hkv"]
    if c["op"] == "rotate":
        T = c["tokens"]
        heads = H * G + H
        return dict(bytes=T * heads * D * 4 + 4 * c["axes"] * T + (8 * D if c["norm"] else 0),
                    flops=T * heads * (4 * D * c["norm"] + 6 * c["pairs"]))
    new, old = _sizes(c)
    T = sum(new)
    total = _total(c, new, old)
    if c["op"] == "append":
        heads = H * G + H
        b = T * (heads + H) * D * 4 + (4 * c["axes"] * T if c["far"] else 0) + 4 * (2 * c["batch"] + 1)
        for n, o in zip(new, old):
            filled = (n + o) // S - o // S
            # table entries, a summary for each page that fills, the older keys of the first of them
            b += 4 * (_pages(n + o) - o // S) + filled * H * D * 2 + (H * D * 2 * (o % S) if filled else 0)
        return dict(bytes=b, flops=T * heads * (4 * D * c["norm"] + 6 * c["pairs"]) + T * H * D)
    seen = sum(n * o + n * (n + 1) // 2 if c["causal"] else n * o for n, o in zip(new, old))
    b = 2 * T * H * G * D * 2 + sum(total) * H * D * 4 + 4 * sum(_pages(n) for n in total) + 4 * (2 * c["batch"] + 1)
    return dict(bytes=b, flops=4 * D * H * G * seen)


# ---------------------------------------------------------------- inputs
def _dev():
    return torch.device("cuda:0" if torch.cuda.is_available() else "cpu")


def _angles(c):
    """(inverse frequency, axis) of every pair: the first quarter of the pairs turns by time, the rest by the other
    axes in equal runs."""
    n = c["pairs"]
    freq = [THETA ** (-i / n) for i in range(n)]
    if c["axes"] == 1:
        return freq, [0] * n
    first = n // 4
    rest = (n - first) // (c["axes"] - 1)
    return freq, [0 if i < first else min(c["axes"] - 1, 1 + (i - first) // rest) for i in range(n)]


def _positions(c, tokens, rng):
    """int32 [axes][tokens]: rows of a picture 8 wide and 8 high inside a text that starts far out."""
    t = np.arange(tokens)
    start = int(rng.integers(0, max(1, c["far"])))
    return np.stack([start + t // 64, start + t % 64 // 8, start + t % 8][:c["axes"]]).astype(np.int32) \
        if c["axes"] > 1 else (start + t)[None].astype(np.int32)


def prepare(c, seed):
    dev = _dev()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    H = c["hkv"]
    ints = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(dev)  # noqa: E731
    normal = lambda *dims: torch.randn(dims, generator=gen, device=dev)  # noqa: E731
    s = dict(case=c, hkv=H)
    if own:
        import sparse_long_context_page_gb300 as moira
        s["lib"] = moira
    if c["op"] != "chunk":
        freq, axis = _angles(c)
        s["inv_freq"] = torch.tensor(freq, dtype=torch.float64, device=dev)
        s["axis"] = torch.tensor(axis, device=dev)
        s["q_norm"] = 1.0 + 0.1 * normal(D) if c["norm"] else None
        s["k_norm"] = 1.0 + 0.1 * normal(D) if c["norm"] else None
        if own:
            s["rotary"] = moira.make_rotary(freq, axis, interleaved=c["interleaved"])
    if c["op"] == "rotate":
        T = c["tokens"]
        heads = H * G + H
        # the projection's rows hold the values too, which this call leaves alone
        rows = normal(T, heads + H, D).to(torch.bfloat16)
        s["q"], s["k"] = rows[:, :H * G], rows[:, H * G:heads]
        s["positions"] = ints(_positions(c, T, rng))
        s["q_out"] = torch.empty((T, H * G, D), dtype=torch.bfloat16, device=dev)
        s["k_out"] = torch.empty((T, H, D), dtype=torch.bfloat16, device=dev)
        if own:
            s["shape"] = moira.Shape.of(H * G, H, 1)
        return s
    new, old = _sizes(c)
    total = _total(c, new, old)
    B, T = c["batch"], sum(new)
    mp = max(1, max(_pages(n) for n in total))
    P = B * mp + 1                                   # the last page belongs to nobody
    table = rng.permutation(P - 1).astype(np.int32).reshape(B, mp)
    s |= dict(batch=B, tokens=T, max_pages=mp, pages=P, most_new=max(new), page_table=ints(table),
              seq_lens=ints(total), token_starts=ints(np.concatenate([[0], np.cumsum(new)])))
    k = normal(P, H, S, D)
    # a few tokens carry large keys, as in real caches: the attention is not flat
    k *= torch.where(torch.rand((P, H, S, 1), generator=gen, device=dev) < 0.02, 3.0, 1.0)
    s["k_pool"] = k.to(torch.bfloat16)
    del k
    s["v_pool"] = normal(P, H, S, D).to(torch.bfloat16)
    if own:
        s["shape"] = moira.Shape.of(H * G, H, P)
    if c["op"] == "append":
        rows = normal(T, (G + 2) * H, D).to(torch.bfloat16)
        s["q"], s["k"], s["v"] = rows[:, :H * G], rows[:, H * G:H * (G + 1)], rows[:, H * (G + 1):]
        s["positions"] = ints(_positions(c, T, rng)) if c["far"] else None
        s["summ"] = s["k_pool"].float().mean(2).to(torch.bfloat16)
        s["q_out"] = torch.empty((T, H * G, D), dtype=torch.bfloat16, device=dev)
        return s
    s["sm_scale"] = 1.0 / math.sqrt(D)
    s["q"] = normal(T, H * G, D).to(torch.bfloat16)
    s["out"] = torch.empty((T, H * G, D), dtype=torch.bfloat16, device=dev)
    if own:
        s["ws"] = moira.make_chunk_workspace(s["shape"], B, mp, T, device=dev)
    return s


# ---------------------------------------------------------------- the operators
def run(s):
    c = s["case"]
    if c["op"] == "rotate":
        if own:
            s["lib"].rotate_qk(s["shape"], s["rotary"], s["q"], s["k"], s["positions"], s["q_out"], s["k_out"],
                               q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        else:
            cs = _cos_sin(s, s["positions"])
            s["q_out"], s["k_out"] = (_turned(s, x, w, cs) for x, w in ((s["q"], s["q_norm"]), (s["k"], s["k_norm"])))
        return {n: s[n] for n in ("q_out", "k_out")}
    if c["op"] == "append":
        if own:
            s["lib"].append_rotated(s["shape"], s["rotary"], s["q"], s["k"], s["v"], s["token_starts"], s["k_pool"],
                                    s["v_pool"], s["summ"], s["page_table"], s["seq_lens"], s["q_out"],
                                    positions=s["positions"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS)
        else:
            _plain_append(s)
        return {n: s[n] for n in ("q_out", "k_pool", "v_pool", "summ")}
    if own:
        s["lib"].attend_chunk(s["shape"], s["q"], s["k_pool"], s["v_pool"], s["page_table"], s["seq_lens"],
                              s["token_starts"], s["sm_scale"], s["out"], s["ws"], causal=c["causal"])
    else:
        s["out"] = _plain_chunk(s)
    return {"out": s["out"]}


def _cos_sin(s, positions):
    """fp32 cosine and sine [T, 1, pairs] of int32 positions [axes][T]; the angles in fp64."""
    turn = positions.double()[s["axis"]] * s["inv_freq"].unsqueeze(1)
    turn = turn.T.unsqueeze(1)
    return torch.cos(turn).float(), torch.sin(turn).float()


def _turned(s, x, weight, cs):
    """Rows [T, heads, d]: norm of each head, then its first 2 * pairs elements turned; rounded once."""
    c, (cos, sin) = s["case"], cs
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    n = c["pairs"]
    if c["interleaved"]:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., 2 * n:]), -1).to(torch.bfloat16)


def _rows(s):
    """(request, number among the request's new tokens) of every row."""
    t = torch.arange(s["tokens"], device=s["token_starts"].device)
    starts = s["token_starts"].long()
    req = torch.searchsorted(starts, t, right=True) - 1
    return req, t - starts[req]


def _plain_append(s):
    B, H = s["batch"], s["hkv"]
    dev = s["q"].device
    req, nth = _rows(s)
    starts, lens = s["token_starts"].long(), s["seq_lens"].long()
    old = lens - (starts[1:] - starts[:-1])
    at = old[req] + nth                                              # index of the token in its request
    positions = s["positions"] if s["positions"] is not None else at.expand(s["case"]["axes"], -1)
    cs = _cos_sin(s, positions)
    s["q_out"] = _turned(s, s["q"], s["q_norm"], cs)
    page, slot = s["page_table"][req, at // S].long(), at % S
    head = torch.arange(H, device=dev)
    s["k_pool"][page.unsqueeze(1), head, slot.unsqueeze(1)] = _turned(s, s["k"], s["k_norm"], cs)
    s["v_pool"][page.unsqueeze(1), head, slot.unsqueeze(1)] = s["v"]
    # summaries of the pages that these tokens fill
    many = _pages(s["most_new"]) + 1
    lp = (old // S).unsqueeze(1) + torch.arange(many, device=dev)
    full = (lp + 1) * S <= lens.unsqueeze(1)
    pages = torch.where(full, s["page_table"].gather(1, lp.clamp_max(s["max_pages"] - 1)).long(), s["pages"] - 1)
    mean = s["k_pool"][pages].double().mean(3).to(torch.bfloat16)
    s["summ"][pages] = torch.where(full.view(B, many, 1, 1), mean, s["summ"][pages])


def _plain_chunk(s):
    B, H, M = s["batch"], s["hkv"], s["most_new"]
    dev = s["q"].device
    req, nth = _rows(s)
    starts, lens = s["token_starts"].long(), s["seq_lens"].long()
    n_new = starts[1:] - starts[:-1]
    row = (starts[:-1].unsqueeze(1) + torch.arange(M, device=dev)).clamp_max(s["tokens"] - 1)       # [B, M]
    q = s["q"].float()[row].view(B, M, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * M, D)
    pages = s["page_table"].long()
    N = s["max_pages"] * S
    k = s["k_pool"][pages].transpose(1, 2).reshape(B, H, N, D).float()
    v = s["v_pool"][pages].transpose(1, 2).reshape(B, H, N, D).float()
    seen = lens.unsqueeze(1).expand(B, M)
    if s["case"]["causal"]:
        seen = lens.unsqueeze(1) - n_new.unsqueeze(1) + 1 + torch.arange(M, device=dev)
        seen = torch.minimum(seen, lens.unsqueeze(1))
    hidden = torch.arange(N, device=dev) >= seen.unsqueeze(-1)                                      # [B, M, N]
    sc = (q @ k.transpose(-1, -2)).view(B, H, G, M, N)
    sc = sc.mul_(s["sm_scale"]).masked_fill_(hidden.view(B, 1, 1, M, N), -math.inf)
    sc = sc.sub_(sc.amax(-1, keepdim=True).clamp_min_(-3.0e38)).exp_().view(B, H, G * M, N)
    # a token that the cache does not hold has weight 0 and may hold anything
    v = torch.where((torch.arange(N, device=dev) < lens.unsqueeze(1)).view(B, 1, N, 1), v, 0.0)
    o = (sc @ v) / sc.sum(-1, keepdim=True).clamp_min(1e-30)
    o = o.view(B, H, G, M, D).permute(0, 3, 1, 2, 4).reshape(B, M, H * G, D)
    return o[req, nth].to(torch.bfloat16)


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(c, seed):
    if c["op"] == "chunk" and work(c)["flops"] > 3e12:
        return None
    s = prepare(c, seed)
    return _exact_chunk(s) if c["op"] == "chunk" else _exact_rows(s)


def _exact_turn(s, x, weight, place):
    """Rows x [n, heads, d] at positions `place` [axes][n], as complex numbers turned by their angle."""
    c = s["case"]
    freq, axis = _angles(c)
    x = x.double()
    if weight is not None:
        x = x / ((x * x).sum(-1, keepdim=True) / D + EPS).sqrt() * weight.double()
    y = x.clone()
    n = c["pairs"]
    first = slice(0, 2 * n, 2) if c["interleaved"] else slice(0, n)
    second = slice(1, 2 * n, 2) if c["interleaved"] else slice(n, 2 * n)
    angle = torch.stack([place[axis[i]].double() * freq[i] for i in range(n)], -1).unsqueeze(1)
    z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rows(s):
    c, H = s["case"], s["hkv"]
    dev = s["q"].device
    if c["op"] == "rotate":
        place = s["positions"].long()
        return dict(q_out=_exact_turn(s, s["q"], s["q_norm"], place), k_out=_exact_turn(s, s["k"], s["k_norm"], place))
    new, old = _sizes(c)
    at = torch.from_numpy(np.concatenate([np.arange(o, o + n) for n, o in zip(new, old)])).to(dev)
    req = torch.from_numpy(np.repeat(np.arange(len(new)), new)).to(dev)
    place = s["positions"].long() if s["positions"] is not None else at.expand(c["axes"], -1)
    kp, vp, summ = s["k_pool"].double(), s["v_pool"].double(), s["summ"].double()
    keys = _exact_turn(s, s["k"], s["k_norm"], place)
    row = s["page_table"][req, at // S].long() * S + at % S           # rows of the pools, token by token
    for pool, x in ((kp, keys), (vp, s["v"].double())):
        flat = pool.transpose(1, 2).reshape(-1, H, D).clone()
        flat[row] = x
        pool.copy_(flat.view(-1, S, H, D).transpose(1, 2))
    done = [(r, p) for r, (n, o) in enumerate(zip(new, old)) for p in range(o // S, (n + o) // S)]
    if done:
        r, p = (torch.tensor(x, device=dev) for x in zip(*done))
        page = s["page_table"][r, p].long()
        # a page's summary is the mean of its keys as the cache holds them
        summ[page] = kp[page].to(torch.bfloat16).double().sum(2) / S
    return dict(q_out=_exact_turn(s, s["q"], s["q_norm"], place), k_pool=kp, v_pool=vp, summ=summ)


def _exact_chunk(s):
    c, H = s["case"], s["hkv"]
    dev = s["q"].device
    new, old = _sizes(c)
    total = _total(c, new, old)
    out = torch.zeros((s["tokens"], H * G, D), dtype=torch.float64, device=dev)
    at = 0
    for r, (n, L) in enumerate(zip(new, total)):
        pages = s["page_table"][r, :_pages(L)].long()
        for j in range(H):
            k, v = (s[x][pages, j].reshape(-1, D)[:L].double() for x in ("k_pool", "v_pool"))
            for lo in range(0, n, 512):
                hi = min(n, lo + 512)
                q = s["q"][at + lo:at + hi, j * G:(j + 1) * G].double()
                last = L - n + hi if c["causal"] else L                 # keys that some row of the piece sees
                sc = torch.einsum("thd,kd->thk", q, k[:last]) * s["sm_scale"]
                if c["causal"]:
                    far = torch.ones((hi - lo, last), dtype=torch.bool, device=dev).triu(L - n + lo + 1)
                    sc.masked_fill_(far.unsqueeze(1), -math.inf)
                out[at + lo:at + hi, j * G:(j + 1) * G] = torch.einsum("thk,kd->thd", torch.softmax(sc, -1), v[:last])
        at += n
    return dict(out=out)
