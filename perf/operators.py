"""Measured cases of the cache operators: attention of a batch that shares a
prefix, attention that accumulates each cached token's attention weight, and
eviction by that weight.

`run` computes an operator in its plain form (elementary torch operations in
fp32) or, with `own` set, through sparse_long_context_page_gb300's calls.
Every case is a paged bf16 KV cache as the package lays it out: pages of 16
tokens, head dimension 128, 4 query heads per KV head.
"""
import math
import random

import numpy as np
import torch

own = False

D, S, G = 128, 16, 4
CHUNK = 64                       # pages per partial sum of the plain attention (1024 tokens)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # four short chats behind one short system prompt: the smallest call, where latency counts
        dict(name="shared_small", op="shared", hkv=2, batch=4, groups=1, prefix=519, own_lo=1, own_hi=48,
             keep=1.0, weights=False),
        # a serving batch behind a long system prompt, every request at its own length
        dict(name="shared_serving", op="shared", hkv=8, batch=32, groups=1, prefix=8192, own_lo=64, own_hi=2048,
             keep=1.0, weights=False),
        # eight questions about one 128k document
        dict(name="shared_document", op="shared", hkv=8, batch=8, groups=1, prefix=131072, own_lo=16, own_hi=512,
             keep=1.0, weights=False),
        # many samples of one long prompt: enough query rows to be bound by arithmetic
        dict(name="shared_wide", op="shared", hkv=8, batch=256, groups=1, prefix=32763, own_lo=128, own_hi=1024,
             keep=1.0, weights=False),
        # six tenants, each with a prompt of its own, weights accumulated for a later eviction
        dict(name="shared_tenants", op="shared", hkv=4, batch=48, groups=6, prefix=16384, own_lo=256, own_hi=4096,
             keep=1.0, weights=True),
        # one short request, weights accumulated
        dict(name="weights_small", op="weights", hkv=2, batch=1, groups=0, prefix=0, own_lo=1000, own_hi=1000,
             keep=1.0, weights=True),
        # one 128k request, every page read
        dict(name="weights_long", op="weights", hkv=8, batch=1, groups=0, prefix=0, own_lo=131072, own_hi=131072,
             keep=1.0, weights=True),
        # a ragged batch over selected pages (about a third of them, as the coverage rule keeps)
        dict(name="weights_selected", op="weights", hkv=8, batch=32, groups=0, prefix=0, own_lo=1024, own_hi=16384,
             keep=0.33, weights=True),
        # one short request a few tokens over its budget
        dict(name="evict_small", op="evict", hkv=2, batch=1, len_lo=1040, len_hi=1040, budget=1024, recent=256,
             sinks=4, primed=True),
        # a serving batch that evicts every 16 decode steps
        dict(name="evict_decode", op="evict", hkv=8, batch=32, len_lo=4112, len_hi=4112, budget=4096, recent=2048,
             sinks=4, primed=True),
        # two 64k prompts cut to an eighth after prefill
        dict(name="evict_prompt", op="evict", hkv=8, batch=2, len_lo=65536, len_hi=65536, budget=8192, recent=4096,
             sinks=4, primed=False),
        # a ragged batch cut to one budget; the short requests keep every token
        dict(name="evict_ragged", op="evict", hkv=8, batch=64, len_lo=500, len_hi=20000, budget=2037, recent=509,
             sinks=1, primed=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most_b = max(work(c)["bytes"] for c in listed())
    most_f = max(work(c)["flops"] for c in listed())
    while True:
        op = rng.choice(("shared", "shared", "weights", "evict"))
        c = dict(op=op, hkv=rng.choice((1, 2, 4, 8)))
        if op == "evict":
            hi = _log(rng, 20, 65536)
            lo = _log(rng, 1, hi)
            budget = _log(rng, 8, 16384)
            recent = rng.randint(0, budget // 2)
            c |= dict(batch=_log(rng, 1, 64), len_lo=lo, len_hi=hi, budget=budget, recent=recent,
                      sinks=rng.randint(0, min(8, budget - recent)), primed=rng.random() < 0.5)
        else:
            hi = _log(rng, 1, 131072 if op == "weights" else 16384)
            c |= dict(batch=_log(rng, 1, 256 if op == "shared" else 64), groups=0, prefix=0,
                      own_lo=_log(rng, 1, hi), own_hi=hi, keep=rng.choice((1.0, 1.0, 0.3)),
                      weights=op == "weights" or rng.random() < 0.5)
            if op == "shared":
                c |= dict(groups=min(c["batch"], rng.choice((1, 1, 2, 5))), prefix=_log(rng, 1, 131072))
        # the gathered plain form stays within a few GB
        big = c["batch"] * c["hkv"] * (c["len_hi"] if op == "evict" else c["own_hi"]) + \
            c.get("groups", 0) * c["hkv"] * c.get("prefix", 0)
        w = work(c)
        if w["bytes"] <= most_b and w["flops"] <= most_f and big <= 32 * 8 * 16384:
            return c


def _sizes(c):
    """Lengths of a case (the same for every seed): own lengths, group starts, prefix lengths."""
    rng = random.Random(repr(sorted((k, v) for k, v in c.items() if k != "name")))
    lo, hi = (c["len_lo"], c["len_hi"]) if c["op"] == "evict" else (c["own_lo"], c["own_hi"])
    lens = [_log(rng, lo, hi) for _ in range(c["batch"])]
    lens[rng.randrange(c["batch"])] = hi
    n = c.get("groups", 0)
    starts, plens = [0], []
    if n:
        starts += sorted(rng.sample(range(1, c["batch"]), n - 1)) + [c["batch"]]
        plens = [c["prefix"]] + [_log(rng, max(1, c["prefix"] // 16), c["prefix"]) for _ in range(n - 1)]
    return lens, starts, plens


def _pages(n):
    return -(-n // S)


def _kept(c, lens):
    """Per (request, KV head): the listed full pages in ascending order (the partial page, if any, follows)."""
    rng = np.random.default_rng(len(lens) * 1000 + c["hkv"])
    out = []
    for n in lens:
        full = n // S
        row = []
        for _ in range(c["hkv"]):
            keep = np.arange(full) if c["keep"] >= 1 else np.flatnonzero(rng.random(full) < c["keep"])
            row.append(np.concatenate([keep, [full]]) if n % S else keep)
        out.append(row)
    return out


def work(c):
    lens, starts, plens = _sizes(c)
    B, H = c["batch"], c["hkv"]
    if c["op"] == "evict":
        b = 4 * 2 * B
        for n in lens:
            m = min(n, c["budget"])
            b += 4 * _pages(n)                                         # page table
            if n > m:
                moves = min(n - m, max(c["recent"], 1))
                # weights and positions of every token; cleared tail; K, V, weight and position of a move;
                # each page that takes a token is read once for its summary
                b += H * (8 * n + 8 * (n - m) + moves * (4 * D * 2 + 8) +
                          min(moves, m // S) * (S * D * 2 + D * 2))
        return dict(bytes=b, flops=H * sum(lens))
    kept = _kept(c, lens)
    toks = sum((len(k) - (n % S > 0)) * S + n % S for n, row in zip(lens, kept) for k in row)
    ptoks = sum(plens) * H
    rows = [(e - s) * G for s, e in zip(starts, starts[1:])]
    b = 2 * 2 * D * (toks + ptoks) + B * H * G * D * (2 + 4) + 4 * sum(len(k) for row in kept for k in row)
    b += 4 * sum(_pages(p) for p in plens) + (8 * toks if c["weights"] else 0)
    f = 4 * D * G * toks + 4 * D * H * sum(r * p for r, p in zip(rows, plens))
    return dict(bytes=b, flops=f)


# ---------------------------------------------------------------- inputs
def _dev():
    return torch.device("cuda:0" if torch.cuda.is_available() else "cpu")


def prepare(c, seed):
    dev = _dev()
    gen = torch.Generator(device=dev).manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    lens, starts, plens = _sizes(c)
    B, H = c["batch"], c["hkv"]
    mp = max(1, max(_pages(n) for n in lens))
    npre = [_pages(p) for p in plens]
    P = B * mp + sum(npre)
    perm = rng.permutation(P).astype(np.int32)
    table = perm[:B * mp].reshape(B, mp)
    k = torch.randn((P, H, S, D), generator=gen, device=dev)
    # a few tokens carry large keys, as in real caches: the attention is not flat
    k *= torch.where(torch.rand((P, H, S, 1), generator=gen, device=dev) < 0.02, 3.0, 1.0)
    k = k.to(torch.bfloat16)
    v = torch.randn((P, H, S, D), generator=gen, device=dev).to(torch.bfloat16)
    ints = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(dev)  # noqa: E731
    s = dict(case=c, hkv=H, batch=B, max_pages=mp, k=k, v=v, page_table=ints(table), seq_lens=ints(lens))
    if c["op"] == "evict":
        s["weights"] = torch.rand((P, H, S), generator=gen, device=dev) ** 4 * 10.0
        pos = torch.full((P, H, S), -1, dtype=torch.int32, device=dev)
        slot = torch.arange(mp * S, device=dev, dtype=torch.int32).view(1, mp, 1, S).expand(B, mp, H, S)
        old = slot < torch.minimum(s["seq_lens"], torch.tensor(c["budget"], device=dev)).view(B, 1, 1, 1)
        if c["primed"]:                    # the first `budget` slots were kept by an earlier eviction
            pos[s["page_table"].long()] = torch.where(old, 3 * slot + 1, -1)
            s["weights"][s["page_table"].long()] *= torch.where(old, 1.0, 0.1)
        s["positions"] = pos
        s["summ"] = k.float().mean(2).to(torch.bfloat16)
        s["new_lens"] = torch.zeros_like(s["seq_lens"])
        if own:
            import sparse_long_context_page_gb300 as moira
            s["lib"], s["shape"] = moira, moira.Shape.of(H * G, H, P)
            s["ws"] = moira.make_evict_workspace(s["shape"], B, mp, device=dev)
        return s
    s["sm_scale"] = 1.0 / math.sqrt(D)
    s["q"] = torch.randn((B, H * G, D), generator=gen, device=dev).to(torch.bfloat16)
    kept = _kept(c, lens)
    lists = np.zeros((B, H, mp), np.int32)
    lengths = np.zeros((B, H), np.int32)
    for r in range(B):
        for j in range(H):
            lists[r, j, :len(kept[r][j])] = table[r, kept[r][j]]
            lengths[r, j] = len(kept[r][j])
    s["lists"], s["lengths"] = ints(lists), ints(lengths)
    if c["op"] == "shared":
        pt = np.full((len(plens), max(npre)), -1, np.int32)
        at = B * mp
        for g, n in enumerate(npre):
            pt[g, :n] = perm[at:at + n]
            at += n
        s["prefix_table"], s["prefix_lens"], s["group_starts"] = ints(pt), ints(plens), ints(starts)
        s["most"] = max(b - a for a, b in zip(starts, starts[1:]))      # requests of the largest group
    s["weights"] = torch.zeros((P, H, S), device=dev) if c["weights"] else None
    s["out"] = torch.empty((B, H * G, D), dtype=torch.float32, device=dev)
    if own:
        import sparse_long_context_page_gb300 as moira
        s["lib"], s["shape"] = moira, moira.Shape.of(H * G, H, P)
        s["ws"] = moira.make_shared_workspace(s["shape"], B, mp, groups=len(plens), weights=bool(c["weights"]),
                                              device=dev)
    return s


# ---------------------------------------------------------------- the operators
def run(s):
    op = s["case"]["op"]
    if own:
        m = s["lib"]
        if op == "evict":
            c = s["case"]
            m.evict(s["shape"], s["k"], s["v"], s["summ"], s["weights"], s["positions"], s["page_table"],
                    s["seq_lens"], c["budget"], c["sinks"], c["recent"], s["new_lens"], s["ws"])
        elif op == "shared":
            m.attend_shared(s["shape"], s["q"], s["k"], s["v"], s["prefix_table"], s["prefix_lens"],
                            s["group_starts"], s["lists"], s["lengths"], s["seq_lens"], s["max_pages"],
                            s["sm_scale"], s["out"], s["ws"], weights=s["weights"])
        else:
            m.attend_weights(s["shape"], s["q"], s["k"], s["v"], s["lists"], s["lengths"], s["seq_lens"],
                             s["max_pages"], s["sm_scale"], s["weights"], s["out"], s["ws"])
    elif op == "evict":
        _plain_evict(s)
    else:
        s["out"] = _plain_attend(s)
    names = ("k", "v", "summ", "weights", "positions", "new_lens") if op == "evict" else ("out", "weights")
    return {n: s[n] for n in names if s[n] is not None}


def _partial(q, k, v, ok, scale):
    """Softmax partials of rows q [.., M, d] over keys k, v [.., N, d] where ok [.., N] (N a multiple of the
    chunk): scores, row maximum, sum and unnormalised output, the long sums taken in two levels."""
    sc = (q @ k.transpose(-1, -2)) * scale
    sc = sc.masked_fill(~ok.unsqueeze(-2), -math.inf)
    m = sc.amax(-1, keepdim=True)
    e = torch.exp(sc - m.clamp_min(-3.0e38))
    M, N = e.shape[-2:]
    lead = e.shape[:-2]
    c = e.view(*lead, M, N // (CHUNK * S), CHUNK * S).transpose(-2, -3)
    o = (c @ v.reshape(*lead, N // (CHUNK * S), CHUNK * S, D)).sum(-3)
    return sc, m, c.sum(-1).sum(-2).unsqueeze(-1), o


def _padded(pages):
    """A page list [.., n] padded with page 0 to whole chunks."""
    return torch.nn.functional.pad(pages, (0, -pages.shape[-1] % CHUNK))


def _plain_attend(s):
    B, H = s["batch"], s["hkv"]
    dev = s["q"].device
    q = s["q"].float().view(B, H, G, D)
    lists = _padded(s["lists"])
    n = lists.shape[-1]
    pid = lists.clamp_min(0).long()                                       # [B, H, n]
    at = torch.arange(n, device=dev)
    tail = (s["seq_lens"] % S).view(B, 1, 1)
    ntok = torch.where((at == s["lengths"].unsqueeze(-1) - 1) & (tail > 0), tail, S)
    ntok = torch.where(at < s["lengths"].unsqueeze(-1), ntok, 0)
    ok = (torch.arange(S, device=dev) < ntok.unsqueeze(-1)).view(B, H, n * S)
    head = torch.arange(H, device=dev).view(1, H, 1)
    sc, m, l, o = _partial(q, s["k"][pid, head].float().view(B, H, n * S, D),
                           s["v"][pid, head].float().view(B, H, n * S, D), ok, s["sm_scale"])
    if s["case"]["op"] == "shared":
        starts, R = s["group_starts"].long(), s["most"]
        NG = starts.numel() - 1
        r = torch.arange(B, device=dev)
        req = (starts[:-1].unsqueeze(1) + torch.arange(R, device=dev)).clamp_max(B - 1)   # [NG, R]
        qg = q[req].transpose(1, 2).reshape(NG, H, R * G, D)
        pt = _padded(s["prefix_table"]).clamp_min(0).long()
        kg = s["k"][pt].float().transpose(1, 2).reshape(NG, H, -1, D)
        vg = s["v"][pt].float().transpose(1, 2).reshape(NG, H, -1, D)
        okg = torch.arange(kg.shape[2], device=dev) < s["prefix_lens"].view(NG, 1, 1)
        _, mg, lg, og = _partial(qg, kg, vg, okg.expand(NG, H, -1), s["sm_scale"])
        gid = torch.searchsorted(starts, r, right=True) - 1
        back = lambda x: x.view(NG, H, R, G, -1)[gid, :, r - starts[gid]]  # noqa: E731
        mg, lg, og = back(mg), back(lg), back(og)
        mj = torch.maximum(m, mg).clamp_min(-3.0e38)
        a, b = torch.exp(m - mj), torch.exp(mg - mj)
        m, l, o = mj, a * l + b * lg, a * o + b * og
    if s["weights"] is not None:
        p = (torch.exp(sc - m.clamp_min(-3.0e38)) / l.clamp_min(1e-30)).sum(2).view(B, H, n, S)
        s["weights"].index_put_((pid, head), torch.where(ok.view(B, H, n, S), p, 0.0), accumulate=True)
    return torch.where(l > 0, o / l.clamp_min(1e-30), 0.0).view(B, H * G, D)


def _plain_evict(s):
    c, B, H = s["case"], s["batch"], s["hkv"]
    dev = s["k"].device
    table = s["page_table"].long()
    T = s["max_pages"] * S
    pick = lambda x: x[table].transpose(1, 2).reshape(B, H, T)  # noqa: E731
    w, pos = pick(s["weights"]), pick(s["positions"])
    t = torch.arange(T, device=dev)
    n = s["seq_lens"].long().view(B, 1, 1)
    m = n.clamp_max(c["budget"])
    live = t < n
    unset = live & (pos < 0)
    last = torch.where(live, pos, -1).amax(-1, keepdim=True)
    first = torch.where(unset, t, T).amin(-1, keepdim=True)
    pos = torch.where(unset, last + 1 + t - first, pos)
    newest = torch.where(live, pos, -1).amax(-1, keepdim=True)
    safe = (pos < c["sinks"]) | (pos > newest - c["recent"])
    # protected tokens first, then by weight, NaN last: one ordered integer per token
    key = (w + 0.0).view(torch.int32).long()
    key = torch.where(key < 0, -(key & 0x7FFFFFFF), key)
    key = torch.where(torch.isnan(w), -(1 << 32), key)
    key = torch.where(safe, 1 << 32, key)
    key = torch.where(live, key, -(1 << 33))
    order = torch.sort(key, dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(-1, order, t.expand(B, H, T).contiguous())
    kept = live & (rank < m)
    hole, mover = ~kept & (t < m), kept & (t >= m)
    # the i-th hole takes the i-th mover
    dump = T
    nth = torch.where(mover, mover.long().cumsum(-1) - 1, dump)
    movers = torch.zeros((B, H, T + 1), dtype=torch.long, device=dev).scatter_(-1, nth, t.expand(B, H, T))
    src = torch.where(hole, movers.gather(-1, (hole.long().cumsum(-1) - 1).clamp_min(0)), t)
    cut = live & (n > m)
    w, pos2 = w.gather(-1, src), pos.gather(-1, src)
    old_pos = pick(s["positions"])
    w = torch.where(cut & (t >= m), 0.0, w)
    pos = torch.where(cut, torch.where(t < m, pos2, -1), old_pos).int()
    unpick = lambda x: x.view(B, H, s["max_pages"], S).transpose(1, 2)  # noqa: E731
    s["weights"][table], s["positions"][table] = unpick(w), unpick(pos)
    few = min(s["max_pages"], _pages(c["budget"]))
    Tk = few * S
    row = (table.repeat_interleave(S, 1).unsqueeze(1) * H + torch.arange(H, device=dev).view(1, H, 1)) * S + t % S
    at = row[..., :Tk]
    frm = row.gather(-1, src[..., :Tk])
    for_pool = s["k"].view(-1, D), s["v"].view(-1, D)
    for_pool[0][at], for_pool[1][at] = for_pool[0][frm], for_pool[1][frm]
    pages = table[:, :few]
    changed = hole.view(B, H, s["max_pages"], S).any(-1)[..., :few] & \
        (torch.arange(1, few + 1, device=dev) * S <= m) & (n > m)
    mean = s["k"][pages].double().mean(3).to(torch.bfloat16)
    s["summ"][pages] = torch.where(changed.transpose(1, 2).unsqueeze(-1), mean, s["summ"][pages])
    s["new_lens"].copy_(m.view(B))


# ---------------------------------------------------------------- the definition, in 64 bits
def exact(c, seed):
    w = work(c)
    if w["flops"] > 4e11:
        return None
    s = prepare(c, seed)
    return _exact_evict(s) if c["op"] == "evict" else _exact_attend(s)


def _exact_attend(s):
    H = s["hkv"]
    lens, starts, plens = _sizes(s["case"])
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=s["q"].device)
    weights = None if s["weights"] is None else s["weights"].double()
    lists, lengths = s["lists"].long(), s["lengths"].tolist()
    q = s["q"].double()

    def joint(rq, parts):
        """Softmax over the concatenated keys of `parts`; one matrix of probabilities."""
        kk = torch.cat([p[0] for p in parts]).double()
        vv = torch.cat([p[1] for p in parts]).double()
        p = torch.softmax((rq @ kk.T) * s["sm_scale"], -1)
        return p, p @ vv

    groups = list(zip(starts, starts[1:], plens)) if plens else [(0, len(lens), 0)]
    for g, (a, b, plen) in enumerate(groups):
        for j in range(H):
            if plen:
                pages = s["prefix_table"][g, :_pages(plen)].long()
                pk, pv = (s[x][pages, j].reshape(-1, D)[:plen].double() for x in ("k", "v"))
                rows = q[a:b, j * G:(j + 1) * G].reshape(-1, D)
                ps = (rows @ pk.T) * s["sm_scale"]
                lse_p = torch.logsumexp(ps, -1).view(b - a, G)
                o_p = (torch.softmax(ps, -1) @ pv).view(b - a, G, D)
                del ps
            for r in range(a, b):
                cnt = lengths[r][j]
                pages = lists[r, j, :cnt]
                toks = cnt * S - (S - lens[r] % S if cnt and lens[r] % S else 0)
                rq = q[r, j * G:(j + 1) * G]
                if toks == 0:
                    if plen:
                        out[r, j * G:(j + 1) * G] = o_p[r - a]
                    continue
                ok, ov = (s[x][pages, j].reshape(-1, D)[:toks] for x in ("k", "v"))
                p, o = joint(rq, [(ok, ov)])
                share = torch.ones(G, 1, dtype=torch.float64, device=q.device)
                if plen:
                    lse_o = torch.logsumexp((rq @ ok.double().T) * s["sm_scale"], -1)
                    share = torch.sigmoid(lse_o - lse_p[r - a]).unsqueeze(-1)
                    o = share * o + (1 - share) * o_p[r - a]
                out[r, j * G:(j + 1) * G] = o
                if weights is not None:
                    add = torch.zeros(cnt * S, dtype=torch.float64, device=q.device)
                    add[:toks] = (share * p).sum(0)
                    weights[pages, j] += add.view(cnt, S)
    return dict(out=out) if weights is None else dict(out=out, weights=weights)


def _exact_evict(s):
    c, H = s["case"], s["hkv"]
    lens = s["seq_lens"].tolist()
    table = s["page_table"].cpu().numpy().astype(np.int64)
    w, pos = s["weights"].cpu().numpy().copy(), s["positions"].cpu().numpy().copy()
    summ = s["summ"].double()
    new, dst, src, touched = [], [], [], []
    for r, n in enumerate(lens):
        m = min(n, c["budget"])
        new.append(m)
        if n == m:
            continue
        page, slot = table[r][np.arange(n) // S], np.arange(n) % S
        for j in range(H):
            wr, pr = w[page, j, slot], pos[page, j, slot].astype(np.int64)
            gone = np.flatnonzero(pr < 0)
            if gone.size:
                pr[gone] = pr.max(initial=-1) + 1 + gone - gone[0]
            safe = (pr < c["sinks"]) | (pr > pr.max() - c["recent"])
            value = np.where(safe, np.inf, np.where(np.isnan(wr), -np.inf, wr.astype(np.float64)))
            keep = np.zeros(n, bool)
            keep[np.lexsort((np.arange(n), -value))[:m]] = True
            holes, movers = np.flatnonzero(~keep[:m]), m + np.flatnonzero(keep[m:])
            wr[holes], pr[holes] = wr[movers], pr[movers]
            wr[m:], pr[m:] = 0, -1
            w[page, j, slot], pos[page, j, slot] = wr, pr
            flat = (page * H + j) * S + slot
            dst.append(flat[holes])
            src.append(flat[movers])
            full = np.unique(holes // S)
            touched.append(table[r][full[full < m // S]] * H + j)
    if dst:
        to, frm, pages = (torch.from_numpy(np.concatenate(x)).to(summ.device) for x in (dst, src, touched))
        for x in ("k", "v"):
            s[x].view(-1, D)[to] = s[x].view(-1, D)[frm]
        summ.view(-1, D)[pages] = s["k"].view(-1, S, D)[pages].double().sum(1) / S
    dev = summ.device
    return dict(k=s["k"], v=s["v"], summ=summ, weights=torch.from_numpy(w).to(dev).double(),
                positions=torch.from_numpy(pos).to(dev), new_lens=torch.tensor(new, dtype=torch.int32, device=dev))
