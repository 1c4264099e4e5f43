"""Norm and rotation of queries and keys, and the append of rotated tokens,
against the plain 64-bit forms.

Tolerance of a rotated element: it is rounded once to bf16, at most 2^-8 of its
value away; before that, in fp32, the mean square (128 products and sums), its
root and quotient, two weights, sine and cosine (angle within 2^-24 of itself,
at most pi) and two products leave less than 64 roundings of 2^-24 relative to
the pair's |a| + |b|: 2^-18.  What is only moved is equal bit for bit, and
summaries are the oracle's of the keys that the cache holds."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from oracle import oracle
from tests import token_reference as ref
from tests.cache_reference import bf16_to_f64
from tests.helpers import u16

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S, G = 128, 16, 4


def bf(*dims, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(dims, generator=g, device="cuda") * scale).to(torch.bfloat16)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


def near(got, want, size):
    got = bf16_to_f64(got)
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * size + 2.0 ** -133)


def rotation(pairs, axes, inter, scale=1.0):
    freq = [10000.0 ** (-i / pairs) for i in range(pairs)]
    axis = [i * axes // pairs for i in range(pairs)]
    return freq, axis, moira.make_rotary(freq, axis, interleaved=inter, scale=scale)


@pytest.mark.parametrize("tokens,hkv,pairs,axes,inter,norm,scale,far", [
    (1, 1, 64, 1, False, True, 1.0, 0),
    (7, 2, 64, 3, False, True, 1.0, 100),
    (3, 32, 32, 2, False, False, 0.75, 5000),
    (333, 8, 24, 4, True, True, 1.0, 2 ** 31 - 400),        # the last positions that int32 holds
    (65, 4, 4, 1, True, False, 1.25, 1000000),
    (4999, 2, 64, 1, True, True, 1.0, -3000),                # negative positions turn back
    (40, 16, 60, 3, False, True, 1.0, 262144),
])
def test_rotate_qk(tokens, hkv, pairs, axes, inter, norm, scale, far):
    freq, axis, rot = rotation(pairs, axes, inter, scale)
    shape = moira.Shape.of(G * hkv, hkv, 1)
    rows = bf(tokens, 6 * hkv, D, seed=tokens)
    q, k = rows[:, :G * hkv], rows[:, G * hkv:5 * hkv]
    rng = np.random.default_rng(tokens)
    pos = (far + rng.integers(0, 399, (axes, tokens))).astype(np.int32)
    qn, kn = ((1 + 0.1 * torch.randn(D, device="cuda")) if norm else None for _ in range(2))
    qo, ko = torch.empty((tokens, G * hkv, D), dtype=torch.bfloat16, device="cuda"), torch.empty_like(k, memory_format=torch.contiguous_format)
    before = u16(rows)
    moira.rotate_qk(shape, rot, q, k, dev(pos), qo, ko, q_norm=qn, k_norm=kn, eps=1e-5)
    for x, w, o in ((q, qn, qo), (k, kn, ko)):
        w = None if w is None else w.cpu().numpy().astype(np.float64)
        near(u16(o), *ref.turned(bf16_to_f64(u16(x)), w, np.float32(1e-5).astype(np.float64), freq, axis, pos, inter, scale))
    assert np.array_equal(u16(rows), before)


def test_rotate_alone_in_place_and_without_a_rotation():
    freq, axis, rot = rotation(64, 1, False)
    shape = moira.Shape.of(8, 2, 1)
    q, k, pos = bf(37, 8, D, seed=1), bf(37, 2, D, seed=2), dev(np.arange(37)[None])
    a, b = torch.empty_like(q), torch.empty_like(k)
    moira.rotate_qk(shape, rot, q, k, pos, a, b)
    c, d = q.clone(), k.clone()
    moira.rotate_qk(shape, rot, c, None, pos, c)
    moira.rotate_qk(shape, rot, None, d, pos, k_out=d)
    assert torch.equal(a, c) and torch.equal(b, d)
    w = torch.linspace(0.5, 2, D, device="cuda")
    moira.rotate_qk(shape, None, q, k, None, a, b, q_norm=w)
    near(u16(a), *ref.turned(bf16_to_f64(u16(q)), w.cpu().numpy().astype(np.float64), np.float32(1e-6).astype(np.float64), [], [], None))
    assert torch.equal(b, k)                                   # neither norm nor rotation: the same values


def test_rotate_rows_of_zeros_and_without_finite_values():
    """A row of zeros stays zero (eps), one with an infinity or NaN spoils no other row."""
    freq, axis, rot = rotation(64, 1, False)
    shape = moira.Shape.of(4, 1, 1)
    q = bf(3, 4, D, seed=3)
    q[0, 1], q[1, 2, 5], q[2, 0, 127] = 0, float("inf"), float("nan")
    o, w = torch.empty_like(q), torch.ones(D, device="cuda")
    moira.rotate_qk(shape, rot, q, None, dev([[5, 6, 7]]), o, q_norm=w)
    assert not o[0, 1].any()
    bad = ~torch.isfinite(o).all(-1)
    assert bad.sum() == 2 and bad[1, 2] and bad[2, 0]


def test_rotate_refuses_wrong_tensors():
    _, _, rot = rotation(64, 2, False)
    shape = moira.Shape.of(8, 2, 1)
    q, pos = bf(5, 8, D), dev(np.zeros((2, 5)))
    o = torch.empty_like(q)
    for args, kind in (((q.float(), None, pos, o), TypeError), ((q[:, :4], None, pos, o), ValueError),
                       ((q.transpose(1, 2).contiguous().transpose(1, 2), None, pos, o), ValueError),
                       ((q, None, pos[:1], o), ValueError), ((q, None, pos.long(), o), TypeError),
                       ((q, None, pos, o[:4]), ValueError), ((q, None, None, o), moira.MoiraError)):
        with pytest.raises(kind):
            moira.rotate_qk(shape, rot, *args)
    with pytest.raises(moira.MoiraError):                      # token rows that are not 16-byte aligned
        moira.rotate_qk(shape, rot, torch.empty(5 * 8 * D + 4, dtype=torch.bfloat16, device="cuda")[4:].view(5, 8, D), None, pos, o)


class Batch:
    """A ragged append: `new` tokens on top of `old` cached ones for each request, rows behind the last one."""

    def __init__(self, hkv, new, old, seed=0, extra=0, fmt=moira.SUMM_BF16, spare=3):
        self.hkv, self.fmt = hkv, fmt
        self.new, self.old = np.asarray(new), np.asarray(old)
        self.lens = (self.new + self.old).astype(np.int32)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.tokens, self.B = int(self.starts[-1]) + extra, len(new)
        self.mp = max(1, -(-int(self.lens.max()) // S))
        self.P = self.B * self.mp + spare
        rng = np.random.default_rng(seed)
        self.table = rng.permutation(self.P)[:self.B * self.mp].reshape(self.B, self.mp).astype(np.int32)
        self.shape = moira.Shape.of(G * hkv, hkv, self.P)
        self.k_pool, self.v_pool = bf(self.P, hkv, S, D, seed=seed + 1), bf(self.P, hkv, S, D, seed=seed + 2)
        self.summ = moira.make_summaries(self.shape, fmt)
        self.summ.view(torch.uint8).fill_(77)
        rows = bf(self.tokens, 6 * hkv, D, seed=seed + 3)
        self.q, self.k, self.v = rows[:, :G * hkv], rows[:, G * hkv:5 * hkv], rows[:, 5 * hkv:]
        self.q_out = torch.full((self.tokens, G * hkv, D), 9.0, dtype=torch.bfloat16, device="cuda")

    def append(self, rot, **kw):
        moira.append_rotated(self.shape, rot, self.q, self.k, self.v, dev(self.starts), self.k_pool, self.v_pool, self.summ,
                             dev(self.table), dev(self.lens), self.q_out, fmt=self.fmt, **kw)

    def check(self, freq, axis, inter, scale, pos=None, qn=None, kn=None, eps=1e-6, act=None):
        """Runs `act` and compares everything that the call may and may not touch."""
        kw, vw, sw, qw = (u16(self.k_pool), u16(self.v_pool), self.summ.view(torch.uint8).cpu().numpy().copy(), u16(self.q_out))
        act()
        kg, vg, sg, qg = u16(self.k_pool), u16(self.v_pool), self.summ.view(torch.uint8).cpu().numpy(), u16(self.q_out)
        place = np.zeros((max(axis, default=0) + 1, self.tokens), np.int64)
        todo = list(ref.request_rows(self.starts, self.lens, self.mp))
        for _, row, at in todo:
            place[:, row] = at
        f64 = lambda w: None if w is None else w.cpu().numpy().astype(np.float64)  # noqa: E731
        args = (np.float64(np.float32(eps)), freq, axis, place if pos is None else pos, inter, scale)
        qr, qs = ref.turned(bf16_to_f64(u16(self.q)), f64(qn), *args)
        kr, ks = ref.turned(bf16_to_f64(u16(self.k)), f64(kn), *args)
        vn = u16(self.v)
        rows = [row for _, row, _ in todo]
        near(qg[rows], qr[rows], qs[rows])
        qw[rows] = qg[rows]
        assert np.array_equal(qg, qw)                          # other rows are left alone
        filled, seen = set(), [x for x in todo if 0 <= self.table[x[0], x[2] // S] < self.P]
        for r, row, at in seen:
            p = self.table[r, at // S]
            near(kg[p, :, at % S], kr[row], ks[row])
            kw[p, :, at % S], vw[p, :, at % S] = kg[p, :, at % S], vn[row]
            if at % S == S - 1:
                filled.add(int(p))
        assert np.array_equal(kg, kw) and np.array_equal(vg, vw)
        filled = sorted(filled)
        if filled:
            want = moira.make_summaries(self.shape, self.fmt)
            if self.fmt == moira.SUMM_BF16:
                m = oracle.summaries(kg[filled].reshape(-1, S, D)).reshape(len(filled), -1)
                sw.reshape(self.P, -1)[filled] = m.view(np.uint8)
            else:
                moira.update_summaries(self.shape, self.k_pool, want, dev(filled), fmt=self.fmt)
                sw[filled] = want.cpu().numpy()[filled]
        assert np.array_equal(sg, sw)                          # renewed bit for bit, untouched elsewhere
        return filled


@pytest.mark.parametrize("hkv,new,old,pairs,axes,inter,norm,fmt,extra", [
    (1, [1], [0], 64, 1, False, True, moira.SUMM_BF16, 0),
    (2, [1, 1, 1, 1], [15, 16, 31, 5], 64, 1, False, False, moira.SUMM_BF16, 0),          # decode: two pages fill
    (8, [16, 32], [0, 16], 64, 1, False, True, moira.SUMM_BF16, 0),                       # whole pages
    (2, [17, 0, 1, 100, 0, 3], [3, 40, 15, 9, 0, 29], 32, 3, True, True, moira.SUMM_BF16, 5),   # ragged, empty, rows behind
    (4, [250, 33], [7, 1], 24, 2, False, True, moira.SUMM_Q8, 1),
    (4, [250, 33], [7, 1], 64, 4, True, False, moira.SUMM_Q2, 0),
    (32, [40], [11], 64, 1, False, True, moira.SUMM_BF16, 0),
    (2, [5003, 1, 700], [13, 2047, 0], 64, 1, False, True, moira.SUMM_BF16, 2),           # many rows a block
    (1, list(range(1, 40)) * 8, [x % 23 for x in range(312)], 60, 1, False, False, moira.SUMM_BF16, 0),
])
@pytest.mark.parametrize("given", [False, True])
def test_append_rotated(hkv, new, old, pairs, axes, inter, norm, fmt, extra, given):
    b = Batch(hkv, new, old, seed=len(new) + hkv, extra=extra, fmt=fmt)
    freq, axis, rot = rotation(pairs, axes, inter, 1.0 if norm else 1.125)
    qn, kn = ((1 + 0.1 * torch.randn(D, device="cuda")) if norm else None for _ in range(2))
    rng = np.random.default_rng(4)
    pos = rng.integers(0, 200000, (axes, b.tokens)).astype(np.int32) if given else None
    filled = b.check(freq, axis, inter, rot.scale, pos, qn, kn, 1e-6, lambda: b.append(
        rot, positions=None if pos is None else dev(pos), q_norm=qn, k_norm=kn))
    assert len(filled) == sum((n + o) // S - o // S for n, o in zip(new, old))


def test_append_without_rotation_queries_or_summaries():
    """An encoder's states: keys and values as they are, no summaries."""
    b = Batch(2, [30, 1, 50], [0, 0, 0], seed=9)
    summ = b.summ.clone()
    moira.append_rotated(b.shape, None, None, b.k, b.v, dev(b.starts), b.k_pool, b.v_pool, None, dev(b.table), dev(b.lens))
    kg, vg, kn, vn = u16(b.k_pool), u16(b.v_pool), u16(b.k), u16(b.v)
    for r, row, at in ref.request_rows(b.starts, b.lens, b.mp):
        assert np.array_equal(kg[b.table[r, at // S], :, at % S], kn[row])
        assert np.array_equal(vg[b.table[r, at // S], :, at % S], vn[row])
    assert torch.equal(b.summ, summ)


def test_append_skips_what_is_out_of_range():
    """Requests shorter than their new tokens or longer than their table, pages outside the pool; nothing else is touched."""
    b = Batch(2, [20, 20, 20, 20, 20], [0, 30, 5, 12, 40], seed=5, extra=3)
    b.lens[1], b.lens[2] = 19, b.mp * S + 1                    # refused
    b.table[3, 1], b.table[4, 2], b.table[4, 3] = -1, b.P, 2 ** 31 - 1
    freq, axis, rot = rotation(64, 1, False)
    b.check(freq, axis, False, 1.0, act=lambda: b.append(rot))


@pytest.mark.parametrize("starts", [[0, 10, 5, 30], [-7, 3, 3, 1000], [40, 30, 20, 10], [0, 2 ** 31 - 1, 2 ** 31 - 1, -2 ** 31]])
def test_append_stays_in_bounds_with_bad_starts(starts):
    """Starts that are no ragged batch: whatever is written lies in the requests' own pages."""
    b = Batch(1, [10, 10, 10], [40, 40, 40], seed=6)
    guard = [p for p in range(b.P) if p not in b.table]
    kw = u16(b.k_pool)[guard]
    b.starts = np.asarray(starts, np.int64).astype(np.int32)
    _, _, rot = rotation(64, 1, False)
    b.append(rot)
    torch.cuda.synchronize()
    assert np.array_equal(u16(b.k_pool)[guard], kw)


def test_append_replayed_and_on_another_stream():
    """A captured append replays with the lengths and rows that its tensors then hold, here as a decode loop on a side stream."""
    hkv, B, mp = 2, 3, 6
    shape = moira.Shape.of(G * hkv, hkv, B * mp)
    freq, axis, rot = rotation(64, 1, False)
    pools = [bf(B * mp, hkv, S, D, seed=i) for i in (1, 2)]
    pools2 = [p.clone() for p in pools]
    summ = moira.make_summaries(shape)
    summ2 = summ.clone()
    table, starts, lens = dev(np.arange(B * mp).reshape(B, mp)), dev([0, 1, 2, 3]), dev([20, 31, 1])
    q, k, v = bf(B, G * hkv, D), bf(B, hkv, D), bf(B, hkv, D)
    out, out2 = torch.empty_like(q), torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def call(p, s, o, **kw):
        moira.append_rotated(shape, rot, q, k, v, starts, *p, s, table, lens, o, **kw)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(pools, summ, out)
    for step in range(40):
        lens += 1
        for x in (q, k, v):
            x.copy_(bf(*x.shape, seed=100 + step))
        g.replay()
        side.wait_stream(torch.cuda.current_stream())
        call(pools2, summ2, out2, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, out2)
    assert all(torch.equal(a, c) for a, c in zip(pools, pools2)) and torch.equal(summ, summ2)
    assert summ.any()
