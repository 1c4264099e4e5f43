"""moira_evict against the plain form: every buffer bit for bit."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from oracle import oracle
from tests import cache_reference as ref
from tests.helpers import pack_lowbit, u16

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S = 128, 16
FMTS = (moira.SUMM_BF16, moira.SUMM_Q8, moira.SUMM_Q2)


class Cache:
    def __init__(self, hkv, max_pages, lens, seed=0, fmt=moira.SUMM_BF16, spare=5, weights="random"):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        B = len(lens)
        P = B * max_pages + spare
        self.shape, self.fmt, self.H = moira.Shape.of(4 * hkv, hkv, P), fmt, hkv
        self.k = torch.randn((P, hkv, S, D), generator=gen, device="cuda").to(torch.bfloat16)
        self.v = torch.randn((P, hkv, S, D), generator=gen, device="cuda").to(torch.bfloat16)
        self.table = rng.permutation(P)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
        self.lens = np.asarray(lens, np.int32)
        w = rng.random((P, hkv, S), dtype=np.float32)
        if weights == "ties":
            w = np.floor(w * 4) / 4
        elif weights == "zeros":
            w[:] = 0
        elif weights == "special":
            pick = rng.integers(0, 9, w.shape)
            for i, x in enumerate((np.nan, np.inf, -np.inf, -0.0, 0.0, -1.0, 1e-42, np.float32(3.4e38))):
                w[pick == i] = x
        self.weights = torch.from_numpy(w.astype(np.float32)).cuda()
        self.positions = torch.full((P, hkv, S), -1, dtype=torch.int32, device="cuda")
        self.summ = moira.make_summaries(self.shape, fmt)
        moira.update_summaries(self.shape, self.k, self.summ, torch.arange(P, dtype=torch.int32, device="cuda"),
                               fmt=fmt)
        self.ws = moira.make_evict_workspace(self.shape, B, max_pages)
        self.new_lens = torch.full((B,), -7, dtype=torch.int32, device="cuda")

    def host(self):
        return [u16(self.k).copy(), u16(self.v).copy(), self.weights.cpu().numpy().copy(),
                self.positions.cpu().numpy().copy(), self.summ.cpu()]

    def evict(self, budget, sinks, recent, new_lens=None, lens=None):
        lens = torch.from_numpy(self.lens).cuda() if lens is None else lens
        moira.evict(self.shape, self.k, self.v, self.summ, self.weights, self.positions,
                    torch.from_numpy(self.table).cuda(), lens, budget, sinks, recent,
                    self.new_lens if new_lens is None else new_lens, self.ws, fmt=self.fmt)

    def check(self, budget, sinks, recent, status=0):
        k, v, w, pos, summ = self.host()
        self.evict(budget, sinks, recent)
        torch.cuda.synchronize()
        assert moira.read_device_status(self.ws) == status
        new, renewed = ref.evict(k, v, w, pos, self.table, self.lens, budget, sinks, recent)
        gk, gv, gw, gpos, gsumm = self.host()
        assert np.array_equal(self.new_lens.cpu().numpy(), new)
        assert np.array_equal(gpos, pos)
        assert np.array_equal(gw.view(np.uint32), w.view(np.uint32))
        assert np.array_equal(gk, k) and np.array_equal(gv, v)
        # summaries: renewed where keys moved into a full page, else untouched
        if self.summ is not None:
            want = summ.clone()
            for p, j in renewed:
                self.put_summary(want, k, p, j)
            assert torch.equal(gsumm.view(torch.uint8), want.view(torch.uint8))
        return new, renewed

    def put_summary(self, want, k, p, j):
        if self.fmt == moira.SUMM_BF16:
            bits = oracle.summaries(k[p, j][None])[0].view(np.int16)
            want[p, j] = torch.from_numpy(bits).view(torch.bfloat16)
            return
        bits = 8 if self.fmt == moira.SUMM_Q8 else 2
        codes, steps = oracle.summaries_lowbit(k[p, j][None], bits)
        H, gh, cb = self.H, min(self.H, 4), D * bits // 8
        rec = pack_lowbit(np.repeat(codes[:, None], H, 1), np.repeat(steps[:, None], H, 1), bits, want.shape[-1])[0]
        o = (j // gh) * (gh * cb + 16)
        for lo, n in ((o + (j % gh) * cb, cb), (o + gh * cb + 4 * (j % gh), 4)):
            want[p, lo:lo + n] = torch.from_numpy(rec[lo:lo + n])


@pytest.mark.parametrize("hkv,lens,budget,sinks,recent", [
    (1, [2], 1, 0, 0), (1, [2], 1, 0, 1), (1, [2], 1, 1, 0),          # the smallest
    (2, [17, 16, 15, 0, 1], 16, 0, 4),                               # at, below and over the budget
    (2, [33, 100, 64], 32, 4, 12), (4, [130], 129, 1, 1), (8, [200, 31, 90, 1], 37, 2, 9),
    (1, [3000, 2999, 1500], 1024, 4, 512), (2, [5000], 17, 17, 0), (2, [5000], 17, 0, 17),
    (1, [16 * 700], 16 * 600 + 5, 3, 1000),
])
@pytest.mark.parametrize("weights", ["random", "ties"])
def test_evict_matches_the_plain_form(hkv, lens, budget, sinks, recent, weights):
    Cache(hkv, -(-max(lens) // S) + 1, lens, seed=len(lens) + budget, weights=weights).check(budget, sinks, recent)


@pytest.mark.parametrize("weights", ["zeros", "special"])
def test_evict_orders_special_weights(weights):
    """Zeros of both signs tie, NaN goes first, infinities keep their place."""
    Cache(2, 30, [300, 470, 33], seed=2, weights=weights).check(64, 2, 8)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hkv", [1, 2, 8])
def test_evict_renews_the_summaries_of_changed_pages(fmt, hkv):
    _, renewed = Cache(hkv, 20, [320, 100, 250], seed=3, fmt=fmt).check(96, 4, 30)
    assert renewed


def test_evict_long_requests():
    Cache(1, 16 * 256, [16 * 16 * 256, 60001], seed=5, weights="ties").check(8192, 4, 4096)


def test_evict_without_summaries_leaves_them():
    c = Cache(2, 10, [150], seed=6)
    before = c.summ.clone()
    summ, c.summ = c.summ, None
    moira.evict(c.shape, c.k, c.v, None, c.weights, c.positions, torch.from_numpy(c.table).cuda(),
                torch.from_numpy(c.lens).cuda(), 64, 0, 8, c.new_lens, c.ws)
    torch.cuda.synchronize()
    assert torch.equal(summ, before) and int(c.new_lens[0]) == 64


def test_evict_in_place_of_seq_lens():
    c = Cache(2, 10, [150, 20, 64], seed=7)
    lens = torch.from_numpy(c.lens).cuda()
    c.evict(64, 0, 8, new_lens=lens, lens=lens)
    assert lens.tolist() == [64, 20, 64]


def test_evict_in_place_of_seq_lens_with_more_lists_than_fit():
    """Blocks that start late must not read a length that another head of their request has already written."""
    c = Cache(8, 8, [128 - i % 5 for i in range(96)], seed=17)
    lens = torch.from_numpy(c.lens).cuda()
    k, v, w, pos, _ = c.host()
    for _ in range(2):                                           # the second call finds nothing to evict
        c.evict(64, 0, 8, new_lens=lens, lens=lens)
        assert lens.tolist() == [64] * 96
    ref.evict(k, v, w, pos, c.table, c.lens, 64, 0, 8)
    got = c.host()
    assert np.array_equal(got[3], pos) and np.array_equal(got[2].view(np.uint32), w.view(np.uint32))
    assert np.array_equal(got[0], k) and np.array_equal(got[1], v)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("batch,hkv,n,budget", [
    (1, 2, 1040, 1024), (3, 1, 1040, 1023), (3, 1, 1039, 1024),     # as many moves as warps, one more, one fewer
    (40, 4, 256, 128), (40, 4, 255, 127), (40, 4, 272, 143),         # a list for every SM: as many as windows, ..
    (160, 1, 100, 3), (20, 8, 300, 299),
])
def test_evict_few_moves_a_list(fmt, batch, hkv, n, budget):
    Cache(hkv, -(-n // S), [n - i % 3 for i in range(batch)], seed=batch + n, fmt=fmt).check(budget, 0, budget // 2)


def test_one_workspace_for_several_sizes():
    """One after another: few moves a list (one launch), many (two), a cluster a list, and again."""
    caches = [Cache(2, 8, [120, 128, 7], seed=21), Cache(8, 40, [600] * 25, seed=22), Cache(1, 400, [6400], seed=23),
              Cache(4, 9, [140, 130], seed=24), Cache(2, 8, [128, 128, 120], seed=25)]
    ws = max((c.ws for c in caches), key=lambda t: t.numel())
    for c, budget in zip(caches, (115, 200, 1000, 129, 113)):
        c.ws = ws
        c.check(budget, 0, 9)


def test_evict_keeps_rows_of_other_requests_and_rows_behind_the_last():
    """Covered bit for bit by the whole-pool comparison: spare pages, other requests' pages, and rows of the cut
    part keep their keys and values; here also the weights and positions behind n."""
    c = Cache(2, 12, [100, 0, 30], seed=8)
    c.positions.fill_(-1)
    tail = [(int(c.table[0, 100 // S]), 100 % S), (int(c.table[0, 8]), 0)]
    for p, t in tail:
        c.weights[p, :, t:] = 5.0
        c.positions[p, :, t:] = 77
    c.check(40, 0, 10)
    for p, t in tail:
        assert torch.all(c.weights[p, :, t:] == 5.0) and torch.all(c.positions[p, :, t:] == 77)


def test_bad_pages_leave_their_request_alone_and_bad_lengths_are_clamped():
    c = Cache(2, 10, [150, 150, 100], seed=9)
    c.table[1, 3] = c.shape.num_phys_pages
    new, _ = c.check(64, 0, 8, status=moira.DEV_BADPAGE)
    assert new.tolist() == [64, 150, 64]
    c = Cache(2, 10, [161, -5], seed=9)
    new, _ = c.check(64, 0, 8, status=moira.DEV_BADLEN)
    assert new.tolist() == [64, 0]


def test_repeated_evictions_of_a_growing_cache():
    """Append a few tokens, evict, over and over: positions count on, recent tokens and sinks stay."""
    rng = np.random.default_rng(10)
    c = Cache(2, 8, [60, 100], seed=10)
    for step in range(6):
        new, _ = c.check(48, 2, 20)
        pos = c.positions.cpu().numpy()
        for r in range(2):
            pg, sl = c.table[r, np.arange(new[r]) // S], np.arange(new[r]) % S
            for j in range(2):
                p = np.sort(pos[pg, j, sl])
                assert len(np.unique(p)) == new[r] and p[0] == 0 and p[1] == 1
                assert np.array_equal(p[-20:], np.arange(p[-1] - 19, p[-1] + 1))
        c.lens = new + rng.integers(1, 30, 2).astype(np.int32)
        for r in range(2):                          # the appended tokens gather weight
            t = np.arange(new[r], c.lens[r])
            pg = torch.from_numpy(c.table[r, t // S].astype(np.int64)).cuda()
            c.weights[pg, :, torch.from_numpy(t % S).cuda()] += torch.rand((len(t), 2), device="cuda")


def test_captured_and_replayed():
    c = Cache(2, 12, [100, 190], seed=12)
    table, lens = torch.from_numpy(c.table).cuda(), torch.from_numpy(c.lens).cuda()
    saved = [x.clone() for x in (c.k, c.v, c.weights, c.positions, c.summ)]
    bufs = (c.k, c.v, c.weights, c.positions, c.summ)

    def call():
        moira.evict(c.shape, c.k, c.v, c.summ, c.weights, c.positions, table, lens, 64, 1, 16, c.new_lens, c.ws)

    call()
    want = [x.clone() for x in bufs]
    graph = torch.cuda.CUDAGraph()
    for x, y in zip(bufs, saved):
        x.copy_(y)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        call()
    for _ in range(2):
        for x, y in zip(bufs, saved):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(bufs, want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
