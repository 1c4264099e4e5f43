"""Attention of a chunk of tokens over the paged cache, against the plain
64-bit form.

Tolerance of an element: the weights enter the product as bf16, each at most
2^-8 of itself away, and the output is rounded to bf16, 2^-8 of its value.  The
scores are fp32 sums of 128 products (error below 2^-16 sum |q k| scale, here
below 2^-11) and the sums over the tokens are fp32 (below 2^-11 of sum w |v| at
these lengths): 2^-8 |out| + (2^-8 + 2^-10) sum w |v|.  The two roundings to
bf16 are independent and uniform, 2^-8 / sqrt 3 each, and the weights' errors
add up like random signs: the whole output's relative L2 error stays below
sqrt(2/3) 2^-8 < 2^-8."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from tests import token_reference as ref
from tests.cache_reference import bf16_to_f64
from tests.helpers import u16

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S, G = 128, 16, 4
SCALE = 1.0 / np.sqrt(D)


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()


class Chunk:
    """`new` rows of each request over a cache of `total` tokens; everything that no token holds is NaN."""

    def __init__(self, hkv, new, total, seed=0, causal=True, extra=0, mp=None, spare=2, stale=float("nan"), peak=3.0):
        self.hkv, self.causal, self.B = hkv, causal, len(new)
        self.lens = np.asarray(total, np.int32)
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.tokens = int(self.starts[-1]) + extra
        self.mp = mp or max(1, -(-int(self.lens.max()) // S))
        self.P = self.B * self.mp + spare
        rng = np.random.default_rng(seed)
        self.table = rng.permutation(self.P)[:self.B * self.mp].reshape(self.B, self.mp).astype(np.int32)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.k, self.v = (torch.full((self.P, hkv, S, D), stale, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        for r, L in enumerate(total):
            if L == 0:
                continue
            t = torch.arange(L, device="cuda")
            page = torch.from_numpy(self.table[r]).cuda().long()[t // S]
            big = torch.where(torch.rand((L, hkv, 1), generator=g, device="cuda") < 0.02, peak, 1.0)
            self.k[page, :, t % S] = (torch.randn((L, hkv, D), generator=g, device="cuda") * big).to(torch.bfloat16)
            self.v[page, :, t % S] = torch.randn((L, hkv, D), generator=g, device="cuda").to(torch.bfloat16)
        self.q = torch.randn((max(1, self.tokens), G * hkv, D), generator=g, device="cuda").to(torch.bfloat16)[:self.tokens]
        self.shape = moira.Shape.of(G * hkv, hkv, self.P)
        self.out = torch.full((self.tokens, G * hkv, D), 5.0, dtype=torch.bfloat16, device="cuda")
        self.ws = moira.make_chunk_workspace(self.shape, self.B, self.mp, max(1, self.tokens))

    def run(self, out=None, ws=None, scale=SCALE, **kw):
        out = self.out if out is None else out
        moira.attend_chunk(self.shape, self.q, self.k, self.v, dev(self.table), dev(self.lens), dev(self.starts), scale,
                           out, self.ws if ws is None else ws, causal=self.causal, **kw)
        return out

    def check(self, got=None, scale=SCALE, pages=None):
        got = u16(self.out if got is None else got)
        want, size = ref.attend_chunk(u16(self.q), u16(self.k), u16(self.v), self.table, self.lens, self.starts, scale,
                                      self.causal, pages)
        n = int(self.starts[-1])
        assert np.all(got[n:] == 0x40A0)                       # rows behind the last request keep their 5.0
        g, w, z = bf16_to_f64(got[:n]), want[:n], size[:n]
        err = np.abs(g - w)
        bad = err > 2.0 ** -8 * np.abs(w) + (2.0 ** -8 + 2.0 ** -10) * z + 1e-30
        assert not bad.any() and np.isfinite(g).all(), (np.argwhere(bad)[:4], err[bad][:4])
        norm = np.linalg.norm(w)
        assert np.linalg.norm(err) <= 2.0 ** -8 * norm
        return want


CASES = [
    # hkv, new tokens, tokens in the cache, rows behind
    (1, [1], [1], 0),
    (2, [1], [17], 0),
    (1, [5], [5], 3),
    (2, [33], [33], 0),                                        # one row more than a stream holds
    (1, [64, 65], [64, 65], 0),
    (2, [7, 1, 30], [526, 1, 100], 0),
    (4, [0, 12, 0, 3, 0], [40, 12, 0, 700, 5], 1),             # requests without rows
    (1, [129, 200], [129, 1003], 0),
    (8, [3] * 20, list(range(3, 63, 3)), 0),
    (2, [300], [2000], 0),
    (1, [1, 2, 31, 32, 34, 63], [128, 129, 256, 255, 384, 4000], 0),
    (16, [70], [90], 0),
    (32, [9, 40], [300, 40], 0),
]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("hkv,new,total,extra", CASES)
def test_chunk(hkv, new, total, extra, causal):
    c = Chunk(hkv, new, total, seed=len(new) + hkv, causal=causal, extra=extra)
    c.run()
    c.check()
    assert moira.read_device_status(c.ws) == 0


@pytest.mark.parametrize("new,total", [([70, 10], [33, 4]), ([40, 200], [0, 17]), ([300], [1])])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing_are_zero(new, total, causal):
    """A cache shorter than the chunk: the first rows of a causal one, or every row over an empty cache."""
    c = Chunk(2, new, total, seed=3, causal=causal)
    c.run()
    want = c.check()
    dead = ~want.any(-1)
    assert dead.any() == (causal or 0 in total)
    assert not u16(c.out)[dead].any()


@pytest.mark.parametrize("new,total", [([3], [9000]), ([64] * 3, [5000, 6100, 8192]), ([1] * 30, [2000 + 37 * i for i in range(30)])])
def test_long_caches_behind_few_rows(new, total):
    """The keys are split over the grid and joined."""
    c = Chunk(2, new, total, seed=8)
    c.run()
    c.check()


def test_a_whole_prompt_of_odd_length():
    c = Chunk(2, [1501, 700], [1501, 900], seed=4)
    c.run()
    c.check()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_a_row_does_not_see_does_not_reach_it(bad):
    """Values and keys that are not finite, on tokens of the chunk itself and before it: only the rows that see them."""
    new, total, at = 90, 300, 250                              # row i sees tokens below 211 + i
    for which in ("v", "k"):
        c = Chunk(1, [new], [total], seed=5)
        clean = c.run().clone()
        page, slot = c.table[0, at // S], at % S
        (c.v if which == "v" else c.k)[page, 0, slot, 7 if which == "v" else slice(None)] = bad
        got = c.run()
        sees = np.arange(new) >= at - (total - new)
        assert torch.equal(got[~sees], clean[~sees])
        hit = ~np.isfinite(bf16_to_f64(u16(got[sees])))
        if which == "v":
            assert hit[:, :, 7].all() and hit.sum() == sees.sum() * G
            if not np.isnan(bad):
                assert (bf16_to_f64(u16(got[sees]))[:, :, 7] == bad).all()
            rest = [i for i in range(D) if i != 7]
            sees_t = torch.from_numpy(sees).cuda()
            assert torch.equal(got[sees_t][:, :, rest], clean[sees_t][:, :, rest])
        elif np.isnan(bad):
            assert hit.all()


def test_large_scores_and_equal_scores():
    """Scores of thousands (one token takes it all) and a cache of one repeated token."""
    c = Chunk(2, [40], [400], seed=6, peak=40.0)
    c.run(scale=2.0)
    want, _ = ref.attend_chunk(u16(c.q), u16(c.k), u16(c.v), c.table, c.lens, c.starts, 2.0, True)
    got = bf16_to_f64(u16(c.out))
    assert np.isfinite(got).all()
    # scores near 2^13 carry fp32 errors near 2^-8: the weights of close rivals are 2^-7 off at most
    assert np.linalg.norm(got - want) <= 2.0 ** -6 * np.linalg.norm(want)
    c = Chunk(1, [50], [200], seed=7)
    c.k[...] = c.k[c.table[0, 0], 0, 0]
    c.run()
    c.check()


def test_pages_outside_the_pool_are_skipped_and_lengths_clamped():
    c = Chunk(2, [20, 20, 9], [300, 333, 100], seed=9)
    c.table[0, 3], c.table[1, 0], c.table[1, 20], c.table[2, 1] = -1, c.P, 2 ** 31 - 1, c.P - 2
    c.table[2, 1] = -5
    c.run()
    c.check()
    assert moira.read_device_status(c.ws) == moira.DEV_BADPAGE
    c = Chunk(1, [20, 20, 5], [50, 64, 64], seed=10, mp=4)
    clean = c.run().clone()
    c.lens[1], c.lens[2] = 1000, -3                            # 1000 counts as the table's 64
    got = c.run()
    assert torch.equal(got[:40], clean[:40]) and not got[40:].any()
    assert moira.read_device_status(c.ws) == moira.DEV_BADLEN


@pytest.mark.parametrize("starts", [[0, 10, 5, 30], [-7, 3, 3, 1000], [40, 30, 20, 10], [0, 2 ** 31 - 1, 2 ** 31 - 1, -2 ** 31]])
def test_bad_starts_stay_in_bounds(starts):
    c = Chunk(1, [10, 10, 10], [40, 80, 300], seed=11)
    big = torch.full((c.tokens + 64, G, D), 5.0, dtype=torch.bfloat16, device="cuda")
    c.starts = np.asarray(starts, np.int64).astype(np.int32)
    c.run(out=big[32:32 + c.tokens])
    torch.cuda.synchronize()
    assert bool((big[:32] == 5).all()) and bool((big[32 + c.tokens:] == 5).all())


def test_no_tokens_and_wrong_tensors():
    c = Chunk(2, [0, 0], [10, 20])
    c.run()
    c = Chunk(2, [4], [40])
    args = [c.shape, c.q, c.k, c.v, dev(c.table), dev(c.lens), dev(c.starts), SCALE, c.out, c.ws]
    for i, wrong, kind in ((1, c.q.float(), TypeError), (1, c.q[:, :4], ValueError), (2, c.k[:-1], ValueError),
                           (4, dev(c.table).long(), TypeError), (6, dev([0, 4, 4]), ValueError), (8, c.out.float(), TypeError),
                           (8, c.out[:, ::2], ValueError), (9, c.ws[:16], moira.MoiraError), (5, torch.tensor([40]), TypeError)):
        bad = list(args)
        bad[i] = wrong
        with pytest.raises(kind):
            moira.attend_chunk(*bad)


def test_equal_calls_give_equal_bits_and_workspaces_serve_other_sizes():
    """One workspace for calls of several sizes and for the selection's and the attention's own, in turn; the same bits
    each time, from a captured graph and from another stream too."""
    a, b = Chunk(2, [300, 5], [1700, 8000], seed=12), Chunk(2, [1] * 9, [999] * 9, seed=13, causal=False)
    for c in (a, b):
        c.run()
        c.check()
    n = max(a.ws.numel(), b.ws.numel(), moira.workspace_bytes(a.shape, 2, a.mp))
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:n]
    moira.workspace_init(ws)
    outs = [torch.empty_like(a.out), torch.empty_like(b.out)]
    q1 = a.q[:2].contiguous()
    summ = moira.make_summaries(a.shape)
    lists = torch.zeros((2, 2, a.mp), dtype=torch.int32, device="cuda")
    lengths = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    att = [torch.empty((2, 8, D), device="cuda") for _ in range(3)]
    for i in range(3):
        for c, o in zip((a, b), outs):
            c.run(out=o, ws=ws)
            assert torch.equal(o, c.out)
        moira.select_attend(a.shape, q1, summ, a.k, a.v, dev(a.table), dev(a.lens), 1.0, SCALE, lists, lengths, att[i], ws)
    assert torch.equal(att[0], att[1]) and torch.equal(att[0], att[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs[0].zero_()
    torch.cuda.synchronize()
    a.run(out=outs[0], stream=side)
    side.synchronize()
    assert torch.equal(outs[0], a.out)
    g = torch.cuda.CUDAGraph()
    t, l, s = dev(a.table), dev(a.lens), dev(a.starts)
    with torch.cuda.graph(g):
        moira.attend_chunk(a.shape, a.q, a.k, a.v, t, l, s, SCALE, outs[0], ws)
    for _ in range(3):
        outs[0].zero_()
        g.replay()
        assert torch.equal(outs[0], a.out)
    assert moira.read_device_status(ws) == 0
