"""moira_attend_shared and moira_attend_weights against the plain 64-bit form.

Tolerances.  Logits: the 128 products are summed in fp32 in chains of 8 MMA
steps and scaled once, so with |s| <= 64 in the log2 domain a logit is off by
at most 11 roundings of 2^-24 * 64, 4.2e-5 (times ln 2 as a relative error of
e^s: 2.9e-5).  P enters as bf16 plus bf16 residual: at most half a step of
half a step, 2^-18.  The fp32 sums over a chain of a few hundred adds: a few
hundred times 2^-24, 3e-5.  Together below 2^-13 of sum_t p_t |v_t| for every
element, which also bounds a weight's relative error.  Over a row the terms'
errors are independent and add in quadrature, like the terms of random values
themselves, and the largest logits (near 64) are rare: the row's relative L2
stays below 2e-5.
"""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from tests import cache_reference as ref
from tests.helpers import out_errors, u16

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S, G = 128, 16, 4
ELEM, ROW = 2.0 ** -13, 2e-5
SCALE = 1.0 / np.sqrt(D)


def pages_of(n):
    return -(-n // S)


class Case:
    """Random pools, prefixes and own lists; `keep` < 1 lists a random part of the full pages."""

    def __init__(self, hkv, starts, plens, lens, keep=1.0, seed=0, spare=3):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.H = len(lens), hkv
        self.mp = max(1, max(pages_of(n) for n in lens))
        need = [pages_of(p) for p in plens]
        P = sum(pages_of(n) for n in lens) + sum(need) + spare
        perm = rng.permutation(P).astype(np.int32)
        self.shape = moira.Shape.of(G * hkv, hkv, P)
        self.k = torch.randn((P, hkv, S, D), generator=gen, device="cuda").to(torch.bfloat16)
        self.v = torch.randn((P, hkv, S, D), generator=gen, device="cuda").to(torch.bfloat16)
        self.q = torch.randn((self.B, G * hkv, D), generator=gen, device="cuda").to(torch.bfloat16)
        self.prefix_table = np.full((max(1, len(plens)), max([1] + need)), -1, np.int32)
        at = 0
        for g, n in enumerate(need):
            self.prefix_table[g, :n] = perm[at:at + n]
            at += n
        self.starts, self.plens = np.asarray(starts, np.int32), np.asarray(plens, np.int32)
        self.lens = np.asarray(lens, np.int32)
        self.lists = np.full((self.B, hkv, self.mp), -1, np.int32)
        self.lengths = np.zeros((self.B, hkv), np.int32)
        for r, n in enumerate(lens):
            own = perm[at:at + pages_of(n)]
            at += pages_of(n)
            for j in range(hkv):
                full = np.flatnonzero(rng.random(n // S) < keep) if keep < 1 else np.arange(n // S)
                idx = np.concatenate([full, [n // S]]).astype(int) if n % S else full
                self.lists[r, j, :len(idx)] = own[idx]
                self.lengths[r, j] = len(idx)

    def dev(self, x):
        return torch.from_numpy(np.ascontiguousarray(x)).cuda()

    def upload(self, weights=True):
        self.d = {n: self.dev(getattr(self, n)) for n in
                  ("prefix_table", "plens", "starts", "lists", "lengths", "lens")}
        self.out = torch.full((self.B, G * self.H, D), float("nan"), device="cuda")
        self.ws = moira.make_shared_workspace(self.shape, self.B, self.mp, groups=len(self.plens), weights=weights)

    def run(self, weights=None):
        d = self.d
        if len(self.plens):
            moira.attend_shared(self.shape, self.q, self.k, self.v, d["prefix_table"], d["plens"], d["starts"],
                                d["lists"], d["lengths"], d["lens"], self.mp, SCALE, self.out, self.ws,
                                weights=weights)
        else:
            moira.attend_weights(self.shape, self.q, self.k, self.v, d["lists"], d["lengths"], d["lens"], self.mp,
                                 SCALE, weights, self.out, self.ws)

    def want(self, weights=None):
        return ref.attend_shared(u16(self.q), u16(self.k), u16(self.v), self.prefix_table, self.plens, self.starts,
                                 self.lists, self.lengths, self.lens, SCALE,
                                 None if weights is None else weights.cpu().numpy())

    def check(self, status=0, weights=True):
        self.upload(weights=weights)
        w0 = torch.rand((self.k.shape[0], self.H, S), device="cuda") * 0.01 if weights else None
        w = w0.clone() if weights else None
        self.run(w)
        torch.cuda.synchronize()
        assert moira.read_device_status(self.ws) == status
        out, size, ww = self.want(w0)
        got = self.out.cpu().numpy().astype(np.float64)
        assert np.isfinite(got).all()
        assert np.all(np.abs(got - out) <= ELEM * size), np.max(np.abs(got - out) / np.maximum(size, 1e-30))
        assert out_errors(got, out)[1] <= ROW
        if weights:
            g = w.cpu().numpy().astype(np.float64)
            assert np.all(np.abs(g - ww) <= ELEM * (ww - w0.cpu().numpy()) + 2.0 ** -23 * np.abs(ww))
        return got


@pytest.mark.parametrize("hkv,starts,plens,lens", [
    (2, [0, 3], [40], [5, 17, 33]),                       # small, odd sizes, page tails
    (1, [0, 1], [1], [1]),                                # one token each
    (8, [0, 33], [1000], [1 + 13 * i for i in range(33)]),   # just over 128 query rows
    (2, [0, 32], [129], [16] * 32),                       # exactly 128 rows, one key over a tile
    (4, [0, 70], [300], [1 + i for i in range(70)]),      # over 256 rows: two row tiles
    (2, [0, 200], [2085], [3] * 200),                     # four row tiles
    (2, [0, 2, 2, 7], [50, 999, 77], [9, 0, 64, 31, 0, 100, 2]),   # an empty group, empty own parts
    (4, [1, 4, 6], [0, 260], [30, 16, 0, 5, 47, 33, 18]),          # requests of no group, an empty prefix
    (8, [0, 2], [128 * 40 + 3], [0, 0]),                  # prefixes only
    (1, [0, 3], [16 * 300], [4000, 1, 900]),
])
@pytest.mark.parametrize("weights", [True, False])
def test_shared_attention_matches_the_plain_form(hkv, starts, plens, lens, weights):
    Case(hkv, starts, plens, lens, seed=hkv + len(lens)).check(weights=weights)


@pytest.mark.parametrize("groups", [33, 100, 256])
def test_many_groups(groups):
    """One to three requests a group, prefixes from none to a few pages."""
    rng = np.random.default_rng(groups)
    sizes = rng.integers(0, 3, groups)
    starts = np.concatenate([[0], np.cumsum(sizes)])
    lens = rng.integers(0, 40, max(1, int(starts[-1])))
    Case(1, starts, rng.integers(0, 90, groups), [int(x) for x in lens], seed=groups).check()


@pytest.mark.parametrize("batch,plen", [(2100, 300), (520, 700), (130, 1000)])
def test_more_row_tiles_than_a_team(batch, plen):
    """33, 9 and 3 row tiles: teams of seven in five rounds (two members idle in the last), of five in two (one
    idle), of three in one."""
    Case(1, [0, batch], [plen], [r % 4 for r in range(batch)], seed=batch).check(weights=False)


def test_groups_of_unequal_row_tiles():
    """Without a common number of row tiles every block works alone."""
    Case(2, [0, 70, 71, 210], [400, 1500, 260], [1 + r % 5 for r in range(210)], seed=2).check()


@pytest.mark.parametrize("hkv,lens,keep", [(2, [1000], 1.0), (8, [1], 1.0), (1, [0, 7, 16, 5000], 1.0),
                                           (8, [100 * i + 1 for i in range(12)], 0.3), (4, [20000], 0.4)])
def test_attention_weights_match_the_plain_form(hkv, lens, keep):
    Case(hkv, [0], [], lens, keep=keep, seed=len(lens)).check()


def test_output_without_groups_agrees_with_moira_attend():
    """Two roundings of one value: each is within ELEM of it."""
    c = Case(8, [0], [], [300, 5, 2000], keep=0.5, seed=4)
    c.upload()
    c.run(torch.zeros((c.k.shape[0], 8, S), device="cuda"))
    out = torch.empty_like(c.out)
    moira.attend(c.shape, c.q, c.k, c.v, c.d["lists"], c.d["lengths"], c.d["lens"], c.mp, SCALE, out, c.ws)
    torch.cuda.synchronize()
    assert np.all((out - c.out).abs().cpu().numpy() <= 2 * ELEM * c.want()[1])


@pytest.mark.parametrize("batch", [1, 300, 512])
def test_many_lists(batch):
    """Up to the most (request, KV head) lists, most of them of a few pages."""
    rng = np.random.default_rng(batch)
    Case(8, [0], [], [int(x) for x in rng.integers(0, 50, batch)], seed=batch).check()


def test_long_prefix():
    """64k tokens shared by 5 requests: long sums over many splits."""
    Case(2, [0, 5], [65536 + 77], [100, 20, 0, 3, 900], seed=9).check()


def test_garbage_beyond_the_lengths_is_not_read_into_the_result():
    """Rows behind a prefix's or an own part's last token hold NaN and infinity."""
    c = Case(2, [0, 3], [70], [5, 17, 33], seed=3)
    bad = [(c.prefix_table[0, 4], 6)] + [(c.lists[r, 0, pages_of(n) - 1], n % S) for r, n in enumerate(c.lens) if n % S]
    for p, t in bad:
        c.k[p, :, t:] = float("nan")
        c.v[p, :, t:] = float("inf")
    ok = c.k.clone(), c.v.clone()
    c.upload()
    w = torch.zeros((c.k.shape[0], 2, S), device="cuda")
    c.run(w)
    assert torch.isfinite(c.out).all() and torch.isfinite(w).all()
    out, size, ww = c.want(torch.zeros_like(w))
    assert np.all(np.abs(c.out.cpu().numpy() - out) <= ELEM * size)
    assert torch.equal(c.k.view(torch.int16), ok[0].view(torch.int16))
    for p, t in bad[1:]:
        assert not w[p, :, t:].any()                       # rows behind the last token keep their weight


def test_large_logits():
    """Queries and keys whose logits reach hundreds: one token takes the row, and rising maxima along the keys
    make the kernels rescale.  exp2 of a logit of 1000 is off by 11 * 1000 * 2^-24 in the log2 domain."""
    c = Case(1, [0, 2], [600], [40, 200], seed=6)
    ramp = torch.arange(c.k.shape[0], device="cuda").view(-1, 1, 1, 1) / c.k.shape[0]
    c.k = (c.k.float() * (0.5 + 8 * ramp)).to(torch.bfloat16)
    c.q = (c.q.float() * 4).to(torch.bfloat16)
    c.upload(weights=False)
    c.run()
    out, size, _ = c.want()
    assert np.all(np.abs(c.out.cpu().numpy() - out) <= 16 * ELEM * size)


def test_scores_of_minus_infinity_and_nan():
    """A key of -inf in the query's direction drops its token; a NaN key spoils the rows that see it, no others."""
    c = Case(1, [0, 2, 3], [40, 30], [20, 20, 20], seed=8)
    c.q = c.q.abs() + 0.1                                    # every query has the same sign everywhere
    c.q = c.q.to(torch.bfloat16)
    c.k[c.prefix_table[0, 1], 0, 3] = float("-inf")
    c.k[c.lists[0, 0, 0], 0, 5] = float("-inf")
    c.k[c.prefix_table[1, 0], 0, 0] = float("nan")
    c.upload()
    w = torch.zeros((c.k.shape[0], 1, S), device="cuda")
    c.run(w)
    out, size, ww = c.want(torch.zeros_like(w))
    got = c.out.cpu().numpy()
    assert np.isnan(got[2]).all() and np.isnan(out[2]).all()
    assert np.all(np.abs(got[:2] - out[:2]) <= ELEM * size[:2])
    assert w[c.lists[0, 0, 0], 0, 5] == 0 and torch.isnan(w[c.lists[2, 0, 0], 0]).all()


def test_bad_pages_and_lengths_are_skipped_and_flagged():
    c = Case(2, [0, 3], [100], [5, 40, 33], seed=5)
    c.prefix_table[0, 2] = c.k.shape[0]
    c.lists[1, 1, 0] = -4
    c.check(status=moira.DEV_BADPAGE)
    c = Case(2, [0, 2], [100], [5, 40], seed=5)
    c.upload()
    c.d["plens"].fill_(16 * c.prefix_table.shape[1] + 1)     # clamped to the table
    c.run(torch.zeros((c.k.shape[0], 2, S), device="cuda"))
    assert moira.read_device_status(c.ws) & moira.DEV_BADLEN
    for starts in ([-3, 9], [2, 0], [0, 5]):                 # outside the batch, descending
        c.d["starts"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
        c.d["plens"].fill_(100)
        c.run(torch.zeros((c.k.shape[0], 2, S), device="cuda"))
        assert moira.read_device_status(c.ws) & moira.DEV_BADLEN
    assert torch.isfinite(c.out).all()


def test_bad_list_lengths_are_clamped_and_flagged():
    c = Case(2, [0, 2], [100], [5, 40], seed=5)
    c.upload()
    c.d["lengths"][0, 0] = -3
    c.d["lengths"][1, 1] = c.mp + 7
    c.run(torch.zeros((c.k.shape[0], 2, S), device="cuda"))
    assert moira.read_device_status(c.ws) & moira.DEV_BADLEN
    assert torch.isfinite(c.out).all()
    c.lengths[0, 0], c.lengths[1, 1] = 0, c.mp
    assert np.all(np.abs(c.out.cpu().numpy() - c.want()[0]) <= ELEM * c.want()[1])


def test_shared_call_without_groups():
    c = Case(2, [0], [], [30, 100], seed=6)
    c.upload()
    empty = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    moira.attend_shared(c.shape, c.q, c.k, c.v, empty, empty[:, 0].contiguous(), c.d["starts"], c.d["lists"],
                        c.d["lengths"], c.d["lens"], c.mp, SCALE, c.out, c.ws)
    out, size, _ = c.want()
    assert np.all(np.abs(c.out.cpu().numpy() - out) <= ELEM * size)


def test_two_calls_at_once_on_two_streams():
    """Each with its own workspace, over the same pools."""
    cases = [Case(2, [0, 4], [700], [100, 30, 64, 1], seed=13), Case(4, [0, 40], [900], [9] * 40, seed=14)]
    streams = [torch.cuda.Stream() for _ in cases]
    want = []
    for c in cases:
        c.upload(weights=False)
        c.run()
        want.append(c.out.clone())
    torch.cuda.synchronize()
    for _ in range(5):
        for c in cases:
            c.out.fill_(float("nan"))
        torch.cuda.synchronize()
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                c.run()
        torch.cuda.synchronize()
        for c, w in zip(cases, want):
            assert torch.equal(c.out, w)


def test_a_workspace_without_room_for_the_logits_is_refused():
    c = Case(1, [0], [], [64], seed=3)
    c.upload(weights=False)
    with pytest.raises(moira.MoiraError) as e:
        c.run(torch.zeros((c.k.shape[0], 1, S), device="cuda"))
    assert e.value.status == 2


def test_a_page_listed_for_two_requests_collects_both_shares():
    c = Case(1, [0], [], [32, 32], seed=7)
    c.lists[1, 0, :2] = c.lists[0, 0, :2]
    c.check()


def test_weights_accumulate_and_repeat_bit_for_bit():
    c = Case(2, [0, 4], [500], [100, 30, 64, 1], seed=11)
    c.upload()
    one = torch.zeros((c.k.shape[0], 2, S), device="cuda")
    c.run(one)
    first = c.out.clone()
    two = torch.zeros_like(one)
    c.run(two)
    assert torch.equal(one, two) and torch.equal(first, c.out)
    c.run(two)
    assert torch.equal(two, one + one)


def test_captured_and_replayed_on_a_side_stream():
    c = Case(2, [0, 4], [500], [100, 30, 64, 1], seed=12)
    c.upload()
    w = torch.zeros((c.k.shape[0], 2, S), device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(w)
        want_out, want_w = c.out.clone(), w.clone()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run(w)
    # new values in the same buffers: the graph reads lengths and groups on the device
    for _ in range(2):
        w.zero_()
        c.out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.out, want_out) and torch.equal(w, want_w)
    c.d["plens"].fill_(33)
    c.plens = np.asarray([33], np.int32)
    w.zero_()
    graph.replay()
    torch.cuda.synchronize()
    out, size, ww = c.want(torch.zeros_like(w))
    assert np.all(np.abs(c.out.cpu().numpy() - out) <= ELEM * size)
