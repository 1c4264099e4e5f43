"""Shared-prefix attention where one block takes many key tiles of one unit:
accumulators that join their partial in the middle, rising maxima, missing
pages far into a share, the ring of key masks going round.

The 64-bit form runs on the GPU here, a prefix of 128k tokens at a time.

Tolerances.  Element by element as in test_gpu_shared.py (ELEM of sum p |v|).
Over a row, in relative L2, the terms' errors are independent and add like the
terms themselves, so their root mean square counts:
  own lists: a logit (|s| mostly below 8 in the log2 domain) rounds 11 times in
  fp32, 8 * sqrt(11 / 3) * 2^-24 * ln 2 = 6.3e-7; the exponential 2^-22 at
  most, 1e-7; P keeps 24 bits and the sums are fp32: below 1e-6, OWN = 1.5e-6.
  prefixes: besides, P keeps 16 bits, at most 2^-18 = 3.8e-6 and 1.3e-6 in root
  mean square; the tensor cores truncate, 1.7e-8 of the accumulator per 16-key
  step and half of P: over chains of 8 tiles (128 steps) 2.2e-6 at most.  With
  the own lists' share, sqrt(1^2 + 1.3^2) + 2.2 = 3.8e-6, PREFIX = 5e-6.  (An
  accumulator that never joins drifts by 1.5e-5 on 128k tokens.)
"""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from tests.test_gpu_shared import Case, ELEM, G, D, S, SCALE, pages_of
from tests.helpers import out_errors

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

OWN, PREFIX = 1.5e-6, 5e-6


def exact(c):
    """(out, sum p |v|) of a Case in fp64 on the GPU; prefix pages outside the pool drop their tokens."""
    out = torch.zeros((c.B, G * c.H, D), dtype=torch.float64, device="cuda")
    size = torch.zeros_like(out)
    q = c.q.double()
    P = c.k.shape[0]
    for j in range(c.H):
        heads = slice(j * G, (j + 1) * G)
        for g, plen in enumerate(c.plens):
            a, b = int(c.starts[g]), int(c.starts[g + 1])
            if a == b:
                continue
            pages = c.prefix_table[g, :pages_of(plen)]
            live = np.repeat((pages >= 0) & (pages < P), S)[:plen]
            idx = torch.from_numpy(np.where((pages >= 0) & (pages < P), pages, 0).astype(np.int64)).cuda()
            k, v = (x[idx, j].reshape(-1, D)[:plen][torch.from_numpy(live).cuda()].double() for x in (c.k, c.v))
            rows = q[a:b, heads].reshape(-1, D)
            s = rows @ k.T * SCALE
            for r in range(a, b):                              # the own tokens join the row's softmax
                n, rr = int(c.lens[r]), slice((r - a) * G, (r - a + 1) * G)
                ln = int(c.lengths[r, j])
                n = ln * S - (S - n % S if ln and n % S else 0)
                own = torch.from_numpy(c.lists[r, j, :ln].astype(np.int64)).cuda()
                ok, ov = (x[own, j].reshape(-1, D)[:n].double() for x in (c.k, c.v))
                p = torch.softmax(torch.cat([s[rr], q[r, heads] @ ok.T * SCALE], 1), 1)
                vv = torch.cat([v, ov])
                out[r, heads], size[r, heads] = p @ vv, p @ vv.abs()
    return out.cpu().numpy(), size.cpu().numpy()


def check(c, elem=ELEM, row=PREFIX, status=0):
    c.upload(weights=False)
    c.run()
    torch.cuda.synchronize()
    assert moira.read_device_status(c.ws) == status
    out, size = exact(c)
    got = c.out.cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    assert np.all(np.abs(got - out) <= elem * size), np.max(np.abs(got - out) / np.maximum(size, 1e-30))
    if row is not None:
        assert out_errors(got, out)[1] <= row


# requests: rows of a unit are 4 times as many; tiles a block takes of one unit in brackets
CASES = [
    (8, 8, 131072 + 5),              # 32 rows, both streams on the same rows (54)
    (8, 40, 65536 + 77),             # 160 rows, a stream each (27)
    (4, 70, 65536 - 3),              # 280 rows: teams of two, the second's 24 rows in both streams (27)
    (1, 130, 131072),                # 520 rows: teams of three (20)
]


@pytest.mark.parametrize("hkv,batch,plen", CASES)
def test_long_shares(hkv, batch, plen):
    check(Case(hkv, [0, batch], [plen], [(7 * r) % 23 for r in range(batch)], seed=batch))


@pytest.mark.parametrize("hkv,batch,plen", CASES)
def test_rising_maxima_within_a_share(hkv, batch, plen):
    """Logits that climb by 5 a tile to 160 and start again: within a share the maximum passes its reference over
    and over, and the partial's by more than 2^60.  A logit of 160 in the log2 domain is off by 11 * 160 * 2^-24,
    7.3e-5 of e^s: less than ELEM besides ELEM."""
    c = Case(hkv, [0, batch], [plen], [(7 * r) % 23 for r in range(batch)], seed=batch + 1)
    c.q[..., 0] = 8.0
    unit = np.log(2.0) / (8.0 * SCALE)                         # of k[..., 0], for a step of 1 in the log2 domain
    tile = np.arange(pages_of(plen) * S) // 128
    level = torch.from_numpy((5.0 * (tile % 33) * unit).astype(np.float32)).to(torch.bfloat16).cuda()
    c.k[torch.from_numpy(c.prefix_table[0].astype(np.int64)).cuda(), :, :, 0] = level.view(-1, 1, S)
    check(c, elem=2 * ELEM, row=None)


@pytest.mark.parametrize("hkv,batch,plen", CASES)
def test_pages_missing_far_into_a_share(hkv, batch, plen):
    """Pages outside the pool, alone, in whole tiles and at the end, all over the prefix."""
    c = Case(hkv, [0, batch], [plen], [(7 * r) % 23 for r in range(batch)], seed=batch + 2)
    n = pages_of(plen)
    rng = np.random.default_rng(batch)
    c.prefix_table[0, rng.integers(0, n, n // 50)] = -1
    for t in rng.integers(0, n // 8, n // 100):
        c.prefix_table[0, 8 * t:8 * t + 8] = c.k.shape[0]
    c.prefix_table[0, n - 1] = -7
    check(c, status=moira.DEV_BADPAGE)


def test_a_share_across_units_of_several_groups():
    """Blocks whose shares end in one unit and go on in the next, narrow and wide ones in turn."""
    sizes, plens = [3, 50, 1, 60, 8], [40000, 20011, 33333, 9000, 50000]
    check(Case(8, np.concatenate([[0], np.cumsum(sizes)]), plens, [(5 * r) % 40 for r in range(sum(sizes))], seed=3))


@pytest.mark.parametrize("hkv,lens", [(8, [20000]), (4, [3000, 1, 700, 16]), (8, [100 * i + 1 for i in range(12)])])
def test_own_lists_to_fp32(hkv, lens):
    """As near to the definition as an fp32 computation (no prefix)."""
    c = Case(hkv, [0, len(lens)], [0], lens, seed=len(lens))
    check(c, row=OWN)
