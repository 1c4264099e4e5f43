"""Keys and values that are not finite, on tokens that only some rows see, where
the attention of a chunk takes them on different ways: wide and narrow tiles,
tiles split between blocks and joined by the last of them or by a launch of
its own, many tiles a block.

A value that is not finite reaches its own column of the rows that see it and
nothing else, so everything else is equal bit for bit to the call without it.
With an infinite key a row's score is +inf (its output is NaN: infinity over
infinity) or -inf (as if the token were not there), within the tolerance of
tests/test_gpu_chunk.py."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from tests import token_reference as ref
from tests.cache_reference import bf16_to_f64
from tests.helpers import u16
from tests.test_gpu_chunk import SCALE, Chunk

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S, G = 128, 16, 4
INF, NAN = float("inf"), float("nan")

CASES = {
    "narrow": (1, [20], [300]),
    "narrow, two key tiles": (2, [17, 30], [140, 250]),
    "no more tokens than rows": (1, [90], [90]),
    "one wide tile, joined by a launch of its own": (1, [64], [9000]),
    "one narrow tile, the same": (1, [20], [9000]),
    "wide tiles of a few parts": (2, [64, 50], [3000, 2500]),
    "a wide tile of many parts among short requests": (1, [64] + [1] * 80, [9000] + [40] * 80),
    "a narrow tile of many parts among short requests": (1, [2] * 80 + [20], [40] * 80 + [9000]),
    "many requests a block": (4, [3, 7, 40, 1, 12, 65] * 8, [50, 7, 290, 130, 500, 1000] * 8),
    "prompts, many tiles a block": (8, [400] * 4, [400, 500, 601, 700]),
}


def sees(c, r, token):
    """Rows of q that see the request's token."""
    lo, hi = int(c.starts[r]), int(c.starts[r + 1])
    first = max(0, token - (int(c.lens[r]) - (hi - lo))) if c.causal else 0
    return slice(lo + first, hi)


def places(c, rng, n):
    """(request, token, KV head) of n tokens that some row of the request does not see, or any where there is none."""
    new = np.diff(c.starts)
    wide = [r for r in range(c.B) if new[r] > 1 and c.lens[r] > 1]
    out = set()
    for _ in range(50 * n):
        r = int(rng.choice(wide))
        out.add((r, int(rng.integers(max(1, c.lens[r] - new[r] + 1), c.lens[r])), int(rng.integers(c.hkv))))
        if len(out) == n:
            break
    return sorted(out)


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("many", [False, True])
def test_values_that_are_not_finite(name, many):
    c = Chunk(*CASES[name], seed=21)
    clean = u16(c.run())
    want, is_nan = clean.copy(), np.zeros(clean.shape, bool)
    rng = np.random.default_rng(22)
    plus, minus = np.zeros(clean.shape, bool), np.zeros(clean.shape, bool)
    for i, (r, t, j) in enumerate(places(c, rng, 12 if many else 1)):
        d, bad = int(rng.integers(D)), (INF, -INF, NAN)[i % 3]
        c.v[int(c.table[r, t // S]), j, t % S, d] = bad
        at = (sees(c, r, t), slice(j * G, (j + 1) * G), d)
        (is_nan if np.isnan(bad) else plus if bad > 0 else minus)[at] = True
    is_nan |= plus & minus
    want[plus], want[minus] = 0x7F80, 0xFF80
    got = u16(c.run())
    assert (plus | minus | is_nan).any() and not (plus | minus | is_nan).all()
    assert np.isnan(bf16_to_f64(got[is_nan])).all()
    assert np.array_equal(got[~is_nan], want[~is_nan])
    assert moira.read_device_status(c.ws) == 0


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
def test_keys_that_are_not_finite(name, bad):
    c = Chunk(*CASES[name], seed=23)
    clean = u16(c.run())
    rng = np.random.default_rng(24)
    seen = np.zeros(clean.shape[:2], bool)
    for r, t, j in places(c, rng, 2):
        c.k[int(c.table[r, t // S]), j, t % S, int(rng.integers(D))] = bad
        seen[sees(c, r, t), j * G:(j + 1) * G] = True
    got = u16(c.run())
    assert seen.any() and not seen.all()
    assert np.array_equal(got[~seen], clean[~seen])
    want, size = ref.attend_chunk(u16(c.q), u16(c.k), u16(c.v), c.table, c.lens, c.starts, SCALE, True)
    g, w, z = bf16_to_f64(got[seen]), want[seen], size[seen]
    dead = np.isnan(w).all(-1)
    assert np.array_equal(np.isnan(w).any(-1), dead) and (dead.all() or not np.isnan(bad))
    assert np.isnan(g[dead]).all()
    g, w, z = g[~dead], w[~dead], z[~dead]
    assert np.all(np.abs(g - w) <= 2.0 ** -8 * np.abs(w) + (2.0 ** -8 + 2.0 ** -10) * z + 1e-30)
    assert moira.read_device_status(c.ws) == 0
