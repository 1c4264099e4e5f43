"""The plain eviction that the GPU tests compare with, on a case worked out by
hand."""
import numpy as np

from tests import cache_reference as ref


def test_the_heaviest_token_and_the_newest_move_into_the_first_slots():
    """40 tokens on pages 2, 0, 1 cut to 5, the newest protected.  Weights: tokens 0 to 2 have 5, token 23 (page 0,
    slot 7) has 9, the rest none.  So 0, 1, 2, 23 and 39 stay, slots 3 and 4 are free, and the movers 23 and 39 take
    them in order."""
    rng = np.random.default_rng(0)
    k, v = (rng.integers(0, 1 << 16, (3, 1, 16, 128)).astype(np.uint16) for _ in range(2))
    w = np.zeros((3, 1, 16), np.float32)
    pos = np.full((3, 1, 16), -1, np.int32)
    w[2, 0, :3], w[0, 0, 7] = 5.0, 9.0
    k0, v0 = k.copy(), v.copy()
    new, renewed = ref.evict(k, v, w, pos, np.array([[2, 0, 1]], np.int32), [40], 5, 0, 1)
    assert new.tolist() == [5] and renewed == []
    assert pos[2, 0].tolist() == [0, 1, 2, 23, 39] + [-1] * 11 and (pos[[0, 1]] == -1).all()
    assert w[2, 0].tolist() == [5, 5, 5, 9, 0] + [0] * 11 and not w[[0, 1]].any()
    for x, x0 in ((k, k0), (v, v0)):
        assert np.array_equal(x[2, 0, 3], x0[0, 0, 7]) and np.array_equal(x[2, 0, 4], x0[1, 0, 7])
        x[2, 0, 3:5] = x0[2, 0, 3:5]
        assert np.array_equal(x, x0)                             # no other row changed


def test_equal_weights_keep_the_lower_slots():
    """40 tokens without weights cut to 5, the newest protected: 0 to 3 stay where they are, 39 takes slot 4."""
    k = np.arange(3 * 16 * 128, dtype=np.uint16).reshape(3, 1, 16, 128)
    w = np.zeros((3, 1, 16), np.float32)
    pos = np.full((3, 1, 16), -1, np.int32)
    ref.evict(k, k.copy(), w, pos, np.array([[2, 0, 1]], np.int32), [40], 5, 0, 1)
    assert pos[2, 0, :5].tolist() == [0, 1, 2, 3, 39]
