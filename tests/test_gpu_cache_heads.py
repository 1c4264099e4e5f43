"""16 and 32 KV heads: the cache operators, and the selection and attention they
stand beside."""
import numpy as np
import pytest
import torch

from tests.test_gpu_evict import Cache, FMTS
from tests.test_gpu_shapes import test_kv_head_counts_formats_and_launch_shapes as check_select_and_attend
from tests.test_gpu_shared import Case

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


@pytest.mark.parametrize("hkv", [16, 32])
@pytest.mark.parametrize("starts,plens,lens", [
    ([0, 2], [300], [33, 7]), ([0, 0, 40, 41], [70, 129, 0], [r % 37 for r in range(41)]),
    ([0, 65], [500], [1 + r % 3 for r in range(65)]),                # two row tiles: teams
])
def test_shared_attention(hkv, starts, plens, lens):
    Case(hkv, starts, plens, lens, seed=hkv).check()


@pytest.mark.parametrize("hkv", [16, 32])
def test_attention_weights(hkv):
    Case(hkv, [0], [], [200, 0, 1, 777], keep=0.5, seed=hkv).check()


def test_as_many_lists_as_there_may_be():
    rng = np.random.default_rng(0)
    Case(32, [0], [], [int(x) for x in rng.integers(0, 40, 128)], seed=1).check()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hkv", [16, 32])
@pytest.mark.parametrize("lens,budget", [([130, 60, 200], 96), ([80] * 20, 70), ([4000], 1000)])
def test_evict(hkv, fmt, lens, budget):
    _, renewed = Cache(hkv, -(-max(lens) // 16), lens, seed=hkv, fmt=fmt).check(budget, 3, budget // 2)
    assert renewed


@pytest.mark.parametrize("persistent", [False, True])
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("hkv", [16, 32])
def test_selection_and_attention(hkv, fmt, persistent):
    check_select_and_attend(hkv, fmt, persistent)
