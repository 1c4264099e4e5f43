"""Eviction in several layers that share their requests' lengths."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from tests import cache_reference as ref
from tests.helpers import u16

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S = 128, 16


@pytest.mark.parametrize("in_place", [False, True])
def test_every_layer_is_cut_to_the_same_lengths(in_place):
    """The new lengths go to their own tensor until the last layer; there they may replace the old ones."""
    L, H, B, mp, budget = 3, 2, 3, 8, 64
    P = B * mp
    shape = moira.Shape.of(4 * H, H, P)
    rng = np.random.default_rng(0)
    table = rng.permutation(P).astype(np.int32).reshape(B, mp)
    lens = np.array([100, 128, 40], np.int32)
    gen = torch.Generator(device="cuda").manual_seed(0)
    k, v = (torch.randn((L, P, H, S, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    weights, positions = moira.make_token_state(shape, layers=L)
    weights.uniform_(generator=gen)
    summ = torch.stack([moira.make_summaries(shape) for _ in range(L)])
    host = [[u16(k[l]).copy(), u16(v[l]).copy(), weights[l].cpu().numpy(), positions[l].cpu().numpy()] for l in range(L)]
    sl, pt = torch.from_numpy(lens).cuda(), torch.from_numpy(table).cuda()
    new_lens = torch.zeros_like(sl)
    ws = moira.make_evict_workspace(shape, B, mp)
    for l in range(L):
        moira.evict(shape, k[l], v[l], summ[l], weights[l], positions[l], pt, sl, budget, 2, 20,
                    sl if in_place and l == L - 1 else new_lens, ws)
    if not in_place:
        sl.copy_(new_lens)
    assert moira.read_device_status(ws) == 0
    assert sl.tolist() == [64, 64, 40]
    for l, (hk, hv, hw, hp) in enumerate(host):
        ref.evict(hk, hv, hw, hp, table, lens, budget, 2, 20)
        assert np.array_equal(u16(k[l]), hk) and np.array_equal(u16(v[l]), hv), l
        assert np.array_equal(weights[l].cpu().numpy(), hw) and np.array_equal(positions[l].cpu().numpy(), hp), l
