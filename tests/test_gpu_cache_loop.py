"""The cache operators together, as a server uses them: requests behind shared
prompts, one token appended a step, pages selected (or all of them kept),
attention over prompt and own pages with the weights accumulated, eviction
when the own part has grown past its budget.  Every step's output, weights and
eviction are compared with the plain 64-bit forms on the state of that step
(the tolerances are those of test_gpu_shared.py; evictions are exact)."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from oracle import oracle
from tests import cache_reference as ref
from tests.helpers import out_errors, u16

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S, G = 128, 16, 4
ELEM, ROW = 2.0 ** -13, 2e-5


@pytest.mark.parametrize("gamma", [1.0, 0.9])
def test_decode_behind_shared_prompts_with_evictions(gamma):
    H, B, mp, budget, sinks, recent = 2, 5, 8, 64, 2, 24
    starts, plens = [0, 3, 5], [200, 37]
    rng = np.random.default_rng(1)
    gen = torch.Generator(device="cuda").manual_seed(1)
    pre = [-(-p // S) for p in plens]
    P = B * mp + sum(pre) + 2
    shape = moira.Shape.of(G * H, H, P)
    perm = rng.permutation(P).astype(np.int32)
    table = perm[:B * mp].reshape(B, mp)
    prefix = np.full((2, max(pre)), -1, np.int32)
    prefix[0, :pre[0]] = perm[B * mp:B * mp + pre[0]]
    prefix[1, :pre[1]] = perm[B * mp + pre[0]:B * mp + sum(pre)]
    k = torch.randn((P, H, S, D), generator=gen, device="cuda").to(torch.bfloat16)
    v = torch.randn((P, H, S, D), generator=gen, device="cuda").to(torch.bfloat16)
    summ = moira.make_summaries(shape)
    weights, positions = moira.make_token_state(shape)
    moira.update_summaries(shape, k, summ, torch.arange(P, dtype=torch.int32, device="cuda"))
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    pt, pf, pl, gs = dev(table), dev(prefix), dev(plens), dev(starts)
    lens = np.array([60, 100, 0, 1, 33], np.int32)
    sl = dev(lens)
    ws = moira.make_shared_workspace(shape, B, mp, groups=2, weights=True)
    wse = moira.make_evict_workspace(shape, B, mp)
    lists = torch.zeros((B, H, mp), dtype=torch.int32, device="cuda")
    lengths = torch.zeros((B, H), dtype=torch.int32, device="cuda")
    out = torch.empty((B, G * H, D), device="cuda")
    scale = 1.0 / np.sqrt(D)
    evicted = 0
    for step in range(12):
        sl += 1
        lens = lens + 1
        kn, vn, q = (torch.randn((B, n, D), generator=gen, device="cuda").to(torch.bfloat16) for n in (H, H, G * H))
        moira.append_kv(shape, kn, vn, k, v, summ, pt, sl)
        moira.select(shape, q, summ, pt, sl, gamma, scale, lists, lengths, ws)
        w0 = weights.cpu().numpy()
        moira.attend_shared(shape, q, k, v, pf, pl, gs, lists, lengths, sl, mp, scale, out, ws, weights=weights)
        want, size, ww = ref.attend_shared(u16(q), u16(k), u16(v), prefix, plens, starts, lists.cpu().numpy(),
                                           lengths.cpu().numpy(), lens, scale, w0)
        got = out.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - want) <= ELEM * size) and out_errors(got, want)[1] <= ROW, step
        g = weights.cpu().numpy().astype(np.float64)
        assert np.all(np.abs(g - ww) <= ELEM * (ww - w0) + 2.0 ** -23 * np.abs(ww)), step
        if step % 4 == 3:
            hk, hv, hw, hp = u16(k).copy(), u16(v).copy(), weights.cpu().numpy(), positions.cpu().numpy()
            moira.evict(shape, k, v, summ, weights, positions, pt, sl, budget, sinks, recent, sl, wse)
            new, _ = ref.evict(hk, hv, hw, hp, table, lens, budget, sinks, recent)
            evicted += int((lens - new).sum())
            lens = new
            assert np.array_equal(sl.cpu().numpy(), lens)
            assert np.array_equal(u16(k), hk) and np.array_equal(u16(v), hv)
            assert np.array_equal(weights.cpu().numpy(), hw) and np.array_equal(positions.cpu().numpy(), hp)
    assert evicted > 0
    assert moira.read_device_status(ws) == 0 and moira.read_device_status(wse) == 0
    for r in range(B):                                    # the summaries kept up with appends and evictions
        for lp in range(lens[r] // S):
            p = table[r, lp]
            assert np.array_equal(u16(summ[p]), oracle.summaries(u16(k[p]).reshape(-1, S, D)).reshape(H, D)), (r, lp)
