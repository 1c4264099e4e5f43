"""The cache operators on pages whose offsets pass 32 bits: the same tokens on
the first pages of a small pool and on the last of a large one give the same
bits."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S, G, H = 128, 16, 4, 8
SCALE = 1.0 / np.sqrt(D)
USED, FAR = 220, 290_000                # pages with tokens; of the large pool: 4.75e9 elements, 9.5 GB


@pytest.fixture(scope="module")
def pools():
    """(near, far): key and value pools whose last USED pages hold the same tokens."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    near = [torch.randn((USED, H, S, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    far = [torch.empty((FAR, H, S, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for a, b in zip(near, far):
        b[-USED:] = a
    assert far[0][:-USED].numel() > 1 << 32
    yield near, far
    del far


def ints(x, offset=0):
    return torch.from_numpy((np.ascontiguousarray(x) + offset).astype(np.int32)).cuda()


def attend(k, v, offset, q, prefix, lists, lengths, lens):
    shape = moira.Shape.of(G * H, H, k.shape[0])
    weights, _ = moira.make_token_state(shape)
    out = torch.empty((len(lens), G * H, D), device="cuda")
    ws = moira.make_shared_workspace(shape, len(lens), lists.shape[-1], groups=1, weights=True)
    moira.attend_shared(shape, q, k, v, ints(prefix, offset), ints([16 * 90 + 3]), ints([0, len(lens)]),
                        ints(lists, offset), ints(lengths), ints(lens), lists.shape[-1], SCALE, out, ws, weights=weights)
    torch.cuda.synchronize()
    assert moira.read_device_status(ws) == 0
    return out, weights[-USED:].clone()


def test_shared_attention_and_weights(pools):
    near, far = pools
    rng = np.random.default_rng(1)
    perm = rng.permutation(USED)
    lens = np.array([16 * 20 + 5, 1, 16 * 30, 0, 700])
    lists = np.zeros((5, H, 44), np.int64)
    lengths = np.zeros((5, H), np.int64)
    at = 91
    for r, n in enumerate(lens):
        cnt = -(-n // S)
        lists[r, :, :cnt], lengths[r] = perm[at:at + cnt], cnt
        at += cnt
    q = torch.randn((5, G * H, D), device="cuda").to(torch.bfloat16)
    args = q, perm[None, :91], lists, lengths, lens
    for a, b in zip(attend(*near, 0, *args), attend(*far, FAR - USED, *args)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("max_pages,lens,budget", [(60, [900, 960, 100], 890), (100, [1600, 1500], 200)])
def test_evict(pools, max_pages, lens, budget):
    """One launch with the moves, and two."""
    near, far = pools
    table = np.random.default_rng(2).permutation(USED)[:len(lens) * max_pages].reshape(len(lens), max_pages)
    gen = torch.Generator(device="cuda").manual_seed(3)
    w0 = torch.rand((USED, H, S), generator=gen, device="cuda")
    got = []
    for (k, v), offset in ((near, 0), (far, FAR - USED)):
        saved = k[-USED:].clone(), v[-USED:].clone()
        shape = moira.Shape.of(G * H, H, k.shape[0])
        weights, positions = moira.make_token_state(shape)
        weights[-USED:] = w0
        summ = torch.zeros((k.shape[0], H, D), dtype=torch.bfloat16, device="cuda")
        new = torch.zeros(len(lens), dtype=torch.int32, device="cuda")
        ws = moira.make_evict_workspace(shape, len(lens), max_pages)
        moira.evict(shape, k, v, summ, weights, positions, ints(table, offset), ints(lens), budget, 2, budget // 2, new, ws)
        torch.cuda.synchronize()
        assert moira.read_device_status(ws) == 0
        assert not weights[:-USED].any() and (positions[:-USED] == -1).all() and not summ[:-USED].any()
        got.append([x[-USED:].clone() for x in (k, v, summ, weights, positions)] + [new])
        k[-USED:], v[-USED:] = saved
    assert not torch.equal(got[0][0], saved[0])
    for a, b in zip(*got):
        assert torch.equal(a, b)
