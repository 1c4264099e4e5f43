"""Shared-prefix attention where its plan is under strain: groups with empty
prefixes beside large ones, the workspace's end watched."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from tests.test_gpu_shared import Case, ELEM, ROW
from tests.helpers import out_errors

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)


def run_watched(c, behind=64 << 20):
    """Runs the call on a workspace of exactly the stated size, with `behind` bytes after it that must not change."""
    c.upload(weights=False)
    n = c.ws.numel()
    big = torch.full((n + behind + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    off = (-big.data_ptr()) % 256
    c.ws = big[off:off + n]
    moira.workspace_init(c.ws)
    c.run()
    torch.cuda.synchronize()
    assert moira.read_device_status(c.ws) == 0
    assert bool((big[:off] == 0x5A).all()) and bool((big[off + n:] == 0x5A).all())


@pytest.mark.parametrize("hkv,empty,requests,plen", [
    (8, 10, 150, 4200),                   # teams of three
    (4, 3, 300, 2100),                    # of five
    (1, 255, 512, 1000),                  # of eight, as many groups as there may be
    (2, 40, 20, 3000),                    # one row tile: no team
])
def test_empty_prefixes_before_a_large_group(hkv, empty, requests, plen):
    starts = list(range(empty + 1)) + [empty + requests]
    c = Case(hkv, starts, [0] * empty + [plen], [1 + r % 3 for r in range(empty + requests)], seed=empty)
    run_watched(c)
    out, size, _ = c.want()
    got = c.out.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - out) <= ELEM * size) and out_errors(got, out)[1] <= ROW


def test_empty_prefixes_among_large_groups():
    """Two groups of two row tiles with empty prefixes of other sizes before, between and behind them."""
    sizes, plens = [5, 70, 200, 1, 100, 3], [0, 900, 0, 0, 1300, 0]
    c = Case(2, np.concatenate([[0], np.cumsum(sizes)]), plens, [r % 5 for r in range(sum(sizes))], seed=4)
    run_watched(c)
    out, size, _ = c.want()
    got = c.out.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - out) <= ELEM * size) and out_errors(got, out)[1] <= ROW


@pytest.mark.parametrize("starts,plens", [([0, 0], [500]), ([3, 3, 3], [100, 40]), ([0, 0, 2, 2], [300, 0, 70])])
def test_groups_without_requests(starts, plens):
    """Nobody behind a prefix: the own lists alone count."""
    c = Case(2, starts, plens, [40, 0, 7], seed=6)
    run_watched(c)
    out, size, _ = c.want()
    got = c.out.cpu().numpy().astype(np.float64)
    assert np.all(np.abs(got - out) <= ELEM * size) and out_errors(got, out)[1] <= ROW
