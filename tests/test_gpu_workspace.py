"""One workspace for calls of several functions and sizes, one after another:
each gives what it gives on a workspace of its own, bit for bit."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S, G, H = 128, 16, 4, 8
SCALE = 1.0 / np.sqrt(D)


class Layer:
    """One layer of `batch` requests with tables of `pages` pages; the first request fills its table."""

    def __init__(self, batch, pages, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        P = batch * pages
        self.pages, self.batch = pages, batch
        self.shape = moira.Shape.of(G * H, H, P)
        self.k, self.v = (torch.randn((P, H, S, D), generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
        self.q = torch.randn((batch, G * H, D), generator=gen, device="cuda").to(torch.bfloat16)
        self.table = torch.from_numpy(rng.permutation(P).astype(np.int32).reshape(batch, pages)).cuda()
        lens = rng.integers(1, pages * S + 1, batch)
        lens[0] = pages * S
        self.lens = torch.from_numpy(lens.astype(np.int32)).cuda()
        self.summ = moira.make_summaries(self.shape)
        moira.update_summaries(self.shape, self.k, self.summ, torch.arange(P, dtype=torch.int32, device="cuda"))

    def bytes(self):
        return moira.make_shared_workspace(self.shape, self.batch, self.pages, groups=1, weights=True).numel()

    def run(self, what, ws):
        lists = torch.zeros((self.batch, H, self.pages), dtype=torch.int32, device="cuda")
        lengths = torch.zeros((self.batch, H), dtype=torch.int32, device="cuda")
        out = torch.zeros((self.batch, G * H, D), device="cuda")
        weights = torch.zeros((self.k.shape[0], H, S), device="cuda")
        if what == "fused":
            moira.select_attend(self.shape, self.q, self.summ, self.k, self.v, self.table, self.lens, 0.9, SCALE, lists,
                                lengths, out, ws)
        else:
            moira.select(self.shape, self.q, self.summ, self.table, self.lens, 0.9, SCALE, lists, lengths, ws)
            if what == "attend":
                moira.attend(self.shape, self.q, self.k, self.v, lists, lengths, self.lens, self.pages, SCALE, out, ws)
            else:
                i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
                groups = self.table[:1], i32(self.pages * S), i32(0, self.batch)
                moira.attend_shared(self.shape, self.q, self.k, self.v, *groups, lists, lengths, self.lens, self.pages,
                                    SCALE, out, ws, weights=weights)
        keep = torch.arange(self.pages, device="cuda") < lengths.unsqueeze(-1)
        return torch.where(keep, lists, -1), lengths, out, weights


def test_calls_of_several_functions_and_sizes_share_a_workspace():
    layers = [Layer(1, 2048, 1), Layer(4, 64, 2), Layer(1, 40, 3), Layer(20, 200, 4), Layer(2, 1000, 5)]
    assert moira.select_attend_is_fused(layers[0].shape, 1, 2048)
    ws = torch.empty(max(l.bytes() for l in layers) + 256, dtype=torch.uint8, device="cuda")
    ws = ws[-ws.data_ptr() % 256:][:ws.numel() - 256]
    moira.workspace_init(ws)
    want = {}
    for i, l in enumerate(layers):
        for what in ("fused", "attend", "shared"):
            own = moira.make_shared_workspace(l.shape, l.batch, l.pages, groups=1, weights=True)
            want[i, what] = l.run(what, own)
            assert moira.read_device_status(own) == 0
    order = np.random.default_rng(0)
    for step in range(60):
        i, what = int(order.integers(len(layers))), ("fused", "attend", "shared")[order.integers(3)]
        got = layers[i].run(what, ws)
        assert all(torch.equal(a, b) for a, b in zip(got, want[i, what])), (step, i, what)
    assert moira.read_device_status(ws) == 0
