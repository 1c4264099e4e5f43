"""The token operators where their plans and addresses change: many requests,
tiles whose keys many blocks share, rows and pages beyond 2^31 elements, calls
at the same time, workspaces that captured graphs share.

Tolerances are those of the operators' own tests; what only lies elsewhere, or
runs at another time, is equal bit for bit."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from sparse_long_context_page_gb300 import _binding as mb
from tests.test_gpu_chunk import SCALE, Chunk, dev
from tests.test_gpu_rotate import Batch, rotation

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S, G = 128, 16, 4
FAR = 2 ** 31 // (8 * S * D) + 50                              # pages of 8 KV heads: the last ones lie behind 2^31 elements


@pytest.mark.parametrize("batch", [32, 33, 100, 384, 385, 1000, 4096])
@pytest.mark.parametrize("causal", [True, False])
def test_many_requests(batch, causal):
    """A thread of the plan takes one request or several; every third has no rows."""
    rng = np.random.default_rng(batch)
    new = rng.integers(1, 9, batch) * (np.arange(batch) % 3 > 0)
    if batch < 1000:
        new[batch // 2] = 150
    total = new + rng.integers(0, 60, batch)
    c = Chunk(1, list(new), list(total), seed=batch, causal=causal, extra=2)
    c.run()
    c.check()


@pytest.mark.parametrize("hkv,new,total", [
    (2, [64] * 3, [3000, 3100, 2900]),                          # few tiles, a few parts each
    (1, [20], [3000]),
    (1, [3] * 80 + [200], [40] * 80 + [20000]),                 # many tiles, of which some have many parts
    (4, [200] + [1] * 30, [20000] + [17] * 30),
    (1, [1] * 76, [300 + 401 * (i % 7) for i in range(76)]),
    (8, [64, 33, 1], [9000, 9000, 9000]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_tiles_of_many_parts(hkv, new, total, causal):
    c = Chunk(hkv, new, total, seed=len(new), causal=causal)
    first = c.run().clone()
    c.check()
    for _ in range(3):
        c.out.fill_(5.0)
        assert torch.equal(c.run(), first)


@pytest.mark.parametrize("starts", [[0, 0, 0], [7, 7, 7]])
def test_a_batch_without_rows_writes_nothing(starts):
    c = Chunk(2, [0, 0], [30, 0], extra=9)
    c.starts = np.asarray(starts, np.int32)
    c.run()
    assert bool((c.out == 5).all()) and moira.read_device_status(c.ws) == 0


def test_pages_behind_2_to_31_elements():
    c = Chunk(8, [70, 3], [900, 400], seed=2)
    c.run()
    c.check()
    k, v = (torch.empty((FAR, 8, S, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[FAR - c.P:], v[FAR - c.P:] = c.k, c.v
    out = torch.empty_like(c.out)
    moira.attend_chunk(moira.Shape.of(32, 8, FAR), c.q, k, v, dev(c.table + FAR - c.P), dev(c.lens), dev(c.starts), SCALE, out, c.ws)
    assert torch.equal(out, c.out)

    b = Batch(8, [40, 1], [9, 31], seed=3)
    _, _, rot = rotation(64, 1, False)
    summ = moira.make_summaries(moira.Shape.of(32, 8, FAR))
    k[FAR - b.P:], v[FAR - b.P:] = b.k_pool, b.v_pool
    summ[FAR - b.P:] = b.summ
    q_out = torch.full_like(b.q_out, 9.0)
    moira.append_rotated(moira.Shape.of(32, 8, FAR), rot, b.q, b.k, b.v, dev(b.starts), k, v, summ, dev(b.table + FAR - b.P),
                         dev(b.lens), q_out)
    b.append(rot)
    assert torch.equal(k[FAR - b.P:], b.k_pool) and torch.equal(v[FAR - b.P:], b.v_pool)
    assert torch.equal(summ[FAR - b.P:], b.summ) and torch.equal(q_out, b.q_out)


def test_rows_behind_2_to_31_elements():
    T, n = 2 ** 31 // (32 * D) + 200, 100
    c = Chunk(8, [n], [120], seed=4)
    c.run()
    c.check()
    q = torch.empty((T, 32, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    q[T - n:] = c.q
    ws = moira.make_chunk_workspace(c.shape, 1, c.mp, T)
    moira.attend_chunk(c.shape, q, c.k, c.v, dev(c.table), dev(c.lens), dev([T - n, T]), SCALE, out, ws)
    assert torch.equal(out[T - n:], c.out)

    _, _, rot = rotation(64, 1, False)
    pos = torch.arange(T, dtype=torch.int32, device="cuda").view(1, T)
    few = torch.empty_like(c.q)
    moira.rotate_qk(c.shape, rot, c.q, None, pos[:, T - n:].contiguous(), few)
    moira.rotate_qk(c.shape, rot, q, None, pos, out)
    assert torch.equal(out[T - n:], few)


def test_graphs_that_share_a_workspace_and_calls_at_the_same_time():
    a, b = Chunk(2, [300, 5], [1700, 8000], seed=5), Chunk(2, [3], [9000], seed=6)
    tensors = [(dev(c.table), dev(c.lens), dev(c.starts)) for c in (a, b)]
    outs = [torch.empty_like(c.out) for c in (a, b)]
    for c in (a, b):
        c.run()
        c.check()
    big = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    graphs = []
    for c, t, o in zip((a, b), tensors, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            moira.attend_chunk(c.shape, c.q, c.k, c.v, *t, SCALE, o, big)
        graphs.append(g)
    for order in ((0, 1), (1, 0), (0, 0, 1, 1)):
        for o in outs:
            o.zero_()
        for i in order:
            graphs[i].replay()
        assert torch.equal(outs[0], a.out) and torch.equal(outs[1], b.out)
    assert moira.read_device_status(big) == 0
    # both at once, each with its own workspace
    for o in outs:
        o.zero_()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, t, o, s in zip((a, b), tensors, outs, streams):
            moira.attend_chunk(c.shape, c.q, c.k, c.v, *t, SCALE, o, c.ws, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], a.out) and torch.equal(outs[1], b.out)


def test_append_of_many_requests():
    """The largest batch: one token each, and a ragged one."""
    n = 4096
    for new in (np.ones(n, int), np.arange(n) % 4):
        b = Batch(1, new, np.arange(n) % 37, seed=7)
        freq, axis, rot = rotation(64, 1, False)
        b.check(freq, axis, False, 1.0, act=lambda: b.append(rot))


def test_an_append_rotates_queries_as_rotate_qk_does():
    """An append's queries and a rotation in place are the same, which attention may read."""
    b = Batch(2, [50, 1], [0, 20], seed=8)
    _, _, rot = rotation(32, 2, True)
    pos = torch.randint(0, 1000, (2, b.tokens), dtype=torch.int32, device="cuda")
    b.append(rot, positions=pos)
    q = b.q.contiguous()
    moira.rotate_qk(b.shape, rot, q, None, pos, q)
    assert torch.equal(q, b.q_out)


def test_a_captured_call_replays_with_other_rows_and_lengths():
    c = Chunk(2, [90, 70, 1], [2000, 2000, 2000], seed=9, extra=19)
    table, lens, starts = dev(c.table), dev(c.lens), dev(c.starts)
    g = torch.cuda.CUDAGraph()
    c.run()
    with torch.cuda.graph(g):
        moira.attend_chunk(c.shape, c.q, c.k, c.v, table, lens, starts, SCALE, c.out, c.ws)
    for new, total in (([90, 70, 1], [2000, 2000, 2000]), ([1, 1, 178], [1, 1999, 500]), ([0, 0, 3], [700, 3, 3]), ([180, 0, 0], [1, 0, 0])):
        c.starts, c.lens = np.concatenate([[0], np.cumsum(new)]).astype(np.int32), np.asarray(total, np.int32)
        starts.copy_(dev(c.starts))
        lens.copy_(dev(c.lens))
        c.out.fill_(5.0)
        g.replay()
        c.check()
    assert moira.read_device_status(c.ws) == 0


def test_a_workspace_after_a_timeout_ends_its_calls_and_serves_again():
    """A workspace that holds MOIRA_DEV_TIMEOUT: a call gives its waits up, lands its copies and ends; cleared, it is right."""
    c = Chunk(2, [90, 3], [3000, 500], seed=10)
    c.run()
    c.check()
    mb.diag_wait_timeout(c.ws, 1000)
    c.run()
    torch.cuda.synchronize()
    assert moira.read_device_status(c.ws) == mb.DEV_TIMEOUT
    moira.workspace_init(c.ws)
    c.out.fill_(5.0)
    c.run()
    c.check()
    assert moira.read_device_status(c.ws) == 0


def test_outputs_beside_and_between_the_inputs_rows():
    """Outputs that touch the inputs' memory nowhere are taken wherever they lie: between the rows of one arena, in place,
    side by side; the results are those of tensors of their own."""
    H, T = 2, 2
    shape = moira.Shape.of(G * H, H, 1)
    _, _, rot = rotation(64, 1, False)
    pos = dev([[3, 70000]])
    # each token's row: q, k, then room for 20 heads
    arena = torch.randn((T, 30, D), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    q, k = arena[:, :G * H], arena[:, G * H:5 * H]
    want_q, want_k = (torch.empty((T, n, D), dtype=torch.bfloat16, device="cuda") for n in (G * H, H))
    moira.rotate_qk(shape, rot, q, k, pos, want_q, want_k)
    before = arena[:, :5 * H].clone()
    room = arena.view(-1, D)[5 * H:30]
    q_out, k_out = room[:T * G * H].view(T, G * H, D), room[T * G * H:T * 5 * H].view(T, H, D)
    moira.rotate_qk(shape, rot, q, k, pos, q_out, k_out)
    assert torch.equal(q_out, want_q) and torch.equal(k_out, want_k) and torch.equal(arena[:, :5 * H], before)
    both = torch.cat((q.reshape(-1, D), k.reshape(-1, D)))     # in place, one behind the other
    a, b = both[:T * G * H].view(T, G * H, D), both[T * G * H:].view(T, H, D)
    moira.rotate_qk(shape, rot, a, b, pos, a, b)
    assert torch.equal(a, want_q) and torch.equal(b, want_k)
    with pytest.raises(moira.MoiraError):
        moira.rotate_qk(shape, rot, want_q, k, pos, want_q, want_q.view(-1, D)[:T * H].view(T, H, D))


@pytest.mark.parametrize("hkv,new,total", [
    (1, [64], [20000]),                                         # a tile of some 39 parts
    (2, [64], [3600]),                                          # of seven
    (1, [5], [9000]),
    (1, [20, 64, 40], [16000, 2500, 300]),
    (2, [3, 1, 2], [3000, 200, 0]),
])
@pytest.mark.parametrize("wide,rows,idle", [(2000, 0, 0), (0, 6000, 0), (0, 0, 100), (16384, 6000, 100)])
def test_padded_calls_give_the_same_bits(hkv, new, total, wide, rows, idle):
    """The order of the sums goes by the requests' rows and lengths: a wider table, rows behind the last request and
    requests without rows change no bit, whichever way the parts of a tile are joined."""
    c = Chunk(hkv, new, total, seed=14)
    c.run()
    c.check()
    table = np.zeros((c.B + idle, max(c.mp, wide)), np.int32)
    table[:c.B, :c.mp] = c.table
    lens = np.concatenate([c.lens, np.full(idle, 77, np.int32)])
    starts = np.concatenate([c.starts, np.full(idle, c.tokens, np.int32)])
    q = torch.cat((c.q, torch.full((rows, G * hkv, D), 3.0, dtype=torch.bfloat16, device="cuda")))
    out = torch.full_like(q, 5.0)
    ws = moira.make_chunk_workspace(c.shape, *table.shape, len(q))
    moira.attend_chunk(c.shape, q, c.k, c.v, dev(table), dev(lens), dev(starts), SCALE, out, ws)
    assert torch.equal(out[:c.tokens].view(torch.int16), c.out.view(torch.int16)) and bool((out[c.tokens:] == 5).all())
    assert moira.read_device_status(ws) == 0
