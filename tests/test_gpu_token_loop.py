"""The operators together, as a server uses them: ragged prompts appended in
pieces with norm and rotation, their attention, decode steps with the selection
and the attention over selected pages, and a cross attention to an encoder's
states; every output against the plain 64-bit forms on the cache of that step."""
import numpy as np
import pytest
import torch

import sparse_long_context_page_gb300 as moira
from tests import cache_reference
from tests import token_reference as ref
from tests.cache_reference import bf16_to_f64
from tests.helpers import MAX_ABS, REL_L2, out_errors, u16

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

D, S, G = 128, 16, 4


@pytest.mark.parametrize("fmt", [moira.SUMM_BF16, moira.SUMM_Q8])
def test_prompts_in_pieces_then_decode_then_cross(fmt):
    H, B, mp = 2, 3, 24
    P = B * mp + B * 8
    shape = moira.Shape.of(G * H, H, P)
    gen = torch.Generator(device="cuda").manual_seed(3)
    rng = np.random.default_rng(3)
    new = lambda *d: torch.randn(d, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x, np.int32)).cuda()  # noqa: E731
    perm = rng.permutation(P).astype(np.int32)
    table, enc_table = perm[:B * mp].reshape(B, mp), perm[B * mp:].reshape(B, 8)
    k, v, summ = new(P, H, S, D), new(P, H, S, D), moira.make_summaries(shape, fmt)
    freq = [10000.0 ** (-i / 64) for i in range(64)]
    rot = moira.make_rotary(freq, [0] * 16 + [1] * 24 + [2] * 24)
    qn, kn = (1 + 0.1 * torch.randn(D, device="cuda") for _ in range(2))
    ws = moira.make_chunk_workspace(shape, B, mp, 400)
    wsd = moira.make_workspace(shape, B, mp)
    scale = 1.0 / np.sqrt(D)
    pt, lens = dev(table), np.zeros(B, np.int32)

    def step(n, out=None):
        """Appends n[r] tokens to each request; (queries, starts)."""
        nonlocal lens
        lens = lens + np.asarray(n, np.int32)
        starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
        T = int(starts[-1])
        rows = new(T, 6 * H, D)
        pos = rng.integers(0, 9000, (3, T)).astype(np.int32)
        q = torch.empty((T, G * H, D), dtype=torch.bfloat16, device="cuda")
        moira.append_rotated(shape, rot, rows[:, :G * H], rows[:, G * H:5 * H], rows[:, 5 * H:], dev(starts), k, v, summ, pt,
                             dev(lens), q, positions=dev(pos), q_norm=qn, k_norm=kn, fmt=fmt)
        want, size = ref.turned(bf16_to_f64(u16(rows[:, G * H:5 * H])), kn.cpu().numpy().astype(np.float64),
                                np.float64(np.float32(1e-6)), freq, [0] * 16 + [1] * 24 + [2] * 24, pos)
        kg = bf16_to_f64(u16(k))
        for r, row, at in ref.request_rows(starts, lens, mp):
            got = kg[table[r, at // S], :, at % S]
            assert np.all(np.abs(got - want[row]) <= 2.0 ** -8 * np.abs(want[row]) + 2.0 ** -18 * size[row])
        return q, starts

    def close(out, want, size):
        got = bf16_to_f64(u16(out))
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -8 + 2.0 ** -10) * size)

    for n in ([70, 33, 129], [5, 40, 1], [64, 0, 100]):        # the prompts, in three pieces
        q, starts = step(n)
        out = torch.empty_like(q)
        moira.attend_chunk(shape, q, k, v, pt, dev(lens), dev(starts), scale, out, ws)
        close(out, *ref.attend_chunk(u16(q), u16(k), u16(v), table, lens, starts, scale, True))
    full = [(r, p) for r in range(B) for p in range(lens[r] // S)]
    fresh = moira.make_summaries(shape, fmt)
    pages = dev([table[r, p] for r, p in full])
    moira.update_summaries(shape, k, fresh, pages, fmt=fmt)
    assert torch.equal(summ[pages.long()], fresh[pages.long()])

    lists = torch.zeros((B, H, mp), dtype=torch.int32, device="cuda")
    lengths = torch.zeros((B, H), dtype=torch.int32, device="cuda")
    att = torch.empty((B, G * H, D), device="cuda")
    enc = [100, 1, 77]                                         # an encoder's states, without rotation or summaries
    enc_starts = np.concatenate([[0], np.cumsum(enc)]).astype(np.int32)
    states = new(int(enc_starts[-1]), 2 * H, D)
    moira.append_rotated(shape, None, None, states[:, :H], states[:, H:], dev(enc_starts), k, v, None, dev(enc_table), dev(enc))
    for _ in range(20):
        q, starts = step([1, 1, 1])
        sl = dev(lens)
        moira.select_ex(shape, fmt, q, summ, pt, sl, moira.RULE_COVERAGE, 0.9, scale, lists, lengths, wsd)
        moira.attend(shape, q, k, v, lists, lengths, sl, mp, scale, att, wsd)
        want, _, _ = cache_reference.attend_shared(u16(q), u16(k), u16(v), np.zeros((0, 1)), [], [0], lists.cpu().numpy(),
                                                   lengths.cpu().numpy(), lens, scale)
        err = out_errors(att.cpu().numpy().astype(np.float64), want)
        assert err[0] <= MAX_ABS and err[1] <= REL_L2
        moira.select_ex(shape, fmt, q, summ, pt, sl, moira.RULE_COVERAGE, 1.0, scale, lists, lengths, wsd)
        moira.attend(shape, q, k, v, lists, lengths, sl, mp, scale, att, wsd)
        out = torch.empty_like(q)                              # one row a request over every page: the dense decode step
        moira.attend_chunk(shape, q, k, v, pt, sl, dev(starts), scale, out, ws)
        want, size = ref.attend_chunk(u16(q), u16(k), u16(v), table, lens, starts, scale, True)
        close(out, want, size)
        assert np.all(np.abs(att.cpu().numpy() - want) <= MAX_ABS)
        moira.rotate_qk(shape, None, q, None, None, q, q_norm=qn)        # the cross attention's queries: norm alone
        moira.attend_chunk(shape, q, k, v, dev(enc_table), dev(enc), dev(starts), scale, out, ws, causal=False)
        close(out, *ref.attend_chunk(u16(q), u16(k), u16(v), enc_table, enc, starts, scale, False))
    assert moira.read_device_status(ws) == 0 and moira.read_device_status(wsd) == 0
