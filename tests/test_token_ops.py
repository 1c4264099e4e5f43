"""Host-side checks of the operators that fill the cache and attend to it with
many tokens a request, without a GPU: bad arguments give the documented codes
before any CUDA call (fake pointers, never dereferenced), the binding refuses
wrong tensors, and moira_make_rotary's table is exact."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

import sparse_long_context_page_gb300 as moira
from sparse_long_context_page_gb300 import _binding as mb
from tests import token_reference as ref

FAKE = 0x10000
OK = moira.Shape.of(32, 8, 1024)
# 2 pi to 60 digits
TWO_PI = Fraction("6.283185307179586476925286766559005768394338798750211641949889")


def rotary(**kw):
    r = moira.make_rotary([10000.0 ** (-i / 64) for i in range(64)])
    for name, value in kw.items():
        setattr(r, name, value)
    return r


def rotate(shape=OK, rot=rotary(), q=FAKE, qs=4096, k=FAKE, ks=1024, qn=None, kn=None, eps=1e-6, pos=FAKE, tokens=4,
           qo=FAKE, ko=FAKE):
    return moira.load_library().moira_rotate_qk(ctypes.byref(shape), None if rot is None else ctypes.byref(rot), q, qs, k,
                                                ks, qn, kn, eps, pos, tokens, qo, ko, None)


def bad_axis():
    r = rotary()
    r.axis[7] = 1
    return r


BAD_ROTARIES = [dict(rot=rotary(pairs=62)), dict(rot=rotary(pairs=-4)), dict(rot=rotary(pairs=68)), dict(rot=rotary(axes=0)),
                dict(rot=rotary(axes=5)), dict(rot=rotary(scale=float("inf"))), dict(rot=bad_axis())]


@pytest.mark.parametrize("kw,code", [(x, 1) for x in BAD_ROTARIES] + [
    (dict(q=None, k=None), 1), (dict(qo=None), 1), (dict(ko=None), 1), (dict(pos=None), 1), (dict(tokens=-1), 1),
    (dict(q=FAKE + 8), 1), (dict(k=FAKE + 8), 1), (dict(qs=4095), 1), (dict(qs=4092), 1), (dict(qs=4100), 1), (dict(ks=1020), 1),
    (dict(qo=FAKE + 8), 1), (dict(ko=FAKE + 8), 1), (dict(qn=FAKE + 4), 1), (dict(kn=FAKE + 8), 1), (dict(eps=-1.0), 1),
    (dict(eps=float("nan")), 1), (dict(shape=moira.Shape.of(16, 8, 1024)), 4),
    (dict(shape=moira.Shape.of(32, 8, 1024, head_dim=64)), 4), (dict(tokens=0), 0), (dict(tokens=0, q=None, k=None), 0),
    # rows that are written over rows of the input that are still to be read
    (dict(qs=6144), 1), (dict(ks=6144), 1), (dict(qo=FAKE + 16), 1), (dict(qo=FAKE - 4 * 8192 + 16), 1), (dict(ko=FAKE + 2048), 1),
])
def test_rotate_qk_refuses(kw, code):
    assert rotate(**kw) == code


def append(shape=OK, fmt=0, rot=rotary(), q=FAKE, qs=4096, k=FAKE, ks=1024, v=FAKE, vs=1024, qn=None, kn=None, eps=1e-6,
           pos=None, ts=FAKE, tokens=4, kp=FAKE, vp=FAKE, summ=FAKE, pt=FAKE, sl=FAKE, batch=4, mp=64, qo=FAKE):
    return moira.load_library().moira_append_rotated(
        ctypes.byref(shape), fmt, None if rot is None else ctypes.byref(rot), q, qs, k, ks, v, vs, qn, kn, eps, pos, ts, tokens,
        kp, vp, summ, pt, sl, batch, mp, qo, None)


@pytest.mark.parametrize("kw,code", [(x, 1) for x in BAD_ROTARIES] + [
    (dict(k=None), 1), (dict(v=None), 1), (dict(ts=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(pt=None), 1),
    (dict(sl=None), 1), (dict(qo=None), 1), (dict(fmt=3), 1), (dict(fmt=-1), 1), (dict(tokens=-1), 1), (dict(eps=-0.5), 1),
    (dict(q=FAKE + 8), 1), (dict(k=FAKE + 2), 1), (dict(v=FAKE + 8), 1), (dict(qs=4094), 1), (dict(ks=1016), 1), (dict(vs=1028), 1),
    (dict(kp=FAKE + 8), 1), (dict(vp=FAKE + 8), 1), (dict(summ=FAKE + 8), 1), (dict(qo=FAKE + 8), 1), (dict(kn=FAKE + 4), 1),
    (dict(batch=0), 1), (dict(mp=0), 1), (dict(mp=mb.MAX_PAGES_PER_SEQ + 1), 4), (dict(batch=mb.MAX_UNITS // 8 + 1), 4),
    (dict(qs=6144), 1), (dict(qo=FAKE + 3 * 8192), 1),
    (dict(shape=moira.Shape.of(16, 8, 1024)), 4), (dict(tokens=0), 0),
])
def test_append_rotated_refuses(kw, code):
    assert append(**kw) == code


def chunk(shape=OK, q=FAKE, kp=FAKE, vp=FAKE, pt=FAKE, sl=FAKE, ts=FAKE, batch=4, mp=64, tokens=9, causal=1, sm=0.088,
          out=2 * FAKE + (1 << 20), ws=FAKE, nb=0):
    return moira.load_library().moira_attend_chunk(ctypes.byref(shape), q, kp, vp, pt, sl, ts, batch, mp, tokens, causal, sm,
                                                   out, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), 1), (dict(kp=None), 1), (dict(vp=None), 1), (dict(pt=None), 1), (dict(sl=None), 1), (dict(ts=None), 1),
    (dict(out=None), 1), (dict(q=FAKE + 8), 1), (dict(kp=FAKE + 8), 1), (dict(vp=FAKE + 8), 1), (dict(out=FAKE + 8), 1),
    (dict(sm=0.0), 1), (dict(sm=float("inf")), 1), (dict(tokens=-1), 1), (dict(batch=0), 1),
    (dict(mp=mb.MAX_PAGES_PER_SEQ + 1), 4), (dict(batch=mb.MAX_UNITS // 8 + 1), 4),
    (dict(shape=moira.Shape.of(16, 8, 1024)), 4), (dict(ws=None), 2), (dict(ws=FAKE + 16, nb=1 << 40), 2), (dict(nb=100), 2),
    (dict(out=FAKE), 1), (dict(out=FAKE + 9 * 8192 - 16), 1), (dict(q=1 << 20, out=(1 << 20) - 16), 1),
    (dict(out=FAKE + 9 * 8192), 2), (dict(tokens=0), 0),
])
def test_attend_chunk_refuses(kw, code):
    assert chunk(**kw) == code


def test_workspace_size_of_invalid_arguments_is_zero():
    lib = moira.load_library()
    assert lib.moira_chunk_workspace_bytes(ctypes.byref(moira.Shape.of(30, 8, 16)), 1, 64, 8) == 0
    assert lib.moira_chunk_workspace_bytes(ctypes.byref(OK), 0, 64, 8) == 0
    assert lib.moira_chunk_workspace_bytes(ctypes.byref(OK), 1, 64, 0) == 0


@pytest.mark.parametrize("freq,axis,kw", [
    ([1.0] * 3, None, {}), ([], None, {}), ([1.0] * 68, None, {}), ([float("nan")] * 4, None, {}), ([2.0 ** 21] * 4, None, {}),
    ([1.0] * 4, [0, 1, 2, 4], {}), ([1.0] * 4, [0, 0, 0, -1], {}), ([1.0] * 4, None, dict(scale=float("nan"))),
])
def test_make_rotary_refuses(freq, axis, kw):
    with pytest.raises(moira.MoiraError):
        moira.make_rotary(freq, axis, **kw)


def test_make_rotary_wants_an_axis_for_every_pair():
    with pytest.raises(ValueError):
        moira.make_rotary([1.0] * 8, [0] * 4)


@pytest.mark.parametrize("freq", [[500000.0 ** (-i / 64) for i in range(64)], [0.0, 1.0, -1.0, 6.283185307179586],
                                  [1e-30, -1e-30, 123456.789, -2.0 ** 20]])
def test_rotary_table_is_the_fraction_of_a_turn(freq):
    """turns = inv_freq / 2 pi mod 1 in units of 2^-64, the sum of two products and roundings: off by a few units, and
    2^-105 of the turns that whole turns were taken from."""
    r = moira.make_rotary(freq, [i % 3 for i in range(len(freq))], interleaved=True, scale=1.5)
    assert (r.pairs, r.axes, r.interleaved, r.scale) == (len(freq), 3, 1, 1.5)
    for i, f in enumerate(freq):
        exact = Fraction(f) / TWO_PI
        off = (Fraction(r.turns[i], 2 ** 64) - exact) % 1
        off = min(off, 1 - off)
        assert off <= Fraction(4, 2 ** 64) + abs(exact) / 2 ** 104, (i, float(off) * 2 ** 64)
        assert r.axis[i] == i % 3


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 32, 128, dtype=torch.bfloat16)
    i = torch.zeros(5, dtype=torch.int32)
    with pytest.raises(TypeError):
        moira.rotate_qk(OK, rotary(), t, None, i, t)
    with pytest.raises(ValueError):
        moira.rotate_qk(OK, rotary(), None, None, i)
    with pytest.raises(TypeError):
        moira.append_rotated(OK, rotary(), None, t, t, i, t, t, None, i.view(1, 5), i)
    with pytest.raises(TypeError):
        moira.attend_chunk(OK, t, t, t, i.view(1, 5), i, i, 0.1, t, t)


def test_plain_rotation_depends_on_distances_alone():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 1, 128))
    freq, axis = [1000.0 ** (-i / 32) for i in range(32)], [i % 2 for i in range(32)]

    def score(p, q, inter):
        y, _ = ref.turned(x, None, 0, freq, axis, np.array([[p, q], [3 * p, 3 * q]]), inter)
        return float(y[0, 0] @ y[1, 0])

    for inter in (False, True):
        assert abs(score(5, 9, inter) - score(1005, 1009, inter)) < 1e-9
        assert abs(score(0, 0, inter) - float(x[0, 0] @ x[1, 0])) < 1e-12


def test_plain_chunk_is_one_token_at_a_time():
    """The i-th row of a causal chunk is a chunk of one row over the shorter cache."""
    rng = np.random.default_rng(1)
    bits = lambda *s: (rng.standard_normal(s).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)  # noqa: E731
    q, k, v = bits(5, 4, 128), bits(4, 1, 16, 128), bits(4, 1, 16, 128)
    table = np.array([[2, 0, 3, 1]], np.int32)
    whole, _ = ref.attend_chunk(q, k, v, table, [40], [0, 5], 0.1, True)
    for i in range(5):
        one, _ = ref.attend_chunk(q[i:i + 1], k, v, table, [36 + i], [0, 1], 0.1, True)
        assert np.allclose(whole[i], one[0], rtol=1e-12)
    cross, _ = ref.attend_chunk(q, k, v, table, [40], [0, 5], 0.1, False)
    assert np.allclose(cross[4], whole[4], rtol=1e-12) and not np.allclose(cross[0], whole[0])
    empty, _ = ref.attend_chunk(q, k, v, table, [3], [0, 5], 0.1, True)
    assert not empty[:2].any() and empty[2].any()


# Overlaps, each the only reason to refuse: tokens' rows of 32 heads take 8192 bytes, of 8 heads 2048.
MB = 1 << 20
APART = dict(q=1 * MB, k=2 * MB, qo=4 * MB, ko=5 * MB)


@pytest.mark.parametrize("kw", [
    dict(qo=2 * MB), dict(qo=2 * MB + 3 * 2048 + 16), dict(qo=2 * MB - 4 * 8192 + 16),          # q_out over k
    dict(ko=1 * MB), dict(ko=1 * MB + 4 * 8192 - 16), dict(ko=1 * MB - 4 * 2048 + 16),          # k_out over q
    dict(ko=4 * MB), dict(ko=4 * MB + 4 * 8192 - 16), dict(ko=4 * MB - 4 * 2048 + 16),          # k_out over q_out
    dict(q=1 * MB, k=1 * MB + 8192, qs=6144, ks=6144, qo=1 * MB + 3 * 12288 + 8192),             # q_out behind the last q, over the last k
    dict(k=2 * MB, ks=1 << 18, ko=2 * MB + (1 << 19) + 2032),                                  # into the second row of a wide stride
    dict(tokens=1, qo=2 * MB), dict(tokens=1, q=1 * MB, qo=1 * MB, ko=1 * MB + 8176),
])
def test_rotate_qk_refuses_outputs_over_other_rows(kw):
    assert rotate(**(APART | kw)) == 1


@pytest.mark.parametrize("kw", [
    dict(qo=2 * MB), dict(qo=2 * MB + 3 * 2048 + 16), dict(qo=2 * MB - 4 * 8192 + 16),          # q_out over k
    dict(qo=3 * MB), dict(qo=3 * MB + 3 * 2048 + 16), dict(qo=3 * MB - 4 * 8192 + 16),          # q_out over v
    dict(q=1 * MB, k=1 * MB + 8192, v=1 * MB + 10240, qs=6144, ks=6144, vs=6144, qo=1 * MB + 3 * 12288 + 10240),
    dict(tokens=1, qo=3 * MB + 2032),
])
def test_append_rotated_refuses_queries_over_keys_or_values(kw):
    base = dict(q=1 * MB, k=2 * MB, v=3 * MB, qo=4 * MB, kp=16 * MB, vp=32 * MB)
    assert append(**(base | kw)) == 1
