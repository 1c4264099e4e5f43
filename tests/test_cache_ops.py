"""The cache operators' host-side checks, without a GPU: bad arguments give the
documented codes before any CUDA call (fake pointers, never dereferenced), and
the binding refuses wrong tensors.  The plain forms that the GPU tests compare
with are checked against each other on small cases."""
import ctypes

import numpy as np
import pytest

import sparse_long_context_page_gb300 as moira
from sparse_long_context_page_gb300 import _binding as mb
from tests import cache_reference as ref

FAKE = 0x10000
OK = moira.Shape.of(32, 8, 1024)


def shared(shape=OK, q=FAKE, kp=FAKE, vp=FAKE, pt=FAKE, pl=FAKE, gs=FAKE, groups=2, pp=16, lists=FAKE, lengths=FAKE,
           sl=FAKE, batch=4, mp=64, sm=0.088, w=None, out=FAKE, ws=FAKE, nb=0):
    return moira.load_library().moira_attend_shared(ctypes.byref(shape), q, kp, vp, pt, pl, gs, groups, pp, lists,
                                                    lengths, sl, batch, mp, sm, w, out, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(kp=0), 1), (dict(vp=0), 1), (dict(lists=0), 1), (dict(lengths=0), 1), (dict(sl=0), 1),
    (dict(out=0), 1), (dict(pt=0), 1), (dict(pl=0), 1), (dict(gs=0), 1),
    (dict(q=FAKE + 2), 1), (dict(kp=FAKE + 8), 1), (dict(vp=FAKE + 8), 1), (dict(out=FAKE + 4), 1),
    (dict(w=FAKE + 4), 1), (dict(sm=0.0), 1), (dict(sm=float("nan")), 1), (dict(groups=-1), 1), (dict(pp=0), 1),
    (dict(groups=mb.MAX_GROUPS + 1), 4), (dict(pp=mb.MAX_PAGES_PER_SEQ + 1), 4), (dict(batch=0), 1),
    (dict(mp=mb.MAX_PAGES_PER_SEQ + 1), 4), (dict(batch=mb.MAX_UNITS // 8 + 1), 4),
    (dict(shape=moira.Shape.of(16, 8, 1024)), 4), (dict(shape=moira.Shape.of(32, 8, 1024, head_dim=64)), 4),
    (dict(shape=moira.Shape.of(32, 8, 0)), 1), (dict(ws=0), 2), (dict(ws=FAKE + 16, nb=1 << 40), 2), (dict(nb=256), 2),
])
def test_attend_shared_refuses(kw, code):
    assert shared(**kw) == code


def test_attend_weights_refuses():
    def call(w=FAKE, sm=0.1, batch=4, q=FAKE, nb=0):
        return moira.load_library().moira_attend_weights(ctypes.byref(OK), q, FAKE, FAKE, FAKE, FAKE, FAKE, batch, 64,
                                                         sm, w, FAKE, FAKE, nb, None)
    assert call(w=None) == 1 and call(w=FAKE + 8) == 1 and call(sm=-1.0) == 1 and call(batch=-1) == 1
    assert call(q=None) == 1 and call() == 2


def evict(shape=OK, fmt=0, kp=FAKE, vp=FAKE, summ=None, w=FAKE, pos=FAKE, pt=FAKE, sl=FAKE, batch=4, mp=64, budget=64,
          sinks=4, recent=16, nl=FAKE, ws=FAKE, nb=0):
    return moira.load_library().moira_evict(ctypes.byref(shape), fmt, kp, vp, summ, w, pos, pt, sl, batch, mp, budget,
                                            sinks, recent, nl, ws, nb, None)


@pytest.mark.parametrize("kw,code", [
    (dict(kp=0), 1), (dict(vp=0), 1), (dict(w=0), 1), (dict(pos=0), 1), (dict(pt=0), 1), (dict(sl=0), 1),
    (dict(nl=0), 1), (dict(kp=FAKE + 8), 1), (dict(w=FAKE + 4), 1), (dict(pos=FAKE + 4), 1), (dict(summ=FAKE + 8), 1),
    (dict(fmt=3), 1), (dict(budget=0), 1), (dict(sinks=-1), 1), (dict(recent=-1), 1), (dict(recent=61), 1),
    (dict(sinks=65, recent=0), 1), (dict(budget=(1 << 31) - 1, sinks=(1 << 31) - 1, recent=1), 1), (dict(batch=0), 1),
    (dict(mp=mb.MAX_PAGES_PER_SEQ + 1), 4), (dict(shape=moira.Shape.of(16, 8, 1024)), 4), (dict(ws=0), 2),
    (dict(ws=FAKE + 8, nb=1 << 40), 2), (dict(nb=1000), 2),
])
def test_evict_refuses(kw, code):
    assert evict(**kw) == code


def test_workspace_sizes_of_invalid_arguments_are_zero():
    lib = moira.load_library()
    bad = moira.Shape.of(30, 8, 16)
    assert lib.moira_evict_workspace_bytes(ctypes.byref(bad), 1, 64) == 0
    assert lib.moira_evict_workspace_bytes(ctypes.byref(OK), 0, 64) == 0
    assert lib.moira_shared_workspace_bytes(ctypes.byref(bad), 1, 64, 1, 1) == 0
    assert lib.moira_shared_workspace_bytes(ctypes.byref(OK), 1, 64, mb.MAX_GROUPS + 1, 0) == 0
    assert lib.moira_evict_workspace_bytes(ctypes.byref(OK), 2, 64) > 256


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 32, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises((TypeError, ValueError)):
        moira.attend_weights(OK, t, t, t, i, i, i, 64, 0.1, t, t, t)
    with pytest.raises((TypeError, ValueError)):
        moira.evict(OK, t, t, None, t, t, i.view(2, 2), i, 4, 0, 1, i, t)


def test_plain_attention_is_a_softmax_over_both_parts():
    """Splitting the same tokens differently between prefix and own part changes nothing."""
    rng = np.random.default_rng(0)
    bits = lambda *s: (rng.standard_normal(s).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)  # noqa: E731
    q, k, v = bits(1, 4, 128), bits(4, 1, 16, 128), bits(4, 1, 16, 128)
    table = np.arange(4, dtype=np.int32)

    def run(split):
        lists = table[None, None, split:]
        return ref.attend_shared(q, k, v, table[None], [16 * split], [0, 1], lists, np.array([[4 - split]]),
                                 [16 * (4 - split)], 0.09, np.zeros((4, 1, 16)))

    a, b = run(0), run(3)
    assert np.allclose(a[0], b[0], rtol=1e-12)
    assert np.allclose(a[2].sum(), 4.0) and np.allclose(b[2][3], a[2][3]) and not b[2][:3].any()


def test_plain_eviction_keeps_the_heaviest():
    k = np.arange(3 * 16 * 128, dtype=np.uint16).reshape(3, 1, 16, 128)
    w = np.zeros((3, 1, 16), np.float32)
    pos = np.full((3, 1, 16), -1, np.int32)
    table = np.array([[2, 0, 1]], np.int32)
    w[2, 0, :3], w[1, 0, 7] = 5.0, 9.0
    key = k[1, 0, 7].copy()
    new, renewed = ref.evict(k, k.copy(), w, pos, table, [40], 5, 0, 1)
    assert new.tolist() == [5] and renewed == []
    assert pos[2, 0, :5].tolist() == [0, 1, 2, 39, 4] or set(pos[2, 0, :5].tolist()) == {0, 1, 2, 39, 3}
    assert not w[1].any() and not np.array_equal(k[2, 0, 3], key)
