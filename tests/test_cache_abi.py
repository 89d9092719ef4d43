"""The paged key-value cache without a GPU: what the C ABI and the binding
refuse, frequencies, and the oracle's own pins.  Every library call here
returns before any launch."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc
from rank_gated_memory_amd import gsi

pytestmark = pytest.mark.skipif(not os.path.exists(gsi.LIB_PATH), reason="libgsi.so not built")

GSI_OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WS, E_HIP, E_ARG = range(8)
FAKE = 0x7F0000000000  # aligned fake device address (never dereferenced)
REF = ctypes.byref


def cache(pages=10, page=16, heads=2, d=64, dtype=1, ps=None, hs=None, ss=None, K=FAKE, V=FAKE, mass=FAKE, age=FAKE):
    return gsi.GsiCacheStruct(pages, page, heads, d, dtype, 0, page * heads * d if ps is None else ps,
                              page * d if hs is None else hs, d if ss is None else ss, K, V, mass, age)


def table(t=FAKE, ld=4, S=3, most=4):
    return gsi.GsiTableStruct(t, ld, S, most)


def heads(p=FAKE, row=512, head=64, n=2):
    return gsi.GsiHeadsStruct(p, row, head, n, 0)


def rotation(d=64, start=0, layout=1, freq=FAKE):
    return gsi.GsiRotationStruct(d, start, layout, 1.0, freq)


def opt(s):
    return None if s is None else REF(s)


def rotary(r=rotation(), x=heads(), y=heads(), T=3, d=64, dtype=1, positions=FAKE, pos_bytes=8):
    return gsi.lib().gsi_rotary(opt(r), opt(x), opt(y), T, d, dtype, positions, pos_bytes, None)


def append(c=cache(), t=table(), seq=FAKE, slots=FAKE, k=heads(), v=heads(), T=3, r=rotation(), positions=FAKE,
           pos_bytes=4, q=heads(n=4), q_out=heads(n=4)):
    return gsi.lib().gsi_cache_append(opt(c), opt(t), seq, slots, opt(k), opt(v), T, opt(r), positions, pos_bytes,
                                      opt(q), opt(q_out), None)


def attend(c=cache(), t=table(), lengths=FAKE, q=heads(n=4), out=heads(n=4), window=0, accumulate=0, lse=FAKE, ws=FAKE,
           ws_bytes=1 << 40):
    return gsi.lib().gsi_cache_attend(opt(c), opt(t), lengths, opt(q), opt(out), 1.0, window, accumulate, lse, ws,
                                      ws_bytes, None)


def evict(c=cache(), t=table(), lengths=FAKE, budget=20, recent=4, to=None, out=FAKE + 64, source=FAKE):
    return gsi.lib().gsi_cache_evict(opt(c), opt(t), lengths, budget, recent, opt(to), out, source, None)


BAD_CACHES = [
    (dict(pages=0), E_SHAPE), (dict(pages=-1), E_SHAPE), (dict(page=4), E_SHAPE), (dict(page=24), E_SHAPE),
    (dict(page=8192), E_SHAPE), (dict(heads=0), E_SHAPE), (dict(heads=1025), E_SHAPE), (dict(d=0), E_SHAPE),
    (dict(d=12), E_SHAPE), (dict(d=264), E_SHAPE), (dict(dtype=2), E_DTYPE), (dict(ss=56), E_SHAPE), (dict(hs=56), E_SHAPE),
    (dict(ps=0), E_SHAPE), (dict(ps=-2048), E_SHAPE), (dict(ps=1 << 60), E_SHAPE), (dict(hs=1 << 60), E_SHAPE),
    (dict(ss=1 << 60), E_SHAPE), (dict(ss=1 << 24), E_SHAPE), (dict(K=None), E_NULL), (dict(V=None), E_NULL), (dict(K=FAKE + 8), E_ALIGN),
    (dict(V=FAKE + 2), E_ALIGN), (dict(ss=68), E_ALIGN), (dict(hs=1028), E_ALIGN), (dict(ps=4100), E_ALIGN),
    (dict(mass=FAKE + 2), E_ALIGN), (dict(age=FAKE + 1), E_ALIGN),
]
BAD_TABLES = [
    (dict(S=-1), E_SHAPE), (dict(S=1 << 24), E_SHAPE), (dict(most=-1), E_SHAPE), (dict(ld=3), E_SHAPE),
    (dict(ld=1 << 61), E_SHAPE), (dict(most=1 << 27, ld=1 << 27), E_SHAPE), (dict(t=None), E_NULL), (dict(t=FAKE + 2), E_ALIGN),
]
BAD_HEADS = [
    (dict(p=None), E_NULL), (dict(p=FAKE + 8), E_ALIGN), (dict(row=56), E_SHAPE), (dict(row=-512), E_SHAPE),
    (dict(row=516), E_ALIGN), (dict(head=56), E_SHAPE), (dict(head=68), E_ALIGN), (dict(row=1 << 60), E_SHAPE),
    (dict(head=1 << 60), E_SHAPE),
]
BAD_ROTATIONS = [
    (dict(d=0), E_SHAPE), (dict(d=7), E_SHAPE), (dict(d=66), E_SHAPE), (dict(start=-1), E_SHAPE), (dict(start=2), E_SHAPE),
    (dict(start=2**31 - 1), E_SHAPE), (dict(layout=2), E_ARG), (dict(layout=-1), E_ARG), (dict(freq=None), E_NULL),
    (dict(freq=FAKE + 4), E_ALIGN),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_refuses_caches(kw, status):
    assert append(c=cache(**kw)) == status
    assert attend(c=cache(**kw)) == status
    assert evict(c=cache(**kw)) == status
    assert gsi.lib().gsi_cache_attend_workspace(REF(cache(**kw)), REF(table()), 4, 1) == 0


@pytest.mark.parametrize("kw,status", BAD_TABLES)
def test_refuses_tables(kw, status):
    assert append(t=table(**kw)) == status
    assert attend(t=table(**kw)) == status
    assert evict(t=table(**kw)) == status
    assert evict(to=table(**kw)) == status
    assert gsi.lib().gsi_cache_attend_workspace(REF(cache()), REF(table(**kw)), 4, 1) == 0


@pytest.mark.parametrize("kw,status", BAD_HEADS)
def test_refuses_heads(kw, status):
    assert rotary(x=heads(**kw)) == status
    assert rotary(y=heads(**kw)) == status
    assert append(k=heads(**kw)) == status
    assert append(v=heads(**kw)) == status
    assert append(q=heads(**{"n": 4, **kw})) == status
    assert append(q_out=heads(**{"n": 4, **kw})) == status
    assert attend(q=heads(**{"n": 4, **kw})) == status
    assert attend(out=heads(**{"n": 4, **kw})) == status


@pytest.mark.parametrize("kw,status", BAD_ROTATIONS)
def test_refuses_rotations(kw, status):
    assert rotary(r=rotation(**kw)) == status
    assert append(r=rotation(**kw)) == status


def test_rotary_refuses():
    assert rotary(r=None) == E_NULL and rotary(x=None) == E_NULL and rotary(y=None) == E_NULL
    assert rotary(dtype=3) == E_DTYPE and rotary(pos_bytes=2) == E_DTYPE
    assert rotary(T=-1) == E_SHAPE and rotary(d=60) == E_SHAPE and rotary(d=264) == E_SHAPE and rotary(d=0) == E_SHAPE
    assert rotary(y=heads(n=3)) == E_SHAPE and rotary(x=heads(n=0), y=heads(n=0)) == E_SHAPE
    assert rotary(x=heads(n=4097), y=heads(n=4097)) == E_SHAPE
    assert rotary(positions=None) == E_NULL
    assert rotary(positions=FAKE + 4) == E_ALIGN and rotary(positions=FAKE + 2, pos_bytes=4) == E_ALIGN
    assert rotary(T=0) == GSI_OK and rotary(T=0, positions=None, x=heads(p=None), y=heads(p=None)) == GSI_OK
    # fp32 rows: multiples of four elements do; strides over one row or head do not count
    assert rotary(T=0, dtype=0, x=heads(row=516, head=68)) == GSI_OK
    assert rotary(T=0, x=heads(row=-1, n=1, head=3), y=heads(n=1, head=0)) == GSI_OK
    # more than a launch holds
    many = heads(row=64 * 4096, n=4096)
    assert rotary(x=many, y=many, T=2**31 - 1) == E_SHAPE


def test_append_refuses():
    assert append(c=None) == E_NULL and append(t=None) == E_NULL and append(k=None) == E_NULL and append(v=None) == E_NULL
    assert append(slots=None) == E_NULL and append(positions=None) == E_NULL
    assert append(q=None) == E_NULL and append(q_out=None) == E_NULL
    assert append(k=heads(n=3)) == E_SHAPE and append(v=heads(n=1)) == E_SHAPE and append(T=-1) == E_SHAPE
    assert append(q=heads(n=4), q_out=heads(n=3)) == E_SHAPE
    assert append(seq=FAKE + 2) == E_ALIGN and append(slots=FAKE + 1) == E_ALIGN
    assert append(pos_bytes=3) == E_DTYPE and append(r=None, pos_bytes=5) == E_DTYPE
    assert append(positions=FAKE + 4, pos_bytes=8) == E_ALIGN
    assert append(T=0) == GSI_OK and append(T=0, r=None, positions=None, pos_bytes=0, q=None, q_out=None) == GSI_OK


def test_attend_refuses():
    assert attend(c=None) == E_NULL and attend(t=None) == E_NULL and attend(q=None) == E_NULL and attend(out=None) == E_NULL
    assert attend(lengths=None) == E_NULL and attend(accumulate=1, c=cache(mass=None)) == E_NULL
    assert attend(q=heads(n=3), out=heads(n=3)) == E_SHAPE and attend(out=heads(n=2)) == E_SHAPE
    assert attend(window=-1) == E_SHAPE
    assert attend(lengths=FAKE + 2) == E_ALIGN and attend(lse=FAKE + 2) == E_ALIGN and attend(ws=FAKE + 8) == E_ALIGN
    need = gsi.lib().gsi_cache_attend_workspace(REF(cache()), REF(table()), 4, 1)
    assert need > 0
    assert attend(accumulate=1, ws_bytes=need - 1) == E_WS and attend(accumulate=1, ws=None) == E_NULL
    assert attend(t=table(S=0)) == GSI_OK and attend(t=table(S=0), lengths=None) == GSI_OK
    for n in (0, 3, -2, 4098):
        assert gsi.lib().gsi_cache_attend_workspace(REF(cache()), REF(table()), n, 1) == 0
    assert gsi.lib().gsi_cache_attend_workspace(None, REF(table()), 4, 1) == 0
    assert gsi.lib().gsi_cache_attend_workspace(REF(cache()), None, 4, 1) == 0


def test_attend_refuses_more_slots_than_it_counts():
    assert attend(t=table(S=(1 << 24) - 1, most=1 << 10, ld=1 << 10), ws_bytes=2**63) == E_SHAPE
    assert attend(t=table(S=1 << 20, most=1 << 13, ld=1 << 13), ws_bytes=2**63) == E_SHAPE


@pytest.mark.parametrize("S,most,page", [((1 << 24) - 1, 1 << 10, 16), (1 << 20, 1 << 13, 16), ((1 << 24) - 1, 1 << 18, 4096)])
def test_no_workspace_for_more_slots_than_it_counts(S, most, page):
    """Sizes that the call refuses, whatever workspace it is given, and whose scores
    would be 2^64 bytes and more."""
    c, t = cache(page=page, ps=page * 128), table(S=S, most=most, ld=most)
    q = heads(row=4096 * 64, n=4096)
    assert gsi.lib().gsi_cache_attend_workspace(REF(c), REF(t), 4096, 1) == 0
    for size in (0, 1 << 40, 2**63):
        assert attend(c=c, t=t, q=q, out=q, accumulate=1, ws_bytes=size) == E_SHAPE
    most = ((2**31 - 1) // S - 3) * 32 // page  # the most that is counted
    t = table(S=S, most=most, ld=most)
    need = gsi.lib().gsi_cache_attend_workspace(REF(c), REF(t), 4096, 1)
    assert need >= S * 4096 * most * page * 4 and attend(c=c, t=t, q=q, out=q, accumulate=1, ws_bytes=need - 1) == E_WS


def test_evict_refuses():
    assert evict(c=None) == E_NULL and evict(t=None) == E_NULL and evict(lengths=None) == E_NULL
    assert evict(source=None) == E_NULL and evict(c=cache(mass=None)) == E_NULL
    assert evict(budget=0) == E_SHAPE and evict(budget=(1 << 20) + 1) == E_SHAPE
    assert evict(recent=-1) == E_SHAPE and evict(recent=21) == E_SHAPE
    assert evict(t=table(most=(1 << 15) + 1, ld=1 << 16)) == E_SHAPE
    assert evict(to=table(S=2)) == E_SHAPE and evict(to=table(most=1)) == E_SHAPE
    assert evict(out=FAKE) == E_ARG
    assert evict(lengths=FAKE + 2) == E_ALIGN and evict(out=FAKE + 66) == E_ALIGN and evict(source=FAKE + 1) == E_ALIGN
    assert evict(t=table(S=0)) == GSI_OK and evict(t=table(S=0), to=table(S=0)) == GSI_OK
    assert evict(c=cache(heads=1024, ps=16 * 1024 * 64), t=table(S=(1 << 24) - 1)) == E_SHAPE


# ---- the binding ----


def pool(pages=6, heads=2, page=8, d=16, dtype=torch.bfloat16):
    return torch.zeros(pages, heads, page, d, dtype=dtype), torch.zeros(pages, heads, page, d, dtype=dtype)


def test_cache_handle_checks():
    K, V = pool()
    c = gsi.Cache(K, V, torch.zeros(6, 2, 8), torch.zeros(6, 2, 8, dtype=torch.int32))
    assert (c.struct.page_stride, c.struct.head_stride, c.struct.slot_stride) == (256, 128, 16)
    t = gsi.Cache(*(torch.zeros(6, 8, 2, 16).transpose(1, 2) for _ in range(2)))
    assert (t.struct.page_stride, t.struct.head_stride, t.struct.slot_stride) == (256, 16, 32)
    one = gsi.Cache(K[:1, :1].transpose(0, 1), V[:1, :1])  # strides of one page and one head do not count
    assert one.struct.page_stride == 16 and one.struct.head_stride == 16
    for bad in (lambda: gsi.Cache(K, V[:5]), lambda: gsi.Cache(K[0], V[0]), lambda: gsi.Cache(K, V.float()),
                lambda: gsi.Cache(K, V.transpose(2, 3).contiguous().transpose(2, 3)),
                lambda: gsi.Cache(K.transpose(2, 3), V.transpose(2, 3)),
                lambda: gsi.Cache(K, V, torch.zeros(6, 2, 7)), lambda: gsi.Cache(K, V, torch.zeros(6, 2, 8).double()),
                lambda: gsi.Cache(K, V, torch.zeros(6, 8, 2).transpose(1, 2)),
                lambda: gsi.Cache(K, V, None, torch.zeros(6, 2, 8))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        gsi.Cache(K.half(), V.half())


def test_binding_refuses_before_any_call():
    K, V = pool()
    c = gsi.Cache(K, V, torch.zeros(6, 2, 8))
    bare = gsi.Cache(K, V)
    tab = torch.zeros(3, 2, dtype=torch.int32)
    lens = torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 4, 16, dtype=torch.bfloat16)
    kv = torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    r = gsi.Rotary(gsi.rotary_freqs(16))
    pos = torch.zeros(3, dtype=torch.int64)
    for bad in (
            lambda: gsi.gsi_rotary(r, q[0], pos), lambda: gsi.gsi_rotary(r, q, pos[:2]), lambda: gsi.gsi_rotary(r, q, pos.float()),
            lambda: gsi.gsi_rotary(r, q, pos, y=q[:, :3]), lambda: gsi.gsi_rotary(r, q, pos, y=q.float()),
            lambda: gsi.gsi_rotary(r, q.transpose(1, 2).contiguous().transpose(1, 2), pos),
            lambda: gsi.gsi_cache_append(c, tab, lens, kv, kv[:2]), lambda: gsi.gsi_cache_append(c, tab, lens, q, q),
            lambda: gsi.gsi_cache_append(c, tab.long(), lens, kv, kv), lambda: gsi.gsi_cache_append(c, tab[0], lens, kv, kv),
            lambda: gsi.gsi_cache_append(c, tab, lens.long(), kv, kv), lambda: gsi.gsi_cache_append(c, tab, lens[:2], kv, kv),
            lambda: gsi.gsi_cache_append(c, tab, lens, kv, kv, seq=lens.long()),
            lambda: gsi.gsi_cache_append(c, tab, lens, kv.float(), kv),
            lambda: gsi.gsi_cache_append(c, tab, lens, kv, kv, q_out=q),
            lambda: gsi.gsi_cache_append(c, tab, lens, kv, kv, rotary=r, positions=pos[:1]),
            lambda: gsi.gsi_cache_attend(c, tab[:2], lens, q), lambda: gsi.gsi_cache_attend(c, tab, lens[:2], q),
            lambda: gsi.gsi_cache_attend(c, tab, lens, q.float()), lambda: gsi.gsi_cache_attend(c, tab, lens, q[..., :8]),
            lambda: gsi.gsi_cache_attend(bare, tab, lens, q, accumulate=True),
            lambda: gsi.gsi_cache_attend(c, tab, lens, q, out=q[:2]), lambda: gsi.gsi_cache_attend(c, tab, lens, q, lse=q),
            lambda: gsi.gsi_cache_attend(c, tab, lens, q, window=1 << 31),
            lambda: gsi.gsi_cache_evict(bare, tab, lens, 4), lambda: gsi.gsi_cache_evict(c, tab, lens, 0),
            lambda: gsi.gsi_cache_evict(c, tab, lens, 1 << 31), lambda: gsi.gsi_cache_evict(c, tab, lens[:2], 4),
            lambda: gsi.gsi_cache_evict(c, tab, lens, 4, to=tab[:2]),
            lambda: gsi.gsi_cache_evict(c, tab, lens, 4, lengths_out=lens.long()),
            lambda: gsi.gsi_cache_evict(c, tab, lens, 4, moved=torch.zeros(3, 2, 5, dtype=torch.int32))):
        with pytest.raises(ValueError):
            bad()
    # all in order, but not on a GPU
    for call in (lambda: gsi.gsi_rotary(r, q, pos), lambda: gsi.gsi_cache_append(c, tab, lens, kv, kv),
                 lambda: gsi.gsi_cache_attend(c, tab, lens, q), lambda: gsi.gsi_cache_evict(c, tab, lens, 4)):
        with pytest.raises(ValueError, match="on the GPU"):
            call()


def test_rotary_handle_checks():
    with pytest.raises(ValueError):
        gsi.Rotary(gsi.rotary_freqs(8), layout="quarters")
    with pytest.raises(ValueError):
        gsi.Rotary(torch.zeros(0))
    with pytest.raises(ValueError):
        gsi.Rotary(torch.zeros(2, 2))
    r = gsi.Rotary(torch.ones(5, dtype=torch.float32), layout="pairs", start=3, amplitude=0.5)
    assert (r.struct.d, r.struct.start, r.struct.layout, r.struct.amplitude) == (10, 3, 0, 0.5)
    assert r.freqs.dtype == torch.float64


def test_frequencies():
    f = gsi.rotary_freqs(8, base=100.0)
    assert np.allclose(f.numpy(), [1.0, 100 ** -0.25, 0.1, 100 ** -0.75], rtol=1e-14)
    assert torch.equal(gsi.rotary_freqs(8, scaling="linear", factor=4.0), gsi.rotary_freqs(8) / 4.0)
    g = gsi.rotary_freqs(16, scaling="base", factor=8.0)
    plain = gsi.rotary_freqs(16)
    assert g[0] == plain[0] and abs(float(g[-1] * 8 / plain[-1]) - 1) < 1e-12  # the fastest stays, the slowest goes 8 times slower
    b = gsi.rotary_freqs(64, scaling="bands", factor=16.0, original=2048)
    plain = gsi.rotary_freqs(64)
    turns = 2048 * plain / (2 * math.pi)
    assert torch.equal(b[turns >= 32], plain[turns >= 32])
    assert torch.allclose(b[turns <= 1], plain[turns <= 1] / 16, rtol=1e-14, atol=0)
    mid = (turns > 1) & (turns < 32)
    assert bool(mid.any()) and bool(((b < plain) & (b > plain / 16))[mid].all())
    for kw in (dict(d=7), dict(d=0), dict(d=8, scaling="other"), dict(d=2, scaling="base"), dict(d=8, factor=0.0),
               dict(d=8, base=-1.0), dict(d=8, scaling="bands"), dict(d=8, scaling="bands", original=9, low=2, high=2)):
        with pytest.raises(ValueError):
            gsi.rotary_freqs(**kw)


# ---- the oracle ----


def small_pool(rng, pages, heads, page, d):
    return {"K": rng.standard_normal((pages, heads, page, d)), "V": rng.standard_normal((pages, heads, page, d)),
            "mass": rng.random((pages, heads, page)), "age": rng.integers(0, 99, (pages, heads, page)).astype(np.int32)}


def test_oracle_rotary_is_a_rotation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 3, 12))
    f = np.array([1.0, 0.3, 0.01])
    for layout, start in (("pairs", 0), ("halves", 4)):
        p = np.array([0, 1, 7, -3])
        y = orc.rotary(x, p, f, layout, start)
        assert np.allclose(y[0], x[0]) and np.allclose(np.linalg.norm(y, axis=2), np.linalg.norm(x, axis=2))
        assert np.allclose(orc.rotary(y, -p, f, layout, start), x)
        keep = np.r_[0:start, start + 6:12]
        assert np.array_equal(y[..., keep], x[..., keep])
        # scores depend on the distance alone
        a = orc.rotary(x, p + 5, f, layout, start)
        assert np.allclose((a[1] * a[2]).sum(1), (y[1] * y[2]).sum(1))
    # by hand: a quarter turn
    z = np.arange(4.0).reshape(1, 1, 4)
    q = np.array([math.pi / 2, math.pi])
    assert np.allclose(orc.rotary(z, [1], q, "pairs")[0, 0], [-1, 0, -2, -3])
    assert np.allclose(orc.rotary(z, [1], q, "halves", amplitude=2.0)[0, 0], [-4, -2, 0, -6])


def test_oracle_attend_closed_forms():
    rng = np.random.default_rng(2)
    p = small_pool(rng, 5, 2, 4, 3)
    tab = np.array([[3, 1], [0, 4]])
    q = rng.standard_normal((2, 4, 3))
    # a zero scale is the mean, one slot is itself, none is zero
    out, lse, mass, _, _ = orc.attend(p, tab, [5, 1], q, 0.0)
    mean = np.concatenate([p["V"][3, :, :4], p["V"][1, :, :1]], axis=1).mean(1)
    assert np.allclose(out[0], mean[[0, 0, 1, 1]]) and np.allclose(lse[0], math.log(5))
    assert np.allclose(out[1], p["V"][0, [0, 0, 1, 1], 0]) and np.allclose(lse[1], 0)
    assert np.allclose(mass.sum(), 8) and np.allclose(mass[3, :, :4], 0.4)
    out, lse, mass, _, _ = orc.attend(p, tab, [0, -5], q, 1.0)
    assert not out.any() and np.all(lse == -np.inf) and not mass.any()
    # a window is a shorter cache; a page that is none is left out
    out, lse, _, _, _ = orc.attend(p, tab, [8, 8], q, 1.0, window=4)
    two, l2, _, _, _ = orc.attend(p, tab[:, 1:], [4, 4], q, 1.0)
    assert np.allclose(out, two) and np.allclose(lse, l2)
    hole, l3, _, _, _ = orc.attend(p, np.array([[9, 1], [-1, 4]]), [8, 8], q, 1.0)
    assert np.allclose(out, hole) and np.allclose(l3, l2)
    # softmax does not see a shift of all scores: a key that is the same everywhere
    p["K"][:] = p["K"][0, 0, 0]
    out, _, _, _, _ = orc.attend(p, tab, [8, 8], q, 7.0)
    assert np.allclose(out[0, 0], np.concatenate([p["V"][3, 0], p["V"][1, 0]]).mean(0))


def test_oracle_evict_by_hand():
    p = {"K": np.arange(8.0).reshape(2, 1, 4, 1), "V": -np.arange(8.0).reshape(2, 1, 4, 1),
         "mass": np.array([[[5, 0, 2, 2.0]], [[1, 2, 0, 0]]]), "age": np.array([[[0, 1, 2, 3]], [[4, 5, 6, 7]]], np.int32)}
    n, src = orc.evict(p, [[0, 1]], [7], 4, 1)
    # slot 6 is the newest; of the others 5, 2, 2 at slots 0, 2, 3 (the tie at slot 5 loses); hole 1 takes slot 6
    assert n.tolist() == [4] and src.tolist() == [[[0, 6, 2, 3]]]
    orc.move(p, [[0, 1]], src)
    assert p["K"].ravel().tolist() == [0, 6, 2, 3, 4, 5, 6, 7] and p["mass"][0, 0].tolist() == [5, 0, 2, 2]
    assert p["age"][0, 0].tolist() == [0, 6, 2, 3]
    n, src = orc.evict(p, [[0, 1]], [3], 4, 1)
    assert n.tolist() == [3] and src.tolist() == [[[0, 1, 2, -1]]]


def test_oracle_evict_counts():
    rng = np.random.default_rng(3)
    p = small_pool(rng, 6, 2, 4, 1)
    tab = rng.permutation(6).reshape(2, 3)
    for budget, recent in ((5, 0), (5, 5), (5, 2), (1, 1)):
        n, src = orc.evict(p, tab, [12, 4], budget, recent)
        assert n.tolist() == [budget, min(4, budget)]
        for s in range(2):
            for h in range(2):
                live = src[s, h][src[s, h] >= 0]
                assert len(set(live.tolist())) == n[s]
                moved = live[live != np.arange(len(live))]
                assert np.all(np.diff(moved) > 0) and np.all(moved >= budget)
