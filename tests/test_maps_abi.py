"""Plain linear maps without a GPU: what the C ABI and the binding refuse, and
the oracle's own pins.  Every library call here returns before any launch."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import maps_oracle as orc
from rank_gated_memory_amd import gsi

pytestmark = pytest.mark.skipif(not os.path.exists(gsi.LIB_PATH), reason="libgsi.so not built")

GSI_OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_WS, E_HIP, E_ARG = range(8)
FAKE = 0x7F0000000000  # aligned fake device address (never dereferenced)


def weights(d=256, d_out=64, n=1, dtype=1, bits=4, group=32, stride=0, W=FAKE, scales=FAKE, zeros=FAKE):
    return gsi.GsiWeightsStruct(d, d_out, n, dtype, bits, group, stride, W, scales, zeros)


def dense(d=256, d_out=64, n=4, dtype=1, stride=None, W=FAKE, group=0):
    return weights(d, d_out, n, dtype, 0, group, d * d_out if stride is None else stride, W, None, None)


def q4(w, x=FAKE, ldx=256, y=FAKE, ldy=64, T=3):
    return gsi.lib().gsi_q4_linear(None if w is None else ctypes.byref(w), x, ldx, y, ldy, T, None)


def grouped(w, x=FAKE, ldx=256, T=5, offsets=FAKE, rows=FAKE, y=FAKE, ldy=64, R=7):
    return gsi.lib().gsi_grouped_linear(None if w is None else ctypes.byref(w), x, ldx, T, offsets, rows, y, ldy, R,
                                        None)


@pytest.mark.parametrize("kw,status", [
    (dict(d=0), E_SHAPE), (dict(d=48), E_SHAPE), (dict(d=-32), E_SHAPE), (dict(d=(1 << 20) + 32), E_SHAPE),
    (dict(d_out=0), E_SHAPE), (dict(d_out=12), E_SHAPE), (dict(d_out=(1 << 24) + 8), E_SHAPE),
    (dict(n=0), E_SHAPE), (dict(n=2), E_SHAPE), (dict(n=4097), E_SHAPE),
    (dict(group=0), E_SHAPE), (dict(group=16), E_SHAPE), (dict(group=256), E_SHAPE), (dict(stride=64), E_SHAPE),
    (dict(dtype=2), E_DTYPE), (dict(bits=8), E_DTYPE), (dict(bits=3), E_DTYPE),
    (dict(W=None), E_NULL), (dict(scales=None), E_NULL),
    (dict(W=FAKE + 8), E_ALIGN), (dict(scales=FAKE + 1), E_ALIGN), (dict(dtype=0, scales=FAKE + 2), E_ALIGN),
])
def test_q4_refuses_weights(kw, status):
    assert q4(weights(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), E_SHAPE), (dict(ldx=248), E_SHAPE), (dict(ldy=56), E_SHAPE),
    (dict(x=None), E_NULL), (dict(y=None), E_NULL),
    (dict(x=FAKE + 8), E_ALIGN), (dict(y=FAKE + 2), E_ALIGN), (dict(ldx=260), E_ALIGN), (dict(ldy=68), E_ALIGN),
])
def test_q4_refuses_operands(kw, status):
    assert q4(weights(), **kw) == status


def test_q4_null_dense_and_empty():
    assert q4(None) == E_NULL
    assert q4(dense(n=1)) == E_DTYPE
    assert q4(weights(), x=None, y=None, T=0) == GSI_OK


@pytest.mark.parametrize("kw,status", [
    (dict(stride=256 * 64 - 8), E_SHAPE), (dict(group=32), E_SHAPE), (dict(d=252), E_SHAPE),
    (dict(stride=256 * 64 + 4), E_ALIGN), (dict(W=FAKE + 4), E_ALIGN), (dict(W=None), E_NULL),
    (dict(n=4097), E_SHAPE), (dict(dtype=5), E_DTYPE),
])
def test_grouped_refuses_weights(kw, status):
    assert grouped(dense(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(R=-1), E_SHAPE), (dict(T=-1), E_SHAPE), (dict(T=0), E_SHAPE), (dict(ldx=128), E_SHAPE),
    (dict(offsets=None), E_NULL), (dict(x=None), E_NULL), (dict(y=None), E_NULL),
    (dict(offsets=FAKE + 2), E_ALIGN), (dict(rows=FAKE + 1), E_ALIGN), (dict(x=FAKE + 4), E_ALIGN),
    (dict(ldy=66), E_ALIGN),
])
def test_grouped_refuses_operands(kw, status):
    assert grouped(dense(), **kw) == status
    assert grouped(weights(n=4), **kw) == status


def test_grouped_empty():
    assert grouped(dense(), R=0, T=0, offsets=None, rows=None, x=None, y=None) == GSI_OK


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), E_SHAPE), (dict(top=0), E_SHAPE), (dict(n=0), E_SHAPE), (dict(n=1025), E_SHAPE),
    (dict(T=1 << 24, top=8), E_SHAPE), (dict(ids_bytes=2), E_DTYPE),
    (dict(ids=None), E_NULL), (dict(offsets=None), E_NULL), (dict(rows=None), E_NULL), (dict(pos=None), E_NULL),
    (dict(ids=FAKE + 4, ids_bytes=8), E_ALIGN), (dict(offsets=FAKE + 2), E_ALIGN), (dict(pos=FAKE + 1), E_ALIGN),
])
def test_group_rows_refuses(kw, status):
    a = dict(ids=FAKE, ids_bytes=4, T=5, top=2, n=8, offsets=FAKE, rows=FAKE, pos=FAKE)
    a.update(kw)
    assert gsi.lib().gsi_group_rows(*a.values(), None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), E_SHAPE), (dict(R=-1), E_SHAPE), (dict(top=0), E_SHAPE), (dict(top=65), E_SHAPE),
    (dict(d=12), E_SHAPE), (dict(d=0), E_SHAPE), (dict(ldy=32), E_SHAPE), (dict(ldb=32), E_SHAPE),
    (dict(ldo=32), E_SHAPE), (dict(dtype=2), E_DTYPE),
    (dict(y=None), E_NULL), (dict(pos=None), E_NULL), (dict(out=None), E_NULL),
    (dict(y=FAKE + 8), E_ALIGN), (dict(base=FAKE + 8), E_ALIGN), (dict(out=FAKE + 2), E_ALIGN),
    (dict(pos=FAKE + 2), E_ALIGN), (dict(weights=FAKE + 2), E_ALIGN), (dict(ldy=68), E_ALIGN),
    (dict(ldb=68), E_ALIGN), (dict(ldo=68), E_ALIGN),
])
def test_group_combine_refuses(kw, status):
    a = dict(y=FAKE, ldy=64, R=9, pos=FAKE, weights=FAKE, base=FAKE, ldb=64, out=FAKE, ldo=64, T=5, top=2, d=64,
             dtype=1)
    a.update(kw)
    assert gsi.lib().gsi_group_combine(*a.values(), None) == status


def test_group_combine_empty():
    assert gsi.lib().gsi_group_combine(None, 64, 0, None, None, None, 0, None, 64, 0, 2, 64, 1, None) == GSI_OK


def test_refuses_what_no_launch_holds():
    """2^32 threads and more, before anything is launched."""
    assert gsi.lib().gsi_group_combine(FAKE, 64, 9, FAKE, None, None, 0, FAKE, 64, 1 << 24, 2, 64, 1, None) == E_SHAPE
    assert q4(weights(dtype=0, d=1 << 14, d_out=1 << 16), ldx=1 << 14, ldy=1 << 16, T=1 << 20) == E_SHAPE
    assert q4(weights(dtype=1, d_out=1 << 16), ldy=1 << 16, T=1 << 24) == E_SHAPE
    assert grouped(dense(dtype=0, d_out=1 << 16), ldy=1 << 16, R=1 << 24, T=1 << 24) == E_SHAPE


@pytest.mark.parametrize("rows", [2**31 - 16, 2**31 - 15, 2**31 - 1])
@pytest.mark.parametrize("dtype", [0, 1], ids=["fp32", "bf16"])
def test_refuses_the_largest_row_counts(rows, dtype):
    """Counts next to 2^31, where sums of 32 bits would wrap: with and without offsets."""
    w = dict(d=32, d_out=8, dtype=dtype)
    assert q4(weights(**w), ldx=32, ldy=8, T=rows) == E_SHAPE
    assert grouped(weights(n=4, **w), ldx=32, ldy=8, R=rows) == E_SHAPE
    assert grouped(weights(n=4096, **w), ldx=32, ldy=8, R=rows) == E_SHAPE


@pytest.mark.skipif(torch.cuda.is_available(), reason="on a GPU these calls would be launched on addresses that are none")
@pytest.mark.parametrize("n", [1, 64, 4096])
@pytest.mark.parametrize("d_out", [8, 24, 136, 144, 264, 800, 8192, 1 << 20])
@pytest.mark.parametrize("d", [32, 5120, 16384])
def test_calls_within_the_documented_size_are_not_refused(d, d_out, n):
    """(R + 16 n)(d_out + 127) just below 2^32, at every form; without a device the launch itself fails."""
    R = (2**32 - 1) // (d_out + 127) - 16 * n
    if R < 1:
        pytest.skip("no rows left")
    for dtype in (0, 1):
        if n == 1:
            assert q4(weights(d=d, d_out=d_out, dtype=dtype), ldx=d, ldy=d_out, T=R) == E_HIP
        assert grouped(weights(d=d, d_out=d_out, n=n, dtype=dtype), ldx=d, ldy=d_out, R=R) == E_HIP
        assert grouped(dense(d=d, d_out=d_out, n=n, dtype=dtype), ldx=d, ldy=d_out, R=R) == E_HIP


def test_combines_the_documented_number_of_workgroups():
    """A workgroup for every token and started 4 KiB of its row, fewer than 2^24 of them."""
    def call(T, d, dtype):
        return gsi.lib().gsi_group_combine(FAKE, d, 9, FAKE, None, None, 0, FAKE, d, T, 2, d, dtype, None)
    for d, dtype, per in ((8, 1, 1), (2048, 1, 1), (2056, 1, 2), (1024, 0, 1), (1032, 0, 2), (1 << 20, 0, 1024)):
        most = ((1 << 24) - 1) // per
        assert call(most + 1, d, dtype) == E_SHAPE
        if not torch.cuda.is_available():
            assert call(most, d, dtype) == E_HIP


def test_refuses_narrow_maps_that_no_launch_holds():
    """A map of 8 outputs takes a whole workgroup for 16 rows."""
    assert q4(weights(d=32, d_out=8, dtype=0), ldx=32, ldy=8, T=1 << 27) == E_SHAPE
    assert grouped(weights(n=4, d=32, d_out=8, dtype=0), ldx=32, ldy=8, R=1 << 27) == E_SHAPE


def test_binding_refuses():
    codes = torch.zeros(64, 128, dtype=torch.uint8)
    scales = torch.ones(64, 2)
    zeros = torch.zeros(64, 2, dtype=torch.uint8)
    w = gsi.Q4(codes, scales, zeros, group=128)
    assert (w.n, w.d_out, w.d) == (1, 64, 256)
    assert gsi.Q4(codes[None].repeat(3, 1, 1), scales[None].repeat(3, 1, 1)).n == 3
    with pytest.raises(ValueError):
        gsi.Q4(codes.int(), scales)
    with pytest.raises(ValueError):
        gsi.Q4(codes, scales, zeros, group=64)
    with pytest.raises(ValueError):
        gsi.Q4(codes, scales, zeros.int())
    with pytest.raises(ValueError):
        gsi.Q4(codes.t().contiguous().t(), scales, zeros)
    with pytest.raises(ValueError):
        gsi.Q4(codes, scales, zeros, group=48)
    with pytest.raises(TypeError):
        gsi.Q4(codes, scales.half())
    x = torch.zeros(5, 256)
    for bad in (x[:, :128], x.double(), x.t(), x.bfloat16(), x[:, ::2], x[0, 0]):
        with pytest.raises(ValueError):
            gsi.gsi_q4_linear(w, bad)
    with pytest.raises(ValueError, match="GPU"):
        gsi.gsi_q4_linear(w, x)
    with pytest.raises(ValueError):
        gsi.gsi_q4_linear(w, x, y=torch.zeros(4, 64))
    W, off = torch.zeros(3, 64, 256), torch.zeros(4, dtype=torch.int32)
    for kw in (dict(offsets=off[:3]), dict(offsets=off.long()), dict(rows=torch.zeros(5)), dict(w=W[0]),
               dict(w=W.transpose(1, 2)), dict(w=W[:, ::2]), dict(y=torch.zeros(6, 64)), dict(x=x.bfloat16())):
        with pytest.raises(ValueError):
            gsi.gsi_grouped_linear(**{**dict(w=W, x=x, offsets=off), **kw})
    with pytest.raises(ValueError):
        gsi.gsi_group_rows(torch.zeros(5), 4)
    with pytest.raises(ValueError):
        gsi.gsi_group_rows(torch.zeros(5, 2, dtype=torch.int16), 4)
    pos = torch.zeros(5, 2, dtype=torch.int32)
    for kw in (dict(pos=pos.long()), dict(weights=torch.ones(5, 3)), dict(weights=torch.ones(5, 2).double()),
               dict(base=torch.zeros(4, 256)), dict(out=torch.zeros(5, 128))):
        with pytest.raises(ValueError):
            gsi.gsi_group_combine(**{**dict(y=x, pos=pos), **kw})


def test_binding_refuses_sizes_past_32_bits():
    """2^32 + 5 rows must not become 5 on their way into the library (meta tensors: no memory behind them)."""
    big = 2**32 + 5

    def meta(*shape, dtype=torch.bfloat16):
        return torch.empty(*shape, dtype=dtype, device="meta")
    i32, u8 = torch.int32, torch.uint8
    w, off = meta(2, 8, 8), meta(3, dtype=i32)
    few = gsi.Q4(meta(8, 16, dtype=u8), meta(8, 1), None, group=32)
    for call in (lambda: gsi.gsi_q4_linear(few, meta(big, 32)),
                 lambda: gsi.gsi_grouped_linear(w, meta(big, 8), off),
                 lambda: gsi.gsi_grouped_linear(w, meta(7, 8), off, rows=meta(big, dtype=i32)),
                 lambda: gsi.gsi_grouped_linear(meta(2, big + 3, 8), meta(7, 8), off),
                 lambda: gsi.Q4(meta(big + 3, 16, dtype=u8), meta(big + 3, 1), None, group=32),
                 lambda: gsi.Q4(meta(big, 8, 16, dtype=u8), meta(big, 8, 1), None, group=32),
                 lambda: gsi.gsi_group_rows(meta(big, 1, dtype=i32), 4),
                 lambda: gsi.gsi_group_rows(meta(3, big, dtype=i32), 4),
                 lambda: gsi.gsi_group_rows(meta(3, 2, dtype=i32), big),
                 lambda: gsi.gsi_group_combine(meta(7, 8), meta(big, 1, dtype=i32)),
                 lambda: gsi.gsi_group_combine(meta(big, 8), meta(3, 2, dtype=i32)),
                 lambda: gsi.gsi_group_combine(meta(7, big + 3), meta(3, 2, dtype=i32))):
        with pytest.raises(ValueError, match="2\\^31"):
            call()


@pytest.mark.parametrize("rows", [0, 1])
def test_one_row_has_no_stride(rows):
    """The stride of a view of one row is never used, so it need not suit the library (257 columns apart here)."""
    wide = torch.zeros(5, 257)
    for view in (wide[2:2 + rows, :256], wide[2:2 + rows, :256].clone(), wide[None, 0, :256].expand(1, 256)[:rows]):
        assert gsi._rows2d(view, "x", torch.float32, wide.device, 256) == 256
    assert gsi._rows2d(wide[:2, :256], "x", torch.float32, wide.device, 256) == 257


# ---- pins of the oracle ----


def test_oracle_q4_closed_form():
    codes = np.array([[0x10, 0x32, 0xFE, 0x8F] * 8], np.uint8)  # columns 0 1 2 3 14 15 15 8
    W = orc.q4_weights(codes, np.array([[0.5, 2.0]]), np.array([[3, 0x18]], np.uint8), 32)
    assert W.shape == (1, 64)
    assert W[0, :8].tolist() == [-1.5, -1.0, -0.5, 0.0, 5.5, 6.0, 6.0, 2.5]
    assert W[0, 32:40].tolist() == [-16.0, -14.0, -12.0, -10.0, 12.0, 14.0, 14.0, 0.0]
    assert orc.q4_weights(codes, np.array([[1.0, 1.0]]), None, 32)[0, :3].tolist() == [-8.0, -7.0, -6.0]


def test_oracle_grouping_inverts():
    rng = np.random.default_rng(3)
    ids = rng.integers(-1, 6, (13, 3))
    offsets, rows, pos = orc.group_rows(ids, 5)
    assert offsets[0] == 0 and offsets[-1] == ((ids >= 0) & (ids < 5)).sum()
    for t in range(13):
        for j in range(3):
            if 0 <= ids[t, j] < 5:
                assert offsets[ids[t, j]] <= pos[t, j] < offsets[ids[t, j] + 1] and rows[pos[t, j]] == t
            else:
                assert pos[t, j] == -1
    # identity maps, weights that sum to one: a token's own row comes back
    x = rng.standard_normal((13, 4))
    y = orc.grouped_linear([np.eye(4)] * 5, x, offsets, rows, np.zeros((39, 4)))
    w = ((ids >= 0) & (ids < 5)) / np.maximum(1, ((ids >= 0) & (ids < 5)).sum(1, keepdims=True))
    out = orc.group_combine(y, pos, w, x)
    some = ((ids >= 0) & (ids < 5)).any(1)
    assert np.allclose(out[some], 2 * x[some]) and np.allclose(out[~some], x[~some])
