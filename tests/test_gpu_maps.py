"""Plain linear maps on the GPU against the fp64 oracle: 4-bit weights, rows
grouped by expert, the grouping itself and the weighted sum that undoes it.

Tolerances.  An output is rounded once: half a step, finfo.eps / 2 relative to
the value.  The fp32 sum before it: every product is exact (bf16 by bf16 and
codes by bf16 parts) or rounded once (fp32 by fp32), a term takes part in at
most d / 16 + 64 rounded additions (instructions of 16 or more columns in a
chain, the additions inside one, the groups, the joined wavefronts), each off
by at most 2^-23 of the sum of the terms' sizes S.  For 4-bit weights the terms
are (16 + q) s x and (16 + z) s x, so S = sum (32 + q + z) s |x|.  Beside that
elementwise bound, every token as a whole is held to a relative L2 error of
2^-8 + 1e-5 (bf16) or 1e-5 (fp32)."""
import numpy as np
import pytest
import torch

from oracle import maps_oracle as orc
from rank_gated_memory_amd import gsi

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def ints(t):
    return t.detach().cpu().numpy()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def make_q4(g, shape, d, group, dtype, zeros=True):
    n = (d + group - 1) // group
    codes = torch.randint(0, 256, (*shape, d // 2), generator=g, device=DEV, dtype=torch.uint8)
    scales = ((0.5 + torch.rand(*shape, n, generator=g, device=DEV)) * d**-0.5).to(dtype)
    z = torch.randint(0, 16, (*shape, n), generator=g, device=DEV, dtype=torch.uint8) if zeros else None
    return gsi.Q4(codes, scales, z, group=group)


def q4_64(w, e=None):
    """(W, the sizes 32 + q + z times |s|) of one map in 64 bits."""
    pick = (lambda t: None if t is None else (t if e is None else t[e]).cpu())
    codes, z = ints(pick(w.codes)), pick(w.zeros)
    z = None if z is None else ints(z)
    s = f64(pick(w.scales))
    q0 = orc.q4_weights(codes, np.ones_like(s), np.zeros(s.shape, np.uint8), w.group)
    zz = np.repeat(np.full(s.shape, 8.0) if z is None else z % 16, w.group, axis=1)[:, :w.d]
    return orc.q4_weights(codes, s, z, w.group), (32 + q0 + zz) * np.repeat(np.abs(s), w.group, axis=1)[:, :w.d]


def close(y, ref, size, d, dtype, what):
    """|y - ref| <= half a step of ref + (d / 16 + 64) 2^-23 size, and the L2 bar per token."""
    y = f64(y)
    half = torch.finfo(dtype).eps / 2
    tol = half * np.abs(ref) * 1.001 + (1 + half) * (d / 16 + 64) * 2.0**-23 * size + 1e-30
    bad = ~(np.abs(y - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
        f"{y[bad][0]} for {ref[bad][0]}"
    norm = np.linalg.norm(ref, axis=-1)
    rel = np.linalg.norm(y - ref, axis=-1)[norm > 0] / norm[norm > 0]
    bar = (2.0**-8 if dtype == BF16 else 0.0) + 1e-5
    assert rel.size == 0 or rel.max() <= bar, f"{what}: L2 {rel.max()}"


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


# ---- 4-bit maps ----


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d,d_out,T", [
    (32, 8, 1), (64, 24, 2), (96, 16, 15), (160, 136, 16), (224, 72, 17), (1056, 1000, 1), (1056, 264, 33),
    (4096, 512, 1), (4096, 1024, 5), (2080, 520, 64), (480, 264, 65), (1024, 392, 130), (992, 640, 300),
    (4096, 264, 257), (8224, 136, 16), (16384, 72, 21),
])
def test_q4_linear(d, d_out, T, dtype, group):
    g = gen(d + d_out + T + group)
    w = make_q4(g, (d_out,), d, group, dtype, zeros=T % 3 != 2)
    x = torch.randn(T, d, generator=g, device=DEV).to(dtype)
    x[:, d // 3] *= 30
    y = gsi.gsi_q4_linear(w, x)
    W, S = q4_64(w)
    X = f64(x)
    close(y, X @ W.T, np.abs(X) @ S.T, d, dtype, f"q4 {d}x{d_out} T={T} group={group}")
    assert torch.equal(bits(gsi.gsi_q4_linear(w, x)), bits(y))


def test_q4_long_rows():
    """The longest row the tests hold, one token and a ragged batch."""
    g = gen(5)
    w = make_q4(g, (40,), 32768 + 96, 64, BF16)
    W, S = q4_64(w)
    for T in (1, 19, 140):
        x = torch.randn(T, w.d, generator=g, device=DEV).to(BF16)
        X = f64(x)
        close(gsi.gsi_q4_linear(w, x), X @ W.T, np.abs(X) @ S.T, w.d, BF16, f"long rows T={T}")


@pytest.mark.parametrize("T", [3, 70, 200])
def test_q4_strides_and_what_is_left(T):
    g = gen(T)
    w = make_q4(g, (72,), 288, 128, BF16)
    wide = torch.full((T, 288 + 40), float("nan"), device=DEV, dtype=BF16)
    x = wide[:, 16:16 + 288]
    x.copy_(torch.randn(T, 288, generator=g, device=DEV))
    out = torch.full((T + 2, 72 + 24), 5.0, device=DEV, dtype=BF16)
    y = out[1:1 + T, 8:80]
    gsi.gsi_q4_linear(w, x, y=y)
    W, S = q4_64(w)
    X = f64(x)
    close(y, X @ W.T, np.abs(X) @ S.T, 288, BF16, "strided")
    out[1:1 + T, 8:80] = 5.0
    assert bool((out == 5.0).all()), "bytes outside y's rows were written"


@pytest.mark.parametrize("T", [2, 17, 150])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_q4_non_finite_tokens_stay_alone(T, dtype):
    g = gen(T + 50)
    w = make_q4(g, (136,), 416, 32, dtype)
    x = torch.randn(T, 416, generator=g, device=DEV).to(dtype)
    ref = gsi.gsi_q4_linear(w, x)
    for bad in (float("inf"), float("-inf"), float("nan")):
        z = x.clone()
        z[T - 1, 415] = bad
        y = gsi.gsi_q4_linear(w, z)
        assert torch.equal(bits(y[:-1]), bits(ref[:-1]))
        assert not torch.isfinite(y[-1]).any()


def test_q4_special_scales():
    """Scales of zero, negative, tiny and infinite: only their own rows notice."""
    g = gen(9)
    w = make_q4(g, (64,), 256, 64, BF16)
    w.scales[3] = 0.0
    w.scales[4] *= -1
    w.scales[5] = 1e-30
    x = torch.randn(20, 256, generator=g, device=DEV).to(BF16)
    W, S = q4_64(w)
    X = f64(x)
    y = gsi.gsi_q4_linear(w, x)
    close(y, X @ W.T, np.abs(X) @ S.T, 256, BF16, "scales")
    assert bool((y[:, 3] == 0).all())
    w.scales[7, 1] = float("inf")
    z = gsi.gsi_q4_linear(w, x)
    keep = [i for i in range(64) if i != 7]
    assert torch.equal(bits(z[:, keep]), bits(y[:, keep])) and not torch.isfinite(z[:, 7]).any()


def test_q4_one_token_vector_and_empty():
    g = gen(10)
    w = make_q4(g, (64,), 128, 64, F32, zeros=False)
    x = torch.randn(128, generator=g, device=DEV)
    W, S = q4_64(w)
    close(gsi.gsi_q4_linear(w, x), f64(x)[None] @ W.T, np.abs(f64(x))[None] @ S.T, 128, F32, "vector")
    assert gsi.gsi_q4_linear(w, x[None][:0]).shape == (0, 64)


def test_one_row_of_a_matrix_with_an_odd_stride():
    """A row sliced from rows that lie no multiple of 16 bytes apart, as x, y and base."""
    g = gen(11)
    w = make_q4(g, (64,), 256, 64, F32)
    wide, out = torch.randn(3, 257, generator=g, device=DEV), torch.full((3, 67), 5.0, device=DEV)
    x, y = wide[:1, :256], out[:1, :64]
    assert gsi.gsi_q4_linear(w, x, y=y) is y
    assert torch.equal(bits(y), bits(gsi.gsi_q4_linear(w, x.clone())))
    base = torch.randn(2, 67, generator=g, device=DEV)[:1, :64]
    want = base + y
    assert gsi.gsi_group_combine(y, torch.zeros(1, 1, device=DEV, dtype=torch.int32), base=base, out=base) is base
    assert torch.equal(bits(base), bits(want))
    assert bool((out[1:] == 5).all()) and bool((out[:, 64:] == 5).all())


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
def test_q4_most_rows_of_a_narrow_map(dtype):
    """(T + 16)(d_out + 127) just below 2^32, the size up to which no call is refused."""
    g = gen(17)
    w = make_q4(g, (8,), 32, 32, dtype)
    T = (2**32 - 1) // (8 + 127) - 16
    x = torch.randn(T, 32, generator=g, device=DEV, dtype=dtype)
    y = gsi.gsi_q4_linear(w, x)
    at = torch.cat([torch.arange(0, T, 300007, device=DEV), torch.arange(T - 40, T, device=DEV)])
    W, S = q4_64(w)
    X = f64(x[at])
    close(y[at], X @ W.T, np.abs(X) @ S.T, 32, dtype, "narrow")


# ---- grouped maps ----


def make_weights(g, kind, n, d_out, d):
    if kind == "q4":
        return make_q4(g, (n, d_out), d, 64, BF16)
    return (torch.randn(n, d_out, d, generator=g, device=DEV) * d**-0.5).to(BF16 if kind == "bf16" else F32)


def check_grouped(w, kind, x, offsets, rows, y, before, what):
    n = len(offsets) - 1
    off, rws = ints(offsets), None if rows is None else ints(rows)
    Ws, Ss = zip(*[q4_64(w, e) if kind == "q4" else (f64(w[e]), np.abs(f64(w[e]))) for e in range(n)])
    X = f64(x)
    with np.errstate(invalid="ignore"):
        ref = orc.grouped_linear(Ws, X, off, rws, f64(before))
        size = orc.grouped_linear(Ss, np.abs(X), off, rws, np.zeros(before.shape))
    lo, hi = int(off[0]), int(off[-1])
    close(y[lo:hi], ref[lo:hi], size[lo:hi], X.shape[1], y.dtype, what)
    assert torch.equal(bits(y[:lo]), bits(before[:lo])) and torch.equal(bits(y[hi:]), bits(before[hi:])), what


def to_offsets(counts, first=0):
    return torch.tensor(np.concatenate([[first], first + np.cumsum(counts)]), dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "q4"])
@pytest.mark.parametrize("d,d_out,counts", [
    (64, 24, [1]), (96, 8, [0, 1, 0]), (160, 40, [3, 0, 16, 17, 1]), (256, 136, [0, 0, 200, 0, 5]),
    (1056, 264, [1] * 9), (288, 72, [i % 4 for i in range(150)]), (512, 384, [130, 127, 0, 1, 129, 257]),
    (672, 520, [64, 65, 63, 0, 300]), (2048, 256, [33, 31, 500]), (128, 128, [1000, 1]),
    (5152, 72, [16, 2, 0, 5]),
])
def test_grouped_linear(d, d_out, counts, kind):
    g = gen(d + d_out + len(counts))
    n, R = len(counts), sum(counts)
    T = max(1, R // 2)
    w = make_weights(g, kind, n, d_out, d)
    x = torch.randn(T, d, generator=g, device=DEV).to(F32 if kind == "fp32" else BF16)
    # three rows before and five behind the experts' are left as they were
    offsets = to_offsets(counts, first=3)
    rows = torch.randint(0, T, (R + 8,), generator=g, device=DEV, dtype=torch.int32)
    before = torch.randn(R + 8, d_out, generator=g, device=DEV).to(x.dtype)
    y = before.clone()
    gsi.gsi_grouped_linear(w, x, offsets, rows, y=y)
    check_grouped(w, kind, x, offsets, rows, y, before, f"grouped {kind} {d}x{d_out} {counts[:8]}")
    again = before.clone()
    gsi.gsi_grouped_linear(w, x, offsets, rows, y=again)
    assert torch.equal(bits(again), bits(y))


@pytest.mark.parametrize("kind", ["bf16", "fp32", "q4"])
@pytest.mark.parametrize("counts", [[2, 0, 3], [90, 0, 170]], ids=["few", "many"])
def test_grouped_without_rows_and_with_rows_that_name_nothing(kind, counts):
    g = gen(sum(counts))
    R, d, d_out = sum(counts), 192, 264
    w = make_weights(g, kind, 3, d_out, d)
    x = torch.randn(R, d, generator=g, device=DEV).to(F32 if kind == "fp32" else BF16)
    offsets = to_offsets(counts)
    before = torch.full((R, d_out), 7.0, device=DEV, dtype=x.dtype)
    check_grouped(w, kind, x, offsets, None, gsi.gsi_grouped_linear(w, x, offsets), before, f"{kind} no rows")
    rows = torch.randint(0, R, (R,), generator=g, device=DEV, dtype=torch.int32)
    rows[0], rows[R // 2], rows[R - 1] = -1, R, 2**31 - 1
    x[0, 0] = float("nan")  # row 0 stands in for no other row
    rows[rows == 0] = 1
    check_grouped(w, kind, x, offsets, rows, gsi.gsi_grouped_linear(w, x, offsets, rows), before, f"{kind} bad rows")


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_grouped_weights_any_stride_apart(kind):
    """Maps as slices of a fused tensor, e.g. the second half of gate and up."""
    g = gen(77)
    both = make_weights(g, kind, 4, 2 * 72, 160)
    w = both[:, 72:]
    x = torch.randn(50, 160, generator=g, device=DEV).to(both.dtype)
    offsets = to_offsets([20, 0, 29, 1])
    y = gsi.gsi_grouped_linear(w, x, offsets)
    check_grouped(w, kind, x, offsets, None, y, torch.zeros_like(y), "fused slice")


@pytest.mark.parametrize("kind", ["bf16", "fp32", "q4"])
def test_grouped_bad_offsets_are_clamped(kind):
    """Offsets outside [0, R] or decreasing write nothing outside y."""
    g = gen(12)
    w = make_weights(g, kind, 4, 136, 128)
    x = torch.randn(40, 128, generator=g, device=DEV).to(F32 if kind == "fp32" else BF16)
    guard = torch.full((60, 136), 3.0, device=DEV, dtype=x.dtype)
    y = guard[10:50]
    gsi.gsi_grouped_linear(w, x, torch.tensor([-9, 30, 5, 2**31 - 1, -5], dtype=torch.int32, device=DEV), y=y)
    torch.cuda.synchronize()
    assert bool((guard[:10] == 3.0).all()) and bool((guard[50:] == 3.0).all())


@pytest.mark.parametrize("kind", ["bf16", "q4"])
@pytest.mark.parametrize("T", [6, 150])
def test_grouped_non_finite_rows_stay_alone(kind, T):
    g = gen(13)
    w = make_weights(g, kind, 2, 136, 224)
    x = torch.randn(T, 224, generator=g, device=DEV).to(BF16)
    offsets = to_offsets([T // 2, T - T // 2])
    ref = gsi.gsi_grouped_linear(w, x, offsets)
    z = x.clone()
    z[T // 2 - 1, 223] = float("inf")
    y = gsi.gsi_grouped_linear(w, z, offsets)
    keep = [t for t in range(T) if t != T // 2 - 1]
    assert torch.equal(bits(y[keep]), bits(ref[keep])) and not torch.isfinite(y[T // 2 - 1]).any()


@pytest.mark.parametrize("kind", ["bf16", "q4"])
@pytest.mark.parametrize("R", [2, 140])
def test_grouped_addresses_past_32_bits(kind, R):
    """The last expert's weights and the last rows of x and y lie beyond 2^32 bytes and 2^31 elements."""
    g = gen(14)
    d, d_out = 8192, 8192
    n = 34 if kind == "bf16" else 66
    if kind == "bf16":
        w = torch.zeros(n, d_out, d, device=DEV, dtype=BF16)
        w[-1].normal_(0, d**-0.5, generator=g)
    else:
        codes = torch.zeros(n, d_out, d // 2, device=DEV, dtype=torch.uint8)
        codes[-1] = torch.randint(0, 256, (d_out, d // 2), generator=g, device=DEV, dtype=torch.uint8)
        w = gsi.Q4(codes, torch.full((n, d_out, d // 128), 0.01, device=DEV, dtype=BF16), None, group=128)
    ld = (1 << 31) // (R - 1) // 8 * 8 + 64
    x = torch.empty_strided((R, d), (ld, 1), device=DEV, dtype=BF16)
    x.copy_(torch.randn(R, d, generator=g, device=DEV))
    y = torch.empty_strided((R, d_out), (ld, 1), device=DEV, dtype=BF16)
    offsets = to_offsets([0] * (n - 1) + [R])
    gsi.gsi_grouped_linear(w, x, offsets, y=y)
    some = torch.arange(0, d_out, 61, device=DEV)
    if kind == "bf16":
        W = f64(w[-1][some])
        S = np.abs(W)
    else:
        W, S = q4_64(gsi.Q4(w.codes[-1][some], w.scales[-1][some].contiguous(), None, group=128))
    X = f64(x)
    close(y[:, some], X @ W.T, np.abs(X) @ S.T, d, BF16, f"far {kind}")


# ---- many rows: the tiled kernels ----

# 256 x 128 tiles for 4 bits, 256 x 256 and 64 x 64 ones for bf16, 64 x 64 for fp32
TILED = [("q4", 1048), ("bf16", 2056), ("bf16", 264), ("fp32", 264)]
RAGGED = [1300, 0, 257, 700, 128, 1, 193]


@pytest.mark.parametrize("d", [96, 288, 1056])
@pytest.mark.parametrize("kind,d_out", TILED)
def test_grouped_many_rows(kind, d_out, d):
    g = gen(d + d_out)
    R, T = sum(RAGGED), 900
    w = make_weights(g, kind, len(RAGGED), d_out, d)
    x = torch.randn(T, d, generator=g, device=DEV).to(F32 if kind == "fp32" else BF16)
    offsets = to_offsets(RAGGED, first=3)
    rows = torch.randint(1, T, (R + 8,), generator=g, device=DEV, dtype=torch.int32)
    rows[3], rows[5 + R // 2], rows[R + 2] = -1, T, 2**31 - 1
    x[0] = float("nan")  # row 0 stands in for no other row
    wide = torch.randn(R + 8, d_out + 16, generator=g, device=DEV).to(x.dtype)
    before, y = wide.clone(), wide.clone()
    gsi.gsi_grouped_linear(w, x, offsets, rows, y=y[:, 8:-8])
    check_grouped(w, kind, x, offsets, rows, y[:, 8:-8], before[:, 8:-8], f"many {kind} {d}x{d_out}")
    assert torch.equal(bits(y[:, :8]), bits(before[:, :8])) and torch.equal(bits(y[:, -8:]), bits(before[:, -8:]))
    again = before.clone()
    gsi.gsi_grouped_linear(w, x, offsets, rows, y=again[:, 8:-8])
    assert torch.equal(bits(again), bits(y))


@pytest.mark.parametrize("kind,d_out", TILED)
def test_grouped_many_rows_non_finite_and_bad_offsets(kind, d_out):
    g = gen(d_out + 1)
    R, d = sum(RAGGED), 160
    w = make_weights(g, kind, len(RAGGED), d_out, d)
    x = torch.randn(R, d, generator=g, device=DEV).to(F32 if kind == "fp32" else BF16)
    offsets = to_offsets(RAGGED)
    ref = gsi.gsi_grouped_linear(w, x, offsets)
    for at, bad in ((0, float("inf")), (1299, float("nan")), (R - 1, float("-inf"))):
        z = x.clone()
        z[at, d - 1] = bad
        y = gsi.gsi_grouped_linear(w, z, offsets)
        keep = [t for t in range(R) if t != at]
        assert torch.equal(bits(y[keep]), bits(ref[keep])) and not torch.isfinite(y[at]).any()
    guard = torch.full((R + 20, d_out), 3.0, device=DEV, dtype=x.dtype)
    bad = torch.tensor([-9, 1500, 5, 2**31 - 1, -5, 900, 2**31 - 1, -2**31], dtype=torch.int32, device=DEV)
    gsi.gsi_grouped_linear(w, x, bad, y=guard[10:10 + R])
    torch.cuda.synchronize()
    assert bool((guard[:10] == 3.0).all()) and bool((guard[10 + R:] == 3.0).all())


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("d,T", [(96, 2305), (416, 2400), (1056, 2560)])
def test_q4_many_tokens(d, T, group):
    g = gen(d + T + group)
    w = make_q4(g, (1048,), d, group, BF16, zeros=T % 2 == 1)
    wide = torch.full((T, d + 24), float("nan"), device=DEV, dtype=BF16)
    x = wide[:, 8:8 + d]
    x.copy_(torch.randn(T, d, generator=g, device=DEV))
    x[:, d // 3] *= 30
    y = gsi.gsi_q4_linear(w, x)
    W, S = q4_64(w)
    X = f64(x)
    close(y, X @ W.T, np.abs(X) @ S.T, d, BF16, f"q4 {d} {T} {group}")


@pytest.mark.parametrize("kind,n,d,d_out,R", [("q4", 10, 131072, 8192, 2400), ("fp32", 17, 8192, 8192, 400)])
def test_grouped_many_rows_past_32_bits(kind, n, d, d_out, R):
    """As above for the tiles: the last expert's weights and the last rows lie far behind the first."""
    g = gen(15)
    dtype = BF16 if kind == "q4" else F32
    if kind == "q4":
        codes = torch.zeros(n, d_out, d // 2, device=DEV, dtype=torch.uint8)
        codes[-1] = torch.randint(0, 256, (d_out, d // 2), generator=g, device=DEV, dtype=torch.uint8)
        w = gsi.Q4(codes, torch.full((n, d_out, d // 128), 0.01, device=DEV, dtype=BF16), None, group=128)
    else:
        w = torch.zeros(n, d_out, d, device=DEV)
        w[-1].normal_(0, d**-0.5, generator=g)
    ld = (1 << 31) // (R - 1) // 8 * 8 + 64
    x = torch.empty_strided((R, d), (max(ld, d), 1), device=DEV, dtype=dtype)
    x.copy_(torch.randn(R, d, generator=g, device=DEV))
    y = torch.empty_strided((R, d_out), (ld, 1), device=DEV, dtype=dtype)
    gsi.gsi_grouped_linear(w, x, to_offsets([0] * (n - 1) + [R]), y=y)
    some, at = torch.arange(0, d_out, 211, device=DEV), torch.arange(0, R, 57, device=DEV)
    if kind == "q4":
        W, S = q4_64(gsi.Q4(w.codes[-1][some], w.scales[-1][some].contiguous(), None, group=128))
    else:
        W = f64(w[-1][some])
        S = np.abs(W)
    X = f64(x[at])
    close(y[at][:, some], X @ W.T, np.abs(X) @ S.T, d, dtype, f"far tiles {kind}")


# full tiles of 256 rows and rests of each of the four heights
TURNS = [1300, 0, 257, 700, 64, 1, 193, 512, 130, 900, 0, 320, 15]


@pytest.mark.parametrize("d,d_out", [(160, 8200), (416, 8200), (1048, 4104), (128, 4104)])
def test_grouped_many_tiles_of_a_workgroup(d, d_out):
    """bf16 tiles for several turns of every workgroup: 792 (d_out 8200) and 408
    tiles on 256 workgroups, each turn another expert, height or column.  All of
    y is compared, on the GPU, against products in 64 bits."""
    g = gen(d + d_out)
    n, R, T = len(TURNS), sum(TURNS), 1500
    w = make_weights(g, "bf16", n, d_out, d)
    x = torch.randn(T, d, generator=g, device=DEV).to(BF16)
    x[0] = float("nan")  # row 0 stands in for no other row
    offsets = to_offsets(TURNS, first=3)
    rows = torch.randint(1, T, (R + 8,), generator=g, device=DEV, dtype=torch.int32)
    rows[3], rows[5 + R // 2], rows[R + 2] = -1, T, 2**31 - 1
    before = torch.full((R + 8, d_out), 7.0, device=DEV, dtype=BF16)
    y, again = before.clone(), before.clone()
    gsi.gsi_grouped_linear(w, x, offsets, rows, y=y)
    gsi.gsi_grouped_linear(w, x, offsets, rows, y=again)
    assert torch.equal(bits(y), bits(again))
    assert bool((y[:3] == 7).all()) and bool((y[R + 3:] == 7).all())
    at = ints(offsets)
    for e in range(n):
        src = rows[at[e]:at[e + 1]].long()
        has = ((src >= 0) & (src < T))[:, None]
        X = torch.where(has, x[src.clamp(0, T - 1)].double(), 0.0)
        W = w[e].double()
        ref, size = X @ W.T, X.abs() @ W.abs().T
        # half a step of y and the fp32 sums, as in close()
        tol = 2.0**-8 * ref.abs() * 1.001 + (1 + 2.0**-8) * (d / 16 + 64) * 2.0**-23 * size + 1e-30
        off = (y[at[e]:at[e + 1]].double() - ref).abs()
        assert bool((off <= tol).all()), f"expert {e}: {int((off > tol).sum())} off"
        norm = ref.norm(dim=1)
        rel = (off.norm(dim=1)[norm > 0] / norm[norm > 0])
        assert rel.numel() == 0 or float(rel.max()) <= 2.0**-8 + 1e-5


@pytest.mark.parametrize("n,d,d_out,R", [(34, 8192, 8192, 2400), (34, 131072, 768, 400)], ids=["large tiles", "small tiles"])
def test_grouped_many_bf16_rows_past_32_bits(n, d, d_out, R):
    """The bf16 tiles: the last expert's weights and the last rows of x and y lie
    beyond 2^32 bytes, the rows beyond 2^31 elements."""
    g = gen(16)
    w = torch.zeros(n, d_out, d, device=DEV, dtype=BF16)
    w[-1].normal_(0, d**-0.5, generator=g)
    ld = (1 << 31) // (R - 1) // 8 * 8 + 64
    x = torch.empty_strided((R, d), (ld, 1), device=DEV, dtype=BF16)
    x.copy_(torch.randn(R, d, generator=g, device=DEV))
    y = torch.empty_strided((R, d_out), (ld, 1), device=DEV, dtype=BF16)
    gsi.gsi_grouped_linear(w, x, to_offsets([0] * (n - 1) + [R]), y=y)
    some, at = torch.arange(0, d_out, 61, device=DEV), torch.arange(R - 1, 0, -57, device=DEV)
    W, X = f64(w[-1][some]), f64(x[at])
    close(y[at][:, some], X @ W.T, np.abs(X) @ np.abs(W).T, d, BF16, f"far bf16 tiles {d_out}")


@pytest.mark.parametrize("zeros", [True, False], ids=["zeros", "eights"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d,d_out,counts", [(96, 24, [1, 0, 2]), (1056, 264, [3, 0, 17, 1, 33]), (416, 1048, RAGGED)],
                         ids=["few", "some", "many"])
def test_grouped_q4_of_every_type(d, d_out, counts, dtype, group, zeros):
    """Experts in 4 bits with bf16 and fp32 x, every group size, with zeros and without."""
    g = gen(d + group + len(counts))
    n, R, T = len(counts), sum(counts), 700
    w = make_q4(g, (n, d_out), d, group, dtype, zeros=zeros)
    x = torch.randn(T, d, generator=g, device=DEV).to(dtype)
    x[:, d // 3] *= 30
    x[0] = float("nan")  # row 0 stands in for no other row
    offsets = to_offsets(counts, first=3)
    rows = torch.randint(1, T, (R + 8,), generator=g, device=DEV, dtype=torch.int32)
    rows[3], rows[R + 2] = -1, T
    wide = torch.randn(R + 8, d_out + 16, generator=g, device=DEV).to(dtype)
    before, y = wide.clone(), wide.clone()
    gsi.gsi_grouped_linear(w, x, offsets, rows, y=y[:, 8:-8])
    check_grouped(w, "q4", x, offsets, rows, y[:, 8:-8], before[:, 8:-8], f"q4 {dtype} {d}x{d_out} group {group}")
    assert torch.equal(bits(y[:, :8]), bits(before[:, :8])) and torch.equal(bits(y[:, -8:]), bits(before[:, -8:]))
    again = before.clone()
    gsi.gsi_grouped_linear(w, x, offsets, rows, y=again[:, 8:-8])
    assert torch.equal(bits(again), bits(y))


@pytest.mark.parametrize("kind", ["bf16", "q4"])
@pytest.mark.parametrize("R", [40, 6000])
def test_grouped_over_thousands_of_experts(kind, R):
    g = gen(R)
    n, d, d_out = 3000, 32, 16
    w = make_weights(g, kind, n, d_out, d)
    ids = torch.randint(0, n, (R, 1), generator=g, device=DEV)
    offsets = torch.searchsorted(torch.sort(ids[:, 0]).values, torch.arange(n + 1, device=DEV)).to(torch.int32)
    x = torch.randn(R, d, generator=g, device=DEV).to(BF16)
    before = torch.zeros(R, d_out, device=DEV, dtype=BF16)
    check_grouped(w, kind, x, offsets, None, gsi.gsi_grouped_linear(w, x, offsets), before, f"{n} experts {kind}")


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,T", [(BF16, 1), (BF16, 40), (BF16, 2560), (F32, 19)])
def test_q4_reads_the_low_four_bits_of_a_zero(dtype, T, group):
    g = gen(T + group)
    w = make_q4(g, (1048,), 416, group, dtype)
    x = torch.randn(T, 416, generator=g, device=DEV).to(dtype)
    y = gsi.gsi_q4_linear(w, x)
    high = w.zeros | (torch.randint(0, 16, w.zeros.shape, generator=g, device=DEV, dtype=torch.uint8) << 4)
    assert torch.equal(bits(gsi.gsi_q4_linear(gsi.Q4(w.codes, w.scales, high, group=group), x)), bits(y))


@pytest.mark.parametrize("kind,d_out", TILED)
def test_many_rows_captured_and_replayed(kind, d_out):
    """The tiles and the three launches of the ordering in one graph, on other
    choices and values at every replay, with eager work between them."""
    g = gen(d_out + 2)
    n, d, T, top = 7, 160, 11000, 3
    dtype = F32 if kind == "fp32" else BF16
    w = make_weights(g, kind, n, d_out, d)
    x, out = torch.empty(T, d, device=DEV, dtype=dtype), torch.empty(T, d_out, device=DEV, dtype=dtype)
    ids = torch.zeros(T, top, device=DEV, dtype=torch.int32)
    weights = torch.rand(T, top, generator=g, device=DEV)

    def block(x, ids, out):
        offsets, rows, pos = gsi.gsi_group_rows(ids, n)
        y = gsi.gsi_grouped_linear(w, x, offsets, rows)
        return gsi.gsi_group_combine(y, pos, weights, out=out)

    def fill():
        x.copy_(torch.randn(T, d, generator=g, device=DEV))
        ids.copy_(torch.randint(-1, n, (T, top), generator=g, device=DEV))
    fill()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        block(x, ids, out)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        block(x, ids, out)
    for k in range(4):
        fill()
        want = block(x.clone(), ids.clone(), torch.empty_like(out))
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(out), bits(want)), f"replay {k}"


# ---- grouping and combining ----


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64], ids=["int32", "int64"])
@pytest.mark.parametrize("T,top,n", [(1, 1, 1), (1, 8, 64), (5, 2, 3), (64, 1, 7), (333, 3, 65), (1024, 6, 256),
                                     (700, 4, 1024), (20000, 2, 16),
                                     (4095, 8, 256), (4096, 8, 3), (33000, 1, 1), (9001, 5, 1024), (16389, 8, 256)])
def test_group_rows(T, top, n, dtype):
    g = gen(T + n)
    ids = torch.randint(-1 if T % 2 else 0, n + T % 2, (T, top), generator=g, device=DEV).to(dtype)
    if T > 300:
        ids[T // 2:T // 2 + 99] = n - 1  # one long run, and numbers far outside
        ids[3, 0] = torch.iinfo(dtype).max
        ids[5, top - 1] = torch.iinfo(dtype).min
        if dtype == torch.int64:
            ids[7, 0] = 1 << 32  # must not wrap to expert 0
    for got, want in zip(gsi.gsi_group_rows(ids, n), orc.group_rows(ints(ids), n)):
        assert np.array_equal(ints(got), want)


def test_group_rows_all_dropped_all_same_and_empty():
    ids = torch.full((70, 2), -1, device=DEV, dtype=torch.int32)
    o, r, p = gsi.gsi_group_rows(ids, 5)
    assert ints(o).tolist() == [0] * 6 and bool((r == -1).all()) and bool((p == -1).all())
    o, r, p = gsi.gsi_group_rows(ids + 5, 5)  # the last expert takes everything
    assert ints(o).tolist() == [0] * 5 + [140] and torch.equal(p.flatten(), torch.arange(140, device=DEV).int())
    o, r, p = gsi.gsi_group_rows(ids[:0], 5)
    assert ints(o).tolist() == [0] * 6


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,top,d,how", [(1, 1, 8, "all"), (3, 8, 4096, "all"), (65, 2, 264, "plain"),
                                         (130, 5, 1000, "base"), (17, 64, 72, "weights"), (300, 3, 2056, "all")])
def test_group_combine(T, top, d, how, dtype):
    g = gen(T + d)
    R = T * top
    y = torch.randn(R, d, generator=g, device=DEV).to(dtype)
    pos = torch.randint(-2, R + 2, (T, top), generator=g, device=DEV, dtype=torch.int32)
    if T > 1:
        pos[1] = -1  # a token without experts, and one that names one row twice
        pos[0, 0] = pos[0, top - 1]
    weights = torch.randn(T, top, generator=g, device=DEV) if how in ("all", "weights") else None
    if weights is not None and T > 1:
        weights[1] = float("nan")  # a weight of nothing
    base = torch.randn(T, d, generator=g, device=DEV).to(dtype) if how in ("all", "base") else None
    out = gsi.gsi_group_combine(y, pos, weights, base=base)
    ref = orc.group_combine(f64(y), ints(pos), f64(weights), f64(base))
    size = orc.group_combine(np.abs(f64(y)), ints(pos), None if weights is None else np.abs(f64(weights)),
                             None if base is None else np.abs(f64(base)))
    half = torch.finfo(dtype).eps / 2
    # top products and additions in fp32, then one rounding
    assert (np.abs(f64(out) - ref) <= half * np.abs(ref) * 1.001 + (top + 2) * 2.0**-23 * size).all()
    if base is not None:  # onto the residual itself
        assert gsi.gsi_group_combine(y, pos, weights, base=base, out=base) is base
        assert torch.equal(bits(base), bits(out))


def test_group_combine_no_rows_and_strides():
    base = torch.randn(9, 96, device=DEV)
    pos = torch.zeros(9, 2, device=DEV, dtype=torch.int32)
    assert torch.equal(gsi.gsi_group_combine(torch.empty(0, 96, device=DEV), pos, base=base), base)
    y = torch.randn(4, 128, device=DEV)[:, 16:112]
    out = torch.full((9, 104), 2.0, device=DEV)
    gsi.gsi_group_combine(y, pos + 3, base=base, out=out[:, 4:100])
    # the documented order: base, then one row after the other
    assert torch.equal(out[:, 4:100], (base + y[3]) + y[3])
    assert bool((out[:, :4] == 2).all()) and bool((out[:, 100:] == 2).all())


# ---- together: the linear maps of an expert block ----


def expert_block(x, router, up, down, n, top, out):
    """Route, group, up, activate, down, combine onto x."""
    score = torch.softmax((x.float() @ router).float(), dim=1)
    weights, ids = torch.topk(score, top, dim=1)
    offsets, rows, pos = gsi.gsi_group_rows(ids, n)
    h = gsi.gsi_grouped_linear(up, x, offsets, rows)
    a, b = h.float().chunk(2, dim=1)
    h = (torch.nn.functional.silu(a) * b).to(x.dtype)
    y = gsi.gsi_grouped_linear(down, h, offsets)
    return ids, weights, gsi.gsi_group_combine(y, pos, weights, base=x, out=out)


@pytest.mark.parametrize("kind", ["bf16", "fp32", "q4"])
@pytest.mark.parametrize("T", [1, 9, 200])
def test_expert_block_eager_and_replayed(T, kind):
    g = gen(T)
    n, top, d, ff = 12, 3, 256, 192
    dtype = F32 if kind == "fp32" else BF16
    x = torch.randn(T, d, generator=g, device=DEV).to(dtype)
    router = torch.randn(d, n, generator=g, device=DEV)
    up, down = make_weights(g, kind, n, 2 * ff, d), make_weights(g, kind, n, d, ff)
    out = torch.empty_like(x)
    ids, weights, _ = expert_block(x, router, up, down, n, top, out)
    ups = [q4_64(up, e)[0] if kind == "q4" else f64(up[e]) for e in range(n)]
    downs = [q4_64(down, e)[0] if kind == "q4" else f64(down[e]) for e in range(n)]
    ref = f64(x).copy()
    for t in range(T):
        for j in range(top):
            h = ups[int(ids[t, j])] @ f64(x[t])
            a, b = h[:ff], h[ff:]
            ref[t] += float(weights[t, j]) * (downs[int(ids[t, j])] @ (a / (1 + np.exp(-a)) * b))
    err = np.linalg.norm(f64(out) - ref, axis=1) / np.linalg.norm(ref, axis=1)
    # bf16: h is rounded twice on its way (up to 3 half steps of h in the product), y once, out once: 6 half steps
    assert err.max() <= (6 * 2.0**-8 if dtype == BF16 else 1e-5), err.max()

    # the same call sequence captured once and replayed on other inputs, with eager work between
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    fixed, result = x.clone(), torch.empty_like(x)
    with torch.cuda.stream(stream):
        expert_block(fixed, router, up, down, n, top, result)
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        expert_block(fixed, router, up, down, n, top, result)
    for k in range(4):
        new = torch.randn(T, d, generator=g, device=DEV).to(dtype)
        want = expert_block(new, router, up, down, n, top, torch.empty_like(x))[2].clone()
        fixed.copy_(new)
        result.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(bits(result), bits(want)), f"replay {k}"


def test_two_streams_at_once():
    """Calls keep no state: two streams running different calls give what each gives alone."""
    g = gen(21)
    w = make_q4(g, (1024,), 1024, 128, BF16)
    xs = [torch.randn(t, 1024, generator=g, device=DEV).to(BF16) for t in (1, 200)]
    alone = [gsi.gsi_q4_linear(w, x) for x in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    ys = [[torch.empty_like(a) for _ in range(20)] for a in alone]
    for k in range(20):
        for s, x, y in zip(streams, xs, ys):
            gsi.gsi_q4_linear(w, x, y=y[k], stream=s)
    torch.cuda.synchronize()
    for a, y in zip(alone, ys):
        assert all(torch.equal(bits(a), bits(v)) for v in y)


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_new_outputs_belong_to_the_stream_of_the_call(raw):
    """An output is not put where work of the current stream is still to write."""
    g = gen(22)
    w = make_q4(g, (1024,), 1024, 128, BF16)
    x = torch.randn(512, 1024, generator=g, device=DEV).to(BF16)
    ids = torch.randint(0, 8, (1 << 19, 1), generator=g, device=DEV).to(torch.int32)
    want, order = gsi.gsi_q4_linear(w, x), gsi.gsi_group_rows(ids, 8)
    a = torch.randn(4096, 4096, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    junk = [torch.empty_like(want), torch.empty(2 * ids.numel() + 9, device=DEV, dtype=torch.int32)]
    for _ in range(20):
        a = a @ a * 1e-3
    for j in junk:
        j.fill_(7)
    del junk, j
    stream = side.cuda_stream if raw else side
    y = gsi.gsi_q4_linear(w, x, stream=stream)
    got = gsi.gsi_group_rows(ids, 8, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(bits(y), bits(want)) and all(torch.equal(p, q) for p, q in zip(got, order))
