"""The paged key-value cache on the GPU against the fp64 oracle: rotary
positions, appending, attention of one new token, eviction.

Tolerances.  A result is rounded once: half a step, finfo.eps / 2 relative to
the value.  Before that
  - a rotation: the angle, reduced to r in [-1/2, 1/2] turns in 64 bits, is
    rounded to fp32 (2^-25 of a half turn: pi 2^-25 rad), sine and cosine are
    off by 2^-22 at most, the amplitude, two products and a sum round by 2^-24
    each: below 2^-20 (|x0| + |x1|) amplitude; and p f in 64 bits 2^-51 p f rad.
  - a score, d products in fp32: off by delta = (d + 8) 2^-24 scale sum |q k|,
    and its exponential by (|score| + |top| + 8) 2^-23 more: together the
    relative error w of a weight, in numerator and denominator: 2 w.  Weights as
    two bf16 parts: 2^-16.  A sum over n slots takes part in at most n / 16 + 64
    rounded additions (joined in tiles of 16 and more): (n / 16 + 64) 2^-23.
Entries that are moved or copied are equal bit for bit."""
import numpy as np
import pytest
import torch

from oracle import cache_oracle as orc
from rank_gated_memory_amd import gsi

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32
DTYPES = pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "fp32"])


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def ints(t):
    return t.detach().cpu().numpy()


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def bits(t):
    return t.contiguous().view(torch.int16 if t.element_size() == 2 else torch.int32)


def within(y, ref, tol, what):
    y = f64(y)
    with np.errstate(invalid="ignore"):  # inf - inf: those are equal or bad
        bad = ~((np.abs(y - ref) <= tol) | ((y == ref) & np.isinf(ref)))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, first at {np.argwhere(bad)[0]}: " \
        f"{y[bad][0]} for {ref[bad][0]}"


def half(dtype):
    return torch.finfo(dtype).eps / 2


# ---- a pool, its tables and its copy for the oracle ----


def make_pool(g, seqs, lengths, heads, page, d, dtype, most=None, spare=3, age=True, transposed=False):
    """Pages in shuffled order; what no sequence's slots hold is NaN (mass, age: far off)."""
    most = max(1, -(-max(max(lengths), 1) // page)) if most is None else most
    count = seqs * most + spare
    shape = (count, page, heads, d) if transposed else (count, heads, page, d)
    K, V = (torch.randn(shape, generator=g, device=DEV).to(dtype) for _ in range(2))
    if transposed:
        K, V = K.transpose(1, 2), V.transpose(1, 2)
    mass = torch.rand(count, heads, page, generator=g, device=DEV)
    ages = torch.randint(0, 1 << 16, (count, heads, page), generator=g, device=DEV, dtype=torch.int32) if age else None
    order = torch.randperm(count, generator=g, device=DEV).int()
    table = order[:seqs * most].view(seqs, most).contiguous()
    used = torch.zeros(count, page, dtype=torch.bool, device=DEV)
    for s, n in enumerate(lengths):
        i = torch.arange(min(n, most * page), device=DEV)
        used[table[s].long()[i // page], i % page] = True
    free = ~used[:, None, :].expand(count, heads, page)
    K[free], V[free] = float("nan"), float("nan")
    mass[free] = float("nan")
    if age:
        ages[free] = 2**31 - 1
    return gsi.Cache(K, V, mass=mass, age=ages), table


def copy_of(c):
    """The pool for the oracle."""
    return {"K": f64(c.K), "V": f64(c.V), "mass": f64(c.mass), "age": None if c.age is None else ints(c.age).copy()}


def same_pool(c, pool, what):
    for name in ("K", "V", "mass", "age"):
        t = getattr(c, name)
        if t is not None:
            y = ints(t) if name == "age" else f64(t)
            assert np.array_equal(y, pool[name], equal_nan=name != "age"), f"{what}: {name}"


# ---- rotary positions ----


def check_rotary(y, x, positions, freqs, layout, start, amplitude, dtype, what):
    ref = orc.rotary(f64(x), ints(positions), f64(freqs), layout, start, amplitude)
    X, n = np.abs(f64(x)), freqs.numel()
    size, slow = np.zeros_like(ref), np.zeros_like(ref)
    e = (start + 2 * np.arange(n), start + 2 * np.arange(n) + 1) if layout == "pairs" \
        else (start + np.arange(n), start + n + np.arange(n))
    angle = np.abs(ints(positions).astype(np.float64))[:, None, None] * np.abs(f64(freqs))
    for k in e:
        size[:, :, k] = (X[:, :, e[0]] + X[:, :, e[1]]) * abs(amplitude)
        slow[:, :, k] = angle
    turned = size > 0
    within(y, ref, half(dtype) * np.abs(ref) * 1.001 * turned + size * (2.0**-20 + slow * 2.0**-51), what)


@DTYPES
@pytest.mark.parametrize("layout", ["pairs", "halves"])
@pytest.mark.parametrize("T,heads,d,turned,start", [
    (1, 1, 8, 2, 0), (1, 16, 256, 64, 0), (3, 5, 80, 80, 0), (7, 3, 128, 128, 0), (2, 40, 128, 64, 64), (5, 2, 72, 20, 6),
    (33, 7, 64, 62, 2), (1, 300, 24, 8, 16), (2049, 3, 64, 64, 0), (2050, 2, 40, 6, 3), (2311, 1, 256, 256, 0),
    (4, 9, 256, 96, 160),
])
def test_rotary(T, heads, d, turned, start, layout, dtype):
    g = gen(T + heads + d + turned)
    freqs = gsi.rotary_freqs(turned)
    amplitude = 1.0 if T % 2 else 1.3465735
    r = gsi.Rotary(freqs, layout=layout, start=start, amplitude=amplitude, device=DEV)
    x = torch.randn(T, heads, d, generator=g, device=DEV).to(dtype)
    pos = torch.randint(-5, 1 << 20, (T,), generator=g, device=DEV, dtype=torch.int32 if T % 3 else torch.int64)
    y = gsi.gsi_rotary(r, x, pos)
    a32 = float(np.float32(amplitude))
    check_rotary(y, x, pos, freqs, layout, start, a32, dtype, "rotary")
    stay = torch.ones(d, dtype=torch.bool, device=DEV)
    stay[start:start + turned] = False
    assert torch.equal(bits(y[..., stay]), bits(x[..., stay]))
    z = x.clone()  # in place
    assert gsi.gsi_rotary(r, z, pos, y=z) is z
    assert torch.equal(bits(z), bits(y))


@DTYPES
@pytest.mark.parametrize("layout", ["pairs", "halves"])
def test_rotary_every_part_of_a_head(layout, dtype):
    """Parts of every size from every element on, in new rows and in place."""
    g = gen(91)
    x = torch.randn(3, 2, 24, generator=g, device=DEV).to(dtype)
    pos = torch.tensor([7, -3, 100003], device=DEV)
    for turned in range(2, 25, 2):
        for start in range(25 - turned):
            freqs = gsi.rotary_freqs(turned)
            r = gsi.Rotary(freqs, layout=layout, start=start, device=DEV)
            y = gsi.gsi_rotary(r, x, pos)
            check_rotary(y, x, pos, freqs, layout, start, 1.0, dtype, f"{turned} from {start}")
            assert torch.equal(bits(y[..., :start]), bits(x[..., :start]))
            assert torch.equal(bits(y[..., start + turned:]), bits(x[..., start + turned:]))
            z = x.clone()
            gsi.gsi_rotary(r, z, pos, y=z)
            assert torch.equal(bits(z), bits(y)), f"{turned} from {start} in place"


@DTYPES
def test_rotary_strides_and_what_is_left(dtype):
    g = gen(3)
    T, heads, d = 19, 6, 48
    wide = torch.full((T, heads + 3, d + 16), 7.0, device=DEV).to(dtype)
    x = wide[:, 1:1 + heads, 8:8 + d]
    x.copy_(torch.randn(T, heads, d, generator=g, device=DEV))
    out = torch.full((heads + 2, T, d + 8), 5.0, device=DEV).to(dtype)
    y = out[1:1 + heads, :, 8:8 + d].transpose(0, 1)
    freqs = gsi.rotary_freqs(32)
    pos = torch.arange(T, device=DEV) * 1000
    gsi.gsi_rotary(gsi.Rotary(freqs, device=DEV), x, pos, y=y)
    check_rotary(y, x, pos, freqs, "halves", 0, 1.0, dtype, "strided")
    y.fill_(5.0)
    assert bool((out == 5.0).all()), "bytes outside y were written"


def test_rotary_far_positions_and_back():
    """Positions up to 2^31 and more, and that -p undoes p."""
    g = gen(4)
    pos = torch.tensor([0, 1, 2**20 + 1, 2**31 - 1, 2**33 + 5, -(2**31)], device=DEV)
    freqs = gsi.rotary_freqs(64, base=500000.0)
    r = gsi.Rotary(freqs, layout="pairs", device=DEV)
    x = torch.randn(6, 2, 64, generator=g, device=DEV)
    y = gsi.gsi_rotary(r, x, pos)
    check_rotary(y, x, pos, freqs, "pairs", 0, 1.0, F32, "far")
    back = gsi.gsi_rotary(r, y, -pos)
    X = np.abs(f64(x))
    size = X + X.reshape(6, 2, 32, 2)[..., ::-1].reshape(6, 2, 64)
    # two rotations, of sizes that the first has made at most |x0| + |x1|
    within(back, f64(x), 2 * size * 2 * (2.0**-20 + 2.0**-23 + np.abs(ints(pos))[:, None, None] * 2.0**-51), "back")


def test_rotary_of_many_tokens():
    """More tokens than workgroups fit side by side, and row addresses past 32 bits."""
    g = gen(6)
    T = 1 << 20
    wide = torch.empty(T, 2200, device=DEV, dtype=BF16)  # 4.6 GB apart from first to last
    x = wide[:, 64:72].view(T, 1, 8)
    x.copy_(torch.randn(T, 1, 8, generator=g, device=DEV))
    freqs = gsi.rotary_freqs(8)
    r = gsi.Rotary(freqs, device=DEV)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device=DEV)
    y = gsi.gsi_rotary(r, x, pos)
    at = torch.randint(0, T, (300,), generator=g, device=DEV)
    at[:2] = torch.tensor([0, T - 1], device=DEV)
    check_rotary(y[at], x[at], pos[at], freqs, "halves", 0, 1.0, BF16, "many tokens")
    z = gsi.gsi_rotary(r, x[T - 2001:].contiguous(), pos[T - 2001:].contiguous())
    assert torch.equal(bits(z), bits(y[T - 2001:]))


def test_rotary_keeps_rows_apart():
    """A row that is not finite, and no rows at all."""
    g = gen(5)
    r = gsi.Rotary(gsi.rotary_freqs(64), device=DEV)
    x = torch.randn(9, 4, 64, generator=g, device=DEV).to(BF16)
    pos = torch.arange(9, device=DEV, dtype=torch.int32)
    ref = gsi.gsi_rotary(r, x, pos)
    x[4, 1, 5] = float("inf")
    y = gsi.gsi_rotary(r, x, pos)
    same = torch.ones(9, 4, dtype=torch.bool, device=DEV)
    same[4, 1] = False
    assert torch.equal(bits(y[same]), bits(ref[same]))
    assert not torch.isfinite(y[4, 1, 5]) and not torch.isfinite(y[4, 1, 37])
    assert gsi.gsi_rotary(r, x[:0], pos[:0]).shape == (0, 4, 64)


# ---- appending ----


@DTYPES
@pytest.mark.parametrize("T,S,heads,qh,d,page,turned,layout", [
    (1, 1, 1, 1, 8, 8, 0, "pairs"), (1, 1, 16, 16, 256, 16, 64, "pairs"), (48, 48, 8, 32, 128, 16, 128, "halves"),
    (37, 3, 2, 6, 80, 8, 20, "halves"), (130, 2, 5, 0, 72, 64, 72, "pairs"), (2100, 4, 1, 3, 64, 256, 64, "halves"),
    (9, 9, 3, 3, 24, 4096, 0, "halves"),
])
def test_append(T, S, heads, qh, d, page, turned, layout, dtype):
    g = gen(T + heads + d + page)
    each = -(-T // S)
    lengths = [each + 11] * S
    c, table = make_pool(g, S, lengths, heads, page, d, dtype, transposed=T % 2 == 0)
    pool, tab = copy_of(c), ints(table)
    t = torch.arange(T, device=DEV)
    seq, slots = (t % S).int(), (t // S + 5).int()
    slots = torch.where(t % 17 == 16, -1, slots).int()  # padding rows
    pos = (t * 977 + 3).to(torch.int64 if T % 2 else torch.int32)
    qkv = torch.randn(T, qh + 2 * heads, d, generator=g, device=DEV).to(dtype)
    q, k, v = qkv[:, :qh], qkv[:, qh:qh + heads], qkv[:, qh + heads:]
    freqs = gsi.rotary_freqs(turned) if turned else None
    r = gsi.Rotary(freqs, layout=layout, device=DEV) if turned else None
    got = gsi.gsi_cache_append(c, table, slots, k, v, seq=None if S == T else seq, rotary=r, positions=pos,
                               q=q if qh else None)
    # the keys as the rotation alone gives them: held to the oracle above and here
    key = k if r is None else gsi.gsi_rotary(r, k, pos)
    if r is not None:
        check_rotary(key, k, pos, freqs, layout, 0, 1.0, dtype, "keys")
        if qh:
            assert torch.equal(bits(got), bits(gsi.gsi_rotary(r, q, pos)))
    elif qh:
        assert torch.equal(bits(got), bits(q))
    if not qh:
        assert got is None
    orc.append(pool, tab, ints(seq), ints(slots), f64(key), f64(v), ints(pos))
    same_pool(c, pool, "append")


def test_append_writes_nothing_where_there_is_no_slot():
    """Sequences, slots and pages that there are none of; the queries are turned all the same."""
    g = gen(8)
    c, table = make_pool(g, 3, [24, 24, 24], 2, 8, 16, BF16)
    table[1, 1] = c.pages
    table[2, 0] = -7
    pool = copy_of(c)
    seq = torch.tensor([0, 0, 0, -1, 3, 1, 1, 2, 2, 0], device=DEV, dtype=torch.int32)
    slots = torch.tensor([3, 24, -1, 2, 2, 9, 23, 1, 10, 2**31 - 1], device=DEV, dtype=torch.int32)
    k, v = (torch.randn(10, 2, 16, generator=g, device=DEV).to(BF16) for _ in range(2))
    q = torch.randn(10, 4, 16, generator=g, device=DEV).to(BF16)
    pos = torch.tensor([5, 2**40, -(2**40), 1, 1, 1, 2**31 + 7, 1, -(2**33), 1], device=DEV)
    r = gsi.Rotary(gsi.rotary_freqs(16), device=DEV)
    key = gsi.gsi_rotary(r, k, pos)
    out = gsi.gsi_cache_append(c, table, slots, k, v, seq=seq, rotary=r, positions=pos, q=q)
    assert torch.equal(bits(out), bits(gsi.gsi_rotary(r, q, pos)))
    orc.append(pool, ints(table), ints(seq), ints(slots), f64(key), f64(v), ints(pos))
    same_pool(c, pool, "append of nothing")
    gsi.gsi_cache_append(c, table, slots[:0], k[:0], v[:0])
    # ages without positions are the slots
    gsi.gsi_cache_append(c, table, slots, k, v, seq=seq)
    orc.append(pool, ints(table), ints(seq), ints(slots), f64(k), f64(v))
    same_pool(c, pool, "append without positions")


# ---- attention ----


def check_attend(c, table, lengths, q, scale=None, window=0, accumulate=False, what="attend", **kw):
    pool = copy_of(c)
    d = c.d
    scale = d**-0.5 if scale is None else scale
    ref, lse, mass, size, big = orc.attend(pool, ints(table), ints(lengths), f64(q), float(np.float32(scale)), window)
    out, l = gsi.gsi_cache_attend(c, table, lengths, q, scale=scale, window=window, accumulate=accumulate, **kw)
    n = min(max(int(lengths.max()), 1), table.shape[1] * c.page) if lengths.numel() else 1
    delta = (d + 8) * 2.0**-24 * big + (2 * big + 8) * 2.0**-23
    chain = (n / 16 + 64) * 2.0**-23
    rel = 2 * delta + 2.0**-16 + chain
    within(out, ref, half(c.dtype) * np.abs(ref) * 1.001 + size * rel[:, :, None] * 1.01 + 1e-30, what)
    within(l, lse, delta + chain + 2.0**-22 + 2.0**-22 * np.abs(np.where(np.isfinite(lse), lse, 0.0)), what + " lse")
    if c.mass is not None:
        want = pool["mass"] + (mass if accumulate else 0.0)
        got = f64(c.mass)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        tol = mass * (rel.max() if rel.size else 0.0) + 2.0**-23 * np.abs(want) if accumulate else 0.0 * want
        assert bool((np.abs(got - want)[~np.isnan(want)] <= (tol * 1.01 + 1e-37 * accumulate)[~np.isnan(want)]).all()), \
            what + " mass"
    return out, l


@DTYPES
@pytest.mark.parametrize("page", [8, 16, 32])
@pytest.mark.parametrize("d", [8, 24, 32, 40, 64, 72, 80, 96, 104, 128, 136, 160, 192, 200, 248, 256])
def test_attend_head_sizes(d, page, dtype):
    """Every size of a head in units of 32, in pages shorter and longer than a step."""
    g = gen(d)
    lengths = torch.tensor([1, 33, 0, 700], device=DEV, dtype=torch.int32)
    c, table = make_pool(g, 4, lengths.tolist(), 2, page, d, dtype)
    q = 2 * torch.randn(4, 6, d, generator=g, device=DEV).to(dtype)
    check_attend(c, table, lengths, q, accumulate=True, what=f"d={d}")


@DTYPES
@pytest.mark.parametrize("heads,group", [(1, 1), (40, 1), (3, 2), (8, 4), (5, 7), (2, 8), (1, 15), (2, 16), (1, 17),
                                         (2, 32), (1, 33), (1, 71), (1, 128), (1, 300)])
def test_attend_groups(heads, group, dtype):
    g = gen(heads * 100 + group)
    lengths = torch.tensor([77, 5, 130], device=DEV, dtype=torch.int32)
    c, table = make_pool(g, 3, lengths.tolist(), heads, 32, 64, dtype)
    q = torch.randn(3, heads * group, 64, generator=g, device=DEV).to(dtype)
    check_attend(c, table, lengths, q, accumulate=group % 2 == 1, what=f"{heads} heads of {group}")


@DTYPES
@pytest.mark.parametrize("page", [8, 16, 32, 64, 256, 4096])
@pytest.mark.parametrize("transposed", [False, True], ids=["by head", "by slot"])
def test_attend_pages(page, transposed, dtype):
    """Lengths around the ends of pages and of the kernels' tiles."""
    g = gen(page + transposed)
    lens = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300]
    lengths = torch.tensor(lens, device=DEV, dtype=torch.int32)
    c, table = make_pool(g, len(lens), lens, 2, page, 32, dtype, transposed=transposed, age=False)
    q = 3 * torch.randn(len(lens), 4, 32, generator=g, device=DEV).to(dtype)
    check_attend(c, table, lengths, q, accumulate=True, what=f"pages of {page}")


@DTYPES
@pytest.mark.parametrize("n,S,heads,group,d,page", [(5000, 1, 2, 4, 128, 16), (4097, 2, 1, 8, 64, 64), (9999, 1, 1, 1, 80, 128),
                                                    (2048, 1, 3, 3, 256, 32), (3001, 3, 4, 1, 128, 8)])
def test_attend_long(n, S, heads, group, d, page, dtype):
    """A few long sequences: split over their length and joined; a workspace of any contents."""
    g = gen(n)
    lengths = torch.tensor([n - 700 * s for s in range(S)], device=DEV, dtype=torch.int32)
    c, table = make_pool(g, S, lengths.tolist(), heads, page, d, dtype, most=-(-n // page) + 3)
    table[:, -3:] = 2**31 - 1  # behind the lengths: never read
    q = 2.5 * torch.randn(S, heads * group, d, generator=g, device=DEV).to(dtype)
    for accumulate in (False, True):
        need = gsi.gsi_cache_attend_workspace(c, table, heads * group, accumulate)
        ws = torch.full((max(need, 16) // 4,), float("nan"), device=DEV)
        out, lse = check_attend(c, table, lengths, q, accumulate=accumulate, what="long", ws=ws)
        before = c.mass.clone()
        again, lse2 = gsi.gsi_cache_attend(c, table, lengths, q, accumulate=False)
        assert torch.equal(bits(before), bits(c.mass)) and torch.equal(bits(lse), bits(lse2))
        assert torch.equal(bits(out), bits(again))


def plain_attend(c, table, lengths, q, scale, window=0):
    """The oracle's formula for many sequences at once: 64-bit products on the
    GPU.  (out, lse, weights by slot, sum of weight |v|, largest scale sum |q k|)."""
    S, H, d = q.shape
    kv = c.heads
    k, v = (t.double()[table.long()].transpose(1, 2).flatten(2, 3) for t in (c.K, c.V))  # [S][kv][slots][d]
    t = torch.arange(k.shape[2], device=DEV)
    n = lengths.long()[:, None]
    first = (n - window).clamp(min=0) if window else torch.zeros_like(n)
    inside = ((t >= first) & (t < n))[:, None, None]
    k, v = (u.masked_fill(~inside.transpose(2, 3), 0.0) for u in (k, v))
    Q = q.double().view(S, kv, H // kv, d)
    score = (scale * (Q @ k.transpose(2, 3).contiguous())).masked_fill(~inside, -float("inf"))
    big = abs(scale) * (Q.abs() @ k.abs().transpose(2, 3).contiguous()).amax(3).view(S, H)
    lse = torch.logsumexp(score, 3)
    w = torch.exp(score - lse.clamp(min=-1e300)[..., None])
    return (w @ v).view(S, H, d), lse.view(S, H), w.sum(2), (w @ v.abs()).view(S, H, d), big


@DTYPES
@pytest.mark.parametrize("page", [8, 32])
@pytest.mark.parametrize("d", [24, 64, 80, 128, 136, 192, 200, 256])
def test_attend_many_rows(d, page, dtype):
    """Many more rows than workgroups: each takes several, cut ones among them,
    and the lengths of more than 64 sequences are counted."""
    g = gen(d + page)
    S, kv, H, most = 250, 8, 24, 160
    lengths = torch.randint(0, most + 1, (S,), generator=g, device=DEV, dtype=torch.int32)
    lengths[torch.rand(S, generator=g, device=DEV) < 0.3] = 3
    lengths[:5] = torch.tensor([0, 0, most, 1, most], device=DEV)
    c, table = make_pool(g, S, lengths.tolist(), kv, page, d, dtype, most=most // page, age=False)
    q = 2 * torch.randn(S, H, d, generator=g, device=DEV).to(dtype)
    before = c.mass.clone()
    ref, lse, w, size, big = (t.cpu().numpy() for t in plain_attend(c, table, lengths, q, d**-0.5))
    out, l = gsi.gsi_cache_attend(c, table, lengths, q, accumulate=True)
    delta = (d + 8) * 2.0**-24 * big + (2 * big + 8) * 2.0**-23
    chain = (most / 16 + 64) * 2.0**-23
    rel = 2 * delta + 2.0**-16 + chain
    within(out, ref, half(dtype) * np.abs(ref) * 1.001 + size * rel[:, :, None] * 1.01 + 1e-30, "many rows")
    within(l, lse, delta + chain + 2.0**-22 + 2.0**-22 * np.abs(np.where(np.isfinite(lse), lse, 0.0)), "many rows lse")
    add = torch.zeros_like(c.mass).double()
    add[table.long()] = torch.from_numpy(w).to(DEV).view(S, kv, most // page, page).transpose(1, 2)
    want = before.double() + add
    off = (c.mass.double() - want).abs() > add * float(rel.max()) * 1.01 + want.abs() * 2.0**-23
    assert not bool((off & ~torch.isnan(before)).any()) and torch.equal(torch.isnan(before), torch.isnan(c.mass))


@pytest.mark.parametrize("window", [0, 50])
def test_attend_more_sequences_than_a_wavefront_counts(window):
    """2500 sequences, most of them short, some empty, in every place."""
    g = gen(41 + window)
    S = 2500
    lengths = torch.randint(0, 30, (S,), generator=g, device=DEV, dtype=torch.int32)
    lengths[torch.randint(0, S, (40,), generator=g, device=DEV)] = 190
    c, table = make_pool(g, S, lengths.tolist(), 1, 16, 16, BF16, most=12, age=False)
    q = 2 * torch.randn(S, 3, 16, generator=g, device=DEV).to(BF16)
    before = c.mass.clone()
    ref, lse, w, size, big = (t.cpu().numpy() for t in plain_attend(c, table, lengths, q, 0.25, window))
    out, l = gsi.gsi_cache_attend(c, table, lengths, q, window=window, accumulate=True)
    delta = 24 * 2.0**-24 * big + (2 * big + 8) * 2.0**-23
    rel = 2 * delta + 2.0**-16 + 76 * 2.0**-23
    within(out, ref, half(BF16) * np.abs(ref) * 1.001 + size * rel[:, :, None] * 1.01 + 1e-30, "sequences")
    within(l, lse, delta + 76 * 2.0**-23 + 2.0**-22 + 2.0**-22 * np.abs(np.where(np.isfinite(lse), lse, 0.0)), "lse")
    add = torch.zeros_like(c.mass).double()
    add[table.long()] = torch.from_numpy(w).to(DEV).view(S, 1, 12, 16).transpose(1, 2)
    off = (c.mass.double() - before.double() - add).abs() > add * float(rel.max()) * 1.01 + (before + add).abs() * 2.0**-23
    assert not bool((off & ~torch.isnan(before)).any()) and torch.equal(torch.isnan(before), torch.isnan(c.mass))


def check_against_plain(c, table, lengths, q, what):
    """Held to plain_attend; n / 16 + 64 additions of a chain at most, as in check_attend."""
    d = c.d
    ref, lse, _, size, big = (t.cpu().numpy() for t in plain_attend(c, table, lengths, q, d**-0.5))
    out, l = gsi.gsi_cache_attend(c, table, lengths, q)
    delta = (d + 8) * 2.0**-24 * big + (2 * big + 8) * 2.0**-23
    chain = (max(int(lengths.max()), 1) / 16 + 64) * 2.0**-23
    rel = 2 * delta + 2.0**-16 + chain
    within(out, ref, half(c.dtype) * np.abs(ref) * 1.001 + size * rel[:, :, None] * 1.01 + 1e-30, what)
    within(l, lse, delta + chain + 2.0**-22 + 2.0**-22 * np.abs(np.where(np.isfinite(lse), lse, 0.0)), what + " lse")


@DTYPES
@pytest.mark.parametrize("d", [16, 128, 256])
@pytest.mark.parametrize("heads,group", [(1, 17), (3, 33), (2, 40), (1, 300), (1, 1000)])
def test_attend_shares_of_many_query_heads(heads, group, d, dtype):
    """Ragged lengths, some empty, over more than 16 query heads of a key head: two
    to 63 workgroups of a share, eight shares of them at least."""
    g = gen(heads + group + d)
    S = 21
    lengths = torch.exp(torch.rand(S, generator=g, device=DEV) * np.log(1500)).int()
    lengths[::5] = 0
    c, table = make_pool(g, S, lengths.tolist(), heads, 16, d, dtype, most=94, age=False)
    q = 2 * torch.randn(S, heads * group, d, generator=g, device=DEV).to(dtype)
    check_against_plain(c, table, lengths, q, f"{heads} heads of {group}")


@pytest.mark.parametrize("n", [49024, 49025, 49152, 65537])
@pytest.mark.parametrize("others", [[], [0], [5, 0, 1, 700]])
def test_attend_shares_by_units_and_by_cost(n, others):
    """A long sequence around the length from which on rows cost too, before and
    behind short ones."""
    g = gen(n + len(others))
    for lens in ([n] + others, others + [n]):
        lengths = torch.tensor(lens, device=DEV, dtype=torch.int32)
        c, table = make_pool(g, len(lens), lens, 1, 64, 256, BF16, most=-(-n // 64), age=False)
        q = 2 * torch.randn(len(lens), 2, 256, generator=g, device=DEV).to(BF16)
        check_against_plain(c, table, lengths, q, f"{lens}")


def test_attend_nothing_at_all():
    """Only empty sequences; tables without a page; no sequence."""
    g = gen(42)
    c, table = make_pool(g, 3, [0, 0, 0], 2, 16, 64, BF16)
    q = torch.randn(3, 4, 64, generator=g, device=DEV).to(BF16)
    zero = torch.zeros(3, device=DEV, dtype=torch.int32)
    for tab, n in ((table, zero), (table[:, :0], zero + 9), (table, zero - 1)):
        before = c.mass.clone()
        out, lse = gsi.gsi_cache_attend(c, tab, n, q, accumulate=True)
        assert bool((out == 0).all()) and bool((lse == -float("inf")).all())
        assert torch.equal(bits(before), bits(c.mass))
    out, lse = gsi.gsi_cache_attend(c, table[:0], zero[:0], q[:0])
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    length, moved = gsi.gsi_cache_evict(c, table[:, :0], zero + 5, 4)
    assert length.tolist() == [0, 0, 0] and bool((moved == -1).all())


def test_attend_a_billion_slots():
    """2^30 slots of one sequence on pages that come again and again: as many
    products as 64-bit counts of shares need.  Equal pages give the average over
    one of them; a lane adds 2^30 / (32 * 768 * 4) = 10923 steps of 8 weights, the
    sum of which is off by 2^-24 each at most, and shares are joined: below
    (8 * 10923 + 1024) 2^-24 = 0.0053 of the sum, and of each sum of values."""
    g = gen(43)
    K, V = (torch.randn(2, 1, 4096, 8, generator=g, device=DEV).to(BF16) for _ in range(2))
    c = gsi.Cache(K, V)
    table = torch.zeros(1, 1 << 18, device=DEV, dtype=torch.int32)
    q = torch.randn(1, 2, 8, generator=g, device=DEV).to(BF16)
    one, lse1 = gsi.gsi_cache_attend(c, table[:, :1].contiguous(), torch.tensor([4096], device=DEV, dtype=torch.int32), q)
    out, lse = gsi.gsi_cache_attend(c, table, torch.tensor([1 << 30], device=DEV, dtype=torch.int32), q)
    _, _, _, size, _ = plain_attend(c, table[:, :1], torch.tensor([4096], device=DEV, dtype=torch.int32), q, 8**-0.5)
    assert bool(((out.double() - one.double()).abs() <= 2 * 0.0053 * size + 2.0**-7 * one.double().abs()).all())
    assert bool(((lse - lse1 - 18 * np.log(2.0)).abs() <= 0.0054 + 1e-5).all())


@DTYPES
@pytest.mark.parametrize("window", [1, 3, 8, 31, 32, 33, 100, 1000, 2**31 - 1])
def test_attend_window(window, dtype):
    g = gen(window % 1000)
    lens = [0, 1, 31, 32, 40, 97, 333, 1500]
    lengths = torch.tensor(lens, device=DEV, dtype=torch.int32)
    c, table = make_pool(g, len(lens), lens, 2, 16, 48, dtype)
    q = 2 * torch.randn(len(lens), 2, 48, generator=g, device=DEV).to(dtype)
    # what lies before the window is not read either
    for s, n in enumerate(lens):
        i = torch.arange(max(0, n - window), device=DEV)
        at = table[s].long()[i // 16]
        c.K[at, :, i % 16] = float("nan")
        c.V[at, :, i % 16] = float("inf")
    check_attend(c, table, lengths, q, window=window, accumulate=True, what=f"window {window}")


@DTYPES
def test_attend_lengths_outside_and_pages_that_are_none(dtype):
    """Lengths below zero and above the table; pages outside the pool hold nothing."""
    g = gen(11)
    lengths = torch.tensor([-4, 10**9, 50, 64, 30, 2], device=DEV, dtype=torch.int32)
    c, table = make_pool(g, 6, [0, 64, 50, 64, 30, 2], 2, 8, 64, dtype)
    table[2, 1], table[2, 6], table[3, :4], table[4, :], table[5, 0] = -1, c.pages, 2**31 - 1, -2**31, c.pages + 5
    q = torch.randn(6, 4, 64, generator=g, device=DEV).to(dtype)
    out, lse = check_attend(c, table, lengths, q, accumulate=True, what="no pages")
    for s in (0, 4, 5):
        assert bool((out[s] == 0).all()) and bool((lse[s] == -float("inf")).all())


@DTYPES
def test_attend_extreme_scores(dtype):
    """Scores far apart, all of one value, very negative ones, a zero scale, -inf scores."""
    g = gen(12)
    n, d = 150, 64
    lengths = torch.tensor([n, n, n, n], device=DEV, dtype=torch.int32)
    c, table = make_pool(g, 4, lengths.tolist(), 1, 16, d, dtype)
    q = torch.randn(4, 2, d, generator=g, device=DEV).to(dtype)
    q[0] = 60.0
    i = torch.arange(n, device=DEV)
    at, off = table[1].long()[i // 16], i % 16
    c.K[at, 0, off] = 1.0
    at = table[2].long()[i // 16]
    c.K[at, 0, off] = -40.0
    q[2] = q[2].abs() + 1
    check_attend(c, table, lengths, q, what="extreme")
    check_attend(c, table, lengths, q, scale=0.0, what="zero scale")
    check_attend(c, table, lengths, q, scale=-0.3, what="negative scale")
    # a slot with score -inf has no weight; a row of them is an empty one
    big = torch.finfo(dtype).max
    q[3] = 1.0
    at = table[3].long()[i // 16]
    c.K[at, 0, off] = -big
    out, lse = gsi.gsi_cache_attend(c, table, lengths, q, scale=4.0, accumulate=True)
    assert bool((out[3] == 0).all()) and bool((lse[3] == -float("inf")).all())
    c.K[table[3, 2].long(), 0, 5] = 0.25
    out, lse = gsi.gsi_cache_attend(c, table, lengths, q, scale=4.0)
    assert torch.equal(bits(out[3, 0]), bits(c.V[table[3, 2].long(), 0, 5])) and bool((lse[3] == 64.0).all())


@DTYPES
def test_attend_non_finite_rows_stay_alone(dtype):
    g = gen(13)
    lengths = torch.tensor([200, 90, 200], device=DEV, dtype=torch.int32)
    c, table = make_pool(g, 3, lengths.tolist(), 2, 32, 40, dtype)
    q = torch.randn(3, 4, 40, generator=g, device=DEV).to(dtype)
    ref, lse = gsi.gsi_cache_attend(c, table, lengths, q)
    for bad in (float("nan"), float("inf")):
        z = q.clone()
        z[1, 2, 3] = bad  # one query head: neither its neighbours of the key head nor other sequences change
        out, l = gsi.gsi_cache_attend(c, table, lengths, z)
        same = torch.ones(3, 4, dtype=torch.bool, device=DEV)
        same[1, 2] = False
        assert torch.equal(bits(out[same]), bits(ref[same])) and torch.equal(bits(l[same]), bits(lse[same]))
        assert not torch.isfinite(out[1, 2]).any()
    c.V[table[0, 1].long(), 1, 7, 11] = float("nan")  # a value of key head 1: element 11 of its heads alone
    out, l = gsi.gsi_cache_attend(c, table, lengths, q)
    assert torch.isnan(out[0, 2:, 11]).all()
    out[0, 2:, 11] = ref[0, 2:, 11]
    assert torch.equal(bits(out), bits(ref)) and torch.equal(bits(l), bits(lse))


@DTYPES
@pytest.mark.parametrize("q_size", [0.0, 0.3, 2.0], ids=["equal weights", "near weights", "weights apart"])
def test_attend_infinite_values(q_size, dtype):
    """An infinite value makes its column infinite, whatever its weight (one slot:
    exactly 1; others on either side of a number with a short significand), two of
    opposite signs make it NaN; other columns and heads do not see them."""
    g = gen(61)
    lens = [1, 2, 3, 7, 40, 700, 2500]
    lengths = torch.tensor(lens, device=DEV, dtype=torch.int32)
    c, table = make_pool(g, len(lens), lens, 2, 16, 64, dtype)
    q = q_size * torch.randn(len(lens), 4, 64, generator=g, device=DEV)
    q = q.to(dtype)
    ref, lse = gsi.gsi_cache_attend(c, table, lengths, q)
    inf = float("inf")
    want = f64(ref)
    for s, n in enumerate(lens):
        a, b = (int(t) for t in torch.randint(0, n, (2,), generator=g, device=DEV))
        at = lambda t: (int(table[s, t // 16]), 0, t % 16)  # noqa: E731
        c.V[at(a)][3], c.V[at(a)][4] = inf, -inf
        want[s, :2, 3], want[s, :2, 4] = inf, -inf
        if a != b:
            c.V[at(a)][60], c.V[at(b)][60] = inf, -inf
            c.V[at(a)][61], c.V[at(b)][61] = inf, inf
            want[s, :2, 60], want[s, :2, 61] = np.nan, inf
    out, l = gsi.gsi_cache_attend(c, table, lengths, q)
    assert np.array_equal(f64(out), want, equal_nan=True)
    assert torch.equal(bits(l), bits(lse))


@DTYPES
@pytest.mark.parametrize("d", [24, 64, 128, 256])
def test_attend_values_near_the_largest(d, dtype):
    """Values up to 2^128 times 0.97: sums of values that are not yet divided by the
    weights' sum would pass the largest number, in some wavefronts and shares and not
    in others; and values of 2^-100, results of which have no fewer digits."""
    g = gen(62 + d)
    lens = [1, 2, 3, 40, 700, 2500, 3000, 0] + torch.randint(1, 120, (100,), generator=g, device=DEV).tolist()
    lengths = torch.tensor(lens, device=DEV, dtype=torch.int32)
    c, table = make_pool(g, len(lens), lens, 4, 16, d, dtype, age=False)
    V = torch.nan_to_num(c.V).clamp(-3.875, 3.875)
    q = torch.randn(len(lens), 8, d, generator=g, device=DEV).to(dtype)
    for values in (V, V.abs()):  # signs that cancel, and sums of n values
        for k in (0, 126, 121, -100):
            c.V.copy_(values.double() * 2.0**k)
            ref, lse, _, size, big = (t.cpu().numpy() for t in plain_attend(c, table, lengths, q, d**-0.5))
            out, l = gsi.gsi_cache_attend(c, table, lengths, q)
            # as in check_attend, but for its 1e-30
            delta = (d + 8) * 2.0**-24 * big + (2 * big + 8) * 2.0**-23
            chain = (max(lens) / 16 + 64) * 2.0**-23
            rel = 2 * delta + 2.0**-16 + chain
            within(out, ref, half(dtype) * np.abs(ref) * 1.001 + size * rel[:, :, None] * 1.01, f"values of 2^{k}")
            within(l, lse, delta + chain + 2.0**-22 + 2.0**-22 * np.abs(np.where(np.isfinite(lse), lse, 0.0)), "lse")


def single_weights(g, dtype, lens, d=256):
    """A pool whose slot i has the value e_i, and queries with one element each: out
    is the weights themselves, and a score a single product.  (cache, table, lengths,
    q, weights in 64 bits)"""
    c, table = make_pool(g, len(lens), lens, 1, 32, d, dtype, most=d // 32)
    q = torch.zeros(len(lens), 3, d, device=DEV, dtype=dtype)
    q[:, :, 5] = torch.tensor([0.3, -0.7, 1.0], device=DEV, dtype=dtype)
    weights = np.zeros((len(lens), 3, d))
    for s, n in enumerate(lens):
        i = torch.arange(n, device=DEV)
        at, off = table[s].long()[i // 32], i % 32
        k = (6 * torch.rand(n, generator=g, device=DEV) - 3).to(dtype)  # scores of at most 3
        c.K[at, 0, off] = torch.randn(n, d, generator=g, device=DEV).to(dtype)
        c.K[at, 0, off, 5] = k
        c.V[at, 0, off] = torch.eye(d, device=DEV, dtype=dtype)[:n]
        e = np.exp(f64(q[s, :, 5])[:, None] * f64(k)[None])
        weights[s, :, :n] = e / e.sum(1, keepdims=True)
    c.mass.zero_()
    return c, table, torch.tensor(lens, device=DEV, dtype=torch.int32), q, weights


# A score is one product (2^-24 of it), times log2 e (rounded itself) rounded: off by 3
# x 2^-24 |s|, |s| <= 3, and by 2^-24 |s - top| <= 6 x 2^-24 where the maximum is taken
# off: 15 x 2^-24; the exponential by 2^-23 more: 17 in all, of a weight and of each in
# the weights' sum.  That sum of n <= 256 takes a term through 4 additions a step of
# one to four steps, 2 across lanes and 4 across wavefronts: 22.  Times a power of two,
# the other wavefronts' factor (2^-23 and 17 as above), the quotient (three roundings) and
# the sum with zeros: 24.  17 + 17 + 22 + 24 = 80.
WEIGHT = 80 * 2.0**-24


def test_attend_fp32_weights_have_all_their_digits():
    """Weights of which no more than a handful of roundings are lost: that they are
    not held in the 16 digits of two bf16 numbers, which the sums' bounds allow."""
    g = gen(71)
    lens = [1, 2, 3, 17, 64, 65, 200, 256]
    c, table, lengths, q, p = single_weights(g, F32, lens)
    out, _ = gsi.gsi_cache_attend(c, table, lengths, q, scale=1.0)
    within(out, p, WEIGHT * p, "weights")
    # the bound sees what it is there for: the same weights with 16 digits
    cut = (p * 2.0**16 / 2.0**np.floor(np.log2(p, where=p > 0, out=np.zeros_like(p)))).round() / 2.0**16 \
        * 2.0**np.floor(np.log2(p, where=p > 0, out=np.zeros_like(p)))
    assert (np.abs(cut - p) > WEIGHT * p).any()


@DTYPES
def test_attend_mass_has_all_its_digits(dtype):
    """What is added to the mass, in both types: three heads' weights, each from its
    score and the softmax's level (their sizes at most 3 + log 256 = 8.6, times log2 e
    13, each rounded where it is written and taken off: 40 x 2^-24 more), added up."""
    g = gen(72)
    lens = [1, 2, 3, 17, 64, 65, 200, 256]
    c, table, lengths, q, p = single_weights(g, dtype, lens)
    gsi.gsi_cache_attend(c, table, lengths, q, scale=1.0, accumulate=True)
    for s, n in enumerate(lens):
        i = torch.arange(n, device=DEV)
        got = c.mass[table[s].long()[i // 32], 0, i % 32]
        want = p[s, :, :n].sum(0)
        within(got, want, (WEIGHT + 44 * 2.0**-24) * want, f"mass of {n}")


@DTYPES
def test_attend_strides_and_what_is_left(dtype):
    g = gen(14)
    S, H, d = 5, 6, 72
    lengths = torch.tensor([40, 3, 0, 77, 12], device=DEV, dtype=torch.int32)
    wide = torch.full((S + 9, 2, 16, d + 8), float("nan"), device=DEV).to(dtype)  # pages with more in them
    K, V = wide[:, 0], torch.empty_like(wide)[:, 0]
    pool = wide.new_empty(30, 3, 16, 2, d + 8).fill_(float("nan"))
    K, V = pool[:, 0, :, :, 8:].transpose(1, 2), pool[:, 2, :, :, 8:].transpose(1, 2)
    K.copy_(torch.randn(30, 2, 16, d, generator=g, device=DEV))
    V.copy_(torch.randn(30, 2, 16, d, generator=g, device=DEV))
    c = gsi.Cache(K, V)
    wide_table = torch.full((S, 9), -3, device=DEV, dtype=torch.int32)
    table = wide_table[:, 2:7]
    table.copy_(torch.randperm(30, generator=g, device=DEV)[:25].view(S, 5))
    q = torch.full((H + 1, S, d + 24), float("nan"), device=DEV).to(dtype)[:H, :, 16:16 + d].transpose(0, 1)
    q.copy_(torch.randn(S, H, d, generator=g, device=DEV))
    out = torch.full((S, H + 2, d + 8), 5.0, device=DEV).to(dtype)
    y = out[:, 1:1 + H, 8:]
    check_attend(c, table, lengths, q, out=y, what="strided")
    y.fill_(5.0)
    assert bool((out == 5.0).all())


def test_attend_addresses_past_32_bits():
    """Pages more than 4 GiB (and 2^31 elements) apart."""
    g = gen(15)
    page, heads, d = 16, 1, 64
    far = (1 << 31) // (page * d) * 2 + 5
    K = torch.empty(far + 3, heads, page, d, device=DEV, dtype=BF16)
    V = torch.empty_like(K)
    at = torch.tensor([0, 7, far // 2 + 1, far, far + 2], device=DEV)
    K[at], V[at] = (torch.randn(5, heads, page, d, generator=g, device=DEV).to(BF16) for _ in range(2))
    small = gsi.Cache(K[at].contiguous(), V[at].contiguous())
    lengths = torch.tensor([75], device=DEV, dtype=torch.int32)
    q = torch.randn(1, 2, d, generator=g, device=DEV).to(BF16)
    order = torch.tensor([[3, 0, 4, 1, 2]], device=DEV)
    a, l = gsi.gsi_cache_attend(gsi.Cache(K, V), at[order].int(), lengths, q)
    b, m = check_attend(small, order.int(), lengths, q)
    assert torch.equal(bits(a), bits(b)) and torch.equal(bits(l), bits(m))
    # appending and evicting there
    mass, age = torch.rand(far + 3, heads, page, device=DEV), torch.zeros(far + 3, heads, page, device=DEV, dtype=torch.int32)
    big = gsi.Cache(K, V, mass, age)
    k, v = (torch.randn(1, heads, d, generator=g, device=DEV).to(BF16) for _ in range(2))
    table = at[order].int()
    gsi.gsi_cache_append(big, table, torch.tensor([76], device=DEV, dtype=torch.int32), k, v)
    assert torch.equal(bits(K[at[2], :, 12]), bits(k[0])) and torch.equal(bits(V[at[2], :, 12]), bits(v[0]))
    assert int(age[at[2], 0, 12]) == 76
    mass[at[2], 0, 12], mass[at[3], 0, 3] = 9.0, -1.0
    lengths.fill_(77)
    _, moved = gsi.gsi_cache_evict(big, table, lengths, 76)
    assert int(moved[0, 0, 3]) == 76 and torch.equal(bits(K[at[3], :, 3]), bits(k[0]))


# ---- eviction ----


def check_evict(c, table, lengths, budget, recent, to=None, what="evict"):
    pool = copy_of(c)
    tab, dest = ints(table), None if to is None else ints(to)
    want_len, want = orc.evict(pool, tab, ints(lengths), budget, recent)
    orc.move(pool, tab, want, dest)
    old = lengths.clone()
    got_len, got = gsi.gsi_cache_evict(c, table, lengths, budget, recent=recent, to=to)
    assert torch.equal(old, lengths)
    assert np.array_equal(ints(got_len), want_len), what
    bad = np.argwhere(ints(got) != want)
    assert bad.size == 0, f"{what}: {len(bad)} sources, first at {bad[0]}: {ints(got)[tuple(bad[0])]} for {want[tuple(bad[0])]}"
    same_pool(c, pool, what)
    return got_len, got


@DTYPES
@pytest.mark.parametrize("n,budget,recent,heads,page,d", [
    (17, 16, 4, 2, 8, 8), (300, 299, 50, 3, 16, 64), (300, 64, 0, 2, 32, 128), (300, 64, 64, 1, 64, 72), (300, 1, 0, 2, 8, 16),
    (300, 1, 1, 2, 8, 16), (1025, 777, 100, 2, 16, 24), (2500, 70, 30, 1, 128, 40), (64, 65, 3, 2, 16, 32), (129, 128, 127, 1, 8, 256),
])
def test_evict_in_place(n, budget, recent, heads, page, d, dtype):
    g = gen(n + budget + recent)
    lens = [n, max(0, n - 3), budget, 0, min(n, budget + 1)]
    lengths = torch.tensor(lens, device=DEV, dtype=torch.int32)
    c, table = make_pool(g, 5, lens, heads, page, d, dtype, transposed=d == 64)
    check_evict(c, table, lengths, budget, recent)


@DTYPES
@pytest.mark.parametrize("n,budget,recent", [(200, 77, 20), (50, 120, 5), (513, 512, 0)])
def test_evict_into_other_pages(n, budget, recent, dtype):
    g = gen(n)
    lens = [n, 3, 0, n // 2]
    most = max(-(-n // 16), -(-budget // 16))
    c, table = make_pool(g, 8, lens + [0] * 4, 2, 16, 48, dtype, most=most)
    lengths = torch.tensor(lens, device=DEV, dtype=torch.int32)
    check_evict(c, table[:4], lengths, budget, recent, to=table[4:].contiguous(), what="into")


def test_evict_without_ages_goes_by_slots():
    g = gen(21)
    for n, budget, recent in ((200, 100, 64), (200, 100, 1), (130, 129, 129), (65, 64, 0), (192, 70, 65)):
        lens = [n, n - 1, budget]
        c, table = make_pool(g, 3, lens, 2, 16, 16, BF16, age=False)
        check_evict(c, table, torch.tensor(lens, device=DEV, dtype=torch.int32), budget, recent, what=f"{n}->{budget}")


@pytest.mark.parametrize("kind", ["all alike", "zeros", "two values", "signs", "not finite", "tiny", "old ties"])
def test_evict_ties_and_odd_weights(kind):
    """Ties go to the lowest slot; NaN is the least; both zeros are alike."""
    g = gen(22)
    n, budget, recent = 700, 250, 37
    c, table = make_pool(g, 2, [n, n - 30], 3, 16, 8, F32)
    m, shape = c.mass, c.mass.shape
    if kind == "all alike":
        m.fill_(0.37)
        c.age.fill_(5)
    elif kind == "zeros":
        m.copy_(torch.where(torch.rand(shape, generator=g, device=DEV) < 0.5, 0.0, -0.0))
    elif kind == "two values":
        m.copy_(torch.where(torch.rand(shape, generator=g, device=DEV) < 0.3, 1.0, 1.0 + 2.0**-23))
    elif kind == "signs":
        m.copy_(torch.randn(shape, generator=g, device=DEV) * 10.0 ** torch.randint(-30, 30, shape, generator=g, device=DEV))
    elif kind == "not finite":
        pick = torch.randint(0, 5, shape, generator=g, device=DEV)
        m[pick == 0], m[pick == 1], m[pick == 2] = float("nan"), float("inf"), -float("inf")
    elif kind == "tiny":
        m.copy_(torch.rand(shape, generator=g, device=DEV) * 1e-40)
    else:
        c.age.copy_(torch.randint(-3, 3, shape, generator=g, device=DEV, dtype=torch.int32) * 700000000)
    check_evict(c, table, torch.tensor([n, n - 30], device=DEV, dtype=torch.int32), budget, recent, what=kind)


def test_evict_pages_that_are_none():
    """Entries without a page go first; where one has to stay, nothing is moved for it."""
    g = gen(23)
    c, table = make_pool(g, 3, [64, 64, 64], 2, 8, 16, BF16)
    table[0, 1], table[1, 7], table[1, 0], table[2, :] = -1, c.pages, 2**31 - 1, -5
    lengths = torch.tensor([64, 2**31 - 1, 64], device=DEV, dtype=torch.int32)
    check_evict(c, table, lengths, 20, 4)
    c, table = make_pool(g, 1, [64], 2, 8, 16, BF16)
    table[0, 2:] = c.pages
    check_evict(c, table, lengths[:1], 30, 3, what="more room than entries")


@pytest.mark.parametrize("n,budget,recent", [(70000, 4096, 500), (131072, 131071, 1000), (524288, 2000, 10)])
def test_evict_long(n, budget, recent):
    """The longest sequences: the oracle's choice by sorting."""
    g = gen(n)
    c, table = make_pool(g, 1, [n], 2, 4096, 8, BF16)
    at = table[0].long()
    mass, age = (t[at].transpose(0, 1).reshape(2, -1)[:, :n] for t in (c.mass, c.age))
    M, A = f64(mass), ints(age)
    _, got = gsi.gsi_cache_evict(c, table, torch.tensor([n], device=DEV, dtype=torch.int32), budget, recent=recent)
    got = ints(got)[0]
    slots = np.arange(n)
    for h in range(2):
        newest = np.lexsort((slots, -A[h].astype(np.int64)))
        rest = np.sort(newest[recent:])
        best = rest[np.lexsort((rest, -M[h][rest]))][:budget - recent]
        keep = np.sort(np.concatenate([newest[:recent], best]))
        want = np.full(budget, -1)
        low = keep[keep < budget]
        want[low] = low
        want[np.setdiff1d(np.arange(budget), low)] = keep[keep >= budget]
        assert np.array_equal(got[h], want)
        at_h = at.cpu().numpy()
        new = f64(c.mass[:, h])[at_h[np.arange(budget) // 4096], np.arange(budget) % 4096]
        assert np.array_equal(new, M[h][want])


@pytest.mark.parametrize("n,budget", [(32768, 16384), (60000, 30000), (8192, 4095), (4096, 2048), (4097, 4000)])
def test_evict_when_the_newest_weigh_most(n, budget):
    """All that stay lie behind the budget as far as they can: every slot below it
    that is given up takes one of them, more of them than a list in LDS holds."""
    g = gen(n)
    c, table = make_pool(g, 1, [n], 1, 256, 16, F32)
    at = table[0].long()
    slots = torch.arange(at.numel() * 256, device=DEV)
    c.mass[at, 0] = slots.float().view(-1, 256)
    K = c.K[at, 0].reshape(-1, 16)[:n].clone()
    age = c.age[at, 0].reshape(-1)[:n].clone()
    _, moved = gsi.gsi_cache_evict(c, table, torch.tensor([n], device=DEV, dtype=torch.int32), budget)
    want = slots[:budget].clone()
    stay = max(0, 2 * budget - n)  # the last slots below the budget stay where they are
    want[:budget - stay] = torch.arange(max(budget, n - budget), n, device=DEV)[:budget - stay]
    assert torch.equal(moved[0, 0].long(), want)
    assert torch.equal(c.K[at, 0].reshape(-1, 16)[:budget], K[want]) and torch.equal(c.age[at, 0].reshape(-1)[:budget], age[want])


def test_evict_of_sequences_beyond_a_wavefront():
    g = gen(52)
    lens = [(7 * i) % 61 for i in range(150)]
    c, table = make_pool(g, 150, lens, 2, 8, 8, BF16, most=8)
    check_evict(c, table, torch.tensor(lens, device=DEV, dtype=torch.int32), 33, 10, what="many sequences")


def test_a_narrower_view_of_a_wide_table():
    """The pages that the longest sequence needs, as a view: the same choice of an
    eviction, attention within its bounds, and a workspace by the view's width."""
    g = gen(81)
    lens = [300, 17, 0, 130]
    lengths = torch.tensor(lens, device=DEV, dtype=torch.int32)
    c, table = make_pool(g, 4, lens, 2, 16, 64, BF16, most=2500)
    narrow = table[:, :19]
    assert narrow.stride(0) == 2500
    wide_bytes, narrow_bytes = (gsi.gsi_cache_attend_workspace(c, t, 4, True) for t in (table, narrow))
    assert wide_bytes > 100 * 4 * 4 * 19 * 16 * 4 and narrow_bytes < wide_bytes / 10
    q = torch.randn(4, 4, 64, generator=g, device=DEV).to(BF16)
    check_attend(c, narrow, lengths, q, accumulate=True, what="narrow")
    copies = [gsi.Cache(*(t.clone() for t in (c.K, c.V, c.mass, c.age))) for _ in range(2)]
    check_evict(copies[0], narrow, lengths, 100, 20, what="narrow")
    check_evict(copies[1], table, lengths, 100, 20, what="wide")
    for name in ("K", "V", "mass"):
        assert torch.equal(bits(getattr(copies[0], name)), bits(getattr(copies[1], name))), name


# ---- the operators together ----


def decode_steps(cache, table, lengths, steps, r, budget, recent, streams=None):
    """A few tokens of a decode: append, attend with weights, cut to the budget."""
    outs = []
    for q, k, v, pos in steps:
        qt = gsi.gsi_cache_append(cache, table, lengths, k, v, rotary=r, positions=pos, q=q)
        n = lengths + 1
        out, lse = gsi.gsi_cache_attend(cache, table, n, qt, accumulate=True)
        new, moved = gsi.gsi_cache_evict(cache, table, n, budget, recent=recent)
        lengths.copy_(new)
        outs += [out, lse, moved]
    return outs


@DTYPES
def test_decode_with_a_budget(dtype):
    """Tokens one after the other through a cache that fills and then stays at its
    budget: every attention against the oracle on the cache as it is, every
    eviction against the oracle's choice."""
    g = gen(31)
    S, heads, group, d, page, budget, recent = 3, 2, 3, 64, 8, 24, 6
    c, table = make_pool(g, S, [32] * S, heads, page, d, dtype)
    freqs = gsi.rotary_freqs(32)
    r = gsi.Rotary(freqs, layout="pairs", device=DEV)
    lengths = torch.tensor([0, 20, 24], device=DEV, dtype=torch.int32)
    pos = torch.tensor([0, 20, 500000], device=DEV)
    for step in range(30):
        q = 2 * torch.randn(S, heads * group, d, generator=g, device=DEV).to(dtype)
        k, v = (torch.randn(S, heads, d, generator=g, device=DEV).to(dtype) for _ in range(2))
        pool = copy_of(c)
        qt = gsi.gsi_cache_append(c, table, lengths, k, v, rotary=r, positions=pos, q=q)
        orc.append(pool, ints(table), None, ints(lengths), f64(gsi.gsi_rotary(r, k, pos)), f64(v), ints(pos))
        same_pool(c, pool, f"step {step}")
        n = lengths + 1
        check_attend(c, table, n, qt, accumulate=True, what=f"step {step}")
        lengths, _ = check_evict(c, table, n, budget, recent, what=f"step {step}")
        pos = pos + 1
    assert lengths.tolist() == [24, 24, 24]


@DTYPES
def test_decode_replayed_from_a_graph(dtype):
    """The same steps eager and replayed, several times, with eager work in between."""
    g = gen(32)
    S, heads, group, d, page, budget, recent = 4, 2, 4, 128, 16, 40, 10
    r = gsi.Rotary(gsi.rotary_freqs(d), device=DEV)
    c, table = make_pool(g, S, [48] * S, heads, page, d, dtype)
    start = torch.tensor([3, 40, 39, 17], device=DEV, dtype=torch.int32)
    steps = []
    for t in range(3):
        steps.append([2 * torch.randn(S, heads * group, d, generator=g, device=DEV).to(dtype)]
                     + [torch.randn(S, heads, d, generator=g, device=DEV).to(dtype) for _ in range(2)]
                     + [torch.arange(S, device=DEV) * 100 + t + 50])
    first = [t.clone() for t in (c.K, c.V, c.mass, c.age)]

    def reset(lengths):
        for t, u in zip((c.K, c.V, c.mass, c.age), first):
            t.copy_(u)
        lengths.copy_(start)

    lengths = start.clone()
    reset(lengths)
    want = decode_steps(c, table, lengths, steps, r, budget, recent) + [c.K.clone(), c.V.clone(), c.mass.clone()]
    torch.cuda.synchronize()
    reset(lengths)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = decode_steps(c, table, lengths, steps, r, budget, recent)
    for k in range(4):
        reset(lengths)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got + [c.K, c.V, c.mass], want):
            assert torch.equal(bits(a), bits(b)), f"replay {k}"
        reset(lengths)
        again = decode_steps(c, table, lengths, steps, r, budget, recent)
        torch.cuda.synchronize()
        assert all(torch.equal(bits(a), bits(b)) for a, b in zip(again, want))


def test_calls_on_two_streams():
    """Calls on streams of their own, outputs and workspaces allocated there."""
    g = gen(33)
    jobs = []
    for k in range(2):
        lens = [900 - 300 * k, 70]
        c, table = make_pool(g, 2, lens, 2, 16, 64, BF16)
        q = torch.randn(2, 4, 64, generator=g, device=DEV).to(BF16)
        lengths = torch.tensor(lens, device=DEV, dtype=torch.int32)
        jobs.append((c, table, lengths, q, torch.cuda.Stream()))
    want = [gsi.gsi_cache_attend(c, t, n, q) for c, t, n, q, _ in jobs]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [gsi.gsi_cache_attend(c, t, n, q, stream=st) for c, t, n, q, st in jobs]
        torch.cuda.synchronize()
        for (a, l), (b, m) in zip(got, want):
            assert torch.equal(bits(a), bits(b)) and torch.equal(bits(l), bits(m))
    # all of a step on a stream of its own, its results read on the current one
    r = gsi.Rotary(gsi.rotary_freqs(64), device=DEV)
    k, v = (torch.randn(2, 2, 64, generator=g, device=DEV).to(BF16) for _ in range(2))
    results = []
    for st in (None, torch.cuda.Stream()):
        c, t, n, q, _ = jobs[0]
        K, V, mass, age = (x.clone() for x in (c.K, c.V, c.mass, c.age))
        c, slots, pos = gsi.Cache(K, V, mass, age), n - 1, n.long()
        torch.cuda.synchronize()  # the inputs are made on the current stream
        qt = gsi.gsi_cache_append(c, t, slots, k, v, rotary=r, positions=pos, q=q, stream=st)
        out, lse = gsi.gsi_cache_attend(c, t, n, qt, accumulate=True, stream=st)
        length, moved = gsi.gsi_cache_evict(c, t, n, 600, recent=40, stream=st)
        y = gsi.gsi_rotary(r, q, pos, stream=st)
        torch.cuda.synchronize()
        results.append([qt, out, lse, length, moved, y, K, V, mass])
    for a, b in zip(*results):
        assert torch.equal(bits(a), bits(b))


def test_between_two_maps_of_a_block():
    """A block's step as the library's user writes it: the map of q, k and v, the
    cache, the map of attention's output, against the oracle from the map's
    stored output on."""
    g = gen(34)
    S, H, d, page = 3, 4, 32, 8
    wide = H * d
    Wqkv = gsi.Q4(torch.randint(0, 256, (3 * wide, wide // 2), generator=g, device=DEV, dtype=torch.uint8),
                  (torch.rand(3 * wide, 1, generator=g, device=DEV) * 0.05).to(BF16), group=128)
    Wout = gsi.Q4(torch.randint(0, 256, (wide, wide // 2), generator=g, device=DEV, dtype=torch.uint8),
                  (torch.rand(wide, 1, generator=g, device=DEV) * 0.05).to(BF16), group=128)
    c, table = make_pool(g, S, [20, 9, 33], H, page, d, BF16)
    lengths = torch.tensor([19, 8, 32], device=DEV, dtype=torch.int32)
    x = torch.randn(S, wide, generator=g, device=DEV).to(BF16)
    freqs = gsi.rotary_freqs(16)
    r = gsi.Rotary(freqs, layout="pairs", device=DEV)
    pos = lengths.long()
    qkv = gsi.gsi_q4_linear(Wqkv, x).view(S, 3 * H, d)
    q = gsi.gsi_cache_append(c, table, lengths, qkv[:, H:2 * H], qkv[:, 2 * H:], rotary=r, positions=pos, q=qkv[:, :H])
    out, _ = check_attend(c, table, lengths + 1, q, accumulate=True, what="block")
    check_rotary(q, qkv[:, :H], pos, freqs, "pairs", 0, 1.0, BF16, "block q")
    y = gsi.gsi_q4_linear(Wout, out.view(S, wide))
    assert y.shape == (S, wide) and bool(torch.isfinite(y).all())
