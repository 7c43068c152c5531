"""Rows held in e4m3 on the GPU: made, read back and attended, against 64-bit
references."""
import math

import numpy as np
import pytest
import torch

import gather_plan_build_amd as gpb
from held_reference import LEAST, MOST, exponents, held_rows, hold, plain_rows, power
from rows_reference import attention, check, rotated, rotation_bound
from test_rows_gpu import Batch, ints, normal, split
import workloads

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def fmt(which, dtype="bf16", hkv=2, held="e4m3", **kw):
    if which == "latent":
        return gpb.RowFormat(dtype, 1, 576, 512, values_in_key=True, held=held, **kw)
    return gpb.RowFormat(dtype, hkv, int(which), int(which), held=held, **kw)


def word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append

def check_codes(got, want64, size, dtype):
    """Held heads `got` (values, scale exponents) of heads that are want64 [...,
    values] but for the rotation's fp32, at most 2^-19 size of it (rotation_bound's
    terms): the scale is that of a value within it, and a value is off by half a
    step, 2^-4 of itself or 2^-10 scales, more by what it was off before."""
    x, e = got
    off = 2.0 ** -19 * size
    low = exponents((want64.abs() - off).clamp(min=0), dtype)
    high = exponents(want64.abs() + off, dtype)
    assert ((e >= low) & (e <= high)).all()
    step = torch.maximum(2.0 ** -4 * want64.abs(), power(e - 10)[..., None])
    assert ((x - want64).abs() <= step + 2 * off).all()


def heads_of(f, rows):
    """Held rows as (values, exponents) of key heads, and of value heads."""
    x = plain_rows(f, rows).double()
    h, kd, vd = f.n_kv_heads, f.k_dim, f.v_dim
    if f.values_in_key:
        at = vd + 2 * (kd - vd)
        return ((x[:, None, :vd], rows[:, at:at + 1].long() - 127), None)
    at = h * (kd + vd)
    return ((x[:, :h * kd].unflatten(1, (h, kd)), rows[:, at:at + h].long() - 127),
            (x[:, h * kd:].unflatten(1, (h, vd)), rows[:, at + h:at + 2 * h].long() - 127))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("h,kd,vd,latent,hq,start,pairs,interleaved,sections", [
    (2, 128, 128, False, 6, 0, 64, False, None),
    (3, 128, 128, False, 3, 0, 64, False, [16, 24, 24]),
    (1, 128, 128, False, 5, 32, 16, True, [1, 15]),
    (4, 64, 64, False, 8, 0, 32, True, None),
    (1, 64, 64, False, 2, 8, 8, False, [0, 3, 5, 0]),
    (1, 576, 512, True, 16, 512, 32, True, None),
    (1, 576, 512, True, 1, 0, 256, False, [100, 156]),
    (2, 128, 128, False, 4, 0, 0, False, None),
    (1, 128, 128, True, 1, 0, 64, False, None),      # an index key: all of it in codes
    (1, 200, 136, True, 3, 72, 64, False, None),     # pairs half in codes, half in 16 bits
    (5, 8, 24, False, 2, 0, 0, False, None),
    (7, 24, 8, False, 1, 8, 8, True, None),
    (2, 1024, 1000, False, 1, 512, 256, False, None),
])
@pytest.mark.parametrize("tokens", [1, 67])
def test_append(dtype, h, kd, vd, latent, hq, start, pairs, interleaved, sections, tokens):
    f = gpb.RowFormat(dtype, h, kd, vd, values_in_key=latent, held="e4m3")
    plain = gpb.RowFormat(dtype, h, kd, vd, values_in_key=latent)
    f = gpb.RowFormat(dtype, h, kd, vd, values_in_key=latent, held="e4m3",
                      row_bytes=f.row_bytes + 16)
    dt = f.dtype
    packed = normal(1, tokens, (hq + h) * kd + (0 if latent else h * vd), dtype=dt)
    q = packed[:, :hq * kd].unflatten(1, (hq, kd))
    k = packed[:, hq * kd:(hq + h) * kd].unflatten(1, (h, kd))
    v = None if latent else packed[:, (hq + h) * kd:].unflatten(1, (h, vd))
    sec = sections or [pairs]
    rng = np.random.default_rng(tokens)
    pos = ints(rng.integers(-5, 2 ** 31 - 1, (len(sec), tokens)) // rng.integers(
        1, 2 ** 20, (len(sec), tokens)))
    freq = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))).float().cuda()
    rot = gpb.Rotation(freq, start, interleaved, sec) if pairs else None
    pool = torch.randint(0, 256, (200, f.row_bytes), dtype=torch.uint8, device="cuda")
    before = pool.clone()
    locs = rng.permutation(200)[:tokens]
    locs[tokens // 2] = -1                       # a padded entry
    rows = torch.full((tokens, f.row_bytes), 0xa5, dtype=torch.uint8, device="cuda")
    q_out = torch.empty(tokens, hq, kd, dtype=dt, device="cuda")
    status = word()
    gpb.row_append(f, k, v, pool, ints(locs), rot, pos, rows=rows, q=q, q_out=q_out,
                   status=status)
    assert int(status) == 0
    k64 = rotated(k, pos, freq, start, interleaved, sec) if pairs else k.double()
    size = k.double().abs().amax(-1, keepdim=True) if pairs else 0.0
    codes = vd if latent else kd
    keys, values = heads_of(f, rows)
    check_codes(keys, k64[..., :codes], size, dt)
    if not pairs:
        want, s = hold(k[..., :codes], dt)
        assert torch.equal(rows[:, :h * codes], want.flatten(1))
    if v is not None:                            # not turned: the very bytes
        c, s = hold(v, dt)
        assert torch.equal(rows[:, h * kd:h * (kd + vd)], c.flatten(1))
        assert torch.equal(rows[:, h * (kd + vd) + h:h * (kd + vd) + 2 * h], s)
    # queries, and what a latent keeps in 16 bits, as the plain append has them
    rows16 = torch.empty(tokens, plain.values, dtype=dt, device="cuda")
    q16 = torch.empty_like(q_out)
    gpb.row_append(plain, k, v, None, None, rot, pos, rows=rows16, q=q, q_out=q16)
    assert torch.equal(q_out, q16)
    if latent and kd > vd:
        assert torch.equal(rows[:, vd:vd + 2 * (kd - vd)],
                           rows16[:, vd:].contiguous().view(torch.uint8))
    # the pool's rows are the packed ones; padding and other rows stay
    payload = f.row_bytes - 16 - (-(codes * h + (0 if latent else h * vd) +
                                    (2 * (kd - vd) + 1 if latent else 2 * h))) % 16
    assert (rows[:, payload:] == 0xa5).all()
    want = before.clone()
    for t, at in enumerate(locs):
        if at >= 0:
            want[at, :payload] = rows[t, :payload]
    assert torch.equal(pool, want)
    # queries in place, and without a pool
    q2, rows2 = q.clone(), torch.full_like(rows, 0xa5)
    gpb.row_append(f, k, v, None, None, rot, pos, rows=rows2, q=q2)
    assert torch.equal(q2, q_out) and torch.equal(rows2, rows)


def one_nan(rows, codes):
    """Rows of `codes` codes with 0x7f for both codes that are NaN."""
    out = rows.clone()
    out[:, :codes][(rows[:, :codes] & 127) == 127] = 127
    return out


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_codes_of_turned_keys_are_the_nearest(dtype, interleaved):
    """The turn is taken in 64 bits, there as here: sines, products and sum are off by
    less than 2^-48 (|x| + |y|) in all (angles to 10^6 rounded to 2^-34 apart: their
    product with 1 / 2 pi is off by 2^-36).  A code other than the nearest then lies
    no further away than the nearest and twice 2^-33 (|x| + |y|)."""
    f = fmt("128", dtype, 8)
    n = 3000
    k, v = normal(91, n, 8, 128, dtype=f.dtype), normal(92, n, 8, 128, dtype=f.dtype)
    freq = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float().cuda()
    pos = ints(np.random.default_rng(5).integers(0, 1000000, n))
    rows = torch.zeros(n, f.row_bytes, dtype=torch.uint8, device="cuda")
    gpb.row_append(f, k, v, None, None, gpb.Rotation(freq, interleaved=interleaved), pos, rows=rows)
    x, a = k.cpu().double(), pos.cpu().double()[:, None] * freq.cpu().double()
    c, s = a.cos()[:, None], a.sin()[:, None]
    p, q = (x[..., 0::2], x[..., 1::2]) if interleaved else x.chunk(2, -1)
    turned, size = [p * c - q * s, q * c + p * s], [p.abs() + q.abs()] * 2
    if interleaved:
        turned, size = (torch.stack(t, -1).flatten(-2) for t in (turned, size))
    else:
        turned, size = (torch.cat(t, -1) for t in (turned, size))
    scale = rows[:, 2048:2056].cpu().int()[..., None] - 127
    got = plain_rows(f, rows)[:, :1024].cpu().double().unflatten(1, (8, 128))
    y, g = torch.ldexp(turned, -scale), torch.ldexp(got, -scale)
    step = torch.ldexp(torch.ones_like(y), torch.frexp(y)[1].clamp(min=-5) - 4)
    off = (torch.round(y / step) * step - y).abs()
    bound = torch.ldexp(2.0 ** -33 * size, -scale)
    assert ((g - y).abs() <= off + 2 * bound).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_of_every_16_bit_pattern(dtype):
    """Every value of the type, infinities, NaN and subnormals among them, beside
    others that set the scale."""
    dt = DT[dtype]
    f = gpb.RowFormat(dtype, 1, 8, 16, held="e4m3")
    bits = torch.arange(65536, dtype=torch.int32, device="cuda")
    x = bits.to(torch.int16).view(dt)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    mixed = x[torch.randperm(65536, generator=g, device="cuda")]
    # one value over another that is up to 2^12 larger, or up to 2^20 smaller
    near = (x.double() * power(torch.randint(-20, 13, (65536,), generator=g,
                                             device="cuda"))).to(dt)
    v = torch.zeros(65536, 1, 16, dtype=dt, device="cuda")
    v[:, 0, 0], v[:, 0, 9] = x, near
    v[1::2, 0, 3] = torch.nan                   # does not count
    k = mixed.view(8192, 1, 8).repeat(8, 1, 1)
    rows = torch.zeros(65536, f.row_bytes, dtype=torch.uint8, device="cuda")
    gpb.row_append(f, k, v, None, None, rows=rows)
    assert torch.equal(one_nan(rows, 24), one_nan(held_rows(f, k, v), 24))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scales_at_their_borders(dtype):
    """448 scales is held by that scale, the next value by the next."""
    dt = DT[dtype]
    f = gpb.RowFormat(dtype, 1, 8, 8, held="e4m3")
    es = torch.arange(max(LEAST[dt], -14) - 3, min(MOST[dt], 100) + 1, device="cuda")
    edge = (448 * power(es)).to(dt)
    edge = edge[torch.isfinite(edge)]
    up = (edge.view(torch.int16) + 1).view(dt)
    x = torch.cat([edge, -edge, up, (edge.view(torch.int16) - 1).view(dt)])
    x = x[torch.isfinite(x)]
    k = torch.zeros(len(x), 1, 8, dtype=dt, device="cuda")
    k[:, 0, 5], k[:, 0, 1] = x, (x.double() / 37).to(dt)
    rows = torch.zeros(len(x), f.row_bytes, dtype=torch.uint8, device="cuda")
    gpb.row_append(f, k, k, None, None, rows=rows)
    assert torch.equal(rows, held_rows(f, k, k))


def test_append_flags_rows_outside_the_pool():
    f = fmt("64", hkv=1)
    k, v = normal(1, 4, 1, 64), normal(2, 4, 1, 64)
    pool = torch.full((8, f.row_bytes), 7, dtype=torch.uint8, device="cuda")
    want = pool.clone()
    status = word()
    gpb.row_append(f, k, v, pool, ints([7, 8, -1, 2]), status=status)
    assert int(status) == gpb.STATUS_BAD_STAGING_ROW
    rows = held_rows(f, k, v)
    for t, at in ((0, 7), (3, 2)):
        want[at, :130] = rows[t, :130]
    assert torch.equal(pool, want)


def test_append_and_read_past_4_gib_of_pool():
    f = fmt("128", hkv=8)
    n = (5 << 30) // f.row_bytes
    pool = torch.zeros(n, f.row_bytes, dtype=torch.uint8, device="cuda")
    k, v = normal(1, 2, 8, 128), normal(2, 2, 8, 128)
    gpb.row_append(f, k, v, pool, ints([n - 1, 0]))
    want = held_rows(f, k, v)
    assert torch.equal(pool[n - 1], want[0]) and torch.equal(pool[0], want[1])
    assert not pool[n - 2].any()
    got = gpb.rows_read(f, pool, ints([n - 1, -1, 0]))
    assert torch.equal(got[[0, 2]], plain_rows(f, want)) and not got[1].any()


# ------------------------------------------------------------------ reading back

@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_read_of_every_code_at_every_scale(dtype):
    dt = DT[dtype]
    f = gpb.RowFormat(dtype, 1, 128, 128, held="e4m3")
    n = MOST[dt] - LEAST[dt] + 1
    rows = torch.zeros(n, f.row_bytes, dtype=torch.uint8, device="cuda")
    rows[:, :256] = torch.arange(256, device="cuda").to(torch.uint8)
    s = torch.arange(LEAST[dt], MOST[dt] + 1, device="cuda") + 127
    rows[:, 256], rows[:, 257] = s.to(torch.uint8), s.flip(0).to(torch.uint8)
    # at the largest scale an append makes no code beyond 240
    for r, part in ((n - 1, slice(0, 128)), (0, slice(128, 256))):
        c = rows[r, part] & 127
        rows[r, part] = torch.where((c > 0x77) & (c < 0x7f), 0, rows[r, part])
    got = gpb.rows_read(f, rows)
    want = plain_rows(f, rows)
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    assert torch.equal(got.nan_to_num(0.0).view(torch.int16), want.nan_to_num(0.0).view(torch.int16))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("h,kd,vd,latent", [
    (2, 128, 128, False), (8, 64, 64, False), (1, 576, 512, True), (1, 128, 128, True),
    (1, 200, 136, True), (5, 8, 24, False), (7, 24, 8, False), (1024, 16, 8, False),
    (1, 1024, 8, True), (3, 1024, 1000, False)])
@pytest.mark.parametrize("n", [1, 3, 130])
def test_read(dtype, h, kd, vd, latent, n):
    f = gpb.RowFormat(dtype, h, kd, vd, values_in_key=latent, held="e4m3")
    k = normal(1, 50, h, kd, dtype=f.dtype)
    v = None if latent else normal(2, 50, h, vd, dtype=f.dtype)
    src = held_rows(f, k, v)
    want = plain_rows(f, src)
    rng = np.random.default_rng(n)
    locs = rng.integers(-1, 50, n)               # some twice, some padded
    out = torch.full((n + 2, f.values + 8), 3.0, dtype=f.dtype, device="cuda")
    status = word()
    got = gpb.rows_read(f, src, ints(locs), out=out[:, :f.values], status=status)
    assert int(status) == 0 and got.data_ptr() == out.data_ptr()
    padded = torch.cat([want, torch.zeros_like(want[:1])])
    assert torch.equal(out[:n, :f.values], padded[torch.from_numpy(locs).cuda()])
    assert (out[:, f.values:] == 3).all() and (out[n:] == 3).all()
    assert torch.equal(gpb.rows_read(f, src), want)
    assert torch.equal(gpb.rows_read(f, src, n_rows=min(n, 50)), want[:min(n, 50)])


def test_read_of_rows_that_are_not_there():
    f = fmt("64", hkv=1)
    src = held_rows(f, normal(1, 9, 1, 64), normal(2, 9, 1, 64))
    want = plain_rows(f, src)
    for wrong in (9, -2, 2 ** 31 - 1, -2 ** 31):
        status = word()
        got = gpb.rows_read(f, src, ints([4, wrong, 8]), status=status)
        assert int(status) == gpb.STATUS_BAD_DESCRIPTOR
        assert torch.equal(got[[0, 2]], want[[4, 8]]) and not got[1].any()
    assert gpb.rows_read(f, src, ints([])).shape == (0, 128)
    assert gpb.rows_read(f, src[:0]).shape == (0, 128)
    status = word()
    assert not gpb.rows_read(f, src[:0], ints([-1, -1]), status=status).any()
    assert int(status) == 0


def test_read_refuses():
    f = fmt("64", hkv=1)
    src = held_rows(f, normal(1, 9, 1, 64), normal(2, 9, 1, 64))
    with pytest.raises(ValueError):
        gpb.rows_read(fmt("64", hkv=1, held=None), src)
    with pytest.raises(ValueError):
        gpb.rows_read(f, src, n_rows=10)
    with pytest.raises(ValueError):
        gpb.rows_read(f, src, ints([1, 2]), n_rows=3)
    with pytest.raises(ValueError):
        gpb.rows_read(f, src, torch.tensor([1, 2], device="cuda"))
    with pytest.raises(ValueError):
        gpb.rows_read(f, src, out=torch.empty(9, 128, device="cuda"))
    with pytest.raises(ValueError):
        gpb.rows_read(f, src, out=torch.empty(8, 128, dtype=f.dtype, device="cuda"))
    with pytest.raises(gpb.GpbError):
        gpb.rows_read(f, src, out=torch.empty(1, 128, dtype=f.dtype, device="cuda").expand(9, 128))
    with pytest.raises(gpb.GpbError):
        gpb.rows_read(f, src, out=torch.empty(9, 132, dtype=f.dtype, device="cuda")[:, :128])


# ------------------------------------------------------------------ attention

class HeldBatch(Batch):
    """A batch whose rows, the stale ones among them, are held."""

    def __init__(self, f, *a, **kw):
        plain = gpb.RowFormat(f.dtype, f.n_kv_heads, f.k_dim, f.v_dim,
                              values_in_key=f.values_in_key)
        super().__init__(plain, *a, **kw)
        self.f = f
        self.hold()

    def hold(self):
        """Rows, dense buffer and pool as they are, held."""
        def held(x):
            f, at = self.f, self.f.n_kv_heads * self.f.k_dim
            k = x[:, :at].unflatten(1, (f.n_kv_heads, f.k_dim))
            v = None if f.values_in_key else x[:, at:].unflatten(1, (f.n_kv_heads, f.v_dim))
            return held_rows(f, k, v)
        self.rows = [plain_rows(self.f, held(x)) for x in self.rows]
        self.dense, self.pool = held(self.dense), held(self.pool)


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 14), ("64", 1, 1), ("128", 2, 8),
                                          ("128", 1, 7), ("latent", 1, 16), ("latent", 1, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q,kv", [
    ([1], [1]),
    ([1, 1, 1], [31, 32, 33]),
    ([1, 1], [63, 65]),
    ([3, 0, 5], [3, 17, 2]),                 # the last: three queries before any key
    ([2, 1], [0, 5]),
    ([129, 40], [129, 300]),
    ([1, 2, 1], [777, 1300, 4]),
])
def test_lengths(which, hkv, hq, dtype, q, kv):
    HeldBatch(fmt(which, dtype, hkv), hq, q, kv).check()


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 14), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 3), (64, 64), (100, 0),
                                          (300, 70), (5000, 4), (2, 5000)])
def test_windows_and_first_tokens(which, hkv, hq, window, sinks):
    HeldBatch(fmt(which, "bf16", hkv), hq, [1, 90, 2, 200], [640, 500, 1000, 200]).check(
        window, sinks)


@pytest.mark.parametrize("hq,hkv,which", [(128, 1, "latent"), (130, 1, "128"), (48, 1, "64"),
                                          (200, 1, "latent"), (33, 3, "128"), (1, 1, "latent")])
def test_heads(hq, hkv, which):
    HeldBatch(fmt(which, "bf16", hkv), hq, [2, 5, 1], [700, 5, 90]).check()


@pytest.mark.parametrize("page", [1, 3, 16, 48, 100, 256])
@pytest.mark.parametrize("which", ["64", "128", "latent"])
def test_page_sizes(page, which):
    HeldBatch(fmt(which, "fp16", 1), 4, [1, 4, 70], [333, 65, 70], page=page).check(window=0)


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 16), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("q,kv,page,groups,window,sinks", [
    ([1, 1, 1], [700, 650, 641], 64, [(0, 3, 640)], 0, 0),
    ([2, 1, 3, 1], [330, 301, 420, 55], 10, [(0, 3, 300)], 0, 0),     # ends inside a tile
    ([1] * 20, [1030 + 3 * r for r in range(20)], 64, [(0, 9, 1024), (9, 11, 512)], 0, 0),
    ([1, 2, 1, 1], [1100, 1200, 1300, 2000], 50, [(0, 3, 1000)], 150, 5),
    ([40, 30, 20], [168, 158, 148], 64, [(0, 3, 128)], 0, 0),
])
def test_shared_prefixes(which, hkv, hq, q, kv, page, groups, window, sinks):
    HeldBatch(fmt(which, "bf16", hkv), hq, q, kv, page=page, groups=groups).check(window, sinks)


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 8), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q,kv", [([1], [1]), ([1, 1], [70, 300]), ([200, 40], [200, 1000])])
def test_a_row_that_sees_one_key_has_its_value(which, hkv, hq, dtype, q, kv):
    f = fmt(which, dtype, hkv)
    b = HeldBatch(f, hq, q, kv)
    out, _ = gpb.attend_paged(b.plan(window=1), b.q, b.pool, b.table, 0.1)
    at = 0
    for r, (n, m) in enumerate(zip(q, kv)):
        _, v = split(f, b.rows[r][m - n:])
        assert torch.equal(out[at:at + n], v.repeat_interleave(hq // v.shape[1], 1))
        at += n


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 14), ("128", 2, 8), ("latent", 1, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scales_far_apart(which, hkv, hq, dtype):
    """Neighbouring rows whose scales differ by up to 2^20 (bf16) or 2^8."""
    f = fmt(which, dtype, hkv)
    b = HeldBatch(f, hq, [1, 90], [700, 300])
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    span = 20 if dtype == "bf16" else 8
    for r in range(2):
        x = normal(60 + r, *b.rows[r].shape, dtype=f.dtype).double()
        x *= power(torch.randint(-span, 3, (len(x), 1), generator=g, device="cuda"))
        at = f.n_kv_heads * f.k_dim
        k = x[:, :at].unflatten(1, (f.n_kv_heads, f.k_dim))
        v = None if f.values_in_key else x[:, at:].unflatten(1, (f.n_kv_heads, f.v_dim))
        rows = held_rows(f, k, v)
        b.rows[r] = plain_rows(f, rows)
        base = int(b.k_bases[r])
        b.dense[base:base + len(rows)] = rows
        for i, p in enumerate(b.lists[r]):
            part = rows[i * 64:(i + 1) * 64]
            b.pool[p * 64:p * 64 + len(part)] = part
    b.check()


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 14), ("128", 2, 8), ("latent", 1, 16)])
@pytest.mark.parametrize("dtype,size", [("bf16", 2.0 ** -97), ("bf16", 2.0 ** 110),
                                        ("fp16", 2.0 ** -12), ("fp16", 2.0 ** 11)])
@pytest.mark.parametrize("q,kv", [([1, 2], [700, 300]), ([90], [500])])
def test_scales_at_both_ends(which, hkv, hq, dtype, size, q, kv):
    """Values near the least and the largest scale; queries so small or large that the
    scores stay ordinary (of latent rows, whose values are keys too)."""
    f = fmt(which, dtype, hkv)
    b = HeldBatch(f, hq, q, kv)
    key = 0.25 / size if f.values_in_key and dtype == "fp16" else 1.0 / size
    if f.values_in_key:
        b.q[..., :512] = (b.q[..., :512].double() * key).to(f.dtype)
    for r in range(len(kv)):
        x = normal(70 + r, *b.rows[r].shape, dtype=f.dtype).double()
        at = f.n_kv_heads * f.k_dim
        if f.values_in_key:
            x[:, :512] *= size
        else:
            x[:, at:] *= size
        k = x[:, :at].unflatten(1, (f.n_kv_heads, f.k_dim)).to(f.dtype)
        v = None if f.values_in_key else x[:, at:].unflatten(1, (f.n_kv_heads, f.v_dim)).to(f.dtype)
        rows = held_rows(f, k, v)
        b.rows[r] = plain_rows(f, rows)
        base = int(b.k_bases[r])
        b.dense[base:base + len(rows)] = rows
        for i, p in enumerate(b.lists[r]):
            part = rows[i * 64:(i + 1) * 64]
            b.pool[p * 64:p * 64 + len(part)] = part
    b.check()


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 14), ("128", 2, 8), ("latent", 1, 16)])
@pytest.mark.parametrize("dtype,small,large", [("bf16", 2.0 ** -95, 2.0 ** 100),
                                               ("fp16", 2.0 ** -10, 240.0 * 2.0 ** 8)])
@pytest.mark.parametrize("q,kv", [([1, 2], [9, 40]), ([1, 2], [700, 300]), ([1], [3001]),
                                  ([90], [500])])
def test_least_scales_beside_the_largest(which, hkv, hq, dtype, small, large, q, kv):
    """Rows of the least scale between rows of the largest, which hold zeros but for
    one value: all other results are of the small rows alone, and as near as without
    the large ones.  (Scores are spread over 2^-19 at most, so that no weight ends
    where its type does.)"""
    f = fmt(which, dtype, hkv)
    b = HeldBatch(f, hq, q, kv)
    b.q *= 1.5
    if f.values_in_key:
        b.q[..., :512] = (b.q[..., :512].double() / small).to(f.dtype)
        b.q[..., 3] = 0
    for r in range(len(kv)):
        x = normal(80 + r, *b.rows[r].shape, dtype=f.dtype).double()
        at = f.n_kv_heads * f.k_dim
        k = x[:, :at].unflatten(1, (f.n_kv_heads, f.k_dim))
        v = k[..., :512] if f.values_in_key else x[:, at:].unflatten(1, (f.n_kv_heads, f.v_dim))
        v *= small
        v[1::2] = 0
        v[1::2, :, 3] = large
        rows = held_rows(f, k, None if f.values_in_key else v)
        scales = rows[:, -16] if f.values_in_key else \
            rows[:, 2 * at + f.n_kv_heads:2 * at + 2 * f.n_kv_heads]
        assert (scales[::2].long() == LEAST[f.dtype] + 127).all()
        b.rows[r] = plain_rows(f, rows)
        base = int(b.k_bases[r])
        b.dense[base:base + len(rows)] = rows
        for i, p in enumerate(b.lists[r]):
            part = rows[i * 64:(i + 1) * 64]
            b.pool[p * 64:p * 64 + len(part)] = part
    b.check()


@pytest.mark.parametrize("which", ["64", "128", "latent"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("narrow", [True, False])
def test_every_code_at_every_scale_has_its_value(which, dtype, narrow):
    """Queries that see one key, over every code that an append makes at every scale
    (of fp16, down to the least subnormal number).  The weight of an only key is a
    power of two, so the result is its value.  One request a row: narrow items; one
    request of all rows: wide ones.  (Of latent rows they are one kernel.)"""
    dt = DT[dtype]
    f = fmt(which, dtype, 1)
    dim = f.v_dim
    codes = torch.arange(256, device="cuda")
    codes = codes[(codes & 127) != 127]
    at = 0 if f.values_in_key else f.k_dim
    parts = []
    for e in range(LEAST[dt], MOST[dt] + 1):
        some = codes if e < MOST[dt] else codes[(codes & 127) <= 0x77]
        row = some.repeat(-(-dim // len(some)) + 1)
        for first in range(0, len(some) if dim < len(some) else 1, dim):
            r = torch.zeros(f.row_bytes, dtype=torch.uint8, device="cuda")
            if not f.values_in_key:
                r[2 * dim] = 127                    # the key's scale: its values are zeros
            r[at:at + dim] = row[first:first + dim].to(torch.uint8)
            r[640 if f.values_in_key else 2 * dim + 1] = e + 127
            parts.append(r)
    rows = torch.stack(parts)
    n = len(rows)
    want = split(f, plain_rows(f, rows))[1].expand(-1, 4, -1)
    q = torch.zeros(n, 4, f.k_dim, dtype=dt, device="cuda")
    if narrow:
        plan = gpb.AttendPlan(f, 4, [1] * n, [1] * n)
        out, _ = gpb.attend_dense(plan, q, rows, ints(range(n)), 1.0)
    else:
        plan = gpb.AttendPlan(f, 4, [n], [n], window=1)
        out, _ = gpb.attend_dense(plan, q, rows, ints([0]), 1.0)
    assert torch.equal(out, want)


@pytest.mark.parametrize("which", ["64", "128", "latent"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("above", [0, 2, 4, 6])
@pytest.mark.parametrize("q,kv", [(1, 2), (1, 130), (1, 1500), (70, 130)])
def test_a_weight_beside_that_of_a_larger_scale(which, dtype, above, q, kv):
    """The last key but q has the largest scale, a score `above` those of the others,
    and one value that is not zero; the others have the least scale."""
    f = fmt(which, dtype, 1)
    g = torch.Generator(device="cuda")
    g.manual_seed(above)
    at, d = kv - q, 512 if f.values_in_key else 0
    k = torch.zeros(kv, 1, f.k_dim, dtype=torch.float64, device="cuda")
    v = torch.randn(kv, 1, f.v_dim, generator=g, dtype=torch.float64, device="cuda")
    v *= power(torch.tensor([LEAST[f.dtype] + 5], device="cuda"))
    v[at] = 0
    v[at, 0, 3] = 240.0 * 2.0 ** (8 if dtype == "fp16" else 100)
    if f.values_in_key:
        k[..., :512] = v
    k[at, 0, d] = above
    rows = held_rows(f, k, None if f.values_in_key else v)
    query = torch.zeros(q, 4, f.k_dim, dtype=f.dtype, device="cuda")
    query[..., d] = 1
    x, y = split(f, plain_rows(f, rows))
    want = attention(query, x, y, torch.arange(kv - q, kv, device="cuda"), 0, 0, 1.0)
    plan = gpb.AttendPlan(f, 4, [q], [kv])
    check(*gpb.attend_dense(plan, query, rows, ints([0]), 1.0), want)


@pytest.mark.parametrize("which", ["64", "128", "latent"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q,kv", [(3, 20), (3, 2000), (60, 200)])
def test_bytes_that_no_append_makes_reach_those_that_see_them_only(which, dtype, q, kv):
    """Codes past the largest value at the largest scale, and scales past that (of
    fp16 both may come out infinite): queries before that row keep their values."""
    f = fmt(which, dtype, 1)
    b = HeldBatch(f, 4, [q], [kv])
    at, n = kv - q // 2, q - q // 2
    values = slice(0, 512) if f.values_in_key else slice(f.k_dim, 2 * f.k_dim)
    scale = 640 if f.values_in_key else 2 * f.k_dim + 1
    clean = b.rows[0].clone()
    clean[at] = 0
    k, v = split(f, clean)
    want = attention(b.q[:q], k, v, torch.arange(kv - q, kv, device="cuda"), 0, 0, 0.05)
    plan = b.plan()
    for byte in (MOST[f.dtype] + 127, MOST[f.dtype] + 128, 144, 200, 254, 255):
        for code in (0, 0x08, 0x7e, 0xfe):
            b.dense[at, values] = code
            b.dense[at, scale] = byte
            out, lse = gpb.attend_dense(plan, b.q, b.dense, b.k_bases, 0.05)
            check(out[:n], lse[:n], [w[:n] for w in want])


@pytest.mark.parametrize("which", ["64", "128"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q,kv,window,sinks,at", [
    ([100], [230], 0, 0, [140, 229, 180]),       # wide items, results at once
    ([20], [500], 40, 2, [1, 445, 470, 499]),    # values that left some windows
    ([1, 3], [70, 40], 0, 0, [39, 38]),          # narrow items
    ([2, 1], [2500, 3000], 0, 0, [7, 2499]),     # narrow items in parts
    ([150, 2], [3000, 700], 0, 0, [9, 2900, 2999]),   # wide items in parts
])
def test_values_that_are_not_numbers_reach_those_that_see_them_only(which, dtype, q, kv, window,
                                                                    sinks, at):
    f = fmt(which, dtype, 1)
    b = HeldBatch(f, 4, q, kv)
    base = b.k_bases.tolist()
    for r, x in enumerate(b.rows):
        for n, i in enumerate(i for i in at if i < len(x)):
            d = 5 + 9 * n
            x[i, f.k_dim + d] = float("nan")
            b.dense[base[r] + i, f.k_dim + d] = 0x7f if n % 2 else 0xff
            b.pool[b.lists[r][i // 64] * 64 + i % 64, f.k_dim + d] = 0x7f
    out, _ = b.check(window, sinks)
    want = b.want(window, sinks, 1.0 / math.sqrt(f.k_dim))[0]
    assert torch.equal(torch.isnan(out), torch.isnan(want)) and torch.isnan(want).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q,kv", [(60, 200), (60, 3000), (3, 2000)])
def test_latent_rows_that_are_not_numbers(dtype, q, kv):
    """Queries before the odd row keep their values, those that see it have none."""
    f = fmt("latent", dtype)
    b = HeldBatch(f, 4, [q], [kv])
    at = kv - q // 2
    b.dense[at, 7] = 0x7f
    out, lse = gpb.attend_dense(b.plan(), b.q, b.dense, b.k_bases, 0.05)
    clean = b.rows[0].clone()
    clean[at] = 0
    k, v = split(f, clean)
    want = attention(b.q[:q], k, v, torch.arange(kv - q, kv, device="cuda"), 0, 0, 0.05)
    n = at - (kv - q)
    check(out[:n], lse[:n], [w[:n] for w in want])
    assert not torch.isfinite(out[n:, :, 7]).any()


@pytest.mark.parametrize("which", ["64", "128", "latent"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_scale_bytes_that_no_append_writes_touch_those_that_see_them_only(which, dtype):
    """Rows of another kind behind the last key, and before a window: every scale
    byte, every code."""
    f = fmt(which, dtype, 1)
    b = HeldBatch(f, 4, [70, 1], [300, 200])
    for r in range(2):
        n, base = b.kv_lens[r], int(b.k_bases[r])
        end = base + -(-n // 64) * 64
        b.dense[base + n:end] = torch.arange((end - base - n) * f.row_bytes, device="cuda").view(
            -1, f.row_bytes).mul(37).to(torch.uint8)
        at = b.lists[r][-1] * 64
        b.pool[at + n % 64:at + 64] = b.dense[base + n:end]
    b.check(window=0)
    for r in range(2):
        b.dense[int(b.k_bases[r]):int(b.k_bases[r]) + 64] = 255
        b.pool[b.lists[r][0] * 64:b.lists[r][0] * 64 + 64] = 255
    b.check(window=50)


@pytest.mark.parametrize("seed", range(40))
def test_random_batches(seed):
    rng = np.random.default_rng(1000 + seed)
    which = str(rng.choice(["64", "128", "latent"]))
    hkv = 1 if which == "latent" else int(rng.integers(1, 4))
    extra = 16 * int(rng.integers(0, 3))
    f = fmt(which, str(rng.choice(["bf16", "fp16"])), hkv)
    f = fmt(which, f.dtype, hkv, row_bytes=f.row_bytes + extra)
    hq = hkv * int(rng.choice([1, 3, 4, 8, 16, 40]))
    bs = int(rng.integers(1, 7))
    q = rng.integers(0, rng.choice([3, 12, 90]), bs)
    kv = rng.integers(0, rng.choice([80, 400, 2500]), bs)
    page = int(rng.choice([1, 3, 8, 16, 50, 64]))
    window = int(rng.choice([0, 0, 1, 12, 33, 200]))
    sinks = int(rng.choice([0, 4, 17, 40]))
    groups = []
    if bs > 1 and rng.random() < 0.6:
        n = int(rng.integers(2, bs + 1))
        shared = page * int(rng.integers(1, 2 + rng.choice([40, 300, 1500]) // page))
        kv[:n] = shared + q[:n] + rng.integers(0, rng.choice([2, 20, 600]), n)
        groups = [(0, n, shared)]
    b = HeldBatch(f, hq, q.tolist(), kv.tolist(), page=page, groups=groups, seed=seed)
    plan = b.plan(window, sinks)
    ws = plan.workspace().fill_(255) if plan.workspace_bytes else None
    status = word()
    scale = 1.0 / math.sqrt(f.k_dim)
    out, lse = gpb.attend_paged(plan, b.q, b.pool, b.table, scale, workspace=ws, status=status)
    assert int(status) == 0
    if sum(q):
        check(out, lse, b.want(window, sinks, scale))


def test_rows_past_4_gib():
    f = fmt("128", "bf16", 8)
    pages = (5 << 30) // (64 * f.row_bytes)
    pool = torch.zeros(pages * 64, f.row_bytes, dtype=torch.uint8, device="cuda")
    rows = held_rows(f, normal(4, 150, 8, 128), normal(5, 150, 8, 128))
    ids = [pages - 1, 0, pages - 2]
    for i, p in enumerate(ids):
        part = rows[i * 64:(i + 1) * 64]
        pool[p * 64:p * 64 + len(part)] = part
    q = normal(5, 3, 16, 128)
    plan = gpb.AttendPlan(f, 16, [3], [150])
    k, v = split(f, plain_rows(f, rows))
    want = attention(q, k, v, torch.arange(147, 150, device="cuda"), 0, 0, 0.1)
    check(*gpb.attend_paged(plan, q, pool, ints([ids]), 0.1), want)
    at = pages * 64 - 150
    pool[at:] = rows
    check(*gpb.attend_dense(plan, q, pool, ints([at]), 0.1), want)


def test_pages_outside_the_pool_are_reported_and_touch_one_request():
    f = fmt("64", "bf16", 1)
    b = HeldBatch(f, 2, [1, 1, 1], [200, 200, 200], stale=0.0)
    plan = b.plan()
    good, _ = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1)
    for wrong in (-1, 10 ** 9, b.pool.shape[0] // 64, -2 ** 31):
        t = b.table.clone()
        t[1, 2] = wrong
        status = word()
        out, _ = gpb.attend_paged(plan, b.q, b.pool, t, 0.1, status=status)
        assert int(status) == gpb.STATUS_BAD_DESCRIPTOR
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        assert torch.isfinite(out).all()
    for call, pages, kw in ((gpb.attend_dense, ints([0, 2 ** 31 - 5, -9]), {}),
                            (gpb.attend_paged, b.table, {"page_base": ints([0, 2 ** 31 - 5, -9])})):
        status = word()
        call(plan, b.q, b.dense if call is gpb.attend_dense else b.pool, pages, 0.1,
             status=status, **kw)
        assert int(status) == gpb.STATUS_BAD_DESCRIPTOR


@pytest.mark.parametrize("which,hkv,hq", [("64", 8, 64), ("128", 2, 8), ("latent", 1, 16)])
def test_results_do_not_change_from_run_to_run(which, hkv, hq):
    b = HeldBatch(fmt(which, "bf16", hkv), hq, [1] * 12, [2000 + 77 * r for r in range(12)],
                  groups=[(0, 7, 1920)])
    plan = b.plan()
    first = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1)
    for _ in range(3):
        again = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.parametrize("which", ["128", "latent"])
def test_strided_queries_and_results_and_rows_behind(which):
    f = fmt(which, "bf16", 1)
    b = HeldBatch(f, 8, [70, 1], [200, 900])
    want = b.want(0, 0, 0.1)
    T = 71
    wide = normal(3, T, 8, f.k_dim + 24)
    wide[..., 8:8 + f.k_dim] = b.q[:T]
    out = torch.full((T + 3, 8, f.v_dim + 8), 9.0, dtype=f.dtype, device="cuda")
    got, lse = gpb.attend_paged(b.plan(), wide[..., 8:8 + f.k_dim], b.pool, b.table, 0.1,
                                out=out[..., :f.v_dim])
    check(out[:T, :, :f.v_dim], lse, want)
    assert (out[..., f.v_dim:] == 9).all() and (out[T:] == 9).all()


# ------------------------------------------------------------------ together

def test_two_captured_graphs_on_streams_of_their_own():
    """Append, attention and reading back captured twice, replayed in turn with eager
    work in between; every replay equals the eager result."""
    f = fmt("128", "bf16", 2)
    b = HeldBatch(f, 8, [1, 1], [1400, 900])
    plan = b.plan()
    rot = gpb.Rotation(torch.full((64,), 0.01, device="cuda"))
    pos = ints([1399, 899])
    locs = ints([b.lists[0][1399 // 64] * 64 + 1399 % 64, b.lists[1][899 // 64] * 64 + 899 % 64])
    k, v, q = normal(1, 2, 2, 128), normal(2, 2, 2, 128), normal(3, 2, 8, 128)
    turned = torch.empty_like(q)

    def step(out, lse, back):
        gpb.row_append(f, k, v, b.pool, locs, rot, pos, q=q, q_out=turned)
        gpb.attend_paged(plan, turned, b.pool, b.table, 0.1, out=out, lse=lse)
        gpb.rows_read(f, b.pool, locs, out=back)

    def buffers():
        return (torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(2, 8, device="cuda"),
                torch.zeros(2, f.values, dtype=torch.bfloat16, device="cuda"))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*buffers())
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for _ in range(2):
        bufs = buffers()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(*bufs)
        graphs.append((g, bufs))
    for turn in range(4):
        k.copy_(normal(20 + turn, 2, 2, 128))
        v.copy_(normal(25 + turn, 2, 2, 128))
        q.copy_(normal(30 + turn, 2, 8, 128))
        eager = buffers()
        step(*eager)
        torch.cuda.synchronize()
        for g, bufs in graphs:
            bufs[0].zero_()
            g.replay()
            torch.cuda.synchronize()
            for x, y in zip(bufs, eager):
                assert torch.equal(x, y)


def test_other_streams():
    f = fmt("128", "bf16", 2)
    b = HeldBatch(f, 8, [1, 90], [1500, 1800])
    plan = b.plan()
    want = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1)
    back = gpb.rows_read(f, b.pool)
    torch.cuda.synchronize()
    for s in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        o, l = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1, stream=s)
        r = gpb.rows_read(f, b.pool, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
        assert torch.equal(r.view(torch.int16), back.view(torch.int16))


def test_append_compose_attend_read_and_decode():
    """A prefill of held rows through the runner (made, composed, attended from the
    dense buffer and from the pool, read back) and a decode step after it."""
    batch = workloads.make_batch("tiny")
    f = fmt("latent")
    assert f.row_bytes == 656
    n_pool = batch.n_pool_pages * 64
    old = held_rows(f, normal(7, n_pool, 1, 576), None)
    pools = [old.clone()]
    T = int(batch.cur_tokens.sum())
    curs = [torch.zeros(T, f.row_bytes, dtype=torch.uint8, device="cuda")]
    meta = gpb.BatchMeta(batch.bs, 64, f.row_bytes, batch.n_pool_pages, 1, 1,
                         T // 64 + batch.bs + 2, batch.prefix_pages, batch.cur_tokens,
                         batch.req_pages)
    r = gpb.ComposeRunner(meta, pools, curs)
    r.begin_batch()
    hq, scale = 16, 0.07
    k, q = normal(1, T, 1, 576), normal(2, T, hq, 576)
    freq = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    rot = gpb.Rotation(freq, start=512, interleaved=True)
    c, P = batch.cur_tokens, batch.prefix_pages
    pos = ints(np.concatenate([P[i] * 64 + np.arange(c[i]) for i in range(batch.bs)]))
    turned = torch.empty_like(q)
    r.append(0, f, k, None, rot, pos, q=q, q_out=turned)
    made = plain_rows(f, curs[0]).double()
    kd = rotated(k, pos[None], freq, 512, True, [32])[:, 0]
    assert torch.equal(curs[0][:, :512], hold(k[:, 0, :512], f.dtype)[0])
    assert ((made[:, 512:] - kd[:, 512:]).abs() <=
            rotation_bound(kd[:, None], k, f.dtype)[:, 0, 512:]).all()
    r.layer(0)
    plan = r.attend_plan(f, hq)
    out, lse = r.attend(0, plan, turned, scale)
    from_pool = r.attend_pool(0, plan, turned, scale)
    dense = r.read(0, f)
    assert int(r.status) == 0
    assert torch.equal(out, from_pool[0]) and torch.equal(lse, from_pool[1])
    at, want = 0, []
    for i in range(batch.bs):
        base, n = int(r.plan.t["k_bases"][i]), int(P[i]) * 64 + int(c[i])
        assert torch.equal(dense[base:base + n], plain_rows(f, r.dense_of(0)[base:base + n]))
        assert torch.equal(dense[base + n - int(c[i]):base + n].double(),
                           made[at:at + int(c[i])])
        keys, vals = split(f, dense[base:base + n])
        want.append(attention(turned[at:at + int(c[i])], keys, vals,
                              torch.arange(n - int(c[i]), n, device="cuda"), 0, 0, scale))
        at += int(c[i])
    check(out, lse, [torch.cat([w[j] for w in want]) for j in range(4)])

    # the same attention over the rows read back, with the plain format: as near
    plain = fmt("latent", held=None)
    p16 = gpb.AttendPlan(plain, hq, c, P * 64 + c)
    check(*gpb.attend_dense(p16, turned, dense, r.plan.t["k_bases"], scale),
          [torch.cat([w[j] for w in want]) for j in range(4)])

    # one more token per request
    n = [int(P[i]) * 64 + int(c[i]) for i in range(batch.bs)]
    base, pages = r.plan.t["slot_base"].tolist(), r.plan.t["slot_pages"].tolist()
    lists = [pages[base[i]:base[i] + -(-n[i] // 64)] for i in range(batch.bs)]
    assert all(x % 64 for x in n)
    width = max(len(x) for x in lists)
    table = ints([x + [0] * (width - len(x)) for x in lists])
    locs = ints([lists[i][n[i] // 64] * 64 + n[i] % 64 for i in range(batch.bs)])
    k1, q1 = normal(8, batch.bs, 1, 576), normal(9, batch.bs, hq, 576)
    gpb.row_append(f, k1, None, pools[0], locs, rot, ints(n), q=q1)
    step = gpb.AttendPlan(f, hq, [1] * batch.bs, [x + 1 for x in n])
    o1, l1 = gpb.attend_paged(step, q1, pools[0], table, scale)
    want = []
    for i in range(batch.bs):
        idx = ints([p * 64 + j for p in lists[i] for j in range(64)][:n[i] + 1])
        keys, vals = split(f, gpb.rows_read(f, pools[0], idx))
        want.append(attention(q1[i:i + 1], keys, vals, ints([n[i]]), 0, 0, scale))
    check(o1, l1, [torch.cat([w[j] for w in want]) for j in range(4)])
    with pytest.raises(ValueError):
        r.read(0, fmt("128"))
