"""The row append and the attentions on the GPU, against 64-bit references."""
import math

import numpy as np
import pytest
import torch

import gather_plan_build_amd as gpb
from rows_reference import attention, check, rotated, rotation_bound
import workloads

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def fmt(which, dtype="bf16", hkv=2, **kw):
    if which == "latent":
        return gpb.RowFormat(dtype, 1, 576, 512, values_in_key=True, **kw)
    return gpb.RowFormat(dtype, hkv, int(which), int(which), **kw)


def normal(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def ints(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append

def row_values(f, k, v):
    return torch.cat([k.flatten(1)] + ([] if v is None else [v.flatten(1)]), 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("which,hkv,hq,start,pairs,interleaved,sections", [
    ("128", 2, 6, 0, 64, False, None),
    ("128", 3, 3, 0, 64, False, [16, 24, 24]),
    ("128", 1, 5, 32, 16, True, [1, 15]),
    ("64", 4, 8, 0, 32, True, None),
    ("64", 1, 2, 8, 8, False, [0, 3, 5, 0]),
    ("latent", 1, 16, 512, 32, True, None),
    ("latent", 1, 1, 0, 256, False, [100, 156]),
    ("128", 2, 4, 0, 0, False, None),
])
@pytest.mark.parametrize("tokens", [1, 67])
def test_append(dtype, which, hkv, hq, start, pairs, interleaved, sections, tokens):
    f = fmt(which, dtype, hkv)
    dt = f.dtype
    # keys, values and queries are parts of one packed tensor, as a projection
    # leaves them
    parts = [hq, f.n_kv_heads] + ([] if f.values_in_key else [f.n_kv_heads])
    packed = normal(1, tokens, sum(parts) * f.k_dim, dtype=dt)
    q = packed[:, :hq * f.k_dim].unflatten(1, (hq, f.k_dim))
    k = packed[:, hq * f.k_dim:(hq + hkv) * f.k_dim].unflatten(1, (hkv, f.k_dim))
    v = None if f.values_in_key else packed[:, (hq + hkv) * f.k_dim:].unflatten(
        1, (hkv, f.v_dim))
    sec = sections or [pairs]
    rng = np.random.default_rng(tokens)
    pos = ints(rng.integers(-5, 2 ** 31 - 1, (len(sec), tokens)) // rng.integers(
        1, 2 ** 20, (len(sec), tokens)))
    freq = (10000.0 ** (-torch.arange(pairs, dtype=torch.float64) / max(pairs, 1))).float().cuda()
    rot = gpb.Rotation(freq, start, interleaved, sec) if pairs else None
    n = f.row_bytes // 2
    pool = normal(2, 200, n, dtype=dt)
    before = pool.clone()
    locs = rng.permutation(200)[:tokens]
    locs[tokens // 2] = -1                       # a padded entry
    rows = torch.empty(tokens, n, dtype=dt, device="cuda")
    q_out = torch.empty(tokens, hq, f.k_dim, dtype=dt, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gpb.row_append(f, k, v, pool, ints(locs), rot, pos, rows=rows, q=q, q_out=q_out,
                   status=status)
    assert int(status) == 0
    kd, qd = (k.double(), q.double())
    if pairs:
        kd = rotated(k, pos, freq, start, interleaved, sec)
        qd = rotated(q, pos, freq, start, interleaved, sec)
    assert ((q_out.double() - qd).abs() <= rotation_bound(qd, q, dt)).all()
    got_k = rows[:, :f.n_kv_heads * f.k_dim].view(tokens, -1, f.k_dim)
    assert ((got_k.double() - kd).abs() <= rotation_bound(kd, k, dt)).all()
    if v is not None:
        assert torch.equal(rows[:, f.n_kv_heads * f.k_dim:], v.flatten(1))
    # what is not rotated is copied
    out = torch.ones(f.k_dim, dtype=torch.bool)
    out[start:start + 2 * pairs] = False
    assert torch.equal(got_k[..., out], k[..., out])
    want = before.clone()
    for t, at in enumerate(locs):
        if at >= 0:
            want[at] = rows[t]
    assert torch.equal(pool, want)
    # in place, and without a pool
    q2 = q.clone()
    rows2 = torch.zeros_like(rows)
    gpb.row_append(f, k, v, None, None, rot, pos, rows=rows2, q=q2)
    assert torch.equal(q2, q_out) and torch.equal(rows2, rows)
    q3 = packed.clone()
    part = q3[:, :hq * f.k_dim].unflatten(1, (hq, f.k_dim))
    gpb.row_append(f, k, v, pool, ints(locs), rot, pos, q=part)
    assert torch.equal(part, q_out)
    assert torch.equal(q3[:, hq * f.k_dim:], packed[:, hq * f.k_dim:])


def test_append_flags_rows_outside_the_pool_and_keeps_the_padding():
    f = fmt("64", hkv=1, row_bytes=64 * 4 + 32)
    k, v = normal(1, 4, 1, 64), normal(2, 4, 1, 64)
    pool = normal(3, 8, f.row_bytes // 2)
    before = pool.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gpb.row_append(f, k, v, pool, ints([7, 8, -1, 2]), status=status)
    assert int(status) == gpb.STATUS_BAD_STAGING_ROW
    want = before.clone()
    for t, at in ((0, 7), (3, 2)):
        want[at, :64], want[at, 64:128] = k[t, 0], v[t, 0]
    assert torch.equal(pool, want)
    status.zero_()
    gpb.row_append(f, k, v, pool, ints([-2, 0, 1, 3]), status=status)
    assert int(status) == gpb.STATUS_BAD_STAGING_ROW


def test_append_past_4_gib_of_pool():
    f = fmt("128", hkv=8)
    n = (5 << 30) // f.row_bytes
    pool = torch.zeros(n, f.row_bytes // 2, dtype=torch.bfloat16, device="cuda")
    k, v = normal(1, 2, 8, 128), normal(2, 2, 8, 128)
    gpb.row_append(f, k, v, pool, ints([n - 1, 0]))
    assert torch.equal(pool[n - 1], row_values(f, k, v)[0])
    assert torch.equal(pool[0], row_values(f, k, v)[1])
    assert not pool[n - 2].any()


# ------------------------------------------------------------------ attention

def split(f, rows):
    """[n, row values] -> keys, values."""
    k = rows[:, :f.n_kv_heads * f.k_dim].reshape(-1, f.n_kv_heads, f.k_dim)
    v = rows[:, :f.v_dim].reshape(-1, 1, f.v_dim) if f.values_in_key else \
        rows[:, f.n_kv_heads * f.k_dim:f.n_kv_heads * (f.k_dim + f.v_dim)].reshape(
            -1, f.n_kv_heads, f.v_dim)
    return k, v


class Batch:
    """Rows of a batch, dense and paged, with stale rows all around them."""

    def __init__(self, f, hq, q_lens, kv_lens, page=64, groups=(), seed=0, stale=float("nan")):
        self.f, self.hq, self.q_lens, self.kv_lens, self.page = f, hq, q_lens, kv_lens, page
        self.groups = list(groups)
        dt, n = f.dtype, f.row_bytes // 2
        rng = np.random.default_rng(seed)
        self.q = normal(seed + 1, sum(q_lens) + 3, hq, f.k_dim, dtype=dt)
        self.rows = [normal(seed + 10 + r, m, n, dtype=dt) for r, m in enumerate(kv_lens)]
        for first, count, shared in self.groups:
            for r in range(first + 1, first + count):
                self.rows[r][:shared] = self.rows[first][:shared]
        need = [-(-m // page) for m in kv_lens]
        base = np.concatenate([[0], np.cumsum([p * page for p in need])])
        self.dense = torch.full((int(base[-1]) + 5, n), stale, dtype=dt, device="cuda")
        for b, x in zip(base, self.rows):
            self.dense[b:b + len(x)] = x
        self.k_bases = ints(base[:-1])
        total = sum(need) + 4
        ids = iter(rng.permutation(total))
        self.pool = torch.full((total * page, n), stale, dtype=dt, device="cuda")
        own = {r: (first, shared // page) for first, count, shared in self.groups
               for r in range(first + 1, first + count)}
        self.lists = []
        for r, m in enumerate(kv_lens):
            first, s = own.get(r, (None, 0))
            pages = (self.lists[first][:s] if s else []) + [int(next(ids)) for _ in range(need[r] - s)]
            self.lists.append(pages)
            for i in range(s, need[r]):
                part = self.rows[r][i * page:(i + 1) * page]
                self.pool[pages[i] * page:pages[i] * page + len(part)] = part
        width = max(need + [1]) + 2
        self.table = ints([p + [-1] * (width - len(p)) for p in self.lists])

    def want(self, window, sinks, scale):
        parts, at = [], 0
        for r, (n, m) in enumerate(zip(self.q_lens, self.kv_lens)):
            pos = torch.arange(m - n, m, device="cuda")
            k, v = split(self.f, self.rows[r])
            parts.append(attention(self.q[at:at + n], k, v, pos, window, sinks, scale))
            at += n
        return [torch.cat([p[i] for p in parts]) for i in range(4)]

    def plan(self, window=0, sinks=0, groups=True):
        return gpb.AttendPlan(self.f, self.hq, self.q_lens, self.kv_lens, window=window,
                              sinks=sinks, page_size=self.page,
                              groups=self.groups if groups else ())

    def check(self, window=0, sinks=0, dense=True):
        T = sum(self.q_lens)
        scale = 1.0 / math.sqrt(self.f.k_dim)
        want = self.want(window, sinks, scale)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        plan = self.plan(window, sinks)
        out, lse = gpb.attend_paged(plan, self.q, self.pool, self.table, scale, status=status)
        assert out.shape == (T, self.hq, self.f.v_dim) and lse.shape == (T, self.hq)
        check(out, lse, want)
        assert int(status) == 0
        if dense:
            flat = self.plan(window, sinks, groups=False) if self.groups else plan
            o2, l2 = gpb.attend_dense(flat, self.q, self.dense, self.k_bases, scale,
                                      status=status)
            check(o2, l2, want)
            assert int(status) == 0
            if not self.groups:      # the same work list: the same sums
                assert torch.equal(out.view(torch.int16), o2.view(torch.int16))
                assert torch.equal(lse, l2)
        return out, lse


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
    Batch(fmt(which, dtype, hkv), hq, q, kv).check()


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 14), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 3), (64, 64), (100, 0),
                                          (300, 70), (5000, 4), (2, 5000)])
def test_windows_and_first_tokens(which, hkv, hq, window, sinks):
    Batch(fmt(which, "bf16", hkv), hq, [1, 90, 2, 200], [640, 500, 1000, 200]).check(window, sinks)


@pytest.mark.parametrize("hq,hkv,which", [(128, 1, "latent"), (130, 1, "128"), (48, 1, "64"),
                                          (200, 1, "latent"), (33, 3, "128"), (1, 1, "latent")])
def test_heads(hq, hkv, which):
    Batch(fmt(which, "bf16", hkv), hq, [2, 5, 1], [700, 5, 90]).check()


@pytest.mark.parametrize("page", [1, 3, 16, 48, 100, 256])
@pytest.mark.parametrize("which", ["64", "128", "latent"])
def test_page_sizes(page, which):
    Batch(fmt(which, "fp16", 1), 4, [1, 4, 70], [333, 65, 70], page=page).check(window=0)


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 16), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("q,kv,page,groups,window,sinks", [
    ([1, 1, 1], [700, 650, 641], 64, [(0, 3, 640)], 0, 0),
    ([2, 1, 3, 1], [330, 301, 420, 55], 10, [(0, 3, 300)], 0, 0),     # ends inside a tile
    ([1] * 20, [1030 + 3 * r for r in range(20)], 64, [(0, 9, 1024), (9, 11, 512)], 0, 0),
    ([1, 2, 1, 1], [1100, 1200, 1300, 2000], 50, [(0, 3, 1000)], 150, 5),
    ([1, 0, 1], [200, 128, 129], 64, [(0, 3, 128)], 0, 0),
    ([40, 30, 20], [168, 158, 148], 64, [(0, 3, 128)], 0, 0),
    ([1, 1], [640, 640], 64, [(0, 1, 64), (1, 1, 64)], 0, 0),
])
def test_shared_prefixes(which, hkv, hq, q, kv, page, groups, window, sinks):
    Batch(fmt(which, "bf16", hkv), hq, q, kv, page=page, groups=groups).check(window, sinks)


@pytest.mark.parametrize("which", ["64", "128"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("q,kv,window,sinks", [
    ([100], [230], 0, 0),            # a later token's values: seen by later queries alone
    ([20], [500], 40, 2),            # values that left the window of some queries
    ([1, 3], [70, 40], 0, 0),
])
def test_values_that_are_not_finite_reach_those_that_see_them_only(which, bad, q, kv, window,
                                                                   sinks):
    f = fmt(which, "bf16", 1)
    b = Batch(f, 4, q, kv)
    for r in range(len(kv)):
        n = kv[r]
        rows = [n - 1, max(0, n - q[r] // 2 - 1)]
        if window:
            rows.append(n - q[r] - window + 3)
        for x in rows:
            b.rows[r][x, f.k_dim + 5] = bad
    base = b.k_bases.tolist()
    for r, x in enumerate(b.rows):
        b.dense[base[r]:base[r] + len(x)] = x
        for i, p in enumerate(b.lists[r]):
            part = x[i * 64:(i + 1) * 64]
            b.pool[p * 64:p * 64 + len(part)] = part
    b.check(window, sinks)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_latent_rows_that_are_not_finite(bad):
    """A latent is key and value: a query that sees the row has no finite score,
    the others must not notice."""
    f = fmt("latent", "bf16")
    b = Batch(f, 4, [60], [200])
    b.rows[0][170, 7] = bad
    b.dense[170] = b.rows[0][170]
    scale = 0.05
    plan = b.plan()
    out, lse = gpb.attend_dense(plan, b.q, b.dense, b.k_bases, scale)
    clean = b.rows[0].clone()
    clean[170] = 0
    k, v = split(f, clean)
    pos = torch.arange(140, 200, device="cuda")
    want = attention(b.q[:60], k, v, pos, 0, 0, scale)
    check(out[:30], lse[:30], [w[:30] for w in want])
    assert not torch.isfinite(out[30:, :, 7]).any()


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 16), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 3)])
def test_values_that_are_not_finite_behind_a_shared_prefix(which, hkv, hq, window, sinks):
    """The last key of each request, which its last query alone sees, and a
    shared key that a window hides from all."""
    f = fmt(which, "bf16", hkv)
    b = Batch(f, hq, [2, 40, 1, 3], [200, 290, 300, 260], groups=[(0, 4, 128)], stale=0.0)
    at = 0 if f.values_in_key else hkv * f.k_dim     # a value
    for r, n in ((0, 200), (1, 290), (3, 260)):
        b.rows[r][n - 1, at] = float("inf")
        b.pool[b.lists[r][(n - 1) // 64] * 64 + (n - 1) % 64, at] = float("inf")
    if window:
        for r in range(4):
            b.rows[r][5, at] = float("nan")
        b.pool[b.lists[0][0] * 64 + 5, at] = float("nan")
    b.check(window, sinks, dense=False)


def test_large_scores_and_a_growing_maximum():
    """Keys that grow along the sequence move the running maximum in every
    tile; scores of some hundreds stay in range."""
    for which in ("64", "128", "latent"):
        f = fmt(which, "fp16", 1)
        b = Batch(f, 4, [1, 70], [900, 300], stale=0.0)
        for r, x in enumerate(b.rows):
            grow = torch.linspace(0.1, 8.0, len(x), device="cuda")[:, None]
            x[:, :f.k_dim] = (x[:, :f.k_dim] * grow).to(f.dtype)
            base = int(b.k_bases[r])
            b.dense[base:base + len(x)] = x
            for i, p in enumerate(b.lists[r]):
                part = x[i * 64:(i + 1) * 64]
                b.pool[p * 64:p * 64 + len(part)] = part
        b.check()


def test_small_weights_in_half_precision():
    """One key far above many others whose weights are below what fp16 holds of
    a weight of 1: together they are a third of the sum."""
    f = fmt("64", "fp16", 1)
    n = 60000
    b = Batch(f, 2, [1], [n], stale=0.0)
    b.rows[0][:, :64] = 0
    b.rows[0][100, :64] = 1
    b.q[:] = 0
    b.q[..., :64] = 11.7 / 8.0          # score 11.7 against 0: weights of 2^-17
    b.rows[0][:, 64:] = 1.0
    b.rows[0][100, 64:] = -1.0
    for i, p in enumerate(b.lists[0]):
        part = b.rows[0][i * 64:(i + 1) * 64]
        b.pool[p * 64:p * 64 + len(part)] = part
    b.dense[:n] = b.rows[0]
    b.check()


@pytest.mark.parametrize("which", ["128", "latent"])
def test_strided_queries_and_results_and_rows_behind(which):
    f = fmt(which, "bf16", 1)
    hq, T = 4, 75
    b = Batch(f, hq, [1, 74], [400, 90])
    want = b.want(0, 0, 0.1)
    plan = b.plan()
    wide = normal(5, hq + 1, T + 9, f.k_dim + 8).transpose(0, 1)[:, :hq, :f.k_dim]
    wide[:T] = b.q[:T]
    assert not wide.is_contiguous()
    full = torch.full((T + 9, hq, f.v_dim + 4), 7.0, dtype=f.dtype, device="cuda")
    lse = torch.full((T + 9, hq), 7.0, device="cuda")
    out, l2 = gpb.attend_paged(plan, wide, b.pool, b.table, 0.1, out=full[..., :f.v_dim], lse=lse)
    assert l2 is lse
    check(out[:T], lse[:T], want)
    assert (full[T:] == 7).all() and (full[..., f.v_dim:] == 7).all() and (lse[T:] == 7).all()
    only, none = gpb.attend_paged(plan, wide, b.pool, b.table, 0.1, lse=None)
    assert none is None and torch.equal(only, out[:T])


def test_page_lists_of_a_compose_plan_form():
    f = fmt("128", "bf16", 2)
    b = Batch(f, 4, [1, 2, 0, 9], [300, 70, 128, 9])
    flat = ints([x for p in b.lists for x in p])
    starts = ints(np.concatenate([[0], np.cumsum([len(p) for p in b.lists])[:-1]]))
    plan = b.plan()
    out, lse = gpb.attend_paged(plan, b.q, b.pool, flat, 0.1, page_base=starts)
    check(out, lse, b.want(0, 0, 0.1))


def test_pages_outside_the_pool_are_reported_and_touch_one_request():
    f = fmt("64", "bf16", 1)
    b = Batch(f, 2, [1, 1, 1], [200, 200, 200], stale=0.0)
    plan = b.plan()
    good, _ = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1)
    for wrong in (-1, 10 ** 9, b.pool.shape[0] // 64, -2 ** 31):
        t = b.table.clone()
        t[1, 2] = wrong
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, _ = gpb.attend_paged(plan, b.q, b.pool, t, 0.1, status=status)
        assert int(status) == gpb.STATUS_BAD_DESCRIPTOR
        assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
        assert torch.isfinite(out).all()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bases = ints([0, 2 ** 31 - 5, -9])
    gpb.attend_dense(plan, b.q, b.dense, bases, 0.1, status=status)
    assert int(status) == gpb.STATUS_BAD_DESCRIPTOR
    status.zero_()
    starts = ints([0, 2 ** 31 - 5, -9])
    gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1, page_base=starts, status=status)
    assert int(status) == gpb.STATUS_BAD_DESCRIPTOR


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 16), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("q,kv,page,window,sinks", [
    ([1, 1], [2000, 700], 16, 100, 0),
    ([1, 2], [2000, 700], 16, 100, 4),
    ([40, 33], [1500, 400], 16, 70, 0),
    ([300], [900], 8, 33, 17),
    ([1], [3000], 256, 1000, 1),
])
def test_pages_that_no_query_sees_are_not_read(which, hkv, hq, q, kv, page, window, sinks):
    """The pages behind a window are no longer the request's: their entries are
    not asked for, whatever tile the window's first keys share."""
    b = Batch(fmt(which, "bf16", hkv), hq, q, kv, page=page)
    for r, (n, m) in enumerate(zip(q, kv)):
        first, sunk = max(0, m - n + 1 - window) // page, -(-sinks // page)
        b.table[r, sunk:max(first, sunk)] = -1
    b.check(window, sinks, dense=False)


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 16), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("window,sinks", [(2 ** 31 - 1, 0), (2 ** 30, 2 ** 31 - 1),
                                          (5, 2 ** 31 - 1), (1, 0)])
def test_largest_windows_and_queries_before_any_key(which, hkv, hq, window, sinks):
    Batch(fmt(which, "bf16", hkv), hq, [150, 1], [100, 64]).check(window, sinks)


@pytest.mark.parametrize("which", ["64", "128", "latent"])
def test_results_with_heads_outermost(which):
    b = Batch(fmt(which, "fp16", 1), 8, [70, 1], [200, 900])
    f, want = b.f, b.want(0, 0, 0.1)
    out = torch.zeros(8, 71, f.v_dim, dtype=f.dtype, device="cuda").transpose(0, 1)
    q = b.q.transpose(0, 1).contiguous().transpose(0, 1)
    got, lse = gpb.attend_paged(b.plan(), q, b.pool, b.table, 0.1, out=out)
    assert got.data_ptr() == out.data_ptr()
    check(out, lse, want)
    with pytest.raises(gpb.GpbError):
        gpb.attend_paged(b.plan(), q, b.pool, b.table, 0.1,
                         out=out[:1].expand(71, 8, f.v_dim))


def test_an_item_whose_rows_end_past_int32_is_reported():
    b = Batch(fmt("64", "bf16", 1), 2, [1, 1], [90, 20], stale=0.0)
    plan = b.plan()
    host = plan.list_host.copy()
    host[1] = 2 ** 31 - 1                       # the first item's first row
    plan.list.copy_(torch.from_numpy(host))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1, status=status)
    assert int(status) == 4          # GPB_STATUS_BAD_PLAN_INPUT


def test_a_list_that_is_not_the_plans_is_reported():
    f = fmt("64", "bf16", 1)
    b = Batch(f, 2, [1, 1], [900, 2000], stale=0.0)
    plan = b.plan()
    assert plan.c.n_joins > 0
    for fill in (-1, 2 ** 30, -2 ** 31):
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        plan.list.fill_(fill)
        gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1, status=status)
        assert int(status) == 4          # GPB_STATUS_BAD_PLAN_INPUT


def test_rows_past_4_gib():
    """Pages at both ends of a pool of more than 4 GiB, and a dense buffer whose
    last request starts past it."""
    f = fmt("128", "bf16", 8)
    pages = (5 << 30) // (64 * f.row_bytes)
    pool = torch.zeros(pages * 64, f.row_bytes // 2, dtype=torch.bfloat16, device="cuda")
    rows = normal(4, 150, f.row_bytes // 2)
    ids = [pages - 1, 0, pages - 2]
    for i, p in enumerate(ids):
        part = rows[i * 64:(i + 1) * 64]
        pool[p * 64:p * 64 + len(part)] = part
    q = normal(5, 3, 16, 128)
    plan = gpb.AttendPlan(f, 16, [3], [150])
    k, v = split(f, rows)
    want = attention(q, k, v, torch.arange(147, 150, device="cuda"), 0, 0, 0.1)
    check(*gpb.attend_paged(plan, q, pool, ints([ids]), 0.1), want)
    at = pages * 64 - 150
    pool[at:] = rows
    check(*gpb.attend_dense(plan, q, pool, ints([at]), 0.1), want)


@pytest.mark.parametrize("which,hkv,hq", [("64", 8, 64), ("128", 2, 8), ("latent", 1, 16)])
def test_results_do_not_change_from_run_to_run(which, hkv, hq):
    b = Batch(fmt(which, "bf16", hkv), hq, [1] * 12, [2000 + 77 * r for r in range(12)],
              groups=[(0, 7, 1920)])
    plan = b.plan()
    first = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1)
    for _ in range(3):
        again = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_other_streams_and_workspaces():
    b = Batch(fmt("128", "bf16", 2), 8, [1, 1], [1500, 1800])
    plan = b.plan()
    want = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1, stream=s) for s in streams]
    got.append(gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1, stream=streams[0].cuda_stream,
                                workspace=plan.workspace()))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])
    with pytest.raises(gpb.GpbError):
        gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1,
                         workspace=plan.workspace()[:-16])
    with pytest.raises(ValueError):
        gpb.attend_paged(plan, b.q.cpu(), b.pool, b.table, 0.1)
    with pytest.raises(ValueError):
        gpb.attend_paged(plan, b.q.half(), b.pool, b.table, 0.1)
    with pytest.raises(ValueError):
        gpb.attend_paged(plan, b.q[:1], b.pool, b.table, 0.1)


def test_two_captured_graphs_of_a_decode_step():
    """Append and attention captured twice, replayed in turn with eager work in
    between; every replay equals the eager result."""
    f = fmt("128", "bf16", 2)
    b = Batch(f, 8, [1, 1], [1400, 900])
    plan = b.plan()
    freq = torch.full((64,), 0.01, device="cuda")
    rot = gpb.Rotation(freq)
    pos = ints([1399, 899])
    locs = ints([b.lists[0][1399 // 64] * 64 + 1399 % 64, b.lists[1][899 // 64] * 64 + 899 % 64])
    k, v, q = normal(1, 2, 2, 128), normal(2, 2, 2, 128), normal(3, 2, 8, 128)
    turned = torch.empty_like(q)

    def step(out, lse):
        gpb.row_append(f, k, v, b.pool, locs, rot, pos, q=q, q_out=turned)
        gpb.attend_paged(plan, turned, b.pool, b.table, 0.1, out=out, lse=lse)

    def buffers():
        return (torch.zeros(2, 8, 128, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(2, 8, device="cuda"))

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
        q.copy_(normal(30 + turn, 2, 8, 128))
        eager = buffers()
        step(*eager)
        torch.cuda.synchronize()
        for g, bufs in graphs:
            bufs[0].zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(bufs[0], eager[0]) and torch.equal(bufs[1], eager[1])


@pytest.mark.parametrize("which", ["64", "128", "latent"])
def test_batches_without_queries_or_without_keys(which):
    f = fmt(which, "bf16", 1)
    none = gpb.AttendPlan(f, 4, [], [])
    out, lse = gpb.attend_paged(none, normal(1, 0, 4, f.k_dim), normal(2, 64, f.row_bytes // 2),
                                torch.zeros(0, 3, dtype=torch.int32, device="cuda"), 0.1)
    assert out.shape == (0, 4, f.v_dim) and lse.shape == (0, 4)
    bare = gpb.AttendPlan(f, 4, [3, 0, 70], [0, 5, 0])
    q, pool = normal(3, 73, 4, f.k_dim), normal(4, 64, f.row_bytes // 2)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = gpb.attend_paged(bare, q, pool, ints([[-1], [0], [-1]]), 0.1, status=status)
    o2, l2 = gpb.attend_dense(bare, q, pool, ints([99, 0, -7]), 0.1, status=status)
    for o, l in ((out, lse), (o2, l2)):
        assert not o.any() and (l == -math.inf).all()
    assert int(status) == 0


@pytest.mark.parametrize("which,hkv,hq", [("64", 1, 8), ("128", 2, 8), ("latent", 1, 16)])
def test_prefill_captured_and_replayed_on_new_rows(which, hkv, hq):
    """Wide items with parts and joins, in a graph: every replay reads what the
    buffers hold then, an odd value in one of them included."""
    b = Batch(fmt(which, "bf16", hkv), hq, [70, 5], [1900, 1100], stale=0.0)
    plan = b.plan()
    assert plan.c.n_joins > 0
    out = torch.empty(75, hq, b.f.v_dim, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(75, hq, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gpb.attend_dense(plan, b.q, b.dense, b.k_bases, 0.1, out=out, lse=lse)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gpb.attend_dense(plan, b.q, b.dense, b.k_bases, 0.1, out=out, lse=lse)
    for turn in range(4):
        b.dense.copy_(normal(50 + turn, *b.dense.shape))
        if turn == 2:
            b.dense[1890, :8] = float("nan")      # seen by the last ten queries of request 0
        eager = gpb.attend_dense(plan, b.q, b.dense, b.k_bases, 0.1)
        torch.cuda.synchronize()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), eager[0].view(torch.int16))
        assert torch.equal(lse.view(torch.int32), eager[1].view(torch.int32))
        odd = ~torch.isfinite(out).flatten(1).all(1)
        want = torch.zeros(75, dtype=torch.bool, device="cuda")
        if turn == 2:
            want[60:70] = True
        assert torch.equal(odd, want)


def test_two_threads_on_two_streams():
    import threading
    parts = [Batch(fmt("128", "bf16", 2), 8, [1, 90], [1500, 1800], seed=7 + i) for i in range(2)]
    plans = [b.plan() for b in parts]
    want = [gpb.attend_paged(p, b.q, b.pool, b.table, 0.1) for p, b in zip(plans, parts)]
    torch.cuda.synchronize()
    got = [[], []]

    def work(i):
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            for _ in range(20):
                got[i].append(gpb.attend_paged(plans[i], parts[i].q, parts[i].pool,
                                               parts[i].table, 0.1))
            stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        assert len(got[i]) == 20
        for o, l in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])


@pytest.mark.parametrize("which,hkv,hq", [("64", 1, 4), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("q,kv,page,groups,window,sinks", [
    ([1, 1], [60, 60], 16, [(0, 2, 48)], 12, 4),
    ([1, 1], [1020, 1018], 16, [(0, 2, 1008)], 8, 4),
    ([1, 2, 1], [57, 60, 58], 1, [(0, 3, 56)], 1, 3),
    ([1, 1], [60, 60], 16, [(0, 2, 48)], 12, 0),
])
def test_shared_keys_behind_the_window(which, hkv, hq, q, kv, page, groups, window, sinks):
    """The window hides the shared keys but for the first tokens, and the batch
    ends in the tile they end in; the workspace holds what was there before."""
    b = Batch(fmt(which, "bf16", hkv), hq, q, kv, page=page, groups=groups)
    plan = b.plan(window, sinks)
    assert plan.c.n_joins > 0
    ws = plan.workspace().fill_(255)        # NaN
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1, workspace=ws, status=status)
    check(out, lse, b.want(window, sinks, 0.1))
    assert int(status) == 0


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 16), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("q,kv,page,shared,window,sinks", [
    ([1, 1], [20, 20], 8, 16, 3, 4),
    ([1, 2, 1], [600, 611, 602], 3, 594, 5, 7),
    ([40, 33], [500, 480], 16, 432, 8, 17),
])
def test_shared_pages_that_no_query_sees_are_not_read(which, hkv, hq, q, kv, page, shared, window,
                                                      sinks):
    b = Batch(fmt(which, "bf16", hkv), hq, q, kv, page=page, groups=[(0, len(q), shared)])
    for r, (n, m) in enumerate(zip(q, kv)):
        first = (m - n + 1 - window) // page
        assert min(kv) - max(q) + 1 - window > shared - page
        b.table[r, -(-sinks // page):min(first, shared // page)] = -1
    b.check(window, sinks, dense=False)


@pytest.mark.parametrize("given", ["stream", "raw", "current"])
def test_a_plan_dropped_while_another_stream_reads_its_list(given):
    """The list's memory is not handed out again before the call that waits on
    the other stream has ended."""
    b = Batch(fmt("128", "bf16", 2), 8, [1, 40], [1500, 1800])
    plan = b.plan()
    want = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1)
    torch.cuda.synchronize()
    place, size = plan.list.data_ptr(), plan.list.numel()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(1 << 26)                     # some tens of milliseconds
        if given == "current":
            got = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1)
    if given != "current":
        got = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1,
                               stream=side if given == "stream" else side.cuda_stream)
    ended = torch.cuda.Event()
    ended.record(side)
    del plan
    others = [torch.full((size,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
    waiting = not ended.query()
    torch.cuda.synchronize()
    assert waiting, "the other stream was done too soon to tell"
    assert place not in [x.data_ptr() for x in others]
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("which,hq", [("64", 32), ("128", 64), ("latent", 64)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_weights_are_rounded_once(which, hq, dtype):
    """One key alone has a value, and its scores are single products, exact in
    fp32.  Its weight is then off by one rounding to the row's type and, with
    the scaling of the score (below 2^5), the exponential, the sum and the
    division, by 2^-18; the result is rounded once more.  The maxima of the two
    halves of a tile lie apart by no whole power of two."""
    f = fmt(which, dtype, 1)
    n = 64
    b = Batch(f, hq, [1] * 60, [n] * 60, stale=0.0)
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    rand = lambda *shape: torch.rand(shape, generator=g, device="cuda")
    b.q.zero_()
    b.q[..., f.k_dim - 1] = (1 + rand(*b.q.shape[:2])).to(f.dtype)
    for r, x in enumerate(b.rows):
        x.zero_()
        x[:, f.k_dim - 1] = -8
        x[3, f.k_dim - 1] = 1 + 2 * rand(1).item()       # the largest, in the first half
        x[40, f.k_dim - 1] = 0.5 * rand(1).item()        # the largest of the second
        x[50, f.k_dim - 1] = -rand(1).item()
        at = 0 if f.values_in_key else f.k_dim
        x[50, at:at + f.v_dim - 64 * f.values_in_key] = (1 + rand(
            f.v_dim - 64 * f.values_in_key)).to(f.dtype)
        b.dense[r * n:(r + 1) * n] = x
    out, lse = gpb.attend_dense(b.plan(), b.q, b.dense, b.k_bases, 1.0)
    want, _, _, _ = b.want(0, 0, 1.0)
    half = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}[f.dtype]
    off = (out.double() - want).abs() - (2 * half + half ** 2 + 2.0 ** -18) * want.abs()
    worst = float((off / want.abs().clamp_min(1e-30)).max())
    assert worst <= 0


def put_rows(b):
    """The batch's rows to the dense buffer and the pool again."""
    base = b.k_bases.tolist()
    for r, x in enumerate(b.rows):
        b.dense[base[r]:base[r] + len(x)] = x
        for i, p in enumerate(b.lists[r]):
            part = x[i * b.page:(i + 1) * b.page]
            b.pool[p * b.page:p * b.page + len(part)] = part


def check_kinds(out, want):
    """NaN where NaN is due, and each infinity where it is."""
    for kind in (torch.isnan, torch.isposinf, torch.isneginf):
        assert torch.equal(kind(out.double()), kind(want)), kind.__name__


@pytest.mark.parametrize("which", ["64", "128"])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("q,kv,window,sinks,at", [
    ([100], [230], 0, 0, [140, 229, 180]),       # wide items, results at once
    ([20], [500], 40, 2, [1, 445, 470, 499]),    # values that left some windows
    ([1, 3], [70, 40], 0, 0, [39, 38]),          # narrow items
    ([2, 1], [2500, 3000], 0, 0, [7, 2499]),     # narrow items in parts
    ([150, 2], [3000, 700], 0, 0, [9, 2900, 2999]),   # wide items in parts
    ([150], [3000], 200, 3, [2, 2700, 2999]),
])
def test_odd_values_of_both_types(which, dtype, bad, q, kv, window, sinks, at):
    """Each result has the infinities and NaN of the formula and no others, the
    rows beside them their values."""
    f = fmt(which, dtype, 1)
    b = Batch(f, 4, q, kv)
    for x in b.rows:
        for n, i in enumerate(i for i in at if i < len(x)):
            x[i, f.k_dim + 5 + 9 * n] = bad
    put_rows(b)
    out, _ = b.check(window, sinks)
    want = b.want(window, sinks, 1.0 / math.sqrt(f.k_dim))[0]
    assert not torch.isfinite(want).all()
    check_kinds(out, want)


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 16), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 3)])
def test_odd_values_behind_a_shared_prefix_in_half_precision(which, hkv, hq, window, sinks):
    f = fmt(which, "fp16", hkv)
    b = Batch(f, hq, [2, 40, 1, 3], [200, 290, 300, 260], groups=[(0, 4, 128)], stale=0.0)
    at = 0 if f.values_in_key else hkv * f.k_dim     # a value
    for r, n in ((0, 200), (1, 290), (3, 260)):
        b.rows[r][n - 1, at] = float("inf")
    if window:
        for r in range(4):
            b.rows[r][5, at] = float("nan")
    put_rows(b)
    b.check(window, sinks, dense=False)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("q,kv", [(60, 200), (60, 3000), (3, 2000)])
def test_odd_latent_rows_in_half_precision(bad, q, kv):
    """Queries before the odd row keep their values, those that see it have none."""
    f = fmt("latent", "fp16")
    b = Batch(f, 4, [q], [kv])
    at = kv - q // 2
    b.rows[0][at, 7] = bad
    put_rows(b)
    out, lse = gpb.attend_dense(b.plan(), b.q, b.dense, b.k_bases, 0.05)
    clean = b.rows[0].clone()
    clean[at] = 0
    k, v = split(f, clean)
    pos = torch.arange(kv - q, kv, device="cuda")
    want = attention(b.q[:q], k, v, pos, 0, 0, 0.05)
    n = at - (kv - q)
    check(out[:n], lse[:n], [w[:n] for w in want])
    assert not torch.isfinite(out[n:, :, 7]).any()


@pytest.mark.parametrize("which,hq,nq", [("64", 2, 1), ("64", 4, 20), ("128", 2, 1), ("128", 4, 20),
                                         ("latent", 2, 1)])
def test_large_values_and_a_maximum_that_grows(which, hq, nq):
    """Scores grow by 5 from tile to tile, less than what moves the running
    maximum, and values are as large as weights of at most 1 allow: 60 of 5e36
    make 3e38, below the largest float."""
    f = fmt(which, "bf16", 1)
    n = 160
    b = Batch(f, hq, [nq], [n], stale=0.0)
    x = b.rows[0]
    x.zero_()
    b.q.zero_()
    b.q[..., f.k_dim - 1] = 1
    x[n - 40 - nq:, f.k_dim - 1] = 5
    at = 0 if f.values_in_key else f.k_dim
    x[:, at:at + 64] = 5e36
    put_rows(b)
    out, lse = gpb.attend_dense(b.plan(), b.q, b.dense, b.k_bases, 1.0)
    want = b.want(0, 0, 1.0)[0]
    assert torch.isfinite(out).all()
    assert ((out.double() - want).abs() <= 2.0 ** -6 * want.abs()).all()


@pytest.mark.parametrize("seed", range(60))
def test_random_batches(seed):
    """Groups, windows, first tokens, pages that end anywhere; the entries of
    pages that no query sees, and the workspace, hold anything."""
    rng = np.random.default_rng(seed)
    which = str(rng.choice(["64", "128", "latent"]))
    hkv = 1 if which == "latent" else int(rng.integers(1, 4))
    f = fmt(which, str(rng.choice(["bf16", "fp16"])), hkv)
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
    b = Batch(f, hq, q.tolist(), kv.tolist(), page=page, groups=groups, seed=seed)
    seen = np.zeros(b.table.shape, bool)           # pages that a query sees
    for r in range(bs):
        home = next((g for g in groups if g[0] < r < g[0] + g[1]), None)
        for x in range(max(0, kv[r] - q[r]), kv[r]):
            keys = np.arange(x + 1)
            if window:
                keys = keys[(x - keys < window) | (keys < sinks)]
            pages = np.unique(keys // page)
            seen[r, pages] = True
            if home:
                seen[home[0], pages[pages < home[2] // page]] = True
    for first, n, shared in groups:                # read through the first request's list
        seen[first + 1:first + n, :shared // page] = False
    b.table[torch.from_numpy(~seen).cuda()] = int(rng.choice([-1, 10 ** 9]))
    plan = b.plan(window, sinks)
    ws = plan.workspace().fill_(255) if plan.workspace_bytes else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    scale = 1.0 / math.sqrt(f.k_dim)
    out, lse = gpb.attend_paged(plan, b.q, b.pool, b.table, scale, workspace=ws, status=status)
    assert int(status) == 0
    if sum(q):
        check(out, lse, b.want(window, sinks, scale))


def test_a_stream_that_goes_before_the_plan_does():
    """A stream made elsewhere, and gone when the plan's list is handed back."""
    import ctypes
    runtime, = gpb.binding._hip_runtimes()        # the one in use
    hip = ctypes.CDLL(runtime)
    b = Batch(fmt("128", "bf16", 2), 8, [1, 40], [1500, 1800])
    want = gpb.attend_paged(b.plan(), b.q, b.pool, b.table, 0.1)
    torch.cuda.synchronize()
    plan = b.plan()
    handle = ctypes.c_void_p()
    assert hip.hipStreamCreate(ctypes.byref(handle)) == 0
    got = gpb.attend_paged(plan, b.q, b.pool, b.table, 0.1, out=torch.empty_like(want[0]),
                           lse=torch.empty_like(want[1]), workspace=plan.workspace(),
                           stream=handle.value)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert list(plan.readers) == [handle.value]
    assert hip.hipStreamDestroy(handle) == 0
    place, size = plan.list.data_ptr(), plan.list.numel()
    del plan
    others = [torch.full((size,), -1, dtype=torch.int32, device="cuda") for _ in range(8)]
    assert place not in [x.data_ptr() for x in others]     # kept until a next plan is made
    again = gpb.attend_paged(b.plan(), b.q, b.pool, b.table, 0.1)
    assert torch.equal(again[0], want[0])
    assert not gpb.binding._lists_in_use


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 8), ("128", 1, 4), ("latent", 1, 16)])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("q,kv", [([1], [1]), ([1, 1], [70, 300]), ([200, 40], [200, 1000])])
def test_a_row_that_sees_one_key_has_its_value(which, hkv, hq, dtype, q, kv):
    """Its weight is the whole sum, and both are a power of two."""
    f = fmt(which, dtype, hkv)
    b = Batch(f, hq, q, kv)
    out, lse = gpb.attend_paged(b.plan(window=1), b.q, b.pool, b.table, 0.1)
    at = 0
    for r, (n, m) in enumerate(zip(q, kv)):
        _, v = split(f, b.rows[r][m - n:])
        assert torch.equal(out[at:at + n], v.repeat_interleave(hq // v.shape[1], 1))
        at += n


# ------------------------------------------------------------------ together

def test_append_compose_attend_and_decode():
    """A prefill through the runner (rows made, composed, attended densely and
    from the pool) and a decode step after it, against the reference on the
    rows read back."""
    batch = workloads.make_batch("tiny")
    f = fmt("latent")
    pools, curs = workloads.make_values(batch, device="cuda")
    r = gpb.ComposeRunner(gpb.BatchMeta.of(batch), pools, curs)
    r.begin_batch()
    T, hq, scale = r.T, 16, 0.07
    k, q = normal(1, T, 1, 576), normal(2, T, hq, 576)
    freq = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float().cuda()
    rot = gpb.Rotation(freq, start=512, interleaved=True)
    c, P = batch.cur_tokens, batch.prefix_pages
    pos = ints(np.concatenate([P[i] * 64 + np.arange(c[i]) for i in range(batch.bs)]))
    turned = torch.empty_like(q)
    r.append(0, f, k, None, rot, pos, q=q, q_out=turned)
    kd = rotated(k, pos[None], freq, 512, True, [32])
    rows = curs[0].view(torch.bfloat16)
    assert ((rows.double()[:, None] - kd).abs() <= rotation_bound(kd, k, torch.bfloat16)).all()
    r.layer(0)
    plan = r.attend_plan(f, hq)
    out, lse = r.attend(0, plan, turned, scale)
    from_pool = r.attend_pool(0, plan, turned, scale)
    assert int(r.status) == 0
    assert torch.equal(out, from_pool[0]) and torch.equal(lse, from_pool[1])
    dense = r.dense_of(0).view(torch.bfloat16)
    at, want = 0, []
    for i in range(batch.bs):
        base, n = int(r.plan.t["k_bases"][i]), int(P[i]) * 64 + int(c[i])
        keys, vals = split(f, dense[base:base + n])
        want.append(attention(turned[at:at + int(c[i])], keys, vals,
                              torch.arange(n - int(c[i]), n, device="cuda"), 0, 0, scale))
        at += int(c[i])
    check(out, lse, [torch.cat([w[j] for w in want]) for j in range(4)])

    # one more token per request: the next row of its last page, or a new page
    n = [int(P[i]) * 64 + int(c[i]) for i in range(batch.bs)]
    used = set(r.plan.t["slot_pages"].tolist())
    free = iter(x for x in range(1, batch.n_pool_pages) if x not in used)
    base = r.plan.t["slot_base"].tolist()
    pages = r.plan.t["slot_pages"].tolist()
    lists = [pages[base[i]:base[i] + -(-n[i] // 64)] for i in range(batch.bs)]
    for i in range(batch.bs):
        if n[i] % 64 == 0:
            lists[i].append(next(free))
    width = max(len(x) for x in lists)
    table = ints([x + [0] * (width - len(x)) for x in lists])
    locs = ints([lists[i][n[i] // 64] * 64 + n[i] % 64 for i in range(batch.bs)])
    k1, q1 = normal(8, batch.bs, 1, 576), normal(9, batch.bs, hq, 576)
    gpb.row_append(f, k1, None, pools[0], locs, rot, ints(n), q=q1)
    step = gpb.AttendPlan(f, hq, [1] * batch.bs, [x + 1 for x in n])
    o1, l1 = gpb.attend_paged(step, q1, pools[0], table, scale)
    pool = pools[0].view(torch.bfloat16)
    want = []
    for i in range(batch.bs):
        idx = torch.tensor([p * 64 + j for p in lists[i] for j in range(64)], device="cuda")
        keys, vals = split(f, pool[idx[:n[i] + 1]])
        want.append(attention(q1[i:i + 1], keys, vals, ints([n[i]]), 0, 0, scale))
    check(o1, l1, [torch.cat([w[j] for w in want]) for j in range(4)])
    with pytest.raises(ValueError):
        r.attend_plan(fmt("128"), 8)
