"""The row append and the attentions on the CPU: what they refuse, and what the
work list covers.  No call here reaches a kernel launch."""
import ctypes

import numpy as np
import pytest
import torch

import gather_plan_build_amd as gpb
from gather_plan_build_amd import binding as B
import rows_list

A = 0x100000  # an address that is never dereferenced


def fmt(which="128", dtype="bf16", hkv=2, **kw):
    if which == "latent":
        return gpb.RowFormat(dtype, 1, 576, 512, values_in_key=True, **kw)
    return gpb.RowFormat(dtype, hkv, int(which), int(which), **kw)


def build(f, hq, q, kv, window=0, sinks=0, page=64, groups=()):
    q, kv, g = (np.asarray(x, np.int32).reshape(-1) for x in (q, kv, list(groups)))
    shape = B.gpb_attend_shape(q.size, hq, window, sinks, page,
                               q.ctypes.data if q.size else None,
                               kv.ctypes.data if kv.size else None, g.size // 3,
                               g.ctypes.data if g.size else None)
    plan = B.gpb_attend_plan()
    rc = B.lib.gpb_attend_plan_build(ctypes.byref(f.c), ctypes.byref(shape), ctypes.byref(plan),
                                     None, 0)
    if rc != B.OK:
        return rc, None, None
    out = np.full(plan.list_ints + 4, -7, np.int32)
    rc = B.lib.gpb_attend_plan_build(ctypes.byref(f.c), ctypes.byref(shape), ctypes.byref(plan),
                                     out.ctypes.data, plan.list_ints)
    assert (out[plan.list_ints:] == -7).all()
    return rc, plan, out[:plan.list_ints]


def test_strerror_names_the_new_status():
    assert "unknown" not in gpb.strerror(B.ENOMEM)


# ------------------------------------------------------------------ append

def append_args(f, **kw):
    a = B.gpb_append()
    a.n_rows, a.n_q_heads = 3, 4
    a.d_k, a.d_v, a.d_pool, a.d_pool_locs, a.d_rows = A, A, A, A, A
    a.n_pool_rows = 64
    a.k_token_stride = a.v_token_stride = f.n_kv_heads * f.k_dim
    a.k_head_stride = a.v_head_stride = f.k_dim
    a.d_q = a.d_q_out = A
    a.q_token_stride = a.qo_token_stride = 4 * f.k_dim
    a.q_head_stride = a.qo_head_stride = f.k_dim
    a.rot_dim, a.n_axes, a.d_inv_freq, a.d_positions = 32, 1, A, A
    a.section[0] = 16
    for k, v in kw.items():
        if k == "section":
            for i, x in enumerate(v):
                a.section[i] = x
        else:
            setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(n_rows=0), B.OK),
    (dict(n_rows=-1), B.EINVAL),
    (dict(d_k=None), B.EINVAL),
    (dict(d_v=None), B.EINVAL),
    (dict(d_pool=None), B.EINVAL),                      # locations without a pool
    (dict(d_pool_locs=None), B.EINVAL),
    (dict(d_pool=None, d_pool_locs=None, n_pool_rows=0, d_rows=None), B.EINVAL),
    (dict(n_pool_rows=-1), B.EINVAL),
    (dict(n_pool_rows=1 << 31), B.ERANGE),
    (dict(d_q_out=None), B.EINVAL),
    (dict(n_q_heads=0), B.EINVAL),
    (dict(n_q_heads=1 << 20), B.EINVAL),
    (dict(rot_dim=24), B.EINVAL),
    (dict(rot_dim=1024), B.EINVAL),
    (dict(rot_start=4), B.EINVAL),
    (dict(rot_start=104), B.EINVAL),                    # past the head's end
    (dict(interleaved=2), B.EINVAL),
    (dict(n_axes=0), B.EINVAL),
    (dict(n_axes=5), B.EINVAL),
    (dict(n_axes=2, section=[20, -4]), B.EINVAL),
    (dict(section=[15]), B.EINVAL),
    (dict(d_inv_freq=None), B.EINVAL),
    (dict(d_positions=None), B.EINVAL),
    (dict(qo_token_stride=1024), B.EINVAL),             # in place with other strides
    (dict(d_k=A + 8), B.EALIGN),
    (dict(d_q=A + 2), B.EALIGN),
    (dict(d_pool_locs=A + 2), B.EALIGN),
    (dict(k_token_stride=260), B.EALIGN),
    (dict(v_head_stride=4), B.EALIGN),
])
def test_append_refuses(kw, code):
    f = fmt()
    a = append_args(f, **kw)
    assert B.lib.gpb_row_append(ctypes.byref(f.c), ctypes.byref(a), None, None) == code


@pytest.mark.parametrize("args,code", [
    ((3, 1, 128, 128, 0, 512), B.EINVAL),
    ((1, 0, 128, 128, 0, 512), B.EINVAL),
    ((1, 1, 100, 128, 0, 512), B.EINVAL),
    ((1, 1, 128, 2048, 0, 8192), B.EINVAL),
    ((1, 1, 128, 128, 0, 496), B.EINVAL),               # rows shorter than their payload
    ((1, 1, 128, 128, 0, 520), B.EALIGN),
    ((1, 2, 576, 512, 1, 2304), B.EINVAL),              # a latent row has one head
    ((1, 1, 512, 576, 1, 1152), B.EINVAL),
    ((1, 1, 576, 512, 2, 1152), B.EINVAL),
])
def test_row_formats_refused(args, code):
    c = B.gpb_row_format(*args)
    a = append_args(fmt())
    assert B.lib.gpb_row_append(ctypes.byref(c), ctypes.byref(a), None, None) == code
    shape = B.gpb_attend_shape(0, 4, 0, 0, 64, None, None, 0, None)
    assert B.lib.gpb_attend_plan_build(ctypes.byref(c), ctypes.byref(shape),
                                       ctypes.byref(B.gpb_attend_plan()), None, 0) == code


def test_append_refuses_null_structs():
    f, a = fmt(), append_args(fmt())
    assert B.lib.gpb_row_append(None, ctypes.byref(a), None, None) == B.EINVAL
    assert B.lib.gpb_row_append(ctypes.byref(f.c), None, None, None) == B.EINVAL


# ------------------------------------------------------------------ work list

@pytest.mark.parametrize("kw", [
    dict(hq=3), dict(hq=0), dict(q=[-1]), dict(kv=[-1]), dict(window=-1), dict(sinks=-1),
    dict(page=0), dict(groups=[(0, 2, 64)]), dict(groups=[(0, 1, 63)]), dict(groups=[(0, 1, 0)]),
    dict(groups=[(-1, 1, 64)]), dict(groups=[(0, 0, 64)]), dict(groups=[(0, 1, 128)]),
])
def test_work_list_refuses(kw):
    base = dict(hq=4, q=[5], kv=[100])
    base.update(kw)
    assert build(fmt(), **base)[0] == B.EINVAL


def test_work_list_refuses_overlapping_groups_and_other_formats():
    q, kv = [1, 1, 1], [200, 200, 200]
    assert build(fmt(), 4, q, kv, groups=[(0, 2, 64), (1, 2, 64)])[0] == B.EINVAL
    assert build(fmt(), 4, q, kv, groups=[(1, 2, 64), (0, 1, 64)])[0] == B.EINVAL
    assert build(fmt(), 4, q, kv, groups=[(0, 2, 64), (2, 1, 64)])[0] == B.OK
    assert build(gpb.RowFormat("bf16", 2, 96, 96), 4, q, kv)[0] == B.EINVAL
    assert build(gpb.RowFormat("bf16", 2, 128, 64), 4, q, kv)[0] == B.EINVAL
    assert build(fmt(), 65536, [1 << 20], [1 << 20])[0] == B.ERANGE


def test_a_list_too_small_is_refused():
    f = fmt()
    q, kv = np.asarray([5], np.int32), np.asarray([100], np.int32)
    shape = B.gpb_attend_shape(1, 4, 0, 0, 64, q.ctypes.data, kv.ctypes.data, 0, None)
    plan, out = B.gpb_attend_plan(), np.zeros(8, np.int32)
    assert B.lib.gpb_attend_plan_build(ctypes.byref(f.c), ctypes.byref(shape),
                                       ctypes.byref(plan), out.ctypes.data, 8) == B.ERANGE
    assert (out == 0).all()


def covered(f, hq, q, kv, window, sinks, page, groups):
    """Run the work list in numpy: how often every (row, key) is added, and by
    which way a row's results come out."""
    rc, p, lst = build(f, hq, q, kv, window, sinks, page, groups)
    assert rc == B.OK
    G, hkv = hq // f.n_kv_heads, f.n_kv_heads
    latent = f.values_in_key
    T = int(np.sum(q))
    pos = lst[p.positions_at:p.positions_at + T]
    req = np.repeat(np.arange(len(q)), q)
    want_pos = np.concatenate([kv[r] - q[r] + np.arange(q[r]) for r in range(len(q))] or [[]])
    assert np.array_equal(pos, want_pos)
    keys = max(kv) if len(kv) else 0
    times = np.zeros((hkv, T * G, keys + 1), np.int32)
    direct = np.zeros((hkv, T * G), np.int32)
    held = {}
    source = {}
    for first, n, shared in groups:
        for r in range(first, first + n):
            source[r] = (first, shared)
    for it in lst[:p.joins_at].reshape(-1, 16):
        (r, row0, n_rows, h, lo, hi, n_tiles, tile0, n_first, tile1, partial, wide, pmin,
         pmax) = it[:14]
        tile = 64 if wide else 32
        assert 1 <= n_rows <= (64 if latent else 256 if wide else 32)
        assert row0 + n_rows <= T * G
        toks = np.arange(row0, row0 + n_rows) // G
        assert pmin == pos[toks].min() and pmax == pos[toks].max()
        seen = set()
        for v in range(n_tiles):
            t = tile0 + v if v < n_first else tile1 + v - n_first
            assert t not in seen
            seen.add(t)
            ks = np.arange(max(t * tile, lo), min((t + 1) * tile, hi))
            for m in range(n_rows):
                tok = toks[m]
                home = source.get(req[tok], (req[tok], 0))
                assert r == req[tok] or (r == home[0] and hi <= home[1])
                x = pos[tok]
                see = (ks <= x) if not window else \
                    (ks <= x) & ((x - ks < window) | (ks < sinks))
                times[h, row0 + m, ks[see]] += 1
        if partial < 0:
            direct[h, row0:row0 + n_rows] += 1
        else:
            for m in range(n_rows):
                assert partial + m not in held
                held[partial + m] = (h, row0 + m)
    assert len(held) == p.n_partial_rows and (not held or max(held) == len(held) - 1)
    refs = lst[p.refs_at:p.positions_at]
    used = np.zeros(len(held), np.int32)
    for j in lst[p.joins_at:p.refs_at].reshape(-1, 8):
        row0, n_rows, h, ref0, n_refs = j[:5]
        assert 1 <= n_rows <= 32 and row0 // G == (row0 + n_rows - 1) // G
        direct[h, row0:row0 + n_rows] += 1
        for x in refs[ref0:ref0 + n_refs]:
            for m in range(n_rows):
                assert held[x + m] == (h, row0 + m)
                used[x + m] += 1
    assert (used == 1).all() and (direct == 1).all()
    for t in range(T):
        x = want_pos[t]
        ks = np.arange(keys + 1)
        see = (ks <= x) & (ks < kv[req[t]])
        if window:
            see &= (x - ks < window) | (ks < sinks)
        assert np.array_equal(times[:, t * G:(t + 1) * G],
                              np.broadcast_to(see, (hkv, G, keys + 1)).astype(np.int32)), t


@pytest.mark.parametrize("which,hkv,hq", [("64", 2, 14), ("128", 1, 3), ("128", 1, 130),
                                          ("latent", 1, 16), ("latent", 1, 100)])
@pytest.mark.parametrize("q,kv,window,sinks,page,groups", [
    ([1], [1], 0, 0, 64, ()),
    ([0, 3], [0, 2], 0, 0, 64, ()),                       # a query before its first key
    ([5, 0, 40], [5, 9, 700], 0, 0, 64, ()),
    ([7, 33], [900, 33], 50, 3, 64, ()),
    ([2, 1], [2000, 130], 1, 0, 64, ()),
    ([1, 1], [1500, 3], 64, 64, 64, ()),
    ([3], [400], 10, 1000, 64, ()),                       # more first tokens than keys
    ([1, 2, 1, 1], [330, 420, 301, 55], 0, 0, 10, [(0, 3, 300)]),
    ([1, 1, 1], [1025, 1100, 1024 + 64], 100, 5, 64, [(0, 2, 1024), (2, 1, 64)]),
    ([0, 0, 1], [64, 64, 70], 0, 0, 64, [(0, 2, 64)]),
])
def test_work_list_covers_every_visible_key_once(which, hkv, hq, q, kv, window, sinks, page,
                                                 groups):
    covered(fmt(which, hkv=hkv), hq, q, kv, window, sinks, page, groups)


def test_work_lists_of_random_batches():
    rng = np.random.default_rng(3)
    for _ in range(40):
        bs = int(rng.integers(1, 6))
        q = rng.integers(0, 12, bs)
        kv = np.maximum(rng.integers(0, 900, bs), 0)
        window = int(rng.choice([0, 1, 33, 200]))
        groups = []
        if rng.random() < 0.5 and bs > 1:
            kv[:2] = np.maximum(kv[:2], 96 + q[:2])
            groups = [(0, 2, 32 * int(rng.integers(1, 4)))]
        which = ["64", "128", "latent"][int(rng.integers(0, 3))]
        hkv = 1 if which == "latent" else int(rng.integers(1, 3))
        covered(fmt(which, hkv=hkv), hkv * int(rng.integers(1, 9)), list(q), list(kv), window,
                int(rng.integers(0, 9)), 32, groups)


# ------------------------------------------------------------------ attend

def attend_args(paged=False, q=(5,), kv=(100,), groups=(), **kw):
    f = fmt()
    rc, plan, _ = build(f, 4, list(q), list(kv), groups=groups)
    assert rc == B.OK
    io = B.gpb_attend_io(A, 512, 128, A, 512, 128, A, 0.1)
    d = dict(plan=ctypes.byref(plan), list=A, rows=A, n_rows=1000, pages=A, n_listed=64, base=A,
             stride=0, ws=A, ws_bytes=1 << 30, status=None)
    for k, v in kw.items():
        if k in d:
            d[k] = v
        elif hasattr(plan, k):
            setattr(plan, k, v)
        else:
            setattr(io, k, v)
    if d["plan"] is not None:
        d["plan"] = ctypes.byref(plan)
    if paged:
        return B.lib.gpb_attend_paged(d["plan"], d["list"], ctypes.byref(io), d["rows"],
                                      d["n_rows"], d["pages"], d["n_listed"], d["base"],
                                      d["stride"], d["ws"], d["ws_bytes"], d["status"], None)
    return B.lib.gpb_attend_dense(d["plan"], d["list"], ctypes.byref(io), d["rows"],
                                  d["n_rows"], d["base"], d["ws"], d["ws_bytes"], d["status"],
                                  None)


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(q=(0,), list=None), B.OK),                     # no query: nothing to launch
    (dict(plan=None), B.EINVAL),
    (dict(list=None), B.EINVAL),
    (dict(d_q=None), B.EINVAL),
    (dict(d_out=None), B.EINVAL),
    (dict(rows=None), B.EINVAL),
    (dict(n_rows=0), B.EINVAL),
    (dict(n_rows=-1), B.EINVAL),
    (dict(n_rows=1 << 31), B.ERANGE),
    (dict(scale=0.0), B.EINVAL),
    (dict(scale=-1.0), B.EINVAL),
    (dict(scale=float("nan")), B.EINVAL),
    (dict(scale=float("inf")), B.EINVAL),
    (dict(kv=(4000,), ws_bytes=16), B.EINVAL),
    (dict(kv=(4000,), ws=None), B.EINVAL),
    (dict(n_items=3), B.EINVAL),                         # not what the builder filled
    (dict(positions_at=0), B.EINVAL),
    (dict(n_heads=5), B.EINVAL),
    (dict(workspace_bytes=4), B.EINVAL),
    (dict(list=A + 4), B.EALIGN),
    (dict(d_q=A + 8), B.EALIGN),
    (dict(q_head_stride=100), B.EALIGN),
    (dict(out_token_stride=2), B.EALIGN),
    (dict(d_out=A + 4), B.EALIGN),
    (dict(rows=A + 8), B.EALIGN),
    (dict(status=A + 2), B.EALIGN),
])
def test_attend_refuses(paged, kw, code):
    assert attend_args(paged, **kw) == code


def test_attend_refuses_what_only_one_of_them_takes():
    # the dense buffer keeps every request's keys: no groups
    assert attend_args(False, q=(1, 1), kv=(100, 100), groups=[(0, 2, 64)]) == B.EINVAL
    assert attend_args(False, base=None) == B.EINVAL
    assert attend_args(True, pages=None) == B.EINVAL
    assert attend_args(True, n_listed=0) == B.EINVAL
    assert attend_args(True, n_rows=63) == B.EINVAL                    # no whole page
    assert attend_args(True, base=None, stride=1) == B.EINVAL          # 100 keys, 64 a page
    assert attend_args(True, base=None, stride=65) == B.EINVAL         # longer than the list
    assert attend_args(True, base=None, stride=-1) == B.EINVAL


def test_binding_refuses_before_the_library():
    f = fmt()
    with pytest.raises(ValueError):
        gpb.RowFormat("fp32", 1, 64, 64)
    with pytest.raises(ValueError):
        gpb.Rotation(torch.ones(16, dtype=torch.float64))
    with pytest.raises(ValueError):
        gpb.Rotation(torch.ones(16), sections=[8, 4])
    with pytest.raises(ValueError):
        gpb.Rotation(torch.ones(16), sections=[4, 4, 4, 2, 2])
    with pytest.raises(ValueError):
        gpb.AttendPlan(f, 4, [1, 2], [3])
    with pytest.raises(ValueError):
        gpb.AttendPlan(f, 4, [1], [3], device="cpu")
    with pytest.raises(gpb.GpbError):
        gpb.AttendPlan(f, 3, [1], [3])
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                       # host memory
        gpb.row_append(f, k, k, torch.zeros(64, 512, dtype=torch.bfloat16),
                       torch.zeros(3, dtype=torch.int32))


@pytest.mark.parametrize("kw", [
    dict(rot_start=2 ** 31 - 8),
    dict(d_q=A, d_q_out=2 * A, qo_head_stride=64),       # heads of 128 values on each other
    dict(d_q=A, d_q_out=2 * A, qo_token_stride=0),
    dict(d_q=A, d_q_out=2 * A, qo_token_stride=256),
    dict(q_token_stride=0, qo_token_stride=0),           # in place on one token's queries
    dict(d_q=A, d_q_out=2 * A, qo_token_stride=-512),
])
def test_append_refuses_results_that_share_a_place(kw):
    a = append_args(fmt(), **kw)
    assert B.lib.gpb_row_append(ctypes.byref(fmt().c), ctypes.byref(a), None, None) == B.EINVAL


def test_append_refuses_more_rows_than_a_launch_holds():
    a = append_args(fmt(), n_rows=1 << 24)
    assert B.lib.gpb_row_append(ctypes.byref(fmt().c), ctypes.byref(a), None, None) == B.ERANGE


@pytest.mark.parametrize("paged", [False, True])
@pytest.mark.parametrize("kw", [dict(out_head_stride=64), dict(out_token_stride=0),
                                dict(out_token_stride=508), dict(out_token_stride=-512),
                                dict(out_head_stride=1 << 62, out_token_stride=64)])
def test_attend_refuses_results_that_share_a_place(paged, kw):
    assert attend_args(paged, **kw) == B.EINVAL


def test_work_list_of_more_queries_than_a_list_holds_is_refused():
    n = 2 ** 31 - 1
    assert build(fmt(), 4, [n] * 5, [n] * 5)[0] == B.ERANGE
    assert build(fmt(), 65536, [n], [5])[0] == B.ERANGE


# ------------------------------------------------------------------ what the kernels make of a list

@pytest.fixture(scope="module")
def check_lists(tmp_path_factory):
    return rows_list.library(tmp_path_factory.mktemp("lists"))


def grouped_batches(seed, n):
    """Random batches whose first requests share keys, with windows and first
    tokens and pages that end anywhere in a tile."""
    rng = np.random.default_rng(seed)
    for _ in range(n):
        bs = int(rng.integers(1, 6))
        q = rng.integers(0, rng.choice([3, 12, 60]), bs)
        kv = rng.integers(0, rng.choice([80, 400, 1500]), bs)
        page = int(rng.choice([1, 3, 8, 16, 32, 50, 64]))
        groups = []
        if bs > 1 and rng.random() < 0.8:
            n_g = int(rng.integers(2, bs + 1))
            shared = page * int(rng.integers(1, 2 + rng.choice([40, 300]) // page))
            kv[:n_g] = shared + q[:n_g] + rng.integers(0, rng.choice([2, 20, 100]), n_g)
            groups = [(0, n_g, shared)]
        window = int(rng.choice([0, 1, 5, 12, 33, 200]))
        sinks = int(rng.choice([0, 1, 4, 17, 40, 1000]))
        which = str(rng.choice(["64", "128", "latent"]))
        hkv = 1 if which == "latent" else int(rng.integers(1, 3))
        yield (fmt(which, hkv=hkv), hkv * int(rng.choice([1, 4, 7, 16, 40])), list(q), list(kv),
               window, sinks, page, groups)


BEHIND_THE_WINDOW = [       # shared keys that the window hides but for the first tokens
    (("128", 1), 4, [1, 1], [60, 60], 12, 4, 16, [(0, 2, 48)]),
    (("64", 1), 4, [1, 1], [1020, 1018], 8, 4, 16, [(0, 2, 1008)]),
]


@pytest.mark.parametrize("f,hq,q,kv,window,sinks,page,groups", BEHIND_THE_WINDOW)
def test_items_of_shared_keys_behind_the_window_are_taken(check_lists, f, hq, q, kv, window,
                                                          sinks, page, groups):
    rc, plan, lst = build(fmt(f[0], hkv=f[1]), hq, q, kv, window, sinks, page, groups)
    assert rc == B.OK
    assert rows_list.outcome(check_lists.list_items_fit, plan, lst) == (0, -1)
    covered(fmt(f[0], hkv=f[1]), hq, q, kv, window, sinks, page, groups)


def test_every_item_of_random_batches_is_taken(check_lists):
    for case in grouped_batches(5, 4000):
        rc, plan, lst = build(*case)
        assert rc == B.OK
        assert rows_list.outcome(check_lists.list_items_fit, plan, lst) == (0, -1), case[1:]
    for case in grouped_batches(6, 60):
        covered(*case)


def test_keys_of_items_behind_the_window_are_seen(check_lists):
    # keys 17 .. 31 of the one tile are past the shared keys, 4 .. 15 seen by no query
    rc, plan, lst = build(fmt("64", hkv=1), 4, [1, 1], [20, 20], 3, 4, 8, [(0, 2, 16)])
    assert rc == B.OK
    assert rows_list.outcome(check_lists.list_keys_seen, plan, lst) == (0, -1)


def test_only_keys_that_a_query_sees_are_read(check_lists):
    for case in grouped_batches(7, 4000):
        rc, plan, lst = build(*case)
        assert rc == B.OK
        assert rows_list.outcome(check_lists.list_keys_seen, plan, lst) == (0, -1), case[1:]


def test_a_plans_list_is_recorded_on_the_stream_that_reads_it(monkeypatch):
    """The allocator must not hand the list's memory out while a stream other
    than the one it was made on may still read it."""
    import contextlib
    from types import SimpleNamespace

    seen = []
    f = fmt()
    plan = gpb.AttendPlan.__new__(gpb.AttendPlan)
    plan.fmt, plan.n_heads, plan.n_tokens, plan.workspace_bytes = f, 4, 3, 0
    plan.device = torch.device("cuda", 0)
    plan.list, plan.list_stream = SimpleNamespace(record_stream=seen.append), 77

    def on(index, stream):
        c = contextlib.nullcontext(stream.cuda_stream)
        c.raw, c.used, c.other = stream.cuda_stream, stream, stream
        return c

    monkeypatch.setattr(B, "_on", on)
    monkeypatch.setattr(B, "_same_device", lambda *a, **kw: None)
    q, out = (torch.zeros(3, 4, 128, dtype=torch.bfloat16) for _ in range(2))
    for raw in (5, 77):
        stream = SimpleNamespace(cuda_stream=raw, stream_id=3)
        B._attend(plan, q, 0.1, out, None, None, None, stream, lambda *a: B.OK, "attend")
        assert seen == ([stream] if raw == 5 else []), raw
        seen.clear()


@pytest.mark.parametrize("paged", [False, True])
def test_a_plan_with_queries_and_no_requests_is_refused(paged):
    for kw in (dict(), dict(base=None, stride=2)):
        assert attend_args(paged, bs=0, **kw) == B.EINVAL
