"""Rows held in e4m3 on the CPU: their formats, what is refused, the work lists
over them, and the reference that the GPU tests hold them to.  No call here
reaches a kernel launch."""
import ctypes

import numpy as np
import pytest
import torch

import gather_plan_build_amd as gpb
from gather_plan_build_amd import binding as B
from held_reference import LEAST, MOST, TOP, code_values, held_rows, hold, plain_rows
from test_rows_host import A, append_args, build

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


def latent(dtype="bf16", **kw):
    return gpb.RowFormat(dtype, 1, 576, 512, values_in_key=True, held="e4m3", **kw)


@pytest.mark.parametrize("args,latent_row,row_bytes,values", [
    ((1, 576, 512), True, 656, 576),
    ((1, 128, 128), True, 144, 128),
    ((8, 128, 128), False, 2064, 2048),
    ((8, 64, 64), False, 1040, 1024),
    ((1, 8, 8), False, 32, 16),
])
def test_sizes_of_rows(args, latent_row, row_bytes, values):
    f = gpb.RowFormat("bf16", *args, values_in_key=latent_row, held="e4m3")
    assert (f.row_bytes, f.values, f.c.dtype) == (row_bytes, values, B.BF16 | B.HELD_E4M3)
    g = gpb.RowFormat("bf16", *args, values_in_key=latent_row)
    assert (g.row_bytes, g.values, g.held) == (2 * values, values, None)
    with pytest.raises(ValueError):
        gpb.RowFormat("bf16", *args, values_in_key=latent_row, held="e5m2")


@pytest.mark.parametrize("args,code", [
    ((17, 2, 128, 128, 0, 528), B.OK),
    ((18, 2, 128, 128, 0, 528), B.OK),
    ((16, 2, 128, 128, 0, 528), B.EINVAL),
    ((19, 2, 128, 128, 0, 528), B.EINVAL),
    ((33, 2, 128, 128, 0, 528), B.EINVAL),
    ((17, 2, 128, 128, 0, 512), B.EINVAL),              # no room for the scales
    ((17, 2, 128, 128, 0, 520), B.EALIGN),
    ((17, 1, 576, 512, 1, 640), B.EINVAL),
    ((17, 1, 576, 512, 1, 656), B.OK),
    ((17, 2, 576, 512, 1, 2304), B.EINVAL),
    ((17, 1, 100, 128, 0, 512), B.EINVAL),
])
def test_formats(args, code):
    c = B.gpb_row_format(*args)
    f = gpb.RowFormat("bf16", args[1], args[2], args[3], values_in_key=args[4])
    a = append_args(f, n_rows=0, rot_dim=0)
    assert B.lib.gpb_row_append(ctypes.byref(c), ctypes.byref(a), None, None) == code
    shape = B.gpb_attend_shape(0, 4, 0, 0, 64, None, None, 0, None)
    assert B.lib.gpb_attend_plan_build(ctypes.byref(c), ctypes.byref(shape),
                                       ctypes.byref(B.gpb_attend_plan()), None, 0) == code
    assert B.lib.gpb_rows_read(ctypes.byref(c), A, 9, None, 0, A, 1 << 16, None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(d_k=None), B.EINVAL),
    (dict(d_v=None), B.EINVAL),
    (dict(d_pool=None, d_pool_locs=None, n_pool_rows=0, d_rows=None), B.EINVAL),
    (dict(n_pool_rows=1 << 31), B.ERANGE),
    (dict(n_rows=1 << 25), B.ERANGE),
    (dict(rot_start=104), B.EINVAL),
    (dict(d_k=A + 8), B.EALIGN),
    (dict(d_rows=A + 8), B.EALIGN),
    (dict(k_token_stride=260), B.EALIGN),
])
def test_append_refuses(kw, code):
    f = gpb.RowFormat("bf16", 2, 128, 128, held="e4m3")
    a = append_args(f, **kw)
    assert B.lib.gpb_row_append(ctypes.byref(f.c), ctypes.byref(a), None, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_rows=0), B.OK),
    (dict(n_rows=-1), B.EINVAL),
    (dict(n_src=-1), B.EINVAL),
    (dict(n_src=1 << 31), B.ERANGE),
    (dict(rows=None), B.EINVAL),
    (dict(out=None), B.EINVAL),
    (dict(locs=None, n_rows=10), B.EINVAL),
    (dict(rows=A + 8), B.EALIGN),
    (dict(out=A + 8), B.EALIGN),
    (dict(locs=A + 2), B.EALIGN),
    (dict(status=A + 1), B.EALIGN),
    (dict(out_bytes=1136), B.EINVAL),
    (dict(out_bytes=1160), B.EALIGN),
    (dict(out_bytes=-16), B.EINVAL),
    (dict(n_rows=2 ** 31 - 1, rows=A + 8), B.EALIGN),
])
def test_read_refuses(kw, code):
    f = latent()
    a = dict(rows=A, n_src=9, locs=A, n_rows=3, out=A, out_bytes=1152, status=None)
    a.update(kw)
    assert B.lib.gpb_rows_read(ctypes.byref(f.c), a["rows"], a["n_src"], a["locs"], a["n_rows"],
                               a["out"], a["out_bytes"], a["status"], None) == code


def test_read_refuses_plain_formats_and_none():
    f = gpb.RowFormat("bf16", 1, 576, 512, values_in_key=True)
    args = (A, 9, A, 3, A, 1152, None, None)
    assert B.lib.gpb_rows_read(ctypes.byref(f.c), *args) == B.EINVAL
    assert B.lib.gpb_rows_read(None, *args) == B.EINVAL
    with pytest.raises(ValueError):
        gpb.rows_read(f, torch.zeros(3, 1152, dtype=torch.uint8))
    with pytest.raises(ValueError):                    # host memory
        gpb.rows_read(latent(), torch.zeros(3, 656, dtype=torch.uint8))


@pytest.mark.parametrize("n,stride,locs,ok", [
    (3, 2 ** 30 - 8, None, True),                      # rows 2^31 - 16 bytes apart
    (3, 2 ** 30, None, False),
    (3, 2 ** 31 + 576, None, False),                   # 1,152 bytes in the low 32 bits
    (3, 2 ** 32 + 576, None, False),
    (1, 2 ** 31 + 576, None, True),                    # one row has no next one
    (3, 576, 3, True),
    (2 ** 31, 576, 2 ** 31, False),
    (2 ** 32 + 3, 576, 2 ** 32 + 3, False),            # 3 in the low 32 bits
])
def test_read_refuses_numbers_past_32_bits(monkeypatch, n, stride, locs, ok):
    """The C call takes the number of rows and their distance as int32.  (Tensors
    without memory, on a device that is not there.)"""
    class Here:
        used = None

        def __init__(self, *a):
            pass

        def __enter__(self):
            return None

        def __exit__(self, *a):
            pass

    calls = []
    monkeypatch.setattr(B, "_device_index", lambda t, what: 0)
    monkeypatch.setattr(B, "_same_device", lambda index, **tensors: None)
    monkeypatch.setattr(B, "_on", Here)
    monkeypatch.setattr(B.lib, "gpb_rows_read", lambda *a: calls.append(a) or B.OK)
    f = latent()
    rows = torch.empty(3, f.row_bytes, dtype=torch.uint8, device="meta")
    out = torch.empty_strided((n, 576), (stride, 1), dtype=f.dtype, device="meta")
    at = None if locs is None else torch.empty(locs, dtype=torch.int32, device="meta")
    if ok:
        gpb.rows_read(f, rows, at, n_rows=n, out=out)
        (_, _, n_src, _, n_rows, _, apart, _, _), = calls
        assert (n_src, n_rows, apart) == (3, n, 1152 if n == 1 else 2 * stride)
    else:
        with pytest.raises(ValueError, match="32 bits"):
            gpb.rows_read(f, rows, at, n_rows=n, out=out)
        assert not calls


@pytest.mark.parametrize("past", [2 ** 31, 2 ** 32 + 64, 2 ** 62, -2 ** 31 - 1])
def test_sizes_past_32_bits_are_refused(past):
    """They would reach the C call as their low 32 bits (2^32 + 64 as 64)."""
    wrong = [
        lambda: gpb.RowFormat("bf16", past, 64, 64),
        lambda: gpb.RowFormat("bf16", 1, past, 64, held="e4m3"),
        lambda: gpb.RowFormat("bf16", 1, 64, past, held="e4m3"),
        lambda: gpb.RowFormat("bf16", 1, 64, 64, row_bytes=past, held="e4m3"),
        lambda: gpb.Rotation(torch.ones(32), start=past),
    ]
    f = gpb.RowFormat("bf16", 1, 64, 64)
    wrong += [lambda: gpb.AttendPlan(f, past, [1], [1]),
              lambda: gpb.AttendPlan(f, 4, [1], [1], window=past),
              lambda: gpb.AttendPlan(f, 4, [1], [1], sinks=past),
              lambda: gpb.AttendPlan(f, 4, [1], [1], page_size=past)]
    if 0 < past < 2 ** 40:                     # (what a tensor can have)
        k = torch.empty(1, 1, 64, dtype=f.dtype, device="meta").expand(past, 1, 64)
        wrong.append(lambda: gpb.row_append(f, k, k, None, None, rows=k))
    for call in wrong:
        with pytest.raises(ValueError, match="32 bits"):
            call()


def test_a_call_of_another_format_is_refused():
    """The plan's format is the rows': their rows hold other bytes."""
    f = gpb.RowFormat("bf16", 2, 128, 128, held="e4m3")
    rc, plan, _ = build(f, 8, [3], [100])
    assert rc == B.OK and plan.format.dtype == 17 and plan.format.row_bytes == 528
    io = B.gpb_attend_io(A, 1024, 128, A, 1024, 128, None, 1.0)
    for dtype in (16, 19):
        plan.format.dtype = dtype
        assert B.lib.gpb_attend_dense(ctypes.byref(plan), A, ctypes.byref(io), A, 200, A, A,
                                      1 << 30, None, None) == B.EINVAL


@pytest.mark.parametrize("which", [64, 128, 576])
def test_every_row_sees_its_keys_once(which):
    """The list of a held format covers each (query row, key) that is seen once."""
    f = latent() if which == 576 else gpb.RowFormat("fp16", 2, which, which, held="e4m3")
    hq = 16 if which == 576 else 8
    rng = np.random.default_rng(which)
    for _ in range(20):
        bs = int(rng.integers(1, 6))
        q = rng.integers(0, 40, bs)
        kv = q + rng.integers(0, 3000, bs)
        rc, p, lst = build(f, hq, q, kv)
        assert rc == B.OK
        G = hq // f.n_kv_heads
        T = int(q.sum())
        pos = lst[p.positions_at:p.positions_at + T]
        times = np.zeros((f.n_kv_heads, T * G, int(kv.max()) + 1), np.int32)
        for it in lst[:p.joins_at].reshape(-1, 16):
            req, row0, n_rows, h, lo, hi, n_tiles, tile0, n_first, tile1, _, wide = it[:12]
            tile = 64 if wide else 32
            for v in range(n_tiles):
                t = tile0 + v if v < n_first else tile1 + v - n_first
                for m in range(row0, row0 + n_rows):
                    a, b = max(t * tile, lo), min((t + 1) * tile, hi, pos[m // G] + 1)
                    times[h, m, a:max(a, b)] += 1
        for m in range(T * G):
            assert (times[:, m, :pos[m // G] + 1] == 1).all()
            assert (times[:, m, pos[m // G] + 1:] == 0).all()


# ------------------------------------------------------------------ the reference

def test_codes_stand_for_what_torch_says():
    mine = code_values().float()
    theirs = torch.arange(256).to(torch.uint8).view(torch.float8_e4m3fn).float()
    assert torch.equal(torch.isnan(mine), torch.isnan(theirs))
    assert torch.equal(mine.nan_to_num(0.0), theirs.nan_to_num(0.0))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_what_is_held(dtype):
    """Off by half a step at most, of the type, and held again as it is."""
    dt = DT[dtype]
    g = torch.Generator().manual_seed(2)
    x = (torch.randn(3000, 32, generator=g).double() *
         2.0 ** torch.randint(-14, 14, (3000, 1), generator=g).double()).to(dt)
    x[5] = 0
    x[6, 3], x[7, 2], x[7, 3] = float("nan"), float("inf"), -float("inf")
    c, s = hold(x, dt)
    e = s.double()[:, None] - 127
    y = code_values()[c.long()] * 2.0 ** e
    want = x.double().clamp(-TOP[dt], TOP[dt])
    half = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** (e - 10))
    ok = ~torch.isnan(want)
    assert ((y - want).abs()[ok] <= half.expand_as(y)[ok]).all()
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert (s[5] == LEAST[dt] + 127) and (s[7] == MOST[dt] + 127)
    assert torch.equal(y.to(dt).double()[ok], y[ok])
    again = hold(y.to(dt), dt)[0]
    assert torch.equal(code_values()[again.long()][ok] * 2.0 ** (
        hold(y.to(dt), dt)[1].double()[:, None] - 127).expand_as(y)[ok], y[ok])
    # the cast of torch, at the same scales
    t = (want / 2.0 ** e).float().to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(t[ok], c[ok])


@pytest.mark.parametrize("f", [latent(), latent("fp16"),
                               gpb.RowFormat("bf16", 3, 64, 40, held="e4m3", row_bytes=352)])
def test_rows_of_the_reference(f):
    k = torch.randn(7, f.n_kv_heads, f.k_dim).to(f.dtype)
    v = None if f.values_in_key else torch.randn(7, f.n_kv_heads, f.v_dim).to(f.dtype)
    rows = held_rows(f, k, v)
    assert rows.shape == (7, f.row_bytes)
    x = plain_rows(f, rows)
    assert x.shape == (7, f.values)
    want = k.flatten(1) if v is None else torch.cat([k.flatten(1), v.flatten(1)], 1)
    assert ((x.double() - want.double()).abs() <= 0.07 * want.double().abs() + 0.02).all()
    if v is None:
        assert torch.equal(x[:, f.v_dim:], want[:, f.v_dim:])


def test_the_compose_counters_do_not_depend_on_row_kernels():
    """The digest that ties the compose's counters to its kernels leaves out each code
    object of kernels that make, read or attend rows."""
    import glob
    import os
    import re

    import bench
    src = os.path.join(os.path.dirname(B.__file__), "csrc")
    seen = 0
    for path in glob.glob(os.path.join(src, "*.hip")):
        with open(path) as f:
            text = f.read()
        if not re.search(r'#include "(held|append|attend_kernel)\.h"', text):
            continue
        text += open(os.path.join(src, "attend_kernel.h")).read() if "attend_kernel.h" in text else ""
        names = re.findall(r"__global__[^;{]*?\b(k_\w+)\(", text)
        assert names
        assert all(any(k.decode() in n for k in bench._OTHER_KERNELS) for n in names), names
        seen += 1
    assert seen >= 4
