"""The cache append and the attention over composed or paged rows, as cases to
measure: inputs, one pass in plain torch or through the package, the work a
pass cannot do without, and the exact results in 64 bits.

Three operators:

``append``  rows of a paged KV cache made from keys and values, with the keys
            (and the queries of the same tokens) rotated by their positions,
            on one axis or on several;
``dense``   ragged attention over the slot-dense buffer that the compose
            fills, causal, or with a sliding window and a few first tokens
            that stay visible;
``paged``   the attention of a decode step over the paged pool, where groups
            of requests may share their first pages and a window may apply.

A row is one token: ``hkv`` key heads of ``kd`` values, then ``hkv`` value
heads of ``vd`` values; with ``latent`` the row is one key head whose first
``vd`` values are the value.  A page holds 64 rows.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}

# Queries:keys of every request in the compose workloads' batches.
TINY = "100:292,37:357"
MEDIUM = "985:8153,574:6142,627:5299,537:3481"
TRACED = ("1407:29311,1577:22441,5883:22651,12652:21484,6864:16912,3:1347,4739:7171,"
          "151:663,2233:7929,1773:28461,6579:27891,739:30691")


# ---------------------------------------------------------------- cases

def listed():
    gqa128 = {"hkv": 8, "kd": 128, "vd": 128, "latent": False}
    gqa64 = {"hkv": 8, "kd": 64, "vd": 64, "latent": False}
    latent = {"hkv": 1, "kd": 576, "vd": 512, "latent": True}
    return [
        # one decode step's append, eight requests: latency
        dict(gqa128, name="append_step", op="append", dtype="bf16", hq=32, tokens=8,
             pages=64, start=0, rot=128, interleaved=False, sections="64",
             positions=8192, to_rows=False),
        # a prompt of images, video and text: three position axes; odd length
        dict(gqa128, name="append_axes", op="append", dtype="fp16", hq=28, hkv=4, tokens=4099,
             pages=160, start=0, rot=128, interleaved=False, sections="16,24,24",
             positions=32768, to_rows=False),
        # the traced prefill batch's current rows: to the pool and token-packed,
        # as the compose takes them; far positions
        dict(latent, name="append_traced", op="append", dtype="bf16", hq=16, tokens=44600,
             pages=1024, start=512, rot=64, interleaved=True, sections="32",
             positions=1000000, to_rows=True),
        # the tiny workload's batch: the smallest prefill
        dict(latent, name="dense_tiny", op="dense", dtype="bf16", hq=16, lens=TINY,
             window=0, sinks=0),
        # the medium workload's batch with grouped heads: an ordinary prefill
        dict(gqa128, name="dense_medium", op="dense", dtype="fp16", hq=32, lens=MEDIUM,
             window=0, sinks=0),
        # long chunks in a model of sliding windows with visible first tokens
        dict(gqa64, name="dense_window", op="dense", dtype="bf16", hq=64,
             lens="4096:4096,8192:12288,2047:30719,1:777,3001:3001", window=1024, sinks=4),
        # the traced workload's batch, the largest
        dict(latent, name="dense_traced", op="dense", dtype="bf16", hq=16, lens=TRACED,
             window=0, sinks=0),
        # one request decodes one token: latency
        dict(gqa128, name="paged_one", op="paged", dtype="bf16", hq=32, lens="1:737",
             groups="", window=0, sinks=0),
        # an ordinary ragged decode batch over latent rows
        dict(latent, name="paged_latent", op="paged", dtype="bf16", hq=16,
             lens=",".join("1:%d" % (613 + 241 * r) for r in range(32)),
             groups="", window=0, sinks=0),
        # long sequences, of which a window and the first tokens are read
        dict(gqa64, name="paged_window", op="paged", dtype="fp16", hq=64,
             lens=",".join("1:%d" % (40001 + 5003 * r) for r in range(8)),
             groups="", window=4096, sinks=4),
        # 48 requests after one long system prompt
        dict(gqa128, name="paged_shared", op="paged", dtype="bf16", hq=32,
             lens=",".join("1:%d" % (16384 + 37 + 19 * r) for r in range(48)),
             groups="0:48:16384", window=0, sinks=0),
        # two shared documents, some requests alone, two tokens a step (drafts)
        dict(latent, name="paged_shared_latent", op="paged", dtype="fp16", hq=16,
             lens=",".join("2:%d" % n for n in
                           [32768 + 101 + 67 * r for r in range(40)]
                           + [8192 + 3 + 129 * r for r in range(16)] + [950, 4001, 77, 2600]),
             groups="0:40:32768,40:16:8192", window=0, sinks=0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = rng.choice([
        {"hkv": rng.choice([1, 2, 4, 8]), "kd": 128, "vd": 128, "latent": False},
        {"hkv": rng.choice([1, 2, 4, 8]), "kd": 64, "vd": 64, "latent": False},
        {"hkv": 1, "kd": 576, "vd": 512, "latent": True}])
    c = dict(c, op=rng.choice(["append", "dense", "paged"]), dtype=rng.choice(["bf16", "fp16"]))
    c["hq"] = rng.choice([8, 16, 32]) if c["latent"] else c["hkv"] * rng.choice([1, 3, 4, 7, 8])
    if c["op"] == "append":
        c["tokens"] = _spread(rng, 1, 20000)
        c["pages"] = c["tokens"] // PAGE + 2 + _spread(rng, 1, 200)
        c["rot"] = 64 if c["kd"] != 128 else rng.choice([32, 64, 128])
        c["start"] = c["kd"] - c["rot"] if c["latent"] else 0
        c["interleaved"] = rng.choice([False, True])
        half = c["rot"] // 2
        if rng.random() < 0.4:
            a, b = sorted(rng.sample(range(1, half), 2))
            c["sections"] = "%d,%d,%d" % (a, b - a, half - b)
        else:
            c["sections"] = str(half)
        c["positions"] = _spread(rng, 100, 1000000)
        c["to_rows"] = rng.choice([False, True])
        return c
    c["window"] = rng.choice([0, 0, _spread(rng, 16, 4096)])
    c["sinks"] = rng.randrange(0, 9) if c["window"] else 0
    lens, groups = [], []
    if c["op"] == "dense":
        for _ in range(rng.randrange(1, 9)):
            q = 0 if lens and rng.random() < 0.1 else _spread(rng, 1, 3000)
            lens.append((q, PAGE * rng.choice([0, rng.randrange(0, 150)]) + q))
    else:
        while len(lens) < rng.randrange(1, 40):
            q, n = rng.choice([1, 1, 1, 2, 4]), rng.choice([1, rng.randrange(1, 24)])
            shared = 0
            if n > 1 and not c["window"]:
                shared = PAGE * _spread(rng, 1, 300)
                groups.append("%d:%d:%d" % (len(lens), n, shared))
            lens += [(q, shared + q + _spread(rng, 1, 4000)) for _ in range(n)]
    c["lens"] = ",".join("%d:%d" % x for x in lens)
    if c["op"] == "paged":
        c["groups"] = ",".join(groups)
    return c


def _lens(case):
    return [tuple(int(x) for x in p.split(":")) for p in case["lens"].split(",")]


def _groups(case):
    return [tuple(int(x) for x in p.split(":")) for p in case["groups"].split(",") if p]


def _sections(case):
    return [int(x) for x in case["sections"].split(",")]


def _row_values(case):
    return case["hkv"] * (case["kd"] + (0 if case["latent"] else case["vd"]))


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]
    hq, hkv, kd, vd, w = case["hq"], case["hkv"], case["kd"], case["vd"], _row_values(case)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    st = {"case": case}
    if case["op"] == "append":
        t, rot = case["tokens"], case["rot"]
        st["k"] = normal(t, hkv, kd)
        st["v"] = None if case["latent"] else normal(t, hkv, vd)
        st["q"] = normal(t, hq, kd)
        st["q_out"] = torch.empty_like(st["q"])
        st["pool"] = torch.zeros(case["pages"] * PAGE, w, device="cuda", dtype=dt)
        st["rows"] = torch.empty(t, w, device="cuda", dtype=dt) if case["to_rows"] else None
        pages = rng.permutation(np.arange(1, case["pages"]))[:-(-t // PAGE)]
        at = np.arange(t)
        st["pool_locs"] = ints(pages[at // PAGE] * PAGE + at % PAGE)
        n = len(_sections(case))
        st["positions"] = ints(rng.integers(0, case["positions"], size=(n, t)))
        freq = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
        st["inv_freq"] = torch.from_numpy(freq.astype(np.float32)).cuda()
        if own:
            import gather_plan_build_amd as gpb
            st["fmt"] = gpb.RowFormat(case["dtype"], hkv, kd, vd, values_in_key=case["latent"])
            st["rotation"] = gpb.Rotation(st["inv_freq"], start=case["start"],
                                          interleaved=case["interleaved"],
                                          sections=_sections(case))
        return st
    lens = _lens(case)
    tokens = sum(q for q, _ in lens)
    st["q"] = normal(tokens, hq, kd)
    st["scale"] = 1.0 / math.sqrt(192 if case["latent"] else kd)
    need = [-(-n // PAGE) for _, n in lens]
    if case["op"] == "dense":
        base = np.concatenate([[0], np.cumsum(need)[:-1]]) * PAGE
        st["dense"] = normal(sum(need) * PAGE, w)
        for (_, n), b, p in zip(lens, base, need):
            st["dense"][b + n:b + p * PAGE] = 0   # the tail rows the compose leaves zero
        st["k_bases"] = ints(base)
    else:
        owner = {}
        for first, count, shared in _groups(case):
            for r in range(first + 1, first + count):
                owner[r] = (first, shared // PAGE)
        own_pages = sum(n - owner.get(r, (0, 0))[1] for r, n in enumerate(need))
        ids = iter(rng.permutation(np.arange(1, own_pages + 9)))
        table = np.zeros((len(lens), max(need)), dtype=np.int32)
        for r, n in enumerate(need):
            first, s = owner.get(r, (0, 0))
            table[r, :s] = table[first, :s]
            table[r, s:n] = [next(ids) for _ in range(n - s)]
        st["pool"] = normal((own_pages + 9) * PAGE, w)
        st["table"] = ints(table)
    if own:
        import gather_plan_build_amd as gpb
        fmt = gpb.RowFormat(case["dtype"], hkv, kd, vd, values_in_key=case["latent"])
        st["plan"] = gpb.AttendPlan(fmt, hq, [q for q, _ in lens], [n for _, n in lens],
                                    window=case["window"], sinks=case["sinks"],
                                    page_size=PAGE,
                                    groups=_groups(case) if case["op"] == "paged" else ())
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    case = st["case"]
    if own:
        import gather_plan_build_amd as gpb
        if case["op"] == "append":
            gpb.row_append(st["fmt"], st["k"], st["v"], st["pool"], st["pool_locs"],
                           st["rotation"], st["positions"], rows=st["rows"],
                           q=st["q"], q_out=st["q_out"])
            return {"pool": st["pool"], "rows": st["rows"], "q": st["q_out"]}
        if case["op"] == "dense":
            out, lse = gpb.attend_dense(st["plan"], st["q"], st["dense"], st["k_bases"],
                                        st["scale"])
        else:
            out, lse = gpb.attend_paged(st["plan"], st["q"], st["pool"], st["table"],
                                        st["scale"])
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        return _plain_append(st)
    return _plain_attend(st)


def _plain_append(st):
    case = st["case"]
    dt = st["k"].dtype
    axis = [a for a, n in enumerate(_sections(case)) for _ in range(n)]
    # angles of far positions lose their fraction in 32 bits
    angle = st["positions"][axis].double().t() * st["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def rotated(x):
        y = x.float()
        a, b = case["start"], case["start"] + case["rot"]
        part = y[..., a:b]
        if case["interleaved"]:
            p, q = part[..., 0::2], part[..., 1::2]
            new = torch.stack([p * cos - q * sin, q * cos + p * sin], dim=-1).flatten(-2)
        else:
            p, q = part.chunk(2, dim=-1)
            new = torch.cat([p * cos - q * sin, q * cos + p * sin], dim=-1)
        return torch.cat([y[..., :a], new, y[..., b:]], dim=-1).to(dt)

    rows = rotated(st["k"]).flatten(1)
    if st["v"] is not None:
        rows = torch.cat([rows, st["v"].flatten(1)], dim=1)
    st["pool"].index_copy_(0, st["pool_locs"].long(), rows)
    if st["rows"] is not None:
        st["rows"].copy_(rows)
    st["q_out"].copy_(rotated(st["q"]))
    return {"pool": st["pool"], "rows": st["rows"], "q": st["q_out"]}


def _visible(case, qpos, kpos):
    """Key position visible from query position, for broadcast tensors."""
    ok = kpos <= qpos
    if case["window"]:
        ok = ok & ((qpos - kpos < case["window"]) | (kpos < case["sinks"]))
    return ok


def _request_rows(st, r, n):
    """The rows of request r's n keys, in sequence order."""
    if st["case"]["op"] == "dense":
        lens = _lens(st["case"])
        base = PAGE * sum(-(-k // PAGE) for _, k in lens[:r])
        return st["dense"][base:base + n]
    pages = st["table"][r, :-(-n // PAGE)].long()
    at = pages[:, None] * PAGE + torch.arange(PAGE, device="cuda")
    return st["pool"][at.flatten()[:n]]


def _plain_attend(st):
    case, q = st["case"], st["q"]
    hq, hkv, kd, vd = case["hq"], case["hkv"], case["kd"], case["vd"]
    out = torch.empty(q.shape[0], hq, vd, device="cuda", dtype=q.dtype)
    lse = torch.empty(q.shape[0], hq, device="cuda", dtype=torch.float32)
    t0 = 0
    for r, (nq, nk) in enumerate(_lens(case)):
        if nq == 0:
            continue
        rows = _request_rows(st, r, nk)
        step = max(1, (1 << 28) // (hq * nk))
        for a in range(0, nq, step):
            b = min(nq, a + step)
            lo, hi = 0, nk - nq + b          # keys that any of these queries sees
            picks = torch.arange(lo, hi, device="cuda")
            if case["window"]:
                first = max(0, nk - nq + a - case["window"] + 1)
                if first > case["sinks"]:
                    picks = torch.cat([picks[:case["sinks"]], picks[first:]])
            part = rows[picks].float()
            k = part[:, :hkv * kd].view(-1, hkv, kd).permute(1, 2, 0).contiguous()
            v = (part[:, :vd] if case["latent"] else part[:, hkv * kd:]).reshape(-1, hkv, vd)
            v = v.permute(1, 0, 2).contiguous()
            x = q[t0 + a:t0 + b].float().view(b - a, hkv, hq // hkv, kd)
            x = x.permute(1, 2, 0, 3).reshape(hkv, -1, kd)
            s = torch.matmul(x, k).mul_(st["scale"]).view(hkv, hq // hkv, b - a, -1)
            qpos = torch.arange(nk - nq + a, nk - nq + b, device="cuda")[:, None]
            s.masked_fill_(~_visible(case, qpos, picks[None, :]), -math.inf)
            top = s.amax(dim=-1, keepdim=True)
            p = s.sub_(top).exp_()
            total = p.sum(dim=-1, keepdim=True)
            y = torch.matmul(p.view(hkv, -1, p.shape[-1]), v).view(hkv, hq // hkv, b - a, vd)
            y = y / total
            out[t0 + a:t0 + b] = y.permute(2, 0, 1, 3).reshape(b - a, hq, vd).to(q.dtype)
            lse[t0 + a:t0 + b] = (top + total.log())[..., 0].permute(2, 0, 1).reshape(b - a, hq)
        t0 += nq
    return {"out": out, "lse": lse}


# ---------------------------------------------------------------- work and exact results

def _sees(case, p):
    """How many keys a query at position p sees."""
    w = case["window"]
    if p < 0:
        return 0
    if not w or p < w:
        return p + 1
    return w + min(case["sinks"], p + 1 - w)


def work(case):
    w, hq = 2 * _row_values(case), case["hq"]
    if case["op"] == "append":
        t = case["tokens"]
        qb = 2 * hq * case["kd"]
        out = t * w * (2 if case["to_rows"] else 1)
        return {"bytes": t * (w + 2 * qb) + out + 4 * t * (1 + len(_sections(case))),
                "flops": 3 * t * case["rot"] * (hq + case["hkv"])}
    lens = _lens(case)
    seen = sum(_sees(case, p) for q, n in lens for p in range(n - q, n))
    keys = 0
    for q, n in lens:
        if q:
            far = max(0, n - q - case["window"] + 1) if case["window"] else 0
            keys += n - far + min(far, case["sinks"])
    if case["op"] == "paged":
        keys -= sum((count - 1) * shared for _, count, shared in _groups(case))
    tokens = sum(q for q, _ in lens)
    return {"bytes": keys * w + tokens * hq * (2 * case["kd"] + 2 * case["vd"] + 4),
            "flops": 2 * seen * hq * (case["kd"] + case["vd"])}


def exact(case, seed):
    st = prepare(case, seed)
    return _exact_append(st) if case["op"] == "append" else _exact_attend(st)


def _exact_append(st):
    """Every rotated pair as a complex number times exp(i angle)."""
    case = st["case"]
    sec, half, a = _sections(case), case["rot"] // 2, case["start"]
    ends = np.cumsum(sec)
    turn = torch.empty(case["tokens"], half, dtype=torch.complex128, device="cuda")
    for i in range(half):
        pos = st["positions"][int(np.searchsorted(ends, i, side="right"))].double()
        x = pos * st["inv_freq"][i].double()
        turn[:, i] = torch.complex(x.cos(), x.sin())

    def spin(x):
        y = x.double().clone()
        one = [a + (2 * i if case["interleaved"] else i) for i in range(half)]
        two = [j + (1 if case["interleaved"] else half) for j in one]
        z = torch.complex(y[:, :, one], y[:, :, two]) * turn[:, None, :]
        y[:, :, one], y[:, :, two] = z.real, z.imag
        return y

    t = case["tokens"]
    rows = torch.zeros(t, _row_values(case), dtype=torch.float64, device="cuda")
    k = spin(st["k"]).reshape(t, -1)
    rows[:, :k.shape[1]] = k
    if st["v"] is not None:
        rows[:, k.shape[1]:] = st["v"].double().reshape(t, -1)
    pool = st["pool"].double()
    pool[st["pool_locs"].long()] = rows
    return {"pool": pool, "rows": rows if case["to_rows"] else None, "q": spin(st["q"])}


def _exact_attend(st):
    """Head by head: log of the sum of exp over the visible keys, then the
    weights exp(s - lse) on the values."""
    case, q = st["case"], st["q"]
    hq, hkv, kd, vd = case["hq"], case["hkv"], case["kd"], case["vd"]
    out = torch.zeros(q.shape[0], hq, vd, dtype=torch.float64, device="cuda")
    lse = torch.full((q.shape[0], hq), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for r, (nq, nk) in enumerate(_lens(case)):
        rows = _request_rows(st, r, nk) if nq else None
        step = max(1, (1 << 27) // max(nk, 1))
        for h in range(hq if nq else 0):
            g = h // (hq // hkv)
            k = rows[:, g * kd:(g + 1) * kd].double()
            off = 0 if case["latent"] else hkv * kd + g * vd
            v = rows[:, off:off + vd].double()
            for a in range(0, nq, step):
                b = min(nq, a + step)
                last = nk - nq + b
                near = max(0, nk - nq + a + 1 - case["window"]) if case["window"] else 0
                near = near if near > case["sinks"] else 0
                at = torch.cat([torch.arange(case["sinks"] if near else 0),
                                torch.arange(near, last)]).cuda()
                s = q[t0 + a:t0 + b, h].double() @ k[at].t().contiguous() * st["scale"]
                back = torch.arange(nk - nq + a, last, device="cuda")[:, None] - at
                hide = back < 0
                if case["window"]:
                    hide |= (back >= case["window"]) & (at >= case["sinks"])
                s[hide] = -math.inf
                z = torch.logsumexp(s, dim=1)
                lse[t0 + a:t0 + b, h] = z
                out[t0 + a:t0 + b, h] = torch.exp(s - z[:, None]) @ v[at]
        t0 += nq
    return {"out": out, "lse": lse}
