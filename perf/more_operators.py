"""The cache held in 8 bits, as cases to measure: rows quantised as they are
written, rows read back, and the attention that reads them where they are;
inputs, one pass in plain torch or through the package, the work a pass cannot
do without, and the exact results in 64 bits.

Three operators:

``append``  rows of a paged KV cache made from keys and values, keys (and the
            queries of the same tokens) rotated by their positions, the rows
            held in e4m3 with one power of two as the scale of a head's values;
``read``    such rows back as rows of the type they were made from;
``attend``  attention over such rows where they lie, in the paged pool or in
            the slot-dense buffer that the compose fills: of chunks of new
            tokens, causal or with a sliding window and a few first tokens that
            stay visible, and of decode steps, where groups of requests may
            share their first pages.

A held row is one token: ``hkv`` key heads of ``kd`` codes of a byte, ``hkv``
value heads of ``vd`` codes, then a byte a head for the scales, keys' first.
With ``latent`` it is one head: ``vd`` codes, which are the value and the key's
first part, then the key's other ``kd - vd`` values in 16 bits, then one scale.
A code stands for code * 2^(scale - 127), the scale being the smallest with
which no value of the head passes 448.  A row takes whole 16 bytes, a page holds
64 rows.
"""
import math

import numpy as np
import torch

own = False

PAGE = 64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
# Least and largest exponent of a scale, and the largest value that is held: all
# that is held stands for a value of the type.
LEAST = {"bf16": -100, "fp16": -15}
MOST = {"bf16": 120, "fp16": 8}
TOP = {"bf16": 240.0 * 2.0 ** 120, "fp16": 240.0 * 2.0 ** 8}

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
        dict(gqa64, name="append_axes", op="append", dtype="fp16", hq=28, hkv=4, tokens=4099,
             pages=160, start=0, rot=64, interleaved=False, sections="8,12,12",
             positions=32768, to_rows=False),
        # the traced prefill batch's current rows: to the pool and token-packed,
        # as the compose takes them; far positions
        dict(latent, name="append_traced", op="append", dtype="bf16", hq=16, tokens=44600,
             pages=1024, start=512, rot=64, interleaved=True, sections="32",
             positions=1000000, to_rows=True),
        # some rows out of the pool, padded entries among them: a short prefix
        # handed to code that knows plain rows
        dict(gqa64, name="read_some", op="read", dtype="fp16", rows=777, pages=64, at="pool"),
        # the traced batch's whole dense buffer
        dict(latent, name="read_dense", op="read", dtype="bf16", rows=217280, pages=3395,
             at="all"),
        # the tiny workload's batch: the smallest chunks
        dict(latent, name="chunk_tiny", op="attend", source="pool", dtype="bf16", hq=16,
             lens=TINY, groups="", window=0, sinks=0),
        # the medium workload's chunks with grouped heads: ordinary ones
        dict(gqa128, name="chunk_medium", op="attend", source="pool", dtype="fp16", hq=32,
             lens=MEDIUM, groups="", window=0, sinks=0),
        # long chunks in a model of sliding windows with visible first tokens,
        # from the dense buffer
        dict(gqa64, name="chunk_window", op="attend", source="dense", dtype="bf16", hq=64,
             lens="4096:4096,8192:12288,2047:30719,1:777,3001:3001", groups="", window=1024,
             sinks=4),
        # the traced workload's batch, the largest
        dict(latent, name="chunk_traced", op="attend", source="pool", dtype="bf16", hq=16,
             lens=TRACED, groups="", window=0, sinks=0),
        # one request decodes one token: latency
        dict(gqa128, name="step_one", op="attend", source="pool", dtype="bf16", hq=32,
             lens="1:737", groups="", window=0, sinks=0),
        # an ordinary ragged decode batch over latent rows
        dict(latent, name="step_ragged", op="attend", source="pool", dtype="fp16", hq=16,
             lens=",".join("1:%d" % (613 + 241 * r) for r in range(32)),
             groups="", window=0, sinks=0),
        # 48 requests after one long system prompt
        dict(gqa128, name="step_shared", op="attend", source="pool", dtype="bf16", hq=32,
             lens=",".join("1:%d" % (16384 + 37 + 19 * r) for r in range(48)),
             groups="0:48:16384", window=0, sinks=0),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = rng.choice([
        {"hkv": rng.choice([1, 2, 4, 8]), "kd": 128, "vd": 128, "latent": False},
        {"hkv": rng.choice([1, 2, 4, 8]), "kd": 64, "vd": 64, "latent": False},
        {"hkv": 1, "kd": 576, "vd": 512, "latent": True}])
    c = dict(c, op=rng.choice(["append", "read", "attend", "attend"]),
             dtype=rng.choice(["bf16", "fp16"]))
    if c["op"] == "read":
        c["rows"] = _spread(rng, 1, 100000)
        c["at"] = rng.choice(["pool", "all"])
        c["pages"] = c["rows"] // PAGE + 2 + _spread(rng, 1, 200)
        return c
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
    c["source"] = rng.choice(["pool", "pool", "dense"])
    lens, groups = [], []
    if c["source"] == "dense" or rng.random() < 0.5:      # chunks of new tokens
        for _ in range(rng.randrange(1, 9)):
            q = 0 if lens and rng.random() < 0.1 else _spread(rng, 1, 3000)
            lens.append((q, PAGE * rng.choice([0, rng.randrange(0, 150)]) + q))
    else:                                                 # a decode step
        while len(lens) < rng.randrange(1, 40):
            q, n = rng.choice([1, 1, 1, 2, 4]), rng.choice([1, rng.randrange(1, 24)])
            shared = 0
            if n > 1 and not c["window"]:
                shared = PAGE * _spread(rng, 1, 300)
                groups.append("%d:%d:%d" % (len(lens), n, shared))
            lens += [(q, shared + q + _spread(rng, 1, 4000)) for _ in range(n)]
    c["lens"] = ",".join("%d:%d" % x for x in lens)
    c["groups"] = ",".join(groups)
    return c


def _lens(case):
    return [tuple(int(x) for x in p.split(":")) for p in case["lens"].split(",")]


def _groups(case):
    return [tuple(int(x) for x in p.split(":")) for p in case["groups"].split(",") if p]


def _sections(case):
    return [int(x) for x in case["sections"].split(",")]


def _values(case):
    """Values of a row in 16 bits."""
    return case["hkv"] * (case["kd"] + (0 if case["latent"] else case["vd"]))


def _layout(case):
    """Bytes of a held row: where the codes end, where the plain values end, where
    the scales end, and where the next row begins."""
    if case["latent"]:
        codes = case["vd"]
        plain = codes + 2 * (case["kd"] - case["vd"])
        scales = plain + 1
    else:
        codes = plain = _values(case)
        scales = plain + 2 * case["hkv"]
    return codes, plain, scales, -(-scales // 16) * 16


# ---------------------------------------------------------------- held rows, plainly

def _held(case, x):
    """Codes (e4m3) and biased exponents (uint8) of x [..., heads, values]."""
    name = case["dtype"]
    x = x.clamp(-TOP[name], TOP[name])
    share, power = torch.frexp(x.abs().amax(-1))
    # amax = share 2^power; the least e with amax <= 448 2^e, 448 being 0.875 2^9
    e = power - torch.where(share <= 0.875, 9, 8)
    e = torch.where(share > 0, e, LEAST[name]).clamp(LEAST[name], MOST[name])
    codes = torch.ldexp(x, -e[..., None]).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8)


def _hold_rows(case, k, v):
    """Held rows [n, row bytes] of keys [n, hkv, kd] and values (None: in the key)."""
    n, dt = k.shape[0], DTYPES[case["dtype"]]
    codes_end, plain_end, scales_end, row = _layout(case)
    out = torch.zeros(n, row, dtype=torch.uint8, device=k.device)
    if case["latent"]:
        codes, e = _held(case, k[..., :case["vd"]])
        out[:, codes_end:plain_end] = k[:, 0, case["vd"]:].to(dt).contiguous().view(torch.uint8)
    else:
        held = [_held(case, x) for x in (k, v)]
        codes = torch.cat([c.view(torch.uint8).flatten(1) for c, _ in held], 1)
        e = torch.cat([e for _, e in held], 1)
    out[:, :codes_end] = codes.view(torch.uint8).flatten(1)
    out[:, plain_end:scales_end] = e.flatten(1)
    return out


def _values_of(case, rows):
    """What held rows stand for, in 32 bits: keys [n, hkv, kd], values [n, hkv, vd]."""
    codes_end, plain_end, scales_end, _ = _layout(case)
    x = rows[:, :codes_end].view(torch.float8_e4m3fn).float()
    e = rows[:, plain_end:scales_end].int() - 127
    hkv, kd, vd = case["hkv"], case["kd"], case["vd"]
    if case["latent"]:
        v = torch.ldexp(x, e)[:, None, :]
        rest = rows[:, codes_end:plain_end].view(DTYPES[case["dtype"]]).float()
        return torch.cat([v, rest[:, None, :]], -1), v
    k = torch.ldexp(x[:, :hkv * kd].unflatten(1, (hkv, kd)), e[:, :hkv, None])
    v = torch.ldexp(x[:, hkv * kd:].unflatten(1, (hkv, vd)), e[:, hkv:, None])
    return k, v


def _parts(case, rows):
    """Held rows as an output: codes, scales and plain values, each as the numbers
    that its bytes are."""
    codes_end, plain_end, scales_end, _ = _layout(case)
    out = {"codes": rows[:, :codes_end].view(torch.float8_e4m3fn),
           "scales": rows[:, plain_end:scales_end].view(torch.float8_e8m0fnu)}
    if case["latent"]:
        out["plain"] = rows[:, codes_end:plain_end].view(DTYPES[case["dtype"]])
    return out


# ---------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rng = np.random.default_rng(seed)
    dt = DTYPES[case["dtype"]]
    hkv, kd, vd = case["hkv"], case["kd"], case["vd"]
    row = _layout(case)[3]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=dt)

    def ints(a):
        return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()

    def held_rows(n):
        """Rows as an append leaves them, a token's values larger or smaller."""
        out = torch.empty(n, row, dtype=torch.uint8, device="cuda")
        for a in range(0, n, 1 << 17):
            b = min(n, a + (1 << 17))
            size = torch.exp2(0.5 * torch.randn(b - a, 1, 1, generator=g, device="cuda"))
            k = (normal(b - a, hkv, kd).float() * size).to(dt)
            v = None if case["latent"] else (normal(b - a, hkv, vd).float() * size).to(dt)
            out[a:b] = _hold_rows(case, k.float(), None if v is None else v.float())
        return out

    st = {"case": case}
    if own:
        import gather_plan_build_amd as gpb
        st["fmt"] = gpb.RowFormat(case["dtype"], hkv, kd, vd, values_in_key=case["latent"],
                                  held="e4m3")
    if case["op"] == "append":
        t, rot, hq = case["tokens"], case["rot"], case["hq"]
        _, plain_end, scales_end, _ = _layout(case)
        st["k"] = normal(t, hkv, kd)
        st["v"] = None if case["latent"] else normal(t, hkv, vd)
        st["q"] = normal(t, hq, kd)
        st["q_out"] = torch.empty_like(st["q"])
        st["pool"] = torch.zeros(case["pages"] * PAGE, row, device="cuda", dtype=torch.uint8)
        st["pool"][:, plain_end:scales_end] = 127   # rows of zeros, their scale 1
        st["rows"] = st["pool"][:t].clone() if case["to_rows"] else None
        pages = rng.permutation(np.arange(1, case["pages"]))[:-(-t // PAGE)]
        at = np.arange(t)
        st["pool_locs"] = ints(pages[at // PAGE] * PAGE + at % PAGE)
        n = len(_sections(case))
        st["positions"] = ints(rng.integers(0, case["positions"], size=(n, t)))
        freq = 10000.0 ** (-np.arange(0, rot, 2, dtype=np.float64) / rot)
        st["inv_freq"] = torch.from_numpy(freq.astype(np.float32)).cuda()
        if own:
            st["rotation"] = gpb.Rotation(st["inv_freq"], start=case["start"],
                                          interleaved=case["interleaved"],
                                          sections=_sections(case))
        return st
    if case["op"] == "read":
        st["pool"] = held_rows(case["pages"] * PAGE)
        st["locs"] = None
        if case["at"] == "pool":
            at = rng.integers(0, case["pages"] * PAGE, size=case["rows"])
            at[rng.random(case["rows"]) < 0.02] = -1      # padded entries
            st["locs"] = ints(at)
        st["out"] = torch.empty(case["rows"], _values(case), dtype=dt, device="cuda")
        return st
    lens = _lens(case)
    tokens = sum(q for q, _ in lens)
    st["q"] = normal(tokens, case["hq"], kd)
    st["scale"] = 1.0 / math.sqrt(192 if case["latent"] else kd)
    need = [-(-n // PAGE) for _, n in lens]
    if case["source"] == "dense":
        base = np.concatenate([[0], np.cumsum(need)[:-1]]) * PAGE
        st["dense"] = held_rows(sum(need) * PAGE)
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
        st["pool"] = held_rows((own_pages + 9) * PAGE)
        st["table"] = ints(table)
    if own:
        st["plan"] = gpb.AttendPlan(st["fmt"], case["hq"], [q for q, _ in lens],
                                    [n for _, n in lens], window=case["window"],
                                    sinks=case["sinks"], page_size=PAGE, groups=_groups(case))
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
        elif case["op"] == "read":
            gpb.rows_read(st["fmt"], st["pool"], st["locs"], n_rows=case["rows"],
                          out=st["out"])
        else:
            if case["source"] == "dense":
                out, lse = gpb.attend_dense(st["plan"], st["q"], st["dense"], st["k_bases"],
                                            st["scale"])
            else:
                out, lse = gpb.attend_paged(st["plan"], st["q"], st["pool"], st["table"],
                                            st["scale"])
            return {"out": out, "lse": lse}
    elif case["op"] == "append":
        _plain_append(st)
    elif case["op"] == "read":
        _plain_read(st)
    else:
        return _plain_attend(st)
    if case["op"] == "read":
        return st["out"]
    rows = None if st["rows"] is None else _parts(case, st["rows"])
    return {"pool": _parts(case, st["pool"]), "rows": rows, "q": st["q_out"]}


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
        return torch.cat([y[..., :a], new, y[..., b:]], dim=-1)

    rows = _hold_rows(case, rotated(st["k"]), None if st["v"] is None else st["v"].float())
    st["pool"].index_copy_(0, st["pool_locs"].long(), rows)
    if st["rows"] is not None:
        st["rows"].copy_(rows)
    st["q_out"].copy_(rotated(st["q"]).to(dt))


def _plain_read(st):
    case, rows = st["case"], st["pool"][:st["case"]["rows"]]
    if st["locs"] is not None:
        rows = st["pool"][st["locs"].long().clamp(min=0)]
    k, v = _values_of(case, rows)
    x = k.flatten(1) if case["latent"] else torch.cat([k.flatten(1), v.flatten(1)], 1)
    if st["locs"] is not None:
        x = x.masked_fill((st["locs"] < 0)[:, None], 0.0)
    st["out"].copy_(x)


def _visible(case, qpos, kpos):
    """Key position visible from query position, for broadcast tensors."""
    ok = kpos <= qpos
    if case["window"]:
        ok = ok & ((qpos - kpos < case["window"]) | (kpos < case["sinks"]))
    return ok


def _request_rows(st, r, n):
    """The held rows of request r's n keys, in sequence order."""
    if st["case"]["source"] == "dense":
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
            k, v = _values_of(case, rows[picks])
            k, v = k.permute(1, 2, 0).contiguous(), v.permute(1, 0, 2).contiguous()
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
    plain, held = 2 * _values(case), _layout(case)[2]
    if case["op"] == "read":
        return {"bytes": case["rows"] * (held + plain + (4 if case["at"] == "pool" else 0)),
                "flops": case["rows"] * _values(case)}
    hq = case["hq"]
    if case["op"] == "append":
        t = case["tokens"]
        qb = 2 * hq * case["kd"]
        out = t * held * (2 if case["to_rows"] else 1)
        return {"bytes": t * (plain + 2 * qb) + out + 4 * t * (1 + len(_sections(case))),
                "flops": 3 * t * case["rot"] * (hq + case["hkv"]) + 2 * t * _values(case)}
    lens = _lens(case)
    seen = sum(_sees(case, p) for q, n in lens for p in range(n - q, n))
    keys = 0
    for q, n in lens:
        if q:
            far = max(0, n - q - case["window"] + 1) if case["window"] else 0
            keys += n - far + min(far, case["sinks"])
    keys -= sum((count - 1) * shared for _, count, shared in _groups(case))
    tokens = sum(q for q, _ in lens)
    return {"bytes": keys * held + tokens * hq * (2 * case["kd"] + 2 * case["vd"] + 4),
            "flops": 2 * seen * hq * (case["kd"] + case["vd"])}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st)
    if case["op"] == "read":
        return _exact_read(st)
    return _exact_attend(st)


def _byte_values():
    """What each of the 256 codes stands for: sign, four bits of exponent, three of
    fraction."""
    c = torch.arange(256)
    power, part = (c >> 3) & 15, (c & 7).double() / 8
    x = torch.where(power > 0, (1 + part) * 2.0 ** (power - 7).double(), part * 2.0 ** -6)
    x[(c & 127) == 127] = math.nan
    return torch.where(c >= 128, -x, x).cuda()


def _exact_rows(case, rows):
    """Values of a held row [n, values], in 64 bits."""
    codes_end, plain_end, scales_end, _ = _layout(case)
    x = _byte_values()[rows[:, :codes_end].long()]
    s = 2.0 ** (rows[:, plain_end:scales_end].double() - 127)
    if case["latent"]:
        plain = rows[:, codes_end:plain_end].view(DTYPES[case["dtype"]]).double()
        return torch.cat([x * s, plain], 1)
    k = case["hkv"] * case["kd"]
    s = torch.cat([s[:, :case["hkv"]].repeat_interleave(case["kd"], 1),
                   s[:, case["hkv"]:].repeat_interleave(case["vd"], 1)], 1)
    assert k + case["hkv"] * case["vd"] == x.shape[1]
    return x * s


def _exact_read(st):
    case = st["case"]
    x = _exact_rows(case, st["pool"])
    if st["locs"] is None:
        return x[:case["rows"]]
    x = torch.cat([x, torch.zeros_like(x[:1])])        # its last row is a padded entry's
    return x[st["locs"].long()]


def _exact_append(st):
    """Every rotated pair as a complex number times exp(i angle); every value to the
    nearest multiple of its step."""
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

    def coded(x):
        name = case["dtype"]
        x = torch.minimum(torch.maximum(x, -torch.full_like(x, TOP[name])),
                          torch.full_like(x, TOP[name]))
        e = torch.ceil(torch.log2(x.abs().amax(-1) / 448.0)).clamp(LEAST[name], MOST[name])
        y = x / torch.exp2(e)[..., None]
        step = torch.exp2(torch.floor(torch.log2(y.abs())).clamp(min=-6.0) - 3.0)
        return torch.round(y / step) * step, torch.exp2(e)

    t = case["tokens"]
    k = spin(st["k"])
    if case["latent"]:
        codes, scales = coded(k[:, :, :case["vd"]])
        parts = {"codes": codes.flatten(1), "scales": scales, "plain": k[:, 0, case["vd"]:]}
    else:
        both = [coded(k), coded(st["v"].double())]
        parts = {"codes": torch.cat([c.flatten(1) for c, _ in both], 1),
                 "scales": torch.cat([s for _, s in both], 1)}
    at = st["pool_locs"].long()
    pool = {}
    for name, x in parts.items():
        pool[name] = torch.full((case["pages"] * PAGE, x.shape[1]), float(name == "scales"),
                                dtype=torch.float64, device="cuda")
        pool[name][at] = x
    assert t == at.numel()
    return {"pool": pool, "rows": parts if case["to_rows"] else None, "q": spin(st["q"])}


def _exact_attend(st):
    """Head by head: log of the sum of exp over the visible keys, then the
    weights exp(s - lse) on the values."""
    case, q = st["case"], st["q"]
    hq, hkv, kd, vd = case["hq"], case["hkv"], case["kd"], case["vd"]
    out = torch.zeros(q.shape[0], hq, vd, dtype=torch.float64, device="cuda")
    lse = torch.full((q.shape[0], hq), -math.inf, dtype=torch.float64, device="cuda")
    t0 = 0
    for r, (nq, nk) in enumerate(_lens(case)):
        rows = _exact_rows(case, _request_rows(st, r, nk)) if nq else None
        step = max(1, (1 << 27) // max(nk, 1))
        for h in range(hq if nq else 0):
            g = h // (hq // hkv)
            k = rows[:, g * kd:(g + 1) * kd]
            off = 0 if case["latent"] else hkv * kd + g * vd
            v = rows[:, off:off + vd]
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
