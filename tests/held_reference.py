"""Plain 64-bit reference of rows held in e4m3: what is held of values, the bytes
of a held row, and what its bytes stand for."""
import torch

LEAST = {torch.bfloat16: -100, torch.float16: -15}
MOST = {torch.bfloat16: 120, torch.float16: 8}
TOP = {torch.bfloat16: 240.0 * 2.0 ** 120, torch.float16: 240.0 * 2.0 ** 8}


def power(e):
    """2^e, of whole e, exactly (float64; the library's pow is off by a last place
    on some devices)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def code_values():
    """What the 256 codes stand for, at scale 1 (float64)."""
    out = []
    for c in range(128):
        e, m = c >> 3, c & 7
        out.append(float("nan") if c == 127 else m / 8 * 2.0 ** -6 if e == 0 else
                   (1 + m / 8) * 2.0 ** (e - 7))
    return torch.tensor(out + [-x for x in out], dtype=torch.float64)


def nearest_codes(y):
    """The codes of y (float64, |y| <= 448 or NaN): the nearest value, of two as near
    the one whose code is even."""
    table = code_values()[:127].to(y.device)
    a = y.abs().nan_to_num(0.0)
    hi = torch.searchsorted(table, a.contiguous()).clamp(max=126)      # table[hi] >= a
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - a, a - table[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = torch.where(torch.isnan(y), torch.full_like(code, 127), code)
    return (code + 128 * torch.signbit(y).long()).to(torch.uint8)


def exponents(x, dtype):
    """The scale's exponent of heads x [..., values] (float64)."""
    top = x.abs().nan_to_num(nan=0.0, posinf=TOP[dtype]).clamp(max=TOP[dtype]).amax(-1)
    e = torch.full(top.shape, LEAST[dtype], dtype=torch.int64, device=x.device)
    for n in range(LEAST[dtype], MOST[dtype]):
        e += top > 448.0 * 2.0 ** n
    return e


def hold(x, dtype):
    """Codes (uint8) and scale bytes of heads x [..., values]."""
    x = x.double()
    e = exponents(x, dtype)
    y = torch.where(torch.isnan(x), x, x.clamp(-TOP[dtype], TOP[dtype]))
    return nearest_codes(y / power(e)[..., None]), (e + 127).to(torch.uint8)


def held_rows(f, keys, values):
    """Rows [n, f.row_bytes] (uint8) of keys [n, hkv, k_dim] and values [n, hkv,
    v_dim] (None: in the key), the bytes behind a row's payload zero."""
    n = keys.shape[0]
    parts = []
    if f.values_in_key:
        c, s = hold(keys[:, 0, :f.v_dim], f.dtype)
        rest = keys[:, 0, f.v_dim:].to(f.dtype).contiguous()
        parts = [c, rest.view(torch.uint8).reshape(n, 2 * (f.k_dim - f.v_dim)), s[:, None]]
    else:
        (kc, ks), (vc, vs) = hold(keys, f.dtype), hold(values, f.dtype)
        parts = [kc.flatten(1), vc.flatten(1), ks, vs]
    out = torch.cat(parts, 1)
    return torch.nn.functional.pad(out, (0, f.row_bytes - out.shape[1]))


def plain_rows(f, rows):
    """What held rows [n, f.row_bytes] stand for: [n, f.values] of f.dtype."""
    table = code_values().to(rows.device)

    def value(codes, scales, dim):
        s = power(scales.long() - 127)
        return (table[codes.long()].unflatten(1, (-1, dim)) * s[..., None]).flatten(1)

    h, kd, vd = f.n_kv_heads, f.k_dim, f.v_dim
    if f.values_in_key:
        at = vd + 2 * (kd - vd)
        rest = rows[:, vd:at].contiguous().view(f.dtype).double().reshape(len(rows), kd - vd)
        x = torch.cat([value(rows[:, :vd], rows[:, at:at + 1], vd), rest], 1)
    else:
        at = h * (kd + vd)
        x = torch.cat([value(rows[:, :h * kd], rows[:, at:at + h], kd),
                       value(rows[:, h * kd:at], rows[:, at + h:at + 2 * h], vd)], 1)
    out = x.to(f.dtype)
    same = (out.double() == x) | torch.isnan(x)
    assert same.all(), "a held value that its type does not have"
    return out
