"""The attention sub-block's operators in binary64, from their formulas, on
whatever device the inputs live on; with each result a bound on the error of a
kernel that works in binary32 and rounds as the header says (u32, ut and tiny
as in sublayer_ref.py, whose check() takes both).
"""
import math

import torch

from sublayer_ref import TINY, U32, UT, check, rounded  # noqa: F401

# pi to 200 bits, from Machin's formula in integers
_BITS = 200


def _arctan_inverse(n):
    one = 1 << (_BITS + 20)
    total, term, k = 0, one // n, 1
    while term:
        total += term // k if k % 4 == 1 else -(term // k)
        term //= n * n
        k += 2
    return total


PI = 4 * (4 * _arctan_inverse(5) - _arctan_inverse(239)) >> 20  # times 2^200


def turns(inv_freq):
    """inv_freq / (2 pi) modulo 1 times 2^64, exactly rounded down, for each."""
    out = []
    for f in inv_freq:
        num, den = float(f).as_integer_ratio()
        out.append((num << (_BITS + 64)) // (2 * PI * den) % (1 << 64))
    return out


def angles(positions, inv_freq):
    """Radians in [-pi, pi) [tokens, pairs], from integers: positions as far
    as they like."""
    wide = 1 << 128
    full = []
    for f in inv_freq:
        num, den = float(f).as_integer_ratio()
        full.append((num << (_BITS + 128)) // (2 * PI * den))
    rows = []
    for p in positions:
        row = []
        for t in full:
            x = int(p) * t % wide
            row.append((x - wide if x >= wide // 2 else x) / wide * 2 * math.pi)
        rows.append(row)
    return torch.tensor(rows, dtype=torch.float64).view(len(rows), len(full))


def _pairs(x, rot, interleaved):
    if interleaved:
        return x[..., 0:rot:2], x[..., 1:rot:2]
    return x[..., :rot // 2], x[..., rot // 2:rot]


def _join(a, b, rest, interleaved):
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, rest], -1)


def rotate(x, angle, rot, interleaved, back=False):
    """The rotation of x [tokens, heads, dim] and, element by element, the sum
    of the magnitudes of its terms and of those with sine and cosine 1."""
    if rot == 0:
        return x, x.abs(), torch.zeros_like(x)
    c, s = torch.cos(angle)[:, None].to(x.device), torch.sin(angle)[:, None].to(x.device)
    if back:
        s = -s
    a, b = _pairs(x, rot, interleaved)
    rest = x[..., rot:]
    both = a.abs() + b.abs()
    return (_join(a * c - b * s, b * c + a * s, rest, interleaved),
            _join((a * c).abs() + (b * s).abs(), (b * c).abs() + (a * s).abs(), rest.abs(), interleaved),
            _join(both, both, torch.zeros_like(rest), interleaved))


def angle_error(positions):
    """Of a cosine or sine in the kernels: the turns are off by 2^-64 at most,
    the angle within a quarter turn by 2^-24 pi / 4, sincospi by 2 ulp, and
    the product with a weight by one rounding: per position."""
    p = torch.as_tensor([abs(float(x)) for x in positions], dtype=torch.float64)
    return (2 * math.pi * 2.0 ** -64 * p + 2.0 ** -24 * math.pi / 4 + 5 * U32)[:, None, None]


def _weight(w, dim, like):
    return torch.ones(dim, dtype=torch.float64, device=like.device) if w is None else w.double()


def head_norm(x, w, angle, positions, rot, interleaved, eps):
    """(value, bound) of the rotated norm of x [tokens, heads, dim]."""
    x, w = x.double(), _weight(w, x.shape[2], x)
    d = x.shape[2]
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    y, terms, ones = rotate(x * w, angle, rot, interleaved)
    # mean: chains of 8 + 5 and three more roundings, halved by the root; rsqrt 2 ulp; four roundings of the result
    err = r * (terms * ((8 + 5 + 3) / 2 + 4 + 4 + min(d, 1)) * U32 + ones * angle_error(positions).to(x.device))
    return y * r, err


def head_norm_backward(dy, x, w, angle, positions, rot, interleaved, eps):
    """{"dx", "dw"}: (value, bound)."""
    dy, x, w = dy.double(), x.double(), _weight(w, x.shape[2], x)
    d, rows = x.shape[2], x.shape[0] * x.shape[1]
    r = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    dz, terms, ones = rotate(dy, angle, rot, interleaved, back=True)
    ez = terms * 3 * U32 + ones * angle_error(positions).to(x.device)
    g, xh = dz * w, x * r
    er = 12 * U32  # relative, of r
    dot = (g * xh).mean(-1, keepdim=True)
    edot = ((ez * w.abs() + g.abs() * 20 * U32) * xh.abs()).mean(-1, keepdim=True)
    dx = r * (g - xh * dot)
    edx = r * (ez * w.abs() + g.abs() * (er + 4 * U32) + xh.abs() * (edot + dot.abs() * (4 * er + 6 * U32)))
    # sums over rows: at worst one chain over all of them
    dw = (dz * xh).sum((0, 1))
    edw = (ez * xh.abs() + (dz * xh).abs() * (er + 3 * U32 + rows * U32)).sum((0, 1))
    return {"dx": (dx, edx), "dw": (dw, edw)}


# ------------------------------------------------------------------ attention

def seen(lq, lk, window, sinks, device="cpu"):
    """bool[lq, lk]: which keys each query sees (window None: no window)."""
    p = torch.arange(lq, device=device)[:, None] + (lk - lq)
    j = torch.arange(lk, device=device)[None]
    near = j > p - (lk + lq + 1 if window is None else window)
    return (j <= p) & (near | (j < sinks))


def _scores(q, k, scale):
    """s [heads, lq, lk] and the bound on its error: exact products summed
    over dim by the tensor cores or in binary32, and the scale's rounding."""
    t = torch.einsum("ihd,jhd->hij", q, k)
    mag = torch.einsum("ihd,jhd->hij", q.abs(), k.abs())
    return t * scale, scale * (mag * (2 * q.shape[2] * U32) + t.abs() * 3 * U32)


def _grouped(x, group):
    return x.repeat_interleave(group, 1)


def attention(q, k, v, window, sinks, scale, dtype):
    """One sequence: {"out", "lse"}: (value, bound), q [lq, heads, dim], k, v
    [lk, key heads, dim].  A weight exp(s - m) is off by its score's error, by
    16 u32 for the exponential's argument and the function itself, and by one
    rounding to dtype before the product with v (absolutely: by tiny, where
    the sum of all is at least 1)."""
    group = q.shape[1] // k.shape[1]
    mask = seen(q.shape[0], k.shape[0], window, sinks, q.device)
    q, k, v = q.double(), _grouped(k.double(), group), _grouped(v.double(), group)
    v0 = torch.where(mask.any(0)[:, None, None], v, 0.0)
    s, es = _scores(q, torch.where(mask.any(0)[:, None, None], k, 0.0), scale)
    s = s.masked_fill(~mask, -math.inf)
    es = es.masked_fill(~mask, 0.0)
    some = mask.any(1)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(some, lse, 0.0)[..., None])
    n = k.shape[0]
    top = torch.where(some, s.amax(-1) if n else lse, 0.0)
    size = torch.where(mask, s.abs() + top[..., None].abs(), 0.0)  # the exponential's argument is rounded at this size
    ep = es + (size * 2 + 16) * U32
    worst = ep.amax(-1) if n else torch.zeros_like(lse)
    out = torch.einsum("hij,jhd->ihd", p, v0)
    rel = ep + worst[..., None] + (UT[dtype] + (2 * n + 8) * U32)
    low = torch.exp(torch.where(some, top - lse, 0.0))  # 1 over the sum of weights
    eo = torch.einsum("hij,jhd->ihd", p * rel, v0.abs()) + \
        torch.einsum("hij,jhd->ihd", mask.double() * low[..., None] * TINY[dtype], v0.abs())
    elz = torch.where(some, worst + (n + 8) * U32 + 4 * U32 * (lse.abs() + top.abs()), 0.0)
    return {"out": (out, eo), "lse": (lse, elz)}


def attention_backward(dout, q, k, v, out, lse, window, sinks, scale, dtype):
    """One sequence: {"dq", "dk", "dv"}: (value, bound); out and lse [heads,
    lq] as the forward pass left them."""
    group = q.shape[1] // k.shape[1]
    heads = k.shape[1]
    mask = seen(q.shape[0], k.shape[0], window, sinks, q.device)
    some = mask.any(1)
    keys = mask.any(0)[:, None, None]
    q, do, o = (torch.where(some[:, None, None], x.double(), 0.0) for x in (q, dout, out))
    k, v = (torch.where(keys, _grouped(x.double(), group), 0.0) for x in (k, v))
    lse = torch.where(some, lse.double(), 0.0)
    s, es = _scores(q, k, scale)
    p = torch.where(mask, torch.exp(s - lse[..., None]), 0.0)
    ep = torch.where(mask, es + (s.abs() * 2 + lse.abs()[..., None] * 2 + 16) * U32, 0.0)
    d = q.shape[2]
    delta = (do * o).sum(-1).T[..., None]
    edelta = ((do * o).abs().sum(-1).T * (d * U32))[..., None]
    dp = torch.einsum("ihd,jhd->hij", do, v)
    edp = torch.einsum("ihd,jhd->hij", do.abs(), v.abs()) * (2 * d * U32)
    ds = p * (dp - delta)
    eds = p * (ep * (dp - delta).abs() + edp + edelta + 4 * U32 * (dp.abs() + delta.abs())) + UT[dtype] * ds.abs() + \
        torch.where(mask, TINY[dtype], 0.0)
    ep16 = p * (ep + UT[dtype]) + torch.where(mask, TINY[dtype], 0.0)
    n, m = k.shape[0], q.shape[0] * group

    def product(spec, a, ea, b, terms, factor):
        return (torch.einsum(spec, a, b) * factor,
                (torch.einsum(spec, ea, b.abs()) + torch.einsum(spec, a.abs(), b.abs()) * (2 * terms * U32)) * factor)

    def over_group(x):
        return tuple(t.view(t.shape[0], heads, group, d).sum(2) for t in x)

    return {"dq": product("hij,jhd->ihd", ds, eds, k, n, scale),
            "dk": over_group(product("hij,ihd->jhd", ds, eds, q, m, scale)),
            "dv": over_group(product("hij,ihd->jhd", p, ep16, do, m, 1.0))}
