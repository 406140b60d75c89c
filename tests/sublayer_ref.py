"""The feed-forward sub-block's operators in binary64, from their formulas, on
whatever device the inputs live on; with each result a bound on the error of
a kernel that works in binary32 and rounds as the header says.

The bounds (u32 = 2^-24 a binary32 rounding, ut that of the output's type,
tiny the half quantum of its subnormals):
  * a sum of n binary32 terms taken in chains of at most `depth` additions is
    off by at most depth * u32 * sum |terms|;
  * a tensor-core product over k terms adds exact products into binary32
    sums that may truncate: k * 2 * u32 * sum |a b|;
  * errors of inputs pass through the first derivative of what follows;
  * sigmoid through the fast exponential: relative 1e-5, plus 1e-30.
"""
import numpy as np
import torch

U32 = 2.0 ** -24
UT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8, torch.float32: U32}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134, torch.float32: 2.0 ** -150}
SILU, GELU = 0, 1


def rounded(ref, err, dtype):
    """The bound after one rounding to dtype."""
    return err + UT[dtype] * (ref.abs() + err) + TINY[dtype]


def check(got, ref, bound, what):
    g = got.double()
    assert g.shape == ref.shape, what
    same = (g == ref) | (torch.isnan(g) & torch.isnan(ref))
    ok = same | ((g - ref).abs() <= bound)
    if not bool(ok.all()):
        i = int((~ok).flatten().nonzero()[0])
        raise AssertionError(f"{what}: {int((~ok).sum())} of {ok.numel()} outside the bound; first at {i}: got "
                             f"{g.flatten()[i]!r} want {ref.flatten()[i]!r} bound {bound.flatten()[i]!r}")


# ------------------------------------------------------------------ dropout

def philox(counter, key):
    """Philox4x32-10 on numpy uint64 arrays holding 32-bit words."""
    m = np.uint64(0xFFFFFFFF)
    c = [np.asarray(x, np.uint64) for x in counter]
    k0, k1 = int(key[0]), int(key[1])
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & m, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & m]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def keep_mask(rows, cols, p, seed, offset):
    """bool[rows, cols] (numpy): the elements a dropout keeps."""
    quads = (cols + 3) // 4
    c, r = np.meshgrid(np.arange(quads, dtype=np.uint64), np.arange(rows, dtype=np.uint64))
    offset &= (1 << 64) - 1
    w = philox([c, r, np.full_like(c, offset & 0xFFFFFFFF), np.full_like(c, offset >> 32)],
               (seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF))
    words = np.stack(w, -1).reshape(rows, quads * 4)[:, :cols]
    return words >= np.uint64(int(np.floor(p * 2.0 ** 32 + 0.5)))


def drop_scale(p):
    return float(np.float32(1.0 / (1.0 - p))) if p < 1 else 0.0


def dropout_add(x, residual, drop):
    """(t, error before rounding): drop a tuple (p, seed, offset) or None."""
    t = x.double()
    if drop is not None:
        keep = torch.from_numpy(keep_mask(x.shape[0], x.shape[1], *drop)).to(x.device)
        t = torch.where(keep, t * drop_scale(drop[0]), torch.zeros_like(t))
    err = U32 * t.abs() if drop is not None else torch.zeros_like(t)
    if residual is not None:
        t = t + residual.double()
        err = err + U32 * (t.abs() + err)
    return t, err


# ------------------------------------------------------------------ layer norm

def layer_norm(x, weight, bias, eps, residual=None, drop=None):
    """dict of (value, error before rounding) for y, mean, rstd, sum."""
    t, e = dropout_add(x, residual, drop)
    n = t.shape[1]
    depth = 32 + n / 128
    mean = t.mean(1, keepdim=True)
    em = (depth + 1) * U32 * t.abs().mean(1, keepdim=True) + e.mean(1, keepdim=True)
    d = t - mean
    ed = e + em + U32 * (d.abs() + e + em)
    var = d.square().mean(1, keepdim=True)
    ev = (2 * d.abs() * ed + ed.square()).mean(1, keepdim=True) + (depth + 3) * U32 * var
    rstd = 1 / torch.sqrt(var + eps)
    # relative: d(rstd)/rstd = -dvar / (2 (var + eps)); the binary32 eps, sum, root and division
    er = rstd * (0.5 * ev / (var + eps - ev).clamp_min(1e-300) + 4 * U32)
    xh = d * rstd
    ex = ed * rstd + d.abs() * er + ed * er + 2 * U32 * xh.abs()
    w = torch.ones(n, dtype=torch.float64, device=t.device) if weight is None else weight.double()
    y = xh * w
    ey = ex * w.abs() + U32 * y.abs()
    if bias is not None:
        y = y + bias.double()
        ey = ey + U32 * (y.abs() + ey)
    return {"y": (y, ey), "mean": (mean[:, 0], em[:, 0]), "rstd": (rstd[:, 0], er[:, 0]), "sum": (t, e)}


def layer_norm_backward(dy, x, weight, mean, rstd, dresidual=None, drop=None):
    """dict of (value, error before rounding) for dx, dropped, dweight, dbias."""
    rows, n = x.shape
    depth = 32 + n / 128
    t, dyd = x.double(), dy.double()
    mu, r = mean.double()[:, None], rstd.double()[:, None]
    xh = (t - mu) * r
    ex = 3 * U32 * (t - mu).abs() * r
    w = torch.ones(n, dtype=torch.float64, device=t.device) if weight is None else weight.double()
    g = dyd * w
    eg = U32 * g.abs()
    s0, s1 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    e0 = ((depth + 2) * U32 * g.abs() + eg).mean(1, keepdim=True)
    e1 = ((depth + 3) * U32 * (g * xh).abs() + eg * xh.abs() + ex * g.abs()).mean(1, keepdim=True)
    dx = r * (g - s0 - xh * s1)
    edx = r * (eg + e0 + ex * s1.abs() + xh.abs() * e1 + 4 * U32 * (g.abs() + s0.abs() + (xh * s1).abs()))
    if dresidual is not None:
        dx = dx + dresidual.double()
        edx = edx + U32 * (dx.abs() + edx)
    out = {"dx": (dx, edx)}
    if drop is not None:
        keep = torch.from_numpy(keep_mask(rows, n, *drop)).to(x.device)
        s = drop_scale(drop[0])
        out["dropped"] = (torch.where(keep, dx * s, torch.zeros_like(dx)),
                          torch.where(keep, edx * s + U32 * dx.abs() * s, torch.zeros_like(dx)))
    rd = 32 + rows / 8
    out["dweight"] = ((dyd * xh).sum(0), (dyd.abs() * (ex + (rd + 1) * U32 * xh.abs())).sum(0))
    out["dbias"] = (dyd.sum(0), rd * U32 * dyd.abs().sum(0))
    return out


# ------------------------------------------------------------------ gated feed-forward

def act(kind, g):
    """(value, slope, value error, slope error) of the gate's activation."""
    if kind == SILU:
        k, dk = g, torch.ones_like(g)
    else:
        a = 2 * np.sqrt(2 / np.pi)
        k, dk = a * (g + 0.044715 * g ** 3), a * (1 + 3 * 0.044715 * g ** 2)
    s = torch.sigmoid(k)
    # binary32 rounding of k moves the sigmoid by 4 u32 |k| of itself
    rel = 1e-5 + 8 * U32 * k.abs()
    value, slope = g * s, s + g * s * (1 - s) * dk
    return value, slope, rel * value.abs() + 1e-30, 3 * rel * (s + (g * s * dk).abs()) + 1e-30


def product(a, b, ea=None, eb=None):
    """a b^T with the error of a tensor-core product and of its inputs."""
    c, m = a @ b.T, a.abs() @ b.abs().T
    e = (a.shape[1] + 1) * 2 * U32 * m
    if ea is not None:
        e = e + ea @ b.abs().T
    if eb is not None:
        e = e + (a.abs() + (ea if ea is not None else 0)) @ eb.T
    return c, e


def gated_ffn(x, wg, wu, wd, kind):
    dt = x.dtype
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    v, slope, ev, es = act(kind, g)
    ev = ev + (slope.abs() + es + 1.1 * eg) * eg  # |act''| < 1.1 for both
    h = v * u
    eh = rounded(h, ev * u.abs() + v.abs() * eu + ev * eu + U32 * h.abs(), dt)
    return {"y": product(h, wd, eh), "gate": (g, eg), "up": (u, eu)}


def gated_ffn_backward(dy, x, wg, wu, wd, gate, up, kind):
    dt = x.dtype
    dy, x, wg, wu, wd, g, u = (t.double() for t in (dy, x, wg, wu, wd, gate, up))
    dh, ed = product(dy, wd.T)
    v, slope, ev, es = act(kind, g)
    dg, du, h = dh * u * slope, dh * v, v * u
    edg = rounded(dg, (ed * slope.abs() + dh.abs() * es + ed * es) * u.abs() + 3 * U32 * dg.abs(), dt)
    edu = rounded(du, ed * v.abs() + dh.abs() * ev + ed * ev + U32 * du.abs(), dt)
    eh = rounded(h, ev * u.abs() + U32 * h.abs(), dt)
    a, ea = product(dg, wg.T, edg)
    b, eb = product(du, wu.T, edu)
    return {"dx": (a + b, ea + eb + 2 * U32 * (a.abs() + b.abs())),
            "dw_gate": product(dg.T, x.T, edg.T), "dw_up": product(du.T, x.T, edu.T),
            "dw_down": product(dy.T, h.T, None, eh.T)}
