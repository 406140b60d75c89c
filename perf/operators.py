"""The operators of the pre-norm feed-forward half of a transformer layer, as
cases to time and compare: dropout with the residual sum, layer norm (alone
and with that sum in front of it) and the gated feed-forward, each forward
and backward.

``run`` computes a case in its plain form (elementary torch operations in
binary32, one rounding at the end) or, with ``own`` set, through the calls of
``zero_partitioned_mixed_layout_gb300``.
"""
import math

import numpy as np
import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5

# ------------------------------------------------------------------ cases

# op "dropout":  out = residual + dropout(x)  (residual 0: the backward form, dropout of a gradient)
# op "norm":     y = layer_norm(t); fused 1: t = residual + dropout(x), also returned
# op "norm_bwd": dx, dweight, dbias; fused 1: the residual path's gradient added, and dx through the mask
# op "ffn":      y = (act(x Wg') * (x Wu')) Wd'; train 1: gate and up kept for the backward pass
# op "ffn_bwd":  dx and the three weight gradients


def listed():
    return [
        # the tiny 2-layer state (hidden 256): one short batch, where the launch is all there is
        dict(name="dropout_tiny", op="dropout", rows=64, cols=256, dtype="f16", p=0.1, residual=1),
        # a ragged batch over an odd width, the gradient's direction
        dict(name="dropout_bwd_odd", op="dropout", rows=4097, cols=1601, dtype="f16", p=0.1, residual=0),
        # the 100B stack's width, two sequences of 8192: the residual stream of a large step
        dict(name="dropout_wide", op="dropout", rows=16384, cols=8192, dtype="bf16", p=0.1, residual=1),
        # one token of GPT-2 1.5B (hidden 1600) while it answers
        dict(name="norm_token", op="norm", rows=1, cols=1600, dtype="f16", wdtype="f16", p=0.0, fused=0),
        # GPT-2 1.5B in training, 8 sequences of its 1024 positions: sum, dropout and norm
        dict(name="norm_train", op="norm", rows=8192, cols=1600, dtype="f16", wdtype="f16", p=0.1, fused=1),
        # its backward pass, gradients in the fp16 that the optimizer step reads
        dict(name="norm_bwd_train", op="norm_bwd", rows=8192, cols=1600, dtype="f16", wdtype="f16", gdtype="f16",
             p=0.1, fused=1),
        # an odd width in binary32 with binary32 weight gradients
        dict(name="norm_bwd_odd", op="norm_bwd", rows=3001, cols=2049, dtype="f32", wdtype="f32", gdtype="f32",
             p=0.0, fused=0),
        # one token through GPT-2 1.5B's inner width: three weight matrices read once
        dict(name="ffn_token", op="ffn", tokens=1, dim=1600, inner=6400, dtype="f16", act="gelu", train=0),
        # a ragged batch of prompts over widths that no vector divides
        dict(name="ffn_odd", op="ffn", tokens=333, dim=1001, inner=2731, dtype="bf16", act="silu", train=0),
        # GPT-2 1.5B in training, forward
        dict(name="ffn_train", op="ffn", tokens=8192, dim=1600, inner=6400, dtype="f16", act="gelu", train=1),
        # and backward
        dict(name="ffn_bwd_train", op="ffn_bwd", tokens=8192, dim=1600, inner=6400, dtype="f16", act="gelu"),
        # the 100B stack's widths (8192, 4 x 8192) on one sequence of 2048, backward
        dict(name="ffn_bwd_stack", op="ffn_bwd", tokens=2048, dim=8192, inner=32768, dtype="bf16", act="silu"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["dropout", "norm", "norm_bwd", "ffn", "ffn_bwd"])
    dtype = rng.choice(["f16", "bf16", "f32"])
    p = rng.choice([0.05, 0.1, 0.25, 0.5])
    if op in ("ffn", "ffn_bwd"):
        case = dict(op=op, dtype=rng.choice(["f16", "bf16"]), act=rng.choice(["gelu", "silu"]))
        case["dim"] = _log_int(rng, 64, 8192)
        case["inner"] = _log_int(rng, 64, 32768)
        if rng.random() < 0.5:  # most models' widths are whole tiles, some are not
            case["dim"], case["inner"] = -(-case["dim"] // 64) * 64, -(-case["inner"] // 64) * 64
        case["tokens"] = _log_int(rng, 1, 8192)
        most = 2048 * 8192 * 32768
        case["tokens"] = max(1, min(case["tokens"], most // (case["dim"] * case["inner"])))
        if op == "ffn":
            case["train"] = rng.randint(0, 1)
        return case
    cols = _log_int(rng, 16, 16384)
    if rng.random() < 0.5:
        cols = -(-cols // 16) * 16
    rows = min(_log_int(rng, 1, 32768), (16384 * 8192) // cols)
    if dtype == "f32":
        rows = max(1, rows // 2)
    case = dict(op=op, rows=rows, cols=cols, dtype=dtype)
    if op == "dropout":
        return {**case, "p": p, "residual": rng.randint(0, 1)}
    fused = rng.randint(0, 1)
    case.update(wdtype=rng.choice([dtype, "f32"]), p=p if fused else 0.0, fused=fused)
    if op == "norm_bwd":
        case["gdtype"] = rng.choice([dtype, "f32"])
    return case


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype, std=1.0, mean=0.0):
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=gen)
    return t.to(TYPES[dtype])


def _inputs(case, seed):
    """The data of a case, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2 + 1)
    s = {"case": case, "key": (int(seed) * 0x9E3779B97F4A7C15 + 12345) % 2**63, "offset": int(seed) % 1000 + 2**32 - 500}
    op, dt = case["op"], case["dtype"]
    if op in ("ffn", "ffn_bwd"):
        m, d, f = case["tokens"], case["dim"], case["inner"]
        s["x"] = _normal(gen, (m, d), dt)
        s["w_gate"] = _normal(gen, (f, d), dt, 1 / math.sqrt(d))
        s["w_up"] = _normal(gen, (f, d), dt, 1 / math.sqrt(d))
        s["w_down"] = _normal(gen, (d, f), dt, 1 / math.sqrt(f))
        if op == "ffn_bwd":
            # the gradient arrives times the loss scale; gate and up as the forward pass left them
            s["dy"] = _normal(gen, (m, d), dt)
            s["gate"] = (s["x"].float() @ s["w_gate"].float().T).to(TYPES[dt])
            s["up"] = (s["x"].float() @ s["w_up"].float().T).to(TYPES[dt])
        return s
    r, c = case["rows"], case["cols"]
    if op == "dropout":
        s["x"] = _normal(gen, (r, c), dt)
        s["residual"] = _normal(gen, (r, c), dt, 2.0) if case["residual"] else None
        return s
    s["weight"] = _normal(gen, (c,), case["wdtype"], 0.1, 1.0)
    s["bias"] = _normal(gen, (c,), case["wdtype"], 0.1)
    s["x"] = _normal(gen, (r, c), dt, 1.0, 0.25)
    if op == "norm":
        s["residual"] = _normal(gen, (r, c), dt, 2.0) if case["fused"] else None
        return s
    s["dy"] = _normal(gen, (r, c), dt)
    s["dresidual"] = _normal(gen, (r, c), dt) if case["fused"] else None
    t = s["x"].float()
    s["mean"] = t.mean(1)
    s["rstd"] = torch.rsqrt((t - s["mean"][:, None]).square().mean(1) + EPS)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if not own:
        return s
    import zero_partitioned_mixed_layout_gb300 as zp
    s["zp"] = zp
    op, dt = case["op"], TYPES[case["dtype"]]

    def like(t, dtype=None):
        return torch.empty_like(t, dtype=dtype)

    if op in ("ffn", "ffn_bwd"):
        m, d, f = case["tokens"], case["dim"], case["inner"]
        s["act"] = {"gelu": zp.ZERO_ACT_GELU_TANH, "silu": zp.ZERO_ACT_SILU}[case["act"]]
        s["ws"] = zp.new_gated_ffn_workspace(m, d, f, backward=op == "ffn_bwd")
        if op == "ffn":
            s["y"] = like(s["x"])
            s["gate"], s["up"] = (torch.empty((m, f), dtype=dt, device="cuda") if case["train"] else None
                                  for _ in range(2))
        else:
            s["dx"] = like(s["x"])
            s["dw_gate"], s["dw_up"], s["dw_down"] = like(s["w_gate"]), like(s["w_up"]), like(s["w_down"])
        return s
    s["drop"] = zp.Dropout(case["p"], s["key"], s["offset"]) if case["p"] else None
    if op == "dropout":
        s["out"] = like(s["x"])
        return s
    c, r = case["cols"], case["rows"]
    if op == "norm":
        s["y"] = like(s["x"])
        s["sum"] = like(s["x"]) if case["fused"] else None
        s["mean"], s["rstd"] = (torch.empty(r, dtype=torch.float32, device="cuda") for _ in range(2))
        return s
    s["ws"] = zp.new_layer_norm_workspace(r, c)
    s["dx"] = like(s["x"])
    s["dx_dropped"] = like(s["x"]) if case["fused"] else None
    s["dweight"], s["dbias"] = (torch.empty(c, dtype=TYPES[case["gdtype"]], device="cuda") for _ in range(2))
    return s


# ------------------------------------------------------------------ plain forms

M32 = 0xFFFFFFFF


def _keep(rows, cols, p, key, offset):
    """Philox4x32-10 at counter (column / 4, row, offset low, offset high);
    element kept where word column % 4 is at least round(p * 2^32).  32-bit
    words in int64: a product wraps at 64 bits, its halves stay right."""
    quads = -(-cols // 4)
    c0 = torch.arange(quads, device="cuda", dtype=torch.int64).expand(rows, quads)
    c1 = torch.arange(rows, device="cuda", dtype=torch.int64)[:, None].expand(rows, quads)
    c2, c3 = torch.full_like(c0, offset & M32), torch.full_like(c0, (offset >> 32) & M32)
    k0, k1 = key & M32, (key >> 32) & M32
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & M32) ^ c1 ^ k0, b & M32, ((a >> 32) & M32) ^ c3 ^ k1, a & M32
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    words = torch.stack([c0, c1, c2, c3], -1).reshape(rows, quads * 4)[:, :cols]
    return words >= int(math.floor(p * 2.0**32 + 0.5))


def _dropped(t, s):
    c = s["case"]
    if not c["p"]:
        return t
    keep = _keep(t.shape[0], t.shape[1], c["p"], s["key"], s["offset"])
    return torch.where(keep, t * float(np.float32(1.0 / (1.0 - c["p"]))), torch.zeros((), device="cuda"))


def _act(g, kind):
    if kind == "silu":
        return g * torch.sigmoid(g)
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_slope(g, kind):
    if kind == "silu":
        q = torch.sigmoid(g)
        return q * (1 + g * (1 - q))
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (g + 0.044715 * g * g * g))
    return 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * a * (1 + 3 * 0.044715 * g * g)


def _plain(s):
    case = s["case"]
    op, dt = case["op"], TYPES[case["dtype"]]
    if op == "dropout":
        t = _dropped(s["x"].float(), s)
        if case["residual"]:
            t = s["residual"].float() + t
        return {"out": t.to(dt)}
    if op == "norm":
        t = s["x"].float()
        if case["fused"]:
            t = s["residual"].float() + _dropped(t, s)
        mean = t.mean(1)
        d = t - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(1) + EPS)
        y = d * rstd[:, None] * s["weight"].float() + s["bias"].float()
        out = {"y": y.to(dt), "mean": mean, "rstd": rstd}
        if case["fused"]:
            out["sum"] = t.to(dt)
        return out
    if op == "norm_bwd":
        dy = s["dy"].float()
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        gdt = TYPES[case["gdtype"]]
        out = {"dweight": (dy * xh).sum(0).to(gdt), "dbias": dy.sum(0).to(gdt)}
        if case["fused"]:
            dx = dx + s["dresidual"].float()
            out["dx_dropped"] = _dropped(dx, s).to(dt)
        return {**out, "dx": dx.to(dt)}
    x, wg, wu, wd = (s[k].float() for k in ("x", "w_gate", "w_up", "w_down"))
    if op == "ffn":
        g, u = x @ wg.T, x @ wu.T
        y = (_act(g, case["act"]) * u) @ wd.T
        out = {"y": y.to(dt)}
        if case["train"]:
            out.update(gate=g.to(dt), up=u.to(dt))
        return out
    dy, g, u = s["dy"].float(), s["gate"].float(), s["up"].float()
    a = _act(g, case["act"])
    dh = dy @ wd
    dg, du = dh * u * _act_slope(g, case["act"]), dh * a
    return {"dx": (dg @ wg + du @ wu).to(dt), "dw_gate": (dg.T @ x).to(dt), "dw_up": (du.T @ x).to(dt),
            "dw_down": (dy.T @ (a * u)).to(dt)}


def run(s):
    if not own:
        return _plain(s)
    zp, case = s["zp"], s["case"]
    op = case["op"]
    if op == "dropout":
        zp.zero_dropout_add(s["x"], s["residual"], s["out"], s["drop"])
        return {"out": s["out"]}
    if op == "norm":
        zp.zero_layer_norm(s["x"], s["weight"], s["bias"], s["y"], s["mean"], s["rstd"], eps=EPS,
                           residual=s["residual"], drop=s["drop"], sum_out=s["sum"])
        out = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
        if case["fused"]:
            out["sum"] = s["sum"]
        return out
    if op == "norm_bwd":
        zp.zero_layer_norm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"],
                                    s["dbias"], s["ws"], dresidual=s["dresidual"], drop=s["drop"],
                                    dx_dropped=s["dx_dropped"])
        out = {"dweight": s["dweight"], "dbias": s["dbias"]}
        if case["fused"]:
            out["dx_dropped"] = s["dx_dropped"]
        return {**out, "dx": s["dx"]}
    if op == "ffn":
        zp.zero_gated_ffn(s["x"], s["w_gate"], s["w_up"], s["w_down"], s["y"], s["ws"], act=s["act"],
                          gate=s["gate"], up=s["up"])
        out = {"y": s["y"]}
        if case["train"]:
            out.update(gate=s["gate"], up=s["up"])
        return out
    zp.zero_gated_ffn_backward(s["dy"], s["x"], s["w_gate"], s["w_up"], s["w_down"], s["gate"], s["up"], s["dx"],
                               s["dw_gate"], s["dw_up"], s["dw_down"], s["ws"], act=s["act"])
    return {k: s[k] for k in ("dx", "dw_gate", "dw_up", "dw_down")}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    if op in ("ffn", "ffn_bwd"):
        m, d, f = case["tokens"], case["dim"], case["inner"]
        if op == "ffn":  # x, y, three weights (gate and up written in training)
            return {"bytes": e * (2 * m * d + 3 * d * f + (2 * m * f if case["train"] else 0)), "flops": 6.0 * m * d * f}
        # dy, x, dx; gate, up; three weights read, three gradients written
        return {"bytes": e * (3 * m * d + 2 * m * f + 6 * d * f), "flops": 12.0 * m * d * f}
    n, c, r = case["rows"] * case["cols"], case["cols"], case["rows"]
    if op == "dropout":
        return {"bytes": e * n * (3 if case["residual"] else 2), "flops": 2.0 * n}
    w = BYTES[case["wdtype"]]
    if op == "norm":  # x (residual), y (sum); weight, bias; mean, rstd
        return {"bytes": e * n * (4 if case["fused"] else 2) + 2 * w * c + 8 * r, "flops": 8.0 * n}
    # dy, x, dx (dresidual, dx_dropped); weight; mean, rstd; dweight, dbias
    return {"bytes": e * n * (5 if case["fused"] else 3) + w * c + 8 * r + 2 * BYTES[case["gdtype"]] * c,
            "flops": 14.0 * n}


# ------------------------------------------------------------------ the definition in 64 bits

def _mul_halves(a, k):
    """High and low 32 bits of a * k through 16-bit limbs (no wrap)."""
    al, ah, kl, kh = a & 0xFFFF, a >> 16, k & 0xFFFF, k >> 16
    mid = ah * kl + ((al * kl) >> 16)
    mid2 = al * kh + (mid & 0xFFFF)
    return ah * kh + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((al * kl) & 0xFFFF)


def _exact_keep(rows, cols, p, key, offset):
    quads = (cols + 3) // 4
    at = torch.arange(rows * quads, device="cuda", dtype=torch.int64)
    x = [at % quads, torch.div(at, quads, rounding_mode="floor"),
         torch.full_like(at, offset % 2**32), torch.full_like(at, offset // 2**32 % 2**32)]
    for i in range(10):
        k0, k1 = (key + i * 0x9E3779B9) % 2**32, (key // 2**32 + i * 0xBB67AE85) % 2**32
        h0, l0 = _mul_halves(x[0], 0xD2511F53)
        h1, l1 = _mul_halves(x[2], 0xCD9E8D57)
        x = [h1 ^ x[1] ^ k0, l1, h0 ^ x[3] ^ k1, l0]
    return (torch.stack(x, 1).view(rows, quads * 4)[:, :cols] < math.floor(p * 2**32 + 0.5)).logical_not_()


def _exact_drop(t, case, s):
    if case["p"] == 0:
        return t
    keep = _exact_keep(case["rows"], case["cols"], case["p"], s["key"], s["offset"])
    return (t / (1.0 - case["p"])).masked_fill_(~keep, 0.0)


def exact(case, seed):
    op = case["op"]
    if op in ("ffn", "ffn_bwd") and 6.0 * case["tokens"] * case["dim"] * case["inner"] * (2 if op == "ffn_bwd" else 1) > 7e12:
        return None
    s = _inputs(case, seed)
    D = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    if op == "dropout":
        t = _exact_drop(D["x"], case, s)
        return {"out": t.add_(D["residual"]) if case["residual"] else t}
    if op == "norm":
        t = D["x"]
        if case["fused"]:
            t = _exact_drop(t, case, s) + D["residual"]
        var, mean = torch.var_mean(t, 1, correction=0, keepdim=True)
        rstd = 1 / torch.sqrt(var + EPS)
        out = {"y": (t - mean) * rstd * D["weight"] + D["bias"], "mean": mean[:, 0], "rstd": rstd[:, 0]}
        if case["fused"]:
            out["sum"] = t
        return out
    if op == "norm_bwd":
        n, rstd = case["cols"], D["rstd"][:, None]
        xh = (D["x"] - D["mean"][:, None]) * rstd
        g = D["dy"] * D["weight"]
        dx = rstd / n * (n * g - g.sum(1, keepdim=True) - xh * (g * xh).sum(1, keepdim=True))
        out = {"dweight": torch.einsum("rc,rc->c", D["dy"], xh), "dbias": D["dy"].sum(0)}
        if case["fused"]:
            dx = dx + D["dresidual"]
            out["dx_dropped"] = _exact_drop(dx.clone(), case, s)
        return {**out, "dx": dx}
    if op == "ffn":
        g, u = D["x"] @ D["w_gate"].T, D["x"] @ D["w_up"].T
        out = {"y": (_exact_act(g, case["act"])[0] * u) @ D["w_down"].T}
        if case["train"]:
            out.update(gate=g, up=u)
        return out
    a, slope = _exact_act(D["gate"], case["act"])
    dh = D["dy"] @ D["w_down"]
    dg, du = dh * D["up"] * slope, dh * a
    return {"dx": dg @ D["w_gate"] + du @ D["w_up"], "dw_gate": dg.T @ D["x"], "dw_up": du.T @ D["x"],
            "dw_down": D["dy"].T @ (a * D["up"])}


def _exact_act(g, kind):
    """The activation and its slope, both as z * sigmoid(k(z))."""
    if kind == "silu":
        k, dk = g, 1.0
    else:
        b = 2 * math.sqrt(2 / math.pi)
        k, dk = b * (g + 0.044715 * g**3), b * (1 + 0.134145 * g**2)
    q = 1 / (1 + torch.exp(-k))
    return g * q, q + g * q * (1 - q) * dk
