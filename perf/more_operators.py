"""The operators of the attention half of a transformer layer, as cases to time
and compare: norms of queries and keys for each head with the position
rotation in the same pass, and attention with a sliding window and a few first
keys that stay visible (over packed sequences, and of new tokens over a cache);
each forward and backward.

``run`` computes a case in its plain form (elementary torch operations in
binary32, one rounding at the end) or, with ``own`` set, through the calls of
``zero_partitioned_mixed_layout_gb300``.
"""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-6
BASE = 10000.0

# ------------------------------------------------------------------ cases

# op "norm":     y = rotation(norm(x)) of the heads of q and k
# op "norm_bwd": dx of both, and the two weights' gradients
# op "attn":     out and lse; kind "packed": sequences in training (as many queries as keys), "cache": `new` tokens
#                for each sequence over a cache with room for `most` keys each
# op "attn_bwd": dq, dk, dv of packed sequences
# window 0: every key up to the query's own; ragged 1: lengths from most / 4 (a cache: most / 8) to most


def listed():
    return [
        # one token of GPT-2 1.5B (25 heads of 64) while it answers: the launch is all there is
        dict(name="norm_token", op="norm", tokens=1, heads=25, kv_heads=25, dim=64, rot=64, pairs="half", dtype="f16",
             wdtype="f16", far=1000),
        # GPT-2 1.5B in training, 8 sequences of its 1024 positions
        dict(name="norm_train", op="norm", tokens=8192, heads=25, kv_heads=25, dim=64, rot=64, pairs="half",
             dtype="f16", wdtype="f16", far=0),
        # its backward pass, gradients in the fp16 that the optimizer step reads
        dict(name="norm_bwd_train", op="norm_bwd", tokens=8192, heads=25, kv_heads=25, dim=64, rot=64, pairs="half",
             dtype="f16", wdtype="f16", gdtype="f16", far=0),
        # binary32, a head dimension that is no power of two, half of it rotated, far positions
        dict(name="norm_bwd_odd", op="norm_bwd", tokens=3001, heads=7, kv_heads=3, dim=80, rot=40, pairs="next",
             dtype="f32", wdtype="f32", gdtype="f32", far=10**6),
        # the 100B stack's 64 heads of 128 (8 of keys) over one long prompt
        dict(name="norm_long", op="norm", tokens=16384, heads=64, kv_heads=8, dim=128, rot=128, pairs="half",
             dtype="bf16", wdtype="bf16", far=10**5),
        # one token of GPT-2 1.5B over the keys of its 1024 positions
        dict(name="attn_token", op="attn", kind="cache", sequences=1, new=1, most=1024, ragged=0, heads=25,
             kv_heads=25, dim=64, window=256, sinks=4, dtype="f16"),
        # 64 requests answering at once over caches of up to 8192 keys, at the 100B stack's heads
        dict(name="attn_answer", op="attn", kind="cache", sequences=64, new=1, most=8192, ragged=1, heads=64,
             kv_heads=8, dim=128, window=4096, sinks=4, dtype="bf16"),
        # ragged chunks of a prompt over what is cached, an odd window, heads of 80 in groups of three
        dict(name="attn_chunk", op="attn", kind="cache", sequences=5, new=333, most=2049, ragged=1, heads=12,
             kv_heads=4, dim=80, window=777, sinks=5, dtype="f16"),
        # GPT-2 1.5B in training, 8 sequences of its 1024 positions
        dict(name="attn_train", op="attn", kind="packed", sequences=8, most=1024, ragged=0, heads=25, kv_heads=25,
             dim=64, window=256, sinks=4, dtype="f16"),
        # its backward pass over packed sequences of uneven lengths
        dict(name="attn_bwd_train", op="attn_bwd", kind="packed", sequences=8, most=1024, ragged=1, heads=25,
             kv_heads=25, dim=64, window=256, sinks=4, dtype="f16"),
        # the 100B stack's heads over one long sequence
        dict(name="attn_long", op="attn", kind="packed", sequences=1, most=16384, ragged=0, heads=64, kv_heads=8,
             dim=128, window=2048, sinks=64, dtype="bf16"),
        # and backward
        dict(name="attn_bwd_long", op="attn_bwd", kind="packed", sequences=1, most=16384, ragged=0, heads=64,
             kv_heads=8, dim=128, window=2048, sinks=64, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    kv = _log_int(rng, 1, 32)
    return min(64, kv * rng.choice([1, 1, 2, 3, 4, 8])) // kv * kv, kv


def draw(rng):
    op = rng.choice(["norm", "norm_bwd", "attn", "attn", "attn_bwd"])
    heads, kv = _heads(rng)
    if op in ("norm", "norm_bwd"):
        dtype = rng.choice(["f16", "bf16", "f32"])
        dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 256, 2 * rng.randint(5, 128)])
        rot = rng.choice([dim, dim, dim // 4 * 2])
        most = 16384 * 72 * 128 // ((heads + kv) * dim) // (2 if dtype == "f32" else 1)
        case = dict(op=op, tokens=max(1, min(_log_int(rng, 1, 32768), most)), heads=heads, kv_heads=kv, dim=dim,
                    rot=rot, pairs=rng.choice(["half", "next"]), dtype=dtype, wdtype=rng.choice([dtype, "f32"]),
                    far=rng.choice([0, 1000, 10**5, 10**6]))
        if op == "norm_bwd":
            case["gdtype"] = rng.choice([dtype, "f32"])
        return case
    case = dict(op=op, kind="packed" if op == "attn_bwd" else rng.choice(["packed", "cache"]),
                sequences=_log_int(rng, 1, 64), ragged=rng.randint(0, 1), heads=heads, kv_heads=kv,
                dim=rng.choice([64, 64, 80, 96, 128, 128, 8 * rng.randint(4, 16)]), dtype=rng.choice(["f16", "bf16"]),
                sinks=rng.choice([0, 1, 4, 64, 130]), window=rng.choice([0, _log_int(rng, 16, 4096), 1024]))
    case["most"] = _log_int(rng, 16, 16384)
    if case["kind"] == "cache":
        case["new"] = min(case["most"], rng.choice([1, 1, 1, 2, 5, _log_int(rng, 8, 1024)]))
    # no more queries, keys or pairs (with those at the window's ends) than the largest listed cases have
    keys = min(case["most"], (case["window"] or case["most"]) + 255) + case["sinks"]
    rows = min(16384 * 64 // heads, 16384 * 2304 * 64 // (heads * keys))
    if case["kind"] == "packed":
        case["most"] = min(case["most"], rows)
    case["sequences"] = max(1, min(case["sequences"], rows // case.get("new", case["most"]),
                                   64 * 8192 * 8 // (case["most"] * kv)))
    return case


def _lengths(case):
    """(queries, keys) of each sequence: from the case alone."""
    rng = random.Random(case["sequences"] * 65537 + case["most"])
    n, most = case["sequences"], case["most"]
    if case["kind"] == "packed":
        q = [rng.randint(max(1, most // 4), most) if case["ragged"] else most for _ in range(n)]
        return q, q
    q = [rng.randint(max(1, case["new"] // 2), case["new"]) if case["ragged"] else case["new"] for _ in range(n)]
    return q, [max(a, rng.randint(max(1, most // 8), most) if case["ragged"] else most) for a in q]


# ------------------------------------------------------------------ inputs

def _normal(gen, shape, dtype, std=1.0, mean=0.0):
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=gen)
    return t.to(TYPES[dtype])


def _before(lengths):
    return [sum(lengths[:i]) for i in range(len(lengths) + 1)]


def _inputs(case, seed):
    """The data of a case, from the seed alone."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 2 + 1)
    s = {"case": case}
    h, g, d, dt = case["heads"], case["kv_heads"], case["dim"], case["dtype"]
    if case["op"] in ("norm", "norm_bwd"):
        t = case["tokens"]
        # queries and keys are slices of one projection's output, as are their gradients
        s["qk"] = _normal(gen, (t, h + g, d), dt, 1.5)
        s["q_weight"], s["k_weight"] = (_normal(gen, (d,), case["wdtype"], 0.1, 1.0) for _ in range(2))
        s["inv_freq"] = [BASE ** (-2.0 * i / case["rot"]) for i in range(case["rot"] // 2)]
        first = torch.randint(0, case["far"] + 1, (1,), device="cuda", generator=gen)
        s["positions"] = torch.arange(t, device="cuda") % 1024 + first if case["far"] < 10**5 else \
            torch.arange(t, device="cuda") + first
        if case["op"] == "norm_bwd":
            s["dqk"] = _normal(gen, (t, h + g, d), dt)
        return s
    ql, kl = _lengths(case)
    room = kl if case["kind"] == "packed" else [case["most"]] * len(kl)
    tq, tk = sum(ql), sum(room)
    s["q"] = _normal(gen, (tq, h, d), dt)
    s["k"], s["v"] = _normal(gen, (tk, g, d), dt), _normal(gen, (tk, g, d), dt)
    s["q_offsets"], s["k_offsets"], s["k_lengths"] = (torch.tensor(x, device="cuda")
                                                      for x in (_before(ql), _before(room), kl))
    if case["op"] == "attn_bwd":
        # the gradient that reaches the output, and what the forward pass left
        s["dout"] = _normal(gen, s["q"].shape, dt)
        s.update(_plain_attention(s))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    h, g, d, dt = case["heads"], case["kv_heads"], case["dim"], TYPES[case["dtype"]]
    if not own:
        return s
    import zero_partitioned_mixed_layout_gb300 as zp
    s["zp"] = zp
    if case["op"] in ("norm", "norm_bwd"):
        s["rotary"] = zp.Rotary(s["inv_freq"], interleaved=case["pairs"] == "next")
        s["to"] = torch.empty_like(s["qk"])
        if case["op"] == "norm_bwd":
            s["ws"] = zp.new_qk_norm_workspace(case["tokens"], h, g, d)
            s["dweights"] = torch.empty((2, d), dtype=TYPES[case["gdtype"]], device="cuda")
        return s
    tq, tk = s["q"].shape[0], s["k"].shape[0]
    s["window"] = case["window"] or None
    s["ws"] = zp.new_window_attention_workspace(tq, tk, case["sequences"], h, g, d, window=s["window"],
                                                sinks=case["sinks"], backward=case["op"] == "attn_bwd")
    if case["op"] == "attn":
        s["out"], s["lse"] = torch.empty_like(s["q"]), torch.empty((h, tq), dtype=torch.float32, device="cuda")
    else:
        s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[k]) for k in "qkv")
    return s


# ------------------------------------------------------------------ plain forms

def _angles(s):
    """cos and sin [tokens, 1, pairs] of the rotation, from binary64 angles."""
    f = torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda")
    a = s["positions"].double()[:, None, None] * f
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(x, cos, sin, case):
    r = case["rot"]
    if case["pairs"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _weights(s):
    """The weight of every head's row: the queries', then the keys'."""
    c = s["case"]
    return torch.cat([s["q_weight"].float().expand(c["heads"], -1), s["k_weight"].float().expand(c["kv_heads"], -1)])


def _plain_norm(s):
    case, dt = s["case"], TYPES[s["case"]["dtype"]]
    h = case["heads"]
    cos, sin = _angles(s)
    x, w = s["qk"].float(), _weights(s)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    if case["op"] == "norm":
        y = _rotate(x * rstd * w, cos, sin, case).to(dt)
        return {"q": y[:, :h], "k": y[:, h:]}
    dz, xh = _rotate(s["dqk"].float(), cos, -sin, case), x * rstd
    g = dz * w
    dx = (rstd * (g - xh * (g * xh).mean(-1, keepdim=True))).to(dt)
    dw, gdt = dz * xh, TYPES[case["gdtype"]]
    return {"dq": dx[:, :h], "dk": dx[:, h:], "dq_weight": dw[:, :h].sum((0, 1)).to(gdt),
            "dk_weight": dw[:, h:].sum((0, 1)).to(gdt)}


def _bands(s):
    """The packed queries in blocks of one sequence, and the keys that a block
    may see: (query rows [n, B], which of them are there, key rows [n, J],
    which of them are seen by each query [n, B, J])."""
    case = s["case"]
    rows = case.get("new", case["most"])
    keys, sinks = case["most"], min(case["sinks"], case["most"])
    block = min(256, rows)
    n = -(-rows // block)
    band = min(keys, (case["window"] or keys) + block - 1)
    at = torch.arange(n, device="cuda").repeat(case["sequences"])                      # block of its sequence
    seq = torch.arange(case["sequences"], device="cuda").repeat_interleave(n)
    ql = (s["q_offsets"][1:] - s["q_offsets"][:-1])[seq]
    kl = s["k_lengths"][seq]
    i = at[:, None] * block + torch.arange(block, device="cuda")                       # query of its sequence
    p = i + (kl - ql)[:, None]                                                         # where it stands
    first = (torch.minimum((at + 1) * block, ql) + kl - ql - band)[:, None]            # the band ends with the block
    j = torch.cat([first + torch.arange(band, device="cuda"),
                   torch.arange(sinks, device="cuda").expand(len(at), -1)], 1)
    there = torch.cat([j[:, :band] >= 0, j[:, band:] < first], 1) & (j < kl[:, None])
    near = j[:, None] > p[:, :, None] - (case["window"] or keys + block)
    seen = there[:, None] & (j[:, None] <= p[:, :, None]) & (near | (j[:, None] < sinks))
    live = i < ql[:, None]
    qr = torch.where(live, s["q_offsets"][seq][:, None] + i, 0)
    kr = torch.where(there, s["k_offsets"][seq][:, None] + j, 0)
    return qr, live, kr, seen & live[:, :, None]


def _scores(s, qr, kr, seen):
    """q, k, v of the blocks ([n, key heads, ...]) and their scores, what is not seen at -inf."""
    c = s["case"]
    g, d = c["kv_heads"], c["dim"]
    group = c["heads"] // g
    # [n, g, group * B, d] and [n, g, J, d]
    q = s["q"][qr].float().view(*qr.shape, g, group, d).permute(0, 2, 3, 1, 4).flatten(2, 3)
    k, v = (s[x][kr].float().transpose(1, 2) for x in "kv")
    t = (q @ k.transpose(-1, -2)).mul_(d ** -0.5).unflatten(2, (group, -1))
    return q, k, v, t.masked_fill_(~seen[:, None, None], -math.inf)


def _rows_of(x, s, qr, live):
    """[n, g, group, B, ...] to the packed rows [tokens, heads, ...]."""
    x = x.movedim(3, 1).flatten(2, 3)
    out = torch.empty((s["q"].shape[0], *x.shape[2:]), dtype=x.dtype, device="cuda")
    out[qr[live]] = x[live]
    return out


def _plain_attention(s):
    dt = TYPES[s["case"]["dtype"]]
    qr, live, kr, seen = _bands(s)
    _, _, v, t = _scores(s, qr, kr, seen)
    top = t.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    t = t.sub_(top).exp_()
    total = t.sum(-1, keepdim=True)
    o = (t.flatten(2, 3) @ v).unflatten(2, t.shape[2:4]) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)
    return {"out": _rows_of(o, s, qr, live).to(dt), "lse": _rows_of(lse, s, qr, live).T.contiguous()}


def _plain_attention_bwd(s):
    c, dt = s["case"], TYPES[s["case"]["dtype"]]
    g, d = c["kv_heads"], c["dim"]
    group, scale = c["heads"] // g, c["dim"] ** -0.5
    qr, live, kr, seen = _bands(s)
    q, k, v, t = _scores(s, qr, kr, seen)
    lse = s["lse"].T[qr].view(*qr.shape, g, group).permute(0, 2, 3, 1)[..., None]
    p = t.sub_(torch.where(lse == -math.inf, 0.0, lse)).exp_().flatten(2, 3)
    do, o = (s[x][qr].float().view(*qr.shape, g, group, d).permute(0, 2, 3, 1, 4).flatten(2, 3) for x in ("dout", "out"))
    dv = p.transpose(-1, -2) @ do
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p).mul_(scale)
    dq = (ds @ k).unflatten(2, (group, -1))
    dk = ds.transpose(-1, -2) @ q
    grads = [torch.zeros((s["k"].shape[0], g, d), dtype=torch.float32, device="cuda").index_add_(
        0, kr.flatten(), x.transpose(1, 2).flatten(0, 1)).to(dt) for x in (dk, dv)]
    return {"dq": _rows_of(dq, s, qr, live).to(dt), "dk": grads[0], "dv": grads[1]}


def run(s):
    case = s["case"]
    op = case["op"]
    if not own:
        return _plain_attention(s) if op == "attn" else _plain_attention_bwd(s) if op == "attn_bwd" else _plain_norm(s)
    zp, h = s["zp"], case["heads"]
    if op == "norm":
        x, y = s["qk"], s["to"]
        q, k = y[:, :h], y[:, h:]
        zp.zero_qk_norm(x[:, :h], x[:, h:], s["q_weight"], s["k_weight"], q, k, rotary=s["rotary"],
                        positions=s["positions"], eps=EPS)
        return {"q": q, "k": k}
    if op == "norm_bwd":
        x, dy, dx = s["qk"], s["dqk"], s["to"]
        dq, dk = dx[:, :h], dx[:, h:]
        dqw, dkw = s["dweights"]
        zp.zero_qk_norm_backward(dy[:, :h], dy[:, h:], x[:, :h], x[:, h:], s["q_weight"], s["k_weight"], dq, dk, dqw,
                                 dkw, s["ws"], rotary=s["rotary"], positions=s["positions"], eps=EPS)
        return {"dq": dq, "dk": dk, "dq_weight": dqw, "dk_weight": dkw}
    where = dict(window=s["window"], sinks=case["sinks"], q_offsets=s["q_offsets"], k_offsets=s["k_offsets"],
                 k_lengths=s["k_lengths"])
    if op == "attn":
        zp.zero_window_attention(s["q"], s["k"], s["v"], s["out"], s["ws"], lse=s["lse"], **where)
        return {"out": s["out"], "lse": s["lse"]}
    zp.zero_window_attention_backward(s["dout"], s["q"], s["k"], s["v"], s["out"], s["lse"], s["dq"], s["dk"], s["dv"],
                                      s["ws"], **where)
    return {"dq": s["dq"], "dk": s["dk"], "dv": s["dv"]}


# ------------------------------------------------------------------ what a pass cannot do without

def _visible(case):
    """(pairs of a query and a key that it sees, keys that any query sees) over all sequences, for one head."""
    def low(p, lk):  # the first key of a window that ends with key p
        return (p + 1 - (case["window"] or lk)).clamp(min=0)

    def pairs(lq, lk):
        p = torch.arange(lk - lq, lk)
        return int((p + 1 - low(p, lk) + low(p, lk).clamp(max=case["sinks"])).sum())

    def keys(lq, lk):
        first = int(low(torch.tensor(lk - lq), lk))
        return lk - first + min(first, case["sinks"])

    lengths = list(zip(*_lengths(case)))
    return sum(pairs(*x) for x in lengths), sum(keys(*x) for x in lengths)


def work(case):
    e, h, g, d = BYTES[case["dtype"]], case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("norm", "norm_bwd"):
        n, w = case["tokens"] * (h + g) * d, 2 * BYTES[case["wdtype"]] * d
        if case["op"] == "norm":  # x, y; weights; positions
            return {"bytes": 2 * e * n + w + 8 * case["tokens"], "flops": 8.0 * n}
        # x, dy, dx; weights and their gradients; positions
        return {"bytes": 3 * e * n + w + 2 * BYTES[case["gdtype"]] * d + 8 * case["tokens"], "flops": 16.0 * n}
    pairs, keys = _visible(case)
    rows = sum(_lengths(case)[0])
    if case["op"] == "attn":  # q, out; k, v; lse
        return {"bytes": 2 * e * d * (rows * h + keys * g) + 4 * rows * h, "flops": 4.0 * d * pairs * h}
    # q, out, dout, dq; k, v, dk, dv; lse
    return {"bytes": 4 * e * d * (rows * h + keys * g) + 4 * rows * h, "flops": 10.0 * d * pairs * h}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_norm(case, s):
    """The rotation as a product of complex numbers."""
    t, h, d, r = case["tokens"], case["heads"], case["dim"], case["rot"]
    x = s["qk"].double()
    w = torch.empty((h + case["kv_heads"], d), dtype=torch.float64, device="cuda")
    w[:h], w[h:] = s["q_weight"].double(), s["k_weight"].double()
    angle = torch.outer(s["positions"].double(), torch.tensor(s["inv_freq"], dtype=torch.float64, device="cuda"))
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotated(z, by):
        z = z.clone()
        part = z[..., :r].unflatten(-1, (2, r // 2) if case["pairs"] == "half" else (r // 2, 2))
        axis = -2 if case["pairs"] == "half" else -1
        c = torch.complex(part.select(axis, 0).contiguous(), part.select(axis, 1).contiguous()) * by
        part.select(axis, 0).copy_(c.real)
        part.select(axis, 1).copy_(c.imag)
        return z

    size = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
    if case["op"] == "norm":
        y = rotated(x / size * w, turn)
        return {"q": y[:, :h], "k": y[:, h:]}
    dz = rotated(s["dqk"].double(), turn.conj())
    dw = torch.einsum("thd,thd->hd", dz, x / size)
    dx = dz * w / size - x * ((dz * w * x).sum(-1, keepdim=True) / (d * size ** 3))
    return {"dq": dx[:, :h], "dk": dx[:, h:], "dq_weight": dw[:h].sum(0), "dk_weight": dw[h:].sum(0)}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] in ("norm", "norm_bwd"):
        return _exact_norm(case, s)
    # attention: a sequence, a key head and 1024 queries at a time, over the keys up to the last of them
    if work(case)["flops"] > 4e12:
        return None
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    group, back = h // g, case["op"] == "attn_bwd"
    q, k, v = (s[x].double() for x in "qkv")
    out, lse = torch.zeros_like(q), torch.empty((h, q.shape[0]), dtype=torch.float64, device="cuda")
    if back:
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        do, o, kept = s["dout"].double(), s["out"].double(), s["lse"].double()
    starts = s["k_offsets"].tolist()
    q0 = 0
    for seq, (lq, lk) in enumerate(zip(*_lengths(case))):
        for i0 in range(0, lq, 1024):
            i1 = min(lq, i0 + 1024)
            at = torch.arange(i0 + lk - lq, i1 + lk - lq, device="cuda")[:, None]
            first = max(0, i0 + lk - lq + 1 - case["window"]) if case["window"] else 0
            j = torch.arange(i1 + lk - lq, device="cuda")
            j = j[(j >= first) | (j < case["sinks"])]
            hidden = (j > at) | ((j <= at - (case["window"] or lk)) & (j >= case["sinks"]))
            rows, cols = slice(q0 + i0, q0 + i1), starts[seq] + j
            for m in range(g):
                hs = slice(m * group, m * group + group)
                kk, vv = k[cols, m], v[cols, m]
                t = torch.einsum("ihd,jd->hij", q[rows, hs], kk) / math.sqrt(d)
                t[:, hidden] = -math.inf
                if not back:
                    lse[hs, rows] = torch.logsumexp(t, -1)
                    out[rows, hs] = torch.einsum("hij,jd->ihd", torch.softmax(t, -1), vv)
                    continue
                p = torch.exp(t - kept[hs, rows, None])
                dv[cols, m] += torch.einsum("hij,ihd->jd", p, do[rows, hs])
                dp = torch.einsum("ihd,jd->hij", do[rows, hs], vv)
                dt = p * (dp - (do[rows, hs] * o[rows, hs]).sum(-1).T[..., None]) / math.sqrt(d)
                dq[rows, hs] = torch.einsum("hij,jd->ihd", dt, kk)
                dk[cols, m] += torch.einsum("hij,ihd->jd", dt, q[rows, hs])
        q0 += lq
    return {"dq": dq, "dk": dk, "dv": dv} if back else {"out": out, "lse": lse}
