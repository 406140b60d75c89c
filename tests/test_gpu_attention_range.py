"""The attention kernels at the ends of their types' ranges: scores up to
10^9, weights and gradients far below and above what 16 bits hold unscaled.
The bounds are derived beside each test, from the formulas in binary64."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_ref as ref  # noqa: E402
from test_gpu_attention import Batch, randn, zp  # noqa: E402, F401

U32, UT = ref.U32, ref.UT


# ------------------------------------------------------------------ one key takes all

class Dominated(Batch):
    """Each query has one element that is not zero, so that its scores are
    single products, exact in binary32 before the scale; of every element one
    key, which all queries see, holds more than twice what any other does.  So
    P is 1 for that key and 0 for the others (their scores are lower by a
    third of the largest, at least 1000)."""

    def __init__(self, lens, heads, kv, dim, dtype, size, scale):
        super().__init__([lens], heads, kv, dim, dtype, std=0.0)
        gen = torch.Generator(device="cuda").manual_seed(int(size))
        (lq, lk), each = lens, math.sqrt(size / scale)

        def uniform(lo, hi, *shape):
            return torch.empty(shape, device="cuda").uniform_(lo * each, hi * each, generator=gen).to(self.dt)
        self.element = torch.arange(lq, device="cuda")[:, None] * 7 % dim + torch.zeros((lq, heads), dtype=torch.int64, device="cuda")
        self.q.zero_().scatter_(2, self.element[..., None], uniform(0.6, 1.0, lq, heads, 1))
        self.k.copy_(uniform(-0.35, 0.35, lk, kv, dim))
        self.winner = torch.randint(0, lk - lq + 1, (kv, dim), device="cuda", generator=gen)  # [key head, element]
        self.k.scatter_(0, self.winner[None], uniform(0.75, 1.0, 1, kv, dim))
        group = heads // kv
        head = torch.arange(heads, device="cuda") // group
        self.key = self.winner[head[None], self.element]  # [query, head]: the key that takes all
        self.key_head = head.expand(lq, heads)
        self.scale = scale

    def score(self):
        k = self.k.double()[self.key, self.key_head]
        return (self.q.double() * k).sum(-1) * self.scale


DOMINATED = [(1e4, 0.1), (1e5, 0.1), (1e6, 0.125), (1e7, 0.7), (1e8, 0.7), (1e9, 0.7)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [(150, 400), (4, 400)], ids=["many", "few"])
@pytest.mark.parametrize("size,scale", DOMINATED, ids=str)
def test_one_key_takes_all_forward(zp, size, scale, lens, dim, dtype):  # noqa: F811
    b = Dominated(lens, 4, 2, dim, dtype, size, scale)
    out, lse = b.forward(zp, None, 0, scale)
    # out: the weight's rounding to 16 bits, the quotient and the output's own rounding; no term with the score
    v = b.v.double()[b.key, b.key_head]
    ref.check(out.t, v, ref.rounded(v, v.abs() * (UT[b.dt] + 16 * U32), b.dt), "out")
    # lse: the scale's, the product's and the sum's rounding, and the logarithm's of a sum that is 1
    s = b.score().T
    ref.check(lse, s, 3 * U32 * s.abs() + 32 * U32, "lse")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens", [(150, 400), (4, 400)], ids=["many", "few"])
@pytest.mark.parametrize("size,scale", DOMINATED, ids=str)
def test_one_key_takes_all_backward(zp, size, scale, lens, dim, dtype):  # noqa: F811
    """P is 1 whatever the score's size: lse is the rounded product that the
    backward pass forms again."""
    b = Dominated(lens, 4, 2, dim, dtype, size, scale)
    out, lse = b.forward(zp, None, 0, scale)
    b.dout.mul_(0.01)
    out.t.mul_(0.5)  # (so that dP - delta is no difference of equal numbers)
    ws = b.workspace(zp, None, 0, True)
    g = [torch.empty_like(x) for x in (b.q, b.k, b.v)]
    zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out.t, lse, *g, ws, None, 0, scale, **b.where)
    do, o, q, k, v = (x.double() for x in (b.dout, out.t, b.q, b.k, b.v))
    vw, kw = v[b.key, b.key_head], k[b.key, b.key_head]
    ds = (do * vw).sum(-1) - (do * o).sum(-1)
    # dP and delta: binary32 sums (which may truncate) of exact products; P: 16 roundings; dS: one to 16 bits
    eds = ((do * vw).abs().sum(-1) * 2 + (do * o).abs().sum(-1)) * (dim * U32) + ds.abs() * (UT[b.dt] + 24 * U32) + ref.TINY[b.dt]
    ep = UT[b.dt] + 16 * U32
    dq = (ds[..., None] * kw * scale, (eds[..., None] + ds.abs()[..., None] * 4 * U32) * kw.abs() * scale)

    def by_key(x):
        to = torch.zeros_like(k)
        return to.index_put_((b.key, b.key_head), x, accumulate=True)
    n = 2 * lens[0] * U32  # the sums over queries
    dk = by_key(ds[..., None] * q) * scale, by_key((eds[..., None] + ds.abs()[..., None] * n) * q.abs()) * scale
    dv = by_key(do), by_key(do.abs() * (ep + n))
    for name, got, (value, err) in zip(("dq", "dk", "dv"), g, (dq, dk, dv)):
        ref.check(got, value, ref.rounded(value, err + 4 * U32 * value.abs(), b.dt), name)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 80, 128])
@pytest.mark.parametrize("std", [100.0, 1000.0])
def test_scores_that_binary32_rounds_are_the_same_in_both_passes(zp, std, dim, dtype):  # noqa: F811
    """Sums of random products of up to 10^8, which one more or one less
    rounding changes by up to 8: lse is of the very scores that the backward
    pass forms, so that the P of a key that takes all is 1 all the same.  (dv
    of a gradient of 1 in one element adds up P.)"""
    b = Batch([(300, 300), (200, 400)], 4, 2, dim, dtype, std=std)
    out, lse = b.forward(zp, None, 0, 1.0)
    want = torch.zeros((b.tk, 2), dtype=torch.float64, device="cuda")
    b.dout.zero_()
    for qs, ks in b.slices():
        s = torch.einsum("ihd,jhd->hij", b.q[qs].double(), b.k[ks].double().repeat_interleave(2, 1))
        s.masked_fill_(~ref.seen(qs.stop - qs.start, ks.stop - ks.start, None, 0, "cuda"), -math.inf)
        top, key = s.topk(min(2, s.shape[2]), -1)
        # by so much that binary32's sums (off by 2 dim u32 of 4 std^2 sqrt(dim) at most) leave it more than 100 above the next
        clear = ~(top[..., 0] - top[..., 1] < 100 + 2 * (2 * dim * U32) * 16 * std ** 2 * dim ** 0.5)
        b.dout[qs, :, 0] = clear.T.to(b.dt)
        for h in range(4):
            want[ks, h // 2] += torch.bincount(key[h, clear[h], 0], minlength=ks.stop - ks.start).double()
    assert float(want.sum()) > 100
    ws = b.workspace(zp, None, 0, True)
    g = [torch.zeros_like(x) for x in (b.q, b.k, b.v)]
    zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out.t, lse, *g, ws, None, 0, 1.0, **b.where)
    # whole numbers of ones, each rounded to 16 bits as it is: one rounding of the sum
    ref.check(g[2][..., 0], want, ref.rounded(want, want * 16 * U32, b.dt), "dv")


# ------------------------------------------------------------------ weights far below the largest

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("few", [False, True], ids=["many", "few"])
@pytest.mark.parametrize("below", [17.5, 16.5, 13.0])
def test_many_keys_far_below_another(zp, below, few, dim, dtype):  # noqa: F811
    """A key of weight 1 among others of exp(-below) each, about 2^-25 at 17.5:
    what those add up to is in out as it is in lse.  The one key comes before
    most of the others in either kernel's order, and in one part of them."""
    heads, queries, n, lens = (32, 1, 1024, [(1, 1025)] * 64) if few else (2, 20, 65536, [(20, 65556)])
    b = Batch(lens, heads, heads, dim, dtype)
    for x in (b.q, b.k, b.v):
        x.zero_()
    b.q[..., 0] = 1.0
    b.v.fill_(1.0)
    one = torch.tensor([ks.start if few else ks.stop - queries for _, ks in b.slices()], device="cuda")
    b.k[one, :, 0] = below
    b.v[one] = 0.0
    out, lse = b.forward(zp, None, 0, 1.0)
    # queries see the one key and n others, and each one more than the query before it
    others = (n + torch.arange(queries, dtype=torch.float64, device="cuda")).repeat(len(lens))[:, None]
    w = others * math.exp(-below)
    want = (w / (1 + w))[..., None].expand(-1, heads, dim)
    # each weight: the exponent's and the exponential's own errors, and one rounding to 16 bits of 2^7 times it (half a
    # step of f16's subnormals is 2^-32 of the weight 1); sums of at most 1024 terms' chains that may truncate
    step = 2.0 ** -32 if dtype == "f16" else 0.0
    err = want * (UT[b.dt] + (4 * below + 16 + 2 * 1024) * U32) + (others * step)[..., None]
    ref.check(out.t, want, ref.rounded(want, err, b.dt), "out")
    ref.check(lse, (below + torch.log1p(w)).T.expand(heads, -1), torch.full_like(lse, 2048 * U32 + 4 * below * U32, dtype=torch.float64), "lse")


# ------------------------------------------------------------------ small and large gradients

def sequence_backward(b, qs, ks, out, lse, window, sinks, scale, rows):
    """dq, dk, dv of one sequence from the formulas in binary64, and what
    binary32 may do to them: the errors of S, dP and delta (sums of d exact
    products that may truncate) in each pair, independent from pair to pair.
    rows: dq is to be compared row by row, where the roundings of dS are as few
    as a row's keys (of the first rows' one or two to a head) and no mean:
    each may be half a step, where the mean is 0.39 of one."""
    group, d = b.heads // b.kv, b.dim
    q, do, o = (x[qs].double() for x in (b.q, b.dout, out))
    k, v = (x[ks].double() for x in (b.k, b.v))
    mask = ref.seen(q.shape[0], k.shape[0], window, sinks, "cuda")
    r = {n: torch.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v))}
    e = {n: torch.zeros_like(x) for n, x in r.items()}  # squares
    for h in range(b.heads):
        g = h // group
        p = torch.exp((q[:, h] @ k[:, g].T) * scale - lse[h, qs].double()[:, None]).masked_fill_(~mask, 0.0)
        delta = (do[:, h] * o[:, h]).sum(-1, keepdim=True)
        ds = p * (do[:, h] @ v[:, g].T - delta)
        ep = p * ((q[:, h].abs() @ k[:, g].abs().T) * scale * (2 * d * U32) + 32 * U32)
        eds = p * (do[:, h].abs() @ v[:, g].abs().T * (2 * d * U32) + (do[:, h] * o[:, h]).abs().sum(-1, keepdim=True) * (d * U32)) + \
            ep * (ds / p.clamp(min=1e-300)).abs()
        r["dq"][:, h] = scale * ds @ k[:, g]
        r["dk"][:, g] += scale * ds.T @ q[:, h]
        r["dv"][:, g] += p.T @ do[:, h]
        half = (UT[b.dt] * ds).square() if rows else 0.0
        e["dq"][:, h] = scale ** 2 * (eds.square() + half) @ k[:, g].square()
        e["dk"][:, g] += scale ** 2 * eds.square().T @ q[:, h].square()
        e["dv"][:, g] += ep.square().T @ do[:, h].square()
    return r, e


def norm_wise(got, want, square, dtype, what, axes):
    """Against the exact result rounded once.  The products' operands are
    rounded once before (each by a relative error of the same distribution,
    independent from term to term), and the output once: the square root of
    two times the error of the output's rounding alone, for which 2 stands."""
    off = (got.double() - want).square().sum(axes).sqrt()
    # (of a value that 16 bits hold the operands were rounded all the same; 0.39 of half a step is the mean over all mantissas)
    once = torch.maximum((want.to(dtype).double() - want).square().sum(axes).sqrt(),
                         0.39 * UT[dtype] * want.square().sum(axes).sqrt())
    assert bool(torch.isfinite(got).all()), what
    assert bool((off <= 2 * once + square.sum(axes).sqrt()).all()), (what, float((off / once).max()))


def check_norm_wise(zp, b, window, sinks, rows=False):  # noqa: F811
    scale = b.dim ** -0.5
    out, lse = b.forward(zp, window, sinks, scale)
    ws = b.workspace(zp, window, sinks, True)
    g = dict(zip(("dq", "dk", "dv"), (torch.zeros_like(x) for x in (b.q, b.k, b.v))))
    zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out.t, lse, *g.values(), ws, window, sinks, scale, **b.where)
    assert zp.zero_workspace_stalls(ws) == 0
    for qs, ks in b.slices():
        want, square = sequence_backward(b, qs, ks, out.t, lse, window, sinks, scale, rows)
        for name, at in (("dq", qs), ("dk", ks), ("dv", ks)):
            norm_wise(g[name][at], want[name], square[name], b.dt, f"{name} {at}",
                      (1, 2) if rows and name == "dq" else (0, 1, 2))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("std", [1.0, 1e-2, 1e-3, 1e-4])
def test_small_gradients_over_many_keys(zp, std, dim, dtype):  # noqa: F811
    """P is about 1 / keys and dS a 4096th of the gradients, which 16 bits do
    not hold as they are; dq, dk and dv are sums that they hold."""
    b = Batch([(4096, 4096)], 4, 2, dim, dtype)
    b.dout.copy_(randn(b.dout.shape, torch.float32, 9, std))
    check_norm_wise(zp, b, None, 0)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_small_gradients_of_first_keys_in_parts(zp, dim, dtype):  # noqa: F811
    """The same where the first keys' queries are dealt out."""
    b = Batch([(3000, 3000), (500, 700)], 4, 1, dim, dtype)
    b.dout.copy_(randn(b.dout.shape, torch.float32, 9, 1e-3))
    check_norm_wise(zp, b, 130, 4)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_large_gradients(zp, dim, dtype):  # noqa: F811
    """dP past 65504 (a scaled loss), over keys and queries so small that dq
    and dk are not."""
    b = Batch([(300, 300), (70, 200)], 4, 2, dim, dtype, std=0.05)
    b.v.mul_(8.0)
    b.dout.mul_(4000.0)
    check_norm_wise(zp, b, None, 0)
    check_norm_wise(zp, b, 40, 3)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
def test_gradients_of_many_sizes_in_one_call(zp, dim, dtype):  # noqa: F811
    """Sequences whose gradients are 10^5 apart, and rows within one that are
    a thousand apart: each sequence's dk and dv, and each row's dq, are as near
    as by themselves."""
    b = Batch([(1000, 1000), (900, 1200), (130, 130)], 4, 2, dim, dtype)
    rows = torch.empty((b.tq, 1, 1), device="cuda").uniform_(-3, 0, generator=torch.Generator(device="cuda").manual_seed(3))
    for (qs, _), size in zip(b.slices(), (100.0, 1e-3, 1.0)):
        rows[qs] = 10 ** rows[qs] * size
    b.dout.copy_(randn(b.dout.shape, torch.float32, 9) * rows)
    b.dout[5:40] = 0.0  # (and rows without any)
    check_norm_wise(zp, b, None, 0, rows=True)
    check_norm_wise(zp, b, 200, 4, rows=True)


@pytest.mark.parametrize("dim", [64, 128])
def test_dq_is_whole_when_the_waits_before_it_give_up(zp, dim):  # noqa: F811
    """dk's and dv's kernel tells dq's how large the values are, also when its
    own waits ran out (bounded, as the test of each kernel's waits has them)."""
    import ctypes
    hook = zp.lib().zero_test_window_attention_waits
    hook.argtypes, hook.restype = [ctypes.c_int32, ctypes.c_uint64], None
    b = Batch([(300, 300), (200, 400)], 4, 2, dim, "f16")
    out, lse = b.forward(zp, 100, 2)
    runs = []
    for kernel in (-1, 1):
        ws = b.workspace(zp, 100, 2, True)
        g = [torch.zeros_like(x) for x in (b.q, b.k, b.v)]
        hook(kernel, 20_000_000)
        try:
            zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out.t, lse, *g, ws, 100, 2, **b.where)
            stalls = zp.zero_workspace_stalls(ws)
        finally:
            hook(-1, 0)
        assert (stalls > 0) == (kernel == 1)
        runs.append(g)
    assert bool(torch.isnan(runs[1][1]).all()) and bool(torch.isnan(runs[1][2]).all())
    assert torch.equal(runs[0][0], runs[1][0])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("what", [math.inf, -math.inf, math.nan], ids=str)
def test_a_gradient_that_overflowed_shows(zp, what, dim, dtype):  # noqa: F811
    """An element of dout that is no number: its query's dq, and dk and dv of
    the keys that it sees, are none either (so that a scaled loss is found to
    be too large), and other sequences' are what they were, to the bit."""
    b = Batch([(200, 200), (300, 400), (70, 70)], 4, 2, dim, dtype)
    out, lse = b.forward(zp, 90, 2)
    ws, runs = b.workspace(zp, 90, 2, True), []
    for value in (None, what):
        if value is not None:
            b.dout[300, 1, 5] = value  # (query 100 of the second sequence, at key 200)
        g = [torch.zeros_like(x) for x in (b.q, b.k, b.v)]
        zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out.t, lse, *g, ws, 90, 2, **b.where)
        runs.append(g)
    assert zp.zero_workspace_stalls(ws) == 0
    dq, dk, dv = runs[1]
    assert not bool(torch.isfinite(dq[300, 1]).any())
    seen = torch.cat([torch.arange(2), torch.arange(111, 201)]) + 200
    assert not bool(torch.isfinite(dk[seen, 0]).any()) and not bool(torch.isfinite(dv[seen, 0, 5]).any())
    for (before, after), parts in zip(zip(*runs), (((0, 200), (500, 570)), ((0, 200), (600, 670)), ((0, 200), (600, 670)))):
        for a, e in parts:
            assert torch.equal(before[a:e], after[a:e])
