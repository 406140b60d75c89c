"""The attention sub-block on the GPU against its formulas in binary64
(attention_ref.py, which also derives each bound), at the sizes, layouts,
masks and values where the kernels can go wrong."""
import math
import random

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import attention_ref as ref  # noqa: E402

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def zp():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from zero_partitioned_mixed_layout_gb300 import _build
    _build.build()
    import zero_partitioned_mixed_layout_gb300 as zp
    zp.lib()
    return zp


def randn(shape, dtype, seed, std=1.0, mean=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(mean, std, generator=gen).to(dtype)


def close(got, want, dtype, what):
    value, err = want
    ref.check(got, value, ref.rounded(value, err, dtype), what)


def placed(shape, dtype, layout, fill):
    """A tensor [tokens, heads, dim] in a buffer of `fill`, and the buffer:
    packed; a slice of a wider projection; heads before tokens; from an odd
    element on."""
    t, h, d = shape
    if layout == "packed":
        buf = torch.full((t, h, d), fill, dtype=dtype, device="cuda")
        return buf, buf
    if layout == "slice":
        buf = torch.full((t, h + 3, d), fill, dtype=dtype, device="cuda")
        return buf[:, 2:2 + h], buf
    if layout == "heads_first":
        buf = torch.full((h, t + 5, d), fill, dtype=dtype, device="cuda")
        return buf.transpose(0, 1)[3:3 + t], buf
    buf = torch.full((t * h * (d + 1) + 8,), fill, dtype=dtype, device="cuda")  # odd
    return buf[1:1 + t * h * (d + 1)].view(t, h, d + 1)[..., :d], buf


def put(x, layout):
    v, _ = placed(x.shape, x.dtype, layout, math.nan)
    return v.copy_(x)


class Out:
    """An output in a buffer of sentinels."""

    def __init__(self, shape, dtype, layout="packed"):
        self.t, self.buf = placed(shape, dtype, layout, 77.0)
        self.shape, self.layout = shape, layout

    def only(self, rows=None):
        """Whether nothing but it (of its rows: `rows`, a bool per token) changed."""
        before = self.buf.clone()
        if rows is None:
            self.t.fill_(77.0)
        else:
            self.t[rows] = 77.0
        ok = bool((self.buf == 77.0).all())
        self.buf.copy_(before)
        return ok


# ------------------------------------------------------------------ norms of queries and keys

# tokens, query heads, key heads, head dim, rotated, layout: every width of a
# piece, rows of one lane to several pieces per lane, rotations of a part
QK = [(1, 1, 1, 64, 64, "packed"), (1, 25, 25, 64, 64, "packed"), (7, 3, 1, 128, 128, "slice"), (33, 5, 2, 80, 40, "packed"),
      (5, 2, 2, 96, 96, "heads_first"), (9, 4, 4, 256, 256, "slice"), (3, 2, 1, 250, 100, "packed"), (4, 3, 3, 50, 20, "slice"),
      (6, 2, 1, 33, 6, "packed"), (8, 1, 1, 1, 0, "packed"), (5, 2, 2, 2, 2, "packed"), (11, 3, 2, 8, 4, "packed"),
      (13, 2, 1, 64, 32, "odd"), (3, 1, 2, 128, 0, "packed"), (2, 1, 1, 251, 250, "packed"), (700, 9, 3, 64, 64, "slice"),
      (5000, 2, 1, 32, 32, "packed"), (4, 1, 0, 64, 64, "packed"), (6, 70, 3, 16, 16, "packed")]


def qk_case(shape, dtype, wdtype, seed=1):
    t, h, g, d, rot, layout = shape
    freq = [100.0 ** (-2 * i / max(rot, 1)) for i in range(rot // 2)]
    rng = random.Random(t * 1000 + d)
    pos = [rng.choice([i, rng.randint(-2000, 10 ** 6)]) for i in range(t)]
    c = dict(q=randn((t, h, d), dtype, seed), k=randn((t, g, d), dtype, seed + 1, 3.0, 0.5),
             qw=randn((d,), wdtype, seed + 2, 0.3, 1.0), kw=randn((d,), wdtype, seed + 3, 0.3, -1.0))
    return c, freq, pos, ref.angles(pos, freq)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairs", ["half", "next"])
@pytest.mark.parametrize("shape", QK, ids=str)
def test_qk_norm(zp, shape, pairs, dtype):
    t, h, g, d, rot, layout = shape
    dt = TYPES[dtype]
    c, freq, pos, angle = qk_case(shape, dt, dt)
    rotary = zp.Rotary(freq, interleaved=pairs == "next") if rot else None
    positions = torch.tensor(pos, device="cuda") if rot else None
    qo, ko = Out((t, h, d), dt, layout), Out((t, g, d), dt, layout)
    zp.zero_qk_norm(put(c["q"], layout), put(c["k"], layout), c["qw"], c["kw"], qo.t, ko.t, rotary, positions, 1e-6)
    for o, x, w in ((qo, c["q"], c["qw"]), (ko, c["k"], c["kw"])):
        close(o.t, ref.head_norm(x, w, angle, pos, rot, pairs == "next", 1e-6), dt, "out")
        assert o.only()


@pytest.mark.parametrize("gdtype", ["own", "f32"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairs", ["half", "next"])
@pytest.mark.parametrize("shape", QK, ids=str)
def test_qk_norm_backward(zp, shape, pairs, dtype, gdtype):
    t, h, g, d, rot, layout = shape
    dt = TYPES[dtype]
    gt = dt if gdtype == "own" else torch.float32
    c, freq, pos, angle = qk_case(shape, dt, torch.float32 if gdtype == "f32" else dt, 11)
    gq, gk = randn((t, h, d), dt, 21), randn((t, g, d), dt, 22)
    rotary = zp.Rotary(freq, interleaved=pairs == "next") if rot else None
    positions = torch.tensor(pos, device="cuda") if rot else None
    dq, dk = Out((t, h, d), dt, layout), Out((t, g, d), dt, layout)
    dw = torch.full((2, d + 6), 77.0, dtype=gt, device="cuda")
    ws = zp.new_qk_norm_workspace(t, h, g, d)
    args = (put(gq, layout), put(gk, layout), put(c["q"], layout), put(c["k"], layout), c["qw"], c["kw"])
    for _ in range(2):  # (the workspace serves again)
        zp.zero_qk_norm_backward(*args, dq.t, dk.t, dw[0, 3:3 + d], dw[1, 3:3 + d], ws, rotary, positions, 1e-6)
    assert bool((dw[:, :3] == 77).all()) and bool((dw[:, 3 + d:] == 77).all())
    for o, w, x, dy, n in ((dq, c["qw"], c["q"], gq, 0), (dk, c["kw"], c["k"], gk, 1)):
        r = ref.head_norm_backward(dy, x, w, angle, pos, rot, pairs == "next", 1e-6)
        close(o.t, r["dx"], dt, f"dx {n}")
        close(dw[n, 3:3 + d], r["dw"], gt, f"dw {n}")
        assert o.only()


def test_qk_norm_in_place_without_weights(zp):
    x = randn((300, 8, 64), torch.float16, 5)
    freq = [0.5 ** i for i in range(16)]
    rotary = zp.Rotary(freq)
    pos = list(range(300))
    want = ref.head_norm(x, None, ref.angles(pos, freq), pos, 32, False, 1e-5)
    both = x.clone()
    zp.zero_qk_norm(both[:, :6], both[:, 6:], None, None, both[:, :6], both[:, 6:], rotary, None, 1e-5)
    close(both, want, torch.float16, "positions 0, 1, 2 ...")
    g = randn((300, 8, 64), torch.float16, 6)
    r = ref.head_norm_backward(g, x, None, ref.angles(pos, freq), pos, 32, False, 1e-5)
    for out in ("dout", "x"):  # dx takes the place of either
        a, b = x.clone(), g.clone()
        to = b if out == "dout" else a
        zp.zero_qk_norm_backward(b[:, :6], b[:, 6:], a[:, :6], a[:, 6:], None, None, to[:, :6], to[:, 6:], None, None,
                                 zp.new_qk_norm_workspace(300, 6, 2, 64), rotary, None, 1e-5)
        close(to, r["dx"], torch.float16, out)


def test_qk_norm_far_positions(zp):
    """Angles of positions up to 2^40, of either sign, as exact as near ones."""
    freq = [1.0, 0.9, 1e-3, 1e-6, 3.0, 0.1, 1e-9, 1e5]
    pos = [2 ** 31 - 1, -2 ** 31, 10 ** 9, 2 ** 40 + 1, -2 ** 40, 12345678901, 0, 1]
    x = randn((len(pos), 4, 16), torch.float32, 7)
    for inter in (False, True):
        y = torch.empty_like(x)
        zp.zero_qk_norm(x, x[:, :0], None, None, y, y[:, :0], zp.Rotary(freq, inter), torch.tensor(pos, device="cuda"), 0.0)
        close(y, ref.head_norm(x, None, ref.angles(pos, freq), pos, 16, inter, 0.0), torch.float32, str(inter))


def test_qk_norm_rows_that_are_not_numbers_stay_apart(zp):
    x = randn((40, 6, 64), torch.bfloat16, 8)
    bad = torch.zeros(40, 6, dtype=torch.bool, device="cuda")
    x[3, 2, 5], x[17, 0, 63], x[39, 5, 0] = math.nan, math.inf, -math.inf
    bad[3, 2] = bad[17, 0] = bad[39, 5] = True
    y, dx, dw = torch.empty_like(x), torch.empty_like(x), torch.empty(64, dtype=torch.float32, device="cuda")
    rotary = zp.Rotary([0.3 ** i for i in range(32)])
    zp.zero_qk_norm(x[:, :4], x[:, 4:], None, None, y[:, :4], y[:, 4:], rotary, None)
    zp.zero_qk_norm_backward(x[:, :4], x[:, 4:], x[:, :4], x[:, 4:], None, None, dx[:, :4], dx[:, 4:], dw, None,
                             zp.new_qk_norm_workspace(40, 4, 2, 64), rotary, None)
    for t in (y, dx):
        assert torch.equal(torch.isnan(t).any(-1), bad)
    zero = torch.zeros_like(x)
    zp.zero_qk_norm(zero[:, :4], zero[:, 4:], None, None, y[:, :4], y[:, 4:], rotary, None)
    assert bool((y == 0).all())


def test_qk_norm_sums_are_the_same_on_every_run(zp):
    x, g = randn((4097, 12, 64), torch.float16, 9), randn((4097, 12, 64), torch.float16, 10)
    ws, runs = zp.new_qk_norm_workspace(4097, 8, 4, 64), []
    for _ in range(20):
        dx, dw = torch.empty_like(x), torch.empty((2, 64), dtype=torch.float32, device="cuda")
        zp.zero_qk_norm_backward(g[:, :8], g[:, 8:], x[:, :8], x[:, 8:], None, None, dx[:, :8], dx[:, 8:], dw[0], dw[1],
                                 ws, zp.Rotary([0.1 ** i for i in range(32)]), None)
        runs.append(dw)
    assert all(torch.equal(r, runs[0]) for r in runs)
    # without tokens the sums are empty
    none = torch.empty((0, 8, 64), dtype=torch.float16, device="cuda")
    zp.zero_qk_norm_backward(none, none, none, none, None, None, none, none, dw[0], dw[1], ws)
    assert bool((dw == 0).all())


# ------------------------------------------------------------------ attention

class Batch:
    """Sequences of (queries, keys): packed, each sequence's keys at the head
    of a room of its own `room` rows larger, `behind` rows after the last."""

    def __init__(self, lens, heads, kv, dim, dtype, seed=1, room=0, behind=0, layout="packed", fill=math.nan, std=1.0):
        self.lens, self.heads, self.kv, self.dim, self.dt = lens, heads, kv, dim, TYPES[dtype]
        ql, kl = [a for a, _ in lens], [b for _, b in lens]
        self.q0 = [sum(ql[:i]) for i in range(len(lens) + 1)]
        self.k0 = [sum(kl[:i]) + room * i for i in range(len(lens) + 1)]
        self.tq, self.tk = self.q0[-1] + behind, self.k0[-1] + behind
        self.q = put(randn((self.tq, heads, dim), self.dt, seed, std), layout)
        self.k = put(randn((self.tk, kv, dim), self.dt, seed + 1, std), layout)
        self.v = put(randn((self.tk, kv, dim), self.dt, seed + 2), layout)
        self.dout = put(randn((self.tq, heads, dim), self.dt, seed + 3), layout)
        self.live = torch.zeros(self.tq, dtype=torch.bool, device="cuda")
        self.keyed = torch.zeros(self.tk, dtype=torch.bool, device="cuda")
        self.live[:self.q0[-1]] = True
        for a, b in zip(self.k0, kl):
            self.keyed[a:a + b] = True
        # what lies outside every sequence is not to matter
        for t, rows in ((self.q, self.live), (self.dout, self.live), (self.k, self.keyed), (self.v, self.keyed)):
            t[~rows] = fill
        dev = dict(dtype=torch.int64, device="cuda")
        self.where = dict(q_offsets=torch.tensor(self.q0, **dev), k_offsets=torch.tensor(self.k0, **dev),
                          k_lengths=torch.tensor(kl, **dev))
        self.layout = layout

    def workspace(self, zp, window, sinks, backward=False):
        return zp.new_window_attention_workspace(self.tq, self.tk, len(self.lens), self.heads, self.kv, self.dim,
                                                 window, sinks, backward)

    def slices(self):
        for i, (a, b) in enumerate(self.lens):
            yield slice(self.q0[i], self.q0[i] + a), slice(self.k0[i], self.k0[i] + b)

    def forward(self, zp, window, sinks, scale=None, **where):
        out, lse = Out((self.tq, self.heads, self.dim), self.dt, self.layout), torch.full((self.heads, self.tq), 77.0,
                                                                                           device="cuda")
        ws = self.workspace(zp, window, sinks)
        zp.zero_window_attention(self.q, self.k, self.v, out.t, ws, window, sinks, scale, lse, **(where or self.where))
        assert zp.zero_workspace_stalls(ws) == 0
        return out, lse

    def check_forward(self, zp, window, sinks, scale=None, **where):
        out, lse = self.forward(zp, window, sinks, scale, **where)
        for qs, ks in self.slices():
            r = ref.attention(self.q[qs], self.k[ks], self.v[ks], window, sinks, scale or self.dim ** -0.5, self.dt)
            close(out.t[qs], r["out"], self.dt, f"out {qs}")
            close(lse[:, qs], r["lse"], torch.float32, f"lse {qs}")
        assert out.only(self.live) and bool((lse[:, ~self.live] == 77).all())
        return out, lse

    def check_backward(self, zp, window, sinks, scale=None, **where):
        out, lse = self.forward(zp, window, sinks, scale, **where)
        out.t[~self.live] = math.nan
        lse[:, ~self.live] = math.nan
        dq = Out((self.tq, self.heads, self.dim), self.dt, self.layout)
        dk, dv = (Out((self.tk, self.kv, self.dim), self.dt, self.layout) for _ in range(2))
        ws = self.workspace(zp, window, sinks, True)
        zp.zero_window_attention_backward(self.dout, self.q, self.k, self.v, out.t, lse, dq.t, dk.t, dv.t, ws, window,
                                          sinks, scale, **(where or self.where))
        assert zp.zero_workspace_stalls(ws) == 0
        for qs, ks in self.slices():
            r = ref.attention_backward(self.dout[qs], self.q[qs], self.k[ks], self.v[ks], out.t[qs], lse[:, qs], window,
                                       sinks, scale or self.dim ** -0.5, self.dt)
            close(dq.t[qs], r["dq"], self.dt, f"dq {qs}")
            close(dk.t[ks], r["dk"], self.dt, f"dk {ks}")
            close(dv.t[ks], r["dv"], self.dt, f"dv {ks}")
        assert dq.only(self.live) and dk.only(self.keyed) and dv.only(self.keyed)


# lens, heads, key heads, dim, window, sinks: one token, tiles' neighbours,
# empty sequences, windows of one, a window's edge in and between tiles, sinks
# past a tile, more queries than keys (rows that see nothing), groups
ATTN = [
    ([(1, 1)], 1, 1, 64, None, 0),
    ([(1, 300)], 4, 2, 128, 100, 3),
    ([(5, 5), (0, 0), (3, 9), (1, 1)], 2, 1, 64, 2, 1),
    ([(127, 127), (128, 128), (129, 129)], 2, 2, 64, None, 0),
    ([(300, 300)], 2, 1, 128, 1, 0),
    ([(300, 300)], 1, 1, 128, 64, 5),
    ([(513, 513), (40, 40)], 3, 3, 80, 128, 130),
    ([(200, 50), (0, 33), (17, 0), (2, 1)], 2, 2, 64, 20, 2),
    ([(260, 700)], 6, 2, 96, 257, 300),
    ([(100, 1000), (3, 5)], 4, 4, 128, 333, 1),
    ([(384, 384)], 8, 1, 64, 129, 0),
    ([(640, 640), (256, 256)], 2, 2, 32, 255, 4),
    ([(257, 257)], 5, 5, 8, None, 3),
    ([(1030, 1030)], 1, 1, 128, 400, 64),
    ([(70, 70)] * 9, 3, 1, 72, 30, 2),
    ([(900, 900)], 2, 1, 112, None, 0),
]
# a few tokens for each sequence, over caches
FEW = [
    ([(1, 1), (1, 17), (1, 16), (1, 15), (1, 2000)], 8, 8, 64, 500, 4),
    ([(1, 600)] * 7, 16, 2, 128, None, 0),
    ([(1, 100), (0, 50), (1, 0), (1, 3000)], 6, 2, 80, 64, 70),
    ([(2, 333), (1, 40), (3, 3), (2, 1)], 12, 4, 96, 50, 1),
    ([(1, 5000)], 25, 25, 64, 256, 4),
    ([(1, 5000)], 64, 2, 128, None, 0),
    ([(4, 777), (4, 9)], 40, 1, 128, 300, 2),
    ([(1, 50), (90, 200), (1, 1)], 4, 2, 64, 33, 2),
    ([(1, 70)], 3, 1, 8, 1, 0),
]


def ids(c):
    return str(c[0][0]) + f"x{len(c[0])}-" + "-".join(map(str, c[1:]))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", ATTN + FEW, ids=ids)
def test_window_attention(zp, case, dtype):
    lens, h, g, d, window, sinks = case
    Batch(lens, h, g, d, dtype, room=3, behind=2).check_forward(zp, window, sinks)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", ATTN + FEW, ids=ids)
def test_window_attention_backward(zp, case, dtype):
    lens, h, g, d, window, sinks = case
    Batch(lens, h, g, d, dtype, room=3, behind=2).check_backward(zp, window, sinks)


@pytest.mark.parametrize("case", [([(2600, 2600)], 2, 1, 64, 100, 4), ([(300, 300), (2400, 2500), (2200, 2200)], 2, 2, 128, 130, 200),
                                  ([(4100, 4100)], 1, 1, 32, 900, 1)], ids=ids)
def test_window_attention_backward_deals_out_the_first_keys(zp, case):
    """Sequences long enough that the first keys' queries go in parts."""
    lens, h, g, d, window, sinks = case
    Batch(lens, h, g, d, "bf16", room=3, behind=2).check_backward(zp, window, sinks)


@pytest.mark.parametrize("short", [6, 12])
def test_window_attention_backward_of_a_long_sequence_among_short_ones(zp, short):
    """The first keys' queries go in parts among few short sequences, and whole among many."""
    lens = [(20, 20)] * (short // 2) + [(2400, 2400)] + [(20, 30)] * (short // 2)
    Batch(lens, 2, 1, 64, "f16", room=3, behind=2).check_backward(zp, 100, 4)


@pytest.mark.parametrize("layout", ["slice", "heads_first"])
@pytest.mark.parametrize("lens", [[(150, 150), (70, 300)], [(1, 400), (1, 30)]], ids=["many", "few"])
def test_window_attention_layouts(zp, lens, layout):
    b = Batch(lens, 4, 2, 64, "bf16", layout=layout)
    b.check_forward(zp, 100, 3)
    b.check_backward(zp, 100, 3)


@pytest.mark.parametrize("lens", [[(300, 300)], [(1, 1)]], ids=["many", "one"])
def test_window_attention_of_one_sequence_without_offsets(zp, lens):
    b = Batch(lens, 2, 2, 64, "f16")
    b.check_forward(zp, 77, 2, q_offsets=None)
    b.check_backward(zp, 77, 2, q_offsets=None)
    c = Batch([(64, 64), (90, 90)], 2, 1, 64, "f16")  # the keys' offsets are the queries'
    c.check_forward(zp, None, 0, q_offsets=c.where["q_offsets"])
    c.check_backward(zp, None, 0, q_offsets=c.where["q_offsets"])


@pytest.mark.parametrize("lens", [(300, 700), (8, 3), (1, 5000), (200, 90)], ids=str)
def test_window_attention_of_one_sequence_over_a_cache(zp, lens):
    """The keys' offsets and length without offsets of the queries."""
    b = Batch([lens], 4, 2, 64, "bf16", room=5)
    where = {name: b.where[name] for name in ("k_offsets", "k_lengths")}
    b.check_forward(zp, 150, 2, **where)
    b.check_backward(zp, 150, 2, **where)


def test_window_attention_in_three_graphs(zp):
    """Captured calls with workspaces of their own, replayed in turn, on
    streams of their own, and twice in a row."""
    batches = [Batch([(1, 900)] * 3, 8, 2, 64, "f16"), Batch([(7, 4000)], 4, 4, 128, "f16"), Batch([(260, 260), (90, 140)], 4, 2, 64, "f16")]
    want, graphs, outs = [], [], []
    for b in batches:
        want.append([x.t if isinstance(x, Out) else x for x in b.check_forward(zp, 300, 3)])
        out, lse, ws = torch.zeros_like(b.q), torch.zeros((b.heads, b.tq), device="cuda"), b.workspace(zp, 300, 3)
        run = lambda: zp.zero_window_attention(b.q, b.k, b.v, out, ws, 300, 3, None, lse, **b.where)
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            run()
            run()
        graphs.append((graph, stream, ws))
        outs.append((out, lse))
    torch.cuda.synchronize()
    for _ in range(3):
        for graph, stream, _ in graphs:
            with torch.cuda.stream(stream):
                graph.replay()
                graph.replay()
    torch.cuda.synchronize()
    for (out, lse), (o, l) in zip(outs, want):
        assert torch.equal(out, o) and torch.equal(lse, l)
    assert all(zp.zero_workspace_stalls(ws) == 0 for _, _, ws in graphs)


@pytest.mark.parametrize("lens", [[(200, 200)], [(1, 200)]], ids=["many", "one"])
@pytest.mark.parametrize("scale,std", [(1.0, 4.0), (1e-3, 1.0), (30.0, 1.0)])
def test_window_attention_scales(zp, lens, scale, std):
    """Scores of several thousand (one key takes all), and flat ones."""
    b = Batch(lens, 2, 1, 128, "bf16", std=std)
    b.check_forward(zp, 90, 2, scale)
    b.check_backward(zp, 90, 2, scale)


@pytest.mark.parametrize("lens", [[(300, 300)], [(2, 300)]], ids=["many", "few"])
def test_window_attention_of_falling_and_rising_scores(zp, lens):
    """The running maximum moves at every tile, or never after the first."""
    for sign in (1.0, -1.0):
        b = Batch(lens, 2, 2, 64, "f16")
        ramp = torch.linspace(0, 8 * sign, 300, device="cuda")[:, None, None]
        b.k.copy_((torch.ones_like(b.k, dtype=torch.float32) * ramp).half())
        b.q.fill_(1.0)
        b.check_forward(zp, None, 0)
        b.check_backward(zp, None, 0)


def test_window_attention_sums_are_the_same_on_every_run(zp):
    b = Batch([(700, 700), (333, 333)], 6, 2, 64, "f16")
    out, lse = b.forward(zp, 100, 40)
    ws, runs = b.workspace(zp, 100, 40, True), []
    for _ in range(10):
        g = [torch.empty_like(x) for x in (b.q, b.k, b.v)]
        zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out.t, lse, *g, ws, 100, 40, **b.where)
        runs.append(g)
    assert all(torch.equal(x, y) for r in runs for x, y in zip(r, runs[0]))
    again = b.forward(zp, 100, 40)
    assert torch.equal(out.t, again[0].t) and torch.equal(lse, again[1])


@pytest.mark.parametrize("lens", [[(150, 200), (200, 260)], [(1, 200), (1, 260)]], ids=["many", "few"])
def test_window_attention_lengths_are_read_when_a_graph_runs(zp, lens):
    """One captured forward and backward over two sets of lengths, on a stream
    of its own."""
    b = Batch(lens, 4, 2, 64, "bf16", room=40, fill=0.0)
    window, sinks = 70, 3
    out, lse = torch.empty_like(b.q), torch.empty((4, b.tq), device="cuda")
    g = [torch.empty_like(x) for x in (b.q, b.k, b.v)]
    ws, bws = b.workspace(zp, window, sinks), b.workspace(zp, window, sinks, True)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())

    def step():
        zp.zero_window_attention(b.q, b.k, b.v, out, ws, window, sinks, None, lse, **b.where)
        zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out, lse, *g, bws, window, sinks, **b.where)
    with torch.cuda.stream(stream):
        step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        step()
    for cut in (0, 37):
        b.where["k_lengths"].sub_(cut)
        graph.replay()
        torch.cuda.synchronize()
        for i, (qs, ks) in enumerate(b.slices()):
            ks = slice(ks.start, ks.stop - cut)
            r = ref.attention(b.q[qs], b.k[ks], b.v[ks], window, sinks, 64 ** -0.5, b.dt)
            close(out[qs], r["out"], b.dt, "out")
            r = ref.attention_backward(b.dout[qs], b.q[qs], b.k[ks], b.v[ks], out[qs], lse[:, qs], window, sinks,
                                       64 ** -0.5, b.dt)
            for got, rows, name in zip(g, (qs, ks, ks), ("dq", "dk", "dv")):
                close(got[rows], r[name], b.dt, name)


@pytest.mark.parametrize("few", [False, True])
def test_window_attention_past_32_bits(zp, few):
    """Rows of keys more than 2^31 elements from the first: a cache of which
    a sequence near its end is read."""
    rows, ld = 70000, 32768  # 2.3 * 10^9 elements
    buf = torch.zeros(rows * ld, dtype=torch.float16, device="cuda").view(rows, ld)
    k, v = buf[:, :128].view(rows, 2, 64), buf[:, 4096:4224].view(rows, 2, 64)
    first = rows - 300
    assert first * ld > 2 ** 31
    k[first:], v[first:] = randn((300, 2, 64), torch.float16, 1), randn((300, 2, 64), torch.float16, 2)
    n = 1 if few else 200
    q = randn((n, 4, 64), torch.float16, 3)
    dev = dict(dtype=torch.int64, device="cuda")
    where = dict(q_offsets=torch.tensor([0, n], **dev), k_offsets=torch.tensor([first, rows], **dev))
    out, lse = torch.empty_like(q), torch.empty((4, n), device="cuda")
    ws = zp.new_window_attention_workspace(n, rows, 1, 4, 2, 64, 100, 4)
    zp.zero_window_attention(q, k, v, out, ws, 100, 4, None, lse, **where)
    r = ref.attention(q, k[first:], v[first:], 100, 4, 0.125, torch.float16)
    close(out, r["out"], torch.float16, "out")
    close(lse, r["lse"], torch.float32, "lse")


def test_window_attention_offsets_outside_the_arrays_are_cut(zp):
    """Offsets and lengths past the rows that there are: as if they ended there."""
    for n in (1, 150):
        b = Batch([(n, 150)], 2, 2, 64, "f16")
        dev = dict(dtype=torch.int64, device="cuda")
        b.check_forward(zp, 60, 1, q_offsets=torch.tensor([-5, 2 ** 40], **dev), k_offsets=torch.tensor([-2 ** 40, 10 ** 6], **dev),
                        k_lengths=torch.tensor([2 ** 50], **dev))
        b.check_backward(zp, 60, 1, q_offsets=torch.tensor([-5, 2 ** 40], **dev),
                         k_offsets=torch.tensor([-2 ** 40, 10 ** 6], **dev))
        out, lse = torch.full_like(b.q, 77.0), torch.full((2, n), 77.0, device="cuda")
        ws = b.workspace(zp, 60, 1)
        zp.zero_window_attention(b.q, b.k, b.v, out, ws, 60, 1, None, lse, q_offsets=torch.tensor([0, n], **dev),
                                 k_offsets=torch.tensor([0, 150], **dev), k_lengths=torch.tensor([-3], **dev))
        assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_window_attention_of_nothing(zp):
    none, q = torch.empty((0, 2, 64), dtype=torch.float16, device="cuda"), randn((3, 2, 64), torch.float16, 1)
    ws = zp.new_window_attention_workspace(3, 3, 1, 2, 2, 64, 5, 0, True)
    out, lse = torch.empty_like(q), torch.empty((2, 3), device="cuda")
    at = dict(q_offsets=torch.tensor([0, 3], device="cuda"), k_offsets=torch.tensor([0, 0], device="cuda"))
    zp.zero_window_attention(q, none, none, out, ws, 5, 0, None, lse, **at)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    dq = torch.full_like(q, 7.0)
    zp.zero_window_attention_backward(q, q, none, none, out, lse, dq, none, none, ws, 5, 0, **at)
    assert bool((dq == 0).all())
    at = dict(q_offsets=torch.tensor([0, 0], device="cuda"), k_offsets=torch.tensor([0, 3], device="cuda"))
    dk, dv = torch.full_like(q, 7.0), torch.full_like(q, 7.0)
    zp.zero_window_attention(none, q, q, none, ws, 5, 0, **at)
    zp.zero_window_attention_backward(none, none, q, q, none, lse[:, :0].contiguous(), none, dk, dv, ws, 5, 0, **at)
    assert bool((dk == 0).all()) and bool((dv == 0).all())


def test_bindings_refuse_on_the_gpu(zp):
    q = randn((4, 2, 64), torch.float16, 1)
    ws = zp.new_window_attention_workspace(4, 4, 1, 2, 2, 64, 4, 0, True)
    out, lse = torch.empty_like(q), torch.empty((2, 4), device="cuda")
    off = torch.tensor([0, 4], device="cuda")
    ok = dict(window=4, lse=lse)
    for call, kind in (
            (lambda: zp.zero_window_attention(q, q.bfloat16(), q, out, ws, **ok), TypeError),
            (lambda: zp.zero_window_attention(q, q, q[:3], out, ws, **ok), ValueError),
            (lambda: zp.zero_window_attention(q, q, q, out[:, :1].expand(4, 2, 64), ws, **ok), ValueError),
            (lambda: zp.zero_window_attention(q, q, q, out, ws, 4, lse=lse.double()), TypeError),
            (lambda: zp.zero_window_attention(q, q, q, out, ws, 4, lse=lse[:, :2]), ValueError),
            (lambda: zp.zero_window_attention(q, q, q, out, ws, 4, q_offsets=off.int()), TypeError),
            (lambda: zp.zero_window_attention(q, q, q, out, ws, 4, q_offsets=off.cpu()), ValueError),
            (lambda: zp.zero_window_attention(q, q, q, out, ws, 4, q_offsets=off, k_offsets=off[:1]), ValueError),
            (lambda: zp.zero_window_attention(q, q, q, out, ws, 4, k_lengths=off[:1]), zp.ZeroError),
            (lambda: zp.zero_window_attention(q, q, q, out, ws, 0), zp.ZeroError),
            (lambda: zp.zero_window_attention(q, q, q, out, ws[:256 - 16], **ok), zp.ZeroError),
            (lambda: zp.zero_window_attention(q.float(), q.float(), q.float(), out.float(), ws, **ok), zp.ZeroError),
            (lambda: zp.zero_window_attention(q[..., 1:9], q[..., 1:9], q[..., 1:9], out[..., :8], ws, **ok), zp.ZeroError),
            (lambda: zp.zero_qk_norm(q, q, None, None, out, out, zp.Rotary([1.0] * 33)), zp.ZeroError),
            (lambda: zp.zero_qk_norm(q, q, None, None, out, out, None, off), ValueError),
            (lambda: zp.zero_qk_norm(q, q, q[0, 0].bfloat16(), None, out, out), zp.ZeroError),
            (lambda: zp.zero_qk_norm(q, q, None, None, out, out, zp.Rotary([1.0]), off), ValueError)):
        with pytest.raises(kind):
            call()


MANY = [(i * 7 % 23, 5 + i * 11 % 60) for i in range(45)]


@pytest.mark.parametrize("lens", [MANY, [(min(q, 2), k) for q, k in MANY]], ids=["many", "few"])
def test_window_attention_of_more_sequences_than_lanes(zp, lens):
    b = Batch(lens, 4, 2, 64, "bf16", room=2, behind=1)
    b.check_forward(zp, 20, 3)
    b.check_backward(zp, 20, 3)


@pytest.mark.parametrize("dim", range(8, 129, 8))
def test_window_attention_head_dims(zp, dim):
    b = Batch([(140, 200), (1, 30)], 4, 2, dim, "f16")
    b.check_forward(zp, 90, 2)
    b.check_backward(zp, 90, 2)
    Batch([(1, 200), (1, 30)], 4, 2, dim, "f16").check_forward(zp, 90, 2)


# up to eight queries for each sequence on average: sets of 8 and of 16 rows
# of queries and heads, windows shorter than the queries, queries without keys,
# and so many blocks that two of them fall to a lane of the join
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("case", [
    ([(8, 700), (5, 5), (6, 1), (7, 40)], 4, 4, 64, None, 0),
    ([(8, 700), (8, 300)], 8, 2, 128, 3, 2),
    ([(8, 9), (8, 3), (8, 8)], 16, 1, 64, 4, 0),
    ([(6, 2000), (7, 65)], 24, 1, 128, 1500, 5),
    ([(5, 30000)], 5, 1, 32, None, 0),
    ([(16, 500), (0, 20), (8, 8)], 3, 1, 80, 100, 130),
], ids=ids)
def test_window_attention_of_up_to_eight_queries(zp, case, dtype):
    lens, h, g, d, window, sinks = case
    Batch(lens, h, g, d, dtype, room=3, behind=2).check_forward(zp, window, sinks)


def test_window_attention_rows_before_the_first_sequence(zp):
    """Offsets that start behind the first rows: those are left as they were."""
    for n in (1, 200):
        b = Batch([(40, 40), (n, 220)], 2, 2, 64, "bf16", fill=math.nan)
        b.q[:40] = b.k[:40] = b.v[:40] = b.dout[:40] = math.nan
        b.where = {k: v[1:].contiguous() for k, v in b.where.items()}
        b.live[:40] = b.keyed[:40] = False
        b.slices = lambda: [(slice(40, 40 + n), slice(40, 260))]
        b.lens = [(n, 220)]
        b.check_forward(zp, 50, 1)
        b.check_backward(zp, 50, 1)


@pytest.mark.parametrize("few", [False, True])
def test_window_attention_offsets_that_fall_touch_nothing_else(zp, few):
    """Results mean nothing, but no other memory is written."""
    b = Batch([(2, 300)] * 3 if few else [(150, 150)] * 3, 2, 1, 64, "f16", fill=0.0)
    dev = dict(dtype=torch.int64, device="cuda")
    last = b.tq
    where = dict(q_offsets=torch.tensor([last, 0, last // 2, 1], **dev), k_offsets=torch.tensor([400, 100, 449, 3], **dev),
                 k_lengths=torch.tensor([500, -3, 2 ** 45], **dev))
    guard = torch.full((64, 2, 64), 77.0, dtype=torch.float16, device="cuda")
    out = torch.full((64 + b.tq + 64, 2, 64), 77.0, dtype=torch.float16, device="cuda")
    lse = torch.full((2, b.tq), 0.0, device="cuda")
    ws = b.workspace(zp, 60, 5, True)
    zp.zero_window_attention(b.q, b.k, b.v, out[64:64 + b.tq], ws, 60, 5, None, lse, **where)
    grads = [torch.full((64 + t.shape[0] + 64, *t.shape[1:]), 77.0, dtype=torch.float16, device="cuda") for t in (b.q, b.k, b.v)]
    zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out[64:64 + b.tq], lse, *(g[64:-64] for g in grads), ws, 60, 5,
                                      **where)
    torch.cuda.synchronize()
    assert torch.equal(out[:64], guard) and torch.equal(out[-64:], guard)
    assert all(bool((g[:64] == 77).all()) and bool((g[-64:] == 77).all()) for g in grads)
    assert zp.zero_workspace_stalls(ws) == 0
    b.check_forward(zp, 60, 5)  # (and the next call is whole)


def test_window_attention_on_two_streams_at_once(zp):
    jobs = []
    for i, lens in enumerate(([(700, 700)], [(1, 3000)] * 5, [(300, 900), (20, 20)])):
        b = Batch(lens, 4, 2, 64, "f16", seed=10 * i)
        jobs.append((b, torch.cuda.Stream(), [b.workspace(zp, 200, 3, True) for _ in range(2)], []))
    torch.cuda.synchronize()
    for _ in range(5):
        for b, stream, ws, outs in jobs:
            with torch.cuda.stream(stream):
                out, lse = torch.empty_like(b.q), torch.empty((4, b.tq), device="cuda")
                g = [torch.empty_like(x) for x in (b.q, b.k, b.v)]
                zp.zero_window_attention(b.q, b.k, b.v, out, ws[0], 200, 3, None, lse, **b.where)
                zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out, lse, *g, ws[0], 200, 3, **b.where)
                outs.append([out, lse, *g])
    torch.cuda.synchronize()
    for b, stream, ws, outs in jobs:
        assert all(torch.equal(x, y) for o in outs for x, y in zip(o, outs[0]))
        for qs, ks in b.slices():
            r = ref.attention(b.q[qs], b.k[ks], b.v[ks], 200, 3, 0.125, b.dt)
            close(outs[0][0][qs], r["out"], b.dt, "out")


def test_window_attention_workspace_serves_other_calls(zp):
    """One workspace, of the largest call, through calls of every kind."""
    big = Batch([(300, 400)] * 3, 4, 2, 64, "bf16")
    ws = big.workspace(zp, 100, 5, True)
    small = [Batch([(1, 390)] * 3, 4, 2, 64, "bf16"), Batch([(2, 50)], 4, 2, 64, "bf16"), Batch([(90, 90)] * 2, 4, 2, 64, "bf16")]
    for b in (big, *small, big, small[0]):
        out, lse = torch.empty_like(b.q), torch.empty((4, b.tq), device="cuda")
        zp.zero_window_attention(b.q, b.k, b.v, out, ws, 100, 5, None, lse, **b.where)
        g = [torch.empty_like(x) for x in (b.q, b.k, b.v)]
        zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out, lse, *g, ws, 100, 5, **b.where)
        for qs, ks in b.slices():
            r = ref.attention(b.q[qs], b.k[ks], b.v[ks], 100, 5, 0.125, b.dt)
            close(out[qs], r["out"], b.dt, "out")
            r = ref.attention_backward(b.dout[qs], b.q[qs], b.k[ks], b.v[ks], out[qs], lse[:, qs], 100, 5, 0.125, b.dt)
            for got, rows, name in zip(g, (qs, ks, ks), ("dq", "dk", "dv")):
                close(got[rows], r[name], b.dt, name)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("kernel", [0, 1, 2])
def test_waits_that_give_up_leave_nan(zp, kernel, dim):
    """A kernel whose tiles of queries never arrive whole: the call ends, the
    workspace counts it, and its results are NaN; the next call is whole."""
    import ctypes
    hook = zp.lib().zero_test_window_attention_waits
    hook.argtypes, hook.restype = [ctypes.c_int32, ctypes.c_uint64], None
    b = Batch([(300, 300), (200, 400)], 4, 2, dim, "f16")
    out, lse = b.forward(zp, 100, 2)
    ws = b.workspace(zp, 100, 2, True)
    o, s = torch.zeros_like(b.q), torch.zeros((4, b.tq), device="cuda")
    g = [torch.zeros_like(x) for x in (b.q, b.k, b.v)]
    hook(kernel, 20_000_000)
    try:
        if kernel == 0:
            zp.zero_window_attention(b.q, b.k, b.v, o, ws, 100, 2, None, s, **b.where)
        else:
            zp.zero_window_attention_backward(b.dout, b.q, b.k, b.v, out.t, lse, *g, ws, 100, 2, **b.where)
        stalls = zp.zero_workspace_stalls(ws)
    finally:
        hook(-1, 0)
    assert stalls > 0
    if kernel == 0:
        assert bool(torch.isnan(o).all()) and bool(torch.isnan(s).all())
    else:
        assert all(bool(torch.isnan(x).all()) == (kernel == 1) for x in g[1:])
        assert bool(torch.isnan(g[0]).all()) == (kernel == 2)
    b.check_forward(zp, 100, 2)
    b.check_backward(zp, 100, 2)


# ------------------------------------------------------------------ together

def test_layer_half_together(zp):
    """Projections' slices through the norms, the rotation and attention and
    back, as a training step runs them, against the formulas one after the
    other; then the next token over the cache that the step's keys make."""
    t, h, g, d = 200, 6, 2, 64
    qkv, gout = randn((t, h + 2 * g, d), torch.bfloat16, 1), randn((t, h, d), torch.bfloat16, 2)
    qw, kw = randn((d,), torch.bfloat16, 3, 0.1, 1.0), randn((d,), torch.bfloat16, 4, 0.1, 1.0)
    freq = [1e-2 ** (i / 32) for i in range(32)]
    rotary, pos = zp.Rotary(freq), list(range(t))
    q, k, v = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
    room = 256
    cache_k, cache_v = (torch.zeros((room, g, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qn, kn = torch.empty_like(q), cache_k[:t]
    zp.zero_qk_norm(q, k, qw, kw, qn, kn, rotary)
    cache_v[:t] = v
    out, lse = torch.empty_like(gout), torch.empty((h, t), device="cuda")
    ws = zp.new_window_attention_workspace(t, room, 1, h, g, d, 50, 4, True)
    zp.zero_window_attention(qn, kn, v, out, ws, 50, 4, None, lse)
    angle = ref.angles(pos, freq)
    for got, x, w in ((qn, q, qw), (kn, k, kw)):
        close(got, ref.head_norm(x, w, angle, pos, d, False, 1e-6), torch.bfloat16, "norm")
    r = ref.attention(qn, kn, v, 50, 4, 0.125, torch.bfloat16)
    close(out, r["out"], torch.bfloat16, "out")
    dqkv = torch.empty_like(qkv)
    dqn, dkn = torch.empty_like(qn), torch.empty_like(kn)
    zp.zero_window_attention_backward(gout, qn, kn, v, out, lse, dqn, dkn, dqkv[:, h + g:], ws, 50, 4)
    dw = torch.empty((2, d), dtype=torch.bfloat16, device="cuda")
    zp.zero_qk_norm_backward(dqn, dkn, q, k, qw, kw, dqkv[:, :h], dqkv[:, h:h + g], dw[0], dw[1],
                             zp.new_qk_norm_workspace(t, h, g, d), rotary)
    r = ref.attention_backward(gout, qn, kn, v, out, lse, 50, 4, 0.125, torch.bfloat16)
    for got, name in ((dqn, "dq"), (dkn, "dk"), (dqkv[:, h + g:], "dv")):
        close(got, r[name], torch.bfloat16, name)
    for n, (got, dy, x, w) in enumerate(((dqkv[:, :h], dqn, q, qw), (dqkv[:, h:h + g], dkn, k, kw))):
        r = ref.head_norm_backward(dy, x, w, angle, pos, d, False, 1e-6)
        close(got, r["dx"], torch.bfloat16, "dx")
        close(dw[n], r["dw"], torch.bfloat16, "dw")
    # the next token
    new = randn((1, h + 2 * g, d), torch.bfloat16, 5)
    q1 = torch.empty((1, h, d), dtype=torch.bfloat16, device="cuda")
    zp.zero_qk_norm(new[:, :h], new[:, h:h + g], qw, kw, q1, cache_k[t:t + 1], rotary, torch.tensor([t], device="cuda"))
    cache_v[t] = new[0, h + g:]
    o1 = torch.empty_like(q1)
    zp.zero_window_attention(q1, cache_k, cache_v, o1, ws, 50, 4, k_offsets=torch.tensor([0, room], device="cuda"),
                             k_lengths=torch.tensor([t + 1], device="cuda"), q_offsets=torch.tensor([0, 1], device="cuda"))
    r = ref.attention(q1, cache_k[:t + 1], cache_v[:t + 1], 50, 4, 0.125, torch.bfloat16)
    close(o1, r["out"], torch.bfloat16, "next token")
