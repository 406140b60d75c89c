"""The feed-forward sub-block on the GPU against its formulas in binary64
(sublayer_ref.py, which also derives each bound), at the sizes, strides and
values where the kernels can go wrong."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sublayer_ref as ref  # noqa: E402

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


def randn(shape, dtype, seed, std=1.0, mean=0.0, ld=None, off=0):
    """N(mean, std) in a buffer with row stride ld and `off` elements before
    the first, the rest of the buffer NaN."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    t = torch.empty(shape, device="cuda").normal_(mean, std, generator=gen).to(dtype)
    if ld is None and off == 0:
        return t
    return strided(shape, dtype, ld, off).copy_(t)


def strided(shape, dtype, ld=None, off=0, fill=float("nan")):
    ld = ld or shape[-1]
    rows = shape[0] if len(shape) == 2 else 1
    buf = torch.full((off + rows * ld + 16,), fill, dtype=dtype, device="cuda")
    return buf[off:off + rows * ld].view(rows, ld)[:, :shape[-1]] if len(shape) == 2 else buf[off:off + shape[0]]


def guarded(shape, dtype, ld=None, off=0):
    """An output in a buffer of sentinels, and a check that only it changed."""
    ld = ld or shape[-1]
    rows = shape[0] if len(shape) == 2 else 1
    buf = torch.full((off + rows * ld + 64,), 77.0, dtype=dtype, device="cuda")
    view = buf[off:off + rows * ld].view(rows, ld)[:, :shape[-1]] if len(shape) == 2 else buf[off:off + shape[0]]

    def untouched():
        c = buf.clone()
        (c[off:off + rows * ld].view(rows, ld)[:, :shape[-1]] if len(shape) == 2 else c[off:off + shape[0]]).fill_(77.0)
        return bool((c == 77.0).all())
    return view, untouched


def close(got, want, dtype, what):
    value, err = want
    ref.check(got, value, ref.rounded(value, err, dtype), what)


# rows, cols: one element, one row, a quad and its neighbours, odd widths,
# whole vectors, wide rows, more rows than blocks
SHAPES = [(1, 1), (1, 5), (3, 4), (2, 7), (5, 8), (4, 31), (33, 64), (7, 255), (129, 256), (64, 257), (17, 1001),
          (1, 1600), (300, 1600), (9, 4097), (3, 8192), (5, 20001), (2, 40000), (5000, 33), (9001, 16)]

# (row stride beyond cols, elements before the first): whole rows, odd starts, padded rows
PLACES = [(0, 0), (0, 1), (3, 2), (8, 8)]


# ------------------------------------------------------------------ dropout

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_dropout_add(zp, shape, dtype):
    dt = TYPES[dtype]
    for k, (pad, off) in enumerate(PLACES):
        x = randn(shape, dt, 1, ld=shape[1] + pad, off=off)
        res = randn(shape, dt, 2, 2.0, ld=shape[1] + pad, off=off) if k % 2 == 0 else None
        out, untouched = guarded(shape, dt, shape[1] + pad, off)
        drop = (0.3, 0x123456789ABCDEF + k, (k << 33) + 5)
        zp.zero_dropout_add(x, res, out, zp.Dropout(*drop))
        close(out, ref.dropout_add(x, res, drop), dt, f"place {pad}, {off}")
        assert untouched()


@pytest.mark.parametrize("p", [0.0, 1e-10, 0.5, 1.0 - 1e-10, 1.0])
def test_dropout_add_extreme_rates(zp, p):
    x, res = randn((50, 99), torch.float32, 3), randn((50, 99), torch.float32, 4)
    out = torch.empty_like(x)
    zp.zero_dropout_add(x, res, out, zp.Dropout(p, 9))
    close(out, ref.dropout_add(x, res, (p, 9, 0)), torch.float32, "out")


def test_dropout_drops_values_that_are_not_numbers(zp):
    x = randn((64, 64), torch.float16, 5)
    x[::2] = float("nan")
    x[1::4] = float("inf")
    out = torch.empty_like(x)
    zp.zero_dropout_add(x, None, out, zp.Dropout(0.5, 11, 12))
    keep = torch.from_numpy(ref.keep_mask(64, 64, 0.5, 11, 12)).cuda()
    assert bool((out[~keep] == 0).all())
    assert torch.equal(torch.isnan(out), torch.isnan(x) & keep) and torch.equal(torch.isinf(out), torch.isinf(x) & keep)


def test_dropout_in_place_and_offset_on_the_device(zp):
    x, res = randn((31, 100), torch.bfloat16, 6), randn((31, 100), torch.bfloat16, 7)
    step = torch.tensor([2 ** 40 + 3], dtype=torch.int64, device="cuda")
    want = torch.empty_like(x)
    zp.zero_dropout_add(x, res, want, zp.Dropout(0.25, 1, 2 ** 40 + 10))
    a, b = x.clone(), res.clone()
    zp.zero_dropout_add(a, res, a, zp.Dropout(0.25, 1, 7, step))
    zp.zero_dropout_add(x, b, b, zp.Dropout(0.25, 1, 7, step))
    assert torch.equal(a, want) and torch.equal(b, want)
    # a captured call draws a new mask when the offset on the device moves on
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    drop = zp.Dropout(0.25, 1, 7, step)
    with torch.cuda.graph(g):
        zp.zero_dropout_add(x, res, out, drop)
    g.replay()
    assert torch.equal(out, want)
    step += 1
    g.replay()
    zp.zero_dropout_add(x, res, want, zp.Dropout(0.25, 1, 2 ** 40 + 11))
    assert torch.equal(out, want)


def test_offsets_past_32_bits(zp):
    """Rows 2^31 elements apart: the third starts past element 2^32."""
    ld = 2 ** 31
    buf = torch.zeros(2 * ld + 1600, dtype=torch.float16, device="cuda")
    out = torch.zeros_like(buf)
    x = torch.as_strided(buf, (3, 1600), (ld, 1))
    x.copy_(randn((3, 1600), torch.float16, 8))
    y = torch.as_strided(out, (3, 1600), (ld, 1))
    zp.zero_dropout_add(x, None, y, zp.Dropout(0.1, 3))
    close(y, ref.dropout_add(x, None, (0.1, 3, 0)), torch.float16, "dropout")
    zp.zero_layer_norm(x, None, None, y)
    r = ref.layer_norm(x, None, None, 1e-5)
    close(y, r["y"], torch.float16, "norm")
    dy = randn((3, 1600), torch.float16, 9)
    mean, rstd = r["mean"][0].float(), r["rstd"][0].float()
    ws, dw, db = zp.new_layer_norm_workspace(3, 1600), *(torch.empty(1600, device="cuda") for _ in range(2))
    zp.zero_layer_norm_backward(dy, x, None, mean, rstd, y, dw, db, ws)
    b = ref.layer_norm_backward(dy, x, None, mean, rstd)
    close(y, b["dx"], torch.float16, "dx")
    close(dw, b["dweight"], torch.float32, "dweight")
    w = [randn(s, torch.float16, 10 + k, 0.03) for k, s in enumerate([(64, 1600), (64, 1600), (1600, 64)])]
    zp.zero_gated_ffn(x, *w, y, zp.new_gated_ffn_workspace(3, 1600, 64))
    close(y, ref.gated_ffn(x, *w, ref.SILU)["y"], torch.float16, "ffn")


def test_matrix_of_more_than_2_to_the_32_elements(zp):
    """A contiguous matrix past 2^32 elements: its last rows."""
    rows, cols = 2 ** 21 + 3, 2048
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda").normal_()
    out = torch.empty_like(x)
    zp.zero_dropout_add(x, None, out, zp.Dropout(0.5, 21))
    quads = cols // 4
    r = np.repeat(np.arange(rows - 4, rows, dtype=np.uint64), quads)
    c = np.tile(np.arange(quads, dtype=np.uint64), 4)
    w = np.stack(ref.philox([c, r, np.zeros_like(c), np.zeros_like(c)], (21, 0)), -1).reshape(4, cols)
    keep = torch.from_numpy(w >= np.uint64(2 ** 31)).cuda()
    assert torch.equal(out[-4:], torch.where(keep, 2 * x[-4:], torch.zeros_like(x[-4:])))
    zp.zero_layer_norm(x, None, None, out)
    close(out[-4:], ref.layer_norm(x[-4:], None, None, 1e-5)["y"], torch.bfloat16, "y")


# ------------------------------------------------------------------ layer norm

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_layer_norm(zp, shape, dtype):
    dt, (rows, cols) = TYPES[dtype], shape
    for k, (pad, off) in enumerate(PLACES):
        wdt = dt if k % 2 else torch.float32
        w = randn((cols,), wdt, 20, 0.2, 1.0, off=off) if k != 2 else None
        b = randn((cols,), wdt, 21, off=off) if k != 3 else None
        x = randn(shape, dt, 22, 1.5, 0.5, ld=cols + pad, off=off)
        y, ok_y = guarded(shape, dt, cols + pad, off)
        mean, ok_m = guarded((rows,), torch.float32, off=off)
        rstd, ok_r = guarded((rows,), torch.float32, off=off)
        zp.zero_layer_norm(x, w, b, y, mean, rstd, eps=1e-5)
        r = ref.layer_norm(x, w, b, 1e-5)
        close(y, r["y"], dt, f"y, place {pad}, {off}")
        close(mean, r["mean"], torch.float32, "mean")
        close(rstd, r["rstd"], torch.float32, "rstd")
        assert ok_y() and ok_m() and ok_r()
        # with the sum in front
        res = randn(shape, dt, 23, 2.0, ld=cols + pad, off=off) if k != 1 else None
        drop = (0.2, 5 + k, k << 32) if k != 2 else None
        s, ok_s = guarded(shape, dt, cols + pad, off)
        zp.zero_layer_norm(x, w, b, y, mean, rstd, eps=1e-5, residual=res, sum_out=s,
                           drop=zp.Dropout(*drop) if drop else None)
        r = ref.layer_norm(x, w, b, 1e-5, res, drop)
        close(y, r["y"], dt, f"y of the sum, place {pad}, {off}")
        close(s, r["sum"], dt, "sum")
        close(rstd, r["rstd"], torch.float32, "rstd of the sum")
        assert ok_y() and ok_s() and ok_m() and ok_r()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_layer_norm_backward(zp, shape, dtype):
    dt, (rows, cols) = TYPES[dtype], shape
    ws = zp.new_layer_norm_workspace(rows, cols)
    for k, (pad, off) in enumerate(PLACES):
        wdt, gdt = (dt, torch.float32) if k % 2 else (torch.float32, dt)
        w = randn((cols,), wdt, 30, 0.2, 1.0, off=off) if k != 2 else None
        x = randn(shape, dt, 31, 1.5, 0.5, ld=cols + pad, off=off)
        dy = randn(shape, dt, 32, ld=cols + pad, off=off)
        r = ref.layer_norm(x, None, None, 1e-5)
        mean, rstd = r["mean"][0].float(), r["rstd"][0].float()
        res = randn(shape, dt, 33, ld=cols + pad, off=off) if k != 1 else None
        drop = (0.4, 6 + k, k << 31) if k != 3 else None
        dx, ok_x = guarded(shape, dt, cols + pad, off)
        dd, ok_d = guarded(shape, dt, cols + pad, off) if drop else (None, lambda: True)
        dw, ok_w = guarded((cols,), gdt, off=off)
        db, ok_b = guarded((cols,), gdt, off=off) if k != 2 else (None, lambda: True)
        zp.zero_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws, dresidual=res, dx_dropped=dd,
                                    drop=zp.Dropout(*drop) if drop else None)
        b = ref.layer_norm_backward(dy, x, w, mean, rstd, res, drop)
        close(dx, b["dx"], dt, f"dx, place {pad}, {off}")
        if drop:
            close(dd, b["dropped"], dt, "dropped")
        close(dw, b["dweight"], gdt, "dweight")
        if db is not None:
            close(db, b["dbias"], gdt, "dbias")
        assert ok_x() and ok_d() and ok_w() and ok_b()
        again = dw.clone()
        zp.zero_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, None, ws)
        assert torch.equal(dw, again), "the same sums in the same order"
        dx2, _ = guarded(shape, dt, cols + pad, off)
        zp.zero_layer_norm_backward(dy, x, w, mean, rstd, dx2, None, None, ws)
        assert torch.equal(dx, dx2), "the same dx whether or not the weight's gradient is taken"


# rows, cols where a block stages its rows: every number of column groups per
# lane, one to sixteen warps per row, last groups that are partly and wholly
# outside the row, rows that do not divide among the blocks
MANY = [(1216, 520), (1300, 1000), (1217, 1280), (1700, 1288), (2501, 1600), (1219, 2048), (1300, 2056), (2433, 2568),
        (2433, 4096), (2440, 4104), (2440, 6400), (2450, 8192), (310, 8200), (400, 16384)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("shape", MANY, ids=str)
def test_layer_norm_of_many_rows(zp, shape, dtype):
    test_layer_norm(zp, shape, dtype)
    test_layer_norm_backward(zp, shape, dtype)


@pytest.mark.parametrize("cols", [1600, 4096])
def test_layer_norm_of_many_rows_keeps_rows_apart(zp, cols):
    """A row that is not finite changes no other row; a rate of one drops everything."""
    rows, dt = 2600, torch.float16
    x, res, w, b = randn((rows, cols), dt, 45), randn((rows, cols), dt, 46), randn((cols,), dt, 47), randn((cols,), dt, 48)
    mean, rstd = (torch.empty(rows, device="cuda") for _ in range(2))
    bad = x.clone()
    bad[7, 3], bad[1999, cols - 1] = float("nan"), float("inf")
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[[7, 1999]] = False
    out = []
    for t in (x, bad):
        y, s, dx, dd = (torch.empty_like(x) for _ in range(4))
        zp.zero_layer_norm(t, w, b, y, mean, rstd, residual=res, sum_out=s, drop=zp.Dropout(2.0 ** -40, 1))
        dw, ws = torch.empty_like(w), zp.new_layer_norm_workspace(rows, cols)
        zp.zero_layer_norm_backward(res, s, w, mean, rstd, dx, dw, None, ws, dresidual=res, dx_dropped=dd,
                                    drop=zp.Dropout(0.3, 2))
        out.append((y[others], s[others], dx[others], dd[others]))
        assert torch.isfinite(y).all(1).eq(others if t is bad else torch.ones_like(others)).all()
    assert all(torch.equal(p, q) for p, q in zip(*out))
    zp.zero_layer_norm(bad, w, b, y, mean, rstd, residual=res, sum_out=s, drop=zp.Dropout(1.0, 1))
    assert torch.equal(s, res)
    zp.zero_layer_norm_backward(bad, s, w, mean, rstd, dx, dw, None, ws, dx_dropped=dd, drop=zp.Dropout(1.0, 1))
    assert torch.equal(dd[others], torch.zeros_like(dd[others]))


def test_layer_norm_gradient_against_differences(zp):
    """Central differences of the binary32 kernel itself.  Step 2^-6 in a unit
    direction of 40 x 96 elements: truncation below step^2 times third
    derivatives of order 1 times |dy|; rounding: y to 2^-22 relative, summed
    with random signs over 3840 terms and divided by 2 step."""
    shape = (40, 96)
    x, dy, v = (randn(shape, torch.float32, 40 + k) for k in range(3))
    w, b = randn((96,), torch.float32, 43, 0.2, 1.0), randn((96,), torch.float32, 44)
    v /= v.norm()
    y, mean, rstd = torch.empty_like(x), *(torch.empty(40, device="cuda") for _ in range(2))
    zp.zero_layer_norm(x, w, b, y, mean, rstd)
    dx, dw, db, ws = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b), zp.new_layer_norm_workspace(*shape)
    zp.zero_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
    step, f = 2.0 ** -6, []
    for s in (step, -step):
        zp.zero_layer_norm((x + s * v), w, b, y)
        f.append(float((y.double() * dy.double()).sum()))
    d = (f[0] - f[1]) / (2 * step)
    assert abs(d - float((dx.double() * v.double()).sum())) < 8 * step ** 2 + 3840 ** 0.5 * 2 ** -20 / step
    # linear in the weight and the bias: exact but for rounding
    for grad, t in ((dw, (v[0], torch.zeros_like(b))), (db, (torch.zeros_like(w), v[1]))):
        zp.zero_layer_norm(x, *t, y)
        want = float((y.double() * dy.double()).sum())
        assert abs(float((grad.double() * (t[0] + t[1]).double()).sum()) - want) < 1e-4


@pytest.mark.parametrize("dtype", TYPES)
def test_layer_norm_of_values_that_are_not_finite(zp, dtype):
    """A row with an inf or a NaN gives NaN; the others stay as they were."""
    dt = TYPES[dtype]
    x = randn((8, 300), dt, 50)
    x[2, 17] = float("inf")
    x[5, 299] = float("nan")
    y, mean, rstd = torch.empty_like(x), *(torch.empty(8, device="cuda") for _ in range(2))
    zp.zero_layer_norm(x, None, None, y, mean, rstd)
    bad = torch.tensor([2, 5], device="cuda")
    good = torch.tensor([0, 1, 3, 4, 6, 7], device="cuda")
    assert bool(torch.isnan(y[bad]).all())
    close(y[good], ref.layer_norm(x[good], None, None, 1e-5)["y"], dt, "y")
    # rows of equal values: variance zero
    x = torch.full((3, 1024), 3.0, dtype=dt, device="cuda")
    y = torch.empty_like(x)
    zp.zero_layer_norm(x, None, None, y, mean[:3].clone(), rstd[:3].clone())
    assert bool((y == 0).all())


def test_layer_norm_with_a_large_mean(zp):
    """mean 1000 times the deviation: the deviations are taken from the mean,
    not from a difference of squares."""
    x = randn((50, 1600), torch.float32, 51, 1.0, 1000.0)
    y, rstd = torch.empty_like(x), torch.empty(50, device="cuda")
    zp.zero_layer_norm(x, None, None, y, None, rstd)
    r = ref.layer_norm(x, None, None, 1e-5)
    close(rstd, r["rstd"], torch.float32, "rstd")
    close(y, r["y"], torch.float32, "y")


def test_empty_sizes(zp):
    z = torch.empty((0, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    zp.zero_dropout_add(z, z, z, zp.Dropout(0.1, 1))
    zp.zero_layer_norm(z, w, w, z)
    dw, db = torch.full_like(w, 5.0), torch.full_like(w, 5.0)
    e = torch.empty(0, device="cuda")
    zp.zero_layer_norm_backward(z, z, w, e, e, z, dw, db, zp.new_layer_norm_workspace(0, 64))
    assert bool((dw == 0).all()) and bool((db == 0).all()), "gradients over no rows are zero"
    z = torch.empty((64, 0), device="cuda")
    zp.zero_layer_norm(z, None, None, z)
    h = lambda *s: torch.full(s, 5.0, dtype=torch.float16, device="cuda")  # noqa: E731
    for m, d, f in ((0, 64, 128), (5, 64, 0), (5, 0, 128), (5, 13, 0), (0, 13, 7)):
        x, wg, wu, wd, gate, up = h(m, d), h(f, d), h(f, d), h(d, f), h(m, f), h(m, f)
        y, ws = h(m, d), zp.new_gated_ffn_workspace(m, d, f, True)
        zp.zero_gated_ffn(x, wg, wu, wd, y, ws, gate=gate, up=up)
        assert bool((y == 0).all()) and (d > 0 or bool((gate == 0).all() and (up == 0).all()))
        gate, up = h(m, f), h(m, f)
        dx, dwg, dwu, dwd = h(m, d), h(f, d), h(f, d), h(d, f)
        zp.zero_gated_ffn_backward(y, x, wg, wu, wd, gate, up, dx, dwg, dwu, dwd, ws)
        assert bool((dx == 0).all() and (dwg == 0).all() and (dwu == 0).all() and (dwd == 0).all())


# ------------------------------------------------------------------ gated feed-forward

# tokens, dim, inner: single elements and tokens, a batch of a few, tile
# edges and their neighbours, odd widths, several tiles of every axis
FFN = [(1, 1, 1), (1, 8, 8), (1, 64, 256), (1, 1600, 640), (2, 257, 96), (3, 24, 40), (4, 512, 1024), (5, 8, 300),
       (8, 1024, 512), (9, 96, 520), (16, 200, 400), (17, 33, 65), (31, 136, 72), (64, 64, 64), (65, 320, 192),
       (127, 128, 256), (128, 256, 128), (129, 264, 136), (200, 101, 203), (256, 512, 768), (300, 72, 1000),
       (513, 640, 264), (700, 1001, 513), (1030, 512, 520), (2049, 1608, 2056), (1999, 1501, 2011),
       (3, 101, 203), (3, 104, 203), (4, 257, 1001), (4, 1001, 264), (2500, 72, 200), (4001, 147, 333)]


def ffn_inputs(m, d, f, dt, seed):
    return (randn((m, d), dt, seed), randn((f, d), dt, seed + 1, d ** -0.5), randn((f, d), dt, seed + 2, d ** -0.5),
            randn((d, f), dt, seed + 3, f ** -0.5))


@pytest.mark.parametrize("kind", [ref.SILU, ref.GELU], ids=["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", FFN, ids=str)
def test_gated_ffn(zp, size, dtype, kind):
    (m, d, f), dt = size, TYPES[dtype]
    x, wg, wu, wd = ffn_inputs(m, d, f, dt, 60)
    r = ref.gated_ffn(x, wg, wu, wd, kind)
    ws = zp.new_gated_ffn_workspace(m, d, f)
    y, ok_y = guarded((m, d), dt)
    zp.zero_gated_ffn(x, wg, wu, wd, y, ws, act=kind)
    close(y, r["y"], dt, "y")
    assert ok_y()
    first = y.clone()
    gate, ok_g = guarded((m, f), dt)
    up, ok_u = guarded((m, f), dt)
    zp.zero_gated_ffn(x, wg, wu, wd, y, ws, act=kind, gate=gate, up=up)
    close(gate, r["gate"], dt, "gate")
    close(up, r["up"], dt, "up")
    assert ok_y() and ok_g() and ok_u()
    assert torch.equal(y, first), "the same bits with gate and up kept"
    assert zp.zero_workspace_stalls(ws) == 0


@pytest.mark.parametrize("kind", [ref.SILU, ref.GELU], ids=["silu", "gelu"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("size", FFN, ids=str)
def test_gated_ffn_backward(zp, size, dtype, kind):
    (m, d, f), dt = size, TYPES[dtype]
    x, wg, wu, wd = ffn_inputs(m, d, f, dt, 70)
    dy, gate, up = randn((m, d), dt, 80), randn((m, f), dt, 81), randn((m, f), dt, 82)
    r = ref.gated_ffn_backward(dy, x, wg, wu, wd, gate, up, kind)
    ws = zp.new_gated_ffn_workspace(m, d, f, True)
    for gdt in (dt, torch.float32):
        outs = {k: guarded(s, g) for k, s, g in (("dx", (m, d), dt), ("dw_gate", (f, d), gdt), ("dw_up", (f, d), gdt),
                                                 ("dw_down", (d, f), gdt))}
        views = [v for v, _ in outs.values()]
        zp.zero_gated_ffn_backward(dy, x, wg, wu, wd, gate, up, *views, ws, act=kind)
        for k, (v, untouched) in outs.items():
            close(v, r[k], v.dtype, f"{k} ({gdt})")
            assert untouched(), k
        first = [v.clone() for v in views]
        zp.zero_gated_ffn_backward(dy, x, wg, wu, wd, gate, up, *views, ws, act=kind)
        assert all(torch.equal(a, b) for a, b in zip(first, views)), "the same bits on every run"
    assert zp.zero_workspace_stalls(ws) == 0


@pytest.mark.parametrize("size", [(1, 64, 128), (40, 136, 264), (300, 128, 256), (70, 51, 99), (70, 51, 100)], ids=str)
def test_gated_ffn_strided_and_offset(zp, size):
    """Row-strided x, y, dy, dx (NaN between the rows); outputs, gate and up
    at odd starts; with odd widths the operands too, but for the last size,
    whose x and dy lie on 16 bytes."""
    (m, d, f), dt = size, torch.bfloat16
    whole = (d | f) % 8 == 0
    pad, off = (24, 8) if whole else (5, 3) if f % 2 else (13, 8)
    x = randn((m, d), dt, 90, ld=d + pad, off=off)
    dy = randn((m, d), dt, 91, ld=d + pad, off=off)
    o = 0 if whole else 1
    wg, wu = (randn((f * d,), dt, 92 + k, d ** -0.5, off=o).view(f, d) for k in range(2))
    wd = randn((d * f,), dt, 94, f ** -0.5, off=o).view(d, f)
    y, ok_y = guarded((m, d), dt, d + 7, 5)
    gate, up = (strided((m * f,), dt, off=k + 1).view(m, f) for k in range(2))
    ws = zp.new_gated_ffn_workspace(m, d, f, True)
    zp.zero_gated_ffn(x, wg, wu, wd, y, ws, gate=gate, up=up)
    r = ref.gated_ffn(x, wg, wu, wd, ref.SILU)
    for got, k in ((y, "y"), (gate, "gate"), (up, "up")):
        close(got, r[k], dt, k)
    assert ok_y()
    dx, ok_x = guarded((m, d), dt, d + 7, 5)
    dw = [strided((f * d,), dt, off=k + 1).view(s) for k, s in enumerate([(f, d), (f, d), (d, f)])]
    zp.zero_gated_ffn_backward(dy, x, wg, wu, wd, gate, up, dx, *dw, ws)
    r = ref.gated_ffn_backward(dy, x, wg, wu, wd, gate, up, ref.SILU)
    for got, k in zip([dx] + dw, ("dx", "dw_gate", "dw_up", "dw_down")):
        close(got, r[k], dt, k)
    assert ok_x()


def test_gated_ffn_refuses_operands_off_16_bytes(zp):
    x, wg, wu, wd = ffn_inputs(4, 64, 128, torch.float16, 95)
    ws, y = zp.new_gated_ffn_workspace(4, 64, 128), torch.empty_like(x)
    odd = randn((4, 64), torch.float16, 96, ld=64, off=1)
    for bad in (odd, randn((4, 64), torch.float16, 96, ld=68)):
        with pytest.raises(zp.ZeroError) as e:
            zp.zero_gated_ffn(bad, wg, wu, wd, y, ws)
        assert e.value.code == -2
    with pytest.raises(zp.ZeroError) as e:
        zp.zero_gated_ffn(x, wg, wu, wd, y, ws[:256])
    assert e.value.code == -5


@pytest.mark.parametrize("m", [1, 5, 40, 300])
def test_gated_ffn_gradients_are_adjoint(zp, m):
    """y is linear in w_down and in w_up: <dw_down, V> = <dy, y at w_down = V>
    and <dw_up, V> = <dy, y at w_up = V>, with V of the weights' type, but for
    the kernels' rounding (binary32 weight gradients)."""
    d, f, dt = 96, 160, torch.float16
    x, wg, wu, wd = ffn_inputs(m, d, f, dt, 100)
    vd, vu, dy = randn((d, f), dt, 104, f ** -0.5), randn((f, d), dt, 105, d ** -0.5), randn((m, d), dt, 106)
    ws, y, gate, up = zp.new_gated_ffn_workspace(m, d, f, True), torch.empty_like(x), *(
        torch.empty((m, f), dtype=dt, device="cuda") for _ in range(2))
    zp.zero_gated_ffn(x, wg, wu, wd, y, ws, act=ref.GELU, gate=gate, up=up)
    g = [torch.empty(s, device="cuda") for s in ((f, d), (f, d), (d, f))]
    dx = torch.empty_like(x)
    zp.zero_gated_ffn_backward(dy, x, wg, wu, wd, gate, up, dx, *g, ws, act=ref.GELU)
    for grad, v, w in ((g[2], vd, (wg, wu, vd)), (g[1], vu, (wg, vu, wd))):
        zp.zero_gated_ffn(x, *w, y, ws, act=ref.GELU)
        left = float((grad.double() * v.double()).sum())
        terms = y.double() * dy.double()
        # every f16 rounding on either side (gate, up, h, dh's products, y): a few 2^-11 of each of the m * d terms
        assert abs(left - float(terms.sum())) < 8 * 2.0 ** -11 * float(
            ref.gated_ffn(x.abs(), wg.abs(), wu.abs(), wd.abs() + vd.abs(), ref.GELU)["y"][0].mul(dy.abs()).sum())


def test_gated_ffn_of_values_that_are_not_finite(zp):
    """An inf or a NaN in a token reaches that token's outputs alone."""
    for m in (3, 200):
        x, wg, wu, wd = ffn_inputs(m, 128, 256, torch.bfloat16, 110)
        y, clean, ws = torch.empty_like(x), torch.empty_like(x), zp.new_gated_ffn_workspace(m, 128, 256)
        zp.zero_gated_ffn(x, wg, wu, wd, clean, ws)
        x[1, 5] = float("nan")
        zp.zero_gated_ffn(x, wg, wu, wd, y, ws)
        assert bool(torch.isnan(y[1]).all())
        rest = [i for i in range(m) if i != 1]
        assert torch.equal(y[rest], clean[rest])
        # large gates of both signs: the activation saturates
        x, big = torch.ones_like(x), torch.full_like(wg, 1.0)
        big[1::2] = -1.0
        zp.zero_gated_ffn(x, big, wu, wd, y, ws)
        close(y, ref.gated_ffn(x, big, wu, wd, ref.SILU)["y"], torch.bfloat16, "y")


# ------------------------------------------------------------------ streams, graphs, repeated use

def test_calls_run_on_the_given_stream(zp):
    """Inputs written late on a side stream are seen, whatever the current
    stream."""
    side = torch.cuda.Stream()
    x, wg, wu, wd = ffn_inputs(64, 128, 256, torch.float16, 120)
    src = randn((64, 128), torch.float16, 121)
    y, t, ws = torch.empty_like(x), torch.empty_like(x), zp.new_gated_ffn_workspace(64, 128, 256, True)
    drop = zp.Dropout(0.1, 4)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        x.copy_(src)
    zp.zero_layer_norm(x, None, None, t, stream=side)
    zp.zero_gated_ffn(t, wg, wu, wd, y, ws, stream=side)
    zp.zero_dropout_add(y, x, y, drop, stream=side)
    side.synchronize()
    t2, y2 = torch.empty_like(x), torch.empty_like(x)
    zp.zero_layer_norm(src, None, None, t2)
    zp.zero_gated_ffn(t2, wg, wu, wd, y2, ws)
    zp.zero_dropout_add(y2, src, y2, drop)
    assert torch.equal(y, y2)


@pytest.mark.parametrize("size", [(1, 64, 128), (40, 128, 256), (300, 136, 520), (70, 51, 99)], ids=str)
def test_calls_can_be_captured(zp, size):
    m, d, f = size
    dt = torch.bfloat16
    x, wg, wu, wd = ffn_inputs(m, d, f, dt, 130)
    dy, w = randn((m, d), dt, 134), randn((d,), dt, 135)
    n, y, dn, dx = (torch.empty_like(x) for _ in range(4))
    gate, up = (torch.empty((m, f), dtype=dt, device="cuda") for _ in range(2))
    mean, rstd = (torch.empty(m, device="cuda") for _ in range(2))
    dwg, dwu, dwd, dw, db = (torch.empty_like(t) for t in (wg, wu, wd, w, w))
    ws, wn = zp.new_gated_ffn_workspace(m, d, f, True), zp.new_layer_norm_workspace(m, d)

    def step():
        zp.zero_layer_norm(x, w, w, n, mean, rstd)
        zp.zero_gated_ffn(n, wg, wu, wd, y, ws, gate=gate, up=up)
        zp.zero_gated_ffn_backward(dy, n, wg, wu, wd, gate, up, dn, dwg, dwu, dwd, ws)
        zp.zero_layer_norm_backward(dn, x, w, mean, rstd, dx, dw, db, wn)

    outs = (y, dx, dwg, dwu, dwd, dw, db)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    want = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        for t in outs:
            t.fill_(float("nan"))
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
    assert zp.zero_workspace_stalls(ws) == 0


def test_one_workspace_serves_calls_of_many_sizes(zp):
    """A workspace of the largest size, back to back over other sizes: no call
    leaves anything behind that the next one trips over."""
    sizes = [(1, 64, 128), (300, 256, 512), (7, 51, 99), (130, 256, 512), (2, 256, 512)]
    ws = torch.zeros(max(zp.zero_gated_ffn_workspace_bytes(*s, True) for s in sizes), dtype=torch.uint8, device="cuda")
    for rep in range(3):
        for k, (m, d, f) in enumerate(sizes):
            x, wg, wu, wd = ffn_inputs(m, d, f, torch.float16, 140 + k)
            a, b = torch.empty_like(x), torch.empty_like(x)
            zp.zero_gated_ffn(x, wg, wu, wd, a, ws)
            zp.zero_gated_ffn(x, wg, wu, wd, b, zp.new_gated_ffn_workspace(m, d, f))
            assert torch.equal(a, b)
