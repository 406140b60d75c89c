"""The feed-forward sub-block on the GPU at the edges of its sizes, values and
waits, against its formulas in binary64 (sublayer_ref.py)."""
import ctypes

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


def randn(shape, dtype, seed, std=1.0, mean=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(shape, device="cuda").normal_(mean, std, generator=gen).to(dtype)


def close(got, want, dtype, what):
    value, err = want
    ref.check(got, value, ref.rounded(value, err, dtype), what)


@pytest.mark.parametrize("rows", [0, 1, 700, 5000])
def test_layer_norm_of_no_columns(zp, rows):
    z = torch.empty((rows, 0), dtype=torch.float16, device="cuda")
    stats = torch.empty(rows, device="cuda")
    none = torch.empty(0, device="cuda")
    zp.zero_layer_norm(z, None, None, z)
    zp.zero_layer_norm_backward(z, z, None, stats, stats, z, none, none, zp.new_layer_norm_workspace(rows, 0))
    torch.cuda.synchronize()


@pytest.mark.parametrize("shape", [(1217, 1600), (1216, 2048), (2433, 4096), (305, 16384)], ids=str)
def test_layer_norm_backward_repeats_its_weight_gradients(zp, shape):
    """Rows that leave some teams without one, and the last copies of all teams
    just behind their last row: the sums over the block, which take the place
    of the staged rows, are right and the same bits on every run."""
    rows, cols = shape
    dt = torch.bfloat16
    x, dy, w = randn(shape, dt, 1, 1.5, 0.5), randn(shape, dt, 2), randn((cols,), dt, 3, 0.2, 1.0)
    r = ref.layer_norm(x, None, None, 1e-5)
    mean, rstd = r["mean"][0].float(), r["rstd"][0].float()
    ws, dx = zp.new_layer_norm_workspace(rows, cols), torch.empty_like(x)
    dw, db = (torch.empty(cols, device="cuda") for _ in range(2))
    b = ref.layer_norm_backward(dy, x, w, mean, rstd)
    first = None
    for _ in range(50):
        dw.fill_(float("nan"))
        db.fill_(float("nan"))
        zp.zero_layer_norm_backward(dy, x, w, mean, rstd, dx, dw, db, ws)
        if first is None:
            first = dw.clone(), db.clone()
            close(dw, b["dweight"], torch.float32, "dweight")
            close(db, b["dbias"], torch.float32, "dbias")
        assert torch.equal(dw, first[0]) and torch.equal(db, first[1])


@pytest.mark.parametrize("tokens", [1, 3])
def test_gated_ffn_with_rows_up_to_the_limit(zp, tokens):
    """An inner width of 2^31 - 512, the largest: the rows of the gate's and
    the up matrix (one element each) end within a grid's step of 2^31.  x is
    one or a power of two, so gate and up are the weights, exactly; w_down is
    zero but for some columns, so y is their sum."""
    inner, dt = 2 ** 31 - 512, torch.float16
    x = torch.tensor([[1.0], [2.0], [0.5]], dtype=dt, device="cuda")[:tokens]
    wg, wu = (torch.empty((inner, 1), dtype=dt, device="cuda") for _ in range(2))
    gen = torch.Generator(device="cuda").manual_seed(7)
    for w in (wg, wu):
        w.uniform_(0.5, 1.5, generator=gen)
    wd = torch.zeros((1, inner), dtype=dt, device="cuda")
    last = slice(inner - 6000, inner)
    wd[:, last] = 2.0 ** -10
    wd[:, :100] = -(2.0 ** -10)
    y = torch.full((tokens, 1), float("nan"), dtype=dt, device="cuda")
    gate, up = (torch.empty((tokens, inner), dtype=dt, device="cuda") for _ in range(2))
    ws = zp.new_gated_ffn_workspace(tokens, 1, inner)
    zp.zero_gated_ffn(x, wg, wu, wd, y, ws, gate=gate, up=up)
    for m in range(tokens):
        # (a product with a power of two is exact: every element normal)
        assert torch.equal(gate[m], wg[:, 0] * x[m]) and torch.equal(up[m], wu[:, 0] * x[m])
    for part, sign in ((slice(0, 100), -1.0), (last, 1.0)):
        g, u = (x.double() @ w[part].double().T for w in (wg, wu))
        v = ref.act(ref.SILU, g)
        terms = v[0] * u * 2.0 ** -10
        # the sum's other terms are zeros: 6100 roundings of it at most
        err = (v[2] * u.abs() * 2.0 ** -10 + 6200 * ref.U32 * terms.abs()).sum(1, keepdim=True)
        want = (sign * terms.sum(1, keepdim=True), err) if part.start == 0 else (
            want[0] + terms.sum(1, keepdim=True), want[1] + err)
    close(y, want, dt, "y")
    del ws, gate, up, wg, wu, wd
    torch.cuda.empty_cache()  # (100 GB)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [256, 1600, 2049, 9001])
def test_layer_norm_workspace_of_the_largest_batch_serves_all(zp, cols, dtype):
    """One workspace, made for the longest batch, at row counts around those
    where the blocks' plan changes."""
    dt, most = TYPES[dtype], 1300
    ws = zp.new_layer_norm_workspace(most, cols)
    x, dy = randn((most, cols), dt, 4, 1.5, 0.5), randn((most, cols), dt, 5)
    dx = torch.empty_like(x)
    dw, db = (torch.empty(cols, device="cuda") for _ in range(2))
    for rows in (1, 2, 7, 8, 9, 151, 152, 153, 304, 305, 456, 457, 608, 609, 760, 761, 912, 913, 1215, 1216, 1300):
        r = ref.layer_norm(x[:rows], None, None, 1e-5)
        mean, rstd = r["mean"][0].float(), r["rstd"][0].float()
        zp.zero_layer_norm_backward(dy[:rows], x[:rows], None, mean, rstd, dx[:rows], dw, db, ws)
        b = ref.layer_norm_backward(dy[:rows], x[:rows], None, mean, rstd)
        close(dx[:rows], b["dx"], dt, f"dx of {rows}")
        close(dw, b["dweight"], torch.float32, f"dweight of {rows}")
        close(db, b["dbias"], torch.float32, f"dbias of {rows}")


@pytest.mark.parametrize("dim,inner", [(64, 256), (51, 99), (1600, 640)])
def test_gated_ffn_workspace_of_the_largest_batch_serves_all(zp, dim, inner):
    for most in (3, 5, 40):
        ws = zp.new_gated_ffn_workspace(most, dim, inner)
        for m in [k for k in (1, 2, 3, 4, 5, 9, 40) if k <= most]:
            dt = torch.float16
            x, wg, wu, wd = (randn(s, dt, 10 + k, std) for k, (s, std) in enumerate(
                [((m, dim), 1.0), ((inner, dim), dim ** -0.5), ((inner, dim), dim ** -0.5), ((dim, inner), inner ** -0.5)]))
            y = torch.empty_like(x)
            zp.zero_gated_ffn(x, wg, wu, wd, y, ws)
            close(y, ref.gated_ffn(x, wg, wu, wd, ref.SILU)["y"], dt, f"{m} tokens")


# ------------------------------------------------------------------ waits that run out

@pytest.fixture
def short_copies(zp):
    """Makes the waits of one kind of product run out after a fifth of a
    second: the copies that they wait for are asked for a little too small."""
    so = zp.lib()
    so.zero_test_gated_ffn_waits.argtypes = [ctypes.c_int32, ctypes.c_uint64]
    so.zero_test_gated_ffn_waits.restype = None
    yield lambda epilogue: so.zero_test_gated_ffn_waits(epilogue, 200_000_000)
    so.zero_test_gated_ffn_waits(-1, 0)


STORE, GATE, GATE_BWD = 0, 1, 2

# pairs of CTAs, several tiles to each; k cut among a cluster; widths whose outputs leave without TMA
STALLED = [(1200, 512, 2048), (40, 512, 1024), (200, 101, 203), (2100, 1001, 1501)]


@pytest.mark.parametrize("size", STALLED, ids=str)
def test_a_wait_that_gave_up_leaves_nan_in_the_outputs(zp, short_copies, size):
    (m, d, f), dt = size, torch.bfloat16
    x, wg, wu, wd = (randn(s, dt, 20 + k, std) for k, (s, std) in enumerate(
        [((m, d), 1.0), ((f, d), d ** -0.5), ((f, d), d ** -0.5), ((d, f), f ** -0.5)]))
    dy = randn((m, d), dt, 25)
    ws = zp.new_gated_ffn_workspace(m, d, f, True)

    def forward():
        y, gate, up = (torch.zeros(s, dtype=dt, device="cuda") for s in ((m, d), (m, f), (m, f)))
        zp.zero_gated_ffn(x, wg, wu, wd, y, ws, gate=gate, up=up)
        return y, gate, up

    def backward(gate, up):
        out = [torch.zeros(s, dtype=t, device="cuda") for s, t in
               (((m, d), dt), ((f, d), torch.float32), ((f, d), torch.float32), ((d, f), torch.float32))]
        zp.zero_gated_ffn_backward(dy, x, wg, wu, wd, gate, up, *out, ws)
        return out

    want = forward()
    grads = backward(*want[1:])
    torch.cuda.synchronize()
    assert zp.zero_workspace_stalls(ws) == 0

    def stalled(kind, call):
        before = zp.zero_workspace_stalls(ws)
        short_copies(kind)
        out = call()
        torch.cuda.synchronize()
        short_copies(-1)
        assert zp.zero_workspace_stalls(ws) > before
        return out

    # no block of any tile's k was whole: everything that the products write is NaN
    for t in stalled(GATE, forward):
        assert bool(torch.isnan(t).all())
    y, gate, up = stalled(STORE, forward)
    assert bool(torch.isnan(y).all()) and torch.equal(gate, want[1]) and torch.equal(up, want[2])
    for t in stalled(GATE_BWD, lambda: backward(*want[1:])):
        assert bool(torch.isnan(t).all())
    for t in stalled(STORE, lambda: backward(*want[1:])):
        assert bool(torch.isnan(t).all())
    # the workspace serves the next calls as before
    assert all(torch.equal(a, b) for a, b in zip(forward(), want))
    assert all(torch.equal(a, b) for a, b in zip(backward(*want[1:]), grads))


# ------------------------------------------------------------------ the mean

@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(3, 30), (3, 1601), (700, 1600), (2, 6001), (1300, 1608), (1300, 1000), (2500, 5000),
                                   (2500, 8008), (5, 20001), (3, 40000)], ids=str)
def test_layer_norm_of_equal_values_is_the_bias(zp, shape, dtype):
    """Sums of 1000 (a multiple of 8) up to 2^27 are exact in binary32 in any
    order, so the mean, their quotient by the width, is exact too, and nothing
    is left for rstd (316 at this eps) to magnify."""
    (rows, cols), dt = shape, TYPES[dtype]
    x = torch.full(shape, 1000.0, dtype=dt, device="cuda")
    b = randn((cols,), dt, 31)
    for weight, bias, want in ((None, None, torch.zeros_like(x)), (b, b, b.expand(rows, cols))):
        y, mean, rstd = torch.empty_like(x), *(torch.empty(rows, device="cuda") for _ in range(2))
        zp.zero_layer_norm(x, weight, bias, y, mean, rstd)
        assert bool((mean == 1000.0).all()) and torch.equal(y, want)
        s = torch.empty_like(x)
        zp.zero_layer_norm(x, weight, bias, y, mean, rstd, residual=torch.zeros_like(x), sum_out=s)
        assert bool((mean == 1000.0).all()) and torch.equal(y, want) and torch.equal(s, x)


@pytest.mark.parametrize("cols", [1, 3, 7, 10, 30, 49, 100, 257, 600, 1000, 1601, 2049, 2568, 5000, 8200, 20001])
def test_layer_norm_mean_is_the_rounded_quotient(zp, cols):
    """Rows of small whole numbers: their sums are exact in binary32 in any
    order, so mean is that sum divided by cols and rounded once."""
    rows = 2500
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randint(-200, 256, (rows, cols), device="cuda", generator=gen)
    for dt in (torch.float32, torch.bfloat16):
        t, mean = x.to(dt), torch.empty(rows, device="cuda")
        y = torch.empty_like(t)
        zp.zero_layer_norm(t, None, None, y, mean)
        want = x.sum(1).float() / torch.full((rows,), float(cols), device="cuda")
        assert torch.equal(mean, want) and torch.equal(mean, (x.sum(1).double() / cols).float())


def test_layer_norm_mean_of_an_infinite_row(zp):
    x = randn((4, 257), torch.float32, 33)
    x[1, 200], x[2, 0] = float("inf"), -float("inf")
    y, mean = torch.empty_like(x), torch.empty(4, device="cuda")
    zp.zero_layer_norm(x, None, None, y, mean)
    assert mean[1] == float("inf") and mean[2] == -float("inf") and bool(torch.isfinite(mean[[0, 3]]).all())
    assert bool(torch.isnan(y[1:3]).any(1).all()) and bool(torch.isfinite(y[[0, 3]]).all())


def test_a_dropout_moved_on_draws_the_next_mask(zp):
    x, out = randn((40, 100), torch.float32, 41), torch.empty((40, 100), device="cuda")
    drop = zp.Dropout(0.5, 3, 10)
    for offset in (10, 11):
        zp.zero_dropout_add(x, None, out, drop)
        close(out, ref.dropout_add(x, None, (0.5, 3, offset)), torch.float32, f"offset {offset}")
        drop.offset += 1
    drop.d_offset = torch.tensor([88], dtype=torch.int64, device="cuda")
    zp.zero_dropout_add(x, None, out, drop)
    close(out, ref.dropout_add(x, None, (0.5, 3, 100)), torch.float32, "offset 100")
