"""The feed-forward sub-block on the GPU at the edges of its sizes, values and
waits, against its formulas in binary64 (sublayer_ref.py)."""
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
