"""The feed-forward sub-block without a GPU: the reference the GPU tests
compare with (Philox against its published answers, the gradients against
differences) and the C calls' argument checks."""
import ctypes

import numpy as np
import pytest
import torch

import sublayer_ref as ref


@pytest.fixture(scope="module")
def zp():
    from zero_partitioned_mixed_layout_gb300 import _build
    _build.build()
    import zero_partitioned_mixed_layout_gb300 as zp
    zp.binding._sublayer_lib()
    return zp


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8)),
    ((0xffffffff,) * 4, (0xffffffff,) * 2, (0x408f276d, 0x41c83b0e, 0xa20bc7c6, 0x6d5451fd)),
    ((0x243f6a88, 0x85a308d3, 0x13198a2e, 0x03707344), (0xa4093822, 0x299f31d0),
     (0xd16cfe09, 0x94fdcceb, 0x5001e420, 0x24126ea1)),
])
def test_philox_known_answers(counter, key, want):
    assert tuple(int(x) for x in ref.philox(counter, key)) == want


def test_keep_mask_rate_and_streams():
    m = ref.keep_mask(200, 1001, 0.3, 7, 5)
    # 200,200 draws: the rate within five standard deviations
    assert abs(m.mean() - 0.7) < 5 * np.sqrt(0.21 / m.size)
    assert ref.keep_mask(3, 9, 0.0, 7, 5).all() and not ref.keep_mask(3, 9, 1.0, 7, 5).any()
    other = ref.keep_mask(200, 1001, 0.3, 7, 5 + 2 ** 32)
    assert abs((m == other).mean() - 0.58) < 0.01
    # a narrower matrix sees the same words
    assert (ref.keep_mask(200, 7, 0.3, 7, 5) == m[:, :7]).all()


def _directional(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


def test_layer_norm_gradient_against_differences():
    gen = torch.Generator().manual_seed(3)
    x, dy, v = (torch.randn(5, 17, dtype=torch.float64, generator=gen) for _ in range(3))
    w, b, vw = (torch.randn(17, dtype=torch.float64, generator=gen) for _ in range(3))
    r = ref.layer_norm(x, w, b, 1e-5)
    g = ref.layer_norm_backward(dy, x, w, r["mean"][0], r["rstd"][0])
    y = lambda x_, w_, b_: (ref.layer_norm(x_, w_, b_, 1e-5)["y"][0] * dy).sum()  # noqa: E731
    # central differences of step 1e-5: truncation about 1e-10, rounding about 1e-10
    assert abs(_directional(lambda t: y(t, w, b), x, v) - (g["dx"][0] * v).sum()) < 1e-6
    assert abs(_directional(lambda t: y(x, t, b), w, vw) - (g["dweight"][0] * vw).sum()) < 1e-6
    assert abs(_directional(lambda t: y(x, w, t), b, vw) - (g["dbias"][0] * vw).sum()) < 1e-6


@pytest.mark.parametrize("kind", [ref.SILU, ref.GELU])
def test_gated_ffn_gradient_against_differences(kind):
    gen = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, dtype=torch.float64, generator=gen)  # noqa: E731
    ref.UT[torch.float64] = ref.TINY[torch.float64] = 0.0
    x, wg, wu, wd, dy = rnd(6, 9), rnd(11, 9), rnd(11, 9), rnd(9, 11), rnd(6, 9)
    f = lambda *a: (ref.gated_ffn(*a, kind)["y"][0] * dy).sum()  # noqa: E731
    got = ref.gated_ffn_backward(dy, x, wg, wu, wd, x @ wg.T, x @ wu.T, kind)
    args = [x, wg, wu, wd]
    for k, name in enumerate(("dx", "dw_gate", "dw_up", "dw_down")):
        v = rnd(*args[k].shape)
        d = _directional(lambda t: f(*args[:k], t, *args[k + 1:]), args[k], v)
        # third derivatives of order 100 times step^2 = 1e-10
        assert abs(d - (got[name][0] * v).sum()) < 1e-6 * max(1.0, abs(d)), name


# ------------------------------------------------------------------ argument checks (nothing is launched)

EINVAL, EALIGN, EDTYPE, ESIZE, EWORKSPACE = -1, -2, -3, -4, -5
F16, BF16, F32 = 0, 1, 2
P = 0x1000  # never dereferenced: the call fails a check that comes before


def test_dropout_add_refusals(zp):
    so = zp.binding._sublayer_lib()
    D = zp.binding._Dropout

    def call(x=P, ld=8, rows=4, cols=8, dtype=F16, p=0.1, drop=True, out=P, res=None):
        return so.zero_dropout_add(x, ld, res, ld, out, ld, rows, cols, dtype,
                                   ctypes.byref(D(p, 1, 2, None)) if drop else None, None)
    assert call(drop=False) == EINVAL
    assert call(dtype=3) == EDTYPE and call(dtype=-1) == EDTYPE
    assert call(rows=-1) == EINVAL and call(cols=-1) == EINVAL
    assert call(p=-0.01) == EINVAL and call(p=1.01) == EINVAL and call(p=float("nan")) == EINVAL
    assert call(ld=7) == ESIZE and call(rows=1 << 32) == ESIZE and call(cols=1 << 35, ld=1 << 35) == ESIZE
    assert call(x=None) == EINVAL
    assert call(x=P + 1) == EALIGN and call(x=P + 2, dtype=F32) == EALIGN
    assert call(rows=0, x=None, out=None) == 0 and call(cols=0, x=None, out=None) == 0


def test_layer_norm_refusals(zp):
    so = zp.binding._sublayer_lib()

    def fwd(x=P, ld=8, res=None, s=None, w=P, wdt=F16, rows=4, cols=8, eps=1e-5, dtype=F16):
        return so.zero_layer_norm(x, ld, res, ld, None, s, ld, w, w, wdt, P, ld, None, None, rows, cols, eps, dtype,
                                  None)
    assert fwd(dtype=3) == EDTYPE and fwd(wdt=BF16) == EDTYPE and fwd(wdt=F16, dtype=F32) == EDTYPE
    assert fwd(rows=-1) == EINVAL and fwd(eps=-1.0) == EINVAL and fwd(eps=float("nan")) == EINVAL
    assert fwd(res=P) == EINVAL      # a sum is formed: it needs its output
    assert fwd(s=P) == EINVAL        # no sum is formed
    assert fwd(ld=7) == ESIZE and fwd(rows=1 << 32) == ESIZE
    assert fwd(x=None) == EINVAL and fwd(x=P + 1) == EALIGN
    assert fwd(rows=0) == EINVAL  # the weight's pointer is looked at (cols > 0) and is no device memory
    assert fwd(rows=0, w=None) == 0 and fwd(cols=0, ld=0) == 0

    def bwd(dtype=F16, wdt=F16, gdt=F16, drop=None, dropped=None, rows=4, cols=8, mean=P, ws=256, wsb=1 << 30, x=P):
        return so.zero_layer_norm_backward(P, 8, x, 8, None, wdt, mean, P, None, 0, P, 8, drop, dropped, 8, None, None,
                                           gdt, rows, cols, dtype, ws, wsb, None)
    assert bwd(dtype=7) == EDTYPE
    assert bwd(rows=-2) == EINVAL
    d = ctypes.byref(zp.binding._Dropout(0.5, 1, 2, None))
    assert bwd(drop=d) == EINVAL and bwd(dropped=P) == EINVAL
    assert bwd(x=None) == EINVAL
    assert bwd(rows=0, ws=None) == EWORKSPACE
    assert bwd(rows=0, ws=128) == EALIGN
    assert bwd(rows=0, wsb=16) == EWORKSPACE
    assert zp.zero_layer_norm_workspace_bytes(1 << 20, 1600) % 256 == 0


def test_gated_ffn_refusals(zp):
    so = zp.binding._sublayer_lib()

    def fwd(x=P, ld=16, wg=P, gate=None, up=None, m=4, d=16, f=32, act=0, dtype=F16, ws=256, wsb=1 << 40):
        return so.zero_gated_ffn(x, ld, wg, P, P, P, d, gate, up, m, d, f, act, dtype, ws, wsb, None)
    assert fwd(dtype=F32) == EDTYPE and fwd(dtype=9) == EDTYPE
    assert fwd(act=2) == EINVAL and fwd(act=-1) == EINVAL and fwd(m=-1) == EINVAL
    assert fwd(gate=P) == EINVAL and fwd(up=P) == EINVAL
    assert fwd(m=(1 << 31) - 1) == ESIZE
    assert fwd(ld=15) == ESIZE
    assert fwd(x=None) == EINVAL and fwd(x=P + 1) == EALIGN
    assert fwd(m=0, d=0, f=0, ld=0, ws=None) == EWORKSPACE
    assert fwd(m=0, d=0, f=0, ld=0, ws=128) == EALIGN
    assert fwd(m=0, d=0, f=0, ld=0, wsb=8) == EWORKSPACE

    def bwd(dtype=F16, gdt=F16, act=0, m=4, d=16, f=32, ws=256, wsb=1 << 40):
        return so.zero_gated_ffn_backward(P, d, P, d, P, P, P, P, P, P, d, P, P, P, gdt, m, d, f, act, dtype, ws, wsb,
                                          None)
    assert bwd(dtype=F32, gdt=F32) == EDTYPE and bwd(gdt=BF16) == EDTYPE
    assert bwd(act=5) == EINVAL and bwd(f=-1) == EINVAL and bwd(d=(1 << 31)) == ESIZE
    assert bwd(m=0, d=0, f=0, ws=None) == EWORKSPACE
    assert zp.zero_gated_ffn_workspace_bytes(100, 64, 256, True) >= 3 * 100 * 256 * 2
    assert zp.zero_gated_ffn_workspace_bytes(-1, 64, 256) == 0


def test_binding_refuses_what_the_call_cannot_take(zp):
    x = torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(ValueError):
        zp.zero_dropout_add(x, None, x, zp.Dropout(0.1, 1))
    with pytest.raises(ValueError):
        zp.zero_layer_norm(x, None, None, x)
    with pytest.raises(ValueError):
        zp.zero_gated_ffn(x, x, x, x, x, x)
    with pytest.raises(ValueError):
        zp.Dropout(0.1, 1, d_offset=torch.zeros(1, dtype=torch.int64))
