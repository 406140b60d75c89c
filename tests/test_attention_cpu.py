"""The attention sub-block without a GPU: the reference that the GPU tests
compare with (the gradients against differences, the angles against known
ones), the rotation's frequencies, and the C calls' argument checks."""
import ctypes
import math

import numpy as np
import pytest
import torch

import attention_ref as ref


@pytest.fixture(scope="module")
def zp():
    from zero_partitioned_mixed_layout_gb300 import _build
    _build.build()
    import zero_partitioned_mixed_layout_gb300 as zp
    zp.binding._attention_lib()
    return zp


def _directional(f, x, v, h=1e-5):
    return (f(x + h * v) - f(x - h * v)) / (2 * h)


# ------------------------------------------------------------------ the reference

def test_pi():
    assert ref.PI / 2 ** ref._BITS == math.pi
    assert hex(ref.PI >> (ref._BITS - 64))[2:] == "3243f6a8885a308d3"  # 3.243F6A8885A308D3 in hexadecimal


def test_angles():
    a = ref.angles([0, 1, -1, 7], [1.0, 0.25])
    assert torch.allclose(a, torch.tensor([[0.0, 0.0], [1.0, 0.25], [-1.0, -0.25], [7 - 2 * math.pi, 1.75]],
                                          dtype=torch.float64), atol=1e-15)
    # 10^22 radians: Payne and Hanek's textbook case, cos(10^22) = 0.5232147853951389
    assert abs(math.cos(float(ref.angles([10 ** 22], [1.0]))) - 0.5232147853951389) < 1e-14


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_is_orthogonal(interleaved):
    gen = torch.Generator().manual_seed(1)
    x = torch.randn(5, 3, 10, dtype=torch.float64, generator=gen)
    angle = ref.angles([0, 3, 100, -7, 12345], [1.0, 0.3, 0.01])
    y = ref.rotate(x, angle, 6, interleaved)[0]
    assert torch.allclose(y.square().sum(-1), x.square().sum(-1)) and torch.equal(y[..., 6:], x[..., 6:])
    assert torch.allclose(ref.rotate(y, angle, 6, interleaved, back=True)[0], x, atol=1e-14)
    # a pair's product with a rotated pair depends on the distance alone
    z = ref.rotate(x, angle + ref.angles([11] * 5, [1.0, 0.3, 0.01]), 6, interleaved)[0]
    w = ref.rotate(x, ref.angles([11] * 5, [1.0, 0.3, 0.01]), 6, interleaved)[0]
    assert torch.allclose((z * w).sum(-1), (y * x).sum(-1))


@pytest.mark.parametrize("interleaved", [False, True])
def test_head_norm_gradient_against_differences(interleaved):
    gen = torch.Generator().manual_seed(2)
    x, dy, vx = (torch.randn(4, 3, 10, dtype=torch.float64, generator=gen) for _ in range(3))
    w, vw = (torch.randn(10, dtype=torch.float64, generator=gen) for _ in range(2))
    pos = [0, 5, 9, -3]
    angle = ref.angles(pos, [1.0, 0.3, 0.01])
    f = lambda x_, w_: (ref.head_norm(x_, w_, angle, pos, 6, interleaved, 1e-6)[0] * dy).sum()  # noqa: E731
    g = ref.head_norm_backward(dy, x, w, angle, pos, 6, interleaved, 1e-6)
    # truncation about 1e-10, rounding about 1e-10
    assert abs(_directional(lambda t: f(t, w), x, vx) - (g["dx"][0] * vx).sum()) < 1e-6
    assert abs(_directional(lambda t: f(x, t), w, vw) - (g["dw"][0] * vw).sum()) < 1e-6


def test_seen():
    def by_hand(lq, lk, window, sinks):
        out = torch.zeros(lq, lk, dtype=torch.bool)
        for i in range(lq):
            p = i + lk - lq
            for j in range(lk):
                out[i, j] = j <= p and (window is None or j > p - window or j < sinks)
        return out
    for args in [(5, 5, 2, 0), (5, 5, 2, 1), (3, 9, 4, 2), (4, 2, 3, 1), (6, 6, None, 0), (1, 7, 1, 9), (3, 0, 2, 1)]:
        assert torch.equal(ref.seen(*args), by_hand(*args)), args


@pytest.mark.parametrize("lq,lk,window,sinks", [(6, 6, None, 0), (7, 7, 3, 2), (3, 8, 4, 1), (5, 3, 2, 0)])
def test_attention_gradient_against_differences(lq, lk, window, sinks):
    gen = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, dtype=torch.float64, generator=gen)  # noqa: E731
    ref.UT[torch.float64] = ref.TINY[torch.float64] = 0.0
    q, k, v, dout = rnd(lq, 4, 5), rnd(lk, 2, 5), rnd(lk, 2, 5), rnd(lq, 4, 5)
    f = lambda *a: (ref.attention(*a, window, sinks, 0.4, torch.float64)["out"][0] * dout).sum()  # noqa: E731
    kept = ref.attention(q, k, v, window, sinks, 0.4, torch.float64)
    got = ref.attention_backward(dout, q, k, v, kept["out"][0], kept["lse"][0], window, sinks, 0.4, torch.float64)
    args = [q, k, v]
    for n, name in enumerate(("dq", "dk", "dv")):
        t = rnd(*args[n].shape)
        d = _directional(lambda z: f(*args[:n], z, *args[n + 1:]), args[n], t)
        # third derivatives of order 100 times step^2 = 1e-10
        assert abs(d - (got[name][0] * t).sum()) < 1e-6 * max(1.0, abs(d)), name


def test_attention_of_queries_before_every_key():
    q, k = torch.ones(4, 1, 8), torch.ones(2, 1, 8)
    r = ref.attention(q, k, k, 5, 0, 1.0, torch.float16)
    assert bool((r["out"][0][:2] == 0).all()) and r["lse"][0][0, :2].tolist() == [-math.inf] * 2
    assert bool(torch.isfinite(r["lse"][0][0, 2:]).all())


# ------------------------------------------------------------------ frequencies

def test_rotary_turns(zp):
    f = [10000.0 ** (-2 * i / 128) for i in range(64)] + [0.0, -0.5, 3.7, 1e-12, -1e-9, 7.0, 2.0 ** 20, -1048575.3]
    for got, want in zip(zp.zero_rotary_turns(f).tolist(), ref.turns(f)):
        off = (got - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1
    assert zp.zero_rotary_turns([]).size == 0
    for bad in (math.nan, math.inf, -math.inf, 2.0 ** 20 + 1):
        with pytest.raises(zp.ZeroError):
            zp.zero_rotary_turns([1.0, bad])
    lib = zp.binding._attention_lib()
    x, y = (ctypes.c_double * 1)(1.0), (ctypes.c_uint64 * 1)()
    assert lib.zero_rotary_turns(x, -1, y) == EINVAL and lib.zero_rotary_turns(None, 1, y) == EINVAL
    assert lib.zero_rotary_turns(x, 1, None) == EINVAL and lib.zero_rotary_turns(None, 0, None) == 0


# ------------------------------------------------------------------ argument checks (nothing is launched)

EINVAL, EALIGN, EDTYPE, ESIZE, EWORKSPACE = -1, -2, -3, -4, -5
F16, BF16, F32 = 0, 1, 2
P = 0x1000  # never dereferenced: the call fails a check that comes before


def qk(zp, **kw):
    a = dict(q=P, q_ld=128, q_hd=64, k=P, k_ld=64, k_hd=64, qw=None, kw=None, wdtype=F16, turns=None, rot=0, pairs=0,
             positions=None, qo=P, qo_ld=128, qo_hd=64, ko=P, ko_ld=64, ko_hd=64, tokens=4, q_heads=2, k_heads=1, dim=64,
             eps=1e-6, dtype=F16)
    assert not set(kw) - set(a)
    a.update(kw)
    r = zp.binding._Rotary(a["turns"], a["rot"], a["pairs"])
    return zp.binding._attention_lib().zero_qk_norm(
        a["q"], a["q_ld"], a["q_hd"], a["k"], a["k_ld"], a["k_hd"], a["qw"], a["kw"], a["wdtype"], ctypes.byref(r),
        a["positions"], a["qo"], a["qo_ld"], a["qo_hd"], a["ko"], a["ko_ld"], a["ko_hd"], a["tokens"], a["q_heads"],
        a["k_heads"], a["dim"], a["eps"], a["dtype"], None)


@pytest.mark.parametrize("change,code", [
    (dict(dtype=3), EDTYPE), (dict(wdtype=BF16), EDTYPE), (dict(dtype=F32, wdtype=F16), EDTYPE),
    (dict(tokens=-1), EINVAL), (dict(q_heads=-1), EINVAL), (dict(k_heads=-1), EINVAL), (dict(dim=-2), EINVAL),
    (dict(eps=-1e-9), EINVAL), (dict(eps=math.nan), EINVAL), (dict(q=None), EINVAL), (dict(ko=None), EINVAL),
    (dict(q=P + 1), EALIGN), (dict(q_ld=-64), EINVAL), (dict(q_ld=1 << 38), ESIZE),
    (dict(q_ld=1 << 37, tokens=1 << 30), ESIZE), (dict(q_hd=1 << 38), ESIZE),
    (dict(tokens=1 << 31), ESIZE), (dict(dim=257), ESIZE), (dict(q_heads=(1 << 20) + 1), ESIZE),
    (dict(q_heads=1 << 20, k_heads=1), ESIZE), (dict(rot=65), ESIZE), (dict(rot=3), ESIZE), (dict(rot=-2), ESIZE),
    (dict(q=P), EINVAL),  # no device memory
], ids=str)
def test_qk_norm_refuses(zp, change, code):
    assert qk(zp, **change) == code


def test_qk_norm_of_nothing(zp):
    none = dict(q=None, k=None, qo=None, ko=None)
    assert qk(zp, tokens=0, **none) == 0 and qk(zp, q_heads=0, k_heads=0, **none) == 0 and qk(zp, dim=0, **none) == 0


def test_qk_norm_workspace(zp):
    f = zp.zero_qk_norm_workspace_bytes
    assert f(1, 1, 1, 64) % 256 == 0 and f(0, 0, 0, 0) == 256 and f(-1, 1, 1, 64) == 0 and f(1, 1, 1, 257) == 0
    # no larger call needs less than a smaller one
    sizes = [f(t, h, g, d) for t in (1, 5000) for h in (1, 64) for g in (0, 8) for d in (1, 64, 256)]
    for i, t in enumerate([(t, h, g, d) for t in (1, 5000) for h in (1, 64) for g in (0, 8) for d in (1, 64, 256)]):
        for j, u in enumerate([(t, h, g, d) for t in (1, 5000) for h in (1, 64) for g in (0, 8) for d in (1, 64, 256)]):
            if all(x <= y for x, y in zip(t, u)):
                assert sizes[i] <= sizes[j]
    lib = zp.binding._attention_lib()
    back = [P, 64, 64] * 4 + [None, None, F16, None, None] + [P, 64, 64] * 2 + [None, None]
    # (sizes are checked first, then the arrays: no device memory)
    assert lib.zero_qk_norm_backward(*back, BF16, 4, 1, 1, 64, 1e-6, F16, P, 1 << 30, None) == EDTYPE
    assert lib.zero_qk_norm_backward(*back, F16, 0, 1, 1, 64, 1e-6, F16, None, 0, None) == EWORKSPACE
    assert lib.zero_qk_norm_backward(*back, F16, 0, 1, 1, 64, 1e-6, F16, 128, 1 << 30, None) == EALIGN
    assert lib.zero_qk_norm_backward(*back, F16, 0, 1, 1, 64, 1e-6, F16, 4096, 256, None) == EWORKSPACE


def attn(zp, backward=False, **kw):
    a = dict(q=P, q_ld=128, q_hd=64, k=P, k_ld=64, k_hd=64, out=P, lse=None, ws=P, wsb=1 << 40, q_tokens=4, k_tokens=4,
             sequences=1, q_heads=2, k_heads=1, dim=64, dtype=F16, window=4, sinks=0, scale=0.125, q_offsets=None,
             k_offsets=None, k_lengths=None)
    assert not set(kw) - set(a)
    a.update(kw)
    s = zp.binding._Attention(a["q_tokens"], a["k_tokens"], a["sequences"], a["q_heads"], a["k_heads"], a["dim"],
                              a["dtype"], a["window"], a["sinks"], a["scale"], a["q_offsets"], a["k_offsets"],
                              a["k_lengths"])
    q, k, o = (a["q"], a["q_ld"], a["q_hd"]), (a["k"], a["k_ld"], a["k_hd"]), (a["out"], a["q_ld"], a["q_hd"])
    lib = zp.binding._attention_lib()
    if backward:
        return lib.zero_window_attention_backward(ctypes.byref(s), *o, *q, *k, *k, *o, a["lse"], *q, *k, *k, a["ws"],
                                                  a["wsb"], None)
    return lib.zero_window_attention(ctypes.byref(s), *q, *k, *k, *o, a["lse"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("change,code", [
    (dict(dtype=F32), EDTYPE), (dict(dtype=-1), EDTYPE), (dict(q_tokens=-1), EINVAL), (dict(k_tokens=-1), EINVAL),
    (dict(sequences=-1), EINVAL), (dict(q_heads=0), EINVAL), (dict(k_heads=0), EINVAL), (dict(dim=0), EINVAL),
    (dict(window=0), EINVAL), (dict(sinks=-1), EINVAL), (dict(scale=0.0), EINVAL), (dict(scale=-1.0), EINVAL),
    (dict(scale=math.nan), EINVAL), (dict(scale=math.inf), EINVAL), (dict(scale=1e300), EINVAL),
    (dict(q_heads=3, k_heads=2), ESIZE), (dict(dim=12), ESIZE), (dict(dim=136), ESIZE),
    (dict(q_heads=1 << 16), ESIZE), (dict(q_tokens=(1 << 31) - 511), ESIZE), (dict(k_tokens=(1 << 31) - 511), ESIZE),
    (dict(sequences=(1 << 31) - 511), ESIZE), (dict(k_tokens=5), ESIZE), (dict(sequences=2), EINVAL),
    (dict(sequences=0), EINVAL), (dict(k_lengths=P), EINVAL), (dict(q_offsets=P + 4), EALIGN), (dict(q_offsets=P), EINVAL),
    (dict(q=None), EINVAL), (dict(q=P + 8), EINVAL), (dict(q_ld=-64), EINVAL), (dict(q_ld=1 << 38), ESIZE),
], ids=str)
def test_window_attention_refuses(zp, change, code, backward):
    assert attn(zp, backward, **change) == code


def test_window_attention_without_rows_checks_its_workspace(zp):
    none = dict(q_tokens=0, k_tokens=0, q=None, k=None, out=None)
    assert attn(zp, ws=None, **none) == EWORKSPACE and attn(zp, ws=128, **none) == EALIGN
    assert attn(zp, wsb=255, **none) == EWORKSPACE


def test_window_attention_workspace(zp):
    f = zp.zero_window_attention_workspace_bytes
    base = dict(q_tokens=100, k_tokens=100, sequences=2, q_heads=4, k_heads=2, head_dim=64, window=10, sinks=2)
    for backward in (False, True):
        least = f(**base, backward=backward)
        assert least >= 256 and least % 256 == 0
        # more of anything needs no less
        for name, more in (("q_tokens", [101, 127, 128, 129, 1000, 5000]), ("k_tokens", [101, 5000, 1 << 20]),
                           ("sequences", [3, 50, 51]), ("head_dim", [72, 128])):
            last = least
            for n in more:
                now = f(**{**base, name: n}, backward=backward)
                assert now >= last, (name, n, backward)
                last = now
        assert f(**{**base, "head_dim": 136}, backward=backward) == 0 and f(**{**base, "window": 0}, backward=backward) == 0
    assert f(**base, backward=True) >= f(**base)
    # sums of first keys' parts, for no more sequences than are long enough to have parts
    many = dict(q_tokens=65536, k_tokens=65536, q_heads=8, k_heads=8, head_dim=128, window=256, sinks=4, backward=True)
    sizes = [f(**many, sequences=n) for n in (1, 64, 256, 257, 513, 4096)]
    assert sizes == sorted(sizes) and sizes[-1] < 500e6


def test_binding_refuses(zp):
    q = torch.zeros(4, 2, 64, dtype=torch.float16)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        zp.zero_window_attention(q, q, q, q.clone(), ws)
    with pytest.raises(ValueError, match="CUDA"):
        zp.zero_qk_norm(q, q, None, None, q.clone(), q.clone())
    with pytest.raises(ValueError, match="three dimensions"):
        zp.zero_window_attention(q[0], q, q, q.clone(), ws)
    with pytest.raises(ValueError, match="head dimension"):
        zp.zero_window_attention(q, q[..., :8], q, q.clone(), ws)
    with pytest.raises(ValueError, match="tokens"):
        zp.zero_qk_norm(q, q[:2], None, None, q.clone(), q.clone())


def test_bounds_follow_the_types():
    """The rounding to a narrower type is most of a bound (so that a kernel
    that lost more than it says would show)."""
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(40, 2, 64, dtype=torch.float64, generator=gen) for _ in range(3))
    r = {t: ref.attention(q, k, v, 16, 1, 0.125, t)["out"][1] for t in (torch.float16, torch.bfloat16)}
    assert float((r[torch.bfloat16] / r[torch.float16]).median()) > 5
    assert float(r[torch.bfloat16].max()) < 2.0 ** -8 * 4
    assert np.isfinite(float(r[torch.float16].max()))
