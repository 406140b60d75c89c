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
