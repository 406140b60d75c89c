"""The feed-forward sub-block's operators together with the optimizer step, as
examples/train_ffn_block.py uses them: one step's flat gradient against the
composition's in binary64 (torch's autograd), and that it trains."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import sublayer_ref as ref  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from zero_partitioned_mixed_layout_gb300 import _build
    _build.build()
    spec = importlib.util.spec_from_file_location("train_ffn_block", os.path.join(ROOT, "examples", "train_ffn_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("tokens", [3, 200])
def test_one_step_against_autograd(example, tokens):
    """Every gradient passes at most five f16 roundings (the norm, gate or up,
    their product, dz, dgate or dup) of relative size 2^-11 each, which enter
    it independently: the difference in norm stays below five of them."""
    dim, inner = 128, 256
    block = example.FeedForwardBlock(tokens, dim, inner, p_drop=0.25, loss_scale=256.0, seed=5)
    gen = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(tokens, dim, device="cuda", generator=gen).half()
    dout = torch.randn(tokens, dim, device="cuda", generator=gen).half()
    out = block.forward(x).clone()
    dx = block.backward(x, dout).clone()
    leaves = [x.double().requires_grad_()] + [w.double().requires_grad_() for w in block.weights]
    xx, wg, wu, wd, w, b = leaves
    n = torch.nn.functional.layer_norm(xx, (dim,), w, b, 1e-5)
    z = (torch.nn.functional.silu(n @ wg.T) * (n @ wu.T)) @ wd.T
    keep = torch.from_numpy(ref.keep_mask(tokens, dim, 0.25, 5, 0)).cuda()
    want = xx + torch.where(keep, z / 0.75, torch.zeros_like(z))
    want.backward(dout.double())
    for got, exact in [(out, want.detach())] + list(zip([dx] + block.grads, [t.grad for t in leaves])):
        assert float((got.double() - exact).norm()) <= 5 * 2.0 ** -11 * float(exact.norm())
    # the padding of the flat gradient is not written
    assert bool((block.grad[sum(g.numel() for g in block.grads):] == 0).all())


def test_the_example_trains(example):
    losses = example.main(steps=60)
    assert losses[-1] < 0.5 * losses[0]


def test_a_captured_step_draws_new_masks(example):
    """The whole step in a CUDA graph: replays equal eager steps bit for bit,
    the dropout's offset moving on with each."""
    def batch(k):
        gen = torch.Generator(device="cuda").manual_seed(100 + k)
        x = torch.randn(64, 128, device="cuda", generator=gen).half()
        return x, torch.tanh(x.float()).half()

    eager, graphed = (example.FeedForwardBlock(64, 128, 256, p_drop=0.3, seed=3) for _ in range(2))
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):  # first calls outside capture
        graphed.step(*batch(0))
    side.synchronize()
    eager.step(*batch(0))
    x, target = batch(1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed.step(x, target)
    for k in range(1, 4):
        new = batch(k)
        x.copy_(new[0])
        target.copy_(new[1])
        graph.replay()
        eager.step(*new)
        assert torch.equal(graphed.out, eager.out) and torch.equal(graphed.master, eager.master)
