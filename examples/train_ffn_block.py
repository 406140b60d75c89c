"""Trains the feed-forward half of a pre-norm transformer layer,

    out = x + dropout(gated_ffn(layer_norm(x))),

on one GPU: its five tensors live in the flat buffers of the optimizer step.
The weights that the forward and backward calls read are views of the fp16
copy that zero_step writes, and the gradients that they write are views of the
flat fp16 gradient that zero_step reads, times the loss scale.

    python examples/train_ffn_block.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import zero_partitioned_mixed_layout_gb300 as zp  # noqa: E402


class FeedForwardBlock:
    """The block and its optimizer state; `step` trains on one batch."""

    def __init__(self, tokens, dim, inner, p_drop=0.1, loss_scale=1024.0, seed=0, lr=1e-3):
        shapes = [(inner, dim), (inner, dim), (dim, inner), (dim,), (dim,)]
        numel = [int(torch.Size(s).numel()) for s in shapes]
        layout = zp.zero_partition_layout(numel, 1, 128)
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def flat(dtype):
            return torch.zeros(layout.shard_numel, dtype=dtype, device="cuda")

        def views(buf):
            return [buf[o:o + n].view(s) for o, n, s in zip(layout.tensor_offset, numel, shapes)]

        self.master, self.m, self.v = flat(torch.float32), flat(torch.float32), flat(torch.float32)
        for w, std in zip(views(self.master)[:3], (dim ** -0.5, dim ** -0.5, inner ** -0.5)):
            w.normal_(0.0, std, generator=gen)
        views(self.master)[3].fill_(1.0)
        self.p16, self.grad = self.master.half(), flat(torch.float16)
        self.weights, self.grads = views(self.p16), views(self.grad)

        def act(*shape, dtype=torch.float16):
            return torch.empty(shape, dtype=dtype, device="cuda")

        self.normed, self.z, self.out, self.dz, self.dn, self.dx = (act(tokens, dim) for _ in range(6))
        self.gate, self.up = act(tokens, inner), act(tokens, inner)
        self.mean, self.rstd = act(tokens, dtype=torch.float32), act(tokens, dtype=torch.float32)
        # the dropout's offset lives on the device, so that a captured step draws new masks too
        self.calls = torch.zeros(1, dtype=torch.int64, device="cuda")
        self.drop = zp.Dropout(p_drop, seed, 0, self.calls)
        self.state = zp.new_state(loss_scale)
        self.ws = zp.new_workspace(1, layout.shard_numel)
        self.ffn_ws = zp.new_gated_ffn_workspace(tokens, dim, inner, backward=True)
        self.norm_ws = zp.new_layer_norm_workspace(tokens, dim)
        self.hp = zp.HParams(lr=lr, max_norm=1.0)
        self.act = zp.ZERO_ACT_SILU

    def forward(self, x):
        w_gate, w_up, w_down, w, b = self.weights
        zp.zero_layer_norm(x, w, b, self.normed, self.mean, self.rstd)
        zp.zero_gated_ffn(self.normed, w_gate, w_up, w_down, self.z, self.ffn_ws, act=self.act, gate=self.gate,
                          up=self.up)
        zp.zero_dropout_add(self.z, x, self.out, self.drop)
        return self.out

    def backward(self, x, dout):
        """dout: the output's gradient times the loss scale; returns x's."""
        w_gate, w_up, w_down, w, _ = self.weights
        zp.zero_dropout_add(dout, None, self.dz, self.drop)
        zp.zero_gated_ffn_backward(self.dz, self.normed, w_gate, w_up, w_down, self.gate, self.up, self.dn,
                                   *self.grads[:3], self.ffn_ws, act=self.act)
        zp.zero_layer_norm_backward(self.dn, x, w, self.mean, self.rstd, self.dx, *self.grads[3:], self.norm_ws,
                                    dresidual=dout)
        return self.dx

    def optimize(self):
        zp.zero_step(self.grad, self.master, self.m, self.v, self.p16, self.hp, self.state, self.ws)
        self.calls += 1

    def step(self, x, target):
        """One step on the mean squared error; returns the loss (a device scalar)."""
        err = self.forward(x).float() - target.float()
        # the loss scale is read on the device: it changes there when a step overflows
        scale = self.state.view(torch.float64)[2].float()
        self.backward(x, (err * (2.0 * scale / err.numel())).half())
        self.optimize()
        return err.square().mean()


def main(steps=60, tokens=512, dim=256, inner=1024):
    """Learns a fixed random map of its inputs; returns the losses."""
    gen = torch.Generator(device="cuda").manual_seed(1)
    block = FeedForwardBlock(tokens, dim, inner)
    teacher = torch.randn(dim, dim, device="cuda", generator=gen) * dim ** -0.5
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, dim, device="cuda", generator=gen).half()
        target = x.float() + torch.tanh(x.float() @ teacher)
        losses.append(block.step(x, target.half()))
    losses = [float(v) for v in losses]
    st = zp.parse_state(block.state)
    print(f"{steps} steps ({st['skipped']} skipped, loss scale {st['loss_scale']:.0f}): "
          f"loss {losses[0]:.4f} -> {losses[-1]:.4f}")
    return losses


if __name__ == "__main__":
    main()
