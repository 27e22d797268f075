"""A block that trains, and its use between two updates.

    python examples/updates.py          # a training step and a few tokens, with their times

TrainBlock   layer norm with residual and dropout, the MoE layer, layer norm; forward,
             backward, and AdamW on all weights (norms in fp32, the layer's in bf16 with
             states in 8 bits or with fp32 copies and 32-bit states).  A step is
             captured into one CUDA graph that reads rate and step number from the device,
             and counters for the numbers that it draws: each replay has its own masks and
             roundings.
few()        the same block for a few tokens, on the weights that the last step has
             written: no conversion, no buffers of the training batch.

Weights and inputs are random.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_layer_softmax_gb300 as moe
from examples.block import BF16, F32, U8, randn, timed


class TrainBlock:
    """h1 = stream + dropout(x), y1 = norm(h1), out = experts(y1),
    h2 = h1 + dropout(out), y2 = norm(h2)."""

    def __init__(self, T, d, E, k, f, p=0.1, eps=1e-5, bits=8, lr=1e-3):
        self.shape, self.p, self.eps, self.seed = moe.shape(T, d, E, k, f), p, eps, 1234
        self.buf = moe.allocate(self.shape)
        self.w_router, self.w_down = randn(E, d), randn(E, d, f)
        self.w_gate, self.w_up = randn(E, f, d), randn(E, f, d)
        self.norms = [torch.ones(d, **F32), torch.zeros(d, **F32), torch.ones(d, **F32), torch.zeros(d, **F32)]
        self.d_norms = [torch.empty(d, **F32) for _ in range(4)]
        self.h = [torch.empty(T, d, **F32) for _ in range(2)]
        self.mean, self.rstd = ([torch.empty(T, **F32) for _ in range(2)] for _ in range(2))
        self.y = [torch.empty(T, d, **BF16) for _ in range(2)]
        self.out, self.d_out, self.dx = (torch.empty(T, d, **BF16) for _ in range(3))
        self.dh, self.dstream = torch.empty(T, d, **F32), torch.empty(T, d, **F32)
        self.ws = torch.empty(moe.add_layer_norm_bwd_workspace(T, d), **U8)
        # the optimiser: two lists, the norms' without weight decay
        self.layer = moe.layer_adamw(self.buf, self.w_router, self.w_gate, self.w_up, self.w_down, bits, master=bits == 32)
        self.norm_list = moe.adamw_list(self.norms, self.d_norms, *moe.adamw_states(self.norms))
        self.lr, self.step = torch.full((1,), lr, **F32), torch.zeros(1, dtype=torch.int64, device="cuda")
        self.drawn = torch.zeros_like(self.step)   # masks of the steps so far, two each

    def _norm(self, i, x, stream, y, h, mean=None, rstd=None, p=0.0):
        moe.add_layer_norm(x, self.norms[2 * i], self.norms[2 * i + 1], y, stream, h, mean, rstd, self.eps, p, self.seed, i,
                           offset_dev=self.drawn)

    def forward(self, x, stream):
        """x [T, d] bf16, stream [T, d] fp32 -> y2."""
        self._norm(0, x, stream, self.y[0], self.h[0], self.mean[0], self.rstd[0], self.p)
        moe.forward(self.buf, self.y[0], self.w_router, None, self.w_gate, self.w_up, self.w_down, self.out)
        self._norm(1, self.out, self.h[0], self.y[1], self.h[1], self.mean[1], self.rstd[1], self.p)
        return self.y[1]

    def _norm_bwd(self, i, dy, dres, dh, dx):
        moe.add_layer_norm_bwd(dy, self.h[i], self.mean[i], self.rstd[i], self.norms[2 * i], dres, dh, dx,
                               self.d_norms[2 * i], self.d_norms[2 * i + 1], self.ws, self.p, self.seed, i, offset_dev=self.drawn)

    def backward(self, dy2, dh2=None):
        """dy2 [T, d] bf16, dh2: what comes back through the stream (or None)."""
        self._norm_bwd(1, dy2, dh2, self.dh, self.d_out)
        moe.backward(self.buf, self.d_out, self.y[0], self.w_router, self.w_gate, self.w_up, self.w_down)
        self._norm_bwd(0, self.buf.grads["dx"], self.dh, self.dstream, self.dx)
        self.drawn.add_(2)   # the next forward's masks are others
        return self.dx, self.dstream

    def update(self, offset=None):
        """One step on all weights.  The numbers of the drawn roundings go with the step's, far
        from those of the masks; with `offset` they are this offset's (at every replay)."""
        self.step.add_(1)
        draws = dict(offset=1 << 32, offset_dev=self.step) if offset is None else dict(offset=offset)
        moe.adamw(self.layer, self.lr, self.step, weight_decay=0.01, seed=self.seed, **draws)
        moe.adamw(self.norm_list, self.lr, self.step, weight_decay=0.0)

    def few(self, x, stream):
        """The block for up to 64 rows, without dropout, on the weights as they are -> y2."""
        t, d = x.shape
        y, h, out = torch.empty_like(x), torch.empty_like(stream), torch.empty_like(x)
        s = moe.shape(t, d, self.shape.n_experts, self.shape.top_k, self.shape.d_ff)
        self.few_ws = torch.zeros(moe.few_workspace(s), **U8)
        self._norm(0, x, stream, y, h)
        moe.forward_few(s, y, self.w_router, None, self.w_gate, self.w_up, self.w_down, out, self.few_ws)
        self._norm(1, out, h, y, h)
        return y


def main(T=8192, d=2048, E=32, k=4, f=1024):
    x, stream, dy = randn(T, d, scale=1.0), torch.randn(T, d, **F32), randn(T, d, scale=1.0)
    for bits in (32, 8):
        block = TrainBlock(T, d, E, k, f, bits=bits)

        def step():
            block.forward(x, stream)
            block.backward(dy)
            block.update()
        us, own = timed(step), timed(block.update)
        assert moe.read_error(block.buf.ws) == 0
        print(f"train  {T} tokens, d {d}, {E} experts of {f}, {k} a token, states in {bits} bits: {us:.0f} us a step, "
              f"{own:.0f} of it the update ({block.step.item()} steps taken)")
    for t in (1, 16, 64):
        us = timed(lambda: block.few(x[:t], stream[:t]))
        assert moe.read_error(block.few_ws) == 0
        print(f"few    {t} tokens: {us:.1f} us")


if __name__ == "__main__":
    moe.init(0)
    torch.manual_seed(0)
    main()
