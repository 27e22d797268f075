"""A transformer block's expert half with the operators around the layer.

    python examples/block.py            # train and serve, with their times
    python examples/block.py train
    python examples/block.py serve

Three ways in which a program uses them:

TrainBlock   the residual stream takes the attention's output (dropout, add, RMS
             norm), the MoE layer runs on the normed rows, the next norm takes the
             layer's output; forward and backward, bf16 activations, fp32 stream.
DenseBlock   a dense SwiGLU on MXFP8 codes that the norm writes itself: no pass
             quantises the activations.
ServeBlock   a few tokens: the same norms, the router, the experts on 4-bit
             weights and a 4-bit projection; captured into one CUDA graph.

Weights and inputs are random.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import moe_expert_layer_softmax_gb300 as moe

BF16 = dict(dtype=torch.bfloat16, device="cuda")
F32 = dict(dtype=torch.float32, device="cuda")
U8 = dict(dtype=torch.uint8, device="cuda")


def randn(*shape, scale=0.02):
    return (scale * torch.randn(*shape, **F32)).to(torch.bfloat16)


class TrainBlock:
    """h1 = stream + dropout(x), y1 = norm(h1), out = experts(y1),
    h2 = h1 + dropout(out), y2 = norm(h2)."""

    def __init__(self, T, d, E, k, f, p=0.1, eps=1e-5):
        self.shape, self.p, self.eps = moe.shape(T, d, E, k, f), p, eps
        self.buf = moe.allocate(self.shape)
        self.w_router, self.w_down = randn(E, d), randn(E, d, f)
        self.w_gate, self.w_up = randn(E, f, d), randn(E, f, d)
        self.w1, self.w2 = torch.ones(d, **F32), torch.ones(d, **F32)
        self.h1, self.h2 = torch.empty(T, d, **F32), torch.empty(T, d, **F32)
        self.r1, self.r2 = torch.empty(T, **F32), torch.empty(T, **F32)
        self.y1, self.y2, self.out = (torch.empty(T, d, **BF16) for _ in range(3))
        # gradients of the streams and branches; those of the layer are in buf.grads
        self.dh, self.dstream = torch.empty(T, d, **F32), torch.empty(T, d, **F32)
        self.d_out, self.dx = torch.empty(T, d, **BF16), torch.empty(T, d, **BF16)
        self.dw1, self.dw2 = torch.empty(d, **F32), torch.empty(d, **F32)
        self.ws = torch.empty(moe.add_norm_bwd_workspace(T, d), **U8)

    def forward(self, x, stream, step):
        """x [T, d] bf16, stream [T, d] fp32 -> y2 (and h2, the next block's stream)."""
        self.seed, self.step = 1234, step
        moe.add_norm(x, self.w1, self.y1, stream, self.h1, self.r1, self.eps, self.p, self.seed, 2 * step)
        moe.forward(self.buf, self.y1, self.w_router, None, self.w_gate, self.w_up, self.w_down, self.out)
        moe.add_norm(self.out, self.w2, self.y2, self.h1, self.h2, self.r2, self.eps, self.p, self.seed,
                     2 * step + 1)
        return self.y2

    def backward(self, dy2, dh2=None):
        """dy2 [T, d] bf16, dh2: what comes back through the stream (or None) ->
        (dx, dstream); the masks are those of the forward."""
        moe.add_norm_bwd(dy2, self.h2, self.r2, self.w2, dh2, self.dh, self.d_out, self.dw2, self.ws,
                         self.p, self.seed, 2 * self.step + 1)
        moe.backward(self.buf, self.d_out, self.y1, self.w_router, self.w_gate, self.w_up, self.w_down)
        moe.add_norm_bwd(self.buf.grads["dx"], self.h1, self.r1, self.w1, self.dh, self.dstream, self.dx,
                         self.dw1, self.ws, self.p, self.seed, 2 * self.step)
        return self.dx, self.dstream


class DenseBlock:
    """h = stream + x, y = norm(h) as MXFP8, out = W_down (silu(W_gate y) * W_up y)."""

    def __init__(self, T, d, f, eps=1e-5):
        self.T, self.eps = T, eps
        self.rows = (T + 127) // 128 * 128
        self.shape = moe.shape(T, d, 1, 1, f, prec=moe.MXFP8)
        self.buf = moe.allocate(self.shape, with_grads=False)
        self.w_gate, self.w_up, self.w_down = randn(1, f, d), randn(1, f, d), randn(1, d, f)
        moe.build_mx_weights(self.shape, self.w_gate, self.w_up, self.w_down, self.buf.mx_weights)
        self.w = torch.ones(d, **F32)
        self.h, self.out = torch.empty(T, d, **F32), torch.empty(self.rows, d, **BF16)
        self.tiles = torch.tensor([0, self.rows // 128], dtype=torch.int32, device="cuda")

    def forward(self, x, stream):
        s, b, mx, w = self.shape, self.buf, self.buf.mx, self.buf.mx_weights
        moe.add_norm(x, self.w, None, stream, self.h, None, self.eps, y_q=mx["xd_q"], y_scales=mx["xd_s"])
        moe.grouped_gemm(s, moe.GEMM_FWD1_SWIGLU, b.ws, tile_offsets=self.tiles, a0=mx["xd_q"], sfa0=mx["xd_s"],
                         w0=w["gu_q"], sfb0=w["gu_s"], out0=b.saved["h"], out1=b.saved["u"], out2=mx["a_q"],
                         osf0=mx["a_s"])
        moe.grouped_gemm(s, moe.GEMM_FWD2, b.ws, tile_offsets=self.tiles, a0=mx["a_q"], sfa0=mx["a_s"],
                         w0=w["down_q"], sfb0=w["down_s"], out0=self.out)
        return self.out[:self.T]


def quantized(w, group):
    """(codes, scales) of bf16 weights [..., K]."""
    q = torch.empty(*w.shape[:-1], w.shape[-1] // 2, **U8)
    s = torch.empty(*w.shape[:-1], w.shape[-1] // group, **BF16)
    moe.quantize_w4(w, q, s)
    return q, s


class ServeBlock:
    """The block for T tokens and a projection of the last norm to `vocab` rows:
    logits = W_proj y2."""

    def __init__(self, T, d, E, k, f, vocab, group=128, eps=1e-5):
        self.shape, self.eps = moe.shape(T, d, E, k, f), eps
        self.w_router = randn(E, d)
        self.w = {}
        for name, shape in (("gate", (E, f, d)), ("up", (E, f, d)), ("down", (E, d, f))):
            self.w[name + "_q"], self.w[name + "_s"] = quantized(randn(*shape), group)
        self.proj = quantized(randn(vocab, d), group)
        self.w1, self.w2 = torch.ones(d, **F32), torch.ones(d, **F32)
        self.h1, self.h2 = torch.empty(T, d, **F32), torch.empty(T, d, **F32)
        self.y1, self.y2, self.out = (torch.empty(T, d, **BF16) for _ in range(3))
        self.logits = torch.empty(T, vocab, **BF16)
        b = moe.allocate(self.shape, with_grads=False)
        self.route_ws = b.ws
        self.route = {n: b.saved[n] for n in ("logits", "topk_idx", "gates", "counts", "offsets", "tile_offsets",
                                              "slot_of_route", "route_of_slot")}
        self.ws = torch.zeros(moe.experts_w4_workspace(T, d, E, k, f), **U8)

    def forward(self, x, stream):
        """x [T, d] bf16 (the attention's output), stream [T, d] fp32 -> logits."""
        moe.add_norm(x, self.w1, self.y1, stream, self.h1, eps=self.eps)
        moe.route(self.shape, self.y1, self.w_router, None, **self.route, ws=self.route_ws)
        moe.experts_w4(self.y1, self.route["topk_idx"], self.route["gates"], self.w, self.out, self.ws)
        moe.add_norm(self.out, self.w2, self.y2, self.h1, self.h2, eps=self.eps)
        moe.matvec_w4(self.y2, *self.proj, self.logits)
        return self.logits


def timed(fn, n=20):
    """Microseconds of a call, captured into a graph and replayed n times."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            fn()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        fn()
    for _ in range(3):
        graph.replay()
    a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    a.record()
    for _ in range(n):
        graph.replay()
    b.record()
    b.synchronize()
    return a.elapsed_time(b) * 1e3 / n


def train(T=8192, d=2048, E=32, k=4, f=1024):
    block = TrainBlock(T, d, E, k, f)
    x, stream, dy = randn(T, d, scale=1.0), torch.randn(T, d, **F32), randn(T, d, scale=1.0)

    def step():
        block.forward(x, stream, 0)
        block.backward(dy)
    us = timed(step)
    assert moe.read_error(block.buf.ws) == 0
    print(f"train  {T} tokens, d {d}, {E} experts of {f}, {k} a token: {us:.0f} us a step "
          f"({T / us:.2f} M tokens/s), |dx| {block.dx.float().norm().item():.4f}")
    dense = DenseBlock(T, d, 4 * d)
    us = timed(lambda: dense.forward(x, stream))
    print(f"dense  {T} tokens, d {d}, f {4 * d}, MXFP8 forward: {us:.0f} us")


def serve(d=2048, E=64, k=4, f=1408, vocab=32000):
    for T in (1, 8, 64):
        block = ServeBlock(T, d, E, k, f, vocab, group=64)
        x, stream = randn(T, d, scale=1.0), torch.randn(T, d, **F32)
        us = timed(lambda: block.forward(x, stream))
        assert moe.read_error(block.ws) == 0 and moe.read_error(block.route_ws) == 0
        print(f"serve  {T} tokens, d {d}, {E} experts of {f}, {k} a token, {vocab} logits: {us:.1f} us a step")


if __name__ == "__main__":
    moe.init(0)
    torch.manual_seed(0)
    what = sys.argv[1:] or ["train", "serve"]
    if "train" in what:
        train()
    if "serve" in what:
        serve()
