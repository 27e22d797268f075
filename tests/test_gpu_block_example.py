"""examples/block.py: the operators around the layer and the layer together, against
the same block in float64 (autograd for the gradients, the oracle's dropout masks,
the device's own choice of experts).

Tolerances, relative to the largest value: the layer's 2e-2 in bf16 and 6e-2 in
MXFP8, and four bf16 roundings of what goes in and out of it, 4 * 2^-9 < 1e-2.
GPU only."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def block(moe_gpu):
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "block.py")
    spec = importlib.util.spec_from_file_location("block_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def norm(h, w, eps=1e-5):
    return h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * w


def experts(y, logits, idx, wg, wu, wd):
    """The routed SwiGLU experts, gates renormalised over the chosen ones."""
    gates = torch.softmax(logits.gather(1, idx), -1)
    out = torch.zeros_like(y)
    for e in range(wg.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        a = torch.nn.functional.silu(y[t] @ wg[e].T) * (y[t] @ wu[e].T)
        out = out.index_add(0, t, gates[t, j, None] * (a @ wd[e].T))
    return out


def near(got, want, tol, what):
    got, want = got.detach().double().cpu(), want.detach()
    worst = ((got - want).abs().max() / want.abs().max()).item()
    assert worst <= tol, f"{what}: {worst:.3e} of the largest value"


def test_train_block(moe_gpu, block):
    m, dev = moe_gpu
    torch.manual_seed(3)
    T, d, E, k, f, p, step = 150, 256, 8, 2, 256, 0.2, 5
    b = block.TrainBlock(T, d, E, k, f, p)
    for w in (b.w_router, b.w_gate, b.w_up, b.w_down):
        w.mul_(4)   # the experts' part of the stream next to what passes them by
    b.w1.copy_(torch.rand(d) + 0.5)
    b.w2.copy_(torch.rand(d) + 0.5)
    x, stream = block.randn(T, d, scale=1.0), torch.randn(T, d, device=dev)
    dy, dh = block.randn(T, d, scale=1.0), torch.randn(T, d, device=dev)
    m.clear_error(b.buf.ws)
    y = b.forward(x, stream, step)
    dx, ds = b.backward(dy, dh)
    assert m.read_error(b.buf.ws) == 0
    c = lambda t, grad=True: t.detach().double().cpu().requires_grad_(grad)
    cx, cs, wr, wg, wu, wd, w1, w2 = (c(t) for t in (x, stream, b.w_router, b.w_gate, b.w_up, b.w_down, b.w1, b.w2))
    one = np.ones((T, d))
    mask = [torch.from_numpy(B.dropout(one, p, 1234, 2 * step + i)) for i in range(2)]
    idx = b.buf.saved["topk_idx"].long().cpu()
    h1 = cs + mask[0] * cx
    y1 = norm(h1, w1)
    out = experts(y1, y1 @ wr.T, idx, wg, wu, wd)
    h2 = h1 + mask[1] * out
    y2 = norm(h2, w2)
    ((y2 * c(dy, False)).sum() + (h2 * c(dh, False)).sum()).backward()
    near(b.out, out, 3e-2, "out")
    near(y, y2, 3e-2, "y2")
    for what, got, want in (("dx", dx, cx), ("dstream", ds, cs), ("dw1", b.dw1, w1), ("dw2", b.dw2, w2),
                            ("dw_router", b.buf.grads["dw_router"], wr), ("dw_gate", b.buf.grads["dw_gate"], wg),
                            ("dw_up", b.buf.grads["dw_up"], wu), ("dw_down", b.buf.grads["dw_down"], wd)):
        near(got, want.grad, 3e-2, what)


def test_dense_block(moe_gpu, block):
    m, dev = moe_gpu
    torch.manual_seed(4)
    T, d, f = 300, 256, 512
    b = block.DenseBlock(T, d, f)
    x, stream = block.randn(T, d, scale=1.0), torch.randn(T, d, device=dev)
    m.clear_error(b.buf.ws)
    out = b.forward(x, stream)
    assert m.read_error(b.buf.ws) == 0
    c = lambda t: t.double().cpu()
    y = norm(c(stream) + c(x), c(b.w))
    a = torch.nn.functional.silu(y @ c(b.w_gate[0]).T) * (y @ c(b.w_up[0]).T)
    near(out, a @ c(b.w_down[0]).T, 7e-2, "out")


@pytest.mark.parametrize("T", [1, 7, 40])
def test_serve_block(moe_gpu, block, T):
    m, dev = moe_gpu
    torch.manual_seed(5)
    d, E, k, f, vocab = 256, 8, 2, 256, 1000
    b = block.ServeBlock(T, d, E, k, f, vocab, group=64)
    x, stream = block.randn(T, d, scale=1.0), torch.randn(T, d, device=dev)
    logits = b.forward(x, stream).clone()
    assert m.read_error(b.ws) == 0 and m.read_error(b.route_ws) == 0
    c = lambda t: t.double().cpu()

    def full(q, s):
        v = torch.empty(*q.shape[:-1], q.shape[-1] * 2, device=dev)
        m.dequantize_w4(q, s, v)
        return c(v)
    h1 = c(stream) + c(x)
    y1 = norm(h1, c(b.w1))
    w = {n: full(b.w[n + "_q"], b.w[n + "_s"]) for n in ("gate", "up", "down")}
    out = experts(y1, y1 @ c(b.w_router).T, b.route["topk_idx"].long().cpu(), w["gate"], w["up"], w["down"])
    near(b.out, out, 3e-2, "out")
    near(logits, norm(h1 + out, c(b.w2)) @ full(*b.proj).T, 3e-2, "logits")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(x, stream)
    x.neg_()
    b.forward(x, stream)
    want = b.logits.clone()
    b.logits.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.logits, want) and not torch.equal(want, logits)
