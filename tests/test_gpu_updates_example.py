"""examples/updates.py: layer norms, the layer, their backward, AdamW and the few-token
layer together, against the same block in float64 (autograd for the gradients, the
oracle's dropout masks, the device's own choice of experts).

Tolerances, relative to the largest value: the layer's 2e-2 and four bf16 roundings of
what goes in and out of it (4 * 2^-9 < 1e-2) for gradients; updates are compared bit for
bit with the oracle's on the gradients that the device left.  GPU only."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu
T, D, E, K, F = 300, 256, 8, 2, 128


@pytest.fixture(scope="module")
def example(moe_gpu):
    path = os.path.join(os.path.dirname(__file__), "..", "examples", "updates.py")
    spec = importlib.util.spec_from_file_location("updates_example", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def norm(h, w, b, eps=1e-5):
    return torch.nn.functional.layer_norm(h, (h.shape[1],), w, b, eps)


def layer(y, logits, idx, wg, wu, wd):
    """The routed SwiGLU experts, gates renormalised over the chosen ones."""
    gates = torch.softmax(logits.gather(1, idx), -1)
    out = torch.zeros_like(y)
    for e in range(wg.shape[0]):
        t, j = (idx == e).nonzero(as_tuple=True)
        a = torch.nn.functional.silu(y[t] @ wg[e].T) * (y[t] @ wu[e].T)
        out = out.index_add(0, t, gates[t, j, None] * (a @ wd[e].T))
    return out


def dropped(x, block, i):
    keep = torch.from_numpy(B.keep_mask(*x.shape, block.p, block.seed, i)).to(x.device)
    return torch.where(keep, x * (65536 / (65536 - round(block.p * 65536))), 0.0)


def rel(got, want):
    return ((got.double() - want).abs().max() / want.abs().max()).item()


def inputs(rows, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, stream, dy, dh = (torch.randn(rows, D, generator=gen, device="cuda") for _ in range(4))
    return x.bfloat16(), stream, dy.bfloat16(), dh


def new_block(example, bits):
    torch.manual_seed(1)
    b = example.TrainBlock(T, D, E, K, F, bits=bits)
    b.w_router.mul_(10)   # so that the choice of experts is not one of equals
    b.norms[0].add_(torch.randn_like(b.norms[0]) * 0.1)
    b.norms[1].add_(torch.randn_like(b.norms[1]) * 0.1)
    if bits == 32:
        b.layer = example.moe.layer_adamw(b.buf, b.w_router, b.w_gate, b.w_up, b.w_down, 32)
    return b


def test_gradients(example):
    b = new_block(example, 8)
    x, stream, dy, dh = inputs(T)
    y = b.forward(x, stream)
    dx, dstream = b.backward(dy, dh)
    assert example.moe.read_error(b.buf.ws) == 0
    leaves = [t.double().detach().clone().requires_grad_() for t in
              (x, stream, b.w_router, b.w_gate, b.w_up, b.w_down, *b.norms)]
    xd, sd, wr, wg, wu, wd, n1, b1, n2, b2 = leaves
    idx = b.buf.saved["topk_idx"].long()
    h1 = sd + dropped(xd, b, 0)
    y1 = norm(h1, n1, b1)
    h2 = h1 + dropped(layer(y1, y1 @ wr.T, idx, wg, wu, wd), b, 1)
    y2 = norm(h2, n2, b2)
    assert rel(y, y2) <= 3e-2
    ((y2 * dy.double()).sum() + (h2 * dh.double()).sum()).backward()
    g = b.buf.grads
    got = [dx, dstream, g["dw_router"], g["dw_gate"], g["dw_up"], g["dw_down"], *b.d_norms]
    for name, a, leaf in zip("dx dstream dw_router dw_gate dw_up dw_down dn1 db1 dn2 db2".split(), got, leaves):
        assert rel(a, leaf.grad) <= 3e-2, name


@pytest.mark.parametrize("bits", [32, 8])
def test_updates_and_few_tokens(example, bits):
    """Two steps captured and replayed; the second step's weights from the first's; then a
    few tokens on them."""
    m = example.moe
    b = new_block(example, bits)
    x, stream, dy, _ = inputs(T)
    names = ("w_router", "w_gate", "w_up", "w_down")
    b.forward(x, stream)
    b.backward(dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.forward(x, stream)
        b.backward(dy)
        b.update(offset=5)
    states = {n: [np.zeros(getattr(b, n).numel(), np.float32)] * 2 for n in names}
    masters = {n: getattr(b, n).float().flatten().cpu().numpy() for n in names}
    roots = states
    for step in (1, 2):
        graph.replay()
        torch.cuda.synchronize()
        assert b.step.item() == step and m.read_error(b.buf.ws) == 0
        for i, n in enumerate(names):
            grad = b.buf.grads["d" + n].flatten().cpu().numpy()
            w, a, v, root = B.adamw(masters[n], grad, *states[n], lr=np.float32(1e-3).item(), step=step, dtype=np.float32)
            size = len(w)
            if bits == 8:
                q, s = B.state8(a, B.numbers16(size, 4 * i, b.seed, 5), False)
                r, t = B.state8(root, B.numbers16(size, 4 * i + 1, b.seed, 5), True)
                a, rt = q * np.repeat(s, 128)[:size], r * np.repeat(t, 128)[:size]
                v = rt * rt
                w = ((w.view(np.uint32) + B.numbers16(size, 4 * i + 2, b.seed, 5).astype(np.uint32)) & 0xFFFF0000).view(np.float32)
            states[n], masters[n] = [a, v], w
            want = torch.from_numpy(w).to(torch.bfloat16)
            assert torch.equal(getattr(b, n).flatten().cpu(), want), (step, n)
    for i, (w, g) in enumerate(zip(b.norms, b.d_norms)):
        assert torch.isfinite(w).all() and (g != 0).any()
    # a few rows through the same block (no dropout), the routing that the device chose
    few = inputs(16, seed=9)
    y = b.few(few[0], few[1])
    assert m.read_error(b.few_ws) == 0
    n1, b1, n2, b2 = (t.double() for t in b.norms)
    h1 = few[1].double() + few[0].double()
    y1 = norm(h1, n1, b1)
    logits = y1 @ b.w_router.double().T
    top = logits.topk(K + 1, -1)
    sure = (top.values[:, K - 1] - top.values[:, K]) > 2e-2   # y1 is rounded to bf16 before the router
    out = layer(y1, logits, top.indices[:, :K], *(getattr(b, n).double() for n in names[1:]))
    want = norm(h1 + out, n2, b2)
    assert sure.sum() >= 12 and rel(y[sure], want[sure]) <= 3e-2


def test_example_runs(example, capsys):
    example.main(T=512, d=256, E=8, k=2, f=128)
    said = capsys.readouterr().out
    assert said.count("train") == 2 and said.count("few") == 3


def test_layer_lists(moe_gpu):
    m, dev = moe_gpu
    s = m.shape(64, 128, 4, 2, 128)
    buf = m.allocate(s)
    w = [torch.zeros(*v, dtype=torch.bfloat16, device=dev) for v in ((4, 128), (4, 128, 128), (4, 128, 128), (4, 128, 128))]
    assert m.layer_adamw(buf, *w).n == 4 and m.layer_adamw(buf, None, *w[1:], bits=8, master=False).n == 3
    with pytest.raises(ValueError):
        m.adamw_states(w, bits=16)
    with pytest.raises((ValueError, TypeError)):
        m.layer_adamw(buf, w[0], *[v.float() for v in w[1:]])
