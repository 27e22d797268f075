"""Calls that draw numbers, captured into a graph: each replay has numbers of its own when
the offset comes from the device.

Replays are compared bit for bit with eager calls that are given the sum of the two offsets,
which other tests compare with the oracle.  How far many roundings stray is compared with
the binomial distribution.  GPU only."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from test_gpu_adamw import HYPER, SEED, Tensors
from test_gpu_updates_example import example, inputs, new_block   # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def captured(fn):
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        fn()
    return graph


# ------------------------------------------------------------------ AdamW
@pytest.mark.parametrize("kind,bits", [(("bf16", "f32", False), 32), (("bf16", "bf16", False), 8), (("bf16", "f32", True), 8),
                                       (("f32", "f32", False), 8), (("f16", "f16", True), 8)], ids=str)
@pytest.mark.parametrize("offset", [0, (1 << 32) - 2, (1 << 64) - 2], ids=hex)
def test_replays_equal_steps_with_offsets_of_their_own(moe_gpu, kind, bits, offset):
    """The sum carries into the upper word and past 64 bits."""
    m, dev = moe_gpu
    t, u = (Tensors(m, dev, [5000, 17, 0, 129], kind, bits) for _ in range(2))
    step = torch.zeros(1, dtype=torch.int64, device=dev)

    def one():
        step.add_(1)
        m.adamw(t.list, step=step, seed=SEED, offset=offset, offset_dev=step, **HYPER)
    graph = captured(one)
    for k in (1, 2, 3):
        graph.replay()
        m.adamw(u.list, step=k, seed=SEED, offset=(offset + k) % (1 << 64), **HYPER)
        torch.cuda.synchronize()
        for a, b in zip(t.list.held, u.list.held):
            assert torch.equal(a, b)


def test_the_counter_is_no_part_of_steps_without_drawn_numbers(moe_gpu):
    m, dev = moe_gpu
    for kind in (("f32", "f32", False), ("bf16", "f32", True)):
        t, u = (Tensors(m, dev, [300], kind, 32) for _ in range(2))
        m.adamw(t.list, step=1, offset_dev=torch.tensor([5], device=dev), **HYPER)
        m.adamw(u.list, step=1, **HYPER)
        for a, b in zip(t.list.held, u.list.held):
            assert torch.equal(a, b)


def test_captured_steps_of_bf16_parameters_follow_their_mean(moe_gpu):
    """A hundred replayed steps of -1e-4 from 1, where bf16 steps by 2^-8: each goes down
    with the probability 1e-4 * 2^8 (16 bits of it: 2^-16 off at most), so that a place has
    taken a binomial number of steps.  The mean of n places strays by five standard errors
    at most, the spread by five of its own (sigma / sqrt(2 n) for a normal distribution; the
    binomial one's fourth moment is below 3.4 sigma^4: 1.1 times that)."""
    m, dev = moe_gpu
    n, steps, lr = 1 << 18, 100, 1e-4
    p = torch.ones(n, dtype=torch.bfloat16, device=dev)
    g = torch.full((n,), 0.25, device=dev)
    lst = m.adamw_list([p], [g], *m.adamw_states([p]))
    step = torch.zeros(1, dtype=torch.int64, device=dev)

    def one():
        step.add_(1)
        m.adamw(lst, lr, step, eps=0.0, weight_decay=0.0, seed=SEED, offset_dev=step)
    graph = captured(one)
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    down = lr * 256
    sigma = 2.0 ** -8 * np.sqrt(steps * down * (1 - down))
    got = p.double()
    assert step.item() == steps
    assert abs(got.mean().item() - (1 - steps * lr)) <= 5 * sigma / np.sqrt(n) + 2 * steps * 2.0 ** -24
    assert abs(got.std().item() / sigma - 1) <= 1.1 * 5 / np.sqrt(2 * n) + steps * 2.0 ** -16
    assert got.max().item() <= 1 and (got == 1).double().mean().item() < 0.1   # (1 - down)^100 = 0.075 never moved


def test_captured_steps_of_8_bit_states_follow_their_mean(moe_gpu):
    """A gradient of 0.4 beside one of 1 each 128, a hundred steps from zeros: the first
    moment is 0.4 (1 - b^100).  A step adds 1 - b of the distance, and a rounding that is
    right in the mean (16 bits of the probability: off by 2^-16 of a code's step at most) and
    strays by at most half of that step, 32 / 448 below the code of 512; each rounding counts
    b of the one before it in the next step.  With the same numbers at every replay a place
    would stand still where its distance no longer reaches its border."""
    m, dev = moe_gpu
    n, steps, beta = 1 << 16, 100, 0.9
    p = torch.zeros(n, device=dev)
    g = torch.full((n,), 0.4, device=dev)
    g[::128] = 1.0
    states = m.adamw_states([p], 8)
    lst = m.adamw_list([p], [g], *states)
    step = torch.zeros(1, dtype=torch.int64, device=dev)

    def one():
        step.add_(1)
        m.adamw(lst, 1e-3, step, beta1=beta, beta2=beta, seed=SEED, offset=3 << 40, offset_dev=step)
    graph = captured(one)
    for _ in range(steps):
        graph.replay()
    torch.cuda.synchronize()
    few = torch.arange(n, device=dev) % 128 != 0
    code, scale = states[0][0]
    v = (code.view(torch.float8_e4m3fn).double() * scale.double().repeat_interleave(128))[few]
    want, unit = 0.4 * (1 - beta ** steps), 32 / 448
    sigma = unit / 2 / np.sqrt(1 - beta ** 2)
    off = 5 * sigma / np.sqrt(len(v)) + 2.0 ** -16 * unit / (1 - beta) + 2.0 ** -20
    assert abs(v.mean().item() - want) <= off and v.std().item() <= sigma


# ------------------------------------------------------------------ norms and dropout
def normal(gen, shape, dtype, dev):
    return torch.randn(shape, generator=gen, device=dev).to(dtype)


def norm_calls(m, dev, rows, d, xt, rt, layer):
    """(call(offset, offset_dev), its outputs): forward, 8-bit forward where there is one, and
    backward of one norm, and the dropout, each on outputs of its own."""
    gen = torch.Generator(device=dev).manual_seed(rows + d)
    x, dy = normal(gen, (rows, d), xt, dev), normal(gen, (rows, d), xt, dev)
    res, w = normal(gen, (rows, d), rt, dev), normal(gen, (d,), xt, dev)
    f = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device=dev)   # noqa: E731
    out = dict(h=f(rows, d, dtype=rt), y=f(rows, d, dtype=xt), rstd=f(rows), dh=f(rows, d, dtype=rt), dx=f(rows, d, dtype=xt),
               dw=f(d), dropped=f(rows, d, dtype=xt), h8=f(rows, d, dtype=rt))
    mean, rstd = normal(gen, (rows,), torch.float32, dev), torch.rand(rows, generator=gen, device=dev)
    size = m.add_layer_norm_bwd_workspace(rows, d)
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    pad = (rows + 127) // 128 * 128
    if xt is torch.bfloat16 and d % 128 == 0:
        out.update(q=f(pad, d, dtype=torch.uint8), s=f(pad * d // 32, dtype=torch.uint8))

    def call(offset, at=None):
        kw = dict(p=0.3, seed=SEED, offset=offset, offset_dev=at)
        if layer:
            fwd = lambda y, h, **k: m.add_layer_norm(x, w, w, y, res, h, None, out["rstd"], **k)   # noqa: E731
            m.add_layer_norm_bwd(dy, res, mean, rstd, w, None, out["dh"], out["dx"], out["dw"], None, ws, **kw)
        else:
            fwd = lambda y, h, **k: m.add_norm(x, w, y, res, h, out["rstd"], **k)   # noqa: E731
            m.add_norm_bwd(dy, res, rstd, w, None, out["dh"], out["dx"], out["dw"], ws, **kw)
        fwd(out["y"], out["h"], **kw)
        if "q" in out:
            fwd(None, out["h8"], y_q=out["q"], y_scales=out["s"], **kw)
        m.dropout(x, out["dropped"], 0.3, SEED, offset, offset_dev=at)
    return call, out


@pytest.mark.parametrize("d", [64, 77, 250, 2048, 9000])
@pytest.mark.parametrize("types", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")], ids="-".join)
@pytest.mark.parametrize("layer", [False, True], ids=["rms", "layer"])
def test_replayed_masks_are_those_of_the_summed_offsets(moe_gpu, d, types, layer):
    m, dev = moe_gpu
    xt, rt = ({"bf16": torch.bfloat16, "f32": torch.float32}[t] for t in types)
    rows, first = 37, (1 << 64) - 2
    call, out = norm_calls(m, dev, rows, d, xt, rt, layer)
    at = torch.zeros(1, dtype=torch.int64, device=dev)
    call(first)   # shared memory limits are raised before the capture

    def one():
        at.add_(1)
        call(first, at)
    graph, seen = captured(one), []
    for k in (1, 2, 3):
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in out.items()}
        call((first + k) % (1 << 64))
        for n, t in out.items():
            assert torch.equal(got[n], t), n
        seen.append(got["dropped"])
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])


def test_a_counter_without_dropout(moe_gpu):
    """p = 0: the counter is not needed and changes nothing."""
    m, dev = moe_gpu
    x, w = torch.randn(9, 256, device=dev), torch.ones(256, device=dev)
    a, b = torch.empty_like(x), torch.empty_like(x)
    at = torch.tensor([3], device=dev)
    m.add_layer_norm(x, w, None, a, offset_dev=at)
    m.add_layer_norm(x, w, None, b)
    assert torch.equal(a, b)
    m.dropout(x, a, 0.0, 1, offset_dev=at)
    assert torch.equal(a, x)


def test_counters_of_a_wrong_kind_are_refused(moe_gpu):
    m, dev = moe_gpu
    x, w = torch.randn(4, 64, device=dev), torch.ones(64, device=dev)
    y = torch.zeros_like(x)
    for bad in (torch.zeros(1, device=dev), torch.zeros(2, dtype=torch.int64, device=dev), torch.zeros(1, dtype=torch.int64)):
        with pytest.raises((TypeError, ValueError)):
            m.dropout(x, y, 0.5, 1, offset_dev=bad)
        with pytest.raises((TypeError, ValueError)):
            m.add_norm(x, w, y, h=y, p=0.5, offset_dev=bad)
    assert (y == 0).all()


# ------------------------------------------------------------------ the example
@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_training_step(example, bits):   # noqa: F811
    """Replays of the example's step: each with the oracle's masks of its own offsets, and the
    weights that eager steps leave."""
    x, stream, dy, _ = inputs(300)
    blocks = []
    for _ in range(2):
        b = new_block(example, bits)
        b.forward(x, stream)
        b.backward(dy)
        blocks.append(b)

    def step(b):
        b.forward(x, stream)
        b.backward(dy)
        b.update()
    graph = captured(lambda: step(blocks[0]))
    kept = []
    for k in (1, 2, 3):
        graph.replay()
        step(blocks[1])
        torch.cuda.synchronize()
        for n in ("w_router", "w_gate", "w_up", "w_down"):
            assert torch.equal(getattr(blocks[0], n), getattr(blocks[1], n)), (k, n)
        for i in range(2):
            assert torch.equal(blocks[0].h[i], blocks[1].h[i])
        got = (blocks[0].h[0] != stream).cpu().numpy()   # places that were kept
        want = B.keep_mask(*x.shape, blocks[0].p, blocks[0].seed, 2 * k)
        # a kept x of zero, or one that is lost beside the stream's value, looks dropped
        assert not (got & ~want).any() and (want & ~got).mean() < 0.02
        kept.append(got)
    assert (kept[0] != kept[1]).any() and (kept[1] != kept[2]).any()


def test_steps_of_the_example_draw_other_roundings(example):   # noqa: F811
    """The same gradients and weights, stepped as step 1 and as step 2 of 8-bit states whose
    constants are the same: the codes differ."""
    blocks = [new_block(example, 8) for _ in range(2)]
    for s, b in enumerate(blocks):
        gen = torch.Generator(device="cuda").manual_seed(7)
        for g in ("dw_router", "dw_gate", "dw_up", "dw_down"):
            b.buf.grads[g].normal_(generator=gen)
        b.step.fill_(1 + s)
        b.update()
    codes = [b.layer.held[0] for b in blocks]   # of the first tensor's first moment
    assert codes[0].dtype == torch.uint8 and not torch.equal(codes[0], codes[1])
