"""AdamW's gradient scale, and its arithmetic where the kernel has two ways for it: roots and
quotients of pairs from the hardware's approximations (second moments within 2^-100 .. 2^100,
first ones within 2^-60 .. 2^60, eps and 1 - beta2 not too small), one by one elsewhere.
Both round each operation as IEEE 754 does, so everything is compared bit for bit with
numpy's float32.  GPU only."""
import numpy as np
import pytest
import torch

from test_gpu_adamw import HYPER, KINDS, SEED, Tensors

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{k[0]}-{k[1]}-{'copy' if k[2] else 'alone'}")
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("scale", [0.25, 0.37, 3.0, 0.0])
def test_gradient_scale(moe_gpu, kind, bits, scale):
    """The gradient is multiplied once, before the moments."""
    m, dev = moe_gpu
    t = Tensors(m, dev, [1, 129, 2050], kind, bits)
    factor = torch.tensor([scale], device=dev)
    for step in (1, 2):
        want = t.expected(step, step, HYPER, grad_scale=np.float32(scale))
        m.adamw(t.list, step=step, seed=SEED, offset=step, grad_scale=factor, **HYPER)
        t.check(want)


def spread(rng, n, low, high):
    """Magnitudes of all exponents from low to high, eight neighbours of one exponent in the
    first half and of any in the second."""
    e = rng.integers(low, high + 1, n)
    e[:n // 2] = np.repeat(e[:n // 2:8], 8)
    return (rng.uniform(1, 2, n) * np.exp2(e)).astype(np.float32)


EDGES = [(-64, -56), (56, 64), (-3, 3)]         # of the first moment
SQUARES = [(-104, -96), (96, 104), (-126, -110), (-6, 6)]


@pytest.mark.parametrize("first", EDGES, ids=str)
@pytest.mark.parametrize("second", SQUARES, ids=str)
@pytest.mark.parametrize("eps,beta2", [(1e-8, 0.99), (2.0 ** -60, 0.99), (2.0 ** -61, 0.99), (1.0, 0.99), (1.5, 0.99),
                                       (1e-8, 1 - 2.0 ** -16), (1e-8, 1 - 2.0 ** -17)], ids=str)
def test_both_ends_of_the_ranges(moe_gpu, first, second, eps, beta2):
    m, dev = moe_gpu
    n = 4096
    rng = np.random.default_rng(abs(first[0]) * 1000 + abs(second[0]))
    t = Tensors(m, dev, [n], ("f32", "f32", False), 32)
    t.m1[0].copy_(torch.from_numpy(spread(rng, n, *first) * rng.choice(np.float32([-1, 1]), n)))
    t.m2[0].copy_(torch.from_numpy(spread(rng, n, *second)))
    t.grad[0][::3] = 0
    if first[0] < -50:   # so that the moments keep their size
        t.grad[0].zero_()
    hyper = {**HYPER, "eps": eps, "beta2": beta2}
    with np.errstate(over="ignore", under="ignore"):
        want = t.expected(3, 0, hyper)
    m.adamw(t.list, step=3, seed=SEED, **hyper)
    t.check(want)


@pytest.mark.parametrize("first", [(-70, -52), (48, 56)], ids=str)
@pytest.mark.parametrize("second", [(-60, -42), (40, 52)], ids=str)
def test_8_bit_states_at_both_ends(moe_gpu, first, second):
    """Scales of blocks from one end of the ranges to beyond it."""
    m, dev = moe_gpu
    n = 128 * 64
    rng = np.random.default_rng(abs(first[0]) * 1000 + abs(second[0]))
    t = Tensors(m, dev, [n], ("f32", "f32", False), 8)
    t.m1[0][1].copy_(torch.from_numpy(spread(rng, 64, *first)))
    t.m2[0][1].copy_(torch.from_numpy(spread(rng, 64, *second)))
    t.grad[0].zero_()
    want = t.expected(3, 7, HYPER)
    m.adamw(t.list, step=3, seed=SEED, offset=7, **HYPER)
    t.check(want)


def quotient(m, dev, first, second):
    """first / sqrt(second) as a step computes it: moments that are halved (exactly), a step
    number at which the corrections are 1, a rate of 1, a weight of 0, and an eps that is
    lost beside roots from 1 on."""
    n = len(first)
    w, g = torch.zeros(n, device=dev), torch.zeros(n, device=dev)
    a, b = (torch.from_numpy(2 * v).to(dev) for v in (first, second))
    m.adamw(m.adamw_list([w], [g], [a], [b]), lr=1.0, step=100, beta1=0.5, beta2=0.5, eps=2.0 ** -60, weight_decay=0.0)
    assert torch.equal(a.cpu(), torch.from_numpy(first)) and torch.equal(b.cpu(), torch.from_numpy(second))
    return -w.cpu().numpy()


def test_roots_of_every_mantissa(moe_gpu):
    """All numbers of [1, 4): the root divided by the right one is 1, and would not be if it
    were a place off (r' = r + u: r / r' <= 1 - 2^-24; r - u: 1 + 2^-24 at least, u = 2^-23)."""
    m, dev = moe_gpu
    v = np.arange(0x3F800000, 0x40800000, dtype=np.uint32).view(np.float32)
    assert (quotient(m, dev, np.sqrt(v), v) == 1).all()


def test_reciprocals_of_every_mantissa_and_quotients(moe_gpu):
    """Divisors are all numbers of [1, 2), as roots of their rounded squares."""
    m, dev = moe_gpu
    d = np.arange(0x3F800000, 0x40000000, dtype=np.uint32).view(np.float32)
    v = d * d
    assert np.array_equal(np.sqrt(v), d)
    rng = np.random.default_rng(0)
    assert np.array_equal(quotient(m, dev, np.ones_like(d), v), np.float32(1) / d)
    for _ in range(8):
        bits = rng.integers(0, 1 << 23, len(d), dtype=np.uint32) | rng.integers(127 - 50, 127 + 50, len(d), dtype=np.uint32) << 23
        a = bits.view(np.float32)
        assert np.array_equal(quotient(m, dev, a, v), a / d)
