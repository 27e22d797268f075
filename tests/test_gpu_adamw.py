"""AdamW over lists of tensors on the GPU.

The definition rounds every operation to 32 bits in a given order, so the results are
compared bit for bit with the oracle's float32 arithmetic (numpy rounds each operation
by itself), and that arithmetic with 64 bits: about ten roundings of 2^-24, the
difference of moment and decayed weight relative to its terms.  GPU only."""
import numpy as np
import pytest
import torch

from gpu_util import f64
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
KINDS = [("f32", "f32", False), ("bf16", "f32", True), ("bf16", "bf16", True), ("bf16", "f32", False),
         ("bf16", "bf16", False), ("f16", "f32", True), ("f16", "f16", True)]
SEED = 0xFEDCBA9876543210
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


class Tensors:
    """A list of tensors with gradients and states; `shift` elements off a boundary."""

    def __init__(self, m, dev, sizes, kind, bits, seed=0, shift=0, zeros=False):
        rng = np.random.default_rng(seed)
        pt, gt, master = kind
        self.m, self.bits, self.kind = m, bits, kind

        def put(v, dtype):
            t = torch.from_numpy(np.ascontiguousarray(v))
            big = torch.zeros(len(v) + shift + 8, dtype=dtype, device=dev)
            big[shift:shift + len(v)] = t.to(dtype)
            return big[shift:shift + len(v)]

        self.param, self.grad, self.master, self.m1, self.m2 = [], [], [] if master else None, [], []
        for n in sizes:
            w = rng.standard_normal(n) * 0.05
            size = 1e-3 * np.exp(rng.standard_normal(n))
            w32 = put(w, torch.float32)
            self.param.append(put(f64(w32), DT[pt]))
            if master:
                self.master.append(w32)
            self.grad.append(put(rng.standard_normal(n) * size, DT[gt]))
            a, b = rng.standard_normal(n) * size * 0.3, size * 0.7
            if zeros:
                a, b = 0 * a, 0 * b
            if bits == 32:
                self.m1.append(put(a, torch.float32))
                self.m2.append(put(b * b, torch.float32))
            else:
                for states, x, least in ((self.m1, a, False), (self.m2, b, True)):
                    q, s = B.state8(x, np.full(n, 32768), least)
                    codes = torch.from_numpy(q).to(torch.float8_e4m3fn).view(torch.uint8)
                    states.append((put(codes.numpy(), torch.uint8), put(s, torch.float32)))
        self.list = m.adamw_list(self.param, self.grad, self.m1, self.m2, master=self.master)

    def state(self, s):
        """An fp32 array of what a state holds."""
        if self.bits == 32:
            return s.cpu().numpy()
        codes, scales = s[0].cpu().numpy(), s[1].cpu().numpy()
        return B.e4m3_values(codes).astype(np.float32) * np.repeat(scales, 128)[:len(codes)]

    def expected(self, step, offset, hyper, grad_scale=1.0, dtype=np.float32):
        """What a step leaves, tensor by tensor (before it is taken)."""
        out = []
        for i in range(len(self.param)):
            w = (self.master if self.kind[2] else self.param)[i].float().cpu().numpy()
            g, a, b = self.grad[i].float().cpu().numpy(), self.state(self.m1[i]), self.state(self.m2[i])
            b = b if self.bits == 32 else b * b
            w, a, b, root = B.adamw(w, g, a, b, step=step, grad_scale=grad_scale, dtype=dtype, **hyper)
            n = len(w)
            d = dict(w=w, m=a, v=b)
            if self.bits == 8:
                d["m"], d["m_scale"] = B.state8(a, B.numbers16(n, 4 * i, SEED, offset), False)
                d["v"], d["v_scale"] = B.state8(root, B.numbers16(n, 4 * i + 1, SEED, offset), True)
            if self.kind[0] == "bf16" and not self.kind[2] and dtype is np.float32:
                bits = (w.view(np.uint32) + B.numbers16(n, 4 * i + 2, SEED, offset).astype(np.uint32)) & 0xFFFF0000
                d["w"] = bits.view(np.float32)
            out.append(d)
        return out

    def check(self, want):
        for i, d in enumerate(want):
            p = self.param[i].float().cpu().numpy()
            if self.kind[2]:
                assert np.array_equal(self.master[i].cpu().numpy(), d["w"]), i
                assert np.array_equal(p, torch.from_numpy(d["w"]).to(DT[self.kind[0]]).float().numpy()), i
            else:
                assert np.array_equal(p, d["w"]), i
            if self.bits == 32:
                assert np.array_equal(self.m1[i].cpu().numpy(), d["m"]) and np.array_equal(self.m2[i].cpu().numpy(), d["v"])
            else:
                for s, n in ((self.m1[i], "m"), (self.m2[i], "v")):
                    assert np.array_equal(B.e4m3_values(s[0].cpu().numpy()), d[n].astype(np.float64)), (i, n)
                    assert np.array_equal(s[1].cpu().numpy(), d[n + "_scale"]), (i, n)


SIZES = [1, 7, 8, 127, 128, 129, 0, 2047, 2048, 2049, 5000, 3]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: f"{k[0]}-{k[1]}-{'copy' if k[2] else 'alone'}")
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("shift", [0, 1])
def test_steps(moe_gpu, kind, bits, shift):
    """Three steps, each from what the one before it left."""
    m, dev = moe_gpu
    t = Tensors(m, dev, SIZES, kind, bits, shift=shift)
    for step in (1, 2, 3):
        want = t.expected(step, step << 33, HYPER)
        m.adamw(t.list, step=step, seed=SEED, offset=step << 33, **HYPER)
        t.check(want)


@pytest.mark.parametrize("bits", [32, 8])
def test_against_64_bits(moe_gpu, bits):
    m, dev = moe_gpu
    t = Tensors(m, dev, [4096, 301], ("f32", "f32", False), bits)
    before = [(t.param[i].cpu().numpy().astype(np.float64), t.state(t.m1[i]).astype(np.float64), t.state(t.m2[i]).astype(np.float64))
              for i in range(2)]
    want = t.expected(5, 0, HYPER, dtype=np.float64)
    m.adamw(t.list, step=5, seed=SEED, **HYPER)
    for i in range(2):
        w0, m0, _ = before[i]
        terms = np.abs(w0) + np.abs(want[i]["w"] - w0)
        # moments and root: 4 roundings of their terms; the quotient and its factors: 6 more.
        # The first moment's terms may cancel: its error is relative to them
        g = f64(t.grad[i])
        moved = HYPER["lr"] / (1 - 0.9 ** 5)
        b = before[i][2] if bits == 32 else before[i][2] ** 2
        root = np.sqrt(0.99 * b + 0.01 * g * g) / np.sqrt(1 - 0.99 ** 5) + 1e-8
        terms = terms + moved * (0.9 * np.abs(m0) + 0.1 * np.abs(g)) / root
        assert (np.abs(f64(t.param[i]) - want[i]["w"]) <= 10 * 2.0 ** -24 * terms).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_a_launch_takes(moe_gpu, bits):
    """Tables of both lengths, several launches, empty tensors in front and behind."""
    m, dev = moe_gpu
    rng = np.random.default_rng(4)
    for count in (16, 17, 224, 225, 500):
        sizes = [0] + [int(v) for v in rng.integers(0, 300, count - 2)] + [0]
        t = Tensors(m, dev, sizes, ("bf16", "f32", False), bits, seed=count)
        want = t.expected(2, 9, HYPER)
        m.adamw(t.list, step=2, seed=SEED, offset=9, **HYPER)
        t.check(want)


def test_rounding_up_follows_the_remainder(moe_gpu):
    """Over many numbers the states' and the parameters' mean is that of the values before
    they were rounded: 2^20 equal values beside a large one each 128; the mean of n
    roundings is off by at most 5 standard deviations, half a step / sqrt(n) each."""
    m, dev = moe_gpu
    n = 1 << 20
    p = torch.full((n,), 1.0 + 2.0 ** -10, device=dev).to(torch.bfloat16)   # 1: its steps are 2^-7
    g = torch.full((n,), 3.1e-3, device=dev)
    g[::128] = 1.0
    codes = [torch.zeros(n, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.zeros(n // 128, device=dev) for _ in range(2)]
    lst = m.adamw_list([p], [g], [(codes[0], scales[0])], [(codes[1], scales[1])])
    m.adamw(lst, lr=1e-3, step=1, beta1=0.9, beta2=0.999, weight_decay=0.0, seed=3)
    few = torch.arange(n, device=dev) % 128 != 0
    for c, s, want in ((codes[0], scales[0], 0.1 * 3.1e-3), (codes[1], scales[1], np.sqrt(0.001) * 3.1e-3)):
        v = c.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128)
        got, values = v[few].mean().item(), v[few].unique()
        assert len(values) == 2
        step = (values[1] - values[0]).item()
        assert values[0] < want < values[1] and abs(got - want) <= 2.5 * step / np.sqrt(n) + 1e-6 * want
    got = p.double()[few]
    assert set(got.unique().tolist()) == {1 - 2.0 ** -8, 1.0}
    assert abs(got.mean().item() - (1 - 1e-3)) <= 2.5 * 2.0 ** -8 / np.sqrt(n) + 1e-6


def test_a_root_above_zero_is_kept(moe_gpu):
    """Beside a root 10^7 times as large a small one keeps the smallest code, and the next
    step, without a gradient, stays small; values that were never moved stay zero."""
    m, dev = moe_gpu
    t = Tensors(m, dev, [128], ("f32", "f32", False), 8, zeros=True)
    t.grad[0].zero_()
    t.grad[0][0], t.grad[0][1] = 10.0, 1e-6
    before = t.param[0].clone()
    m.adamw(t.list, step=1, lr=1e-3, weight_decay=0.0, seed=1)
    codes = t.m2[0][0]
    assert codes[0] == 0x7E and codes[1] == 1 and (codes[2:] == 0).all() and (t.m1[0][0][2:] == 0).all()
    t.grad[0].zero_()
    for step in range(2, 30):
        m.adamw(t.list, step=step, lr=1e-3, weight_decay=0.0, seed=1, offset=step)
    moved = (t.param[0] - before).abs()
    assert moved[1] < 0.1 and torch.isfinite(t.param[0]).all() and (moved[2:] == 0).all()


def test_infinities_and_nan(moe_gpu):
    """A gradient that is not finite reaches its own value alone, states included."""
    m, dev = moe_gpu
    for bits in (32, 8):
        for kind in (("f32", "f32", False), ("bf16", "f32", False), ("bf16", "f32", True)):
            t, u = (Tensors(m, dev, [400], kind, bits) for _ in range(2))
            t.grad[0][5], t.grad[0][130], u.grad[0][5], u.grad[0][130] = float("nan"), float("-inf"), 0, 0
            for x in (t, u):
                for state in (x.m1[0], x.m2[0]):   # so that the two places are not their blocks' largest
                    (state if bits == 32 else state[0])[[5, 130]] = 0
                m.adamw(x.list, step=2, seed=SEED, **HYPER)
            keep = torch.ones(400, dtype=torch.bool, device=dev)
            keep[[5, 130]] = False
            assert torch.equal(t.param[0][keep], u.param[0][keep]) and torch.isfinite(t.param[0][keep]).all()
            assert torch.isnan(t.param[0][[5, 130]]).all()   # -inf / inf
            if bits == 8:
                assert torch.equal(t.m1[0][0][keep], u.m1[0][0][keep]) and torch.equal(t.m2[0][0][keep], u.m2[0][0][keep])
                for s in (t.m1[0], t.m2[0]):
                    assert (s[0][[5, 130]] & 127 == 127).all() and torch.isfinite(s[1]).all()
            else:
                assert torch.isnan(t.m1[0][5]) and torch.isinf(t.m1[0][130]) and torch.isinf(t.m2[0][130])


def test_tiny_values(moe_gpu):
    """Blocks whose largest value has no inverse in 32 bits become zeros, others keep theirs."""
    m, dev = moe_gpu
    for size in (1e-45, 1e-38, 2.0 ** -99 * 10, 1e-20):
        t = Tensors(m, dev, [128], ("f32", "f32", False), 8, zeros=True)
        t.grad[0].fill_(size)
        want = t.expected(1, 0, HYPER)
        m.adamw(t.list, step=1, seed=SEED, **HYPER)
        t.check(want)


@pytest.mark.parametrize("bits", [32, 8])
def test_scalars_on_the_device_and_graph(moe_gpu, bits):
    """A captured step follows rate, number and gradient scale; replays equal eager steps
    with numbers, on another stream."""
    m, dev = moe_gpu
    kind = ("bf16", "bf16", True)
    t, u = (Tensors(m, dev, [3000, 17], kind, bits) for _ in range(2))
    lr, step = torch.tensor([1e-3], device=dev), torch.zeros(1, dtype=torch.int64, device=dev)
    scale = torch.ones(1, device=dev)
    hyper = dict(HYPER)
    del hyper["lr"]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step.add_(1)
        m.adamw(t.list, lr=lr, step=step, grad_scale=scale, seed=SEED, offset=4, **hyper)
    side = torch.cuda.Stream()
    for k, rate in ((1, 1e-3), (2, 5e-4), (3, 2.5e-4)):
        lr.fill_(rate)
        scale.fill_(0.5 ** k)
        graph.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            m.adamw(u.list, lr=float(np.float32(rate)), step=k, grad_scale=scale, seed=SEED, offset=4, **hyper)
        side.synchronize()
        for a, b in zip(t.list.held, u.list.held):
            assert torch.equal(a, b)


def test_a_number_of_steps_that_is_large(moe_gpu):
    m, dev = moe_gpu
    t, u = (Tensors(m, dev, [300], ("f32", "f32", False), 32) for _ in range(2))
    step = torch.tensor([(1 << 40) + 3], device=dev)
    m.adamw(t.list, step=step, **HYPER)
    m.adamw(u.list, step=(1 << 40) + 3, **HYPER)
    assert torch.equal(t.param[0], u.param[0]) and torch.isfinite(t.param[0]).all()


def test_places_past_32_bits(moe_gpu):
    """A tensor of more than 2^32 bytes of parameters and 2^31 values: its last places."""
    m, dev = moe_gpu
    n = (1 << 31) + 1000
    p = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    g = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    tail = slice(n - 999, n)
    rng = np.random.default_rng(5)
    p[tail] = torch.from_numpy(rng.standard_normal(999)).to(torch.bfloat16).to(dev)
    g[tail] = torch.from_numpy(rng.standard_normal(999)).to(torch.bfloat16).to(dev)
    codes = [torch.zeros(n, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.zeros((n + 127) // 128, device=dev) for _ in range(2)]
    w, gt = p[tail].float().cpu().numpy(), g[tail].float().cpu().numpy()
    m.adamw(m.adamw_list([p], [g], [(codes[0], scales[0])], [(codes[1], scales[1])]), step=1, seed=SEED, offset=2, **HYPER)
    w, a, _, root = B.adamw(w, gt, 0 * w, 0 * w, step=1, dtype=np.float32, **HYPER)
    first = (n - 999) // 8 * 8   # counters count groups of eight
    skip = n - 999 - first

    def numbers(what):
        nb = (n - first + 7) // 8
        ctr = np.zeros((nb, 4), dtype=np.uint64)
        ctr[:, 0] = first // 8 + np.arange(nb)
        ctr[:, 1], ctr[:, 2] = what, 2
        words = B.philox4x32_10(ctr, (SEED % (1 << 32), SEED >> 32))
        return words.astype("<u4").view("<u2").reshape(-1)[skip:skip + 999].astype(np.int64)

    bits = (w.view(np.uint32) + numbers(2).astype(np.uint32)) & 0xFFFF0000
    assert np.array_equal(p[tail].float().cpu().numpy(), bits.view(np.float32))
    # whole blocks of 128 places at the end
    start = (n - 999 + 127) // 128 * 128 - (n - 999)
    for c, s, x, what in ((codes[0], scales[0], a, 0), (codes[1], scales[1], root, 1)):
        q, sc = B.state8(x[start:], numbers(what)[start:], what == 1)
        assert np.array_equal(B.e4m3_values(c[tail][start:].cpu().numpy()), q.astype(np.float64))
        assert np.array_equal(s[-len(sc):].cpu().numpy(), sc)
    assert (p[:1 << 20] == 0).all() and (codes[1][:1 << 20] == 0).all()


def test_what_lies_beside_a_tensor_is_left(moe_gpu):
    m, dev = moe_gpu
    for bits in (32, 8):
        big = {}

        def view(name, dtype, n, fill):
            big[name] = torch.full((n + 40,), fill, dtype=dtype, device=dev)
            return big[name][16:16 + n]
        n = 133
        states = []
        for s in ("m", "v"):
            states.append(view(s, torch.float32, n, 7.0) if bits == 32 else
                          (view(s, torch.uint8, n, 0x55), view(s + "s", torch.float32, 2, 7.0)))
        lst = m.adamw_list([view("p", torch.bfloat16, n, 7.0)], [torch.ones(n, device=dev)], [states[0]], [states[1]],
                           [view("w", torch.float32, n, 7.0)])
        before = {k: v.clone() for k, v in big.items()}
        m.adamw(lst, lr=0.1, step=1)
        for k, v in big.items():
            inner = 2 if k[-1] == "s" else n
            assert torch.equal(v[:16], before[k][:16]) and torch.equal(v[16 + inner:], before[k][16 + inner:])
            assert not torch.equal(v, before[k])


def test_refused_lists(moe_gpu):
    m, dev = moe_gpu
    f = lambda n=64, dtype=torch.float32: torch.zeros(n, dtype=dtype, device=dev)   # noqa: E731
    p, g, a, b = f(), f(), f(), f()
    errors = (ValueError, TypeError, m.MoEError)
    q, s = f(64, torch.uint8), f(1)
    for args in (([p], [g, g], [a], [b]), ([p], [g], [a], [a]), ([p], [g], [p], [b]), ([p, p], [g, g], [a, f()], [b, f()]),
                 ([p], [f(63)], [a], [b]), ([p], [g], [a.half()], [b]), ([p], [g.cpu()], [a], [b]),
                 ([p], [g], [(q, s)], [b]), ([p], [g], [(q, f(2))], [(f(64, torch.uint8), f(1))]),
                 ([p.double()], [g], [a], [b]), ([f(128)[::2]], [g], [a], [b]), ([p, p.half()], [g, g], [a, f()], [b, f()]),
                 ([p], [g], [a], [b], [p])):
        with pytest.raises(errors):
            m.adamw_list(*args)
    for lst in (m.adamw_list([f(64, torch.float16)], [g], [a], [b]),              # fp16 without a copy
                m.adamw_list([p], [g.half()], [a], [b]), m.adamw_list([p], [g], [a], [b], [f()])):
        with pytest.raises(m.MoEError):
            m.adamw(lst, lr=1e-3, step=1)
    lst = m.adamw_list([p], [g], [a], [b])
    for bad in (dict(step=0), dict(beta1=1.0), dict(beta2=-0.1), dict(eps=-1.0), dict(lr=float("nan")),
                dict(weight_decay=float("inf")), dict(lr=f(2)), dict(step=f(1)), dict(grad_scale=f(1).half())):
        with pytest.raises(errors):
            m.adamw(lst, **{**dict(lr=1e-3, step=1), **bad})
    assert (p == 0).all()
    m.adamw(m.adamw_list([], [], [], []), lr=1e-3, step=1)
    m.adamw(m.adamw_list([f(0)], [f(0)], [f(0)], [f(0)]), lr=1e-3, step=1)


def test_gradients_that_overlap(moe_gpu):
    """A gradient may serve two tensors, but not lie in what the step writes: a block
    would read there what another has written."""
    m, dev = moe_gpu
    f = lambda n=64: torch.zeros(n, dtype=torch.float32, device=dev)   # noqa: E731
    p, a, b, more = f(), f(), f(), f(256)
    for g in (p, a, b):
        with pytest.raises(ValueError):
            m.adamw_list([p], [g], [a], [b])
    for at in (129, 191, 64):   # its end and its beginning in what is written, all of it
        with pytest.raises(ValueError):
            m.adamw_list([f(64 if at > 64 else 192)], [more[at:at + 64] if at > 64 else more[64:256]],
                         [more[128:192] if at > 64 else f(192)], [f(64 if at > 64 else 192)] if at > 64 else [more[:192]])
    g = more[64:128]
    g.fill_(1.0)
    q = f()
    m.adamw(m.adamw_list([p, q], [g, g], [more[:64], more[128:192]], [f(), f()]), lr=0.5, step=1, eps=0.0, weight_decay=0.0)
    # about eight roundings of 2^-24 each
    assert torch.allclose(p, torch.full_like(p, -0.5), rtol=1e-6) and torch.equal(p, q) and (g == 1).all()
    assert (more[192:] == 0).all()
