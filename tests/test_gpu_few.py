"""The layer for a few tokens against the definition in 64 bits.

Tolerances: a product sum over n columns in 32 bits takes n / 16 partial sums of the
tensor cores, each cut off by at most 2^-22 of the terms' sizes, plus the fixed ones:
sums(n) = (n / 16 + 16) 2^-22.  The activation a is rounded to bf16 (half a step,
2^-8) and carries what h and u are off by (|silu'| <= 1.1); out adds the error of its
own sum and half a step.  Logits that decide about an expert by less than their error
are not used: inputs are drawn so that this has no effect.  GPU only."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
BF = dict(dtype=torch.bfloat16, device="cuda")
HALF = 2.0 ** -8


def sums(n):
    return (n / 16 + 16) * 2.0 ** -22


def inputs(T, d, E, f, seed=0, scale=1.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, scale):
        return (torch.randn(shape, generator=gen, device="cuda") * scale).to(torch.bfloat16)
    w = 0.02 * (1024 / d) ** 0.5
    return (normal(T, d, scale=scale), normal(E, d, scale=w), normal(E, f, d, scale=w), normal(E, f, d, scale=w),
            normal(E, d, f, scale=0.05))


def routing(x, w_router, bias, k):
    """(logits, indices, gates) in 64 bits, larger logits first, then lower experts."""
    logits = x.double() @ w_router.double().T
    if bias is not None:
        logits = logits + bias.double()
    idx = torch.sort(logits, stable=True, dim=-1, descending=True).indices[:, :k]
    return logits, idx, torch.softmax(logits.gather(1, idx), -1)


def experts(x, idx, gates, w_gate, w_up, w_down):
    """(out, bound of its error) in 64 bits; indices outside [0, E) add nothing."""
    T, d, f = x.shape[0], x.shape[1], w_gate.shape[1]
    out, err = torch.zeros(T, d, dtype=torch.float64, device="cuda"), torch.zeros(T, d, dtype=torch.float64, device="cuda")
    xd = x.double()
    for e in idx.unique().tolist():
        if not 0 <= e < w_gate.shape[0]:
            continue
        t, j = (idx == e).nonzero(as_tuple=True)
        g = gates[t, j].double()[:, None]
        wg, wu, wd = (v[e].double() for v in (w_gate, w_up, w_down))
        h, u = xd[t] @ wg.T, xd[t] @ wu.T
        dh, du = xd[t].abs() @ wg.abs().T * sums(d), xd[t].abs() @ wu.abs().T * sums(d)
        s = h * torch.sigmoid(h)
        a = s * u
        da = 1.1 * dh * (u.abs() + du) + s.abs() * du + (HALF + 2.0 ** -18) * a.abs() + 1e-38
        out.index_add_(0, t, a @ wd.T * g)
        err.index_add_(0, t, (da @ wd.abs().T + (a.abs() + da) @ wd.abs().T * (sums(f) + 34 * 2.0 ** -24)) * g.abs())
    return out, err + HALF * (out.abs() + err) + 1e-38


def close(got, want, err):
    off = (got.double() - want).abs()
    assert torch.isfinite(got).all()
    assert (off <= err).all(), f"{(off / err).max().item():.2f} of the bound"


def call(m, x, wr, bias, wg, wu, wd, k, **kw):
    T, d = x.shape
    E, f = wg.shape[:2]
    s = m.shape(T, d, E, k, f)
    ws = torch.full((m.few_workspace(s),), 0x7F, dtype=torch.uint8, device="cuda")
    m.clear_error(ws)
    out = torch.full((T, d), 9.0, **BF)
    m.forward_few(s, x, wr, bias, wg, wu, wd, out, ws, **kw)
    return out, m.read_error(ws)


SHAPES = [(1, 128, 1, 1, 128), (1, 128, 4, 2, 128), (2, 256, 8, 2, 128), (3, 384, 8, 8, 256), (5, 512, 9, 3, 384),
          (16, 512, 32, 4, 256), (17, 640, 33, 1, 128), (31, 256, 64, 8, 640), (32, 1024, 16, 5, 128),
          (33, 128, 129, 6, 128), (64, 256, 256, 32, 128), (64, 512, 8, 8, 256), (7, 2048, 64, 4, 1408),
          (1, 4096, 64, 8, 2048), (64, 8192, 4, 2, 128), (48, 128, 2, 1, 2048)]


@pytest.mark.parametrize("T,d,E,k,f", SHAPES, ids=str)
@pytest.mark.parametrize("with_bias", [False, True], ids=["plain", "bias"])
def test_layer(moe_gpu, T, d, E, k, f, with_bias):
    m, _ = moe_gpu
    x, wr, wg, wu, wd = inputs(T, d, E, f, seed=T + d + E)
    bias = torch.randn(T, E, device="cuda") if with_bias else None
    idx, gates = torch.full((T, k), -9, dtype=torch.int32, device="cuda"), torch.full((T, k), -9.0, device="cuda")
    logits = torch.full((T, E), -9.0, device="cuda")
    out, error = call(m, x, wr, bias, wg, wu, wd, k, topk_idx=idx, gates=gates, logits=logits)
    assert error == 0
    l64, i64, _ = routing(x, wr, bias, k)
    size = x.double().abs() @ wr.double().abs().T
    off = sums(d) * size + 2.0 ** -23 * l64.abs()
    assert ((logits.double() - l64).abs() <= off).all()
    # the selection is that of the logits as they came out: larger first, lower expert first
    want = torch.sort(logits, stable=True, dim=-1, descending=True).indices[:, :k]
    assert torch.equal(idx.long(), want)
    g = torch.softmax(logits.double().gather(1, want), -1)
    assert ((gates.double() - g).abs() <= 2.0 ** -20 * g).all()
    want_out, err = experts(x, want, g, wg, wu, wd)
    close(out, want_out, err + 2.0 ** -20 * want_out.abs())
    # the same bits without the optional outputs, and with the routing given
    again, error = call(m, x, wr, bias, wg, wu, wd, k)
    assert error == 0 and torch.equal(again, out)
    given, error = call(m, x, None, None, wg, wu, wd, k, topk_idx=idx, gates=gates)
    assert error == 0 and torch.equal(given, out)


def test_equal_logits_and_routing_of_the_layer(moe_gpu):
    """Rows of W_router that are equal give equal logits: lower experts go first; the
    whole call beside the layer's own on the same tokens."""
    m, _ = moe_gpu
    T, d, E, k, f = 40, 512, 24, 5, 256
    x, wr, wg, wu, wd = inputs(T, d, E, f)
    wr[8:16] = wr[:8]
    wr[16:] = wr[:8]
    idx = torch.empty(T, k, dtype=torch.int32, device="cuda")
    gates, logits = torch.empty(T, k, device="cuda"), torch.empty(T, E, device="cuda")
    out, _ = call(m, x, wr, None, wg, wu, wd, k, topk_idx=idx, gates=gates, logits=logits)
    assert torch.equal(logits[:, :8], logits[:, 8:16]) and torch.equal(logits[:, :8], logits[:, 16:])
    assert torch.equal(idx.long(), torch.sort(logits, stable=True, dim=-1, descending=True).indices[:, :k])
    assert ((idx[:, 1] - idx[:, 0]) % 8 == 0).all() and (idx[:, 1] > idx[:, 0]).all()
    s = m.shape(T, d, E, k, f)
    buf = m.allocate(s, with_grads=False)
    buf.saved["logits"].copy_(logits)
    full = torch.empty_like(out)
    m.forward(buf, x, None, None, wg, wu, wd, full)
    assert torch.equal(buf.saved["topk_idx"], idx) and torch.equal(buf.saved["gates"], gates)
    want, err = experts(x, idx, gates, wg, wu, wd)
    close(out, want, err)
    # the layer rounds y to bf16 too: half a step of each route's product
    assert ((full.double() - want).abs() <= err + 3 * HALF * want.abs().max()).all()


def test_given_routing(moe_gpu):
    """No expert (-1), an expert twice, tokens without any, indices out of range."""
    m, _ = moe_gpu
    T, d, E, k, f = 37, 256, 12, 4, 256
    x, _, wg, wu, wd = inputs(T, d, E, f)
    gen = torch.Generator(device="cuda").manual_seed(3)
    idx = torch.randint(-1, E, (T, k), generator=gen, device="cuda", dtype=torch.int32)
    idx[5] = -1
    idx[6] = 7            # one expert four times
    idx[7] = torch.tensor([3, 3, -1, 3], device="cuda")
    idx[36, 0] = 11
    gates = torch.randn(T, k, generator=gen, device="cuda")
    out, error = call(m, x, None, None, wg, wu, wd, k, topk_idx=idx, gates=gates)
    assert error == 0
    want, err = experts(x, idx, gates, wg, wu, wd)
    # gates of one expert are added in 32 bits before they multiply
    extra = experts(x, idx, gates.abs(), wg.abs(), wu.abs(), wd.abs())[0] * 4 * 2.0 ** -24 * 64
    close(out, want, err + extra)
    assert (out[5] == 0).all()
    none = torch.full_like(idx, -1)
    out, error = call(m, x, None, None, wg, wu, wd, k, topk_idx=none, gates=gates)
    assert error == 0 and (out == 0).all()
    bad = idx.clone()
    bad[9, 1], bad[20, 3], bad[21, 0] = E, -2, 2 ** 31 - 1
    out, error = call(m, x, None, None, wg, wu, wd, k, topk_idx=bad, gates=gates)
    assert error == m.DEVERR_BOUNDS
    want, err = experts(x, bad, gates, wg, wu, wd)
    close(out, want, err + extra)


def test_rows_keep_to_themselves(moe_gpu):
    """What is not finite in one row or in one expert's weights stays with it.  With the
    same routing the other tokens keep their bits; rows that change take other experts, and
    the parts in which a sum over d_ff is taken depend on how many routes there are: both
    results are within the bound of the sums' errors, so they differ by twice that and no
    more."""
    m, _ = moe_gpu
    T, d, E, k, f = 24, 512, 16, 3, 256
    x, wr, wg, wu, wd = inputs(T, d, E, f)
    idx, gates = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    out, _ = call(m, x, wr, None, wg, wu, wd, k, topk_idx=idx, gates=gates)
    bound = experts(x, idx, gates, wg, wu, wd)[1]
    odd = x.clone()
    odd[3], odd[4, 7], odd[5] = float("nan"), float("inf"), 0
    got, error = call(m, odd, wr, None, wg, wu, wd, k)
    assert error == m.DEVERR_NONFINITE_LOGIT
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[[3, 4, 5]] = False
    assert ((got[keep].double() - out[keep].double()).abs() <= 2 * bound[keep]).all() and (got[5] == 0).all()
    for w in (wg, wu, wd):   # an expert of NaN: tokens that do not take it stay as they are
        e = idx[0, 0].item()
        was = w[e].clone()
        w[e] = float("nan")
        got, _ = call(m, x, wr, None, wg, wu, wd, k)
        takes = (idx == e).any(1)
        assert takes.any() and not takes.all()
        assert torch.equal(got[~takes], out[~takes]) and torch.isnan(got[takes]).all()
        w[e] = was


def test_logits_that_are_not_finite(moe_gpu):
    """A NaN in the bias: below every other logit, gates of zero, the error word's bit."""
    m, _ = moe_gpu
    T, d, E, k, f = 6, 256, 8, 2, 128
    x, wr, wg, wu, wd = inputs(T, d, E, f)
    bias = torch.zeros(T, E, device="cuda")
    bias[2, 3], bias[4, 1] = float("nan"), float("inf")
    idx, gates = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    out, error = call(m, x, wr, bias, wg, wu, wd, k, topk_idx=idx, gates=gates)
    assert error == m.DEVERR_NONFINITE_LOGIT
    assert 3 not in idx[2].tolist() and idx[4, 0] == 1 and (gates[[2, 4]] == 0).all() and (out[[2, 4]] == 0).all()
    assert (gates[[0, 1, 3, 5]].sum(1) - 1).abs().max() < 1e-6


def test_more_rows_than_32_bits_of_weights(moe_gpu):
    """Experts whose weights begin more than 2^32 bytes into their matrix."""
    m, _ = moe_gpu
    T, d, E, k, f = 3, 4096, 130, 2, 4480
    wg, wu, wd = (torch.zeros(E, *s, **BF) for s in ((f, d), (f, d), (d, f)))
    x = inputs(T, d, 1, 128)[0]
    for e in (0, 128, 129):
        for w in (wg, wu, wd):
            w[e] = (torch.randn(w[e].shape, device="cuda") * 0.02).to(torch.bfloat16)
    idx = torch.tensor([[129, 0], [128, 129], [0, 128]], dtype=torch.int32, device="cuda")
    gates = torch.rand(T, k, device="cuda")
    out, error = call(m, x, None, None, wg, wu, wd, k, topk_idx=idx, gates=gates)
    assert error == 0
    close(out, *experts(x, idx, gates, wg, wu, wd))


def test_graph_streams_and_repeats(moe_gpu):
    """Captured and replayed on new tokens, on another stream, calls back to back: the
    same bits; two graphs with one workspace, one after the other."""
    m, _ = moe_gpu
    T, d, E, k, f = 9, 1024, 32, 4, 256
    x, wr, wg, wu, wd = inputs(T, d, E, f)
    s = m.shape(T, d, E, k, f)
    ws = torch.zeros(m.few_workspace(s), dtype=torch.uint8, device="cuda")
    out, other = torch.empty_like(x), torch.empty_like(x)

    def run(o):
        m.forward_few(s, x, wr, None, wg, wu, wd, o, ws)
    run(out)
    torch.cuda.synchronize()
    graphs = []
    for o in (out, other):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(o)
            run(o)
        graphs.append(g)
    side, eager = torch.cuda.Stream(), torch.empty_like(x)
    for seed in range(4):
        x.copy_(inputs(T, d, 1, 128, seed=seed)[0])
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            run(eager)
        side.synchronize()
        for _ in range(50):
            run(other)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.equal(other, eager)
    assert m.read_error(ws) == 0


def test_in_place_and_two_streams(moe_gpu):
    """out in x's buffer; two calls at once, each with its stream and workspace."""
    m, _ = moe_gpu
    T, d, E, k, f = 20, 1024, 16, 4, 512
    x, wr, wg, wu, wd = inputs(T, d, E, f)
    out, _ = call(m, x, wr, None, wg, wu, wd, k)
    s = m.shape(T, d, E, k, f)
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.zeros(m.few_workspace(s), dtype=torch.uint8, device="cuda") for _ in range(2)]
    outs = [torch.empty_like(x) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(30):
        for st, w, o in zip(streams, ws, outs):
            m.forward_few(s, x, wr, None, wg, wu, wd, o, w, stream=st)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], out) and torch.equal(outs[1], out)
    assert m.read_error(ws[0]) == 0 and m.read_error(ws[1]) == 0
    m.forward_few(s, x, wr, None, wg, wu, wd, x, ws[0])
    assert torch.equal(x, out)


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(moe_gpu, seed):
    """Shapes, routing and expert loads of all kinds: one expert for most tokens, tokens
    without any, more columns than a stage holds."""
    m, _ = moe_gpu
    rng = np.random.default_rng(seed)
    T, E = int(rng.integers(1, 65)), int(rng.integers(1, 100))
    k = int(rng.integers(1, min(E, 12) + 1))
    d, f = 128 * int(rng.integers(1, 24)), 128 * int(rng.integers(1, 12))
    x, _, wg, wu, wd = inputs(T, d, E, f, seed=seed)
    idx = torch.from_numpy(np.stack([rng.permutation(E)[:k] for _ in range(T)])).to(torch.int32).cuda()
    if seed % 3 == 0:
        idx[rng.random(T) < 0.7, 0] = E - 1
    if seed % 4 == 1:
        idx[torch.from_numpy(rng.random((T, k)) < 0.5).cuda()] = -1
    gates = torch.rand(T, k, device="cuda")
    out, error = call(m, x, None, None, wg, wu, wd, k, topk_idx=idx, gates=gates)
    assert error == 0
    want, err = experts(x, idx, gates, wg, wu, wd)
    extra = experts(x, idx, gates, wg.abs(), wu.abs(), wd.abs())[1] * 2.0 ** -20   # gates of one expert added
    close(out, want, err + extra)


def test_refused_tensors(moe_gpu):
    m, _ = moe_gpu
    T, d, E, k, f = 4, 256, 8, 2, 128
    x, wr, wg, wu, wd = inputs(T, d, E, f)
    s = m.shape(T, d, E, k, f)
    good = dict(s=s, x=x, w_router=wr, logit_bias=None, w_gate=wg, w_up=wu, w_down=wd, out=torch.zeros_like(x),
                ws=torch.zeros(m.few_workspace(s), dtype=torch.uint8, device="cuda"))
    idx, gates = torch.zeros(T, k, dtype=torch.int32, device="cuda"), torch.ones(T, k, device="cuda")
    for bad in (dict(x=x.float()), dict(x=x[:3]), dict(x=x.cpu()), dict(w_gate=wg[:7]), dict(w_down=wd.half()),
                dict(out=torch.zeros(d, T, **BF).t()), dict(ws=good["ws"][:100]), dict(topk_idx=idx.long()),
                dict(gates=gates[:, :1]), dict(w_router=None), dict(w_router=None, topk_idx=idx),
                dict(w_router=None, gates=gates), dict(logit_bias=gates), dict(s=m.shape(65, d, E, k, f)),
                dict(w_router=None, topk_idx=idx, gates=gates, logit_bias=torch.zeros(T, E, device="cuda")),
                dict(s=m.shape(T, d, E, k, f, prec=m.MXFP8)), dict(s=m.shape(T, d, E, 9, f))):
        with pytest.raises((ValueError, TypeError, m.MoEError)):
            m.forward_few(**{**good, **bad})
    none = m.shape(0, d, E, k, f)
    m.forward_few(none, x[:0], wr, None, wg, wu, wd, x[:0], good["ws"])
