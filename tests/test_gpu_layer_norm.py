"""Residual addition + layer norm (forward, backward, 8-bit output) on the GPU against
the float64 oracle.

Tolerances: as for the RMS norm, a stored value is off by at most half a step of its
type and fp32 work by REL = 2^-18 (64 roundings) relative to the terms that enter it.
The mean of a row is off by REL of its mean |h| (`size`), and so is every deviation
from it: a term of its own beside the deviation.  The squares' mean takes that error
squared (its first order adds up to the sum of the deviations, zero).  GPU only."""
import numpy as np
import pytest
import torch

from gpu_util import f64, sf_unpack
from oracle import block_oracle as B
from test_gpu_norm import DT, REL, SHAPES, TYPES, close, e4m3_step, half, normal, strided

pytestmark = pytest.mark.gpu
SEED, OFFSET = 0x1234567890ABCDEF, (7 << 32) + 9


def stream_of(rng, rows, d, dtype, dev, offset=1.5):
    """Rows whose means differ, by `offset` times the deviations."""
    return normal(rng, (rows, d), torch.float32, dev, 2.0).add_(normal(rng, (rows, 1), torch.float32, dev, 2.0 * offset)).to(dtype)


def check_forward(m, dev, rows, d, xt, rt, wt, p=0.0, residual=True, bias=True, layout=lambda t: t, eps=1e-5, stream=None,
                  offset=1.5):
    rng = np.random.default_rng(rows * 131 + d)
    x = layout(normal(rng, (rows, d), DT[xt], dev))
    res = layout(stream_of(rng, rows, d, DT[rt], dev, offset)) if residual else None
    w, b = normal(rng, (d,), DT[wt], dev), normal(rng, (d,), DT[wt], dev) if bias else None
    y, h = layout(torch.zeros(rows, d, dtype=DT[xt], device=dev)), None
    if residual or p:
        h = layout(torch.zeros(rows, d, dtype=DT[rt], device=dev))
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    m.add_layer_norm(x, w, b, y, residual=res, h=h, mean=mean, rstd=rstd, eps=eps, p=p, seed=SEED, offset=OFFSET,
                     stream=stream)
    torch.cuda.synchronize()
    drop = B.dropout(f64(x), p, SEED, OFFSET)
    if h is not None:
        close(h, drop + (f64(res) if residual else 0), h.dtype, np.abs(drop) + (np.abs(f64(res)) if residual else 0))
    hd = f64(h) if h is not None else f64(x)   # the norm is that of the stored stream
    _, want, mu, r = B.add_layer_norm(hd, None, f64(w), f64(b) if bias else None, eps)
    size = np.abs(hd).mean(-1)
    assert (np.abs(f64(mean) - mu) <= REL * size).all()
    shift = (REL * size * r) ** 2   # of the squares' mean plus eps, relative to it
    assert (np.abs(f64(rstd) - r) <= (REL + shift) * r).all()
    scale = r[:, None] * np.abs(f64(w))
    terms = (np.abs(hd - mu[:, None]) * (1 + shift[:, None] / REL) + size[:, None]) * scale
    close(y, want, y.dtype, terms + (np.abs(f64(b)) if bias else 0))
    return x, res, w, b, h, y, mean, rstd


@pytest.mark.parametrize("rows,d", SHAPES, ids=str)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_forward(moe_gpu, rows, d, types):
    m, dev = moe_gpu
    check_forward(m, dev, rows, d, *types)


@pytest.mark.parametrize("rows,d", [(5, 31), (3, 256), (65, 1000), (9, 1001), (2, 9000)], ids=str)
@pytest.mark.parametrize("types", [TYPES[0], TYPES[1], TYPES[4], TYPES[5]], ids="-".join)
@pytest.mark.parametrize("residual,bias", [(True, False), (False, True)], ids=["res", "bias"])
def test_forward_with_dropout(moe_gpu, rows, d, types, residual, bias):
    m, dev = moe_gpu
    check_forward(m, dev, rows, d, *types, p=0.3, residual=residual, bias=bias)


@pytest.mark.parametrize("d", [33, 64, 250, 1001, 2048, 8192, 9000])
def test_forward_of_rows_far_from_zero(moe_gpu, d):
    """Means of a thousand deviations: the variance is that of the deviations."""
    m, dev = moe_gpu
    check_forward(m, dev, 40, d, "f32", "f32", "f32", offset=1000.0)


@pytest.mark.parametrize("extra,shift", [(8, 0), (64, 0), (1, 0), (8, 8), (5, 3), (0, 1)], ids=str)
@pytest.mark.parametrize("d", [64, 77, 2048])
def test_forward_strides_and_alignment(moe_gpu, extra, shift, d):
    m, dev = moe_gpu
    out = check_forward(m, dev, 9, d, "bf16", "f32", "bf16", p=0.2, layout=lambda t: strided(t, extra, shift))
    for v in out[4:6]:   # what lies between the rows keeps its NaN
        big = torch.as_strided(v, (9, d + extra + shift), (d + extra + shift, 1), 0)
        assert torch.isnan(big[:, :shift]).all() and torch.isnan(big[:, shift + d:]).all()


@pytest.mark.parametrize("place", ["w", "b"])
def test_forward_with_weights_off_the_boundary(moe_gpu, place):
    """A weight or a bias that starts two bytes off a vector's boundary."""
    m, dev = moe_gpu
    x, _, w, b, h, y, _, _ = check_forward(m, dev, 5, 256, "bf16", "bf16", "bf16", residual=False)
    off = {"w": w, "b": b}
    off[place] = torch.cat([w[:1], off[place]])[1:]
    z = torch.empty_like(y)
    m.add_layer_norm(x, off["w"], off["b"], z)
    assert (f64(z) - f64(y)).__abs__().max() <= 2 * half(torch.bfloat16) * f64(y).__abs__().max()


def test_forward_in_place(moe_gpu):
    m, dev = moe_gpu
    for d in (1001, 2048):
        x, res, w, b, h, y, _, _ = check_forward(m, dev, 12, d, "bf16", "bf16", "bf16", p=0.25)
        m.add_layer_norm(x, w, b, x, residual=res, h=res, p=0.25, seed=SEED, offset=OFFSET)
        assert torch.equal(res, h) and torch.equal(x, y)


def test_forward_of_extreme_rows(moe_gpu):
    """Equal values (eps alone), one column, an infinity, a NaN; the rows beside them
    keep their values, and no rows are no work."""
    m, dev = moe_gpu
    rng = np.random.default_rng(1)
    d = 256
    x = normal(rng, (5, d), torch.float32, dev)
    x[0], x[1, 5], x[2, 9] = 7.0, float("inf"), float("nan")
    x[3] *= 1e15
    w, b = torch.ones(d, device=dev), normal(rng, (d,), torch.float32, dev)
    y, mean, rstd = torch.empty_like(x), torch.empty(5, device=dev), torch.empty(5, device=dev)
    m.add_layer_norm(x, w, b, y, mean=mean, rstd=rstd, eps=1e-6)
    assert torch.equal(y[0], b) and mean[0].item() == 7.0 and abs(rstd[0].item() - 1e3) < 1e-2
    assert torch.isnan(y[1:3]).all()
    for r in (3, 4):
        c = f64(x[r]) - f64(x[r]).mean()
        want = c / np.sqrt((c * c).mean() + 1e-6) + f64(b)
        assert (np.abs(f64(y[r]) - want) <= REL * (4 + np.abs(want) + np.abs(f64(b)))).all()
    one = torch.full((3, 1), 5.0, device=dev)
    m.add_layer_norm(one, w[:1], b[:1], one)
    assert (one == b[0]).all()
    none = torch.empty(0, d, device=dev)
    m.add_layer_norm(none, w, b, none, mean=mean[:0], rstd=rstd[:0])


@pytest.mark.parametrize("rows,d", [(1, 128), (3, 256), (129, 1408), (70, 2048), (2, 4096), (5, 16384)], ids=str)
@pytest.mark.parametrize("rt,wt,p,bias", [("bf16", "bf16", 0.0, True), ("f32", "f32", 0.1, True), ("f32", "bf16", 0.0, False)])
def test_forward_mxfp8(moe_gpu, rows, d, rt, wt, p, bias):
    m, dev = moe_gpu
    rng = np.random.default_rng(rows + d)
    x, res = normal(rng, (rows, d), torch.bfloat16, dev), stream_of(rng, rows, d, DT[rt], dev)
    w, b = normal(rng, (d,), DT[wt], dev), normal(rng, (d,), DT[wt], dev)
    w[32:64] = 0
    b[32:64] = 0
    pad = (rows + 127) // 128 * 128
    q = torch.full((pad, d), 0x55, dtype=torch.uint8, device=dev)
    sc = torch.full((pad * d // 32,), 0x55, dtype=torch.uint8, device=dev)
    dq, out = (torch.full((pad, d), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(2))
    h, mean, rstd = torch.empty(rows, d, dtype=DT[rt], device=dev), torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    m.add_layer_norm(x, w, b if bias else None, None, residual=res, h=h, mean=mean, rstd=rstd, p=p, seed=5, offset=1,
                     y_q=q, y_scales=sc, y_dq=dq)
    m.dequantize_mxfp8(pad, d, q, sc, out)
    assert torch.equal(out.view(torch.int16), dq.view(torch.int16))
    s = sf_unpack(sc.cpu().numpy(), pad, d // 32).astype(np.int64) - 127
    assert (q[rows:] == 0).all() and (out[rows:] == 0).all() and (s[rows:] == 0).all()
    s = s[:rows]
    c = f64(h) - f64(mean)[:, None]
    y = c * f64(rstd)[:, None] * f64(w) + (f64(b) if bias else 0)
    # fp32 work on deviations, products and the sum with the bias, of the saved mean and rstd
    off = 4 * REL * (np.abs(c) * f64(rstd)[:, None] * np.abs(f64(w)) + np.abs(f64(b)))
    top, slack = np.abs(y.reshape(rows, -1, 32)).max(-1), off.reshape(rows, -1, 32).max(-1)
    lim = 448 * np.exp2(s)
    zero = top == 0
    assert (s[zero] == 0).all()
    assert (top <= lim + slack)[~zero].all() and (top > lim / 2 - slack)[~zero].all()
    unit = np.repeat(np.exp2(s), 32, axis=1)
    err = np.abs(f64(out[:rows]) - y)
    assert (err <= e4m3_step(np.minimum(np.abs(y) / unit, 448)) * unit / 2 + off).all()


# ------------------------------------------------------------------ backward
def check_backward(m, dev, rows, d, xt, rt, wt, p=0.0, with_dres=True, layout=lambda t: t, outs=("dh", "dx", "dw", "db"),
                   stream=None):
    rng = np.random.default_rng(rows * 17 + d)
    dy = layout(normal(rng, (rows, d), DT[xt], dev))
    h = layout(stream_of(rng, rows, d, DT[rt], dev))
    dres = layout(normal(rng, (rows, d), DT[rt], dev)) if with_dres else None
    w = normal(rng, (d,), DT[wt], dev)
    _, _, mu, r = B.add_layer_norm(f64(h), None, 1.0, None, 1e-5)
    mean, rstd = (torch.from_numpy(v).float().to(dev) for v in (mu, r))
    o = {"dh": layout(torch.zeros(rows, d, dtype=DT[rt], device=dev)),
         "dx": layout(torch.zeros(rows, d, dtype=DT[xt], device=dev)),
         "dw": torch.full((d,), 9.0, device=dev), "db": torch.full((d,), 9.0, device=dev)}
    o = {n: v for n, v in o.items() if n in outs}
    ws = torch.full((m.add_layer_norm_bwd_workspace(rows, d),), 0xA5, dtype=torch.uint8, device=dev)
    m.add_layer_norm_bwd(dy, h, mean, rstd, w, dres=dres, ws=ws, p=p, seed=SEED, offset=3, stream=stream, **o)
    torch.cuda.synchronize()
    a = [f64(t) if t is not None else None for t in (dy, h, mean, rstd, w, dres)]
    dh, dx, dw, db = B.add_layer_norm_bwd(*a, p, SEED, 3)
    g, r = a[0] * a[4], a[3][:, None]
    # (h - mean) is rounded once: half a step of itself; the row's means by REL of those of |g| and |g n|
    n = np.abs(a[1] - a[2][:, None]) * r
    terms = r * (np.abs(g) + np.abs(g).mean(-1, keepdims=True) + n * np.abs(g * n).mean(-1, keepdims=True))
    terms = terms + (np.abs(a[5]) if with_dres else 0)
    if "dh" in o:
        close(o["dh"], dh, DT[rt], terms)
    if "dx" in o:
        close(o["dx"], dx, DT[xt], B.dropout(terms, p, SEED, 3))
    for name, want, size in (("dw", dw, np.abs(a[0]) * n), ("db", db, np.abs(a[0]))):
        if name in o:
            lim = (rows + 64) * 2.0 ** -24 * size.sum(0) + 1e-37
            assert (np.abs(f64(o[name]) - want) <= lim).all(), name
    return o


@pytest.mark.parametrize("rows,d", SHAPES, ids=str)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_backward(moe_gpu, rows, d, types):
    m, dev = moe_gpu
    check_backward(m, dev, rows, d, *types)


@pytest.mark.parametrize("rows,d", [(5, 31), (3, 256), (65, 1000), (9, 1001), (2, 9000), (3000, 64), (2500, 1024)], ids=str)
@pytest.mark.parametrize("types", [TYPES[0], TYPES[1], TYPES[4], TYPES[5]], ids="-".join)
@pytest.mark.parametrize("with_dres", [True, False], ids=["dres", "nodres"])
def test_backward_with_dropout(moe_gpu, rows, d, types, with_dres):
    m, dev = moe_gpu
    check_backward(m, dev, rows, d, *types, p=0.3, with_dres=with_dres)


@pytest.mark.parametrize("outs", [("dh",), ("dx",), ("dw",), ("db",), ("dh", "dx"), ("dx", "dw", "db")], ids="-".join)
@pytest.mark.parametrize("d", [77, 512])
def test_backward_of_some_outputs(moe_gpu, outs, d):
    m, dev = moe_gpu
    check_backward(m, dev, 40, d, "bf16", "f32", "f32", p=0.1, outs=outs)


@pytest.mark.parametrize("extra,shift", [(8, 0), (1, 0), (8, 8), (5, 3)], ids=str)
@pytest.mark.parametrize("d", [64, 77, 2048])
def test_backward_strides_and_alignment(moe_gpu, extra, shift, d):
    m, dev = moe_gpu
    check_backward(m, dev, 9, d, "bf16", "bf16", "bf16", p=0.2, layout=lambda t: strided(t, extra, shift))


def test_a_row_that_is_not_finite_keeps_to_itself(moe_gpu):
    """An infinite mean in one row: the other rows' gradients stay, also where its group
    of threads has no row afterwards (64 columns: four rows a warp)."""
    m, dev = moe_gpu
    rng = np.random.default_rng(3)
    for d in (64, 77, 512):
        rows = 152 * 64 + 1   # some groups of a block go one row further than others
        dy, h = normal(rng, (rows, d), torch.bfloat16, dev), normal(rng, (rows, d), torch.bfloat16, dev)
        w, mean, rstd = torch.ones(d, dtype=torch.bfloat16, device=dev), torch.zeros(rows, device=dev), torch.ones(rows, device=dev)
        dh, ref = torch.empty_like(h), torch.empty_like(h)
        m.add_layer_norm_bwd(dy, h, mean, rstd, w, dh=ref)
        mean[5] = float("inf")
        m.add_layer_norm_bwd(dy, h, mean, rstd, w, dh=dh)
        assert not torch.isfinite(dh[5]).any()
        keep = torch.arange(rows, device=dev) != 5
        assert torch.equal(dh[keep], ref[keep])


def test_backward_is_deterministic_and_in_place(moe_gpu):
    m, dev = moe_gpu
    rng = np.random.default_rng(2)
    rows = 3000
    for d in (1001, 1024):
        dy, h, dres = (normal(rng, (rows, d), torch.bfloat16, dev) for _ in range(3))
        w, mean, rstd = normal(rng, (d,), torch.bfloat16, dev), torch.rand(rows, device=dev), torch.rand(rows, device=dev)
        ws = torch.empty(m.add_layer_norm_bwd_workspace(rows, d), dtype=torch.uint8, device=dev)
        first = None
        for _ in range(3):
            o = torch.empty_like(h), torch.empty_like(dy), torch.empty(d, device=dev), torch.empty(d, device=dev)
            m.add_layer_norm_bwd(dy, h, mean, rstd, w, dres, *o, ws=ws, p=0.1, seed=1)
            first = first or o
            assert all(torch.equal(a, b) for a, b in zip(first, o))
        m.add_layer_norm_bwd(dy, h, mean, rstd, w, dres, dres, dy, *o[2:], ws=ws, p=0.1, seed=1)
        assert torch.equal(dres, first[0]) and torch.equal(dy, first[1])


def test_backward_without_rows(moe_gpu):
    m, dev = moe_gpu
    e, none = torch.empty(0, 64, device=dev), torch.empty(0, device=dev)
    dw, db = torch.full((64,), 3.0, device=dev), torch.full((64,), 3.0, device=dev)
    ws = torch.empty(256, dtype=torch.uint8, device=dev)
    m.add_layer_norm_bwd(e, e, none, none, torch.ones(64, device=dev), dh=e, dw=dw, db=db, ws=ws)
    assert (dw == 0).all() and (db == 0).all()


def test_forward_and_backward_against_differences(moe_gpu):
    """A loss through the forward kernel, its slope along a direction against the
    backward kernel's gradients (fp32, dropout included)."""
    m, dev = moe_gpu
    rng = np.random.default_rng(6)
    rows, d, p, seed = 9, 200, 0.2, 77
    x, res, dy, dres, vx, vr = (normal(rng, (rows, d), torch.float32, dev) for _ in range(6))
    w, b, vw, vb = (normal(rng, (d,), torch.float32, dev) for _ in range(4))

    def forward(t):
        h, y, mu, r = torch.empty_like(res), torch.empty_like(x), torch.empty(rows, device=dev), torch.empty(rows, device=dev)
        m.add_layer_norm(x + t * vx, w + t * vw, b + t * vb, y, residual=res + t * vr, h=h, mean=mu, rstd=r, p=p, seed=seed)
        return h, y, mu, r

    def loss(t):
        h, y, _, _ = forward(t)
        return ((y.double() * dy).sum() + (h.double() * dres).sum()).item()

    h, _, mu, r = forward(0.0)
    dh, dx, dw, db = torch.empty_like(h), torch.empty_like(x), torch.empty(d, device=dev), torch.empty(d, device=dev)
    ws = torch.empty(m.add_layer_norm_bwd_workspace(rows, d), dtype=torch.uint8, device=dev)
    m.add_layer_norm_bwd(dy, h, mu, r, w, dres, dh, dx, dw, db, ws, p=p, seed=seed)
    slope = sum((a.double() * v).sum().item() for a, v in ((dx, vx), (dh, vr), (dw, vw), (db, vb)))
    step = 2.0 ** -7
    # the difference is off by the third derivative's share (step^2) and by rounding (1e-7 / step)
    assert abs((loss(step) - loss(-step)) / (2 * step) - slope) <= 5e-3 * max(abs(slope), np.sqrt(rows * d))


# ------------------------------------------------------------------ use
def test_rows_past_32_bits(moe_gpu):
    m, dev = moe_gpu
    ld, cols = (1 << 31) + 8, 40
    big = torch.empty(2 * ld + cols, dtype=torch.bfloat16, device=dev)
    x = torch.as_strided(big, (3, cols), (ld, 1))
    vals = normal(np.random.default_rng(0), (3, cols), torch.bfloat16, dev)
    x.copy_(vals)
    w = torch.ones(cols, dtype=torch.bfloat16, device=dev)
    y, z = torch.empty_like(vals), torch.empty_like(vals)
    mean, rstd = torch.empty(3, device=dev), torch.empty(3, device=dev)
    m.add_layer_norm(x, w, w, y, mean=mean, rstd=rstd)
    m.add_layer_norm(vals, w, w, z)
    assert torch.equal(y, z)
    m.add_layer_norm_bwd(vals, vals, mean, rstd, w, dx=y)
    m.add_layer_norm_bwd(x, x, mean, rstd, w, dx=x)   # written there, too
    assert torch.equal(x, y)


def test_refused_tensors(moe_gpu):
    m, dev = moe_gpu
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev), torch.ones(64, dtype=torch.bfloat16, device=dev)
    one = torch.ones(4, device=dev)
    errors = (ValueError, TypeError, m.MoEError)
    for bad in (x[:3], torch.zeros(4, 65, dtype=torch.bfloat16, device=dev), x.float(), x.t().contiguous().t(), x.cpu(),
                x[:1].expand(4, 64)):
        with pytest.raises(errors):
            m.add_layer_norm(x, w, w, bad)
        with pytest.raises(errors):
            m.add_layer_norm_bwd(x, bad, one, one, w, dh=torch.zeros_like(x))
    for bad in (dict(bias=w[:32]), dict(bias=w.float()), dict(mean=one[:3]), dict(mean=one.half()), dict(residual=x)):
        with pytest.raises(errors):
            m.add_layer_norm(x, w, **{**dict(bias=w, y=torch.zeros_like(x)), **bad})
    for bad in (dict(mean=None), dict(db=one), dict(ws=torch.empty(16, dtype=torch.uint8, device=dev)), dict(ws=None)):
        with pytest.raises(errors):
            m.add_layer_norm_bwd(x, x, **{**dict(mean=one, rstd=one, weight=w, db=torch.zeros(64, device=dev),
                                                 ws=torch.empty(4096, dtype=torch.uint8, device=dev)), **bad})


def test_another_stream_and_graph(moe_gpu):
    m, dev = moe_gpu
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        check_forward(m, dev, 33, 1000, "bf16", "f32", "bf16", p=0.1)
    check_backward(m, dev, 33, 1000, "bf16", "f32", "bf16", p=0.1, stream=torch.cuda.current_stream())
    rng = np.random.default_rng(9)
    rows, d = 64, 512
    x, res, dy = (normal(rng, (rows, d), torch.bfloat16, dev) for _ in range(3))
    w, b = normal(rng, (d,), torch.bfloat16, dev), normal(rng, (d,), torch.bfloat16, dev)
    ws = torch.empty(m.add_layer_norm_bwd_workspace(rows, d), dtype=torch.uint8, device=dev)

    def step(o):
        m.add_layer_norm(x, w, b, o[0], residual=res, h=o[1], mean=o[2], rstd=o[3], p=0.1, seed=4)
        m.add_layer_norm_bwd(dy, o[1], o[2], o[3], w, dh=o[4], dx=o[5], dw=o[6], db=o[7], ws=ws, p=0.1, seed=4)

    def outputs():
        return [torch.empty(s, dtype=t, device=dev) for s, t in
                (((rows, d), torch.bfloat16),) * 2 + (((rows,), torch.float32),) * 2 + (((rows, d), torch.bfloat16),) * 2
                + (((d,), torch.float32),) * 2]

    a, c = outputs(), outputs()
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for seed in (1, 2):
        x.copy_(normal(np.random.default_rng(seed), (rows, d), torch.bfloat16, dev))
        graph.replay()
        step(c)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(a, c))
