"""Residual addition + RMS norm (forward, backward, 8-bit output) and dropout on
the GPU against the float64 oracle.

Tolerances: a stored value is off by at most half a step of its type (`half`),
fp32 intermediates by REL relative to the terms that enter them: a row's sum of
squares is taken by at most 32 sequential and 10 tree additions, 42 roundings of
2^-24, which the square root halves; the products add a few.  REL = 2^-18 is
64 roundings.  GPU only."""
import numpy as np
import pytest
import torch

from gpu_util import f64, sf_unpack
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu
REL = 2.0 ** -18
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def half(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half of the smallest step of a type."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def close(got, want, dtype, terms):
    """got (stored in dtype) against want, fp32 work on terms of size `terms`."""
    got, want = f64(got), np.asarray(want)
    err = np.abs(got - want)
    lim = half(dtype) * np.abs(want) + REL * (1 + 2 * half(dtype)) * terms + tiny(dtype)
    assert np.isfinite(got).all()
    assert (err <= lim).all(), f"worst {np.max(err / lim):.3f} of the limit at {np.unravel_index(np.argmax(err / lim), err.shape)}"


def normal(rng, shape, dtype, dev, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(dtype).to(dev)


def strided(t, extra, shift=0):
    """The same matrix with `extra` more columns of NaN between its rows."""
    big = torch.full((t.shape[0], t.shape[1] + extra + shift), float("nan"), dtype=t.dtype, device=t.device)
    v = big[:, shift:shift + t.shape[1]]
    v.copy_(t)
    return v


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 31), (2, 33), (130, 64), (257, 128), (7, 250), (3, 256), (65, 1000), (9, 1001),
          (33, 2048), (4, 4096), (3, 5000), (2, 8192), (2, 9000), (1, 16385), (2, 32768)]
TYPES = [("bf16", "bf16", "bf16"), ("bf16", "f32", "bf16"), ("bf16", "bf16", "f32"), ("f16", "f16", "f16"),
         ("f16", "f32", "f32"), ("f32", "f32", "f32")]


def check_forward(m, dev, rows, d, xt, rt, wt, p=0.0, residual=True, layout=lambda t: t, eps=1e-5, stream=None):
    rng = np.random.default_rng(rows * 131 + d)
    x = layout(normal(rng, (rows, d), DT[xt], dev))
    res = layout(normal(rng, (rows, d), DT[rt], dev, 2.0)) if residual else None
    w = normal(rng, (d,), DT[wt], dev)
    y, h = layout(torch.zeros(rows, d, dtype=DT[xt], device=dev)), None
    if residual or p:
        h = layout(torch.zeros(rows, d, dtype=DT[rt], device=dev))
    rstd = torch.empty(rows, device=dev)
    seed, offset = 0x1234567890ABCDEF, (7 << 32) + 9
    m.add_norm(x, w, y, residual=res, h=h, rstd=rstd, eps=eps, p=p, seed=seed, offset=offset, stream=stream)
    torch.cuda.synchronize()
    drop = B.dropout(f64(x), p, seed, offset)
    if h is not None:
        want = drop + (f64(res) if residual else 0)
        close(h, want, h.dtype, np.abs(drop) + (np.abs(f64(res)) if residual else 0))
    hd = f64(h) if h is not None else f64(x)   # the norm is that of the stored stream
    want_r = 1 / np.sqrt((hd * hd).mean(-1) + eps)
    assert (np.abs(f64(rstd) - want_r) <= REL * want_r).all()
    want_y = hd * want_r[:, None] * f64(w)
    close(y, want_y, y.dtype, np.abs(want_y))
    return x, res, w, h, y, rstd


@pytest.mark.parametrize("rows,d", SHAPES, ids=str)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_forward(moe_gpu, rows, d, types):
    m, dev = moe_gpu
    check_forward(m, dev, rows, d, *types)


@pytest.mark.parametrize("rows,d", [(5, 31), (3, 256), (65, 1000), (9, 1001), (2, 9000)], ids=str)
@pytest.mark.parametrize("types", [TYPES[0], TYPES[1], TYPES[4], TYPES[5]], ids="-".join)
@pytest.mark.parametrize("residual", [True, False], ids=["res", "nores"])
def test_forward_with_dropout(moe_gpu, rows, d, types, residual):
    m, dev = moe_gpu
    check_forward(m, dev, rows, d, *types, p=0.3, residual=residual)


@pytest.mark.parametrize("rows,d", [(1, 1), (5, 31), (65, 1000), (3, 2048)], ids=str)
@pytest.mark.parametrize("types", [TYPES[0], TYPES[3], TYPES[5]], ids="-".join)
def test_forward_without_residual(moe_gpu, rows, d, types):
    m, dev = moe_gpu
    check_forward(m, dev, rows, d, *types, residual=False)


@pytest.mark.parametrize("extra,shift", [(8, 0), (64, 0), (1, 0), (3, 0), (8, 8), (5, 3), (0, 1)], ids=str)
@pytest.mark.parametrize("d", [64, 77, 2048])
def test_forward_strides_and_alignment(moe_gpu, extra, shift, d):
    m, dev = moe_gpu
    check_forward(m, dev, 9, d, "bf16", "f32", "bf16", p=0.2, layout=lambda t: strided(t, extra, shift))


def test_forward_writes_its_rows_alone(moe_gpu):
    m, dev = moe_gpu
    out = check_forward(m, dev, 6, 77, "f16", "f16", "f16", layout=lambda t: strided(t, 11, 2))
    for v in (out[3], out[4]):   # what lies between the rows keeps its NaN
        big = torch.as_strided(v, (6, 90), (90, 1), 0)
        assert torch.isnan(big[:, :2]).all() and torch.isnan(big[:, 79:]).all()


def test_forward_in_place(moe_gpu):
    """h in the residual's buffer and y in that of x: the same bits."""
    m, dev = moe_gpu
    for d in (1001, 2048):
        x, res, w, h, y, _ = check_forward(m, dev, 12, d, "bf16", "bf16", "bf16", p=0.25)
        m.add_norm(x, w, x, residual=res, h=res, p=0.25, seed=0x1234567890ABCDEF, offset=(7 << 32) + 9)
        assert torch.equal(res, h) and torch.equal(x, y)


def test_forward_extreme_rows(moe_gpu):
    """A zero row (eps alone), an infinity, a NaN, large and tiny values; the
    rows beside them keep their values."""
    m, dev = moe_gpu
    rng = np.random.default_rng(1)
    d = 256
    x = normal(rng, (6, d), torch.float32, dev)
    x[0] = 0
    x[1, 5] = float("inf")
    x[2, 9] = float("nan")
    x[3] *= 1e18
    x[4] *= 1e-30
    w = torch.ones(d, device=dev)
    y, rstd = torch.empty_like(x), torch.empty(6, device=dev)
    m.add_norm(x, w, y, rstd=rstd, eps=1e-6)
    assert torch.equal(y[0], torch.zeros(d, device=dev)) and abs(rstd[0].item() - 1e3) < 1e-2
    assert rstd[1].item() == 0 and torch.isnan(y[1, 5]) and (y[1, :5] == 0).all()
    assert torch.isnan(y[2]).all()
    for r, e in ((3, 1e-6), (4, 1e-6), (5, 1e-6)):
        v = f64(x[r])
        want = v / np.sqrt((v * v).mean() + e)
        assert (np.abs(f64(y[r]) - want) <= 2 * REL * np.abs(want) + 1e-37).all()
    m.add_norm(x[:1], w, y[:1], eps=0.0)   # 0 / 0 of a zero row without eps
    assert torch.isnan(y[0]).all()


# ------------------------------------------------------------------ 8-bit output
def e4m3_step(z):
    """Distance of neighbouring E4M3 values at |z| (2^-9 among the subnormals)."""
    return np.exp2(np.maximum(np.floor(np.log2(np.maximum(np.abs(z), 2.0 ** -6))), -6) - 3)


@pytest.mark.parametrize("rows,d", [(1, 128), (3, 256), (127, 128), (128, 384), (129, 1408), (70, 2048), (2, 4096),
                                    (5, 16384)], ids=str)
@pytest.mark.parametrize("rt,wt,p", [("bf16", "bf16", 0.0), ("f32", "f32", 0.1)])
@pytest.mark.parametrize("with_dq", [True, False], ids=["dq", "nodq"])
def test_forward_mxfp8(moe_gpu, rows, d, rt, wt, p, with_dq):
    m, dev = moe_gpu
    rng = np.random.default_rng(rows + d)
    x, res = normal(rng, (rows, d), torch.bfloat16, dev), normal(rng, (rows, d), DT[rt], dev)
    # columns of very different sizes, an all-zero block: every kind of scale
    w = normal(rng, (d,), DT[wt], dev) * torch.exp2(torch.randint(-12, 12, (d,), device=dev).float()).to(DT[wt])
    w[32:64] = 0
    pad = (rows + 127) // 128 * 128
    q = torch.full((pad, d), 0x55, dtype=torch.uint8, device=dev)
    sc = torch.full((pad * d // 32,), 0x55, dtype=torch.uint8, device=dev)
    dq = torch.full((pad, d), 7.0, dtype=torch.bfloat16, device=dev) if with_dq else None
    h, rstd = torch.empty(rows, d, dtype=DT[rt], device=dev), torch.empty(rows, device=dev)
    m.add_norm(x, w, None, residual=res, h=h, rstd=rstd, p=p, seed=5, offset=1, y_q=q, y_scales=sc, y_dq=dq)
    drop = B.dropout(f64(x), p, 5, 1)
    close(h, drop + f64(res), h.dtype, np.abs(drop) + np.abs(f64(res)))
    out = torch.empty(pad, d, dtype=torch.bfloat16, device=dev)
    m.dequantize_mxfp8(pad, d, q, sc, out)
    if with_dq:
        assert torch.equal(out.view(torch.int16), dq.view(torch.int16))
    assert (q[rows:] == 0).all() and (out[rows:] == 0).all()
    scales = sf_unpack(sc.cpu().numpy(), pad, d // 32).astype(np.int64) - 127
    assert (scales[rows:] == 0).all()
    y = f64(h) * f64(rstd)[:, None] * f64(w)
    top = np.abs(y.reshape(rows, -1, 32)).max(-1)
    s = scales[:rows]
    lim = 448 * np.exp2(s)
    zero = top == 0
    assert (s[zero] == 0).all()
    assert (top <= lim * (1 + 2 * REL))[~zero].all() and (top > lim / 2 * (1 - 2 * REL))[~zero].all()
    unit = np.repeat(np.exp2(s), 32, axis=1)
    err = np.abs(f64(out[:rows]) - y) / unit
    z = np.minimum(np.abs(y) / unit, 448)
    assert (err <= e4m3_step(z) / 2 + 4 * REL * z).all()


def test_mxfp8_output_feeds_the_grouped_gemm(moe_gpu):
    """The codes as they are: one expert's SwiGLU on them equals that on the same
    rows quantised by moe_quantize_mxfp8 from the dequantised values."""
    m, dev = moe_gpu
    rng = np.random.default_rng(8)
    T, d, f = 200, 256, 256
    s = m.shape(T, d, 1, 1, f, prec=m.MXFP8)
    n = m.rows_max(s)
    x, w = normal(rng, (T, d), torch.bfloat16, dev), normal(rng, (d,), torch.bfloat16, dev)
    q = torch.zeros(n, d, dtype=torch.uint8, device=dev)
    sc = torch.full((n * d // 32,), 127, dtype=torch.uint8, device=dev)
    dq = torch.zeros(n, d, dtype=torch.bfloat16, device=dev)
    m.add_norm(x, w, None, y_q=q, y_scales=sc, y_dq=dq)
    q2, sc2 = torch.empty_like(q), torch.empty_like(sc)
    m.quantize_mxfp8(1, n, d, 1, dq, q2, sc2)
    buf = m.allocate(s, with_grads=False)
    wg, wu = (normal(rng, (1, f, d), torch.bfloat16, dev, 0.05) for _ in range(2))
    m.build_mx_weights(s, wg, wu, normal(rng, (1, d, f), torch.bfloat16, dev, 0.05), buf.mx_weights)
    tiles = torch.tensor([0, (T + 127) // 128], dtype=torch.int32, device=dev)
    got = []
    for codes, scales in ((q, sc), (q2, sc2)):
        h, u = (torch.zeros(n, f, dtype=torch.bfloat16, device=dev) for _ in range(2))
        m.grouped_gemm(s, m.GEMM_FWD1_SWIGLU, buf.ws, tile_offsets=tiles, a0=codes, sfa0=scales,
                       w0=buf.mx_weights["gu_q"], sfb0=buf.mx_weights["gu_s"], out0=h, out1=u,
                       out2=buf.mx["a_q"], osf0=buf.mx["a_s"])
        got.append((h[:T].clone(), u[:T].clone()))
    assert m.read_error(buf.ws) == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)
    want = f64(dq[:T]) @ f64(wg[0]).T
    assert np.abs(f64(got[0][0]) - want).max() <= 6e-2 * np.abs(want).max()


# ------------------------------------------------------------------ backward
def check_backward(m, dev, rows, d, xt, rt, wt, p=0.0, with_dres=True, layout=lambda t: t, outs=("dh", "dx", "dw"),
                   stream=None):
    rng = np.random.default_rng(rows * 17 + d)
    dy = layout(normal(rng, (rows, d), DT[xt], dev))
    h = layout(normal(rng, (rows, d), DT[rt], dev, 2.0))
    dres = layout(normal(rng, (rows, d), DT[rt], dev)) if with_dres else None
    w = normal(rng, (d,), DT[wt], dev)
    rstd = torch.from_numpy(1 / np.sqrt((f64(h) ** 2).mean(-1) + 1e-5)).float().to(dev)
    o = {"dh": layout(torch.zeros(rows, d, dtype=DT[rt], device=dev)),
         "dx": layout(torch.zeros(rows, d, dtype=DT[xt], device=dev)),
         "dw": torch.full((d,), 9.0, device=dev)}
    o = {n: v for n, v in o.items() if n in outs}
    ws = torch.full((m.add_norm_bwd_workspace(rows, d),), 0xA5, dtype=torch.uint8, device=dev)
    seed, offset = 0xFEDCBA9876543210, 3
    m.add_norm_bwd(dy, h, rstd, w, dres=dres, ws=ws, p=p, seed=seed, offset=offset, stream=stream, **o)
    torch.cuda.synchronize()
    a = [f64(t) if t is not None else None for t in (dy, h, rstd, w, dres)]
    dh, dx, dw = B.add_norm_bwd(*a, p, seed, offset)
    g, r = a[0] * a[3], a[2][:, None]
    # the row's mean of g h is off by REL of the mean of |g h|
    terms = r * np.abs(g) + np.abs(a[1]) * r ** 3 * np.abs(g * a[1]).mean(-1, keepdims=True)
    terms = terms + (np.abs(a[4]) if with_dres else 0)
    if "dh" in o:
        close(o["dh"], dh, DT[rt], terms)
    if "dx" in o:
        close(o["dx"], dx, DT[xt], B.dropout(terms, p, seed, offset))
    if "dw" in o:
        lim = (rows + 64) * 2.0 ** -24 * np.abs(a[0] * a[1] * r).sum(0) + 1e-37
        assert (np.abs(f64(o["dw"]) - dw) <= lim).all()
    return o


@pytest.mark.parametrize("rows,d", SHAPES, ids=str)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
def test_backward(moe_gpu, rows, d, types):
    m, dev = moe_gpu
    check_backward(m, dev, rows, d, *types)


@pytest.mark.parametrize("rows,d", [(5, 31), (3, 256), (65, 1000), (9, 1001), (2, 9000), (3000, 64), (2500, 1024)],
                         ids=str)
@pytest.mark.parametrize("types", [TYPES[0], TYPES[1], TYPES[4], TYPES[5]], ids="-".join)
@pytest.mark.parametrize("with_dres", [True, False], ids=["dres", "nodres"])
def test_backward_with_dropout(moe_gpu, rows, d, types, with_dres):
    m, dev = moe_gpu
    check_backward(m, dev, rows, d, *types, p=0.3, with_dres=with_dres)


@pytest.mark.parametrize("outs", [("dh",), ("dx",), ("dw",), ("dh", "dx"), ("dx", "dw")], ids="-".join)
@pytest.mark.parametrize("d", [77, 512])
def test_backward_of_some_outputs(moe_gpu, outs, d):
    m, dev = moe_gpu
    check_backward(m, dev, 40, d, "bf16", "f32", "f32", p=0.1, outs=outs)


@pytest.mark.parametrize("extra,shift", [(8, 0), (1, 0), (8, 8), (5, 3)], ids=str)
@pytest.mark.parametrize("d", [64, 77, 2048])
def test_backward_strides_and_alignment(moe_gpu, extra, shift, d):
    m, dev = moe_gpu
    check_backward(m, dev, 9, d, "bf16", "bf16", "bf16", p=0.2, layout=lambda t: strided(t, extra, shift))


def test_backward_is_deterministic_and_in_place(moe_gpu):
    m, dev = moe_gpu
    rng = np.random.default_rng(2)
    rows, d = 3000, 1001
    for d in (1001, 1024):
        dy, h, dres = (normal(rng, (rows, d), torch.bfloat16, dev) for _ in range(3))
        w, rstd = normal(rng, (d,), torch.bfloat16, dev), torch.rand(rows, device=dev)
        ws = torch.empty(m.add_norm_bwd_workspace(rows, d), dtype=torch.uint8, device=dev)
        first = None
        for _ in range(3):
            dh, dx, dw = torch.empty_like(h), torch.empty_like(dy), torch.empty(d, device=dev)
            m.add_norm_bwd(dy, h, rstd, w, dres=dres, dh=dh, dx=dx, dw=dw, ws=ws, p=0.1, seed=1)
            first = first or (dh, dx, dw)
            assert all(torch.equal(a, b) for a, b in zip(first, (dh, dx, dw)))
        m.add_norm_bwd(dy, h, rstd, w, dres=dres, dh=dres, dx=dy, dw=dw, ws=ws, p=0.1, seed=1)
        assert torch.equal(dres, first[0]) and torch.equal(dy, first[1]) and torch.equal(dw, first[2])


def test_backward_without_rows(moe_gpu):
    m, dev = moe_gpu
    e = torch.empty(0, 64, device=dev)
    dw = torch.full((64,), 3.0, device=dev)
    ws = torch.empty(m.add_norm_bwd_workspace(0, 64) + 256, dtype=torch.uint8, device=dev)
    m.add_norm_bwd(e, e, torch.empty(0, device=dev), torch.ones(64, device=dev), dh=e, dw=dw, ws=ws)
    assert (dw == 0).all()


def test_forward_and_backward_against_differences(moe_gpu):
    """A loss through the forward kernel, its slope along a direction against the
    backward kernel's gradients (fp32, dropout included)."""
    m, dev = moe_gpu
    rng = np.random.default_rng(6)
    rows, d, p, seed = 9, 200, 0.2, 77
    x, res = (normal(rng, (rows, d), torch.float32, dev) for _ in range(2))
    w, dy, dres = (normal(rng, s, torch.float32, dev) for s in ((d,), (rows, d), (rows, d)))
    vx, vr, vw = (normal(rng, s, torch.float32, dev) for s in ((rows, d), (rows, d), (d,)))

    def forward(x, res, w):
        h, y, r = torch.empty_like(res), torch.empty_like(x), torch.empty(rows, device=dev)
        m.add_norm(x, w, y, residual=res, h=h, rstd=r, p=p, seed=seed)
        return h, y, r

    def loss(t):
        h, y, _ = forward(x + t * vx, res + t * vr, w + t * vw)
        return ((y.double() * dy).sum() + (h.double() * dres).sum()).item()

    h, _, r = forward(x, res, w)
    dh, dx, dw = torch.empty_like(h), torch.empty_like(x), torch.empty(d, device=dev)
    ws = torch.empty(m.add_norm_bwd_workspace(rows, d), dtype=torch.uint8, device=dev)
    m.add_norm_bwd(dy, h, r, w, dres=dres, dh=dh, dx=dx, dw=dw, ws=ws, p=p, seed=seed)
    slope = ((dx.double() * vx).sum() + (dh.double() * vr).sum() + (dw.double() * vw).sum()).item()
    step = 2.0 ** -7
    # the difference is off by the third derivative's share (step^2) and by rounding (1e-7 / step)
    assert abs((loss(step) - loss(-step)) / (2 * step) - slope) <= 5e-3 * max(abs(slope), np.sqrt(rows * d))


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 5), (3, 8), (17, 129), (1000, 24), (5, 1001), (2, 70000), (9, 2048)],
                         ids=str)
@pytest.mark.parametrize("dt", list(DT))
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999, 1.0])
def test_dropout(moe_gpu, rows, cols, dt, p):
    m, dev = moe_gpu
    rng = np.random.default_rng(cols)
    x = normal(rng, (rows, cols), DT[dt], dev)
    y = torch.empty_like(x)
    seed, offset = 0xABCDEF0123456789, (1 << 40) + 3
    m.dropout(x, y, p, seed, offset)
    want = B.dropout(f64(x), p, seed, offset)
    got = f64(y)
    big = torch.finfo(DT[dt]).max
    fits = np.abs(want) < big     # fp16 at p = 0.999: values past its range become infinite
    # one fp32 product with a rounded scale, then the store
    assert (np.abs(got - want)[fits] <= (half(DT[dt]) * np.abs(want) + 2.0 ** -22 * np.abs(want) + tiny(DT[dt]))[fits]).all()
    assert ((got == 0) == (want == 0)).all()
    z = x.clone()
    m.dropout(z, z, p, seed, offset)   # in place
    assert torch.equal(z, y)


@pytest.mark.parametrize("extra,shift", [(8, 0), (1, 0), (5, 3)], ids=str)
def test_dropout_mask_is_of_the_place_alone(moe_gpu, extra, shift):
    """Strides, alignment and type do not enter the mask, and the norm's fused
    dropout has the same."""
    m, dev = moe_gpu
    x = torch.ones(37, 203, device=dev)
    y = torch.empty_like(x)
    m.dropout(x, y, 0.4, 9, 2)
    for dt in DT.values():
        a = strided(x.to(dt), extra, shift)
        b = strided(torch.zeros_like(x).to(dt), extra, shift)
        m.dropout(a, b, 0.4, 9, 2)
        assert torch.equal(b != 0, y != 0)
        h, n = torch.empty_like(b), torch.empty_like(b)
        m.add_norm(a, torch.ones(203, dtype=dt, device=dev), n, h=h, p=0.4, seed=9, offset=2)
        assert torch.equal(h != 0, y != 0)


def test_dropout_of_nan_and_infinity(moe_gpu):
    m, dev = moe_gpu
    x = torch.full((8, 512), float("nan"), device=dev)
    x[4:] = float("inf")
    y = torch.empty_like(x)
    m.dropout(x, y, 0.5, 4)
    keep = torch.from_numpy(B.keep_mask(8, 512, 0.5, 4, 0)).to(dev)
    assert torch.isnan(y[:4][keep[:4]]).all() and torch.isinf(y[4:][keep[4:]]).all()
    assert (y[~keep] == 0).all()


def test_rows_past_32_bits(moe_gpu):
    """Rows that start more than 2^32 elements into their buffer."""
    m, dev = moe_gpu
    ld, cols = (1 << 31) + 8, 40
    big = torch.empty(2 * ld + cols, dtype=torch.bfloat16, device=dev)
    x = torch.as_strided(big, (3, cols), (ld, 1))
    vals = normal(np.random.default_rng(0), (3, cols), torch.bfloat16, dev)
    x.copy_(vals)
    y = torch.empty(3, cols, dtype=torch.bfloat16, device=dev)
    w = torch.ones(cols, dtype=torch.bfloat16, device=dev)
    a, b = torch.empty_like(y), torch.empty_like(y)
    m.dropout(x, y, 0.3, 1)
    m.dropout(vals, a, 0.3, 1)
    assert torch.equal(y, a)
    m.add_norm(x, w, y)
    m.add_norm(vals, w, b)
    assert torch.equal(y, b)
    m.dropout(vals, x, 0.3, 1)   # written there, too
    assert torch.equal(x, a)


def test_many_rows(moe_gpu):
    """More rows than any grid dimension but the first can count."""
    m, dev = moe_gpu
    rows = 600_011
    x = torch.ones(rows, 8, dtype=torch.bfloat16, device=dev)
    x[:, 3] = torch.arange(rows, device=dev).remainder(7).to(torch.bfloat16)
    y, z = torch.empty_like(x), torch.empty_like(x)
    w = torch.ones(8, dtype=torch.bfloat16, device=dev)
    m.add_norm(x, w, y)
    v = x.double()
    want = v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-5)
    assert ((y.double() - want).abs() <= (2.0 ** -8 + REL) * want.abs()).all()
    m.dropout(x, z, 0.5, 3)
    last = B.keep_mask(rows, 8, 0.5, 3, 0)
    assert torch.equal(z != 0, torch.from_numpy(last).to(dev) & (x != 0))


# ------------------------------------------------------------------ use
def test_refused_tensors(moe_gpu):
    m, dev = moe_gpu
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16, device=dev), torch.ones(64, dtype=torch.bfloat16, device=dev)
    y = torch.zeros_like(x)
    for bad in (x[:3], torch.zeros(4, 65, dtype=torch.bfloat16, device=dev), x.float(), x.t().contiguous().t(), x.cpu(),
                x[:1].expand(4, 64)):
        with pytest.raises((ValueError, TypeError, m.MoEError)):
            m.add_norm(x, w, bad)
        with pytest.raises((ValueError, TypeError, m.MoEError)):
            m.dropout(x, bad, 0.1, 0)
        with pytest.raises((ValueError, TypeError, m.MoEError)):
            m.add_norm_bwd(x, bad, torch.ones(4, device=dev), w, dh=y)
    with pytest.raises(ValueError):
        m.add_norm(x, w[:32], y)
    with pytest.raises(m.MoEError):
        m.add_norm(x, w, y, residual=x)   # a residual without a place for the stream
    with pytest.raises((ValueError, m.MoEError)):   # workspace too small
        m.add_norm_bwd(x, x, torch.ones(4, device=dev), w, dw=torch.empty(64, device=dev),
                       ws=torch.empty(16, dtype=torch.uint8, device=dev))
    with pytest.raises((ValueError, m.MoEError)):   # 8-bit buffers without the last tile's padding
        m.add_norm(x.repeat(1, 2), w.repeat(2), None, y_q=torch.zeros(4, 128, dtype=torch.uint8, device=dev),
                   y_scales=torch.zeros(512, dtype=torch.uint8, device=dev))


def test_another_stream_and_graph(moe_gpu):
    """On a stream of its own, and captured in a graph that is replayed on new inputs."""
    m, dev = moe_gpu
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        check_forward(m, dev, 33, 1000, "bf16", "f32", "bf16", p=0.1)
    check_backward(m, dev, 33, 1000, "bf16", "f32", "bf16", p=0.1, stream=torch.cuda.current_stream())
    rng = np.random.default_rng(9)
    rows, d = 64, 512
    x, res, dy = (normal(rng, (rows, d), torch.bfloat16, dev) for _ in range(3))
    w = normal(rng, (d,), torch.bfloat16, dev)
    ws = torch.empty(m.add_norm_bwd_workspace(rows, d), dtype=torch.uint8, device=dev)

    def step(o):
        m.add_norm(x, w, o[0], residual=res, h=o[1], rstd=o[2], p=0.1, seed=4)
        m.add_norm_bwd(dy, o[1], o[2], w, dh=o[3], dx=o[4], dw=o[5], ws=ws, p=0.1, seed=4)
        m.dropout(o[0], o[6], 0.5, 8)

    def outputs():
        return [torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device=dev), torch.empty_like(x),
                torch.empty_like(x), torch.empty(d, device=dev), torch.empty_like(x)]

    a, b = outputs(), outputs()
    step(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(a)
    for seed in (1, 2):
        x.copy_(normal(np.random.default_rng(seed), (rows, d), torch.bfloat16, dev))
        graph.replay()
        step(b)
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(a, b))
