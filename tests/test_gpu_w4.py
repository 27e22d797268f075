"""4-bit weights on the GPU: quantiser, products with a few vectors and the
SwiGLU experts, against the float64 oracle.

Tolerances: products of a 16-column step are added to an fp32 sum by the tensor
core, which may truncate (2^-23 a step); a K-long sum has K/16 such steps and at
most 32 more additions (groups, warps), so it is off by ACC(K) of the sum of the
terms' sizes.  A stored result is off by half a step of its type.  GPU only."""
import numpy as np
import pytest
import torch

from gpu_util import f64
from oracle import block_oracle as B

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f16": torch.float16}


def acc(K):
    return (K / 8 + 64) * 2.0 ** -23


def half(dtype):
    return torch.finfo(dtype).eps / 2


def normal(rng, shape, dtype, dev, scale=1.0):
    return torch.from_numpy(rng.standard_normal(shape) * scale).to(dtype).to(dev)


def weights(m, rng, shape, group, dtype, dev, scale=0.05):
    """Random codes and scales (every code, both signs, zero scales among them)
    and the float64 values that they stand for."""
    codes = rng.integers(0, 16, shape).astype(np.uint8)
    s = torch.from_numpy(np.abs(rng.standard_normal((*shape[:-1], shape[-1] // group))) * scale).to(dtype)
    s.view(-1)[::7] = 0
    q = torch.from_numpy(B.w4_pack(codes)).to(dev)
    return q, s.to(dev), B.w4_values(codes, f64(s))


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("rows,K", [(1, 128), (3, 256), (17, 128), (64, 1408), (5, 4096)], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", list(DT))
def test_quantize(moe_gpu, rows, K, group, dt):
    m, dev = moe_gpu
    rng = np.random.default_rng(K + rows)
    w = rng.standard_normal((rows, K)) * 0.02 * np.exp2(rng.integers(-4, 4, (rows, K)))
    w[0, :group] = 0
    w[-1, -1] = -0.0
    w = torch.from_numpy(w).to(DT[dt]).to(dev)
    q = torch.empty(rows, K // 2, dtype=torch.uint8, device=dev)
    s = torch.empty(rows, K // group, dtype=DT[dt], device=dev)
    m.quantize_w4(w, q, s)
    top = np.abs(f64(w).reshape(rows, -1, group)).max(-1) / 7
    tiny = torch.finfo(DT[dt]).smallest_normal * torch.finfo(DT[dt]).eps / 2
    assert (np.abs(f64(s) - top) <= (half(DT[dt]) + 2.0 ** -23) * top + tiny).all()
    # codes from the stored scales: exact but where w / s lies next to a border
    b, sv = f64(w).reshape(rows, -1, group), f64(s)[..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        z = np.where(sv > 0, b / sv, 0.0)
    packed = q.cpu().numpy()
    codes = np.stack([packed & 15, packed >> 4], -1).reshape(b.shape).astype(int) - 8
    assert (np.abs(codes - np.clip(z, -8, 7)) <= 0.5 + 2.0 ** -20).all()
    assert (codes[0, 0] == 0).all() and f64(s)[0, 0] == 0
    out = torch.empty(rows, K, device=dev)
    m.dequantize_w4(q, s, out)
    assert np.array_equal(f64(out), (codes * sv).reshape(rows, K))


# ------------------------------------------------------------------ matvec
def check_matvec(m, dev, M, N, K, group, dt, x=None, y=None):
    rng = np.random.default_rng(M * 7 + N + K)
    dtype = DT[dt]
    q, s, w = weights(m, rng, (N, K), group, dtype, dev)
    vals = normal(rng, (M, K), dtype, dev)
    x = vals if x is None else x(vals)
    y = torch.full((M, N), 9.0, dtype=dtype, device=dev) if y is None else y
    m.matvec_w4(x, q, s, y)
    want = f64(vals) @ w.T
    lim = half(dtype) * np.abs(want) + 1.01 * acc(K) * (np.abs(f64(vals)) @ np.abs(w).T)
    lim = lim + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    assert (np.abs(f64(y) - want) <= lim).all()


@pytest.mark.parametrize("M", [1, 2, 7, 8, 9, 16, 17, 32, 33, 70])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", list(DT))
def test_matvec_vectors(moe_gpu, M, group, dt):
    m, dev = moe_gpu
    check_matvec(m, dev, M, 200, 640, group, dt)


@pytest.mark.parametrize("N,K", [(1, 128), (15, 128), (16, 256), (17, 384), (33, 4096), (1000, 896), (2001, 2048),
                                 (3, 16384)], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 3, 12])
def test_matvec_sizes(moe_gpu, N, K, group, M):
    m, dev = moe_gpu
    check_matvec(m, dev, M, N, K, group, "bf16")


@pytest.mark.parametrize("K,group", [(32, 32), (96, 32), (64, 64), (192, 64), (128, 128), (1056, 32)])
def test_matvec_short_and_odd_k(moe_gpu, K, group):
    m, dev = moe_gpu
    check_matvec(m, dev, 2, 50, K, group, "f16")


def test_matvec_strides(moe_gpu):
    m, dev = moe_gpu
    big = torch.full((5, 1000), float("nan"), dtype=torch.bfloat16, device=dev)

    def strided(v):
        big[:, 8:8 + v.shape[1]] = v
        return big[:, 8:8 + v.shape[1]]

    out = torch.full((5, 131), 3.0, dtype=torch.bfloat16, device=dev)
    check_matvec(m, dev, 5, 77, 256, 64, "bf16", x=strided, y=out[:, 1:78])
    assert (out[:, 0] == 3).all() and (out[:, 78:] == 3).all()


def test_matvec_nan_and_infinity_stay_in_their_vector(moe_gpu):
    m, dev = moe_gpu
    rng = np.random.default_rng(3)
    q, s, _ = weights(m, rng, (64, 256), 64, torch.bfloat16, dev)
    x = normal(rng, (11, 256), torch.bfloat16, dev)
    clean, y = torch.empty(11, 64, dtype=torch.bfloat16, device=dev), torch.empty(11, 64, dtype=torch.bfloat16, device=dev)
    m.matvec_w4(x, q, s, clean)
    x[2, 100] = float("nan")
    x[9, 5] = float("inf")
    m.matvec_w4(x, q, s, y)
    keep = [i for i in range(11) if i not in (2, 9)]
    assert torch.equal(y[keep], clean[keep])
    assert torch.isnan(y[2]).all() and not torch.isfinite(y[9]).all()


# ------------------------------------------------------------------ experts
def check_experts(m, dev, T, d, E, k, f, group, dt="bf16", idx=None, gates=None, expect_error=0, seed=0):
    rng = np.random.default_rng(T * 31 + d + E + f + seed)
    dtype = DT[dt]
    x = normal(rng, (T, d), dtype, dev)
    w, val = {}, {}
    for n, shape in (("gate", (E, f, d)), ("up", (E, f, d)), ("down", (E, d, f))):
        w[n + "_q"], w[n + "_s"], val[n] = weights(m, rng, shape, group, dtype, dev, 0.3 / np.sqrt(shape[-1]))
    if idx is None:
        idx = np.argsort(-rng.standard_normal((T, E)), 1)[:, :k]
    if gates is None:
        gates = rng.random((T, k))
    ti = torch.from_numpy(np.ascontiguousarray(idx, dtype=np.int32)).to(dev)
    tg = torch.from_numpy(np.ascontiguousarray(gates)).float().to(dev)
    out = torch.full((T, d), 9.0, dtype=dtype, device=dev)
    ws = torch.full((m.experts_w4_workspace(T, d, E, k, f),), 0xFF, dtype=torch.uint8, device=dev)   # NaN everywhere
    m.clear_error(ws)
    m.experts_w4(x, ti, tg, w, out, ws)
    assert m.read_error(ws) == expect_error
    xs, g = f64(x), f64(tg)
    want = B.experts(xs, idx, g, val["gate"], val["up"], val["down"])
    # errors of both products through the activation, its two bf16 parts (2^-16), the last sum
    size = np.zeros_like(want)
    for t in range(T):
        for j in range(idx.shape[1]):
            e = int(idx[t, j])
            if not 0 <= e < E:
                continue
            h, u = val["gate"][e] @ xs[t], val["up"][e] @ xs[t]
            eh, eu = (acc(d) * (np.abs(val[n][e]) @ np.abs(xs[t])) for n in ("gate", "up"))
            sg = 1 / (1 + np.exp(-h))
            a = np.abs(h * sg * u)
            ea = 1.1 * np.abs(u) * eh + np.abs(h * sg) * eu + (2.0 ** -16 + 2.0 ** -20) * a + eh * eu
            size[t] += abs(g[t, j]) * (np.abs(val["down"][e]) @ (ea + acc(2 * f) * a))
    lim = half(dtype) * np.abs(want) + 1.02 * size + k * 2.0 ** -23 * np.abs(want) + 1e-6
    err = np.abs(f64(out) - want)
    assert (err <= lim).all(), f"{np.max(err / lim)}"
    return x, ti, tg, w, out, ws


@pytest.mark.parametrize("T,d,E,k,f", [
    (1, 128, 1, 1, 128), (1, 256, 8, 2, 384), (1, 1024, 64, 8, 256), (2, 128, 8, 8, 128), (3, 384, 5, 3, 128),
    (4, 256, 16, 4, 256), (5, 256, 16, 4, 256), (8, 128, 4, 2, 128), (9, 128, 4, 2, 128), (17, 256, 2, 1, 128),
    (33, 128, 3, 3, 256), (64, 256, 8, 2, 128), (100, 128, 4, 1, 128), (1, 2048, 32, 4, 1024), (2, 128, 256, 32, 128),
], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_experts(moe_gpu, T, d, E, k, f, group):
    m, dev = moe_gpu
    check_experts(m, dev, T, d, E, k, f, group)


@pytest.mark.parametrize("T", [1, 6, 40])
def test_experts_fp16(moe_gpu, T):
    m, dev = moe_gpu
    check_experts(m, dev, T, 256, 8, 2, 384, 64, "f16")


@pytest.mark.parametrize("T", [1, 3, 20, 1024])
def test_experts_all_routes_to_one(moe_gpu, T):
    m, dev = moe_gpu
    check_experts(m, dev, T, 128, 8, 1, 128, 64, idx=np.full((T, 1), 5))


def test_experts_the_same_expert_twice(moe_gpu):
    m, dev = moe_gpu
    check_experts(m, dev, 3, 128, 8, 3, 128, 64, idx=np.array([[2, 2, 2], [1, 2, 1], [7, 0, 7]]))


def test_experts_places_without_an_expert(moe_gpu):
    """Tokens with some or no experts: zeros for the latter, no error."""
    m, dev = moe_gpu
    for T in (2, 4, 30):
        idx = np.argsort(-np.random.default_rng(T).standard_normal((T, 8)), 1)[:, :4].astype(int)
        idx[0] = -1
        idx[1, 1:] = -1
        out = check_experts(m, dev, T, 256, 8, 4, 128, 32, idx=idx)[4]
        assert (out[0] == 0).all()
    out = check_experts(m, dev, 3, 128, 8, 2, 128, 32, idx=np.full((3, 2), -1))[4]
    assert (out == 0).all()


def test_experts_index_out_of_range_is_reported(moe_gpu):
    m, dev = moe_gpu
    for bad in (8, -2, 1 << 30, -(1 << 31)):
        for T in (2, 20):
            idx = np.argsort(-np.random.default_rng(T).standard_normal((T, 8)), 1)[:, :2].astype(int)
            idx[1, 0] = bad
            check_experts(m, dev, T, 128, 8, 2, 128, 64, idx=idx, expect_error=m.DEVERR_BOUNDS)


def test_experts_gates_of_zero_and_negative(moe_gpu):
    m, dev = moe_gpu
    check_experts(m, dev, 2, 128, 8, 2, 128, 64, gates=np.array([[0.0, -1.5], [0.0, 0.0]]))


def test_experts_large_activations(moe_gpu):
    """fp16 activations whose products pass 65504 between the two GEMMs."""
    m, dev = moe_gpu
    d, f = 128, 128
    x = torch.full((1, d), 60.0, dtype=torch.float16, device=dev)
    w = {}
    for n, shape, s in (("gate", (1, f, d), 0.02), ("up", (1, f, d), 0.02), ("down", (1, d, f), 1e-6)):
        codes = np.full(shape, 15, dtype=np.uint8)
        w[n + "_q"] = torch.from_numpy(B.w4_pack(codes)).to(dev)
        w[n + "_s"] = torch.full((*shape[:-1], shape[-1] // 32), s, dtype=torch.float16, device=dev)
    out = torch.empty(1, d, dtype=torch.float16, device=dev)
    ws = torch.zeros(m.experts_w4_workspace(1, d, 1, 1, f), dtype=torch.uint8, device=dev)
    m.experts_w4(x, torch.zeros(1, 1, dtype=torch.int32, device=dev), torch.ones(1, 1, device=dev), w, out, ws)
    h = 60.0 * 7 * d * float(w["gate_s"][0, 0, 0])
    assert h * h > 65504
    want = h * h * 7 * f * float(w["down_s"][0, 0, 0])
    assert torch.isfinite(out).all() and abs(out[0, 0].item() - want) <= (2.0 ** -11 + 2.0 ** -13) * want


def test_experts_match_the_layer(moe_gpu):
    """Next to the bf16 layer on the dequantised weights, with its own routing."""
    m, dev = moe_gpu
    rng = np.random.default_rng(21)
    T, d, E, k, f = 24, 256, 8, 2, 256
    s = m.shape(T, d, E, k, f)
    buf = m.allocate(s, with_grads=False)
    x, wr = normal(rng, (T, d), torch.bfloat16, dev), normal(rng, (E, d), torch.bfloat16, dev, 0.1)
    w, full = {}, {}
    for n, shape in (("gate", (E, f, d)), ("up", (E, f, d)), ("down", (E, d, f))):
        src = normal(rng, shape, torch.bfloat16, dev, 0.02)
        w[n + "_q"] = torch.empty(*shape[:-1], shape[-1] // 2, dtype=torch.uint8, device=dev)
        w[n + "_s"] = torch.empty(*shape[:-1], shape[-1] // 64, dtype=torch.bfloat16, device=dev)
        m.quantize_w4(src, w[n + "_q"], w[n + "_s"])
        v = torch.empty(shape, device=dev)
        m.dequantize_w4(w[n + "_q"], w[n + "_s"], v)
        full[n] = v.bfloat16()
    out = torch.empty(T, d, dtype=torch.bfloat16, device=dev)
    m.clear_error(buf.ws)
    m.forward(buf, x, wr, None, full["gate"], full["up"], full["down"], out)
    got = torch.empty_like(out)
    ws = torch.zeros(m.experts_w4_workspace(T, d, E, k, f), dtype=torch.uint8, device=dev)
    m.experts_w4(x, buf.saved["topk_idx"], buf.saved["gates"], w, got, ws)
    assert m.read_error(buf.ws) == 0 and m.read_error(ws) == 0
    # the layer rounds weights, activations and expert outputs to bf16: its own tolerance
    assert (got.float() - out.float()).abs().max() <= 2e-2 * out.float().abs().max()


def test_experts_stream_graph_and_repeat(moe_gpu):
    """The same bits again, on another stream, and from a replayed graph on new routes."""
    m, dev = moe_gpu
    x, ti, tg, w, out, ws = check_experts(m, dev, 12, 256, 8, 2, 256, 64)
    again = torch.empty_like(out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.experts_w4(x, ti, tg, w, again, ws)
    torch.cuda.synchronize()
    assert torch.equal(out, again)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.experts_w4(x, ti, tg, w, out, ws)
    for shift in (1, 3):
        ti.add_(shift).remainder_(8)
        graph.replay()
        m.experts_w4(x, ti, tg, w, again, ws)
        torch.cuda.synchronize()
        assert torch.equal(out, again)


def test_refused_tensors(moe_gpu):
    m, dev = moe_gpu
    x, ti, tg, w, out, ws = check_experts(m, dev, 2, 128, 8, 2, 128, 64)
    for args in ((x[:1], ti, tg, w, out, ws), (x, ti.long(), tg, w, out, ws), (x, ti, tg.double(), w, out, ws),
                 (x, ti, tg[:, :1], w, out, ws), (x, ti, tg, w, out[:, :64], ws), (x, ti, tg, w, out, ws[:256]),
                 (x.half(), ti, tg, w, out.half(), ws), (x, ti, tg, {**w, "down_q": w["down_q"][:4]}, out, ws),
                 (x, ti, tg, {**w, "up_s": w["up_s"][..., :1].contiguous()}, out, ws), (x.cpu(), ti, tg, w, out, ws)):
        with pytest.raises((ValueError, TypeError, m.MoEError)):
            m.experts_w4(*args)
    q, s = w["gate_q"][0], w["gate_s"][0]
    y = torch.empty(2, 128, dtype=torch.bfloat16, device=dev)
    for args in ((x[:, :96], q, s, y), (x, q, s.half(), y), (x, q, s, y[:, :100]), (x, q, s, y.float()),
                 (x, q[:, ::2], s, y), (x.t().contiguous().t(), q, s, y)):
        with pytest.raises((ValueError, TypeError, m.MoEError)):
            m.matvec_w4(*args)
