"""4-bit weights at their edges.  GPU only."""
import numpy as np
import pytest
import torch

from gpu_util import f64
from oracle import block_oracle as B
from test_gpu_w4 import DT, check_experts, normal

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", list(DT))
def test_weights_that_are_no_numbers_show(moe_gpu, bad, group, dt):
    """A group with one becomes NaN, also in a product; the other groups keep their bits."""
    m, dev = moe_gpu
    rng = np.random.default_rng(group)
    rows, K = 40, 512
    w = normal(rng, (rows, K), DT[dt], dev, 0.05)

    def quantized():
        q = torch.empty(rows, K // 2, dtype=torch.uint8, device=dev)
        s, out = torch.empty(rows, K // group, dtype=DT[dt], device=dev), torch.empty(rows, K, device=dev)
        m.quantize_w4(w, q, s)
        m.dequantize_w4(q, s, out)
        return q, s, out

    clean = quantized()[2]
    places = [(0, 0), (3, K - 1), (17, 130), (39, 77)]
    for r, c in places:
        w[r, c] = bad
    w[5, 128:256] = bad   # whole groups
    q, s, out = quantized()
    hit = torch.zeros(rows, K // group, dtype=torch.bool, device=dev)
    for r, c in places:
        hit[r, c // group] = True
    hit[5, 128 // group:256 // group] = True
    assert torch.equal(torch.isnan(s), hit)
    hit = hit.repeat_interleave(group, 1)
    assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])
    for M in (1, 9):
        y = torch.empty(M, rows, dtype=DT[dt], device=dev)
        m.matvec_w4(normal(rng, (M, K), DT[dt], dev), q, s, y)
        assert np.array_equal(np.isnan(f64(y)), np.tile(f64(hit.any(1)) > 0, (M, 1)))


# ------------------------------------------------------------------ codes around zero
@pytest.mark.parametrize("kind", ["normal", "one sign", "one large value"])
@pytest.mark.parametrize("codes", ["all zero", "one in eight", "any"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dt", list(DT))
def test_error_where_the_weights_are_small(moe_gpu, kind, codes, group, dt):
    """Values beside which the others are small, under weights that are zero or small.
    The limit allows for sums of the codes themselves with 8 times the vector's sum
    taken off (2^-22 of their terms a step of sixteen columns, 2^-24 an addition of the
    vector's sum, at most eleven, and of the result); weights that are all zero give
    exact zeros."""
    m, dev = moe_gpu
    rng = np.random.default_rng(group)
    N, K = 300, 512
    c = np.full((N, K), 8, dtype=np.uint8)
    if codes != "all zero":
        some = rng.random((N, K)) < (0.125 if codes == "one in eight" else 1.0)
        c[some] = rng.integers(0, 16, some.sum())
    s = torch.from_numpy(0.5 + rng.random((N, K // group))).to(DT[dt])
    q, w = torch.from_numpy(B.w4_pack(c)).to(dev), B.w4_values(c, f64(s))
    for M in (1, 9):
        x = rng.standard_normal((M, K))
        if kind == "one sign":
            x = rng.random((M, K))
        if kind == "one large value":
            x[:, ::128] *= 1000
        x = torch.from_numpy(x).to(DT[dt]).to(dev)
        y = torch.empty(M, N, dtype=DT[dt], device=dev)
        m.matvec_w4(x, q, s.to(dev), y)
        want = f64(x) @ w.T
        if codes == "all zero":
            assert (y == 0).all()
        steps = (group / 8 + 8) * 2.0 ** -23
        ax = np.abs(f64(x)).reshape(M, 1, -1, group)
        lost = steps * ((c.reshape(N, -1, group) + 8.0) * ax).sum(-1)
        # the vector itself, held down to 2^-34 of the largest of 128 columns, and the sum over groups
        top = np.abs(f64(x)).reshape(M, -1, 128).max(-1).repeat(128 // group, -1)[:, None]
        lost = ((lost + 2.0 ** -34 * 15 * group * top) * f64(s)).sum(-1) + 32 * 2.0 ** -24 * (np.abs(f64(x)) @ np.abs(w).T)
        lim = torch.finfo(DT[dt]).eps / 2 * np.abs(want) + 1.01 * lost + torch.finfo(DT[dt]).smallest_normal
        err = np.abs(f64(y) - want)
        assert (err <= lim).all(), f"M {M}: {np.max(err / lim):.3f} of the limit"


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M", [1, 9])
def test_values_near_the_end_of_bf16(moe_gpu, group, M):
    """Results are finite where the 32-bit sums are."""
    m, dev = moe_gpu
    rng = np.random.default_rng(group)
    x = rng.standard_normal((M, 256))
    x[:, 5], x[:, 200] = 2.0 ** 120, -1.5 * 2.0 ** 121
    x = torch.from_numpy(x).bfloat16().to(dev)
    c = rng.integers(0, 16, (100, 256)).astype(np.uint8)
    c[7, 5] = c[7, 200] = 8
    s = torch.from_numpy(0.01 * (1 + rng.random((100, 256 // group)))).bfloat16()
    y = torch.empty(M, 100, dtype=torch.bfloat16, device=dev)
    m.matvec_w4(x, torch.from_numpy(B.w4_pack(c)).to(dev), s.to(dev), y)
    w = B.w4_values(c, f64(s))
    want = f64(x) @ w.T
    lim = torch.finfo(torch.bfloat16).eps / 2 * np.abs(want) + (256 / 8 + 64) * 2.0 ** -23 * (np.abs(f64(x)) @ np.abs(w).T)
    # a vector on its own is held down to 2^-38 of the largest of its 128 columns
    top = np.abs(f64(x)).reshape(M, -1, 128).max(-1)
    lim = lim + 2.0 ** -38 * (top @ np.abs(w).reshape(100, -1, 128).sum(-1).T)
    assert torch.isfinite(y).all() and (np.abs(f64(y) - want) <= lim).all()


# ------------------------------------------------------------------ one token
@pytest.mark.parametrize("idx", [[-1, 3, 5, 2], [3, -1, 5, 2], [3, 5, -1, -1], [3, 5, 2, -1], [-1, -1, -1, 6]], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_one_token_with_missing_experts(moe_gpu, idx, group):
    m, dev = moe_gpu
    check_experts(m, dev, 1, 256, 8, 4, 384, group, idx=np.array([idx]))


@pytest.mark.parametrize("dt", list(DT))
def test_one_token_without_experts(moe_gpu, dt):
    m, dev = moe_gpu
    for k in (1, 8):
        out = check_experts(m, dev, 1, 256, 8, k, 128, 64, dt, idx=np.full((1, k), -1))[4]
        assert (out == 0).all()


@pytest.mark.parametrize("bad", [8, -2, 1 << 30, -(1 << 31)])
def test_one_token_with_an_index_out_of_range(moe_gpu, bad):
    m, dev = moe_gpu
    for idx in ([bad, 1, 7], [1, bad, -1], [7, 1, bad], [bad, bad, bad]):
        out = check_experts(m, dev, 1, 256, 8, 3, 256, 128, idx=np.array([idx]), expect_error=m.DEVERR_BOUNDS)[4]
    assert (out == 0).all()


@pytest.mark.parametrize("k", [2, 8, 32])
def test_one_token_with_one_expert_in_every_place(moe_gpu, k):
    m, dev = moe_gpu
    check_experts(m, dev, 1, 256, 8, k, 128, 64, idx=np.full((1, k), 5))


@pytest.mark.parametrize("T,d,E,k,f", [
    (1, 128, 8, 8, 4096),     # the activations of one token's routes do not fit side by side
    (1, 128, 2, 1, 32768), (2, 128, 2, 2, 32768),   # nor those of one route
    (1, 32768, 2, 1, 128),
], ids=str)
@pytest.mark.parametrize("group", [32, 128])
def test_activations_too_long_to_be_staged(moe_gpu, T, d, E, k, f, group):
    m, dev = moe_gpu
    check_experts(m, dev, T, d, E, k, f, group)
    check_experts(m, dev, T, d, E, k, f, group, idx=np.full((T, k), -1))
