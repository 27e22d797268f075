"""4-bit weights at their edges.  GPU only."""
import numpy as np
import pytest
import torch

from gpu_util import f64
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
