"""4-bit weights at their edges.  GPU only."""
import numpy as np
import pytest
import torch

from gpu_util import f64
from test_gpu_w4 import DT, normal

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
