"""The layer norm with MXFP8 output: the stream, the mean and the deviation that its kernels
leave, against the float64 oracle (that the codes are those of these statistics is compared
in test_gpu_layer_norm, with its tolerances).  Widths for one to four groups of columns a
thread, with and without a ring.  GPU only."""
import numpy as np
import pytest
import torch

from gpu_util import f64
from oracle import block_oracle as B
from test_gpu_layer_norm import stream_of
from test_gpu_norm import DT, REL, close, normal

pytestmark = pytest.mark.gpu
SEED, OFFSET = 0xABCDEF0123, (5 << 32) + 3


@pytest.mark.parametrize("d", [128, 256, 384, 640, 2048, 4096, 5120, 8192, 12288, 16384, 20480, 32768])
@pytest.mark.parametrize("rows", [1, 37, 130])
@pytest.mark.parametrize("rt,p,offset", [("bf16", 0.0, 1.5), ("bf16", 0.3, 1.5), ("f32", 0.3, 1.5), ("f32", 0.0, 1000.0)])
def test_stream_and_statistics(moe_gpu, d, rows, rt, p, offset):
    m, dev = moe_gpu
    rng = np.random.default_rng(rows * 7 + d)
    x, res = normal(rng, (rows, d), torch.bfloat16, dev), stream_of(rng, rows, d, DT[rt], dev, offset)
    w, b = normal(rng, (d,), DT[rt], dev), normal(rng, (d,), DT[rt], dev)
    pad = (rows + 127) // 128 * 128
    q = torch.full((pad, d), 0x55, dtype=torch.uint8, device=dev)
    sc = torch.full((pad * d // 32,), 0x55, dtype=torch.uint8, device=dev)
    h = torch.full((rows, d), 9.0, dtype=DT[rt], device=dev)
    mean, rstd = torch.full((rows,), 9.0, device=dev), torch.full((rows,), 9.0, device=dev)
    m.add_layer_norm(x, w, b, None, residual=res, h=h, mean=mean, rstd=rstd, p=p, seed=SEED, offset=OFFSET, y_q=q, y_scales=sc)
    drop = B.dropout(f64(x), p, SEED, OFFSET)
    close(h, drop + f64(res), h.dtype, np.abs(drop) + np.abs(f64(res)))
    hd = f64(h)   # the norm is that of the stored stream
    mu, r = B.add_layer_norm(hd, None, 1.0, None, 1e-5)[2:]
    size = np.abs(hd).mean(-1)
    assert (np.abs(f64(mean) - mu) <= REL * size).all()
    assert (np.abs(f64(rstd) - r) <= (REL + (REL * size * r) ** 2) * r).all()
    # the same stream as the 16-bit output's kernels leave
    y, h2 = torch.empty_like(x), torch.empty_like(h)
    m.add_layer_norm(x, w, b, y, residual=res, h=h2, p=p, seed=SEED, offset=OFFSET)
    assert torch.equal(h, h2)
    # codes against that output: half a code's step (2^-4, below the smallest one 2^-10) of
    # the block's unit and half a bf16 step
    dq = torch.empty(pad, d, dtype=torch.bfloat16, device=dev)
    m.dequantize_mxfp8(pad, d, q, sc, dq)
    top = f64(y).reshape(rows, -1, 32)
    unit = np.repeat(np.abs(top).max(-1) / 224, 32, -1)   # the scale 2^s < largest / 224
    got, want = f64(dq[:rows]), f64(y)
    assert (np.abs(got - want) <= (2.0 ** -4 + 2 * 2.0 ** -8) * np.abs(want) + 2.0 ** -10 * unit * (1 + 2.0 ** -6) + 1e-5 * unit).all()
