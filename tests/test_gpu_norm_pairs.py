"""Norm, backward and dropout where rows are read by pairs of columns (an even width
that is no multiple of eight, or rows on a pair's boundary alone), from one warp a
row to the widest rows, fp32 rows with the largest ring, and the 8-bit output's inverse
root mean square.  GPU only."""
import numpy as np
import pytest
import torch

from gpu_util import f64, sf_unpack
from oracle import block_oracle as B
from test_gpu_norm import DT, REL, TYPES, check_backward, check_forward, close, e4m3_step, half, normal, strided, tiny

pytestmark = pytest.mark.gpu
# widths of a row group of 16 threads, of several warps, of 512 threads, and of more
# than one group of columns a thread
WIDTHS = [66, 126, 250, 1002, 2050, 5006, 10002]
ROWS = 21


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_forward(moe_gpu, d, types, p):
    m, dev = moe_gpu
    check_forward(m, dev, ROWS, d, *types, p=p)


@pytest.mark.parametrize("d", WIDTHS)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("p", [0.0, 0.3])
def test_backward(moe_gpu, d, types, p):
    m, dev = moe_gpu
    check_backward(m, dev, ROWS, d, *types, p=p)


@pytest.mark.parametrize("d", [8, 64, 128, 1000, 2048, 4096, 10000])
@pytest.mark.parametrize("types", [TYPES[0], TYPES[1], TYPES[5]], ids="-".join)
def test_base_on_a_pair(moe_gpu, d, types):
    """Widths that take vector loads, from a base one pair past their boundary."""
    m, dev = moe_gpu
    layout = lambda t: strided(t, 6, 2)   # noqa: E731
    check_forward(m, dev, ROWS, d, *types, p=0.2, layout=layout)
    check_backward(m, dev, ROWS, d, *types, p=0.2, layout=layout)


def test_many_rows(moe_gpu):
    """More rows than the grid has groups, and a last row group without one."""
    m, dev = moe_gpu
    check_forward(m, dev, 9001, 66, "bf16", "bf16", "bf16", p=0.2)
    check_forward(m, dev, 2003, 1002, "f32", "f32", "f32", p=0.2)
    check_backward(m, dev, 5003, 126, "bf16", "f32", "bf16", p=0.2)
    check_backward(m, dev, 2003, 1002, "f16", "f16", "f16")


@pytest.mark.parametrize("rows,p", [(310, 0.0), (2003, 0.0), (701, 0.2)], ids=str)
def test_rows_with_the_largest_ring(moe_gpu, rows, p):
    """fp32 rows whose ring leaves room for one block: one round of blocks, or two."""
    m, dev = moe_gpu
    check_forward(m, dev, rows, 7176, "f32", "f32", "f32", p=p)


@pytest.mark.parametrize("cols", [2, 10, 62, 66, 126, 130, 254, 258, 1002, 2050])
@pytest.mark.parametrize("rows", [1, 2, 37])
@pytest.mark.parametrize("dt", list(DT))
def test_dropout(moe_gpu, cols, rows, dt):
    m, dev = moe_gpu
    check_dropout(m, dev, rows, cols, dt)


@pytest.mark.parametrize("cols", [64, 128, 2048])
@pytest.mark.parametrize("dt", list(DT))
def test_dropout_base_on_a_pair(moe_gpu, cols, dt):
    m, dev = moe_gpu
    check_dropout(m, dev, 11, cols, dt, lambda t: strided(t, 4, 2))


def check_dropout(m, dev, rows, cols, dt, layout=lambda t: t):
    rng = np.random.default_rng(rows + cols)
    x = layout(normal(rng, (rows, cols), DT[dt], dev))
    y = layout(torch.full((rows, cols), 9.0, dtype=DT[dt], device=dev))
    m.dropout(x, y, 0.3, 99, (5 << 32) + 1)
    want = B.dropout(f64(x), 0.3, 99, (5 << 32) + 1)
    # the factor and the product are rounded to 32 bits, the result to its type
    lim = (half(DT[dt]) + 2.0 ** -22) * np.abs(want) + tiny(DT[dt])
    assert (np.abs(f64(y) - want) <= lim).all() and ((f64(y) == 0) == (want == 0)).all()


@pytest.mark.parametrize("rows,d", [(3, 128), (130, 512), (5, 640), (70, 2048), (9, 4096), (3, 8192), (2, 12288),
                                    (2, 32768)], ids=str)
@pytest.mark.parametrize("rt,wt,p", [("bf16", "f32", 0.0), ("f32", "bf16", 0.25)])
def test_mxfp8_output_against_the_formula(moe_gpu, rows, d, rt, wt, p):
    """rstd is that of the stored stream, and the codes are those of y made with it."""
    m, dev = moe_gpu
    rng = np.random.default_rng(rows * 3 + d)
    eps = 0.5   # large enough to be seen
    x, res = normal(rng, (rows, d), torch.bfloat16, dev), normal(rng, (rows, d), DT[rt], dev)
    w = normal(rng, (d,), DT[wt], dev)
    pad = (rows + 127) // 128 * 128
    q = torch.empty(pad, d, dtype=torch.uint8, device=dev)
    sc = torch.empty(pad * d // 32, dtype=torch.uint8, device=dev)
    h, rstd = torch.empty(rows, d, dtype=DT[rt], device=dev), torch.empty(rows, device=dev)
    m.add_norm(x, w, None, residual=res, h=h, rstd=rstd, eps=eps, p=p, seed=5, offset=1, y_q=q, y_scales=sc)
    drop = B.dropout(f64(x), p, 5, 1)
    close(h, drop + f64(res), h.dtype, np.abs(drop) + np.abs(f64(res)))
    want_r = 1 / np.sqrt((f64(h) ** 2).mean(-1) + eps)
    assert (np.abs(f64(rstd) - want_r) <= REL * want_r).all()
    out = torch.empty(pad, d, dtype=torch.bfloat16, device=dev)
    m.dequantize_mxfp8(pad, d, q, sc, out)
    y = f64(h) * want_r[:, None] * f64(w)
    unit = np.repeat(np.exp2(sf_unpack(sc.cpu().numpy(), pad, d // 32)[:rows].astype(np.float64) - 127), 32, axis=1)
    z = np.minimum(np.abs(y) / unit, 448)
    # half a step of the code, and what 32 bits lose before it
    assert (np.abs(f64(out[:rows]) - y) / unit <= e4m3_step(z) / 2 + 4 * REL * z).all()
