"""Every way the kernels around the layer split their work: row groups of 8, 16 and
multiples of 32 threads, one to four groups of columns a thread, rows through the
ring and past it, several rows of a warp of which the last are missing; staged
vectors in rounds of eight and sixteen, fewer where memory is short, and vectors
read where they are.  Checks and tolerances are those of test_gpu_norm.py and
test_gpu_w4.py.  GPU only."""
import numpy as np
import pytest

import test_gpu_norm as N
import test_gpu_w4 as W

pytestmark = pytest.mark.gpu

# rows that do not fill their warps; widths on both sides of each change
ROWS = [(37, 40), (70, 64), (33, 72), (41, 128), (2437, 128), (19, 136), (700, 768), (9, 1152), (5, 1536), (6, 5120),
        (4, 6000), (330, 8192), (3, 8200), (3, 12288), (170, 16384), (2, 16392), (2, 24576), (2, 20000)]
ODD = [(37, 39), (70, 65), (33, 127), (9, 2047), (5, 2049), (3, 4095), (4, 4097), (3, 8191), (2, 8193), (2, 16387)]
TYPES = [("bf16", "bf16", "bf16"), ("f16", "f32", "f16"), ("f32", "f32", "f32")]


@pytest.mark.parametrize("rows,d", ROWS + ODD, ids=str)
@pytest.mark.parametrize("types", TYPES, ids="-".join)
@pytest.mark.parametrize("p", [0.0, 0.2])
def test_norm(moe_gpu, rows, d, types, p):
    m, dev = moe_gpu
    N.check_forward(m, dev, rows, d, *types, p=p)
    N.check_backward(m, dev, rows, d, *types, p=p)


@pytest.mark.parametrize("rows,d", [(1, 128), (17, 128), (300, 128), (35, 256), (9, 512), (7, 640), (130, 768), (5, 896),
                                    (3, 1536), (9, 5120), (3, 8192), (3, 12288), (2, 24576)], ids=str)
@pytest.mark.parametrize("rt,wt,p", [("bf16", "bf16", 0.0), ("f32", "f32", 0.1)])
def test_norm_mxfp8(moe_gpu, rows, d, rt, wt, p):
    N.test_forward_mxfp8(moe_gpu, rows, d, rt, wt, p, True)


@pytest.mark.parametrize("rows,cols", [(1, 40), (37, 64), (129, 72), (4099, 128), (65, 120), (37, 63), (129, 97),
                                       (65, 127), (4099, 768), (3, 131)], ids=str)
@pytest.mark.parametrize("dt", list(N.DT))
def test_dropout(moe_gpu, rows, cols, dt):
    N.test_dropout(moe_gpu, rows, cols, dt, 0.3)


# more than six routes an expert on average; vectors that fill memory, or pass it
@pytest.mark.parametrize("T,d,E,k,f", [
    (12, 128, 1, 1, 128), (16, 256, 4, 4, 256), (17, 128, 2, 2, 256), (40, 256, 2, 2, 256), (64, 384, 8, 8, 128),
    (10, 8192, 2, 1, 128), (10, 128, 2, 1, 4096), (3, 128, 2, 2, 4096), (10, 16384, 2, 1, 128), (10, 128, 2, 1, 8192),
    (1, 128, 8, 8, 8192), (1, 128, 4, 2, 16384), (20, 128, 200, 2, 128),
], ids=str)
@pytest.mark.parametrize("group", [32, 128])
def test_experts(moe_gpu, T, d, E, k, f, group):
    m, dev = moe_gpu
    W.check_experts(m, dev, T, d, E, k, f, group)


def test_experts_of_very_different_load(moe_gpu):
    """One expert with most of the routes, others with one to seventeen, some with none."""
    m, dev = moe_gpu
    T, E = 60, 12
    idx = np.zeros((T, 2), np.int32)
    idx[:, 1] = np.where(np.arange(T) < 17, 3, np.where(np.arange(T) < 25, 5, np.where(np.arange(T) < 34, 7, -1)))
    idx[59, 1] = 11
    W.check_experts(m, dev, T, 256, E, 2, 256, 64, idx=idx)


@pytest.mark.parametrize("M,n,K", [(8, 19500, 128), (3, 5000, 256), (4, 5000, 256), (1, 40, 512), (2, 40, 512),
                                   (3, 4096, 16384), (8, 20000, 8192), (20, 300, 8192)], ids=str)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_matvec(moe_gpu, M, n, K, group):
    m, dev = moe_gpu
    W.check_matvec(m, dev, M, n, K, group, "bf16")
