"""Layer norm on the host: refusals of the C entry points (nothing here reaches a GPU)
and the oracle against torch's float64 autograd."""
import ctypes
import os
import shutil

import numpy as np
import pytest
import torch

import moe_expert_layer_softmax_gb300 as m
from moe_expert_layer_softmax_gb300 import _build
from oracle import block_oracle as B

INVALID, UNSUPPORTED, ALIGN, NOT_INIT = -1, -2, -3, -5
P = 1 << 20   # an address on a 16-byte boundary that no call below may touch


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    _build.build()
    return m.load()


FWD = dict(rows=8, d=256, dt=0, rt=0, wt=0, x=P, ld_x=256, res=P, ld_res=256, w=P, b=P, h=P, ld_h=256, y=P, ld_y=256,
           mean=P, rstd=P, y_q=0, y_s=0, y_dq=0, seed=1, offset=0, eps=1e-5, p=0.0)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(d=0), INVALID), (dict(d=32769, ld_x=1 << 16), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(dt=3), INVALID), (dict(rt=1), INVALID), (dict(wt=1), INVALID), (dict(dt=2, rt=0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(p=-0.1), INVALID), (dict(p=float("nan")), INVALID),
    (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(y=0), INVALID), (dict(ld_x=255), INVALID), (dict(ld_h=-256), INVALID),
    (dict(b=P + 1), ALIGN), (dict(mean=P + 2), ALIGN), (dict(rstd=P + 2), ALIGN), (dict(w=P + 1), ALIGN), (dict(x=P + 1), ALIGN),
    (dict(h=0), INVALID), (dict(res=0, h=0, p=0.5), INVALID),
    (dict(y_q=P, y_s=P), INVALID), (dict(y=0, y_q=P), INVALID), (dict(y=0, y_q=P, y_s=P, d=192), UNSUPPORTED),
    # the 8-bit output needs vector loads of the bias too
    (dict(y=0, y_q=P, y_s=P, b=P + 2), ALIGN), (dict(y=0, y_q=P, y_s=P, y_dq=P + 2), ALIGN),
])
def test_forward_refusals(lib, change, code):
    assert lib.moe_add_layer_norm(m._ADD_LAYER_NORM.pack(*{**FWD, **change}.values()), None) == code


BWD = dict(rows=8, d=256, dt=0, rt=0, wt=0, dy=P, ld_dy=256, h=P, ld_h=256, dres=P, ld_dres=256, mean=P, rstd=P, w=P,
           dh=P, ld_dh=256, dx=P, ld_dx=256, dw=P, db=P, seed=1, offset=0, p=0.0)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(d=0), INVALID), (dict(d=40000), UNSUPPORTED), (dict(dt=-1), INVALID), (dict(rt=1), INVALID),
    (dict(p=2.0), INVALID), (dict(dy=0), INVALID), (dict(h=0), INVALID), (dict(mean=0), INVALID), (dict(rstd=0), INVALID),
    (dict(w=0), INVALID), (dict(dh=0, dx=0, dw=0, db=0), INVALID), (dict(ws=0), INVALID), (dict(dw=0, ws=0), INVALID),
    (dict(ws=P + 4), ALIGN), (dict(ld_dy=8), INVALID), (dict(ld_dx=0), INVALID), (dict(mean=P + 1), ALIGN),
    (dict(dw=P + 2), ALIGN), (dict(db=P + 2), ALIGN), (dict(dres=P + 1), ALIGN), (dict(rstd=P + 1), ALIGN),
])
def test_backward_refusals(lib, change, code):
    a = {**BWD, **change}
    ws = a.pop("ws", P)
    assert lib.moe_add_layer_norm_bwd(m._ADD_LAYER_NORM_BWD.pack(*a.values()), ws or None, None) == code


def test_calls_without_rows(lib):
    assert lib.moe_add_layer_norm(m._ADD_LAYER_NORM.pack(*{**FWD, "rows": 0, "x": 0, "y": 0}.values()), None) == 0
    a = {**BWD, "rows": 0, "dw": 0, "db": 0, "dy": 0}
    assert lib.moe_add_layer_norm_bwd(m._ADD_LAYER_NORM_BWD.pack(*a.values()), None, None) == 0


def test_workspace(lib):
    assert m.add_layer_norm_bwd_workspace(8, 100) >= 8 * 100 * 8 and m.add_layer_norm_bwd_workspace(0, 100) == 0
    assert m.add_layer_norm_bwd_workspace(1 << 20, 64) == m.add_layer_norm_bwd_workspace(1 << 21, 64)
    v = ctypes.c_size_t()
    for bad in ((-1, 8), (4, 0)):
        assert lib.moe_add_layer_norm_bwd_workspace_size(*bad, ctypes.byref(v)) == INVALID
    assert lib.moe_add_layer_norm_bwd_workspace_size(4, 40000, ctypes.byref(v)) == UNSUPPORTED
    assert lib.moe_add_layer_norm_bwd_workspace_size(4, 64, None) == INVALID


@pytest.mark.parametrize("bias", [True, False])
def test_oracle_against_autograd(bias):
    rng = np.random.default_rng(0)
    rows, d, p, seed, offset = 6, 40, 0.3, 11, 5
    x, res, dy, dres = (torch.from_numpy(rng.standard_normal((rows, d))).requires_grad_() for _ in range(4))
    w, b = (torch.from_numpy(rng.standard_normal(d)).requires_grad_() for _ in range(2))
    mask = torch.from_numpy(B.keep_mask(rows, d, p, seed, offset))
    h = res + torch.where(mask, x * (65536 / (65536 - round(p * 65536))), 0.0)
    y = torch.nn.functional.layer_norm(h, (d,), w, b if bias else None, 1e-5)
    (y * dy.detach() + h * dres.detach()).sum().backward()
    a = [t.detach().numpy() for t in (x, res, w, b, dy, dres)]
    hn, yn, mean, rstd = B.add_layer_norm(a[0], a[1], a[2], a[3] if bias else None, 1e-5, p, seed, offset)
    assert np.allclose(hn, h.detach().numpy(), 1e-12) and np.allclose(yn, y.detach().numpy(), 1e-11, 1e-12)
    dh, dx, dw, db = B.add_layer_norm_bwd(a[4], hn, mean, rstd, a[2], a[5], p, seed, offset)
    for got, want in ((dh, res.grad), (dx, x.grad), (dw, w.grad), (db, b.grad if bias else None)):
        if want is not None:
            assert np.allclose(got, want.numpy(), 1e-10, 1e-11)
