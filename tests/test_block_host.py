"""Refusals of the block operators: the C entry points turn every bad argument
into an error before anything is enqueued, and the Python wrappers refuse
tensors that do not fit.  Host only: nothing here reaches a GPU."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

import moe_expert_layer_softmax_gb300 as m
from moe_expert_layer_softmax_gb300 import _build

INVALID, UNSUPPORTED, ALIGN = -1, -2, -3
P = 1 << 20   # an address on a 16-byte boundary that no call below may touch


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    _build.build()
    return m.load()


FWD = dict(rows=8, d=256, dt=0, rt=0, wt=0, x=P, ld_x=256, res=P, ld_res=256, w=P, h=P, ld_h=256, y=P,
           ld_y=256, rstd=P, y_q=0, y_s=0, y_dq=0, seed=1, offset=0, eps=1e-5, p=0.0)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(d=0), INVALID), (dict(d=32769, ld_x=1 << 16), UNSUPPORTED),
    (dict(rows=1 << 31), UNSUPPORTED),
    (dict(dt=3), INVALID), (dict(rt=1), INVALID), (dict(wt=1), INVALID), (dict(dt=2, rt=0), INVALID),
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(p=-0.1), INVALID), (dict(p=1.1), INVALID), (dict(p=float("nan")), INVALID),
    (dict(x=0), INVALID), (dict(w=0), INVALID), (dict(y=0), INVALID),
    (dict(ld_x=255), INVALID), (dict(ld_res=0), INVALID), (dict(ld_h=-256), INVALID), (dict(ld_y=1), INVALID),
    (dict(x=P + 1), ALIGN), (dict(res=P + 1), ALIGN), (dict(w=P + 1), ALIGN), (dict(y=P + 1), ALIGN),
    (dict(rstd=P + 2), ALIGN), (dict(rt=2, h=P + 2), ALIGN),
    (dict(h=0), INVALID), (dict(res=0, h=0, p=0.5), INVALID),
    # 8-bit output: beside y, without scales, of another type or width, off the boundary
    (dict(y_q=P, y_s=P), INVALID), (dict(y=0, y_q=P), INVALID), (dict(y_s=P), INVALID), (dict(y_dq=P), INVALID),
    (dict(y=0, y_q=P, y_s=P, dt=1, rt=1, wt=1), UNSUPPORTED),
    (dict(y=0, y_q=P, y_s=P, d=192), UNSUPPORTED),
    (dict(y=0, y_q=P + 8, y_s=P), ALIGN), (dict(y=0, y_q=P, y_s=P + 4), ALIGN),
    (dict(y=0, y_q=P, y_s=P, y_dq=P + 2), ALIGN), (dict(y=0, y_q=P, y_s=P, x=P + 2), ALIGN),
])
def test_add_norm_refusals(lib, change, code):
    assert lib.moe_add_norm(m._ADD_NORM.pack(*{**FWD, **change}.values()), None) == code


BWD = dict(rows=8, d=256, dt=0, rt=0, wt=0, dy=P, ld_dy=256, h=P, ld_h=256, dres=P, ld_dres=256, rstd=P, w=P,
           dh=P, ld_dh=256, dx=P, ld_dx=256, dw=P, seed=1, offset=0, p=0.0)


@pytest.mark.parametrize("change,code", [
    (dict(rows=-1), INVALID), (dict(d=0), INVALID), (dict(d=40000), UNSUPPORTED),
    (dict(dt=-1), INVALID), (dict(rt=1), INVALID), (dict(wt=1), INVALID),
    (dict(p=2.0), INVALID), (dict(p=float("nan")), INVALID),
    (dict(dy=0), INVALID), (dict(h=0), INVALID), (dict(rstd=0), INVALID), (dict(w=0), INVALID),
    (dict(dh=0, dx=0, dw=0), INVALID), (dict(ws=0), INVALID), (dict(ws=P + 4), ALIGN),
    (dict(ld_dy=8), INVALID), (dict(ld_dres=255), INVALID), (dict(ld_dh=0), INVALID), (dict(ld_dx=0), INVALID),
    (dict(dy=P + 1), ALIGN), (dict(h=P + 1), ALIGN), (dict(dres=P + 1), ALIGN), (dict(dh=P + 1), ALIGN),
    (dict(dx=P + 1), ALIGN), (dict(dw=P + 2), ALIGN), (dict(rstd=P + 1), ALIGN), (dict(w=P + 1), ALIGN),
])
def test_add_norm_bwd_refusals(lib, change, code):
    a = {**BWD, **change}
    ws = a.pop("ws", P)
    assert lib.moe_add_norm_bwd(m._ADD_NORM_BWD.pack(*a.values()), ws or None, None) == code


@pytest.mark.parametrize("args,code", [
    ((-1, 8, 0, P, 8, P, 8, 0.1), INVALID), ((4, 0, 0, P, 8, P, 8, 0.1), INVALID),
    ((4, 8, 9, P, 8, P, 8, 0.1), INVALID), ((4, 8, 0, None, 8, P, 8, 0.1), INVALID),
    ((4, 8, 0, P, 8, None, 8, 0.1), INVALID), ((4, 8, 0, P, 7, P, 8, 0.1), INVALID),
    ((4, 8, 0, P, 8, P, 0, 0.1), INVALID), ((4, 8, 0, P, 8, P, 8, 1.5), INVALID),
    ((4, 8, 0, P, 8, P, 8, float("nan")), INVALID), ((4, 8, 2, P + 2, 8, P, 8, 0.1), ALIGN),
    ((4, 8, 0, P, 8, P + 1, 8, 0.1), ALIGN), ((1 << 31, 8, 0, P, 8, P, 8, 0.1), UNSUPPORTED),
    ((1, (1 << 30) + 1, 0, P, 1 << 31, P, 1 << 31, 0.1), UNSUPPORTED),
])
def test_dropout_refusals(lib, args, code):
    assert lib.moe_dropout(*args, 1, 0, None) == code


@pytest.mark.parametrize("rows,K,g,dt,ptrs,code", [
    (-1, 128, 32, 0, (P, P, P), INVALID), (4, 0, 32, 0, (P, P, P), INVALID), (4, 128, 32, 2, (P, P, P), INVALID),
    (4, 128, 16, 0, (P, P, P), UNSUPPORTED), (4, 96, 64, 0, (P, P, P), UNSUPPORTED),
    (4, 128, 32, 0, (None, P, P), INVALID), (4, 128, 32, 0, (P, None, P), INVALID),
    (4, 128, 32, 0, (P, P, None), INVALID), (4, 128, 32, 0, (P + 2, P, P), ALIGN),
    (4, 128, 32, 0, (P, P + 4, P), ALIGN), (4, 128, 32, 0, (P, P, P + 2), ALIGN),
])
def test_quantize_w4_refusals(lib, rows, K, g, dt, ptrs, code):
    assert lib.moe_quantize_w4(rows, K, g, dt, *ptrs, None) == code
    assert lib.moe_dequantize_w4(rows, K, g, dt, *ptrs, None) == code


MV = dict(M=2, N=64, K=256, g=64, dt=0, x=P, ld_x=256, q=P, s=P, y=P, ld_y=64)


@pytest.mark.parametrize("change,code", [
    (dict(M=-1), INVALID), (dict(N=0), INVALID), (dict(K=0), INVALID), (dict(dt=2), INVALID),
    (dict(g=48), UNSUPPORTED), (dict(K=224, g=128), UNSUPPORTED), (dict(N=1 << 20, ld_y=1 << 20), UNSUPPORTED),
    (dict(x=None), INVALID), (dict(q=None), INVALID), (dict(s=None), INVALID), (dict(y=None), INVALID),
    (dict(ld_x=255), INVALID), (dict(ld_y=63), INVALID), (dict(ld_x=260), ALIGN), (dict(x=P + 8), ALIGN),
    (dict(q=P + 8), ALIGN), (dict(s=P + 2), ALIGN), (dict(y=P + 1), ALIGN),
])
def test_matvec_w4_refusals(lib, change, code):
    assert lib.moe_matvec_w4(*{**MV, **change}.values(), None) == code


EX = dict(T=2, d=256, E=8, k=2, f=128, g=64, dt=0, x=P, idx=P, gates=P, gq=P, gs=P, uq=P, us=P, dq=P, ds=P, out=P)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(d=0), INVALID), (dict(f=0), INVALID),
    (dict(d=192), UNSUPPORTED), (dict(f=64), UNSUPPORTED), (dict(E=257), UNSUPPORTED), (dict(k=33), UNSUPPORTED),
    (dict(T=2049), UNSUPPORTED), (dict(g=16), UNSUPPORTED), (dict(dt=2), INVALID), (dict(ws=0), INVALID),
    (dict(ws=P + 4), ALIGN),
    *[({n: 0}, INVALID) for n in ("x", "idx", "gates", "gq", "gs", "uq", "us", "dq", "ds", "out")],
    *[({n: P + 8}, ALIGN) for n in ("x", "idx", "gates", "gq", "gs", "uq", "us", "dq", "ds", "out")],
])
def test_experts_w4_refusals(lib, change, code):
    a = {**EX, **change}
    ws = a.pop("ws", P)
    assert lib.moe_experts_w4(m._EXPERTS_W4.pack(*a.values()), ws or None, None) == code


def test_null_argument_blocks(lib):
    assert lib.moe_add_norm(None, None) == INVALID
    assert lib.moe_add_norm_bwd(None, None, None) == INVALID
    assert lib.moe_experts_w4(None, None, None) == INVALID


def test_calls_without_rows_do_nothing(lib):
    assert lib.moe_add_norm(m._ADD_NORM.pack(*{**FWD, "rows": 0, "x": 0, "y": 0}.values()), None) == 0
    assert lib.moe_dropout(0, 8, 0, None, 8, None, 8, 0.1, 1, 0, None) == 0
    assert lib.moe_matvec_w4(*{**MV, "M": 0, "x": None, "y": None}.values(), None) == 0
    assert lib.moe_quantize_w4(0, 128, 32, 0, None, None, None, None) == 0
    assert lib.moe_experts_w4(m._EXPERTS_W4.pack(*{**EX, "T": 0, "x": 0}.values()), None, None) == 0


def test_workspace_sizes(lib):
    assert m.add_norm_bwd_workspace(0, 128) >= 0
    for rows, d in ((1, 1), (32768, 4096), (100, 32768)):
        n = m.add_norm_bwd_workspace(rows, d)
        assert 4 * d <= n <= 4 * d * 1216 + 256
    assert m.experts_w4_workspace(0, 128, 1, 1, 128) >= 256
    assert m.experts_w4_workspace(64, 4096, 64, 8, 2048) >= 64 * 8 * 4 * (4096 + 2048)
    with pytest.raises(m.MoEError):
        m.add_norm_bwd_workspace(4, 40000)
    with pytest.raises(m.MoEError):
        m.experts_w4_workspace(4, 100, 8, 2, 128)


def test_argument_blocks_match_the_header(tmp_path):
    """The binding packs the C structs itself: sizes and offsets of the header's."""
    src = tmp_path / "s.cpp"
    src.write_text('''#include <cstdio>
#include <cstddef>
#include "moe.h"
int main() {
  printf("%zu %zu %zu\\n", sizeof(moe_add_norm_args_t), sizeof(moe_add_norm_bwd_args_t), sizeof(moe_experts_w4_args_t));
  printf("%zu %zu %zu\\n", offsetof(moe_add_norm_args_t, p), offsetof(moe_add_norm_bwd_args_t, p), offsetof(moe_experts_w4_args_t, out));
}''')
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe = tmp_path / "s"
    subprocess.run(["g++", "-I", os.path.join(_build.ROOT, "include"), str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    packs = (m._ADD_NORM, m._ADD_NORM_BWD, m._EXPERTS_W4)
    assert [int(v) for v in out[:3]] == [s.size for s in packs]
    assert int(out[3]) == m._ADD_NORM.size - 4
    assert int(out[4]) == m._ADD_NORM_BWD.size - 8
    assert int(out[5]) == m._EXPERTS_W4.size - ctypes.sizeof(ctypes.c_void_p)


def test_wrappers_refuse_host_tensors_and_other_types():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        m.add_norm(x, w, x.clone())
    with pytest.raises(TypeError):
        m.add_norm(x.double(), w, x.clone())
    with pytest.raises(ValueError, match="not a CUDA tensor"):
        m.dropout(x, x.clone(), 0.1, 1)
    q, s = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        m.matvec_w4(x, q, s, torch.zeros(4, 8, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        m.matvec_w4(x, q.int(), s, x)
    with pytest.raises(ValueError, match="do not belong together"):
        m.matvec_w4(x, q, s[:4], x)
