"""AdamW on the host: refusals of the C entry (nothing here reaches a GPU), tensors of
another device, and the oracle against torch's optimiser in 64 bits."""
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


TENSOR = dict(param=P, grad=P, master=0, m=P, v=P, ms=0, vs=0, n=100)
ARGS = dict(n_tensors=1, pt=2, gt=2, bits=32, scale=0, lr_dev=0, step_dev=0, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.01,
            step=1, seed=0, offset=0)


@pytest.mark.parametrize("change,tensor,code", [
    (dict(n_tensors=-1), {}, INVALID), (dict(pt=3), {}, INVALID), (dict(gt=-1), {}, INVALID), (dict(gt=0), {}, INVALID),
    (dict(bits=16), {}, INVALID), (dict(b1=1.0), {}, INVALID), (dict(b1=-0.1), {}, INVALID), (dict(b2=1.0), {}, INVALID),
    (dict(b2=float("nan")), {}, INVALID), (dict(eps=-1.0), {}, INVALID), (dict(eps=float("inf")), {}, INVALID),
    (dict(wd=-0.1), {}, INVALID), (dict(lr=-1.0), {}, INVALID), (dict(lr=float("nan")), {}, INVALID), (dict(step=0), {}, INVALID),
    (dict(scale=P + 2), {}, ALIGN), (dict(lr_dev=P + 1), {}, ALIGN), (dict(step_dev=P + 4), {}, ALIGN),
    (dict(n_tensors=(1 << 24) + 1), {}, UNSUPPORTED), ({}, dict(n=-1), INVALID), ({}, dict(n=(1 << 34) + 1), UNSUPPORTED),
    ({}, dict(param=0), INVALID), ({}, dict(grad=0), INVALID), ({}, dict(m=0), INVALID), ({}, dict(v=0), INVALID),
    (dict(bits=8), {}, INVALID), (dict(bits=8), dict(ms=P), INVALID), (dict(bits=8), dict(ms=P, vs=P + 2), ALIGN),
    ({}, dict(param=P + 2), ALIGN), ({}, dict(grad=P + 2), ALIGN), ({}, dict(m=P + 1), ALIGN), ({}, dict(v=P + 1), ALIGN),
    (dict(pt=0, gt=0), dict(param=P + 1), ALIGN), (dict(pt=0), dict(master=P + 2), ALIGN),
    ({}, dict(master=P), UNSUPPORTED), (dict(pt=1), {}, UNSUPPORTED),   # fp32 with a copy, fp16 without
])
def test_refusals(lib, change, tensor, code):
    t = ctypes.create_string_buffer(m._ADAMW_TENSOR.pack(*{**TENSOR, **tensor}.values()))
    args = m._ADAMW.pack(ctypes.addressof(t), *{**ARGS, **change}.values())
    assert lib.moe_adamw(args, None) == code


def test_lists_with_and_without_copies(lib):
    t = ctypes.create_string_buffer(b"".join(m._ADAMW_TENSOR.pack(*{**TENSOR, "master": w}.values()) for w in (P, 0)))
    args = {**ARGS, "n_tensors": 2, "pt": 0}
    assert lib.moe_adamw(m._ADAMW.pack(ctypes.addressof(t), *args.values()), None) == INVALID
    assert lib.moe_adamw(m._ADAMW.pack(0, *args.values()), None) == INVALID
    assert lib.moe_adamw(m._ADAMW.pack(0, *{**args, "n_tensors": 0}.values()), None) == 0
    assert lib.moe_adamw(None, None) == INVALID


class Placed(torch.Tensor):
    """A tensor that claims to lie on device `at`."""

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.at


def placed(n, at, dtype=torch.float32):
    t = torch.zeros(n, dtype=dtype).as_subclass(Placed)
    t.at = at
    return t


def test_tensors_of_another_device(monkeypatch):
    m._dtype(torch.zeros(1), "x")
    for odd in range(5):
        ts = [placed(8, 0 if i == odd else 1) for i in range(5)]
        ts[0] = placed(8, 0 if odd == 0 else 1, torch.bfloat16)
        with pytest.raises(ValueError, match="device"):
            m.adamw_list([ts[0]], [ts[1]], [ts[2]], [ts[3]], [ts[4]])
    calls = []

    class Library:
        def moe_adamw(self, *args):
            calls.append(args)
            return 0
    lst = m.adamw_list(*([placed(8, 1)] for _ in range(4)))
    monkeypatch.setattr(m, "load", Library)
    monkeypatch.setattr(m, "_stream", lambda stream: 0)
    monkeypatch.setattr(m, "_several", True)
    for current in (0, 1):
        monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
        if current == lst.device:
            m.adamw(lst, lr=0.1, step=1)
        else:
            with pytest.raises(ValueError, match="current device"):
                m.adamw(lst, lr=0.1, step=1)
    assert len(calls) == 1


def test_oracle_against_torch():
    """Steps of torch's AdamW on the same gradients, in 64 bits."""
    rng = np.random.default_rng(0)
    w = torch.from_numpy(rng.standard_normal(50)).requires_grad_()
    opt = torch.optim.AdamW([w], lr=3e-3, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.2)
    x, a, b = w.detach().numpy().copy(), np.zeros(50), np.zeros(50)
    for step in range(1, 6):
        g = rng.standard_normal(50)
        w.grad = torch.from_numpy(g.copy())
        opt.step()
        x, a, b, _ = B.adamw(x, 2 * g, a, b, 3e-3, step, 0.8, 0.95, 1e-6, 0.2, grad_scale=0.5)
        assert np.allclose(x, w.detach().numpy(), 1e-12, 1e-14)


def test_e4m3_values_and_states():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(B.e4m3_values(codes), want, equal_nan=True)
    rng = np.random.default_rng(1)
    x = (rng.standard_normal(300) * np.exp(4 * rng.standard_normal(300))).astype(np.float32)
    low, s = B.state8(x, np.zeros(300, dtype=np.int64), False)      # number 0: down
    high, _ = B.state8(x, np.full(300, 65535), False)               # up, but for the smallest remainders
    scale = np.repeat(s, 128)[:300].astype(np.float64)
    values = np.unique(np.abs(want[np.isfinite(want)]))
    for v, lo, hi, sc in zip(np.abs(x).astype(np.float64), np.abs(low), np.abs(high), scale):
        z = min(v / sc, 448.0)
        assert lo <= z * (1 + 1e-6) and hi >= z * (1 - 2.0 ** -16)
        assert lo in values and hi in values and np.searchsorted(values, hi) - np.searchsorted(values, lo) <= 1
    assert (B.state8(x, np.zeros(300, dtype=np.int64), True)[0] != 0).all()
