"""The few-token layer on the host: refusals of the C entry points (nothing here reaches a
GPU), sizes, tensors of another device."""
import ctypes
import os
import shutil

import pytest
import torch

import moe_expert_layer_softmax_gb300 as m
from moe_expert_layer_softmax_gb300 import _build

INVALID, UNSUPPORTED, ALIGN, NOT_INIT = -1, -2, -3, -5
P = 1 << 20   # an address on a 16-byte boundary that no call below may touch


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    _build.build()
    return m.load()


ARGS = dict(x=P, wr=P, bias=0, wg=P, wu=P, wd=P, logits=0, idx=0, gates=0, out=P)


@pytest.mark.parametrize("change,code", [
    *[({n: 0}, INVALID) for n in ("x", "wg", "wu", "wd", "out", "ws")],
    *[({n: P + 8}, ALIGN) for n in ("x", "wr", "bias", "wg", "wu", "wd", "logits", "idx", "gates", "out", "ws")],
    (dict(wr=0), INVALID), (dict(wr=0, idx=P), INVALID), (dict(wr=0, gates=P), INVALID),
    (dict(wr=0, idx=P, gates=P, logits=P), INVALID), (dict(wr=0, idx=P, gates=P, bias=P), INVALID),
])
def test_refused_arguments(lib, change, code):
    a = {**ARGS, **change}
    ws = a.pop("ws", P)
    s = m.shape(4, 256, 8, 2, 128)
    assert lib.moe_few_fwd(ctypes.byref(s), m._FEW.pack(*a.values()), ws or None, None) == code


@pytest.mark.parametrize("bad,code", [
    ((-1, 128, 8, 2, 128, 0), INVALID), ((65, 128, 8, 2, 128, 0), UNSUPPORTED), ((16, 128, 8, 9, 128, 0), INVALID),
    ((16, 100, 8, 2, 128, 0), UNSUPPORTED), ((16, 128, 8, 2, 200, 0), UNSUPPORTED), ((16, 128, 300, 2, 128, 0), UNSUPPORTED),
    ((16, 128, 64, 33, 128, 0), UNSUPPORTED), ((16, 128, 8, 2, 128, 1), UNSUPPORTED), ((16, 128, 8, 2, 128, 7), INVALID),
    ((4, 128, 256, 2, 1 << 23, 0), UNSUPPORTED), ((4, 1 << 23, 256, 2, 128, 0), UNSUPPORTED),
])
def test_refused_shapes(lib, bad, code):
    s = m.shape(*bad)
    assert lib.moe_few_fwd(ctypes.byref(s), m._FEW.pack(*ARGS.values()), P, None) == code
    with pytest.raises(m.MoEError) as e:
        m.few_workspace(s)
    assert e.value.code == code


def test_no_tokens_and_sizes(lib):
    s = m.shape(0, 128, 8, 2, 128)
    assert lib.moe_few_fwd(ctypes.byref(s), m._FEW.pack(*[0] * 10), None, None) == 0
    assert lib.moe_few_fwd(ctypes.byref(s), None, None, None) == INVALID
    assert lib.moe_few_fwd(None, m._FEW.pack(*ARGS.values()), P, None) == INVALID
    one, many = (m.few_workspace(m.shape(t, 4096, 64, 8, 2048)) for t in (1, 64))
    assert one >= 256 + 8 * 8 + 8 * 2048 * 2 and many >= 512 * 2048 * 2 and m.few_workspace(s) > 0
    assert lib.moe_few_workspace_size(ctypes.byref(s), None) == INVALID
    assert m.FEW_MAX_TOKENS == 64


class Placed(torch.Tensor):
    """A tensor that claims to lie on device `at`."""

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.at


BF, F, U, I = torch.bfloat16, torch.float32, torch.uint8, torch.int32
CALLS = {
    "forward_few": dict(x=((4, 128), BF), w_router=((8, 128), BF), logit_bias=((4, 8), F), w_gate=((8, 128, 128), BF),
                        w_up=((8, 128, 128), BF), w_down=((8, 128, 128), BF), out=((4, 128), BF), ws=((256,), U),
                        topk_idx=((4, 2), I), gates=((4, 2), F), logits=((4, 8), F)),
    "add_layer_norm": dict(x=((4, 128), BF), weight=((128,), BF), bias=((128,), BF), y=((4, 128), BF), residual=((4, 128), F),
                           h=((4, 128), F), mean=((4,), F), rstd=((4,), F)),
    "add_layer_norm_bwd": dict(dy=((4, 128), BF), h=((4, 128), BF), mean=((4,), F), rstd=((4,), F), weight=((128,), BF),
                               dres=((4, 128), BF), dh=((4, 128), BF), dx=((4, 128), BF), dw=((128,), F), db=((128,), F),
                               ws=((256,), U)),
}


@pytest.mark.parametrize("name,odd", [(c, n) for c, ts in CALLS.items() for n in [None, *ts]])
def test_a_tensor_of_another_device_is_refused(monkeypatch, name, odd):
    calls = []

    class Library:
        def __getattr__(self, name):
            return lambda *args: calls.append(args) or 0
    m._dtype(torch.zeros(1), "x")
    lib = Library()
    monkeypatch.setattr(m, "load", lambda: lib)
    monkeypatch.setattr(m, "_stream", lambda stream: 0)
    monkeypatch.setattr(m, "add_layer_norm_bwd_workspace", lambda rows, d: 256)
    monkeypatch.setattr(m, "few_workspace", lambda s: 256)
    monkeypatch.setattr(m, "_several", True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    t = {}
    for n, (shape, dtype) in CALLS[name].items():
        t[n] = torch.zeros(shape, dtype=dtype).as_subclass(Placed)
        t[n].at = 0 if n == odd else 1
    if name == "forward_few":
        t["s"] = m.shape(4, 128, 8, 2, 128)
    if odd is None:
        getattr(m, name)(**t)
        assert len(calls) == 1
    else:
        with pytest.raises(ValueError, match="current device"):
            getattr(m, name)(**t)
        assert not calls
