"""Tensors on another device than the current one are refused.  Host only: tensors of
the host that say they lie on one of two devices, and a library that is not to be called."""
import pytest
import torch

import moe_expert_layer_softmax_gb300 as m


class Placed(torch.Tensor):
    """A tensor that claims to lie on device `at`."""

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.at


class Library:
    """Every entry point counts its call and succeeds."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    m._dtype(torch.zeros(1), "x")   # the binding knows torch
    monkeypatch.setattr(m, "load", lambda: lib)
    monkeypatch.setattr(m, "_stream", lambda stream: 0)
    monkeypatch.setattr(m, "add_norm_bwd_workspace", lambda rows, d: 256)
    monkeypatch.setattr(m, "experts_w4_workspace", lambda *shape: 256)
    monkeypatch.setattr(m, "_several", True, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    return lib


BF, F, U, I = torch.bfloat16, torch.float32, torch.uint8, torch.int32
TENSORS = {   # name: (shape, type) of every tensor of each call
    "add_norm": dict(x=((4, 128), BF), weight=((128,), BF), y=((4, 128), BF), residual=((4, 128), BF), h=((4, 128), BF),
                     rstd=((4,), F)),
    "add_norm mx": dict(x=((4, 128), BF), weight=((128,), BF), y_q=((128, 128), U), y_scales=((512,), U),
                        y_dq=((128, 128), BF)),
    "add_norm_bwd": dict(dy=((4, 128), BF), h=((4, 128), BF), rstd=((4,), F), weight=((128,), BF), dres=((4, 128), BF),
                         dh=((4, 128), BF), dx=((4, 128), BF), dw=((128,), F), ws=((256,), U)),
    "dropout": dict(x=((4, 128), BF), y=((4, 128), BF)),
    "quantize_w4": dict(src=((4, 128), BF), q=((4, 64), U), scales=((4, 2), BF)),
    "dequantize_w4": dict(q=((4, 64), U), scales=((4, 2), BF), out=((4, 128), F)),
    "matvec_w4": dict(x=((2, 128), BF), q=((4, 64), U), scales=((4, 2), BF), y=((2, 4), BF)),
    "experts_w4": dict(x=((2, 128), BF), topk_idx=((2, 1), I), gates=((2, 1), F), out=((2, 128), BF), ws=((256,), U),
                       gate_q=((3, 128, 64), U), gate_s=((3, 128, 2), BF), up_q=((3, 128, 64), U),
                       up_s=((3, 128, 2), BF), down_q=((3, 128, 64), U), down_s=((3, 128, 2), BF)),
}


def call(name, odd=None):
    """The call with tensors on device 1, `odd` on device 0."""
    t = {}
    for n, (shape, dtype) in TENSORS[name].items():
        t[n] = torch.zeros(shape, dtype=dtype).as_subclass(Placed)
        t[n].at = 0 if n == odd else 1
    if name == "experts_w4":
        t["w"] = {n: t.pop(n) for n in list(t) if n[-2:] in ("_q", "_s")}
    if name == "add_norm mx":
        t["y"] = None
    if name == "dropout":
        t.update(p=0.1, seed=1)
    getattr(m, name.split()[0])(**t)


@pytest.mark.parametrize("name", list(TENSORS))
def test_tensors_of_the_current_device_are_taken(lib, name):
    call(name)
    assert lib.calls == 1


@pytest.mark.parametrize("name,odd", [(c, n) for c, ts in TENSORS.items() for n in ts])
def test_a_tensor_of_another_device_is_refused(lib, name, odd):
    with pytest.raises(ValueError, match="current device"):
        call(name, odd)
    assert lib.calls == 0
