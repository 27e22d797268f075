"""Calls whose offset of the drawn numbers lies on the device: refusals of the C entries
and of the binding, and which entry the binding takes.  Host only."""
import ctypes
import os
import shutil

import pytest
import torch

import moe_expert_layer_softmax_gb300 as m
from moe_expert_layer_softmax_gb300 import _build
from test_adamw_host import ARGS, P, TENSOR, Placed, placed
from test_block_host import BWD, FWD
from test_layer_norm_host import BWD as LN_BWD, FWD as LN_FWD

INVALID, ALIGN = -1, -3


@pytest.fixture(scope="module")
def lib():
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("nvcc not available")
    _build.build()
    return m.load()


def test_adamw_refusals(lib):
    t = ctypes.create_string_buffer(m._ADAMW_TENSOR.pack(*TENSOR.values()))

    def pack(**change):
        return m._ADAMW.pack(ctypes.addressof(t), *{**ARGS, **change}.values())
    assert lib.moe_adamw_at(None, P, None) == INVALID
    assert lib.moe_adamw_at(pack(), P + 4, None) == ALIGN
    assert lib.moe_adamw_at(pack(b1=1.0), P, None) == INVALID
    assert lib.moe_adamw_at(pack(n_tensors=0), P, None) == 0


def test_norm_and_dropout_refusals(lib):
    """A counter off its boundary is refused, also without dropout; the other checks stay."""
    fwd, ln = m._ADD_NORM.pack(*FWD.values()), m._ADD_LAYER_NORM.pack(*LN_FWD.values())
    bwd, ln_bwd = m._ADD_NORM_BWD.pack(*BWD.values()), m._ADD_LAYER_NORM_BWD.pack(*LN_BWD.values())
    assert lib.moe_add_norm_at(fwd, P + 4, None) == ALIGN and lib.moe_add_layer_norm_at(ln, P + 4, None) == ALIGN
    assert lib.moe_add_norm_bwd_at(bwd, P, P + 4, None) == ALIGN and lib.moe_add_layer_norm_bwd_at(ln_bwd, P, P + 4, None) == ALIGN
    assert lib.moe_add_norm_bwd_at(bwd, None, P, None) == INVALID and lib.moe_add_layer_norm_bwd_at(ln_bwd, None, P, None) == INVALID
    for f in (lib.moe_add_norm_at, lib.moe_add_layer_norm_at):
        assert f(None, P, None) == INVALID
    for f in (lib.moe_add_norm_bwd_at, lib.moe_add_layer_norm_bwd_at):
        assert f(None, P, P, None) == INVALID
    assert lib.moe_dropout_at(4, 8, 0, P, 8, P, 8, 0.1, 1, 0, P + 2, None) == ALIGN
    assert lib.moe_dropout_at(4, 0, 0, P, 8, P, 8, 0.1, 1, 0, P, None) == INVALID
    assert lib.moe_dropout_at(0, 8, 0, P, 8, P, 8, 0.1, 1, 0, P, None) == 0


class Library:
    """Takes the calls down; every entry answers 0."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture
def fake(monkeypatch):
    m._dtype(torch.zeros(1), "x")
    lib = Library()
    monkeypatch.setattr(m, "load", lambda: lib)
    monkeypatch.setattr(m, "_stream", lambda stream: 77)
    monkeypatch.setattr(m, "_several", False)
    return lib


def counter(n=1, dtype=torch.int64):
    return placed(n, 0, dtype)


def calls():
    lst = m.adamw_list(*([placed(8, 0)] for _ in range(4)))
    x, w, f = (torch.zeros(4, 64).as_subclass(Placed) for _ in range(3))
    w, f = w[0], f[:, 0].contiguous()
    for t in (x, w, f):
        t.at = 0
    return {"adamw": lambda **kw: m.adamw(lst, lr=0.1, step=1, **kw),
            "add_norm": lambda **kw: m.add_norm(x, w, x, h=x, p=0.1, **kw),
            "add_norm_bwd": lambda **kw: m.add_norm_bwd(x, x, f, w, dx=x, p=0.1, **kw),
            "add_layer_norm": lambda **kw: m.add_layer_norm(x, w, w, x, h=x, p=0.1, **kw),
            "add_layer_norm_bwd": lambda **kw: m.add_layer_norm_bwd(x, x, f, f, w, dx=x, p=0.1, **kw),
            "dropout": lambda **kw: m.dropout(x, x, 0.1, 1, **kw)}


NAMES = ["adamw", "add_norm", "add_norm_bwd", "add_layer_norm", "add_layer_norm_bwd", "dropout"]


@pytest.mark.parametrize("name", NAMES)
def test_the_entry_that_is_called(fake, name):
    call, at = calls()[name], counter()
    call()
    call(offset_dev=at)
    (plain, a), (other, b) = fake.calls
    assert plain == "moe_" + name and other == plain + "_at"
    assert len(b) == len(a) + 1 and a[-1] == b[-1] == 77 and b[-2] == at.data_ptr()


@pytest.mark.parametrize("name", NAMES)
def test_counters_that_are_refused(fake, name):
    call = calls()[name]
    for bad, error in ((counter(2), ValueError), (counter(0), ValueError), (counter(1, torch.int32), TypeError),
                       (counter(1, torch.float32), TypeError), (torch.zeros(1, dtype=torch.int64), ValueError)):
        with pytest.raises(error):
            call(offset_dev=bad)
    assert not fake.calls


def test_a_device_that_is_not_set_up(fake, monkeypatch):
    """The call with a counter sets the device up and is made again, itself and not the form
    without."""
    answers, made = [m.ERR_NOT_INIT, 0], []
    monkeypatch.setattr(m, "load", lambda: type("L", (), {"__getattr__": lambda s, n: lambda *a: made.append((n, a)) or answers.pop(0)})())
    monkeypatch.setattr(m, "_capturing", lambda handle: False)
    monkeypatch.setattr(m, "init", lambda: made.append("init"))
    calls()["dropout"](offset_dev=counter())
    (first, a), init, (second, b) = made
    assert first == second == "moe_dropout_at" and init == "init" and a == b
