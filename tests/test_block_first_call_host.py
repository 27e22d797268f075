"""What the wrappers do when the library says that the device is not set up, with
the library and the stream's state replaced: host only."""
import pytest

import moe_expert_layer_softmax_gb300 as m


class Library:
    """moe_dropout as on a device that moe_init has not seen; `after`: its answer then."""

    def __init__(self, after=0):
        self.ready, self.after, self.calls = False, after, []

    def moe_dropout(self, *args):
        self.calls.append(args)
        return self.after if self.ready else m.ERR_NOT_INIT


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(m, "load", lambda: lib)
    monkeypatch.setattr(m, "init", lambda: setattr(lib, "ready", True))
    monkeypatch.setattr(m, "_capturing", lambda handle: False)
    return lib


def test_the_device_is_set_up_and_the_call_made_again(lib):
    m._failed("moe_dropout", m.ERR_NOT_INIT, 1, 2, 3)
    assert lib.ready and lib.calls == [(1, 2, 3)]


def test_other_errors_are_raised_at_once(lib):
    with pytest.raises(m.MoEError) as e:
        m._failed("moe_dropout", -3, 1, 2, 3)
    assert e.value.code == -3 and not lib.ready and not lib.calls


def test_an_error_of_the_second_call_is_raised(lib):
    lib.after = -4
    with pytest.raises(m.MoEError) as e:
        m._failed("moe_dropout", m.ERR_NOT_INIT, 1, 2, 3)
    assert e.value.code == -4 and len(lib.calls) == 1


def test_nothing_is_set_up_within_a_capture(lib, monkeypatch):
    monkeypatch.setattr(m, "_capturing", lambda handle: handle == 3)
    with pytest.raises(m.MoEError) as e:
        m._failed("moe_dropout", m.ERR_NOT_INIT, 1, 2, 3)
    assert e.value.code == m.ERR_NOT_INIT and not lib.ready and not lib.calls
