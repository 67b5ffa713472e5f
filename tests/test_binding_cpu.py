"""What the binding takes for an address."""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from heterogeneous_adapters_lora_gb300 import lora as L


class Address(int):
    """An address that an allocator hands out, with a tensor's accessor of its own kind."""

    def data_ptr(self):
        raise AssertionError("an integer is taken as it is")


def test_addresses():
    t, a = torch.zeros(3), np.zeros(3)
    assert L.ptr(None) is None
    assert L.ptr(t) == t.data_ptr()
    assert L.ptr(a) == a.ctypes.data
    assert L.ptr(t.data_ptr() + 4) == t.data_ptr() + 4
    assert L.ptr(Address(4096)) == 4096
    with pytest.raises(TypeError):
        L.ptr("no address")
    with pytest.raises(TypeError):
        L.ptr(ctypes.c_void_p(8))


def test_an_integer_costs_no_exception():
    """No attribute of an integer is asked for: each call of the library has up to twenty of them."""
    seen = []

    class Counted(int):
        def __getattr__(self, name):
            seen.append(name)
            raise AttributeError(name)

    assert L.ptr(Counted(64)) == 64
    assert not seen


def test_tensors_before_and_after_their_type_is_known(monkeypatch):
    t, p = torch.zeros(3), torch.nn.Parameter(torch.zeros(2))
    for known in (None, torch.Tensor):
        monkeypatch.setattr(L, "_tensor", known)
        assert L.ptr(t) == t.data_ptr() and L.ptr(p) == p.data_ptr()
        assert L.ptr(None) is None and L.ptr(7) == 7 and L.ptr(t[1:]) == t.data_ptr() + 4
