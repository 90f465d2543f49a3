"""How the binding takes pointers: tensors and whole numbers, and nothing that merely converts to one."""
import ctypes
import timeit

import numpy as np
import pytest
import torch

import heterogeneous_adapters_sgmv_b200 as L


def test_pointer_of_tensors_and_numbers():
    t = torch.zeros(4)
    assert L._ptr(t) == t.data_ptr() and L._ptr(None) is None and L._ptr(1 << 40) == 1 << 40 and L._ptr(0) == 0


# a host array of one id would otherwise pass for the address 3 (or, at id 0, for no ids at all)
@pytest.mark.parametrize("obj", [np.array([3], dtype=np.int32), np.array([0]), np.int64(1 << 20), 4096.0, "4096",
                                 ctypes.c_void_p(4096), [4096]], ids=repr)
def test_pointer_of_anything_else_is_refused(obj):
    with pytest.raises(AttributeError):
        L._ptr(obj)


def test_pointer_of_a_number_costs_no_more_than_that_of_a_tensor():
    """A raw address needs no attribute lookup that fails first (ten times a tensor's cost; the bound is three)."""
    t, best = torch.zeros(4), {}
    for k, obj in (("number", 1 << 40), ("tensor", t)):
        best[k] = min(timeit.repeat(lambda: L._ptr(obj), number=5000, repeat=15))
    assert best["number"] < 3 * best["tensor"], best
