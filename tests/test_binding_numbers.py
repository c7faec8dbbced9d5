"""Numbers that a caller hands to the tensor binding may run code of the caller's when they are read, which changes the
list that they come from, or the tensors. They are read first, from a list of the binding's own. (CPU tensors: the calls end with
their refusal, no GPU.)"""
import os

import pytest


@pytest.fixture(scope="module")
def bl():
    import matrix_dense_linear_spd_gb300 as m
    if not os.path.exists(m.LIB_PATH):
        from matrix_dense_linear_spd_gb300 import build
        build.build()
    return m


class Number:
    def __init__(self, value, then):
        self.value, self.then, self.read = value, then, 0

    def __float__(self):
        self.read += 1
        self.then()
        return self.value

    def __index__(self):
        self.read += 1
        self.then()
        return int(self.value)


def test_coefficients_are_read_before_the_list_changes(bl):
    import torch
    given = []
    numbers = [Number(v, given.clear) for v in (3.4445, -4.775, 2.0315)]
    given.extend(numbers)
    with pytest.raises(ValueError, match="CUDA"):
        bl.orth(torch.zeros(4, 8), coefficients=given)
    assert [n.read for n in numbers] == [1, 1, 1] and not given


def test_numbers_are_read_before_the_tensors_are_looked_at(bl):
    import torch
    x = torch.zeros(4, 8)
    t = torch.zeros(4, dtype=torch.int64)
    steps, top = Number(5, lambda: x.resize_(4)), Number(3, lambda: x.resize_(4))
    with pytest.raises(ValueError, match="rows, cols"):
        bl.orth(x, steps=steps)
    x.resize_(4, 8)
    with pytest.raises(ValueError, match="rows, cols"):
        bl.score(x, x, t, top)
    assert steps.read == top.read == 1


@pytest.mark.parametrize("bad", [3, (1.0, 2.0), (1.0, 2.0, 3.0, 4.0), (1.0, "x", 2.0)])
def test_other_coefficients_are_refused(bl, bad):
    import torch
    with pytest.raises((TypeError, ValueError)):
        bl.orth(torch.zeros(4, 8), coefficients=bad)
