"""The variant options' marshalling: what counts as frequencies."""

import numpy as np
import pytest
import torch


def _freq(v, n):
    return [v.inv_freq[i] for i in range(n)]


@pytest.mark.parametrize("make", [list, tuple, np.array, torch.tensor, lambda f: [str(x) for x in f], iter,
                                  lambda f: np.array(f, dtype=np.float32), lambda f: [np.float64(x) for x in f]])
def test_any_sequence_of_numbers(lib, make):
    f = [2.0 ** -i for i in range(32)]
    assert _freq(lib.functional._variant(inv_freq=make(f), dim=64), 32) == f
    assert _freq(lib.functional._variant(inv_freq=make(f), dim=128, rotary_dim=64), 32) == f
    if make is not iter:
        assert _freq(lib.variant(inv_freq=make(f)), 32) == f


def test_a_struct_keeps_its_frequencies(lib):
    many = [lib.variant(inv_freq=[float(i + j) for j in range(32)]) for i in range(600)]
    assert all(_freq(v, 32) == [float(i + j) for j in range(32)] for i, v in enumerate(many))


def test_how_many(lib):
    f = lib.functional
    for bad in (dict(inv_freq=[1.0] * 31, dim=64), dict(inv_freq=[1.0] * 32, dim=64, rotary_dim=32)):
        with pytest.raises(ValueError, match="frequencies"):
            f._variant(**bad)
