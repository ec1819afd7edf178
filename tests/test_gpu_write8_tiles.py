"""The 8-bit write at every way of dividing its tokens among CTAs: one wave of tiles that
several CTAs share, blocks longer than a tile, many waves; against the float64 oracle as in
test_gpu_pool_write8.py. Slots are 304 on 152 SMs."""

import numpy as np
import pytest

from test_gpu_pool_write8 import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("shape", [(32, 8, 128), (64, 16, 64), (4, 1, 64)])
@pytest.mark.parametrize("page_size, block", [(128, 64), (64, 16), (256, 256)])
def test_one_wave(lib, cuda, shape, page_size, block):
    _check(lib, cuda, shape, "interleaved", [5], [3], page_size, block)
    _check(lib, cuda, shape, "sectioned", [257, 40], [0, 77], page_size, block)
    _check(lib, cuda, shape, "interleaved", [1, 900], [600, 31], page_size, block)


@pytest.mark.parametrize("shape", [(4, 2, 128), (16, 16, 64)])
def test_more_than_a_wave(lib, cuda, shape):
    for page_size, block in ((96, 32), (128, 128), (48, 24), (8, 8)):
        _check(lib, cuda, shape, "sectioned", [2128 - 7, 7], [5, 0], page_size, block)   # the last of one wave
        _check(lib, cuda, shape, "interleaved", [100, 2029], [5, 33], page_size, block)  # the first of more


@pytest.mark.parametrize("block", [8, 64])
def test_single_tokens_of_many_sequences(lib, cuda, block):
    rng = np.random.default_rng(block)
    for n in (300, 2200):
        past = [int(p) for p in rng.integers(0, 70, n)]
        _check(lib, cuda, (8, 8, 64), "interleaved", [1] * n, past, 64, block)
