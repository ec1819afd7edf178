"""The rotary layouts over so many tokens that every CTA of the pipelined kernels takes
several tiles: the ring of stages is used again, and the weight and bias gradients are
carried from tile to tile. Against the float64 oracle, and bit for bit against the general
kernels; shapes, options and tolerances as in test_gpu_rotary.py."""

import pytest

from test_gpu_rotary import _check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["interleaved", "sectioned"])
@pytest.mark.parametrize("rot, adjacent, opts", [
    (32, False, {}), (48, True, {}), (64, True, {"norm": False}), (32, True, {"bias": True, "scale": 1.125}),
    (16, False, {"norm": False, "bias": True, "table": True})])
def test_many_tiles(lib, cuda, kind, rot, adjacent, opts):
    _check(lib, cuda, (8, 2, 64, 6001), kind, rot, adjacent, opts)
    _check(lib, cuda, (16, 4, 128, 2003), kind, rot, adjacent, opts)


@pytest.mark.parametrize("adjacent", [False, True])
def test_many_tiles_of_wide_rows(lib, cuda, adjacent):
    _check(lib, cuda, (64, 8, 64, 1201), "sectioned", 32, adjacent, {"bias": True})
    _check(lib, cuda, (32, 8, 128, 1021), "interleaved", 64, adjacent, {"bias": True})
    _check(lib, cuda, (128, 16, 64, 1021), "interleaved", 32, adjacent, {})
