"""Attention of single tokens over the 8-bit pool at the ends of its numbers' range:
scores far beyond the weights' exponents, scales at and beyond their bounds, queries
whose values lie far apart. Against the float64 oracle, bounds as in
test_gpu_attention_decode8.py."""

import numpy as np
import pytest
import torch

import oracle.attention as A
import oracle.pool8 as E8
from attention_parity import U, assert_lse, assert_within
from test_gpu_attention_decode8 import F8, Batch, bound, f64

pytestmark = pytest.mark.gpu


def refill(b, codes=None, scale=None):
    """The batch's keys and values from its tables again, with every stored code
    (codes(i, shape) of pool i) or scale (scale(i, shape)) replaced."""
    for i, (c, s) in enumerate(zip(b.codes, b.scale)):
        if codes is not None and (x := codes(i, c.shape)) is not None:
            c[:] = np.where(c != 127, x, 127)
        if scale is not None and (x := scale(i, s.shape)) is not None:
            s[:] = np.where(np.isfinite(s), x, np.nan)
    page, block = b.codes[0].shape[1], b.codes[0].shape[1] // b.scale[0].shape[1]
    b.keys, b.values = [], []
    for row, n in zip(b.table, b.lengths):
        at = np.arange(n)
        p, o = row[at // page], at % page
        for c, s, to in zip(b.codes, b.scale, (b.keys, b.values)):
            held = np.float64(s[p, o // block])
            held = np.where(np.isnan(held), E8.LEAST, np.clip(held, E8.LEAST, E8.MOST))
            to.append(E8.VALUES[c[p, o]] * held[..., None])


@pytest.mark.parametrize("D, group", [(64, 4), (64, 12), (128, 8), (128, 16)])
@pytest.mark.parametrize("power", [10, 24, 26, 27, 28, 30, 37, 60])
def test_scores_far_beyond_the_weights_exponents(lib, cuda, D, group, power):
    """Scores of about 2^power, of both signs, whose steps in float32 are up to 2^(power
    - 23): one key of each sequence leads by an eighth of that and takes all the weight; or
    all are equal, and the values are averaged. One channel carries the scores, so that a
    score has the rounding of three products and no sum's."""
    g = np.random.default_rng(power)
    for sign, lead in ((1, 1.125), (-1, 0.875), (1, 1.0)):
        b = Batch(group, 1, D, 16, 8, [700, 33, 1, 64], power, spread=20.0)
        key = np.zeros(b.codes[0].shape, np.float64)
        key[..., 0] = sign
        for row, n in zip(b.table, b.lengths):
            at = int(g.integers(n))
            key[row[at // 16], at % 16, :, 0] = sign * lead
        refill(b, codes=lambda i, _: None if i else E8.to_e4m3(key), scale=lambda i, shape: None if i else np.full(shape, 1.0))
        b.q.zero_()
        b.q[:, :, 0] = 2.0 ** power
        ref = b.want(1.0)
        out, lse = b.run(lib, cuda, scale=1.0, save_lse=True)
        what = f"2^{power} {sign} {lead}"
        assert_within(f64(out), ref["out"], bound(ref), what)
        ref["s_abs"] = np.full_like(ref["lse"], 2.0 ** power)
        assert_lse(lse.cpu().numpy(), ref, 700, D, what)


@pytest.mark.parametrize("D, group", [(64, 4), (64, 12), (128, 8)])
@pytest.mark.parametrize("bad", [float("inf"), 3e38, 2.0 ** 121, 2.0 ** 100])
def test_key_scales_at_and_beyond_the_largest(lib, cuda, D, group, bad):
    """Blocks of such a scale among ordinary ones, ordinary queries: the block's largest
    score takes all the weight where it is positive, the other blocks share it where none
    is. Scores beyond float32 are no infinities that cancel."""
    b = Batch(group, 1, D, 16, 8, [100, 33, 8], 41, spread=0.5)
    for row, n in zip(b.table, b.lengths):
        b.scale[0][row[0], 0] = bad
        if n > 90:
            b.scale[0][row[5], 1] = bad
    refill(b)
    ref = b.want()
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    out = b.run(lib, cuda, dev_status=status)
    assert_within(f64(out), ref["out"], bound(ref), f"{bad}")
    assert int(status) == 0


def test_a_key_of_zeros_beyond_the_largest_score(lib, cuda):
    # a query and a scale whose product is no float32, and a key of zeros: its score is 0
    b = Batch(4, 1, 64, 16, 16, [16], 42)
    refill(b, codes=lambda i, shape: None if i else np.zeros(shape, np.uint8), scale=lambda i, shape: np.full(shape, 1.0 if i else 2.0 ** 120))
    b.q = (b.q.double() * 2.0 ** 100).to(torch.bfloat16)
    ref = b.want()
    assert_within(f64(b.run(lib, cuda)), ref["out"], bound(ref), "zeros")
