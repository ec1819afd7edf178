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


@pytest.mark.parametrize("bad", [float("inf"), 3e38, 2.0 ** 121, 2.0 ** 120])
def test_value_scales_at_and_beyond_the_largest(lib, cuda, bad):
    # codes of at most 32, so that the results are finite in bf16
    b = Batch(8, 2, 64, 16, 8, [100, 33, 8], 43)
    g = np.random.default_rng(44)
    refill(b, codes=lambda i, shape: E8.to_e4m3(np.clip(g.standard_normal(shape) * 8, -32, 32)) if i else None)
    for row in b.table:
        b.scale[1][row[0], 0] = bad
    refill(b)
    ref = b.want()
    down = 2.0 ** -100
    assert_within(f64(b.run(lib, cuda)) * down, ref["out"] * down, bound(ref) * down, f"{bad}")


def test_a_scale_that_grows_past_2_to_120_is_read_back(lib, cuda):
    """A block with the scale 1.1 2^119 gets a value of 3.35e38: the least power of two
    that holds it makes 1.1 2^120. What is written has to be what is read, and what a later
    token finds."""
    F, n_q, n_kv, D = lib.functional, 2, 1, 64
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    pools = [torch.full((1, 16, n_kv, D), 0x60, dtype=torch.uint8, device=cuda).view(F8) for _ in range(2)]  # 32
    scales = [torch.full((1, 2, n_kv), 1.1 * 2.0 ** 119, device=cuda) for _ in range(2)]
    first = float(scales[0][0, 0, 0])
    held = 32.0 * first

    def append(value, at):
        rows = torch.zeros(1, (n_q + 2 * n_kv) * D, dtype=torch.bfloat16, device=cuda)
        rows[:, n_q * D:] = value
        F.prologue_pool_write8(rows, None, None, None, i32(0), i32(at), *pools, *scales, n_q, n_kv, D, "sectioned",
                               norm=False, nope=True)

    def read(at):
        """The value at a place: attention to it alone, as if its block began there."""
        one = [torch.full((1, 16, n_kv, D), 127, dtype=torch.uint8, device=cuda).view(F8) for _ in range(2)]
        for p, o in zip(pools, one):
            o.view(torch.uint8)[0, 0] = p.view(torch.uint8)[0, at]
        q = torch.zeros(1, n_q, D, dtype=torch.bfloat16, device=cuda)
        return f64(F.attention_decode8(q, *one, *scales, i32(0)[None], i32(1)))

    big = float(torch.tensor(3.35e38).to(torch.bfloat16))
    append(big, 3)
    for s in scales:
        assert float(s[0, 0, 0]) == 2.0 * first and float(s[0, 1, 0]) == first
    assert np.all(np.abs(read(3) - big) <= (2.0 ** -4 + 2.0 ** -8) * big)
    assert np.all(np.abs(read(0) - held) <= 2.0 ** -8 * held)
    append(1.0, 4)  # no reason to grow, and none to shrink
    for s in scales:
        assert float(s[0, 0, 0]) == 2.0 * first
    assert np.all(np.abs(read(3) - big) <= (2.0 ** -4 + 2.0 ** -8) * big)
    assert np.all(np.abs(read(0) - held) <= 2.0 ** -8 * held)


@pytest.mark.parametrize("D, group", [(64, 4), (64, 12), (128, 8)])
@pytest.mark.parametrize("power", [12, 16, 20, 25, 30])
def test_a_query_value_far_above_the_others(lib, cuda, D, group, power):
    """A channel of the query 2^power times the others, which no key has anything in: the
    scores are those of the others. They are of 1/2 to 2 in magnitude (scaled by the
    channel), so that every one lies within 2^-32 of the row's largest."""
    b = Batch(group, 1, D, 16, 8, [100, 33, 3], 50 + power)
    g = np.random.default_rng(power)
    q = np.exp2(g.uniform(-1, 1, b.q.shape)) * g.choice((-1, 1), b.q.shape)
    q[..., 5] = -1.5 * 2.0 ** power
    b.q = torch.from_numpy(q).to(torch.bfloat16)
    b.codes[0][..., 5] = np.where(b.codes[0][..., 5] == 127, 127, 0)
    refill(b)
    ref = b.want()
    out, lse = b.run(lib, cuda, save_lse=True)
    assert_within(f64(out), ref["out"], bound(ref), f"2^{power}")
    assert_lse(lse.cpu().numpy(), ref, 100, D, f"2^{power}")
    b.q = (b.q.double() * 2.0 ** -126).to(torch.bfloat16)  # down to the least normal numbers
    want = A.attention_decode(f64(b.q), b.keys, b.values, 2.0 ** 123)
    assert_within(f64(b.run(lib, cuda, scale=2.0 ** 123)), want["out"], bound(want), f"2^{power - 126}")


@pytest.mark.parametrize("spread", [5.0, 20.0])
def test_key_scales_far_apart(lib, cuda, spread):
    # blocks whose key scales lie apart by up to e^(2 spread), queries that keep the largest
    # scores moderate: several keys of the large blocks share the weight with all the small ones
    b = Batch(8, 2, 64, 16, 8, [200, 33, 1, 40], 45, spread=spread)
    scale = 0.125 * 8 * np.exp(-spread)
    ref = b.want(scale)
    scores = max(np.abs(k[:, h // 4] @ f64(b.q)[i, h]).max() * scale for i, k in enumerate(b.keys) for h in range(8))
    assert 1 < scores < 64
    out, lse = b.run(lib, cuda, save_lse=True, scale=float(scale))
    assert_within(f64(out), ref["out"], bound(ref), f"{spread}")
    assert_lse(lse.cpu().numpy(), ref, 200, 64, f"{spread}")


def test_a_length_beyond_the_table_attends_what_the_table_names(lib, cuda):
    b = Batch(8, 2, 64, 16, 8, [40, 96, 7], 46)
    b.table = b.table[:, :6]
    b.lengths[0] = 1 << 30
    b.table[0, 3:] = (-1, 1 << 20, 1 << 30)  # no pages of the pool: nothing there is attended
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    # (the oracle's keys of row 0: its three pages, the last of which holds 8 tokens and NaN codes behind them)
    b.codes[0][b.table[0, 2], 8:], b.codes[1][b.table[0, 2], 8:] = 0, E8.to_e4m3(np.float64(3.0))
    for s in b.scale:
        s[b.table[0, 2], 1] = 0.5
    keys, values = np.zeros((48, 2, 64)), np.full((48, 2, 64), 1.5)
    keys[:40], values[:40] = b.keys[0], b.values[0]
    b.keys[0], b.values[0] = keys, values
    ref = b.want()
    out, lse = b.run(lib, cuda, save_lse=True, dev_status=status)
    assert_within(f64(out), ref["out"], bound(ref), "rows")
    assert_lse(lse.cpu().numpy(), ref, 96, 64, "rows")
    assert int(status) == lib.QKVP_DEV_BAD_LENGTH | lib.QKVP_DEV_BAD_PAGE
