"""Error bounds of the attention kernels against the float64 oracle.

bf16 rounds with relative error at most u = 2^-8 (half a step), fp32 with 2^-24.

out_i = sum_j p_ij v_j / l_i. Each p_ij is rounded to bf16 (u); around that the
kernel works in fp32: a score is a sum of D products in fp32 (relative to
sum_d |q_d k_d| at most (D + 2) 2^-24; tensor-core sums may truncate, which
doubles that), and e^x is taken of an argument with a relative rounding of
2^-24 a few times over. With scores up to 2^6 in magnitude the weights' fp32
error stays below 2^-10, for numerator and denominator together, hence

    |out - exact| <= u |exact| + (u + 2^-10) (1 + u) sum_j p_ij |v_j|.

lse_i: the score errors, the e^x errors (2^-22) and a sum of n terms in fp32,
in chunks: |lse - exact| <= 2^-24 (2 (D + 4) s_abs + 4 |lse| + n / 2 + 64).
The tests stay below 2^6 in s_abs and 4096 in n.

Gradients: the bounds that oracle.attention_bwd forms, plus the result's own
rounding u |exact|.
"""

import numpy as np

U = 2.0 ** -8
EDGE = 2.0 ** -10


def out_bound(ref):
    return U * np.abs(ref["out"]) + (U + EDGE) * (1 + U) * ref["out_abs"]


def assert_within(got, exact, bound, what):
    got, exact, bound = (np.asarray(x, dtype=np.float64) for x in (got, exact, bound))
    assert got.shape == exact.shape, (what, got.shape, exact.shape)
    assert np.all(np.isfinite(got)), f"{what}: non-finite values"
    over = np.abs(got - exact) - bound
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else None
    assert over.size == 0 or over[at] <= 1e-30, (
        f"{what}: at {at} got {got[at]:.6g}, exact {exact[at]:.6g}, bound {bound[at]:.3g}; "
        f"{int((over > 1e-30).sum())} of {over.size} values beyond their bound")


def assert_lse(got, ref, n, D, what):
    got = np.asarray(got, dtype=np.float64)
    none = np.isneginf(ref["lse"])
    assert np.array_equal(np.isneginf(got), none), f"{what}: rows without keys"
    s_abs = ref.get("s_abs", np.full_like(ref["lse"], 64.0))
    lse = np.where(none, 0.0, ref["lse"])
    bound = 2.0 ** -24 * (2 * (D + 4) * s_abs + 4 * np.abs(lse) + n / 2 + 64)
    assert_within(np.where(none, 0.0, got), lse, bound, what)
