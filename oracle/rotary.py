"""Rotary layouts in float64 from their definition: the first R values of a head
rotated pair by pair, the pairs (i, i + R/2) or (2i, 2i + 1), the others left
alone; and the prologue and its gradient around it. Each pair is turned by its
own 2 x 2 matrix; shares no code with the kernels.
"""

import numpy as np

from .bf16 import bf16_bits_to_f64
from .prologue import add_bias, merge_heads, rms_norm, rms_norm_backward, split_heads


def pair_indices(R, adjacent):
    """(first, second) value of each of the R/2 pairs."""
    i = np.arange(R // 2)
    return (2 * i, 2 * i + 1) if adjacent else (i, i + R // 2)


def rotate(y, pos, R, adjacent, base, inv_freq=None, scale=1.0, transpose=False):
    """y [T, heads, D] with the first R values of each head rotated (transpose:
    by the transposed matrices), times `scale` on what is rotated."""
    y = np.asarray(y, dtype=np.float64)
    f = float(base) ** (-2.0 * np.arange(R // 2) / R) if inv_freq is None else np.asarray(inv_freq, dtype=np.float64)
    assert f.shape == (R // 2,)
    out = y.copy()
    a, b = pair_indices(R, adjacent)
    for t, p in enumerate(np.asarray(pos, dtype=np.float64)):
        c, s = np.cos(p * f) * scale, np.sin(p * f) * scale
        m = np.array([[c, -s], [s, c]])  # [2, 2, R/2]
        if transpose:
            m = m.transpose(1, 0, 2)
        pairs = np.stack([y[t][:, a], y[t][:, b]])  # [2, heads, R/2]
        turned = np.einsum("xyp,yhp->xhp", m, pairs)
        out[t][:, a], out[t][:, b] = turned[0], turned[1]
    return out


def prologue_fwd(layout, packed_bits, pos, w_q, w_k, eps, base, R, adjacent, norm=True, bias=None, inv_freq=None,
                 rope_scale=1.0):
    """float64 q, k, v of bf16 packed rows (uint16 bits)."""
    x = add_bias(bf16_bits_to_f64(np.asarray(packed_bits).reshape(-1, layout.row_width)), bias)
    q, k, v = split_heads(layout, x)
    if norm:
        q, k = rms_norm(q, w_q, eps), rms_norm(k, w_k, eps)
    return tuple(rotate(t, pos, R, adjacent, base, inv_freq, rope_scale) for t in (q, k)) + (v,)


def prologue_bwd(layout, dq, dk, dv, packed_bits, pos, w_q, w_k, eps, base, R, adjacent, norm=True, bias=None,
                 inv_freq=None, rope_scale=1.0):
    """float64 gradients of sum(q dq + k dk + v dv): dpacked, dw_q, dw_k (None
    without the norm) and dbias (summed over tokens)."""
    x = add_bias(bf16_bits_to_f64(np.asarray(packed_bits).reshape(-1, layout.row_width)), bias)
    xq, xk, _ = split_heads(layout, x)
    gq, gk = (rotate(t, pos, R, adjacent, base, inv_freq, rope_scale, transpose=True) for t in (dq, dk))
    dw_q = dw_k = None
    if norm:
        gq, tq = rms_norm_backward(xq, w_q, gq, eps)
        gk, tk = rms_norm_backward(xk, w_k, gk, eps)
        dw_q, dw_k = tq.sum((0, 1)), tk.sum((0, 1))
    dpacked = merge_heads(layout, gq, gk, np.asarray(dv, dtype=np.float64))
    return dpacked, dw_q, dw_k, dpacked.sum(0)
