"""Attention in float64 from its definition: causal over packed sequences with
its gradients, and single query rows over paged keys. One sequence and one
query head at a time, every score formed; shares no code with the kernels.

Inputs are float64 arrays (the values of the bf16 tensors). Each function also
returns the sums of absolute values that error bounds are made of, so that a
test can bound a kernel's rounding element by element.
"""

import numpy as np


def _softmax_rows(s):
    """Softmax and log-sum-exp of each row; a row of -inf gives zeros and -inf."""
    top = s.max(axis=1, keepdims=True) if s.shape[1] else np.full((s.shape[0], 1), -np.inf)
    safe = np.where(np.isfinite(top), top, 0.0)
    e = np.exp(s - safe)
    total = e.sum(axis=1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (safe + np.log(total))[:, 0]
    return e / np.where(total > 0, total, 1.0), lse


def attention_fwd(q, k, v, cu, scale=None):
    """q [T, n_q, D], k, v [T, n_kv, D], cu [batch + 1]. Returns out [T, n_q, D]
    and lse [n_q, T] (zeros and -inf for rows of no sequence), out_abs =
    sum_j p_ij |v_j| and s_abs [n_q, T] = max_j scale sum_d |q_d k_d|."""
    T, n_q, D = q.shape
    G = n_q // k.shape[1]
    scale = D ** -0.5 if scale is None else scale
    out, out_abs = np.zeros((T, n_q, D)), np.zeros((T, n_q, D))
    lse, s_abs = np.full((n_q, T), -np.inf), np.zeros((n_q, T))
    for a, b in zip(cu[:-1], cu[1:]):
        later = np.triu(np.ones((b - a, b - a), dtype=bool), 1)
        for h in range(n_q if b > a else 0):
            kh, vh = k[a:b, h // G], v[a:b, h // G]
            s = q[a:b, h] @ kh.T * scale
            s[later] = -np.inf
            p, lse[h, a:b] = _softmax_rows(s)
            out[a:b, h] = p @ vh
            out_abs[a:b, h] = p @ np.abs(vh)
            s_abs[h, a:b] = (np.abs(q[a:b, h]) @ np.abs(kh).T).max(axis=1) * scale
    return {"out": out, "lse": lse, "out_abs": out_abs, "s_abs": s_abs}


def attention_bwd(dout, q, k, v, cu, scale=None, out_err=None):
    """Gradients (dq, dk, dv) of sum(out * dout). With out_err [T, n_q, D], a
    bound on the saved output's error, also e_dq, e_dk, e_dv: the gradients'
    error bounds when every weight p and every score gradient ds is rounded
    with relative error `r` (r = 2^-8 + 2^-10, bf16 and the fp32 arithmetic
    around it), delta_i = dout_i . out_i is taken with the saved output, and
    dp_ij = dout_i . v_j has relative error 2^-16 of sum_d |dout_d v_d|."""
    T, n_q, D = q.shape
    n_kv = k.shape[1]
    G = n_q // n_kv
    scale = D ** -0.5 if scale is None else scale
    r = 2.0 ** -8 + 2.0 ** -10
    z = {n: np.zeros_like(x) for n, x in (("dq", q), ("dk", k), ("dv", v), ("e_dq", q), ("e_dk", k), ("e_dv", v))}
    for a, b in zip(cu[:-1], cu[1:]):
        later = np.triu(np.ones((b - a, b - a), dtype=bool), 1)
        for h in range(n_q if b > a else 0):
            g = h // G
            qh, kh, vh, do = q[a:b, h], k[a:b, g], v[a:b, g], dout[a:b, h]
            s = qh @ kh.T * scale
            s[later] = -np.inf
            p, _ = _softmax_rows(s)
            out = p @ vh
            dp = do @ vh.T
            ds = p * (dp - (do * out).sum(axis=1, keepdims=True))
            z["dv"][a:b, g] += p.T @ do
            z["dq"][a:b, h] = ds @ kh * scale
            z["dk"][a:b, g] += ds.T @ qh * scale
            if out_err is not None:
                d_delta = (np.abs(do) * out_err[a:b, h]).sum(axis=1, keepdims=True)
                e_ds = r * np.abs(ds) + p * (d_delta + 2.0 ** -16 * (np.abs(do) @ np.abs(vh).T))
                z["e_dv"][a:b, g] += r * (p.T @ np.abs(do))
                z["e_dq"][a:b, h] = e_ds @ np.abs(kh) * scale
                z["e_dk"][a:b, g] += e_ds.T @ np.abs(qh) * scale
    return z


def attention_decode(q, keys, values, scale=None):
    """One query row per sequence: q [B, n_q, D]; keys[b], values[b] [n_b, n_kv, D]
    in the order they are attended (n_b may be 0). Returns out [B, n_q, D] (zeros
    without keys), lse [B, n_q], out_abs."""
    B, n_q, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    out, out_abs, lse = np.zeros((B, n_q, D)), np.zeros((B, n_q, D)), np.full((B, n_q), -np.inf)
    for b in range(B):
        n = keys[b].shape[0]
        for h in range(n_q if n else 0):
            g = h // (n_q // keys[b].shape[1])
            p, ls = _softmax_rows((keys[b][:, g] @ q[b, h] * scale)[None, :])
            lse[b, h] = ls[0]
            out[b, h] = p[0] @ values[b][:, g]
            out_abs[b, h] = p[0] @ np.abs(values[b][:, g])
    return {"out": out, "lse": lse, "out_abs": out_abs}
