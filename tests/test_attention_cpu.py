"""Attention without a GPU: the float64 oracle against differences, closed forms
and its own symmetries, and the entry points' refusals (fake addresses that
nothing dereferences; only where no CUDA device is visible)."""

import numpy as np
import pytest
import torch

import oracle.attention as A

P = 0x10000  # a 16-byte aligned fake device address


def _no_gpu():
    try:
        return not torch.cuda.is_available()
    except Exception:
        return True


cpu_only = pytest.mark.skipif(not _no_gpu(), reason="fake-pointer argument checks run only without a GPU")


def _case(lengths, n_q, n_kv, D, seed, before=0, after=0):
    rng = np.random.default_rng(seed)
    cu = np.cumsum([before] + list(lengths))
    T = int(cu[-1]) + after
    return cu, [rng.normal(size=(T, n, D)) for n in (n_q, n_kv, n_kv, n_q)]


def test_oracle_single_key_and_two_keys():
    cu, (q, k, v, _) = _case([1, 2], 4, 2, 8, 1)
    r = A.attention_fwd(q, k, v, cu, 0.5)
    for h in range(4):
        g = h // 2
        assert np.allclose(r["out"][0, h], v[0, g]) and np.allclose(r["lse"][h, 0], 0.5 * q[0, h] @ k[0, g])
        a, b = 0.5 * q[2, h] @ k[1, g], 0.5 * q[2, h] @ k[2, g]
        w = 1 / (1 + np.exp(a - b))
        assert np.allclose(r["out"][2, h], (1 - w) * v[1, g] + w * v[2, g])
        assert np.allclose(r["lse"][h, 2], np.logaddexp(a, b))


def test_oracle_gradients_against_differences():
    cu, (q, k, v, do) = _case([3, 0, 5], 4, 2, 6, 2, before=1, after=1)
    z = A.attention_bwd(do, q, k, v, cu)
    rng = np.random.default_rng(3)
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for _ in range(12):
            i = tuple(rng.integers(n) for n in x.shape)
            keep, step = x[i], 1e-6
            x[i] = keep + step
            up = (A.attention_fwd(q, k, v, cu)["out"] * do).sum()
            x[i] = keep - step
            down = (A.attention_fwd(q, k, v, cu)["out"] * do).sum()
            x[i] = keep
            assert abs((up - down) / (2 * step) - z[name][i]) < 1e-7, (name, i)


def test_oracle_rows_of_no_sequence():
    cu, (q, k, v, do) = _case([4, 2], 2, 1, 4, 4, before=2, after=3)
    r, z = A.attention_fwd(q, k, v, cu), A.attention_bwd(do, q, k, v, cu)
    rest = [0, 1, 8, 9, 10]
    assert not r["out"][rest].any() and np.isneginf(r["lse"][:, rest]).all()
    assert not any(z[n][rest].any() for n in ("dq", "dk", "dv"))


def test_oracle_decode_is_the_last_row_of_the_prompt():
    cu, (q, k, v, _) = _case([9], 6, 3, 8, 5)
    r = A.attention_fwd(q, k, v, cu)
    d = A.attention_decode(q[-1:], [k], [v])
    assert np.allclose(d["out"][0], r["out"][-1]) and np.allclose(d["lse"][0], r["lse"][:, -1])
    none = A.attention_decode(q[-1:], [k[:0]], [v[:0]])
    assert not none["out"].any() and np.isneginf(none["lse"]).all()


def test_oracle_heads_share_keys_by_group():
    cu, (q, k, v, do) = _case([7], 6, 2, 4, 6)
    wide = [np.repeat(x, 3, axis=1) for x in (k, v)]
    a, b = A.attention_fwd(q, k, v, cu), A.attention_fwd(q, *wide, cu)
    assert np.array_equal(a["out"], b["out"])
    za, zb = A.attention_bwd(do, q, k, v, cu), A.attention_bwd(do, q, *wide, cu)
    for n in ("dk", "dv"):
        assert np.allclose(za[n], zb[n].reshape(7, 2, 3, 4).sum(axis=2))


# ------------------------------------------------------------- refusals ----

def _fwd(C, L=None, T=4, batch=1, cu=P, q=P, k=P, v=P, scale=0.0, flags=0, out=P, lse=None, status=None):
    L = L or C.layout("sectioned", 8, 2, 64)
    return C.qkv_attention_fwd(L, T, batch, cu, q, k, v, scale, flags, out, lse, status, stream=0, check=False)


@cpu_only
def test_forward_refusals(lib):
    C = lib
    assert _fwd(C) == C.QKVP_ERR_ARCH  # valid arguments: it gets as far as the device check
    assert _fwd(C, L=C.layout("interleaved", 7, 7, 128), flags=C.QKVP_ZERO_REST, lse=P) == C.QKVP_ERR_ARCH
    assert _fwd(C, T=0) == C.QKVP_OK
    assert _fwd(C, T=-1) == C.QKVP_ERR_SHAPE
    assert _fwd(C, T=2 ** 31) == C.QKVP_ERR_SHAPE
    assert _fwd(C, batch=-1) == C.QKVP_ERR_SHAPE and _fwd(C, batch=2 ** 20 + 1) == C.QKVP_ERR_SHAPE
    assert _fwd(C, batch=0) == C.QKVP_ERR_ARCH
    for bad in (C.layout("sectioned", 8, 3, 64), C.layout("sectioned", 8, 2, 96), C.layout("sectioned", 0, 2, 64),
                C.layout("latent", norm_dim=512, rope_dim=64)):
        assert _fwd(C, L=bad) == C.QKVP_ERR_SHAPE
    for scale in (-1.0, float("nan"), float("inf")):
        assert _fwd(C, scale=scale) == C.QKVP_ERR_VALUE
    for flags in (1, 64, C.QKVP_ZERO_REST | C.QKVP_NORM_OFF):
        assert _fwd(C, flags=flags) == C.QKVP_ERR_FLAGS
    for name in ("cu", "q", "k", "v", "out"):
        assert _fwd(C, **{name: None}) == C.QKVP_ERR_NULL
    for name in ("q", "k", "v", "out"):
        assert _fwd(C, **{name: P + 8}) == C.QKVP_ERR_ALIGN
    for name in ("cu", "lse", "status"):
        assert _fwd(C, **{name: P + 2}) == C.QKVP_ERR_ALIGN


@cpu_only
def test_backward_refusals(lib):
    C = lib
    L = C.layout("sectioned", 8, 2, 64)
    # delta [n_q, T], and the sums of the group's four heads apart: [4, dv and dk, T, n_kv, D]
    need = C.qkv_attention_bwd_workspace(L, 4, 1)
    assert need == 4 * (8 * 4 + 4 * 2 * 4 * 2 * 64) and C.qkv_attention_bwd_workspace(L, 0, 1) == 0
    assert C.qkv_attention_bwd_workspace(C.layout("sectioned", 32, 8, 128), 8192, 1) == 4 * 32 * 8192  # one part
    assert C.qkv_attention_bwd_workspace(C.layout("sectioned", 5, 5, 128), 100, 3) == 4 * 5 * 100  # no group to divide
    assert C.qkv_attention_bwd_workspace(L, -1, 1, check=False) == C.QKVP_ERR_SHAPE
    assert C.qkv_attention_bwd_workspace(L, 4, -1, check=False) == C.QKVP_ERR_SHAPE

    def bwd(**kw):
        a = dict(L=L, T=4, batch=1, cu=P, do=P, q=P, k=P, v=P, out=P, lse=P, scale=0.0, flags=0, dq=P, dk=P, dv=P,
                 status=None, ws=P, n=need)
        a.update(kw)
        return C.qkv_attention_bwd(a["L"], a["T"], a["batch"], a["cu"], a["do"], a["q"], a["k"], a["v"], a["out"],
                                   a["lse"], a["scale"], a["flags"], a["dq"], a["dk"], a["dv"], a["status"], a["ws"],
                                   a["n"], stream=0, check=False)

    assert bwd() == C.QKVP_ERR_ARCH
    assert bwd(T=0, ws=None, n=0) == C.QKVP_OK
    assert bwd(T=-1) == C.QKVP_ERR_SHAPE
    assert bwd(L=C.layout("sectioned", 8, 2, 80)) == C.QKVP_ERR_SHAPE
    assert bwd(flags=16) == C.QKVP_ERR_FLAGS
    assert bwd(scale=-0.5) == C.QKVP_ERR_VALUE
    for name in ("cu", "do", "q", "k", "v", "out", "lse", "dq", "dk", "dv"):
        assert bwd(**{name: None}) == C.QKVP_ERR_NULL
    for name in ("do", "q", "k", "v", "out", "dq", "dk", "dv", "ws"):
        assert bwd(**{name: P + 8}) == C.QKVP_ERR_ALIGN
    assert bwd(ws=None) == C.QKVP_ERR_WORKSPACE and bwd(n=need - 1) == C.QKVP_ERR_WORKSPACE


@cpu_only
def test_decode_refusals(lib):
    C = lib
    L = C.layout("sectioned", 8, 2, 64)

    def dec(**kw):
        a = dict(L=L, B=3, q=P, k=P, v=P, pages=9, size=16, table=P, most=4, stride=4, lengths=P, prefix=None, n=0,
                 scale=0.0, out=P, lse=None, status=None, ws=P, nb=1 << 30)
        a.update(kw)
        return C.qkv_attention_decode(a["L"], a["B"], a["q"], a["k"], a["v"], a["pages"], a["size"], a["table"],
                                      a["most"], a["stride"], a["lengths"], a["prefix"], a["n"], a["scale"], a["out"],
                                      a["lse"], a["status"], a["ws"], a["nb"], stream=0, check=False)

    assert dec() == C.QKVP_ERR_ARCH
    assert dec(B=0) == C.QKVP_OK
    assert dec(n=100, prefix=P, most=0, stride=0, table=None) == C.QKVP_ERR_ARCH
    assert dec(B=-1) == C.QKVP_ERR_SHAPE and dec(B=2 ** 20 + 1) == C.QKVP_ERR_SHAPE
    assert dec(most=-1) == C.QKVP_ERR_SHAPE and dec(stride=3) == C.QKVP_ERR_SHAPE
    assert dec(n=-1, prefix=P) == C.QKVP_ERR_SHAPE
    assert dec(most=2 ** 28, stride=2 ** 28) == C.QKVP_ERR_SHAPE  # more keys than 31 bits
    assert dec(L=C.layout("sectioned", 8, 2, 32)) == C.QKVP_ERR_SHAPE
    assert dec(pages=0) == C.QKVP_ERR_VALUE and dec(size=0) == C.QKVP_ERR_VALUE
    assert dec(pages=2 ** 30) == C.QKVP_ERR_VALUE  # pool rows beyond 31 bits
    assert dec(scale=float("inf")) == C.QKVP_ERR_VALUE
    for name in ("q", "k", "v", "lengths", "out", "table"):
        assert dec(**{name: None}) == C.QKVP_ERR_NULL
    assert dec(n=5) == C.QKVP_ERR_NULL  # a prefix without its pages
    for name in ("q", "k", "v", "out"):
        assert dec(**{name: P + 8}) == C.QKVP_ERR_ALIGN
    for name in ("lengths", "table", "lse", "status"):
        assert dec(**{name: P + 2}) == C.QKVP_ERR_ALIGN
    ws = C.qkv_attention_decode_workspace
    assert ws(L, 3, 16, 4, 0, check=False) == C.QKVP_ERR_ARCH  # the split depends on the device
    assert ws(L, 0, 16, 4, 0) == 0
    assert ws(L, 3, 0, 4, 0, check=False) == C.QKVP_ERR_VALUE


@cpu_only
def test_functional_refuses_cpu_tensors_and_shapes(lib):
    F = lib.functional
    bf = dict(dtype=torch.bfloat16)
    q, k = torch.zeros(4, 8, 64, **bf), torch.zeros(4, 2, 64, **bf)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    for args in ((q, k, k, cu), (q.float(), k, k, cu), (q, k[:, :, :32], k, cu), (q, k[:3], k[:3], cu),
                 (q.transpose(0, 1), k, k, cu)):
        with pytest.raises(ValueError):
            F.attention_forward(*args)
    pool = torch.zeros(3, 16, 2, 64, **bf)
    table, n = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    for args in ((q, pool, pool, table, n), (q, pool, pool[:2], table, n), (q.float(), pool, pool, table, n)):
        with pytest.raises(ValueError):
            F.attention_decode(*args)
