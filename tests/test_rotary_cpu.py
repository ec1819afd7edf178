"""The rotary layouts without a GPU: pins of the oracle, and the host's refusals."""

import numpy as np
import pytest

import oracle.prologue as P
import oracle.rotary as R
import workloads
from oracle.bf16 import to_bf16_rne
from test_abi_cpu import cpu_only
from workloads import bits_u16 as u16

A = 0x10000  # a fake device address (never dereferenced)


def test_halves_of_the_whole_head_is_rotate_half(rng):
    y, pos = rng.standard_normal((5, 3, 64)), rng.integers(0, 1 << 17, 5)
    want = P.rope_rotate_half(y, pos, 1e4, scale=1.25)
    assert np.allclose(R.rotate(y, pos, 64, False, 1e4, scale=1.25), want, rtol=0, atol=1e-12)


@pytest.mark.parametrize("dim", [16, 48, 64])
def test_pairs_are_halves_in_another_order(rng, dim):
    y, pos = rng.standard_normal((4, 2, 64)), rng.integers(0, 1000, 4)
    order = np.arange(64)
    order[:dim] = np.concatenate([np.arange(0, dim, 2), np.arange(1, dim, 2)])
    halves = R.rotate(y[..., order], pos, dim, False, 1e4)
    back = np.empty_like(y)
    back[..., order] = halves
    assert np.allclose(R.rotate(y, pos, dim, True, 1e4), back, rtol=0, atol=1e-13)


@pytest.mark.parametrize("adjacent", [False, True])
def test_rotation_is_that_of_a_complex_number(rng, adjacent):
    y, pos = rng.standard_normal((3, 2, 128)), np.array([0, 1, 131071])
    got = R.rotate(y, pos, 96, adjacent, 5e5, scale=0.75)
    a, b = R.pair_indices(96, adjacent)
    z = (y[..., a] + 1j * y[..., b]) * 0.75 * np.exp(1j * pos[:, None, None] * 5e5 ** (-2 * np.arange(48) / 96))
    assert np.allclose(got[..., a] + 1j * got[..., b], z, rtol=0, atol=1e-10)
    assert np.array_equal(got[..., 96:], y[..., 96:])  # untouched, the factor too
    assert np.allclose(R.rotate(got, pos, 96, adjacent, 5e5, scale=1 / 0.75, transpose=True), y, rtol=0, atol=1e-10)


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("adjacent", [False, True])
def test_gradient_against_differences(adjacent, norm):
    wl = workloads.gqa_inputs(3, 4, 2, 64, seed=9, rope_base=1e4, pos_high=5000, with_grads=True)
    L = P.PackedLayout("interleaved", 4, 2, 64)
    bits, pos = u16(wl.packed_rows()), wl.pos.numpy()
    w_q, w_k = (w.numpy().astype(np.float64) for w in (wl.w_q, wl.w_k))
    d = [P.bf16_bits_to_f64(u16(t)) for t in (wl.dq, wl.dk, wl.dv)]
    bias = np.linspace(-1, 1, L.row_width)
    opts = dict(norm=norm, rope_scale=1.1)

    def loss(b, wq, wk):
        out = R.prologue_fwd(L, bits, pos, wq, wk, 1e-6, 1e4, 32, adjacent, bias=b, **opts)
        return sum((o * g).sum() for o, g in zip(out, d))

    _, dw_q, dw_k, db = R.prologue_bwd(L, *d, bits, pos, w_q, w_k, 1e-6, 1e4, 32, adjacent, bias=bias, **opts)
    h = 1e-5
    for i in (0, 5, 31, 40, 63, 64 * 4 + 3, L.row_width - 1):  # through the bias: d(packed) summed over tokens
        e = np.zeros(L.row_width)
        e[i] = h
        assert (loss(bias + e, w_q, w_k) - loss(bias - e, w_q, w_k)) / (2 * h) == pytest.approx(db[i], rel=1e-6, abs=1e-6)
    if norm:
        for i in (0, 17, 63):
            e = np.zeros(64)
            e[i] = h
            assert (loss(bias, w_q + e, w_k) - loss(bias, w_q - e, w_k)) / (2 * h) == pytest.approx(dw_q[i], rel=1e-6)
            assert (loss(bias, w_q, w_k + e) - loss(bias, w_q, w_k - e)) / (2 * h) == pytest.approx(dw_k[i], rel=1e-6)


def test_flags_match_header(lib):
    import os
    import re

    src = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "qkv_prologue.h")).read()
    for name in ("QKVP_ROPE_PAIRS", "QKVP_ROPE_PART"):
        assert int(re.search(rf"\b{name}\s*=\s*(\d+)", src).group(1)) == getattr(lib, name)


@cpu_only
def test_refusals(lib):
    C = lib
    PAIRS, PART = C.QKVP_ROPE_PAIRS, C.QKVP_ROPE_PART

    def layout(rope_dim=0, kind="interleaved"):
        return C.layout(kind, 8, 2, 64, rope_dim=rope_dim)

    def fwd(flags, L):
        return C.qkv_prologue_fwd(L, 4, A, A, A, A, 1e-6, 1e4, flags, A, A, A, stream=0, check=False)

    def pool(flags, L):
        return C.qkv_prologue_pool_write(L, 4, A, A, A, A, 1e-6, 1e4, flags, A, A, A, A, A, 16, 16, stream=0, check=False)

    def bwd(flags, L):
        return C.qkv_prologue_bwd(L, 4, A, A, A, A, A, A, A, A, 1e-6, 1e4, flags, A, A, A, A, 1 << 20, stream=0,
                                  check=False)

    for call in (fwd, pool, bwd):
        ok = C.QKVP_ERR_ARCH  # as far as the device check
        assert call(PAIRS, layout()) == call(PAIRS, layout(24)) == ok  # without PART rope_dim is not looked at
        for dim in (16, 32, 48, 64):
            assert call(PART, layout(dim)) == call(PART | PAIRS, layout(dim, "sectioned")) == ok
        for dim in (0, 8, 24, 40, 80, 128, -16):
            assert call(PART, layout(dim)) == C.QKVP_ERR_SHAPE
        for flags in (PAIRS, PART, PAIRS | PART):
            assert call(flags | C.QKVP_NOPE, layout(32)) == C.QKVP_ERR_FLAGS
        assert call(256, layout()) == C.QKVP_ERR_FLAGS
    latent = C.layout("latent", norm_dim=512, rope_dim=64)
    for flags in (PAIRS, PART):
        assert C.qkv_prologue_fwd(latent, 4, A, A, None, A, 1e-6, 1e4, flags, None, A, None, stream=0,
                                  check=False) == C.QKVP_ERR_FLAGS
        assert C.qkv_prologue_gemm_fwd(layout(32), 4, 64, A, A, A, A, A, 1e-6, 1e4, flags, A, A, A, stream=0,
                                       check=False) == C.QKVP_ERR_FLAGS


@cpu_only
def test_the_caller_s_table_has_one_frequency_per_rotated_pair(lib):
    C = lib
    # 8 finite frequencies, and what lies behind them is not looked at
    V = C.variant(inv_freq=[1.0] * 8 + [float("nan")] * 24)
    part = C.layout("interleaved", 8, 2, 64, rope_dim=16)
    call = lambda flags, L: C.qkv_prologue_fwd_ex(L, V, 4, A, A, A, A, 1e-6, 1e4, flags, A, A, A, stream=0,  # noqa: E731
                                                  check=False)
    assert call(C.QKVP_ROPE_PART, part) == C.QKVP_ERR_ARCH
    assert call(0, part) == C.QKVP_ERR_VALUE
    assert C.qkv_prologue_bwd_workspace_size_ex(part, V, 4) == C.qkv_prologue_bwd_workspace_size(part, 4)
    with pytest.raises(ValueError, match="frequencies"):
        lib.functional._variant(inv_freq=[1.0] * 16, rotary_dim=16)
    assert lib.functional._variant(inv_freq=[1.0] * 8, rotary_dim=16) is not None


def test_oracle_is_not_the_old_one_by_another_name():
    # a part in pairs differs from a part in halves and from the whole head
    y = np.arange(64.0)[None, None]
    got = [R.rotate(y, [3], *a) for a in ((32, True, 1e4), (32, False, 1e4), (64, True, 1e4), (64, False, 1e4))]
    for i in range(4):
        for j in range(i):
            assert not np.array_equal(to_bf16_rne(got[i]), to_bf16_rne(got[j]))


def test_too_few_frequencies_are_refused(lib):
    F = lib.functional
    for dim, rot in ((64, None), (128, None), (64, 32), (128, 128)):
        n = (rot or dim) // 2
        assert F._variant(inv_freq=[0.5] * n, dim=dim, rotary_dim=rot) is not None
        with pytest.raises(ValueError, match="frequencies"):
            F._variant(inv_freq=[0.5] * (n - 1), dim=dim, rotary_dim=rot)
