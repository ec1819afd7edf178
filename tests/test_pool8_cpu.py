"""The 8-bit pool without a GPU: pins of the oracle, and the host's refusals."""

import numpy as np
import pytest
import torch

import oracle.pool8 as E
from test_abi_cpu import cpu_only

A = 0x10000  # fake device addresses, far from each other (never dereferenced)
B = [A + (i << 32) for i in range(16)]


def test_e4m3_is_torch_s():
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(E.VALUES, codes.view(torch.float8_e4m3fn).double().numpy(), equal_nan=True)
    g = np.random.default_rng(1)
    x = np.concatenate([g.standard_normal(20000) * 10.0 ** g.integers(-4, 3, 20000), E.VALUES[:127],
                        (E.VALUES[:126] + E.VALUES[1:127]) / 2, -(E.VALUES[:126] + E.VALUES[1:127]) / 2, [-0.0]])
    x = np.clip(x, -448, 448).astype(np.float32).astype(np.float64)
    want = torch.from_numpy(x).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(E.to_e4m3(x), want)
    assert E.to_e4m3(1e9) == 126 and E.to_e4m3(np.nan) == 127
    assert np.all(np.abs(E.VALUES[E.to_e4m3(x)] - x) <= E.half_step(x, 1.0))


def test_append_by_hand():
    codes, scale = np.zeros((1, 4, 1, 2), np.uint8), np.ones((1, 2, 1))
    x = np.array([[[448.0, -7.0]], [[3.0, 896.0]]])
    codes, scale = E.append(codes, scale, x[:1], [0], [0])
    assert scale[0, 0, 0] == 1.0 and E.VALUES[codes[0, 0, 0]].tolist() == [448.0, -7.0]
    codes, scale = E.append(codes, scale, x[1:], [0], [1])  # grows by two: the held codes are halved
    assert scale[0].ravel().tolist() == [2.0, 1.0]
    assert E.VALUES[codes[0, 0, 0]].tolist() == [224.0, -3.5] and E.VALUES[codes[0, 1, 0]].tolist() == [1.5, 448.0]
    codes, scale = E.append(codes, scale, np.zeros((1, 1, 2)), [0], [0])  # begins the block again
    assert scale[0, 0, 0] == 2.0 ** -100 and E.VALUES[codes[0, 1, 0]].tolist() == [1.5, 448.0]
    assert E.grow(448.0, 1.0) == 0 and E.grow(448.1, 1.0) == 1 and E.grow(896.0, 1.0) == 1 and E.grow(0.0, 1.0) == 0


def _write(C, L=None, V=None, T=4, packed=B[0], pos=B[1], wq=B[2], wk=B[3], eps=1e-6, base=1e4, flags=0, q=B[4],
           page=B[5], off=B[6], kp=B[7], vp=B[8], ks=B[9], vs=B[10], pages=64, size=16, block=8, status=None):
    L = L or C.layout("interleaved", 8, 2, 64)
    return C.qkv_prologue_pool_write8(L, V, T, packed, pos, wq, wk, eps, base, flags, q, page, off, kp, vp, ks, vs, pages,
                                      size, block, status, stream=0, check=False)


@cpu_only
def test_write_refusals(lib):
    C = lib
    ok = C.QKVP_ERR_ARCH  # as far as the device check
    assert _write(C) == ok and _write(C, T=0) == C.QKVP_OK
    for block in (1, 2, 4, 8, 16):
        assert _write(C, block=block) == ok
    for bad in (dict(block=0), dict(block=-1), dict(block=3), dict(block=32), dict(size=0), dict(pages=0),
                dict(pages=1 << 20, size=1 << 12), dict(eps=-1.0), dict(base=0.0), dict(eps=float("nan"))):
        assert _write(C, **bad) == C.QKVP_ERR_VALUE, bad
    for name in ("packed", "pos", "wq", "wk", "q", "page", "off", "kp", "vp", "ks", "vs"):
        assert _write(C, **{name: None}) == C.QKVP_ERR_NULL, name
    for name in ("packed", "wq", "q", "kp", "vp"):
        assert _write(C, **{name: B[15] + 8}) == C.QKVP_ERR_ALIGN, name
    for name in ("pos", "page", "off", "ks", "vs", "status"):
        assert _write(C, **{name: B[15] + 2}) == C.QKVP_ERR_ALIGN, name
    assert _write(C, pos=None, flags=C.QKVP_NOPE) == ok
    assert _write(C, wq=None, wk=None, flags=C.QKVP_NORM_OFF) == ok
    assert _write(C, flags=C.QKVP_ROPE_PAIRS) == ok
    assert _write(C, L=C.layout("sectioned", 8, 2, 64, rope_dim=32), flags=C.QKVP_ROPE_PART) == ok
    assert _write(C, L=C.layout("sectioned", 8, 2, 64, rope_dim=24), flags=C.QKVP_ROPE_PART) == C.QKVP_ERR_SHAPE
    for flags in (C.QKVP_SAVE_PRE, C.QKVP_FORCE_GENERIC, C.QKVP_ACCUMULATE_DW, C.QKVP_ZERO_REST, 256,
                  C.QKVP_NOPE | C.QKVP_ROPE_PAIRS):
        assert _write(C, flags=flags) == C.QKVP_ERR_FLAGS
    assert _write(C, L=C.layout("latent", norm_dim=512, rope_dim=64)) == C.QKVP_ERR_SHAPE
    assert _write(C, L=C.layout("interleaved", 8, 2, 96)) == C.QKVP_ERR_SHAPE
    assert _write(C, T=-1) == C.QKVP_ERR_SHAPE


def _decode(C, L=None, batch=3, q=B[0], kp=B[1], vp=B[2], ks=B[3], vs=B[4], pages=64, size=16, block=8, table=B[5],
            most=4, stride=4, lengths=B[6], scale=0.0, out=B[7], lse=None, status=None, ws=B[8], wsb=1 << 30):
    L = L or C.layout("interleaved", 8, 2, 64)
    return C.qkv_attention_decode8(L, batch, q, kp, vp, ks, vs, pages, size, block, table, most, stride, lengths, scale,
                                   out, lse, status, ws, wsb, stream=0, check=False)


@cpu_only
def test_decode_refusals(lib):
    C = lib
    ok = C.QKVP_ERR_ARCH
    assert _decode(C) == ok and _decode(C, batch=0) == C.QKVP_OK
    for bad in (dict(block=0), dict(block=5), dict(pages=0), dict(size=0), dict(scale=-1.0), dict(scale=float("inf"))):
        assert _decode(C, **bad) == C.QKVP_ERR_VALUE, bad
    for bad in (dict(batch=-1), dict(batch=(1 << 20) + 1), dict(most=-1), dict(stride=3), dict(most=1 << 28, stride=1 << 28),
                dict(L=C.layout("interleaved", 8, 3, 64)), dict(L=C.layout("interleaved", 8, 2, 32))):
        assert _decode(C, **bad) == C.QKVP_ERR_SHAPE, bad
    for name in ("q", "kp", "vp", "ks", "vs", "table", "lengths", "out"):
        assert _decode(C, **{name: None}) == C.QKVP_ERR_NULL, name
    for name in ("q", "kp", "vp", "out"):
        assert _decode(C, **{name: B[15] + 8}) == C.QKVP_ERR_ALIGN, name
    for name in ("ks", "vs", "table", "lengths", "lse", "status"):
        assert _decode(C, **{name: B[15] + 2}) == C.QKVP_ERR_ALIGN, name
    assert C.qkv_attention_decode8_workspace(C.layout("interleaved", 8, 2, 64), 0, 16, 4) == 0
    assert C.qkv_attention_decode8_workspace(C.layout("interleaved", 8, 2, 64), -1, 16, 4, check=False) == C.QKVP_ERR_SHAPE


def test_tensor_checks(lib):
    F, f8 = lib.functional, torch.float8_e4m3fn
    pool = torch.zeros(4, 16, 2, 64, dtype=f8)
    scale = torch.zeros(4, 2, 2)
    assert F._check_pool8(pool, pool, scale, scale, pool.device) == 8
    for k, s in ((pool.view(torch.uint8), scale), (pool[:, :8], scale), (pool[0], scale), (pool, scale.double()),
                 (pool, torch.zeros(4, 3, 2)), (pool, torch.zeros(4, 2, 1)), (pool, torch.zeros(3, 2, 2)),
                 (pool, torch.zeros(4, 0, 2)), (pool, scale[:, :, :1].expand(4, 2, 2)), (pool, torch.zeros(4, 32, 2))):
        with pytest.raises(ValueError):
            F._check_pool8(k, k, s, s, pool.device)
    with pytest.raises(ValueError):
        F._check_pool8(pool, torch.zeros(5, 16, 2, 64, dtype=f8), scale, scale, pool.device)
    cpu = torch.zeros(1, 12 * 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        F.prologue_pool_write8(cpu, None, None, None, None, None, pool, pool, scale, scale, 8, 2)
    with pytest.raises(ValueError, match="CUDA"):
        F.attention_decode8(torch.zeros(1, 8, 64, dtype=torch.bfloat16), pool, pool, scale, scale, None, None)
