"""Paths through the rotary layouts and the 8-bit pool that a model takes: a training
region with attention behind the prologue, the backward without an allocation, packed
rows that lie apart, layers that share one pool's calls on several streams."""

import numpy as np
import pytest
import torch

import oracle.attention as A
import oracle.pool8 as E8
import oracle.prologue as P
import oracle.rotary as R
import workloads
from oracle.bf16 import bf16_bits_to_f64
from parity import assert_bf16_close, assert_dw_close
from test_gpu_pool_write8 import Pool, _check_pool
from workloads import bits_u16 as u16

pytestmark = pytest.mark.gpu


def f64(t):
    return bf16_bits_to_f64(u16(t))


@pytest.mark.parametrize("rot, pairs", [(64, True), (32, False)])
def test_training_region(lib, cuda, rot, pairs):
    """packed -> rotary prologue -> packed attention -> gradients, against float64 from
    end to end. On the way q, k, v, out, dout's products and dq, dk, dv are rounded to
    bf16, and the weights and score gradients within attention. A score is then off by at
    most 2 u sum|q k| scale, about 2^-7 of scores up to 3, hence the weights by 2.4 %; the
    other roundings are 2^-8 each. 5 % of the whole tensor's norm bounds it."""
    n_q, n_kv, D, lengths = 4, 2, 64, [23, 1, 40]
    T = sum(lengths)
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=31, rope_base=1e4, pos_high=4096, with_grads=True)
    F = lib.functional
    cu = np.concatenate([[0], np.cumsum(lengths)])
    x = wl.packed_rows().to(cuda).requires_grad_()
    w_q, w_k = wl.w_q.to(cuda).requires_grad_(), wl.w_k.to(cuda).requires_grad_()
    q, k, v = F.GQAttentionPrologue.apply(x, wl.pos.to(cuda), w_q, w_k, None, n_q, n_kv, D, "interleaved", wl.eps,
                                          wl.rope_base, False, True, None, 1.0, rot, pairs)
    out = F.PackedAttention.apply(q, k, v, torch.tensor(cu, dtype=torch.int32, device=cuda))
    out.backward(wl.dq.to(cuda))  # (of out's shape)
    L = P.PackedLayout("interleaved", n_q, n_kv, D)
    w64 = (wl.w_q.numpy().astype(np.float64), wl.w_k.numpy().astype(np.float64))
    args = (u16(wl.packed_rows()), wl.pos.numpy(), *w64, wl.eps, wl.rope_base, rot, pairs)
    q64, k64, v64 = R.prologue_fwd(L, *args)
    ref = A.attention_fwd(q64, k64, v64, cu)
    g = A.attention_bwd(f64(wl.dq), q64, k64, v64, cu)
    dx, dw_q, dw_k, _ = R.prologue_bwd(L, g["dq"], g["dk"], g["dv"], *args)
    for name, got, want in (("out", f64(out), ref["out"]), ("dx", f64(x.grad), dx), ("dw_q", w_q.grad.cpu().numpy(), dw_q),
                            ("dw_k", w_k.grad.cpu().numpy(), dw_k)):
        off = np.linalg.norm(got - want) / np.linalg.norm(want)
        assert off <= 0.05, f"{name}: {off:.3g}"


@pytest.mark.parametrize("pairs", [False, True])
def test_backward_without_allocation(lib, cuda, pairs):
    C = lib
    wl = workloads.gqa_inputs(33, 8, 2, 64, seed=32, rope_base=1e4, pos_high=4096, with_grads=True)
    L = C.layout("interleaved", 8, 2, 64, rope_dim=48)
    flags = C.QKVP_ROPE_PART | (C.QKVP_ROPE_PAIRS if pairs else 0)
    dev = lambda t: t.to(cuda)  # noqa: E731
    out = C.functional.prologue_forward(dev(wl.packed_rows()), dev(wl.pos), dev(wl.w_q), dev(wl.w_k), 8, 2, 64,
                                        rope_base=1e4, save_pre=True, rotary_dim=48, rotary_pairs=pairs)
    dp = torch.empty(33, 12 * 64, dtype=torch.bfloat16, device=cuda)
    dw = [torch.empty(64, device=cuda) for _ in range(2)]
    C.qkv_prologue_bwd_noalloc(L, 33, dev(wl.dq), dev(wl.dk), dev(wl.dv), out[3], out[4], dev(wl.pos), dev(wl.w_q),
                               dev(wl.w_k), wl.eps, 1e4, flags, dp, *dw)
    oL = P.PackedLayout("interleaved", 8, 2, 64)
    w64 = (wl.w_q.numpy().astype(np.float64), wl.w_k.numpy().astype(np.float64))
    want = R.prologue_bwd(oL, f64(wl.dq), f64(wl.dk), f64(wl.dv), u16(wl.packed_rows()), wl.pos.numpy(), *w64, wl.eps, 1e4,
                          48, pairs)
    assert_bf16_close(u16(dp), want[0], "dpacked")
    for a, b in zip(dw, want[1:3]):
        assert_dw_close(a.cpu().numpy(), b, "dw")


def test_rows_apart_and_accumulated_gradients(lib, cuda):
    # row_stride of the C calls: forward, pool write in 8 bits, backward into rows apart, weight gradients added
    C, T, n_q, n_kv, D = lib, 21, 8, 2, 64
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=33, rope_base=1e4, pos_high=4096, with_grads=True)
    width, stride = 12 * 64, 12 * 64 + 40
    rows = torch.full((T, stride), float("nan"), dtype=torch.bfloat16, device=cuda)
    rows[:, :width] = wl.packed_rows().to(cuda)
    L = C.layout("interleaved", n_q, n_kv, D, row_stride=stride, rope_dim=32)
    flags = C.QKVP_ROPE_PART | C.QKVP_ROPE_PAIRS
    pos, w_q, w_k = wl.pos.to(cuda), wl.w_q.to(cuda), wl.w_k.to(cuda)
    want = C.functional.prologue_forward(rows[:, :width].contiguous(), pos, w_q, w_k, n_q, n_kv, D, rope_base=1e4,
                                         save_pre=True, rotary_dim=32, rotary_pairs=True)
    got = [torch.empty_like(t) for t in want]
    C.qkv_prologue_fwd(L, T, rows, pos, w_q, w_k, wl.eps, 1e4, flags | C.QKVP_SAVE_PRE, *got)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    pool = Pool(3, 16, 8, n_kv, D, cuda)
    before, before_scale = pool.read()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    page, offset = [t // 16 for t in range(T)], [t % 16 for t in range(T)]
    q = torch.empty_like(want[0])
    C.qkv_prologue_pool_write8(L, None, T, rows, pos, w_q, w_k, wl.eps, 1e4, flags, q, i32(page), i32(offset), *pool.args, 3,
                               16, 8)
    assert torch.equal(q, want[0])
    codes, scale = pool.read()
    oL = P.PackedLayout("interleaved", n_q, n_kv, D)
    w64 = (wl.w_q.numpy().astype(np.float64), wl.w_k.numpy().astype(np.float64))
    args = (u16(wl.packed_rows()), wl.pos.numpy(), *w64, wl.eps, 1e4, 32, True)
    _, k, v = R.prologue_fwd(oL, *args)
    _check_pool(before[0], before_scale[0], codes[0], scale[0], k, page, offset, False, "k")
    _check_pool(before[1], before_scale[1], codes[1], scale[1], v, page, offset, True, "v")
    dp = torch.full((T, stride), 3.0, dtype=torch.bfloat16, device=cuda)
    dw = [torch.ones(D, device=cuda) for _ in range(2)]
    need = C.qkv_prologue_bwd_workspace_size(L, T)
    ws = torch.empty(need, dtype=torch.uint8, device=cuda)
    C.qkv_prologue_bwd(L, T, wl.dq.to(cuda), wl.dk.to(cuda), wl.dv.to(cuda), want[3], want[4], pos, w_q, w_k, wl.eps, 1e4,
                       flags | C.QKVP_ACCUMULATE_DW, dp, *dw, ws, need)
    ref = R.prologue_bwd(oL, f64(wl.dq), f64(wl.dk), f64(wl.dv), *args)
    assert_bf16_close(u16(dp[:, :width].contiguous()), ref[0], "dpacked")
    assert bool((dp[:, width:] == 3.0).all())
    for a, b in zip(dw, ref[1:3]):
        assert_dw_close(a.cpu().numpy() - 1.0, b, "dw")


def test_layers_on_streams(lib, cuda):
    """Several layers' pools, each appended to and attended on a stream of its own."""
    n_q, n_kv, D = 8, 2, 64
    F = lib.functional
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    table, lengths = i32([[2, 0], [1, 3]]), i32([20, 9])
    where = [(2, t) for t in range(16)] + [(0, t) for t in range(4)] + [(1, t) for t in range(9)]
    page, offset = i32([p for p, _ in where]), i32([o for _, o in where])
    pos = i32(list(range(20)) + list(range(9)))
    layers = []
    for layer in range(4):
        wl = workloads.gqa_inputs(29, n_q, n_kv, D, seed=40 + layer, rope_base=1e4, pos_high=100)
        pool = Pool(4, 16, 16, n_kv, D, cuda, seed=layer, codes=127)
        layers.append((wl.packed_rows().to(cuda), wl.w_q.to(cuda), wl.w_k.to(cuda), pool))
    streams = [torch.cuda.Stream() for _ in layers]
    torch.cuda.synchronize()
    outs = []
    for s, (rows, w_q, w_k, pool) in zip(streams, layers):
        q = F.prologue_pool_write8(rows, pos, w_q, w_k, page, offset, *pool.args, n_q, n_kv, D, rope_base=1e4,
                                   rotary_pairs=True, stream=s)
        with torch.cuda.stream(s):
            last = q[[19, 28]].contiguous()
        outs.append((last, F.attention_decode8(last, *pool.args, table, lengths, stream=s)))
    torch.cuda.synchronize()
    for (last, out), (*_, pool) in zip(outs, layers):
        codes, scale = pool.read()
        keys, values = (E8.stored(c, s) for c, s in zip(codes, scale))
        pick = lambda x: [x[[2] * 16 + [0] * 4, list(range(16)) + list(range(4))], x[[1] * 9, list(range(9))]]  # noqa: E731
        ref = A.attention_decode(f64(last), pick(keys), pick(values))
        bound = 2.0 ** -8 * np.abs(ref["out"]) + (2.0 ** -11 + 2.0 ** -10) * 1.01 * ref["out_abs"]
        assert np.all(np.abs(f64(out) - ref["out"]) <= bound)


def _spoil(x, at, value):
    """x [T, heads, D] with `value` at the places of `at`."""
    y = x.clone()
    for i in at:
        y[i] = value
    return y


# token, head, value behind the rotated 32
SPOTS = [(0, 0, 40), (2, 1, 63), (5, 1, 32), (6, 0, 55)]


@pytest.mark.parametrize("generic", [False, True])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_what_is_not_rotated_keeps_to_itself(lib, cuda, value, pairs, generic):
    """Without the norm an infinity or NaN in a value that is not rotated is that value's
    alone: every other output has the bits that it has without it, forward and back."""
    C = lib
    n_q, n_kv, D, rot, T = 2, 2, 64, 32, 7
    g = workloads._gen(41)
    x = torch.randn(T, n_q + 2 * n_kv, D, generator=g).bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device=cuda) * 37
    bf = dict(dtype=torch.bfloat16, device=cuda)
    L = C.layout("sectioned", n_q, n_kv, D, rope_dim=rot)
    flags = C.QKVP_ROPE_PART | C.QKVP_NORM_OFF | (C.QKVP_ROPE_PAIRS if pairs else 0) | (C.QKVP_FORCE_GENERIC if generic else 0)

    def forward(x):
        q, k, v = (torch.empty(T, n, D, **bf) for n in (n_q, n_kv, n_kv))
        C.qkv_prologue_fwd(L, T, x.to(cuda), pos, None, None, 1e-6, 1e4, flags, q, k, v)
        return torch.cat([q, k, v], 1).cpu()

    def pool_write(x):
        q = torch.empty(T, n_q, D, **bf)
        pools = [torch.zeros(1, T, n_kv, D, **bf) for _ in range(2)]
        page, offset = (torch.tensor(y, dtype=torch.int32, device=cuda) for y in ([0] * T, list(range(T))))
        C.qkv_prologue_pool_write(L, T, x.to(cuda), pos, None, None, 1e-6, 1e4, flags, q, page, offset, *pools, 1, T)
        return torch.cat([q, pools[0][0], pools[1][0]], 1).cpu()

    def backward(x):
        d = [y.contiguous().to(cuda) for y in x.split([n_q, n_kv, n_kv], 1)]
        dp = torch.empty(T, n_q + 2 * n_kv, D, **bf)
        need = C.qkv_prologue_bwd_workspace_size(L, T)
        C.qkv_prologue_bwd(L, T, *d, None, None, pos, None, None, 1e-6, 1e4, flags, dp, None, None,
                           torch.empty(max(need, 16), dtype=torch.uint8, device=cuda), need)
        return dp.cpu()

    at = [(t, h, e) for t, h, e in SPOTS] + [(t, n_q + h, e) for t, h, e in SPOTS]
    for call in (forward, pool_write, backward):
        clean, spoilt = call(_spoil(x, at, 0.0)), call(_spoil(x, at, value))
        for i in at:
            got = float(spoilt[i])
            assert got != got if value != value else got == value, (call.__name__, i, got)
        assert np.array_equal(u16(_spoil(spoilt, at, 0.0)), u16(_spoil(clean, at, 0.0))), call.__name__


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_the_8_bit_pool_takes_what_is_not_rotated_alone(lib, cuda, value, pairs):
    n_q, n_kv, D, T = 2, 2, 64, 7
    x = torch.randn(T, n_q + 2 * n_kv, D, generator=workloads._gen(42)).bfloat16()
    pos = torch.arange(T, dtype=torch.int32, device=cuda) * 37
    page, offset = (torch.tensor(y, dtype=torch.int32, device=cuda) for y in ([1] * T, list(range(T))))

    def write(x):
        pool = Pool(2, 8, 8, n_kv, D, cuda, codes=0)
        q = lib.functional.prologue_pool_write8(x.to(cuda), pos, None, None, page, offset, *pool.args, n_q, n_kv, D, "sectioned",
                                                rope_base=1e4, norm=False, rotary_dim=32, rotary_pairs=pairs)
        codes, scales = pool.read()
        return q.cpu(), codes, scales

    at = [(t, h, e) for t, h, e in SPOTS] + [(t, n_q + h, e) for t, h, e in SPOTS]
    (q0, codes0, scales0), (q1, codes1, scales1) = write(_spoil(x, at, 0.0)), write(_spoil(x, at, value))
    assert np.array_equal(u16(_spoil(q1, SPOTS, 0.0)), u16(_spoil(q0, SPOTS, 0.0)))
    for a, b in zip(scales0, scales1):
        assert np.array_equal(a, b)
    k = codes1[0]
    for t, h, e in SPOTS:
        assert k[1, t, h, e] & 127 == 127 and codes0[0][1, t, h, e] & 127 == 0
        k[1, t, h, e] = codes0[0][1, t, h, e]
    assert np.array_equal(k, codes0[0]) and np.array_equal(codes1[1], codes0[1])
