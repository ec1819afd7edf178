"""The rotary layouts of the prologue (part of the head, adjacent pairs) on the
GPU against the float64 oracle: forward, pool write and gradients, pipelined and
general kernels, both packings. Tolerances are those of parity.py."""

import numpy as np
import pytest
import torch

import oracle.prologue as P
import oracle.rotary as R
import workloads
from parity import assert_bf16_close, assert_dw_close
from workloads import bits_u16 as u16

pytestmark = pytest.mark.gpu

# n_q, n_kv, head_dim, T
SHAPES = [(8, 2, 64, 1), (6, 3, 64, 67), (32, 8, 128, 33), (128, 16, 64, 19), (5, 1, 128, 130), (64, 8, 64, 40)]
LAYOUTS = [(16, False), (16, True), (32, False), (48, True), (48, False), (64, True)]
WIDE = [(96, False), (112, True), (128, True), (80, False)]


def _case(shape, kind, opts, dev, seed=1, rot=None):
    n_q, n_kv, D, T = shape
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=seed, rope_base=5e5, pos_high=131072, with_grads=True)
    g = workloads._gen(seed + 100)
    L = P.PackedLayout(kind, n_q, n_kv, D)
    rows = wl.packed_rows() if kind == "interleaved" else wl.sectioned_rows()
    more = {"norm": opts.get("norm", True), "rope_scale": opts.get("scale", 1.0), "bias": None, "inv_freq": None}
    if opts.get("bias"):
        more["bias"] = workloads.qkv_bias(L.row_width, g)
    if opts.get("table"):
        more["inv_freq"] = [1.5 * 1e4 ** (-2 * i / rot) for i in range(rot // 2)]
    return wl, L, rows, more


def _oracle(more):
    o = dict(more)
    if o["bias"] is not None:
        o["bias"] = o["bias"].numpy().astype(np.float64)
    return o


def _device(more, dev):
    o = dict(more)
    if o["bias"] is not None:
        o["bias"] = o["bias"].to(dev)
    return o


def _generic_forward(lib, wl, kind, rows, more, rot, adjacent, dev):
    """The general kernel through the C call."""
    C, T, D = lib, wl.T, wl.head_dim
    bf = dict(dtype=torch.bfloat16, device=dev)
    q, k, v = (torch.empty(T, n, D, **bf) for n in (wl.n_q, wl.n_kv, wl.n_kv))
    qp, kp = torch.empty_like(q), torch.empty_like(k)
    m = _device(more, dev)
    V = C.variant(inv_freq=m["inv_freq"], rope_scale=m["rope_scale"], bias=m["bias"])
    flags = C.QKVP_SAVE_PRE | C.QKVP_FORCE_GENERIC | C.QKVP_ROPE_PART | (C.QKVP_ROPE_PAIRS if adjacent else 0) | (
        0 if more["norm"] else C.QKVP_NORM_OFF)
    C.qkv_prologue_fwd_ex(C.layout(kind, wl.n_q, wl.n_kv, D, rope_dim=rot), V, T, rows.to(dev), wl.pos.to(dev),
                          wl.w_q.to(dev), wl.w_k.to(dev), wl.eps, wl.rope_base, flags, q, k, v, qp, kp)
    return q, k, v, qp, kp


def _generic_backward(lib, wl, kind, pre, more, rot, adjacent, dev):
    C, T, D = lib, wl.T, wl.head_dim
    m = _device(more, dev)
    V = C.variant(inv_freq=m["inv_freq"], rope_scale=m["rope_scale"], bias=m["bias"])
    L = C.layout(kind, wl.n_q, wl.n_kv, D, rope_dim=rot)
    flags = C.QKVP_FORCE_GENERIC | C.QKVP_ROPE_PART | (C.QKVP_ROPE_PAIRS if adjacent else 0) | (
        0 if more["norm"] else C.QKVP_NORM_OFF)
    width = (wl.n_q + 2 * wl.n_kv) * D
    dp = torch.empty(T, width, dtype=torch.bfloat16, device=dev)
    dw = [torch.empty(D, device=dev) for _ in range(2)]
    db = torch.empty(width, device=dev)
    need = C.qkv_prologue_bwd_workspace_size_ex(L, V, T)
    ws = torch.empty(need, dtype=torch.uint8, device=dev)
    C.qkv_prologue_bwd_ex(L, V, T, wl.dq.to(dev), wl.dk.to(dev), wl.dv.to(dev), *pre, wl.pos.to(dev), wl.w_q.to(dev),
                          wl.w_k.to(dev), wl.eps, wl.rope_base, flags, dp, *dw, db, ws, need)
    return dp, dw, db


def _check(lib, dev, shape, kind, rot, adjacent, opts):
    wl, L, rows, more = _case(shape, kind, opts, dev, rot=rot)
    F, m = lib.functional, _device(more, dev)
    heads = (wl.n_q, wl.n_kv, wl.head_dim, kind, wl.eps, wl.rope_base)
    weights = (wl.w_q.to(dev), wl.w_k.to(dev)) if more["norm"] else (None, None)
    layout = dict(rotary_dim=rot, rotary_pairs=adjacent)
    got = F.prologue_forward(rows.to(dev), wl.pos.to(dev), *weights, *heads, save_pre=True, **m, **layout)
    w64 = (wl.w_q.numpy().astype(np.float64), wl.w_k.numpy().astype(np.float64))
    args = (u16(rows), wl.pos.numpy(), *w64, wl.eps, wl.rope_base, rot, adjacent)
    want = R.prologue_fwd(L, *args, **_oracle(more))
    what = f"{shape} {kind} {rot} {'pairs' if adjacent else 'halves'} {opts}"
    for name, a, b in zip("qkv", got, want):
        assert_bf16_close(u16(a), b, f"{what} {name}")
    generic = _generic_forward(lib, wl, kind, rows, more, rot, adjacent, dev)
    for name, a, b in zip(("q", "k", "v", "q_pre", "k_pre"), got, generic):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16)), f"{what}: {name} of the two kernels"

    pre = (got[3], got[4])
    back = F.prologue_backward(wl.dq.to(dev), wl.dk.to(dev), wl.dv.to(dev), *(pre if more["norm"] else (None, None)),
                               wl.pos.to(dev), *weights, *heads, **m, **layout)
    d = [P.bf16_bits_to_f64(u16(t)) for t in (wl.dq, wl.dk, wl.dv)]
    dp, dw_q, dw_k, db = R.prologue_bwd(L, *d, *args, **_oracle(more))
    assert_bf16_close(u16(back[0]), dp, f"{what} dpacked")
    other = _generic_backward(lib, wl, kind, pre, more, rot, adjacent, dev)
    assert torch.equal(back[0].view(torch.int16), other[0].view(torch.int16)), f"{what}: dpacked of the two kernels"
    if more["norm"]:
        for name, a, b, c in (("dw_q", back[1], dw_q, other[1][0]), ("dw_k", back[2], dw_k, other[1][1])):
            assert_dw_close(a.cpu().numpy(), b, f"{what} {name}")
            assert_dw_close(c.cpu().numpy(), b, f"{what} {name} general")
    else:
        assert back[1] is None and back[2] is None
    if more["bias"] is not None:
        assert_dw_close(back[3].cpu().numpy(), db, f"{what} dbias")
        assert_dw_close(other[2].cpu().numpy(), db, f"{what} dbias general")


@pytest.mark.parametrize("kind", ["interleaved", "sectioned"])
@pytest.mark.parametrize("shape", SHAPES)
def test_layouts_and_gradients(lib, cuda, shape, kind):
    for i, (rot, adjacent) in enumerate(LAYOUTS + (WIDE if shape[2] == 128 else [])):
        opts = [{}, {"norm": False}, {"bias": True, "scale": 1.125}, {"table": True, "scale": 0.75},
                {"norm": False, "bias": True, "table": True}][i % 5]
        _check(lib, cuda, shape, kind, rot, adjacent, opts)


@pytest.mark.parametrize("opts", [{}, {"norm": False}, {"bias": True}, {"norm": False, "bias": True}])
@pytest.mark.parametrize("adjacent", [False, True])
def test_every_option_at_one_shape(lib, cuda, adjacent, opts):
    for kind in ("interleaved", "sectioned"):
        _check(lib, cuda, (8, 2, 64, 21), kind, 32, adjacent, opts)
        _check(lib, cuda, (8, 2, 128, 21), kind, 32, adjacent, opts)


def test_halves_of_the_whole_head_are_the_old_call(lib, cuda):
    wl, _, rows, _ = _case((32, 8, 128, 50), "sectioned", {}, cuda)
    args = (rows.to(cuda), wl.pos.to(cuda), wl.w_q.to(cuda), wl.w_k.to(cuda), 32, 8, 128, "sectioned")
    a = lib.functional.prologue_forward(*args, save_pre=True)
    b = lib.functional.prologue_forward(*args, save_pre=True, rotary_dim=128)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("adjacent", [False, True])
def test_pool_write_is_the_forward_in_the_pool(lib, cuda, adjacent):
    wl, _, rows, _ = _case((8, 2, 64, 37), "interleaved", {}, cuda)
    F, T = lib.functional, 37
    layout = dict(rotary_dim=48, rotary_pairs=adjacent)
    args = (rows.to(cuda), wl.pos.to(cuda), wl.w_q.to(cuda), wl.w_k.to(cuda))
    q, k, v = F.prologue_forward(*args, 8, 2, 64, **layout)
    page, offset = (t.to(cuda) for t in workloads.random_slots(T, 5, 16, workloads._gen(4)))
    pools = [torch.full((5, 16, 2, 64), 7.0, dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    got = F.prologue_pool_write(*args, page, offset, *pools, 8, 2, 64, **layout)
    assert torch.equal(got, q)
    for pool, rows_ in zip(pools, (k, v)):
        want = torch.full_like(pool, 7.0)
        want[page.long(), offset.long()] = rows_
        assert torch.equal(pool, want)


def test_autograd_region(lib, cuda):
    wl, L, rows, _ = _case((8, 2, 64, 29), "interleaved", {}, cuda)
    x = rows.to(cuda).requires_grad_()
    w_q, w_k = wl.w_q.to(cuda).requires_grad_(), wl.w_k.to(cuda).requires_grad_()
    out = lib.functional.GQAttentionPrologue.apply(x, wl.pos.to(cuda), w_q, w_k, None, 8, 2, 64, "interleaved", wl.eps,
                                                   wl.rope_base, False, True, None, 1.0, 32, True)
    torch.autograd.backward(out, [t.to(cuda) for t in (wl.dq, wl.dk, wl.dv)])
    w64 = (wl.w_q.numpy().astype(np.float64), wl.w_k.numpy().astype(np.float64))
    d = [P.bf16_bits_to_f64(u16(t)) for t in (wl.dq, wl.dk, wl.dv)]
    dp, dw_q, dw_k, _ = R.prologue_bwd(L, *d, u16(rows), wl.pos.numpy(), *w64, wl.eps, wl.rope_base, 32, True)
    assert_bf16_close(u16(x.grad), dp, "dpacked")
    assert_dw_close(w_q.grad.cpu().numpy(), dw_q, "dw_q")
    assert_dw_close(w_k.grad.cpu().numpy(), dw_k, "dw_k")


def test_captured_with_moving_positions(lib, cuda):
    wl, _, rows, _ = _case((8, 2, 64, 9), "interleaved", {}, cuda)
    F = lib.functional
    args = (rows.to(cuda), wl.pos.to(cuda).clone(), wl.w_q.to(cuda), wl.w_k.to(cuda))
    call = lambda: F.prologue_forward(*args, 8, 2, 64, rotary_dim=32, rotary_pairs=True)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    args[1].add_(1000)
    graph.replay()
    for a, b in zip(out, call()):
        assert torch.equal(a, b)


def test_refusals(lib, cuda):
    wl, _, rows, _ = _case((8, 2, 64, 5), "interleaved", {}, cuda)
    F = lib.functional
    args = (rows.to(cuda), wl.pos.to(cuda), wl.w_q.to(cuda), wl.w_k.to(cuda), 8, 2, 64)
    for bad in (dict(rotary_dim=24), dict(rotary_dim=0), dict(rotary_dim=80), dict(rotary_dim=-16),
                dict(rotary_dim=32, nope=True), dict(rotary_pairs=True, nope=True)):
        with pytest.raises(lib.QkvpError):
            F.prologue_forward(*args, **bad)
    with pytest.raises(ValueError, match="frequencies"):
        F.prologue_forward(*args, rotary_dim=32, inv_freq=[1.0] * 32)
    assert [t.shape[0] for t in F.prologue_forward(args[0][:0], args[1][:0], *args[2:], rotary_dim=32)] == [0, 0, 0]
