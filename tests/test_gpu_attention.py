"""Attention over packed sequences on the GPU against the float64 oracle: out,
lse and the gradients, element by element within the bounds of
attention_parity; what is exact (rows of no sequence, repeat runs, independence
of the sequences) is checked bit for bit."""

import numpy as np
import pytest
import torch

import oracle.attention as A
from attention_parity import U, assert_lse, assert_within, out_bound
from oracle.bf16 import bf16_bits_to_f64
from workloads import bits_u16 as u16

pytestmark = pytest.mark.gpu


def f64(t):
    return bf16_bits_to_f64(u16(t))


def offsets(lengths, first=0):
    return np.cumsum([first] + list(lengths)).astype(np.int32)


def inputs(T, n_q, n_kv, D, seed, sharp=1.0):
    g = torch.Generator(device="cpu")
    g.manual_seed(seed)
    q = (torch.randn(T, n_q, D, generator=g) * sharp).to(torch.bfloat16)
    k = torch.randn(T, n_kv, D, generator=g).to(torch.bfloat16)
    v = torch.randn(T, n_kv, D, generator=g).to(torch.bfloat16)
    do = torch.randn(T, n_q, D, generator=g).to(torch.bfloat16)
    return q, k, v, do


def no_error(lib):
    torch.cuda.synchronize()
    assert lib.qkv_prologue_device_error(clear=True) == 0


# lengths from one token to several blocks of 128, uneven, empty ones among
# them, sequences that begin and end inside a block, rows before and after
PACKED = [
    ([1], 0, 0),
    ([2, 1, 3], 0, 0),
    ([127, 128, 129], 0, 0),
    ([0, 37, 0, 256, 1, 0], 0, 3),
    ([300, 5, 77, 640], 11, 40),
    ([1000], 0, 0),
    ([50] * 9, 2, 1),
]
HEADS = [(8, 2, 64), (4, 2, 128), (3, 3, 64), (3, 1, 128), (5, 5, 128), (16, 1, 64)]


@pytest.mark.parametrize("lengths,before,after", PACKED)
@pytest.mark.parametrize("n_q,n_kv,D", HEADS)
def test_forward(lib, cuda, lengths, before, after, n_q, n_kv, D):
    cu = offsets(lengths, before)
    T = int(cu[-1]) + after
    q, k, v, _ = inputs(T, n_q, n_kv, D, 100 + T)
    out, lse = lib.functional.attention_forward(q.to(cuda), k.to(cuda), v.to(cuda), torch.from_numpy(cu).to(cuda),
                                                save_lse=True)
    no_error(lib)
    ref = A.attention_fwd(f64(q), f64(k), f64(v), cu)
    assert_within(f64(out), ref["out"], out_bound(ref), "out")
    assert_lse(lse.cpu().numpy(), ref, max(lengths), D, "lse")


@pytest.mark.parametrize("lengths,before,after", PACKED)
@pytest.mark.parametrize("n_q,n_kv,D", HEADS)
def test_backward(lib, cuda, lengths, before, after, n_q, n_kv, D):
    F = lib.functional
    cu = offsets(lengths, before)
    T = int(cu[-1]) + after
    q, k, v, do = inputs(T, n_q, n_kv, D, 200 + T)
    dev = [t.to(cuda) for t in (q, k, v, do)]
    cu_dev = torch.from_numpy(cu).to(cuda)
    out, lse = F.attention_forward(*dev[:3], cu_dev, save_lse=True)
    grads = F.attention_backward(dev[3], *dev[:3], out, lse, cu_dev)
    no_error(lib)
    fwd = A.attention_fwd(f64(q), f64(k), f64(v), cu)
    ref = A.attention_bwd(f64(do), f64(q), f64(k), f64(v), cu, out_err=out_bound(fwd))
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert_within(f64(got), ref[name], ref["e_" + name] + U * np.abs(ref[name]), name)


@pytest.mark.parametrize("n_q,n_kv,D", [(8, 2, 64), (4, 2, 128), (3, 3, 64)])
@pytest.mark.parametrize("scale,sharp", [(0.02, 1.0), (None, 4.0), (1.0, 0.5)])
def test_scales_and_sharp_rows(lib, cuda, n_q, n_kv, D, scale, sharp):
    # scores far apart, so that a row's maximum moves by many powers of two from
    # block to block; the largest |scale q k| stays below 2^6
    F = lib.functional
    cu = offsets([700, 130], 0)
    q, k, v, do = inputs(830, n_q, n_kv, D, 5, sharp)
    ref = A.attention_fwd(f64(q), f64(k), f64(v), cu, scale)
    assert ref["s_abs"].max() < (64 if scale is None else 128)
    dev = [t.to(cuda) for t in (q, k, v, do)]
    cu_dev = torch.from_numpy(cu).to(cuda)
    out, lse = F.attention_forward(*dev[:3], cu_dev, scale, save_lse=True)
    grads = F.attention_backward(dev[3], *dev[:3], out, lse, cu_dev, scale)
    no_error(lib)
    assert_within(f64(out), ref["out"], out_bound(ref), "out")
    assert_lse(lse.cpu().numpy(), ref, 700, D, "lse")
    g = A.attention_bwd(f64(do), f64(q), f64(k), f64(v), cu, scale, out_err=out_bound(ref))
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert_within(f64(got), g[name], g["e_" + name] + U * np.abs(g[name]), name)


def test_growing_maxima(lib, cuda):
    # keys that each outdo the ones before by far: every block rescales the result
    n_q, n_kv, D, T = 2, 1, 128, 600
    q = torch.ones(T, n_q, D, dtype=torch.bfloat16)
    k = (torch.arange(T).float()[:, None, None] / 150).expand(T, n_kv, D).to(torch.bfloat16).contiguous()
    v = inputs(T, n_q, n_kv, D, 6)[2]
    cu = offsets([T])
    out, lse = lib.functional.attention_forward(q.to(cuda), k.to(cuda), v.to(cuda), torch.from_numpy(cu).to(cuda),
                                                save_lse=True)
    no_error(lib)
    ref = A.attention_fwd(f64(q), f64(k), f64(v), cu)
    assert_within(f64(out), ref["out"], out_bound(ref), "out")
    assert_lse(lse.cpu().numpy(), ref, T, D, "lse")


@pytest.mark.parametrize("batch", [33, 200, 700])
def test_many_sequences(lib, cuda, batch):
    # more sequences than a warp, than the kernels keep counts of, and than work items per CTA
    F = lib.functional
    rng = np.random.default_rng(batch)
    lengths = rng.integers(0, 9, size=batch).tolist()
    lengths[batch // 2] = 200
    cu = offsets(lengths)
    T = int(cu[-1])
    q, k, v, do = inputs(T, 4, 2, 64, batch)
    dev = [t.to(cuda) for t in (q, k, v, do)]
    cu_dev = torch.from_numpy(cu).to(cuda)
    out, lse = F.attention_forward(*dev[:3], cu_dev, save_lse=True)
    grads = F.attention_backward(dev[3], *dev[:3], out, lse, cu_dev)
    no_error(lib)
    ref = A.attention_fwd(f64(q), f64(k), f64(v), cu)
    assert_within(f64(out), ref["out"], out_bound(ref), "out")
    g = A.attention_bwd(f64(do), f64(q), f64(k), f64(v), cu, out_err=out_bound(ref))
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert_within(f64(got), g[name], g["e_" + name] + U * np.abs(g[name]), name)


def test_rows_of_no_sequence_are_left_alone_and_never_used(lib, cuda):
    # NaN in every row of no sequence; out, lse and gradients of the others are
    # those without them, bit for bit, and a given out keeps its other rows
    F = lib.functional
    cu = offsets([5, 260, 0, 64], 7)
    T = int(cu[-1]) + 30
    q, k, v, do = (t.to(cuda) for t in inputs(T, 8, 2, 64, 9))
    cu_dev = torch.from_numpy(cu).to(cuda)
    inside = torch.zeros(T, dtype=torch.bool, device=cuda)
    inside[7:int(cu[-1])] = True
    out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True)
    grads = F.attention_backward(do, q, k, v, out, lse, cu_dev)
    for t in (out, *grads):
        assert not t[~inside].any() and torch.isfinite(t[inside].float()).all()
    assert torch.isneginf(lse[:, ~inside]).all()
    bad = [t.clone() for t in (q, k, v, do)]
    for t in bad:
        t[~inside] = float("nan")
    mine = torch.full_like(q, 3.0)
    out2, lse2 = F.attention_forward(*bad[:3], cu_dev, save_lse=True, out=mine)
    assert out2 is mine and (mine[~inside] == 3.0).all() and torch.isneginf(lse2[:, ~inside]).all()
    assert torch.equal(mine[inside], out[inside]) and torch.equal(lse2[:, inside], lse[:, inside])
    keep = out.clone()
    keep[~inside] = float("nan")
    for a, b in zip(F.attention_backward(bad[3], *bad[:3], keep, lse, cu_dev), grads):
        assert torch.equal(a, b)
    no_error(lib)


def test_sequences_do_not_touch_each_other(lib, cuda):
    # an infinity and a NaN in one sequence leave the others' bits alone, in both directions
    F = lib.functional
    lengths = [100, 30, 200]
    cu = offsets(lengths)
    T = int(cu[-1])
    q, k, v, do = (t.to(cuda) for t in inputs(T, 4, 2, 64, 10))
    cu_dev = torch.from_numpy(cu).to(cuda)

    def step(q, k, v, do):
        out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True)
        return (out, *F.attention_backward(do, q, k, v, out, lse, cu_dev))

    good = step(q, k, v, do)
    bad = [t.clone() for t in (q, k, v, do)]
    for i, t in enumerate(bad):
        t[100:130] = float("nan") if i % 2 else float("inf")
    others = torch.ones(T, dtype=torch.bool, device=cuda)
    others[100:130] = False
    for a, b in zip(step(*bad), good):
        assert torch.equal(a[others], b[others])
    # and a sequence alone gives what it gives in the pack
    one = torch.tensor([0, 200], dtype=torch.int32, device=cuda)
    alone = F.attention_forward(q[130:].contiguous(), k[130:].contiguous(), v[130:].contiguous(), one)
    assert torch.equal(alone, good[0][130:])
    no_error(lib)


def test_offsets_that_do_not_ascend_are_refused_on_the_device(lib, cuda):
    F = lib.functional
    q, k, v, do = (t.to(cuda) for t in inputs(300, 4, 2, 64, 11))
    for cu in ([0, 200, 100, 300], [-1, 300], [0, 301], [5, 2], [0, 2 ** 31 - 1]):
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        cu_dev = torch.tensor(cu, dtype=torch.int32, device=cuda)
        mine = torch.full_like(q, 2.0)
        F.attention_forward(q, k, v, cu_dev, out=mine, dev_status=status)
        assert status.item() == lib.QKVP_DEV_BAD_SEQUENCE and (mine == 2.0).all()
        out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True, dev_status=status)
        assert not out.any() and torch.isneginf(lse).all()
        status.zero_()
        grads = F.attention_backward(do, q, k, v, out, lse, cu_dev, dev_status=status)
        assert status.item() == lib.QKVP_DEV_BAD_SEQUENCE and not any(g.any() for g in grads)
    no_error(lib)


def test_nothing_to_do(lib, cuda):
    F = lib.functional
    q, k, v, do = (t.to(cuda) for t in inputs(5, 4, 2, 64, 12))
    none = torch.zeros(1, dtype=torch.int32, device=cuda)
    out, lse = F.attention_forward(q, k, v, none, save_lse=True)  # no sequence
    assert not out.any() and torch.isneginf(lse).all()
    assert not any(g.any() for g in F.attention_backward(do, q, k, v, out, lse, none))
    empty = torch.zeros(4, dtype=torch.int32, device=cuda)  # three empty ones
    assert not F.attention_forward(q, k, v, empty).any()
    out, lse = F.attention_forward(q[:0], k[:0], v[:0], none, save_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (4, 0)
    assert [tuple(g.shape) for g in F.attention_backward(do[:0], q[:0], k[:0], v[:0], out, lse, none)] == [
        (0, 4, 64), (0, 2, 64), (0, 2, 64)]
    no_error(lib)


@pytest.mark.parametrize("n_q,n_kv,D", [(8, 2, 64), (6, 2, 128)])
def test_repeats_bit_for_bit_and_in_a_graph(lib, cuda, n_q, n_kv, D):
    F = lib.functional
    cu = offsets([333, 1, 129, 700])
    T = int(cu[-1])
    q, k, v, do = (t.to(cuda) for t in inputs(T, n_q, n_kv, D, 13))
    cu_dev = torch.from_numpy(cu).to(cuda)

    def step():
        out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True)
        return (out, lse, *F.attention_backward(do, q, k, v, out, lse, cu_dev))

    first = [t.clone() for t in step()]
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(step(), first))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        captured = step()
    for _ in range(2):
        for t in captured:
            t.fill_(float("nan"))
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(captured, first))
    # other data and other sequence lengths through the same graph
    for t, new in zip((q, k, v, do), inputs(T, n_q, n_kv, D, 14)):
        t.copy_(new)
    cu_dev.copy_(torch.from_numpy(offsets([1000, 50, 0, 113])))
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(captured, step()))
    no_error(lib)


def test_on_a_given_stream(lib, cuda):
    F = lib.functional
    cu_dev = torch.tensor([0, 500], dtype=torch.int32, device=cuda)
    q, k, v, do = (t.to(cuda) for t in inputs(500, 8, 2, 64, 15))
    want = F.attention_forward(q, k, v, cu_dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for s in (side, side.cuda_stream):
        out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True, stream=s)
        grads = F.attention_backward(do, q, k, v, out, lse, cu_dev, stream=s)
        junk = [torch.full((n,), float("nan"), device=cuda) for n in (4000, 500 * 8, 10 ** 6)]  # takes freed memory
        side.synchronize()
        assert torch.equal(out, want) and all(torch.isfinite(x.float()).all() for x in grads)
        del junk
    no_error(lib)


def test_autograd_and_gradients_against_differences(lib, cuda):
    # PackedAttention's gradients are attention_backward's; and along random
    # directions they are the oracle's central differences, within the same bounds
    F = lib.functional
    cu = offsets([3, 140, 1, 20])
    T = int(cu[-1])
    n_q, n_kv, D = 4, 2, 64
    host = inputs(T, n_q, n_kv, D, 16)
    q, k, v = (t.to(cuda).requires_grad_() for t in host[:3])
    do = host[3].to(cuda)
    cu_dev = torch.from_numpy(cu).to(cuda)
    out = F.PackedAttention.apply(q, k, v, cu_dev)
    got = torch.autograd.grad(out, (q, k, v), do)
    with torch.no_grad():
        o, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True)
        want = F.attention_backward(do, q, k, v, o, lse, cu_dev)
    assert torch.equal(out, o) and all(torch.equal(a, b) for a, b in zip(got, want))
    # an expanded (broadcast) upstream gradient
    one = torch.ones(1, 1, 1, dtype=torch.bfloat16, device=cuda).expand(T, n_q, D)
    a = torch.autograd.grad(F.PackedAttention.apply(q, k, v, cu_dev), (q, k, v), one)
    b = F.attention_backward(one.contiguous(), q.detach(), k.detach(), v.detach(), o, lse, cu_dev)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    no_error(lib)

    x = [f64(t) for t in host[:3]]
    d = f64(host[3])
    ref = A.attention_fwd(*x, cu)
    err = A.attention_bwd(d, *x, cu, out_err=out_bound(ref))
    rng = np.random.default_rng(17)
    for i, name in enumerate(("dq", "dk", "dv")):
        way = rng.normal(size=x[i].shape)
        step = 1e-5
        loss = []
        for sign in (1, -1):
            y = list(x)
            y[i] = x[i] + sign * step * way
            loss.append((A.attention_fwd(*y, cu)["out"] * d).sum())
        slope = (loss[0] - loss[1]) / (2 * step)
        g = f64(got[i])
        bound = ((err["e_" + name] + U * np.abs(err[name])) * np.abs(way)).sum()
        assert abs((g * way).sum() - slope) <= bound + 1e-5 * abs(slope), name


def test_behind_the_prologue(lib, cuda):
    # one training step's attention region: packed qkv -> prologue -> attention, and back
    import workloads

    F = lib.functional
    wl = workloads.gqa_inputs(300, 8, 2, 64, seed=21, rope_base=10000.0)
    packed = wl.packed_rows().to(cuda).requires_grad_()
    w_q, w_k = (w.to(cuda).requires_grad_() for w in (wl.w_q, wl.w_k))
    cu = offsets([120, 180])
    cu_dev = torch.from_numpy(cu).to(cuda)
    q, k, v = F.QKVPrologue.apply(packed, wl.pos.to(cuda), w_q, w_k, 8, 2, 64, "interleaved", wl.eps, wl.rope_base,
                                  False)
    out = F.PackedAttention.apply(q, k, v, cu_dev)
    do = torch.randn(300, 8, 64, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    d_packed, d_wq, d_wk = torch.autograd.grad(out, (packed, w_q, w_k), do.to(cuda))
    no_error(lib)
    ref = A.attention_fwd(f64(q), f64(k), f64(v), cu)
    assert_within(f64(out), ref["out"], out_bound(ref), "out")
    assert d_packed.shape == packed.shape and torch.isfinite(d_packed.float()).all() and d_packed.any()
    assert torch.isfinite(d_wq).all() and torch.isfinite(d_wk).all()


@pytest.mark.parametrize("n_q,n_kv,D", [(32, 4, 64), (8, 2, 128)])
def test_many_steps_of_ragged_sequences(lib, cuda, n_q, n_kv, D):
    # the pipelines' barriers over some ten million phases: no wait runs out, and
    # the last step has the first one's bits
    F = lib.functional
    cu = offsets([3, 176, 122, 359, 532, 951, 473, 440, 796, 121, 123])
    q, k, v, do = (t.to(cuda) for t in inputs(int(cu[-1]), n_q, n_kv, D, 18))
    cu_dev = torch.from_numpy(cu).to(cuda)

    def step():
        out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True)
        return (out, lse, *F.attention_backward(do, q, k, v, out, lse, cu_dev))

    first = step()
    for _ in range(400):
        last = step()
    assert all(torch.equal(a, b) for a, b in zip(first, last))
    no_error(lib)


@pytest.mark.parametrize("n_q,n_kv,D", [(6, 2, 64), (7, 1, 128), (8, 1, 64), (5, 5, 128)])
@pytest.mark.parametrize("lengths,before,after", [([1], 0, 0), ([300], 2, 5), ([0, 129, 1, 0, 257], 0, 40)])
def test_heads_of_a_group_in_parts(lib, cuda, lengths, before, after, n_q, n_kv, D):
    # small problems divide a group's query heads among CTAs, whose sums lie in the
    # workspace: the same bits again from one full of NaN
    F = lib.functional
    cu = offsets(lengths, before)
    T = int(cu[-1]) + after
    need = F.attention_backward_workspace_bytes(n_q, n_kv, D, T, len(lengths))
    assert (need > 4 * (n_q * T + 3)) == (n_q != n_kv)
    q, k, v, do = inputs(T, n_q, n_kv, D, 700 + T)
    dev = [t.to(cuda) for t in (q, k, v, do)]
    cu_dev = torch.from_numpy(cu).to(cuda)
    out, lse = F.attention_forward(*dev[:3], cu_dev, save_lse=True)
    grads = F.attention_backward(dev[3], *dev[:3], out, lse, cu_dev)
    room = torch.full((need,), 255, dtype=torch.uint8, device=cuda)
    again = F.attention_backward(dev[3], *dev[:3], out, lse, cu_dev, workspace=room)
    no_error(lib)
    fwd = A.attention_fwd(f64(q), f64(k), f64(v), cu)
    ref = A.attention_bwd(f64(do), f64(q), f64(k), f64(v), cu, out_err=out_bound(fwd))
    for name, got, other in zip(("dq", "dk", "dv"), grads, again):
        assert torch.equal(got, other)
        assert_within(f64(got), ref[name], ref["e_" + name] + U * np.abs(ref[name]), name)


def test_rows_beyond_32_bit_offsets(lib, cuda):
    # the last sequence of tensors of more than 2^31 values
    F = lib.functional
    n_q, n_kv, D, before = 128, 1, 128, 2 ** 17
    T = before + 100
    host = inputs(100, n_q, n_kv, D, 800)
    dev = [torch.zeros(T, t.shape[1], D, dtype=torch.bfloat16, device=cuda) for t in host]
    for t, last in zip(dev, host):
        t[before:] = last.to(cuda)
    cu_dev = torch.tensor([before - 300, before - 1, before, T], dtype=torch.int32, device=cuda)
    out, lse = F.attention_forward(*dev[:3], cu_dev, save_lse=True)
    grads = F.attention_backward(dev[3], *dev[:3], out, lse, cu_dev)
    no_error(lib)
    cu = offsets([100])
    x = [f64(t) for t in host]
    ref = A.attention_fwd(*x[:3], cu)
    assert_within(f64(out[before:]), ref["out"], out_bound(ref), "out")
    assert_lse(lse[:, before:].cpu().numpy(), ref, 100, D, "lse")
    g = A.attention_bwd(x[3], *x[:3], cu, out_err=out_bound(ref))
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert_within(f64(got[before:]), g[name], g["e_" + name] + U * np.abs(g[name]), name)
        assert not got[:before].any()
    assert not out[:before].any()


def test_refusals_of_what_overlaps_or_lies_elsewhere(lib, cuda):
    F = lib.functional
    q, k, v, do = (t.to(cuda) for t in inputs(60, 2, 2, 64, 18))
    cu_dev = torch.tensor([0, 60], dtype=torch.int32, device=cuda)
    out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True)
    for bad in (q, k, v):
        with pytest.raises(lib.QkvpError):
            F.attention_forward(q, k, v, cu_dev, out=bad)
    need = F.attention_backward_workspace_bytes(2, 2, 64, 60, 1)
    room = torch.zeros(need, dtype=torch.uint8, device=cuda)
    for bad in (room.cpu(), torch.zeros(2 * need, dtype=torch.uint8, device=cuda)[::2]):
        with pytest.raises(ValueError):
            F.attention_backward(do, q, k, v, out, lse, cu_dev, workspace=bad)
    for bad in (room[:need - 16], lse, do):  # too small, or an input
        with pytest.raises(lib.QkvpError):
            F.attention_backward(do, q, k, v, out, lse, cu_dev, workspace=bad)
    with pytest.raises(ValueError):
        F.attention_forward(q, k, v, cu_dev, dev_status=torch.zeros(1, dtype=torch.int32))
    L = lib.layout("sectioned", 2, 2, 64)
    grads = [torch.empty_like(q) for _ in range(3)]

    def raw(dq, dk, dv):
        return lib.qkv_attention_bwd(L, 60, 1, cu_dev, do, q, k, v, out, lse, 0.0, 0, dq, dk, dv, None, room, need,
                                     check=False)

    assert raw(*grads) == lib.QKVP_OK
    for bad in ((grads[0], grads[0], grads[2]), (q, *grads[1:]), (grads[0], k, grads[2]), (*grads[:2], out)):
        assert raw(*bad) == lib.QKVP_ERR_VALUE
    no_error(lib)


def test_two_calls_at_once(lib, cuda):
    # on two streams, each result its own; the caller's stream is busy meanwhile
    F = lib.functional
    cu_dev = torch.tensor([3, 500, 900], dtype=torch.int32, device=cuda)
    sets = [[t.to(cuda) for t in inputs(950, 8, 2, 64, 900 + i)] for i in range(2)]

    def step(q, k, v, do, stream=None):
        mine = torch.zeros_like(q)
        torch.cuda.synchronize()
        out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True, out=mine, stream=stream)
        return (out, lse, *F.attention_backward(do, q, k, v, out, lse, cu_dev, stream=stream))

    want = [step(*s) for s in sets]
    mine = [torch.zeros_like(s[0]) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    busy = torch.randn(8192, 8192, device=cuda)
    for _ in range(3):
        busy = busy @ busy * 1e-4
    got = []
    for (q, k, v, do), s, o in zip(sets, streams, mine):
        out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True, out=o, stream=s)
        got.append((out, lse, *F.attention_backward(do, q, k, v, out, lse, cu_dev, stream=s)))
    for s in streams:
        s.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    no_error(lib)


def test_autograd_in_a_graph_and_twice(lib, cuda):
    F = lib.functional
    q, k, v, do = (t.to(cuda) for t in inputs(200, 4, 2, 128, 19))
    cu_dev = torch.tensor([0, 150, 200], dtype=torch.int32, device=cuda)

    def step():
        x = [t.detach().requires_grad_() for t in (q, k, v)]
        return torch.autograd.grad(F.PackedAttention.apply(*x, cu_dev), x, do)

    want = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = step()
    for t in got:
        t.fill_(float("nan"))
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # gradients of the gradients are refused, not silently zero
    x = q.clone().requires_grad_()
    first, = torch.autograd.grad(F.PackedAttention.apply(x, k, v, cu_dev), x, do, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first.float().square().sum(), x)
    no_error(lib)


# sequences at the lengths where a tile of 128 rows holds four heads, two, or one, enough
# of them that the heads of a group are not divided among CTAs (`times`), and few
@pytest.mark.parametrize("n_q,n_kv,D", [(16, 2, 64), (16, 1, 128), (8, 2, 128), (12, 3, 64), (6, 3, 64), (10, 2, 64),
                                        (6, 2, 128), (14, 2, 64), (12, 1, 64), (3, 3, 128)])
@pytest.mark.parametrize("lengths,times,before,after", [
    ([1, 31, 32, 33, 0, 63, 64, 65, 5, 130], 16, 0, 0),
    ([32, 33, 1, 64], 1, 3, 70),
    ([2] * 40 + [129, 0, 40], 4, 1, 0),
    ([1, 31, 32, 33, 0, 63, 64, 65, 5, 130], 4, 2, 1),  # in several parts of several heads
])
def test_short_sequences_with_several_heads_in_a_tile(lib, cuda, lengths, times, before, after, n_q, n_kv, D):
    F = lib.functional
    cu = offsets(lengths * times, before)
    T = int(cu[-1]) + after
    q, k, v, do = inputs(T, n_q, n_kv, D, 1000 + T)
    dev = [t.to(cuda) for t in (q, k, v, do)]
    for t in dev:  # rows of no sequence are in the tiles, but in no result
        t[:before] = t[T - after:] = float("nan")
    cu_dev = torch.from_numpy(cu).to(cuda)
    out, lse = F.attention_forward(*dev[:3], cu_dev, save_lse=True)
    grads = F.attention_backward(dev[3], *dev[:3], out, lse, cu_dev)
    no_error(lib)
    ref = A.attention_fwd(f64(q), f64(k), f64(v), cu)
    assert_within(f64(out), ref["out"], out_bound(ref), "out")
    assert_lse(lse.cpu().numpy(), ref, max(lengths), D, "lse")
    g = A.attention_bwd(f64(do), f64(q), f64(k), f64(v), cu, out_err=out_bound(ref))
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert_within(f64(got), g[name], g["e_" + name] + U * np.abs(g[name]), name)


def test_as_many_sequences_as_allowed(lib, cuda):
    # 2^20, all but a few empty
    F = lib.functional
    lengths = np.zeros(2 ** 20, dtype=np.int64)
    for at, n in ((0, 3), (500000, 200), (2 ** 20 - 2, 60), (2 ** 20 - 1, 129)):
        lengths[at] = n
    cu = offsets(lengths)
    T = int(cu[-1])
    host = inputs(T, 2, 1, 64, 1100)
    dev = [t.to(cuda) for t in host]
    cu_dev = torch.from_numpy(cu).to(cuda)
    out, lse = F.attention_forward(*dev[:3], cu_dev, save_lse=True)
    grads = F.attention_backward(dev[3], *dev[:3], out, lse, cu_dev)
    no_error(lib)
    few = offsets([3, 200, 60, 129])
    x = [f64(t) for t in host]
    ref = A.attention_fwd(*x[:3], few)
    assert_within(f64(out), ref["out"], out_bound(ref), "out")
    g = A.attention_bwd(x[3], *x[:3], few, out_err=out_bound(ref))
    for name, got in zip(("dq", "dk", "dv"), grads):
        assert_within(f64(got), g[name], g["e_" + name] + U * np.abs(g[name]), name)
    more = torch.zeros(2 ** 20 + 2, dtype=torch.int32, device=cuda)
    with pytest.raises(lib.QkvpError):
        F.attention_forward(*dev[:3], more)


@pytest.mark.parametrize("n_q,n_kv,D", [(8, 2, 64), (4, 2, 128), (3, 1, 64)])
def test_what_the_next_sequence_holds_does_not_show(lib, cuda, n_q, n_kv, D):
    # not in the last bits either: large queries (and keys) behind a sequence that ends
    # inside a warp's rows, where every block would move their maxima
    F = lib.functional
    lengths = [168, 300, 430, 140]
    cu_dev = torch.from_numpy(offsets(lengths)).to(cuda)
    T = sum(lengths)
    q, k, v, do = (t.to(cuda) for t in inputs(T + 60, n_q, n_kv, D, 1200))
    want = None
    for factor in (1.0, 30.0):
        x = [t.clone() for t in (q, k, v, do)]
        for t in x:
            t[168:468] *= factor
            t[T:] *= factor
        out, lse = F.attention_forward(*x[:3], cu_dev, save_lse=True)
        got = [t[i] for t in (out, *F.attention_backward(x[3], *x[:3], out, lse, cu_dev))
               for i in (slice(0, 168), slice(468, T))]
        if want is not None:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        want = got
    no_error(lib)


def test_a_work_item_of_more_than_two_seconds(lib, cuda):
    # 640 blocks of 128 rows and 4094 query heads over one key/value head: the first keys'
    # block goes through 2.6 million blocks of queries at about 1 us, longer than any wait may
    # last without progress, while the warp that finds work has nothing to do. All is zero but the
    # last row: with k = v = 0 and lse = 12 ln 2 every p is 2^-12, so that
    # dv_j = 4094 2^-12 dout and ds = -2^-12 dout . out = -2^-6 in that row.
    F = lib.functional
    n_q, D, T = 4094, 64, 640 * 128
    if torch.cuda.mem_get_info()[0] < 110 * 2 ** 30:
        pytest.skip("needs 110 GB of device memory")
    x = torch.zeros(T, n_q, D, dtype=torch.bfloat16, device=cuda)  # q, dout and out
    x[-1] = 1.0
    k, v = (torch.zeros(T, 1, D, dtype=torch.bfloat16, device=cuda) for _ in range(2))
    lse = torch.full((n_q, T), 12 * float(np.log(2.0)), dtype=torch.float32, device=cuda)
    cu_dev = torch.tensor([0, T], dtype=torch.int32, device=cuda)
    dq, dk, dv = F.attention_backward(x, x, k, v, x, lse, cu_dev)
    no_error(lib)
    assert not dq.any()
    # one rounding to bf16 (p and ds are powers of two, their sums exact in fp32)
    for got, exact in ((dv, n_q / 4096), (dk, -n_q / 64 * D ** -0.5)):
        assert float((got.double() - exact).abs().max()) <= U * abs(exact)
    del x, dq
    torch.cuda.empty_cache()  # 90 GB that the tests behind this one need not carry


def test_inputs_dropped_after_a_call_on_another_stream(lib, cuda):
    # what a call on a given stream reads is not handed out again while it may still be
    # reading: the inputs are gone when the call returns, their sizes are taken and filled on
    # the caller's stream, and the other stream has not begun
    F = lib.functional
    cu_dev = torch.tensor([0, 700, 1500], dtype=torch.int32, device=cuda)
    q, k, v, do = (t.to(cuda) for t in inputs(1500, 16, 8, 64, 1300))
    out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True)
    grads = F.attention_backward(do, q, k, v, out, lse, cu_dev)
    pool = torch.randn(300, 16, 8, 64, device=cuda).to(torch.bfloat16)
    rows = torch.randn(64, 16, 64, device=cuda).to(torch.bfloat16)
    table = torch.randperm(300, device=cuda)[:256].to(torch.int32).view(64, 4)
    lengths = torch.full((64,), 50, dtype=torch.int32, device=cuda)
    one = F.attention_decode(rows, pool, pool, table, lengths)
    side = torch.cuda.Stream()
    calls = {
        "forward": ((q, k, v), lambda s, *t: F.attention_forward(*t, cu_dev, stream=s), (out,)),
        "backward": ((do, q, k, v, out, lse), lambda s, *t: F.attention_backward(*t, cu_dev, stream=s), grads),
        "decode": ((rows, pool), lambda s, r, p: F.attention_decode(r, p, p, table, lengths, stream=s), (one,)),
    }
    for name, (given, call, want) in calls.items():
        for stream in (side, side.cuda_stream):
            torch.cuda.synchronize()
            temporary = [t.clone() for t in given]
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                torch.cuda._sleep(200_000_000)  # about 0.1 s
            got = call(stream, *temporary)
            del temporary
            junk = [torch.full_like(t, float("nan")) for t in given for _ in range(2)]
            side.synchronize()
            got = got if isinstance(got, tuple) else (got,)
            assert all(torch.equal(a, b) for a, b in zip(got, want)), name
            del junk, got
    no_error(lib)
