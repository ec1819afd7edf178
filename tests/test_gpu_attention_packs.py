"""Packs of very many and of very long sequences: the order in which the kernels
take their work, the time that finding it costs, and the error of whole tensors."""

import numpy as np
import pytest
import torch

import oracle.attention as A
from attention_parity import U, assert_lse, assert_within, out_bound
from test_gpu_attention import f64, inputs, no_error, offsets

pytestmark = pytest.mark.gpu


def step(F, dev, cu_dev):
    q, k, v, do = dev
    out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True)
    return (out, lse, *F.attention_backward(do, q, k, v, out, lse, cu_dev))


def milliseconds(call):
    for _ in range(2):
        call()
    best = float("inf")
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("rows,n_q,n_kv", [(8, 4, 1), (70, 2, 2)])
def test_time_grows_with_the_number_of_sequences_not_its_square(lib, cuda, rows, n_q, n_kv):
    # eight times the sequences are eight times the work; a search through all of them for
    # every work item would be sixty-four
    F = lib.functional
    took = []
    for batch in (4096, 32768):
        dev = [t.to(cuda) for t in inputs(batch * rows, n_q, n_kv, 64, batch)]
        cu_dev = torch.arange(batch + 1, dtype=torch.int32, device=cuda) * rows
        q, k, v, do = dev
        out, lse = F.attention_forward(q, k, v, cu_dev, save_lse=True)
        took.append([milliseconds(lambda: F.attention_forward(q, k, v, cu_dev)),
                     milliseconds(lambda: F.attention_backward(do, q, k, v, out, lse, cu_dev))])
    no_error(lib)
    print("ms:", took)
    assert took[1][0] < 16 * took[0][0] and took[1][1] < 16 * took[0][1], took


@pytest.mark.parametrize("n_q,n_kv,D", [(4, 1, 64), (3, 3, 64), (2, 1, 128)])
@pytest.mark.parametrize("batch,rows", [(20001, 3), (5000, 33), (2003, 140)])
def test_thousands_of_sequences(lib, cuda, batch, rows, n_q, n_kv, D):
    # all of one length, so that the definition is one batched product in float64
    F = lib.functional
    T = batch * rows
    dev = [t.to(cuda) for t in inputs(T, n_q, n_kv, D, 2000 + batch)]
    cu_dev = torch.arange(batch + 1, dtype=torch.int32, device=cuda) * rows
    out, lse, dq, dk, dv = step(F, dev, cu_dev)
    no_error(lib)
    G = n_q // n_kv

    def heads(t):  # [batch, heads, rows, D]
        return t.double().view(batch, rows, -1, D).transpose(1, 2)

    def back(t):
        return t.transpose(1, 2).reshape(T, -1, D)

    q, do = heads(dev[0]), heads(dev[3])
    k, v = (heads(t).repeat_interleave(G, 1) for t in dev[1:3])
    s = q @ k.transpose(2, 3) * D ** -0.5
    s.masked_fill_(torch.ones(rows, rows, dtype=torch.bool, device=cuda).triu(1), float("-inf"))
    p = s.softmax(3)
    o = p @ v
    dp = do @ v.transpose(2, 3)
    ds = p * (dp - (do * o).sum(3, keepdim=True)) * D ** -0.5
    fold = lambda t: t.view(batch, n_kv, G, rows, D).sum(2)
    ref = {"out": back(o).cpu().numpy(), "out_abs": back(p @ v.abs()).cpu().numpy()}
    assert_within(out.double().cpu().numpy(), ref["out"], out_bound(ref), "out")
    want = s.logsumexp(3).transpose(0, 1).reshape(n_q, T)
    s_abs = float((q.abs() @ k.abs().transpose(2, 3)).max()) * D ** -0.5
    bound = 2.0 ** -24 * (2 * (D + 4) * s_abs + 4 * float(want.abs().max()) + rows / 2 + 64)
    assert float((lse - want).abs().max()) <= bound
    for name, got, exact in (("dq", dq, ds @ k), ("dk", dk, fold(ds.transpose(2, 3) @ q)),
                             ("dv", dv, fold(p.transpose(2, 3) @ do))):
        assert_norm(got, back(exact), name)


def assert_norm(got, exact, name):
    # a bf16 rounding is off by up to 2^-8 of the power of two below the value, evenly spread:
    # 2^-8 / 3^0.5 = 0.0023 as root mean square, over values of 1 to 2 about 0.0016 of them. One for
    # the result, one for p or ds as an operand, one for out inside delta; independent ones add
    # as squares, 3^0.5 0.0016 = 0.0028
    got, exact = (torch.as_tensor(x).double().cpu() for x in (got, exact))
    off = float((got - exact).norm() / exact.norm())
    assert off <= 0.005, f"{name}: {off:.5f} of its norm"


@pytest.mark.parametrize("n_q,n_kv,D", [(16, 1, 64), (8, 2, 128), (3, 3, 64)])
def test_error_of_whole_tensors(lib, cuda, n_q, n_kv, D):
    # bounds for single elements are wide where many rows are added up; a part left out of
    # dk or dv would show here
    lengths = [300, 5, 77, 640, 129]
    cu = offsets(lengths)
    host = inputs(int(cu[-1]), n_q, n_kv, D, 2100)
    got = step(lib.functional, [t.to(cuda) for t in host], torch.from_numpy(cu).to(cuda))
    no_error(lib)
    x = [f64(t) for t in host]
    fwd, bwd = A.attention_fwd(*x[:3], cu), A.attention_bwd(x[3], *x[:3], cu)
    assert_norm(f64(got[0]), fwd["out"], "out")
    for name, g in zip(("dq", "dk", "dv"), got[2:]):
        assert_norm(f64(g), bwd[name], name)


@pytest.mark.parametrize("n_q,n_kv,D", [(4, 2, 64), (3, 1, 64), (2, 1, 128)])
def test_long_sequences_among_many(lib, cuda, n_q, n_kv, D):
    # up to 36 blocks of 128 rows, so that blocks of neighbouring costs are taken together,
    # beside some two hundred short sequences and empty ones
    rng = np.random.default_rng(7)
    lengths = [4500, 0, 2300, 2049] + rng.integers(0, 700, size=12).tolist() + rng.integers(0, 90, size=200).tolist()
    rng.shuffle(lengths)
    cu = offsets(lengths, 5)
    T = int(cu[-1]) + 3
    host = inputs(T, n_q, n_kv, D, 2200)
    got = step(lib.functional, [t.to(cuda) for t in host], torch.from_numpy(cu).to(cuda))
    no_error(lib)
    x = [f64(t) for t in host]
    fwd = A.attention_fwd(*x[:3], cu)
    assert_within(f64(got[0]), fwd["out"], out_bound(fwd), "out")
    assert_lse(got[1].cpu().numpy(), fwd, max(lengths), D, "lse")
    bwd = A.attention_bwd(x[3], *x[:3], cu, out_err=out_bound(fwd))
    for name, g in zip(("dq", "dk", "dv"), got[2:]):
        assert_within(f64(g), bwd[name], bwd["e_" + name] + U * np.abs(bwd[name]), name)
        assert_norm(f64(g), bwd[name], name)
