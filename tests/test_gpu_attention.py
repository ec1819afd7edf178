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
