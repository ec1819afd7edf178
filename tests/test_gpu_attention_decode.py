"""Attention of single tokens over the paged pool, with and without a shared
prefix, against the float64 oracle. Every pool slot that no sequence names
holds a NaN, and page numbers are a random permutation."""

import numpy as np
import pytest
import torch

import oracle.attention as A
from attention_parity import assert_lse, assert_within, out_bound
from oracle.bf16 import bf16_bits_to_f64
from workloads import bits_u16 as u16

pytestmark = pytest.mark.gpu


def f64(t):
    return bf16_bits_to_f64(u16(t))


class Batch:
    """A decode batch with its pools: `lengths` own tokens after `prefix` shared ones."""

    def __init__(self, n_q, n_kv, D, page_size, lengths, prefix, seed, spare=2, wide=0):
        g = torch.Generator(device="cpu")
        g.manual_seed(seed)
        need = [-(-n // page_size) for n in lengths]
        n_prefix = -(-prefix // page_size)
        pages = sum(need) + n_prefix + spare
        order = torch.randperm(pages, generator=g).to(torch.int32)
        shape = (pages, page_size, n_kv, D)
        self.k_pool = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        self.v_pool = torch.full(shape, float("nan"), dtype=torch.bfloat16)
        self.q = torch.randn(len(lengths), n_q, D, generator=g).to(torch.bfloat16)
        self.table = torch.full((len(lengths), max(need + [0]) + wide), -7, dtype=torch.int32)
        self.lengths = torch.tensor(lengths, dtype=torch.int32)
        self.prefix, self.page_size = prefix, page_size

        def fill(page_list, n):
            k = torch.randn(n, n_kv, D, generator=g).to(torch.bfloat16)
            v = torch.randn(n, n_kv, D, generator=g).to(torch.bfloat16)
            for t in range(n):
                self.k_pool[page_list[t // page_size], t % page_size] = k[t]
                self.v_pool[page_list[t // page_size], t % page_size] = v[t]
            return f64(k), f64(v)

        self.prefix_pages = order[:n_prefix].contiguous()
        pk, pv = fill(self.prefix_pages.tolist(), prefix)
        self.keys, self.values = [], []
        at = n_prefix
        for b, n in enumerate(lengths):
            mine = order[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = mine
            k, v = fill(mine.tolist(), n)
            self.keys.append(np.concatenate([pk, k]))
            self.values.append(np.concatenate([pv, v]))

    def run(self, lib, dev, **kw):
        return lib.functional.attention_decode(
            self.q.to(dev), self.k_pool.to(dev), self.v_pool.to(dev), self.table.to(dev), self.lengths.to(dev),
            self.prefix_pages.to(dev) if self.prefix else None, self.prefix, **kw)

    def check(self, lib, got, lse, what=""):
        torch.cuda.synchronize()
        assert lib.qkv_prologue_device_error(clear=True) == 0
        ref = A.attention_decode(f64(self.q), self.keys, self.values)
        assert_within(f64(got), ref["out"], out_bound(ref), what + " out")
        if lse is not None:
            n = max([k.shape[0] for k in self.keys] + [1])
            assert_lse(lse.cpu().numpy(), ref, n, self.q.shape[2], what + " lse")


HEADS = [(8, 2, 64), (4, 2, 128), (3, 3, 64), (7, 1, 128), (40, 2, 64)]


@pytest.mark.parametrize("n_q,n_kv,D", HEADS)
@pytest.mark.parametrize("page_size", [1, 16, 24, 64, 100])
@pytest.mark.parametrize("lengths", [[1], [0], [17, 0, 64, 1, 300], [2500, 16]])
def test_own_keys(lib, cuda, n_q, n_kv, D, page_size, lengths):
    w = Batch(n_q, n_kv, D, page_size, lengths, 0, 7 + page_size, wide=1)
    w.check(lib, *w.run(lib, cuda, save_lse=True))


@pytest.mark.parametrize("n_q,n_kv,D", HEADS)
@pytest.mark.parametrize("page_size", [1, 8, 24, 64, 256])
@pytest.mark.parametrize("prefix", [1, 127, 128, 700])
@pytest.mark.parametrize("lengths", [[3], [0, 0], [17, 0, 64, 1, 300], [5] * 37])
def test_shared_prefix(lib, cuda, n_q, n_kv, D, page_size, prefix, lengths):
    w = Batch(n_q, n_kv, D, page_size, lengths, prefix, 70 + page_size + prefix)
    w.check(lib, *w.run(lib, cuda, save_lse=True))
