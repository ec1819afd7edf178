"""The 8-bit write's codes, bit for bit where its inputs are exact: v as it is packed, k
without norm and rotation. A code is x / s as float32 division rounds it, rounded to the
nearest e4m3 value, ties to even; a scale is amax / 448 as float32 division rounds it."""

import pytest
import torch

from test_gpu_pool_write8 import F8, Pool

pytestmark = pytest.mark.gpu


def codes_of(x, s):
    """Codes of x [T, n_kv, D] with scales s [T, n_kv], by torch's division."""
    return (x.float() / s[..., None]).clamp(-448, 448).to(F8).view(torch.uint8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("block", [1, 4, 64])
@pytest.mark.parametrize("size", [1.0, 1e-25, 1e34])
def test_codes_are_those_of_a_division(lib, cuda, D, block, size):
    n_q, n_kv, pages, page_size = 4, 4, 96, 64
    g = torch.Generator(device=cuda).manual_seed(block + D)
    T = pages * page_size - 5
    at = 3 + torch.arange(T, device=cuda, dtype=torch.int32)  # behind 3 held tokens, in any block size
    pool = Pool(pages, page_size, block, n_kv, D, cuda, 7)
    for s in pool.dev_scale:
        s.mul_(size * torch.exp(0.01 * torch.randn(s.shape, generator=g, device=cuda)))
    before = [s.clone() for s in pool.dev_scale]
    rows = torch.randn(T, n_q + 2 * n_kv, D, generator=g, device=cuda)
    rows = (rows * torch.exp(torch.randn(T, 1, 1, generator=g, device=cuda)) * size).to(torch.bfloat16)
    rows[5::97, :, 3::7] = -0.0
    lib.functional.prologue_pool_write8(rows.view(T, -1), None, None, None, at // page_size, at % page_size, *pool.args, n_q,
                                        n_kv, D, "sectioned", norm=False, nope=True)
    for i in range(2):
        x = rows[:, n_q + i * n_kv:n_q + (i + 1) * n_kv]
        scale = pool.dev_scale[i].view(-1, n_kv)
        of = (at // block).long()
        fresh = at[0] % block if block > 1 else 0
        first = int(3 // block + (1 if fresh else 0))  # the first block that begins in the call
        top = torch.zeros(scale.shape, device=cuda).scatter_reduce_(0, of[:, None].expand(T, n_kv), x.float().abs().amax(-1),
                                                                    "amax")
        begun = slice(first, int(of[-1]) + 1)
        # (a tensor of 448s: a division by a number is a product with its reciprocal)
        assert torch.equal(scale[begun], (top / torch.full_like(top, 448.0)).clamp(min=2.0 ** -100)[begun])
        if fresh:
            grown = scale[0] / before[i].view(-1, n_kv)[0]
            assert torch.all(grown == torch.exp2(torch.log2(grown).round()))
        got = pool.dev[i].view(torch.uint8).view(-1, n_kv, D)[3:3 + T]
        want = codes_of(x, scale[of])
        assert torch.equal(got, want), f"pool {i}: {int((got != want).sum())} of {want.numel()} codes"
