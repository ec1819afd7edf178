"""The 8-bit write's launches with many sizes of shared memory, from several threads."""

import threading

import pytest
import torch

from test_gpu_pool_write8 import Pool

pytestmark = pytest.mark.gpu


def test_many_sizes_from_many_threads(lib, cuda):
    """The blocks' sizes set how much shared memory a launch takes. Behind hundreds of them
    calls that take much and calls that take little, from a thread each: none takes away what
    another's launch needs."""
    F, n_q, n_kv, D = lib.functional, 2, 1, 64
    g = torch.Generator(device=cuda).manual_seed(1)
    w, zero = torch.ones(D, device=cuda), torch.zeros(1, dtype=torch.int32, device=cuda)

    def call(block, **options):
        pool = Pool(1, block, block, n_kv, D, cuda)
        rows = torch.randn(1, (n_q + 2 * n_kv) * D, generator=g, device=cuda).to(torch.bfloat16)
        args = (rows, zero, w, w, zero, zero, *pool.args, n_q, n_kv, D)
        return lambda: F.prologue_pool_write8(*args, **options)

    for block in range(1, 161):  # (a table of 160 tokens is the largest)
        call(block)()
        call(block, norm=False)()
    L, flags = lib.layout("interleaved", n_q, n_kv, D), lib.QKVP_ROPE_PAIRS

    def bare(block):
        """The C call with its arguments at hand: little time goes by outside of it."""
        pool = Pool(1, block, block, n_kv, D, cuda)
        rows = torch.randn(1, (n_q + 2 * n_kv) * D, generator=g, device=cuda).to(torch.bfloat16)
        q = torch.empty(1, n_q, D, dtype=torch.bfloat16, device=cuda)
        keep = (rows, zero, w, w, 1e-6, 1e4, flags, q, zero, zero, *pool.args)
        args = [t.data_ptr() if isinstance(t, torch.Tensor) else t for t in keep]
        f = lambda: lib.qkv_prologue_pool_write8(L, None, 1, *args, 1, block, block, None, stream, check=False)  # noqa: E731
        return f, keep

    stream = torch.cuda.current_stream().cuda_stream
    calls = [bare(b) for b in (1, 400) * 4]
    torch.cuda.synchronize()
    failed = []

    def work(f):
        torch.cuda.set_device(cuda)
        for i in range(10000):
            status = f()
            if status != lib.QKVP_OK:
                failed.append((i, lib.qkv_prologue_status_string(status)))
                return

    threads = [threading.Thread(target=work, args=(f,)) for f, _ in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]
