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


def test_prefix_in_several_ranges(lib, cuda):
    # a prefix longer than one CTA's keys, for more rows than a tile, in both head sizes
    for n_q, n_kv, D, B in ((16, 1, 64, 20), (8, 2, 128, 70)):
        w = Batch(n_q, n_kv, D, 32, [3] * (B - 1) + [40], 9000, 3)
        w.check(lib, *w.run(lib, cuda, save_lse=True), what=f"D {D}")


@pytest.mark.parametrize("prefix", [0, 300])
def test_bad_pages_are_not_attended(lib, cuda, prefix):
    w = Batch(8, 2, 64, 16, [100, 7, 33], prefix, 4)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    w.run(lib, cuda, dev_status=status)
    assert status.item() == 0
    keep = [list(range(n)) for n in (100, 7, 33)]
    w.table[0, 2] = -1
    w.table[2, 1] = w.k_pool.shape[0]
    drop = {0: range(32, 48), 2: range(16, 32)}
    for b, rows in drop.items():
        keep[b] = [t for t in keep[b] if t not in rows]
    shared = list(range(prefix))
    if prefix:
        w.prefix_pages[5] = 2 ** 31 - 1
        w.prefix_pages[-1] = -2 ** 31
        shared = [t for t in shared if t // 16 not in (5, len(w.prefix_pages) - 1)]
    for b in range(3):
        rows = shared + [prefix + t for t in keep[b]]
        w.keys[b], w.values[b] = w.keys[b][rows], w.values[b][rows]
    got = w.run(lib, cuda, save_lse=True, dev_status=status)
    w.check(lib, *got)
    assert status.item() == lib.QKVP_DEV_BAD_PAGE


def test_bad_lengths_are_clamped(lib, cuda):
    w = Batch(8, 2, 64, 16, [64, 5], 0, 5)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    want = w.run(lib, cuda)
    w.lengths[0] = 10 ** 6
    got = w.run(lib, cuda, dev_status=status)
    assert status.item() == lib.QKVP_DEV_BAD_LENGTH and torch.equal(got, want)
    w.lengths[0] = -3
    got = w.run(lib, cuda, dev_status=status)
    assert not got[0].any() and torch.equal(got[1], want[1])
    torch.cuda.synchronize()
    assert lib.qkv_prologue_device_error(clear=True) == 0


def test_table_slices_out_and_workspace(lib, cuda):
    F = lib.functional
    w = Batch(8, 2, 128, 64, [200, 64, 1], 130, 6)
    want = w.run(lib, cuda)
    wide = torch.full((3, 11), 10 ** 6, dtype=torch.int32)
    wide[:, 2:2 + w.table.shape[1]] = w.table
    table = wide.to(cuda)[:, 2:2 + w.table.shape[1]]
    need = F.attention_decode_workspace_bytes(8, 2, 128, 3, 64, table.shape[1], 130)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=cuda)
    out = torch.full((3, 8, 128), 7.0, dtype=torch.bfloat16, device=cuda)
    args = [t.to(cuda) for t in (w.q, w.k_pool, w.v_pool)]
    got = F.attention_decode(*args, table, w.lengths.to(cuda), w.prefix_pages.to(cuda), 130, out=out, workspace=ws)
    assert got is out and torch.equal(out, want)
    with pytest.raises(lib.QkvpError):
        F.attention_decode(*args, table, w.lengths.to(cuda), w.prefix_pages.to(cuda), 130, workspace=ws[:need - 16])
    with pytest.raises(ValueError):
        F.attention_decode(*args, table, w.lengths.to(cuda), w.prefix_pages.to(cuda)[:2], 130)
    with pytest.raises(ValueError):
        F.attention_decode(*args, table[:2], w.lengths.to(cuda))
    with pytest.raises(ValueError):  # rows that overlap
        F.attention_decode(*args, table[:1].expand(3, -1), w.lengths.to(cuda))
    torch.cuda.synchronize()
    assert lib.qkv_prologue_device_error(clear=True) == 0


@pytest.mark.parametrize("prefix", [0, 200])
def test_captured_call_follows_lengths_that_grow(lib, cuda, prefix):
    F = lib.functional
    w = Batch(8, 2, 64, 16, [90, 17, 260, 33], prefix, 7)
    args = [t.to(cuda) for t in (w.q, w.k_pool, w.v_pool, w.table, w.lengths)]
    pages = w.prefix_pages.to(cuda) if prefix else None
    n = args[4]
    F.attention_decode(*args, pages, prefix)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = F.attention_decode(*args, pages, prefix)
    for lengths in ([1, 1, 1, 1], [0, 17, 100, 0], [90, 17, 260, 33]):
        n.copy_(torch.tensor(lengths, dtype=torch.int32))
        out.fill_(float("nan"))
        g.replay()
        short = [k[:prefix + m] for k, m in zip(w.keys, lengths)], [v[:prefix + m] for v, m in zip(w.values, lengths)]
        ref = A.attention_decode(f64(w.q), *short)
        assert_within(f64(out), ref["out"], out_bound(ref), str(lengths))
        assert torch.equal(out, F.attention_decode(*args, pages, prefix))  # repeats bit for bit
    torch.cuda.synchronize()
    assert lib.qkv_prologue_device_error(clear=True) == 0


def test_pool_beyond_32_bit_offsets(lib, cuda):
    # the last pages of a pool of more than 2^32 bytes (and 2^31 values)
    n_kv, D, page_size = 8, 128, 64
    pages = (2 ** 31 + 2 ** 27) // (n_kv * D * page_size)
    w = Batch(16, n_kv, D, page_size, [100, 70], 150, 8)
    small = w.k_pool.shape[0]
    big = [torch.empty(pages, page_size, n_kv, D, dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    for b, s in zip(big, (w.k_pool, w.v_pool)):
        b[:small] = float("nan")
        b[-small:] = s.to(cuda)
    table, shared = w.table.clone(), w.prefix_pages.clone()
    table[table >= 0] += pages - small
    shared += pages - small
    got = lib.functional.attention_decode(w.q.to(cuda), *big, table.to(cuda), w.lengths.to(cuda), shared.to(cuda), 150)
    w.check(lib, got, None, "far pages")
    got = lib.functional.attention_decode(w.q[:1].to(cuda), *big, table[:1].to(cuda), w.lengths[:1].to(cuda),
                                          shared.to(cuda), 150)
    assert_within(f64(got), *(lambda r: (r["out"], out_bound(r)))(A.attention_decode(f64(w.q[:1]), w.keys[:1],
                                                                                     w.values[:1])), "one sequence")


def test_nothing_to_do(lib, cuda):
    F = lib.functional
    w = Batch(8, 2, 64, 16, [5], 0, 9)
    args = [t.to(cuda) for t in (w.q, w.k_pool, w.v_pool, w.table, w.lengths)]
    assert F.attention_decode(args[0][:0], *args[1:3], args[3][:0], args[4][:0]).shape == (0, 8, 64)
    out, lse = F.attention_decode(*args[:3], args[3][:, :0], torch.zeros_like(args[4]), save_lse=True)
    assert not out.any() and torch.isneginf(lse).all()
    torch.cuda.synchronize()
    assert lib.qkv_prologue_device_error(clear=True) == 0


def test_pool_write_then_decode_is_the_prompt(lib, cuda):
    # the prompt's k and v written into the pool by the prologue; the decode of its
    # last token is the last row of the prompt's attention, each within its bound
    import workloads

    F = lib.functional
    T, n_q, n_kv, D, page_size = 150, 8, 2, 64, 16
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=31, rope_base=10000.0)
    g = torch.Generator().manual_seed(1)
    order = torch.randperm(12, generator=g).to(torch.int32)
    at = torch.arange(T)
    page, off = order[at // page_size].to(cuda), (at % page_size).to(torch.int32).to(cuda)
    pools = [torch.full((12, page_size, n_kv, D), float("nan"), dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    rows, pos = wl.packed_rows().to(cuda), wl.pos.to(cuda)
    w_q, w_k = wl.w_q.to(cuda), wl.w_k.to(cuda)
    q = F.prologue_pool_write(rows, pos, w_q, w_k, page, off, *pools, n_q, n_kv, D, eps=wl.eps, rope_base=wl.rope_base)
    _, k, v = F.prologue_forward(rows, pos, w_q, w_k, n_q, n_kv, D, eps=wl.eps, rope_base=wl.rope_base)
    cu = np.array([0, T])
    ref = A.attention_fwd(f64(q), f64(k), f64(v), cu)
    prompt = F.attention_forward(q, k, v, torch.tensor([0, T], dtype=torch.int32, device=cuda))
    assert_within(f64(prompt), ref["out"], out_bound(ref), "prompt")
    n = torch.tensor([T], dtype=torch.int32, device=cuda)
    one = F.attention_decode(q[-1:].contiguous(), *pools, order[None].to(cuda), n)
    assert_within(f64(one)[0], ref["out"][-1], out_bound(ref)[-1], "decode")
    torch.cuda.synchronize()
    assert lib.qkv_prologue_device_error(clear=True) == 0


def test_pages_named_twice(lib, cuda):
    # two sequences with the same pages, a page twice in one sequence, and the
    # prefix's first page among the own ones
    w = Batch(8, 2, 64, 16, [48, 48, 20], 144, 41)
    w.table[1, :3] = w.table[0, :3]
    w.table[2, 0], w.table[2, 1] = w.prefix_pages[0], w.prefix_pages[0]
    for b, pages in ((1, w.table[1, :3]), (2, w.table[2, :2])):
        n = int(w.lengths[b])
        for kept, pool in ((w.keys, w.k_pool), (w.values, w.v_pool)):
            own = f64(pool[pages.long()].reshape(-1, *pool.shape[2:])[:n].contiguous())
            kept[b] = np.concatenate([kept[b][:144], own])
    w.check(lib, *w.run(lib, cuda, save_lse=True))


@pytest.mark.parametrize("prefix", [0, 300])
def test_two_calls_at_once_and_refusals(lib, cuda, prefix):
    F = lib.functional
    sets = [Batch(8, 2, 64, 16, [700, 30, 0, 5], prefix, 50 + i) for i in range(2)]
    want = [w.run(lib, cuda, save_lse=True) for w in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    dev = [[t.to(cuda) for t in (w.q, w.k_pool, w.v_pool, w.table, w.lengths, w.prefix_pages)] for w in sets]
    torch.cuda.synchronize()
    busy = torch.randn(8192, 8192, device=cuda)
    for _ in range(3):
        busy = busy @ busy * 1e-4
    got = [[F.attention_decode(*x, prefix, save_lse=True, stream=s) for _ in range(4)] for x, s in zip(dev, streams)]
    for s in streams:
        s.synchronize()
    for each, ref in zip(got, want):
        assert all(torch.equal(a, b) for one in each for a, b in zip(one, ref))
    x = dev[0]
    need = F.attention_decode_workspace_bytes(8, 2, 64, 4, 16, x[3].shape[1], prefix)
    for bad in (torch.zeros(need, dtype=torch.uint8), torch.zeros(2 * need, dtype=torch.uint8, device=cuda)[::2]):
        with pytest.raises(ValueError):
            F.attention_decode(*x, prefix, workspace=bad)
    with pytest.raises(lib.QkvpError):
        F.attention_decode(*x, prefix, out=x[0])
    with pytest.raises(lib.QkvpError):
        F.attention_decode(*x, prefix, out=x[1].flatten()[:x[0].numel()].view(x[0].shape))
    torch.cuda.synchronize()
    assert lib.qkv_prologue_device_error(clear=True) == 0


@pytest.mark.parametrize("n_q,n_kv,D", [(160, 1, 64), (130, 1, 128)])
@pytest.mark.parametrize("prefix", [0, 200])
def test_groups_wider_than_a_tile(lib, cuda, n_q, n_kv, D, prefix):
    # more query heads per key/value head than the shared prefix's kernel has rows
    w = Batch(n_q, n_kv, D, 16, [70, 0, 33], prefix, 60)
    w.check(lib, *w.run(lib, cuda, save_lse=True))


def test_results_on_a_side_stream_in_a_graph(lib, cuda):
    # a captured call on a stream forked from the capturing one
    F = lib.functional
    w = Batch(8, 2, 64, 16, [70, 0, 33], 150, 61)
    x = [t.to(cuda) for t in (w.q, w.k_pool, w.v_pool, w.table, w.lengths, w.prefix_pages)]
    want = F.attention_decode(*x, 150)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = F.attention_decode(*x, 150, stream=side)
        torch.cuda.current_stream().wait_stream(side)
    got.fill_(float("nan"))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want) and lib.qkv_prologue_device_error(clear=True) == 0


@pytest.mark.parametrize("prefix", [0, 130])
def test_as_many_sequences_as_allowed(lib, cuda, prefix):
    # 2^20, all but a few without tokens of their own
    F = lib.functional
    n_q, n_kv, D, size, batch = 2, 1, 64, 16, 2 ** 20
    w = Batch(n_q, n_kv, D, size, [3, 40, 17], prefix, 70)
    at = torch.tensor([0, 500000, batch - 1])
    q = torch.zeros(batch, n_q, D, dtype=torch.bfloat16)
    table, lengths = torch.zeros(batch, w.table.shape[1], dtype=torch.int32), torch.zeros(batch, dtype=torch.int32)
    q[at], table[at], lengths[at] = w.q, w.table, w.lengths
    x = [t.to(cuda) for t in (q, w.k_pool, w.v_pool, table, lengths, w.prefix_pages)]
    out, lse = F.attention_decode(*x[:5], x[5] if prefix else None, prefix, save_lse=True)
    w.check(lib, out[at.to(cuda)], lse[at.to(cuda)])
    if not prefix:
        rest = torch.ones(batch, dtype=torch.bool, device=cuda)
        rest[at.to(cuda)] = False
        assert not out[rest].any() and torch.isneginf(lse[rest]).all()


@pytest.mark.parametrize("n_q,n_kv,D", [(5, 1, 64), (14, 2, 128), (6, 2, 64)])
def test_the_same_bits_whatever_ran_before(lib, cuda, n_q, n_kv, D):
    # groups whose rows do not fill the prefix kernel's tiles: what an earlier kernel left
    # in shared memory is in the rest, and does not show
    F = lib.functional
    w = Batch(n_q, n_kv, D, 16, [30] * 60, 2000, 80)
    want = w.run(lib, cuda, save_lse=True)
    w.check(lib, *want)
    other = Batch(128 * n_kv, n_kv, D, 16, [3, 5], 400, 81)
    for factor in (1.0, 1e4, float("nan")):
        other.q.copy_(torch.randn_like(other.q.float()) * factor)
        for _ in range(3):
            other.run(lib, cuda)
            assert all(torch.equal(a, b) for a, b in zip(w.run(lib, cuda, save_lse=True), want))


def test_a_refused_call_leaves_no_workspace_size_behind(lib, cuda, monkeypatch):
    # sizes are kept by device: not the current device's under the tensors' one
    F = lib.functional
    x = Batch(4, 2, 64, 16, [37], 0, 70, wide=5)
    kept = F._decode_workspace.cache_info().currsize
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: cuda.index + 1)
        with pytest.raises(ValueError):
            x.run(lib, cuda)
    assert F._decode_workspace.cache_info().currsize == kept
    x.check(lib, *x.run(lib, cuda, save_lse=True))


def test_one_sequence_in_more_parts_than_factors_fit(lib, cuda):
    # 70,000 keys of one head: more than 1024 partial results, joined in two rounds
    x = Batch(4, 1, 64, 64, [70000], 0, 71)
    x.check(lib, *x.run(lib, cuda, save_lse=True))


@pytest.mark.parametrize("n_q,n_kv,D", [(4, 1, 64), (3, 1, 128)])
def test_one_long_sequence_among_many_short_ones(lib, cuda, n_q, n_kv, D):
    # nearly all parts are one sequence's: one warp joins them, 128 a round
    lengths = [3 + i % 7 for i in range(200)]
    lengths[77] = 60000
    x = Batch(n_q, n_kv, D, 64, lengths, 0, 72)
    x.check(lib, *x.run(lib, cuda, save_lse=True))
