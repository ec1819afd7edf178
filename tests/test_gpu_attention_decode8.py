"""Attention of single tokens over the 8-bit pool against the float64 oracle on
the values that the pool holds. Slots that no sequence names hold NaN codes and
blocks that none names NaN scales; page numbers are a random permutation.

Bound: the softmax weights (times the values' scales) are rounded to f16, half a
step is 2^-11; the fp32 arithmetic around them and q's own rounding (2^-25 of a
row's largest magnitude) stay below 2^-10 as in attention_parity.py; the result
is rounded to bf16."""

import numpy as np
import pytest
import torch

import oracle.attention as A
import oracle.pool8 as E8
import workloads
from attention_parity import EDGE, U, assert_lse, assert_within
from oracle.bf16 import bf16_bits_to_f64
from workloads import bits_u16 as u16

pytestmark = pytest.mark.gpu
F8 = torch.float8_e4m3fn


def f64(t):
    return bf16_bits_to_f64(u16(t))


def bound(ref):
    return U * np.abs(ref["out"]) + (2.0 ** -11 + EDGE) * (1 + U) * ref["out_abs"]


class Batch:
    def __init__(self, n_q, n_kv, D, page_size, block, lengths, seed, spare=2, wide=0, spread=2.0, size=1.0):
        g = np.random.default_rng(seed)
        need = [-(-n // page_size) for n in lengths]
        pages = sum(need) + spare
        order = g.permutation(pages)
        shape = (pages, page_size, n_kv, D)
        self.codes = [np.full(shape, 127, np.uint8) for _ in range(2)]
        self.scale = [np.full((pages, page_size // block, n_kv), np.nan, np.float32) for _ in range(2)]
        self.q = torch.from_numpy(g.standard_normal((len(lengths), n_q, D)) * size).to(torch.bfloat16)
        self.table = np.full((len(lengths), max(need + [0]) + wide), -7, np.int32)
        self.lengths = np.array(lengths, np.int32)
        self.keys, self.values = [], []
        at = 0
        for b, n in enumerate(lengths):
            mine = order[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = mine
            rows = []
            for c, s in zip(self.codes, self.scale):
                x = g.standard_normal((n, n_kv, D))
                i = np.arange(n)
                p, o = mine[i // page_size], i % page_size
                # a scale for each block that is used, apart by powers of e
                for pg, j in {(int(a), int(b) // block) for a, b in zip(p, o)}:
                    s[pg, j] = np.exp(g.uniform(-spread, spread, n_kv)) / 448
                c[p, o] = E8.to_e4m3(x / 4 * 448)
                rows.append(E8.VALUES[c[p, o]] * s[p, o // block].astype(np.float64)[..., None])
            self.keys.append(rows[0])
            self.values.append(rows[1])

    def args(self, dev):
        put = lambda x: torch.from_numpy(x).to(dev)  # noqa: E731
        return (self.q.to(dev), *(put(c).view(F8) for c in self.codes), *(put(s) for s in self.scale), put(self.table),
                put(self.lengths))

    def run(self, lib, dev, **kw):
        return lib.functional.attention_decode8(*self.args(dev), **kw)

    def want(self, scale=None):
        return A.attention_decode(f64(self.q), self.keys, self.values, scale)


def check(lib, dev, b, scale=None, what=""):
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    out, lse = b.run(lib, dev, save_lse=True, scale=scale, dev_status=status)
    ref = b.want(scale)
    assert_within(f64(out), ref["out"], bound(ref), what)
    assert_lse(lse.cpu().numpy(), ref, max([k.shape[0] for k in b.keys] + [0]), b.q.shape[2], what)
    assert int(status) == 0
    again = b.run(lib, dev, scale=scale)
    assert torch.equal(out, again), f"{what}: two runs"


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n_q, n_kv", [(1, 1), (2, 1), (6, 2), (9, 3), (16, 4), (5, 1), (14, 2), (32, 4), (32, 2), (20, 1), (40, 1)])
def test_groups(lib, cuda, n_q, n_kv, D):
    check(lib, cuda, Batch(n_q, n_kv, D, 16, 8, [1, 31, 0, 32, 33, 200, 64, 65], 1), what=f"{n_q} over {n_kv}")


@pytest.mark.parametrize("page_size, block", [(1, 1), (8, 2), (24, 24), (24, 3), (64, 16), (64, 1), (100, 25), (100, 4),
                                              (256, 128)])
def test_pages_and_blocks(lib, cuda, page_size, block):
    check(lib, cuda, Batch(8, 2, 64, page_size, block, [1, 99, 100, 101, 0, 517], 2), what=f"page {page_size}")
    check(lib, cuda, Batch(4, 2, 128, page_size, block, [257, 3], 3, wide=3), what=f"page {page_size}")


@pytest.mark.parametrize("lengths", [[1], [2], [31], [32], [33], [63], [64], [65], [127], [0, 0, 0], [0, 5, 0], [4097],
                                     [1] * 70, [0] * 40 + [3] + [0] * 40, [3000, 1, 0, 700]])
def test_lengths(lib, cuda, lengths):
    for D in (64, 128):
        check(lib, cuda, Batch(8, 2, D, 16, 16, lengths, 4), what=f"{lengths[:4]}")


def test_many_sequences(lib, cuda):
    rng = np.random.default_rng(5)
    check(lib, cuda, Batch(16, 2, 64, 16, 8, [int(n) for n in rng.integers(0, 300, 150)], 5))
    check(lib, cuda, Batch(32, 8, 128, 64, 16, [int(n) for n in rng.integers(0, 900, 20)], 6))


@pytest.mark.parametrize("spread", [20.0, 60.0])
def test_scales_far_apart(lib, cuda, spread):
    # keys of tiny and of huge values among each other: scores from one block alone, or ties of many
    b = Batch(8, 2, 64, 16, 8, [200, 33, 1, 40], 7, spread=spread)
    for s in b.scale[:1]:  # the keys' scales stay moderate, so the weights are spread; the values' are apart
        s[np.isfinite(s)] = 1 / 448
    b.keys = [E8.VALUES[b.codes[0]][b.table[i, np.arange(n) // 16], np.arange(n) % 16] / np.float64(np.float32(448)) * 1.0
              for i, n in enumerate(b.lengths)]
    b.keys = [k * (np.float64(np.float32(1 / 448)) * 448) for k in b.keys]
    check(lib, cuda, b, what=f"spread {spread}")


def test_sharp_scores(lib, cuda):
    # scores up to about 60 in magnitude, of both signs, in rising and falling order of length
    check(lib, cuda, Batch(8, 2, 64, 16, 8, [700, 40, 3], 8, spread=0.5, size=6.0), what="sharp")
    check(lib, cuda, Batch(8, 2, 128, 64, 64, [700, 40, 3], 9, spread=0.5), scale=0.5, what="scale")


@pytest.mark.parametrize("D, group", [(64, 1), (64, 12), (128, 8)])
@pytest.mark.parametrize("power", [20, 26, 30])
def test_a_key_that_takes_the_weight_and_gives_nothing(lib, cuda, D, group, power):
    # the first key's weight is 2^power times the others', its value 0: the result is theirs.
    # 16 bits hold weights to 2^-25 of the reference, which lies 2^11 or more below the largest.
    b = Batch(group, 1, D, 16, 16, [60], 30 + power)
    for s in b.scale:
        s[np.isfinite(s)] = 1.0
    at = b.table[0, 0]
    used = b.codes[0] != 127
    b.codes[0][used] = 0
    b.codes[0][at, 0, 0, 0] = E8.to_e4m3(np.float64(power))
    b.codes[1][at, 0] = 0
    b.q.zero_()
    b.q[:, :, 0] = 1
    n = np.arange(60)
    rows = b.table[0, n // 16], n % 16
    b.keys, b.values = [E8.VALUES[b.codes[0][rows]]], [E8.VALUES[b.codes[1][rows]]]
    scale = float(np.log(2.0))
    ref = b.want(scale)
    assert np.abs(ref["out"]).max() > 2.0 ** -power
    lost = 2.0 ** -36 * np.abs(b.values[0]).sum(0)[None]  # (the largest weight is at most 1)
    assert_within(f64(b.run(lib, cuda, scale=scale)), ref["out"], bound(ref) + lost, f"2^{power}")


def test_the_smallest_scales(lib, cuda):
    # every value below 2^-91, many equal weights: no factor on the way falls out of float32
    b = Batch(4, 2, 64, 16, 8, [3000, 70], 61)
    b.q.zero_()
    for s in b.scale[1:]:
        s[np.isfinite(s)] = 2.0 ** -100
    b.values = [E8.VALUES[b.codes[1][b.table[i, np.arange(n) // 16], np.arange(n) % 16]] * 2.0 ** -100
                for i, n in enumerate(b.lengths)]
    ref = b.want()
    got = f64(b.run(lib, cuda))
    assert_within(got * 2.0 ** 100, ref["out"] * 2.0 ** 100, bound(ref) * 2.0 ** 100, "2^-100")


def test_large_and_small_queries(lib, cuda):
    # a row's power of two: queries of 2^-100 .. 2^100 with a scale that undoes it
    for e in (-120, -60, -1, 0, 1, 60, 100):
        b = Batch(4, 1, 64, 16, 8, [90, 17], 10)
        ref = b.want()
        b.q = (b.q.double() * 2.0 ** e).to(torch.bfloat16)
        out = b.run(lib, cuda, scale=0.125 * 2.0 ** -e)
        assert_within(f64(out), ref["out"], bound(ref), f"2^{e}")


def test_zero_queries_average(lib, cuda):
    b = Batch(4, 2, 64, 16, 8, [50], 11)
    b.q.zero_()
    check(lib, cuda, b)


def test_bad_pages_and_lengths(lib, cuda):
    b = Batch(8, 2, 64, 16, 8, [40, 100, 7, 33], 12, wide=1)
    ref_all = b.want()
    table, lengths = b.table.copy(), b.lengths.copy()
    b.table[1, 2] = -3           # tokens 32 .. 47 are not attended
    b.table[2, 0] = 1 << 30      # no token is left
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    out, lse = b.run(lib, cuda, save_lse=True, dev_status=status)
    assert int(status) == lib.QKVP_DEV_BAD_PAGE
    keep = np.r_[0:32, 48:100]
    b.keys[1], b.values[1] = b.keys[1][keep], b.values[1][keep]
    b.keys[2], b.values[2] = b.keys[2][:0], b.values[2][:0]
    ref = b.want()
    assert_within(f64(out), ref["out"], bound(ref), "bad pages")
    assert torch.all(out[2] == 0) and torch.all(lse[2] == float("-inf"))
    # lengths are clamped to what a row can name
    b.table, b.lengths = table[:, :7], lengths.copy()
    b.lengths[0], b.lengths[2] = -5, 7
    status.zero_()
    out = b.run(lib, cuda, dev_status=status)
    assert int(status) == lib.QKVP_DEV_BAD_LENGTH and torch.all(out[0] == 0)
    assert_within(f64(out)[3], ref_all["out"][3], bound(ref_all)[3], "others")
    b.lengths[0] = 1 << 30
    b.table[0, :] = b.table[1, :]
    status.zero_()
    out = b.run(lib, cuda, dev_status=status)
    assert int(status) & lib.QKVP_DEV_BAD_LENGTH


def test_nan_reaches_only_its_readers(lib, cuda):
    b = Batch(8, 2, 64, 16, 8, [40, 100], 13)
    b.codes[0][b.table[0, 1], 3, 1, 9] = 127  # token 19 of sequence 0, key head 1
    out = b.run(lib, cuda)
    ref = b.want()
    got = f64(out)
    assert np.all(np.isnan(got[0, 4:])) and np.all(np.isfinite(got[0, :4]))
    assert_within(got[1], ref["out"][1], bound(ref)[1], "the other sequence")


def test_scales_out_of_range_are_clamped(lib, cuda):
    b = Batch(4, 1, 64, 16, 16, [16], 14)
    q, k, v, ks, vs, table, lengths = b.args(cuda)
    p = int(b.table[0, 0])
    for bad in (0.0, -2.0, float("nan"), 1e-38):
        vs[p] = bad
        assert torch.all(lib.functional.attention_decode8(q, k, v, ks, vs, table, lengths).float().abs() < 1e-26)
        ks[p] = bad
        assert torch.isfinite(lib.functional.attention_decode8(q, k, v, ks, vs, table, lengths).float()).all()


def test_strided_table_given_workspace_and_out(lib, cuda):
    b = Batch(8, 2, 64, 16, 8, [40, 100, 7], 15)
    q, k, v, ks, vs, table, lengths = b.args(cuda)
    F = lib.functional
    want = F.attention_decode8(q, k, v, ks, vs, table, lengths)
    wide = torch.full((3, 20), -1, dtype=torch.int32, device=cuda)
    wide[:, 5:5 + table.shape[1]] = table
    view = wide[:, 5:5 + table.shape[1]]
    need = F.attention_decode8_workspace_bytes(8, 2, 64, 3, 16, table.shape[1])
    ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=cuda)
    out = torch.full_like(want, 5.0)
    got = F.attention_decode8(q, k, v, ks, vs, view, lengths, out=out, workspace=ws[:need])
    assert got is out and torch.equal(got, want) and bool((ws[need:] == 255).all())
    with pytest.raises(lib.QkvpError):
        F.attention_decode8(q, k, v, ks, vs, view, lengths, workspace=ws[:need - 16])


def test_two_at_once_and_captured_while_lengths_grow(lib, cuda):
    b = Batch(8, 2, 64, 16, 8, [400, 100, 7], 16)
    args = b.args(cuda)
    F = lib.functional
    lengths = args[-1]
    want = F.attention_decode8(*args)
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    outs = [F.attention_decode8(*args, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = F.attention_decode8(*args)
    for cut in (1, 30, 0, 399):
        lengths.copy_(torch.tensor([400 - cut, 100 - min(cut, 100), 7 - min(cut, 7)], dtype=torch.int32))
        graph.replay()
        assert torch.equal(out, F.attention_decode8(*args))


def test_pool_past_32_bits(lib, cuda):
    n_kv, D, page_size, block = 8, 128, 64, 16
    pages = 2 ** 32 // (page_size * n_kv * D) + 3
    pools = [torch.full((pages, page_size, n_kv, D), 127, dtype=torch.uint8, device=cuda).view(F8) for _ in range(2)]
    scales = [torch.full((pages, page_size // block, n_kv), float("nan"), device=cuda) for _ in range(2)]
    b = Batch(16, n_kv, D, page_size, block, [130, 64], 17, spare=0)
    place = torch.tensor([pages - 1, 1, pages - 2, 0], device=cuda)[:b.codes[0].shape[0]]
    for pool, scale, c, s in zip(pools, scales, b.codes, b.scale):
        pool.view(torch.uint8)[place] = torch.from_numpy(c).to(cuda)
        scale[place] = torch.from_numpy(s).to(cuda)
    table = place[torch.from_numpy(b.table.clip(0)).to(cuda).long()].to(torch.int32)
    out = lib.functional.attention_decode8(b.q.to(cuda), *pools, *scales, table, torch.from_numpy(b.lengths).to(cuda))
    ref = b.want()
    assert_within(f64(out), ref["out"], bound(ref), "far")


def test_refusals(lib, cuda):
    b = Batch(8, 2, 64, 16, 8, [40, 100], 18)
    q, k, v, ks, vs, table, lengths = b.args(cuda)
    F = lib.functional
    bad = [(q.float(), k, v, ks, vs, table, lengths), (q[:1], k, v, ks, vs, table, lengths),
           (q, k.view(torch.uint8), v, ks, vs, table, lengths), (q, k, v[:1], ks, vs, table, lengths),
           (q, k, v, ks[:, :, :1], vs, table, lengths), (q, k, v, ks.double(), vs, table, lengths),
           (q, k, v, ks, vs, table.long(), lengths), (q, k, v, ks, vs, table, lengths[:1]),
           (q, k, v, ks, vs, table, lengths.cpu()), (q[..., :32].contiguous(), k, v, ks, vs, table, lengths),
           (q, k, v, ks, vs, table.t(), lengths)]
    for args in bad:
        with pytest.raises(ValueError):
            F.attention_decode8(*args)
    with pytest.raises(lib.QkvpError):
        F.attention_decode8(q[:, :7].contiguous(), k, v, ks, vs, table, lengths)  # 7 heads over 2
    with pytest.raises(lib.QkvpError):
        F.attention_decode8(q, k, v, ks, vs, table, lengths, out=q)
    with pytest.raises(ValueError):
        F.attention_decode8(q, k, v, ks, vs, table, lengths, out=q[:1])
    none = F.attention_decode8(q[:0], k, v, ks, vs, table[:0], lengths[:0], save_lse=True)
    assert none[0].shape == (0, 8, 64) and none[1].shape == (0, 8)


@pytest.mark.parametrize("rotary", [dict(), dict(rotary_dim=32, rotary_pairs=True)])
def test_the_path_behind_the_prologue(lib, cuda, rotary):
    """A prompt written into the pool, then decode steps: append, attend. Against
    attention over the float64 values that the pool holds after each step, and near
    the attention over the unquantised keys and values."""
    n_q, n_kv, D, page_size, block = 8, 2, 64, 16, 8
    lengths = [37, 5, 64]
    steps = 12
    F = lib.functional
    pages = 24
    pools = [torch.zeros(pages, page_size, n_kv, D, dtype=torch.uint8, device=cuda).view(F8) for _ in range(2)]
    scales = [torch.ones(pages, page_size // block, n_kv, device=cuda) for _ in range(2)]
    order = np.random.default_rng(19).permutation(pages).astype(np.int32)
    table = np.stack([order[8 * i:8 * i + 8] for i in range(3)])
    i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int32), device=cuda)  # noqa: E731

    def write(where, seed):
        """Tokens [(sequence, position)]; returns q and the unquantised k, v."""
        wl = workloads.gqa_inputs(len(where), n_q, n_kv, D, seed=seed, rope_base=1e4, pos_high=10)
        pos = i32([p for _, p in where])
        page, offset = i32([table[s, p // page_size] for s, p in where]), i32([p % page_size for _, p in where])
        args = (wl.packed_rows().to(cuda), pos, wl.w_q.to(cuda), wl.w_k.to(cuda))
        q = F.prologue_pool_write8(*args, page, offset, *pools, *scales, n_q, n_kv, D, rope_base=1e4, **rotary)
        plain = F.prologue_forward(*args, n_q, n_kv, D, rope_base=1e4, **rotary)
        assert torch.equal(q, plain[0])
        return q, f64(plain[1]), f64(plain[2])

    where = [(s, p) for s, n in enumerate(lengths) for p in range(n)]
    _, k, v = write(where, 100)
    true = [[[k[i] for i, (x, _) in enumerate(where) if x == s] for s in range(3)],
            [[v[i] for i, (x, _) in enumerate(where) if x == s] for s in range(3)]]
    for step in range(steps):
        q, k, v = write([(s, lengths[s]) for s in range(3)], 200 + step)
        for s in range(3):
            true[0][s].append(k[s])
            true[1][s].append(v[s])
            lengths[s] += 1
        out = F.attention_decode8(q, *pools, *scales, i32(table), i32(lengths))
        held = []
        for pool, scale in zip(pools, scales):
            x = E8.stored(pool.view(torch.uint8).cpu().numpy(), scale.cpu().numpy())
            held.append([x[table[s, np.arange(n) // page_size], np.arange(n) % page_size] for s, n in enumerate(lengths)])
        ref = A.attention_decode(f64(q), *held)
        assert_within(f64(out), ref["out"], bound(ref), f"step {step}")
        for i in range(2):  # each value within half a step of its block's scale, and bf16's of the comparison
            for s in range(3):
                t = np.stack(true[i][s])
                assert np.all(np.abs(held[i][s] - t) <= 2.0 ** -4 * 1.01 * np.abs(t) + 2.0 ** -9 * np.abs(t).max())
