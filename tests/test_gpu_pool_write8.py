"""Appending to the 8-bit pool on the GPU against the float64 oracle.

k is computed in float32 before it is quantised. Its error: a row's mean square
is a sum of D <= 128 products (relative error of its root at most (D + 1) 2^-25
< 2^-17.9), rsqrt 2^-22, two products 2^-23, cos and sin 2^-21 of one, and the
rotation adds two such terms of at most sqrt(2) the row's largest pair: below
2^-16 of the row's largest magnitude, before and after the rotation. E = 2^-15
of the largest magnitude of a block's rows bounds it. Its maximum, hence the
scale, has the relative error 2^-15; a code differs from x / s by half a step
and what E and the scale's error make. v is exact, and so is its scale but for
float32's rounding.
"""

import numpy as np
import pytest
import torch

import oracle.pool8 as E8
import oracle.prologue as P
import oracle.rotary as R
import workloads
from workloads import bits_u16 as u16

pytestmark = pytest.mark.gpu

E = 2.0 ** -15
F8 = torch.float8_e4m3fn


class Pool:
    """Pools full of codes and scales of earlier use, on the host and the device."""

    def __init__(self, pages, page_size, block, n_kv, D, dev, seed=1, codes=None):
        g = np.random.default_rng(seed)
        shape = (pages, page_size, n_kv, D)
        self.codes = [g.integers(0, 256, shape).astype(np.uint8) if codes is None else np.full(shape, codes, np.uint8)
                      for _ in range(2)]
        for c in self.codes:
            c[c & 127 == 127] = 3  # (NaN codes only where a test puts them)
        self.scale = [np.exp2(g.uniform(-8, 4, (pages, page_size // block, n_kv))).astype(np.float32) for _ in range(2)]
        self.to(dev)

    def to(self, dev):
        self.dev = [torch.from_numpy(c).to(dev).view(F8) for c in self.codes]
        self.dev_scale = [torch.from_numpy(s).to(dev) for s in self.scale]

    @property
    def args(self):
        return (*self.dev, *self.dev_scale)

    def read(self):
        return [c.view(torch.uint8).cpu().numpy() for c in self.dev], [s.cpu().numpy() for s in self.dev_scale]


def _check_pool(before, before_scale, got, got_scale, x, page, offset, exact, what):
    """One pool (codes, scales before and after) that x [T, n_kv, D] was written into."""
    want, want_scale = E8.append(before, before_scale, x, page, offset)
    block = before.shape[1] // before_scale.shape[1]
    rel = 2.0 ** -23 if exact else E
    assert np.all(np.abs(got_scale - want_scale) <= rel * np.abs(want_scale)), f"{what}: scales"
    written = np.zeros(before.shape[:2], bool)
    for p, o in zip(page, offset):
        if p >= 0:
            written[p, o] = True
    # codes that were not written: untouched, or moved by a power of two
    assert np.array_equal(E8.VALUES[got[~written]], E8.VALUES[want[~written]], equal_nan=True), f"{what}: held codes"
    slot = {(p, o): t for t, (p, o) in enumerate(zip(page, offset))}
    for (p, o), t in slot.items():
        if p < 0:
            continue
        s = got_scale[p, o // block].astype(np.float64)[:, None]
        value = E8.VALUES[got[p, o]] * s
        row = np.where(np.isfinite(x[t]), x[t], np.nan)
        assert np.array_equal(np.isnan(value), np.isnan(row)), f"{what}: token {t}, NaN"
        fine = ~np.isnan(row)
        top = np.max(np.where(fine, np.abs(row), 0), axis=1, keepdims=True)
        err = (0.0 if exact else E) * top + 2.0 ** -22 * np.abs(row)
        bound = E8.half_step(np.abs(row) + err, s) + err
        over = np.where(fine, np.abs(value - row) - bound, 0)
        assert over.max() <= 1e-30, f"{what}: token {t} off by {over.max():.3g} more than {bound.max():.3g}"


def _slots(rng, lengths, past, page_size, pages):
    """Page and offset of new tokens behind `past` ones of each sequence, on pages of its own."""
    order = rng.permutation(pages)
    page, offset, at = [], [], 0
    for n, p in zip(lengths, past):
        need = -(-(n + p) // page_size)
        mine = order[at:at + need]
        at += need
        page += [int(mine[i // page_size]) for i in range(p, p + n)]
        offset += [i % page_size for i in range(p, p + n)]
    assert at <= pages
    return page, offset


def _run(lib, dev, wl, kind, pool, page, offset, opts=None, status=None, **kw):
    opts = dict(opts or {})
    rows = wl.packed_rows() if kind == "interleaved" else wl.sectioned_rows()
    bias = opts.pop("bias", None)
    norm = opts.get("norm", True)
    put = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)  # noqa: E731
    q = lib.functional.prologue_pool_write8(
        rows.to(dev), wl.pos.to(dev), wl.w_q.to(dev) if norm else None, wl.w_k.to(dev) if norm else None, put(page),
        put(offset), *pool.args, wl.n_q, wl.n_kv, wl.head_dim, kind, wl.eps, wl.rope_base,
        bias=None if bias is None else bias.to(dev), dev_status=status, **opts, **kw)
    return q, rows


def _exact(wl, kind, rows, opts):
    opts = dict(opts or {})
    L = P.PackedLayout(kind, wl.n_q, wl.n_kv, wl.head_dim)
    bias = opts.get("bias")
    nope = opts.get("nope", False)
    w = (wl.w_q.numpy().astype(np.float64), wl.w_k.numpy().astype(np.float64))
    _, k, v = R.prologue_fwd(L, u16(rows), np.zeros(wl.T) if nope else wl.pos.numpy(), *w, wl.eps, wl.rope_base,
                             opts.get("rotary_dim") or wl.head_dim, opts.get("rotary_pairs", False),
                             norm=opts.get("norm", True), bias=None if bias is None else bias.numpy().astype(np.float64),
                             rope_scale=opts.get("rope_scale", 1.0))
    return k, v


def _check(lib, dev, shape, kind, lengths, past, page_size, block, opts=None, seed=3):
    n_q, n_kv, D = shape
    rng = np.random.default_rng(seed)
    T = sum(lengths)
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=seed, rope_base=5e5, pos_high=131072)
    pages = sum(-(-(n + p) // page_size) for n, p in zip(lengths, past)) + 2
    page, offset = _slots(rng, lengths, past, page_size, pages)
    pool = Pool(pages, page_size, block, n_kv, D, dev, seed)
    opts = dict(opts or {})
    if opts.get("bias"):
        opts["bias"] = workloads.qkv_bias((n_q + 2 * n_kv) * D, workloads._gen(seed))
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    before, before_scale = pool.read()
    q, rows = _run(lib, dev, wl, kind, pool, page, offset, opts, status)
    codes, scale = pool.read()
    k, v = _exact(wl, kind, rows, opts)
    what = f"{shape} {kind} {lengths} {past} page {page_size} block {block} {opts.keys()}"
    _check_pool(before[0], before_scale[0], codes[0], scale[0], k, page, offset, False, what + " k")
    _check_pool(before[1], before_scale[1], codes[1], scale[1], v, page, offset, opts.get("bias") is None, what + " v")
    assert int(status) == 0
    # q has the bits of the prologue without a pool
    norm = opts.get("norm", True)
    bias = opts.pop("bias", None)
    other = lib.functional.prologue_forward(
        rows.to(dev), wl.pos.to(dev), wl.w_q.to(dev) if norm else None, wl.w_k.to(dev) if norm else None, n_q, n_kv, D,
        kind, wl.eps, wl.rope_base, bias=None if bias is None else bias.to(dev), **opts)
    assert torch.equal(q, other[0]), f"{what}: q"


SHAPES = [(8, 2, 64), (6, 3, 128), (5, 1, 64), (32, 8, 128), (128, 16, 64)]


@pytest.mark.parametrize("kind", ["interleaved", "sectioned"])
@pytest.mark.parametrize("shape", SHAPES)
def test_prompts_into_an_empty_pool(lib, cuda, shape, kind):
    _check(lib, cuda, shape, kind, [1], [0], 16, 16)
    _check(lib, cuda, shape, kind, [70], [0], 32, 16)
    _check(lib, cuda, shape, kind, [33, 1, 0, 17, 64], [0] * 5, 64, 32)


@pytest.mark.parametrize("page_size, block", [(1, 1), (16, 1), (16, 4), (24, 12), (100, 25), (64, 64), (128, 128), (300, 300),
                                              (300, 100), (256, 2)])
def test_pages_and_blocks(lib, cuda, page_size, block):
    _check(lib, cuda, (4, 2, 64), "interleaved", [90, 3, 41], [0, 5, 77], page_size, block)
    _check(lib, cuda, (4, 2, 128), "sectioned", [330], [11], page_size, block)


@pytest.mark.parametrize("opts", [
    dict(nope=True), dict(norm=False), dict(bias=True), dict(norm=False, bias=True, rope_scale=1.25),
    dict(rotary_dim=32), dict(rotary_pairs=True), dict(rotary_dim=48, rotary_pairs=True, bias=True)])
def test_options(lib, cuda, opts):
    for kind in ("interleaved", "sectioned"):
        for D in (64, 128):
            _check(lib, cuda, (8, 2, D), kind, [21, 1, 40], [0, 30, 7], 32, 16, opts)


def test_many_tokens_and_many_runs(lib, cuda):
    rng = np.random.default_rng(8)
    lengths = [int(n) for n in rng.integers(0, 120, 40)]
    _check(lib, cuda, (8, 2, 64), "interleaved", lengths, [int(p) for p in rng.integers(0, 50, 40)], 16, 8)
    _check(lib, cuda, (4, 1, 64), "sectioned", [6000], [3], 64, 16)  # tiles of 16 tokens
    _check(lib, cuda, (4, 1, 128), "sectioned", [1] * 700, [int(p) for p in rng.integers(0, 20, 700)], 16, 16)


def test_token_by_token(lib, cuda):
    # values that grow and shrink, one token at a time into one block, then again over what was there
    n_q, n_kv, D, T = 4, 2, 64, 16
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=5, rope_base=1e4, pos_high=1000)
    rows = wl.sectioned_rows()
    size = torch.tensor([0.0, 1e-3, 1.0, 0.5, 3.0, 64.0, 1.0, 1e-2, 500.0, 7.0, 1e4, 1e-30, 0.0, 1e30, 1.0, 1e36])
    rows = (rows.float() * size[:, None]).to(torch.bfloat16)
    pool = Pool(2, 16, 16, n_kv, D, cuda)
    opts = dict(norm=False)
    F = lib.functional

    def write(t, o):
        before, before_scale = pool.read()
        put = lambda x: torch.tensor([x], dtype=torch.int32, device=cuda)  # noqa: E731
        F.prologue_pool_write8(rows[t:t + 1].to(cuda), wl.pos[t:t + 1].to(cuda), None, None, put(1), put(o), *pool.args,
                               n_q, n_kv, D, "sectioned", rope_base=1e4, norm=False)
        codes, scale = pool.read()
        L = P.PackedLayout("sectioned", n_q, n_kv, D)
        _, k, v = R.prologue_fwd(L, u16(rows[t:t + 1]), wl.pos.numpy()[t:t + 1], None, None, 1e-6, 1e4, D, False, norm=False)
        _check_pool(before[0], before_scale[0], codes[0], scale[0], k, [1], [o], False, f"token {t} k")
        _check_pool(before[1], before_scale[1], codes[1], scale[1], v, [1], [o], True, f"token {t} v")

    assert opts["norm"] is False
    for t in range(T):
        write(t, t)
    for t, o in ((2, 9), (8, 10), (0, 0), (5, 1), (4, 15), (3, 3)):  # a place below others: those are not held
        write(t, o)


def test_runs_out_of_order_and_not_stored(lib, cuda):
    # descending places in a block, pages and offsets out of range, blocks in any order
    n_q, n_kv, D, T = 8, 2, 64, 40
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=6, rope_base=1e4, pos_high=1000)
    page = [2, 2, 2, -1, 0, 0, 5, 1, 1, 1, 1, 1, 3, 4] + [4] * 7 + [-5, 99, 6] + [3] * 4 + [0] * 12
    offset = [7, 6, 5, 3, 0, 15, 16, 8, 9, 10, 11, 12, 2, 0] + list(range(8, 15)) + [0, 0, -1] + [10, 9, 12, 11] + [0] * 12
    page[28:40] = [5] * 8 + [-1] * 4
    offset[28:40] = list(range(8)) + [0] * 4
    pool = Pool(6, 16, 8, n_kv, D, cuda)
    before, before_scale = pool.read()
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    q, rows = _run(lib, cuda, wl, "interleaved", pool, page, offset, status=status)
    codes, scale = pool.read()
    assert int(status) == lib.QKVP_DEV_BAD_PAGE | lib.QKVP_DEV_BAD_OFFSET
    k, v = _exact(wl, "interleaved", rows, {})
    ok = [p if 0 <= p < 6 and 0 <= o < 16 else -1 for p, o in zip(page, offset)]
    _check_pool(before[0], before_scale[0], codes[0], scale[0], k, ok, offset, False, "k")
    _check_pool(before[1], before_scale[1], codes[1], scale[1], v, ok, offset, True, "v")
    want = lib.functional.prologue_forward(rows.to(cuda), wl.pos.to(cuda), wl.w_q.to(cuda), wl.w_k.to(cuda), n_q, n_kv, D,
                                           rope_base=1e4)[0]
    assert torch.equal(q, want)  # of the tokens that are not stored too
    # the same without a status word
    _run(lib, cuda, wl, "interleaved", pool, page, offset)


@pytest.mark.parametrize("block", [8, 64])
def test_infinities_and_nan(lib, cuda, block):
    n_q, n_kv, D, T = 4, 2, 64, 64
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=7, rope_base=1e4, pos_high=1000)
    rows = wl.sectioned_rows().clone().view(T, n_q + 2 * n_kv, D)
    rows[3, n_q + n_kv, 5] = float("inf")   # v
    rows[4, n_q + n_kv, 6] = float("-inf")
    rows[9, n_q + n_kv + 1, 7] = float("nan")
    rows[17, n_q + n_kv] = float("nan")     # a whole row
    rows[20:28, n_q + n_kv + 1] = float("inf")
    rows[40, n_q, 8] = float("inf")         # k, without the norm
    rows[41, n_q + 1, 9] = float("nan")
    wl.sectioned_rows = lambda: rows.view(T, -1)
    page, offset = [0] * T, list(range(T))
    pool = Pool(1, 64, block, n_kv, D, cuda)
    before, before_scale = pool.read()
    _run(lib, cuda, wl, "sectioned", pool, page, offset, dict(norm=False, nope=True))
    codes, scale = pool.read()
    v = rows[:, n_q + n_kv:].double().numpy()
    k = rows[:, n_q:n_q + n_kv].double().numpy()
    _check_pool(before[0], before_scale[0], codes[0], scale[0], k, page, offset, True, "k")
    _check_pool(before[1], before_scale[1], codes[1], scale[1], v, page, offset, True, "v")


def test_scales_out_of_range_and_nan_codes(lib, cuda):
    n_q, n_kv, D = 4, 2, 64
    wl = workloads.gqa_inputs(1, n_q, n_kv, D, seed=8, rope_base=1e4, pos_high=1000)
    for old in (0.0, -1.0, float("nan"), float("inf"), 1e-38, 3e38, 1e-45):
        pool = Pool(1, 16, 16, n_kv, D, cuda)
        pool.codes[1][0, 2] = 127
        pool.scale = [np.full_like(s, old) for s in pool.scale]
        pool.to(cuda)
        before, before_scale = pool.read()
        _, rows = _run(lib, cuda, wl, "sectioned", pool, [0], [5])
        codes, scale = pool.read()
        k, v = _exact(wl, "sectioned", rows, {})
        _check_pool(before[0], before_scale[0], codes[0], scale[0], k, [0], [5], False, f"{old} k")
        _check_pool(before[1], before_scale[1], codes[1], scale[1], v, [0], [5], True, f"{old} v")


def test_pool_past_32_bits(lib, cuda):
    n_q, n_kv, D, page_size, block = 8, 8, 128, 64, 16
    pages = 2 ** 32 // (page_size * n_kv * D) + 3  # code offsets past 2^32
    k_pool = torch.zeros(pages, page_size, n_kv, D, dtype=torch.uint8, device=cuda).view(F8)
    v_pool = torch.zeros(pages, page_size, n_kv, D, dtype=torch.uint8, device=cuda).view(F8)
    scales = [torch.ones(pages, page_size // block, n_kv, device=cuda) for _ in range(2)]
    T = 4
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=9, rope_base=1e4, pos_high=1000)
    page, offset = [pages - 1, pages - 1, 0, pages - 2], [62, 63, 0, 5]
    pool = Pool(1, page_size, block, n_kv, D, cuda)
    pool.dev, pool.dev_scale = [k_pool, v_pool], scales
    _, rows = _run(lib, cuda, wl, "interleaved", pool, page, offset)
    k, v = _exact(wl, "interleaved", rows, {})
    small = {pages - 1: 0, 0: 1, pages - 2: 2}
    for cache, sc, x, exact in ((k_pool, scales[0], k, False), (v_pool, scales[1], v, True)):
        at = torch.tensor(list(small), device=cuda)
        codes = cache.view(torch.uint8)[at].cpu().numpy()
        before = np.zeros_like(codes)
        _check_pool(before, np.ones(sc[at].shape, np.float32), codes, sc[at].cpu().numpy(), x, [small[p] for p in page],
                    offset, exact, "far")
        assert int((cache.view(torch.uint8)[1:pages - 2] != 0).sum()) == 0


def test_captured_and_on_a_stream(lib, cuda):
    n_q, n_kv, D, T = 8, 2, 64, 5
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=10, rope_base=1e4, pos_high=1000)
    F = lib.functional
    rows = wl.packed_rows().to(cuda)
    put = lambda x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    page, offset, pos = put([0, 1, 2, 3, 4]), put([0, 3, 6, 9, 12]), wl.pos.to(cuda)
    pool = Pool(5, 16, 8, n_kv, D, cuda)
    mirror = Pool(5, 16, 8, n_kv, D, cuda)
    w = (wl.w_q.to(cuda), wl.w_k.to(cuda))
    call = lambda p: F.prologue_pool_write8(rows, pos, *w, page, offset, *p.args, n_q, n_kv, D)  # noqa: E731
    graph = torch.cuda.CUDAGraph()
    call(pool), call(mirror)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q = call(pool)
    for _ in range(4):  # the next token of each sequence
        offset.add_(1)
        pos.add_(1)
        rows.mul_(1.5)
        graph.replay()
        want = call(mirror)
        assert torch.equal(q, want)
        for a, b in zip(pool.args, mirror.args):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    q = F.prologue_pool_write8(rows, pos, *w, page, offset, *pool.args, n_q, n_kv, D, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(q, call(mirror))
    for a, b in zip(pool.args, mirror.args):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def test_refusals(lib, cuda):
    n_q, n_kv, D, T = 8, 2, 64, 3
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=11, rope_base=1e4, pos_high=1000)
    F = lib.functional
    pool = Pool(2, 16, 8, n_kv, D, cuda)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=cuda)  # noqa: E731
    good = dict(packed=wl.packed_rows().to(cuda), pos=wl.pos.to(cuda), w_q=wl.w_q.to(cuda), w_k=wl.w_k.to(cuda),
                page=i32(0, 0, 0), offset=i32(0, 1, 2), k_pool=pool.dev[0], v_pool=pool.dev[1], k_scale=pool.dev_scale[0],
                v_scale=pool.dev_scale[1], n_q=n_q, n_kv=n_kv, head_dim=D)
    F.prologue_pool_write8(**good)
    for name, bad in (("packed", good["packed"].float()), ("packed", good["packed"][:, :-1]), ("pos", good["pos"].long()),
                      ("page", i32(0, 0)), ("offset", good["offset"].cpu()), ("w_q", good["w_q"].double()),
                      ("w_k", None), ("k_pool", pool.dev[0][:, :, :1]), ("n_kv", 4), ("dev_status", torch.zeros(1, device=cuda)),
                      ("bias", torch.zeros(5, device=cuda)), ("k_scale", pool.dev_scale[0][:1])):
        with pytest.raises((ValueError, AttributeError)):
            F.prologue_pool_write8(**{**good, name: bad})
    for more in (dict(rotary_dim=24), dict(rotary_dim=32, nope=True), dict(eps=-1.0)):
        with pytest.raises(lib.QkvpError):
            F.prologue_pool_write8(**{**good, **more})
    with pytest.raises(lib.QkvpError):  # one tensor for both pools
        F.prologue_pool_write8(**{**good, "v_pool": pool.dev[0]})
    empty = {**good, "packed": good["packed"][:0], "pos": good["pos"][:0], "page": good["page"][:0],
             "offset": good["offset"][:0]}
    assert F.prologue_pool_write8(**empty).shape == (0, n_q, D)
