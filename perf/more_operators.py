"""Rotary layouts, and a key/value cache in 8 bits, as cases to measure.

Three operators on the tensors of the packed-QKV prologue:

  rotary  the prologue with the rotary layouts that models use beside rotate-half
          over the whole head: the first `rot` values of each head only, in
          halves or in adjacent pairs, frequencies scaled for long contexts;
          with its gradients (a training step's region), or forward alone;
  append  the prologue of new tokens whose keys and values go into a paged cache
          in 8 bits: e4m3 codes [num_pages, page_size, n_kv, D] and a float32
          scale for each block of `block` tokens and head, [num_pages,
          page_size / block, n_kv]. A block whose first token is written here
          gets the scale max(amax / 448, 2^-100) of what is written into it; one
          that holds earlier tokens keeps its scale s, times the least power of
          two 2^k (k >= 0) with which the new values fit, and its earlier codes
          are divided by 2^k;
  decode  attention of one new token per sequence over such a cache.

``run`` computes a case with elementary torch operations in float32, or with
the package's operators when ``own`` is true. ``exact`` is the definition in
float64; where the result is held in 8 bits it gives the value before that
rounding. Head counts are those of the package's workloads (Muse Spark 128 over
16 heads of 64, Llama 3 / Qwen3 32 over 8 heads of 128, GPT-OSS 64 over 8 heads
of 64) and, in ``draw``, generic ones.
"""

import math
import random

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
EPS = 1e-6
LEAST = 2.0 ** -100  # smallest scale


# ---------------------------------------------------------------- the cases ----

def listed():
    return [
        # training on one long document, half of each head rotated, frequencies scaled for a longer context
        dict(name="rotary_train_16384_half_64_of_128", op="rotary", train=True, n_q=32, n_kv=8, dim=128, rot=64,
             pairs=False, kind="sectioned", norm=True, bias=False, scaled=True, tokens=16384, mix=1),
        # training with rotated pairs on the GPT-OSS heads (bias, no norm)
        dict(name="rotary_train_4096_pairs_64_bias", op="rotary", train=True, n_q=64, n_kv=8, dim=64, rot=64,
             pairs=True, kind="interleaved", norm=False, bias=True, scaled=False, tokens=4096, mix=2),
        # a small training step, an odd number of tokens, Muse Spark heads, pairs in half of the head
        dict(name="rotary_train_1021_pairs_32_of_64", op="rotary", train=True, n_q=128, n_kv=16, dim=64, rot=32,
             pairs=True, kind="interleaved", norm=True, bias=False, scaled=True, tokens=1021, mix=3),
        # one short question, forward alone: latency
        dict(name="rotary_prompt_37_pairs_128", op="rotary", train=False, n_q=32, n_kv=8, dim=128, rot=128,
             pairs=True, kind="sectioned", norm=True, bias=False, scaled=False, tokens=37, mix=4),
        # one long document into an empty cache
        dict(name="append_1x16384_d128", op="append", n_q=32, n_kv=8, dim=128, rot=128, pairs=False,
             kind="interleaved", norm=True, bias=False, scaled=True, seqs=1, tokens=16384, past=0, page=64, block=16,
             mix=5),
        # the next pieces of 23 prompts, blocks that are begun already, bias, a quarter of the head in pairs
        dict(name="append_23x4001_d64", op="append", n_q=64, n_kv=8, dim=64, rot=16, pairs=True, kind="sectioned",
             norm=False, bias=True, scaled=False, seqs=23, tokens=4001, past=100, page=32, block=8, mix=6),
        # a decode step of a large batch, one token each, Muse Spark heads
        dict(name="append_256x1_d64", op="append", n_q=128, n_kv=16, dim=64, rot=64, pairs=False, kind="interleaved",
             norm=True, bias=False, scaled=False, seqs=256, tokens=256, past=300, page=64, block=16, mix=7),
        # a decode step of a few requests: latency
        dict(name="append_3x1_d128", op="append", n_q=32, n_kv=8, dim=128, rot=64, pairs=True, kind="sectioned",
             norm=True, bias=False, scaled=False, seqs=3, tokens=3, past=100, page=64, block=64, mix=8),
        # one user, a long conversation
        dict(name="decode_1x131072_d128", op="decode", n_q=32, n_kv=8, dim=128, batch=1, low=131072, high=131072,
             page=64, block=16, mix=9),
        # a large serving batch of unrelated requests of uneven length
        dict(name="decode_256x4096_d64", op="decode", n_q=64, n_kv=8, dim=64, batch=256, low=1, high=4096, page=64,
             block=64, mix=10),
        # a batch of long documents: the largest
        dict(name="decode_48x32768_d128", op="decode", n_q=32, n_kv=8, dim=128, batch=48, low=1, high=32768, page=64,
             block=16, mix=11),
        # the first tokens of a few short requests: latency
        dict(name="decode_3x33_d64", op="decode", n_q=128, n_kv=16, dim=64, batch=3, low=1, high=33, page=16,
             block=16, mix=12),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(("rotary", "append", "decode"))
    dim = rng.choice((64, 128))
    n_kv = rng.choice((1, 2, 3, 4, 8, 16))
    n_q = n_kv * rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    case = dict(op=op, n_q=n_q, n_kv=n_kv, dim=dim, mix=rng.randrange(1 << 20))
    if op == "decode":
        batch = _log_int(rng, 1, 256)
        page = rng.choice((1, 8, 16, 24, 32, 64, 100, 128, 256))
        block = rng.choice([b for b in (1, 2, 4, 8, 12, 16, 25, 32, 50, 64) if page % b == 0])
        room = 48 * 16384 * 8 * 128 // (n_kv * dim)  # keys of the largest listed case
        high = _log_int(rng, 1, max(1, min(131072, room // batch)))
        low = rng.choice((0, 1, high // 2, high))
        while batch * n_q * high > 1 << 28:  # the scores that the plain form holds
            batch = max(1, batch // 2)
        return dict(case, batch=batch, low=min(low, high), high=high, page=page, block=block)
    row = (n_q + 2 * n_kv) * dim
    bias = rng.choice((True, False)) and row <= 12288
    case.update(rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= dim]), pairs=rng.choice((True, False)),
                kind=rng.choice(("interleaved", "sectioned")), norm=rng.choice((True, False)), bias=bias,
                scaled=rng.choice((True, False)))
    most = min(16384, 16384 * 48 * 128 // row)  # values of the largest listed case
    tokens = _log_int(rng, 1, most)
    if op == "rotary":
        return dict(case, train=rng.choice((True, True, False)), tokens=tokens)
    page = rng.choice((1, 8, 16, 24, 32, 64, 100, 128, 256))
    block = rng.choice([b for b in (1, 2, 4, 8, 12, 16, 25, 32, 50, 64) if page % b == 0])
    seqs = rng.choice((_log_int(rng, 1, min(64, tokens)), min(tokens, 256)))
    if seqs == 256 or rng.random() < 0.3:
        tokens = seqs  # a decode step
    return dict(case, seqs=seqs, tokens=tokens, past=rng.choice((0, 33, 300)), page=page, block=block)


def _new_lengths(case):
    """`seqs` lengths that add up to `tokens`: all 1, or uniform cuts (uneven, some perhaps zero)."""
    if case["tokens"] == case["seqs"]:
        return [1] * case["seqs"]
    rng = random.Random(case["mix"])
    ends = sorted(rng.randrange(case["tokens"] + 1) for _ in range(case["seqs"] - 1)) + [case["tokens"]]
    return [b - a for a, b in zip([0] + ends, ends)]


def _past_lengths(case):
    rng = random.Random(case["mix"] + 1)
    return [rng.randint(0, case["past"]) for _ in range(case["seqs"])]


def _own_lengths(case):
    rng = random.Random(case["mix"])
    return [rng.randint(case["low"], case["high"]) for _ in range(case["batch"])]


# --------------------------------------------------------------- the inputs ----

def _frequencies(case):
    """rot / 2 frequencies: base^(-2i/rot), the slow ones divided by 8 with a ramp between when `scaled`."""
    base, rot = 500000.0, case["rot"]
    freq = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if not case["scaled"]:
        return freq
    out = []
    for f in freq:
        turns = 8192 * f / (2 * math.pi)  # over the context that the model was trained on
        keep = min(1.0, max(0.0, (turns - 1.0) / 3.0))
        out.append(f * (keep + (1.0 - keep) / 8.0))
    return out


def _quantised(x, block):
    """Codes and scales of float32 values [pages, page, n_kv, D] by blocks of tokens."""
    pages, page, n_kv, dim = x.shape
    x = x.view(pages, page // block, block, n_kv, dim)
    scale = x.abs().amax((2, 4)).div_(448.0).clamp_(min=LEAST)
    codes = x.div_(scale[:, :, None, :, None]).clamp_(-448, 448).to(F8)
    return codes.view(pages, page, n_kv, dim), scale


def _pools(g, pages, page, n_kv, dim, block):
    """A cache that holds earlier tokens' keys and values, some heads larger than others."""
    out = []
    for _ in range(2):
        x = torch.randn(pages, page, n_kv, dim, generator=g, device=DEV)
        x *= torch.exp(torch.randn(pages, 1, n_kv, 1, generator=g, device=DEV))
        out.append(_quantised(x, block))
    return out[0][0], out[1][0], out[0][1], out[1][1]


def _page_tables(g, counts):
    """Pages of each sequence, in any order: a row each, zero past its last page; and the number of all."""
    total = sum(counts) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    n = torch.tensor(counts, device=DEV)
    at = torch.arange(max(1, max(counts)), device=DEV)[None, :]
    before = torch.cumsum(n, 0) - n
    taken = order[(before[:, None] + at).clamp_(max=total - 1)]
    return torch.where(at < n[:, None], taken, torch.zeros_like(taken)).contiguous(), total


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    n_q, n_kv, dim = case["n_q"], case["n_kv"], case["dim"]
    s = dict(op=case["op"], n_q=n_q, n_kv=n_kv, dim=dim)
    if case["op"] == "decode":
        lengths = _own_lengths(case)
        s["page_table"], total = _page_tables(g, [-(-n // case["page"]) for n in lengths])
        s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _pools(g, total, case["page"], n_kv, dim, case["block"])
        s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
        s["q"] = torch.randn(case["batch"], n_q, dim, generator=g, device=DEV).to(torch.bfloat16)
        return s
    T, row = case["tokens"], (n_q + 2 * n_kv) * dim
    packed = torch.randn(T, row, generator=g, device=DEV)
    packed *= torch.exp(0.5 * torch.randn(T, 1, generator=g, device=DEV))  # some tokens larger than others
    s["packed"] = packed.to(torch.bfloat16)
    s["w_q"] = 0.5 + torch.rand(dim, generator=g, device=DEV) if case["norm"] else None
    s["w_k"] = 0.5 + torch.rand(dim, generator=g, device=DEV) if case["norm"] else None
    s["bias"] = torch.randn(row, generator=g, device=DEV) if case["bias"] else None
    s["inv_freq"] = _frequencies(case)
    s["rope_scale"] = 1.125 if case["scaled"] else 1.0
    for name in ("rot", "pairs", "kind", "norm"):
        s[name] = case[name]
    if case["op"] == "rotary":
        first = random.Random(int(seed) * 7919 + case["mix"]).randrange(1 << 17)
        s["pos"] = torch.arange(first, first + T, dtype=torch.int32, device=DEV)
        s["train"] = case["train"]
        if case["train"]:
            s["grads"] = [torch.randn(T, n, dim, generator=g, device=DEV).to(torch.bfloat16) for n in (n_q, n_kv, n_kv)]
        return s
    new, past, page = _new_lengths(case), _past_lengths(case), case["page"]
    table, total = _page_tables(g, [-(-(a + b) // page) for a, b in zip(past, new)])
    s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"] = _pools(g, total, page, n_kv, dim, case["block"])
    new, past = torch.tensor(new, device=DEV), torch.tensor(past, device=DEV)
    which = torch.repeat_interleave(torch.arange(case["seqs"], device=DEV), new, output_size=T)
    at = past[which] + torch.arange(T, device=DEV) - (torch.cumsum(new, 0) - new)[which]
    s["pos"] = at.to(torch.int32)
    s["page"] = table[which, at // page].contiguous()
    s["offset"] = (at % page).to(torch.int32)
    return s


# ----------------------------------------------------------- the plain form ----

def _split(s, x):
    """Heads [T, n, D] of q, k, v in a row of either packing."""
    T, n_q, n_kv, dim = x.shape[0], s["n_q"], s["n_kv"], s["dim"]
    if s["kind"] == "sectioned":
        return x.view(T, -1, dim).split((n_q, n_kv, n_kv), 1)
    x = x.view(T, n_kv, n_q // n_kv + 2, dim)
    return x[:, :, :-2].reshape(T, n_q, dim), x[:, :, -2], x[:, :, -1]


def _joined(s, q, k, v):
    if s["kind"] == "sectioned":
        return torch.cat((q, k, v), 1).flatten(1)
    T, n_kv, dim = k.shape
    return torch.cat((q.view(T, n_kv, -1, dim), k[:, :, None], v[:, :, None]), 2).flatten(1)


def _turned(s, x, back=False):
    """The first `rot` values of each head rotated by the position's angles (back: by their negatives)."""
    rot = s["rot"]
    turn = s["pos"].double()[:, None] * torch.tensor(s["inv_freq"], dtype=torch.float64, device=DEV)
    c, n = (turn.cos() * s["rope_scale"]).float()[:, None], (turn.sin() * s["rope_scale"]).float()[:, None]
    n = -n if back else n
    if s["pairs"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * c - b * n, b * c + a * n), -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat((a * c - b * n, b * c + a * n), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _plain_prologue(s):
    """float32 q, k, v, and the norms' inputs."""
    x = s["packed"].float()
    if s["bias"] is not None:
        x = x + s["bias"]
    q_in, k_in, v = _split(s, x)
    q, k = q_in, k_in
    if s["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["w_q"]
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["w_k"]
    return _turned(s, q), _turned(s, k), v, q_in, k_in


def _norm_gradients(x, g, w):
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    wg = w * g
    dx = r * wg - x * (r ** 3 * (x * wg).mean(-1, keepdim=True))
    return dx, (g * x * r).sum((0, 1), dtype=torch.float64).float()


def _plain_rotary(s):
    q, k, v, q_in, k_in = _plain_prologue(s)
    out = [t.to(torch.bfloat16) for t in (q, k, v)]
    if not s["train"]:
        return out
    dq, dk, dv = (t.float() for t in s["grads"])
    dq, dk = _turned(s, dq, True), _turned(s, dk, True)
    dw = []
    if s["norm"]:
        dq, dw_q = _norm_gradients(q_in, dq, s["w_q"])
        dk, dw_k = _norm_gradients(k_in, dk, s["w_k"])
        dw = [dw_q, dw_k]
    dx = _joined(s, dq, dk, dv)
    if s["bias"] is not None:
        dw.append(dx.sum(0, dtype=torch.float64).float())
    return out + [dx.to(torch.bfloat16)] + dw


def _store(codes, scale, x, block_of, page, offset):
    """Rows x [T, n_kv, D] into the cache; block_of: the number of each row's block."""
    pages, per, n_kv = scale.shape
    block = codes.shape[1] // per
    touched, run = torch.unique_consecutive(block_of, return_inverse=True)
    n = touched.shape[0]
    top = torch.zeros(n, n_kv, device=DEV).index_reduce_(0, run, x.abs().amax(-1), "amax")
    first = torch.full((n,), block, device=DEV).index_reduce_(0, run, offset.long() % block, "amin")
    old = scale.view(-1, n_kv)[touched].clamp(LEAST, 2.0 ** 120)
    m_top, e_top = torch.frexp(top)
    m_old, e_old = torch.frexp(448.0 * old)
    grow = (e_top - e_old + (m_top > m_old).int()).clamp_(min=0)
    fresh = (first == 0)[:, None]
    grow = torch.where(fresh | (top == 0), torch.zeros_like(grow), grow)
    new = torch.where(fresh, (top / 448.0).clamp(min=LEAST), torch.ldexp(old, grow))
    scale.view(-1, n_kv)[touched] = new
    held = codes.view(-1, block, n_kv, codes.shape[3])[touched].float()
    moved = torch.ldexp(held, -grow[:, None, :, None]).to(F8)
    kept = (torch.arange(block, device=DEV)[None, :] < first[:, None])[:, :, None, None] & (grow > 0)[:, None, :, None]
    moved = torch.where(kept, moved.view(torch.uint8), codes.view(torch.uint8).view(-1, block, n_kv, codes.shape[3])[touched])
    codes.view(torch.uint8).view(-1, block, n_kv, codes.shape[3])[touched] = moved
    rows = (x / new[run][:, :, None]).clamp(-448, 448).to(F8)
    codes.view(torch.uint8)[page.long(), offset.long()] = rows.view(torch.uint8)


def _plain_append(s):
    q, k, v, _, _ = _plain_prologue(s)
    per = s["k_scale"].shape[1]
    block = s["k_pool"].shape[1] // per
    block_of = s["page"].long() * per + s["offset"].long() // block
    _store(s["k_pool"], s["k_scale"], k, block_of, s["page"], s["offset"])
    _store(s["v_pool"], s["v_scale"], v, block_of, s["page"], s["offset"])
    return q.to(torch.bfloat16), s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]


def _plain_decode(s):
    n_kv, D, page = s["n_kv"], s["dim"], s["k_pool"].shape[1]
    block, B = page // s["k_scale"].shape[1], s["q"].shape[0]
    q = s["q"].float().view(B, n_kv, -1, D)
    wide = s["page_table"].shape[1] * page
    at = torch.arange(wide, device=DEV)
    rows = s["page_table"].long()[:, at // page] * page + at % page  # [B, wide]

    def values(pool, scale):
        x = pool.view(torch.uint8).view(-1, n_kv, D)[rows].view(F8).float()
        return x.mul_(scale.view(-1, n_kv)[rows // block][..., None])

    w = torch.einsum("bhgd,bnhd->bhgn", q, values(s["k_pool"], s["k_scale"])).mul_(1.0 / math.sqrt(D))
    w.masked_fill_((at[None, :] >= s["lengths"][:, None])[:, None, None, :], float("-inf"))
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = w.sum(-1, keepdim=True)
    w.div_(torch.where(total > 0, total, torch.ones_like(total)))
    out = torch.einsum("bhgn,bnhd->bhgd", w, values(s["v_pool"], s["v_scale"]))
    return out.reshape(B, -1, D).to(torch.bfloat16)


def run(state):
    s = state
    if own:
        from rope_qkv_prologue_gb300 import functional as F

        if s["op"] == "decode":
            return F.attention_decode8(s["q"], s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"], s["page_table"],
                                       s["lengths"])
        options = dict(kind=s["kind"], eps=EPS, norm=s["norm"], bias=s["bias"], inv_freq=s["inv_freq"],
                       rope_scale=s["rope_scale"], rotary_dim=s["rot"], rotary_pairs=s["pairs"])
        heads = (s["n_q"], s["n_kv"], s["dim"])
        if s["op"] == "append":
            q = F.prologue_pool_write8(s["packed"], s["pos"], s["w_q"], s["w_k"], s["page"], s["offset"], s["k_pool"],
                                       s["v_pool"], s["k_scale"], s["v_scale"], *heads, **options)
            return q, s["k_pool"], s["v_pool"], s["k_scale"], s["v_scale"]
        saved = s["train"] and s["norm"]
        out = F.prologue_forward(s["packed"], s["pos"], s["w_q"], s["w_k"], *heads, save_pre=saved, **options)
        if not s["train"]:
            return list(out)
        q_pre, k_pre = out[3:] if saved else (None, None)
        back = F.prologue_backward(*s["grads"], q_pre, k_pre, s["pos"], s["w_q"], s["w_k"], *heads, **options)
        return list(out[:3]) + [t for t in back if t is not None]
    return {"rotary": _plain_rotary, "append": _plain_append, "decode": _plain_decode}[s["op"]](s)


# ------------------------------------------------------------ what it costs ----

def work(case):
    n_q, n_kv, D = case["n_q"], case["n_kv"], case["dim"]
    if case["op"] == "decode":
        lengths = _own_lengths(case)
        keys, blocks = sum(lengths), sum(-(-n // case["block"]) for n in lengths)
        return {"bytes": 2 * keys * n_kv * D + 8 * blocks * n_kv + 4 * case["batch"] * n_q * D,
                "flops": 4 * D * n_q * keys}
    T, row = case["tokens"], (n_q + 2 * n_kv) * D
    turned = 8 * T * (n_q + n_kv) * D  # norm and rotation of q and k
    if case["op"] == "rotary":
        # packed read, q, k, v written; and dq, dk, dv read, the packed gradient written
        return {"bytes": (8 if case["train"] else 4) * T * row + 4 * T, "flops": (3 if case["train"] else 1) * turned}
    block = case["block"]
    blocks = sum((p + n - 1) // block - p // block + 1 for p, n in zip(_past_lengths(case), _new_lengths(case)) if n)
    return {"bytes": 2 * T * row + 2 * T * n_q * D + 2 * T * n_kv * D + 8 * blocks * n_kv + 12 * T, "flops": turned}


# ------------------------------------------------- the definition in 64 bits ----

def _exact_heads(s):
    """float64 lists of heads: norms' inputs x, weights, of q, k, v."""
    x = s["packed"].double()
    if s["bias"] is not None:
        x = x + s["bias"].double()
    n_q, n_kv, dim = s["n_q"], s["n_kv"], s["dim"]
    G = n_q // n_kv
    x = x.view(x.shape[0], n_q + 2 * n_kv, dim)
    if s["kind"] == "interleaved":
        slot = torch.arange(n_q + 2 * n_kv, device=DEV)
        kind = torch.clamp(slot % (G + 2) - (G - 1), min=0)
        return x[:, kind == 0], x[:, kind == 1], x[:, kind == 2], (kind == 0, kind == 1, kind == 2)
    slot = torch.arange(n_q + 2 * n_kv, device=DEV)
    which = (slot < n_q, (slot >= n_q) & (slot < n_q + n_kv), slot >= n_q + n_kv)
    return x[:, which[0]], x[:, which[1]], x[:, which[2]], which


def _exact_rotation(s, x, sign):
    """Each rotated pair as a complex number times e^(i sign angle)."""
    half = s["rot"] // 2
    i = torch.arange(half, device=DEV)
    lo, hi = (2 * i, 2 * i + 1) if s["pairs"] else (i, i + half)
    angle = s["pos"].double()[:, None, None] * torch.tensor(s["inv_freq"], dtype=torch.float64, device=DEV)
    z = torch.complex(x[..., lo], x[..., hi]) * torch.polar(torch.full_like(angle, s["rope_scale"]), sign * angle)
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def _exact_rotary(s):
    q, k, v, which = _exact_heads(s)

    def forward(x, w):
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / s["dim"] + EPS) * w.double() if s["norm"] else x
        return _exact_rotation(s, y, 1.0)

    out = [forward(q, s["w_q"]), forward(k, s["w_k"]), v]
    if s["op"] == "append" or not s["train"]:
        return out

    def backward(x, d, w):
        g = _exact_rotation(s, d.double(), -1.0)
        if not s["norm"]:
            return g, None
        rms = torch.sqrt((x * x).sum(-1, keepdim=True) / s["dim"] + EPS)
        u = x / rms
        gw = g * w.double()
        return (gw - u * (u * gw).sum(-1, keepdim=True) / s["dim"]) / rms, (g * u).sum((0, 1))

    dq, dk, dv = s["grads"]
    (dq, dw_q), (dk, dw_k) = backward(q, dq, s["w_q"]), backward(k, dk, s["w_k"])
    dx = torch.zeros(q.shape[0], len(which[0]), s["dim"], dtype=torch.float64, device=DEV)
    for here, d in zip(which, (dq, dk, dv.double())):
        dx[:, here] = d
    dx = dx.flatten(1)
    out.append(dx)
    if s["norm"]:
        out += [dw_q, dw_k]
    if s["bias"] is not None:
        out.append(dx.sum(0))
    return out


def _exact_cache(s, x, pool, scale):
    """Codes before rounding and scales, block by block in a dense picture of the whole cache."""
    pages, page, n_kv, dim = pool.shape
    per = scale.shape[1]
    block = page // per
    at = s["page"].long() * page + s["offset"].long()
    value = torch.zeros(pages * page, n_kv, dim, dtype=torch.float64, device=DEV)
    fresh = torch.zeros(pages * page, dtype=torch.bool, device=DEV)
    value[at], fresh[at] = x, True
    value = value.view(pages * per, block, n_kv, dim)
    fresh = fresh.view(pages * per, block)
    top = value.abs().amax((1, 3))  # [blocks, n_kv]
    hit = fresh.any(1)
    first = torch.where(hit, fresh.int().argmax(1), block)
    before = torch.arange(block, device=DEV) < first[:, None]
    old = scale.view(-1, n_kv).double()
    k = torch.ceil(torch.log2(torch.clamp(top / (448.0 * old), min=1.0)))
    k = torch.where((first > 0)[:, None] & hit[:, None], k, torch.zeros_like(k))
    new = torch.where((first == 0)[:, None], torch.clamp(top / 448.0, min=LEAST), old * 2.0 ** k)
    held = pool.double().view(pages * per, block, n_kv, dim)
    moved = torch.where((before & hit[:, None])[:, :, None, None], held / (2.0 ** k)[:, None, :, None], held)
    codes = torch.where(fresh[:, :, None, None], value / new[:, None, :, None], moved)
    return codes.view(pool.shape), torch.where(hit[:, None], new, old).view(scale.shape)


def _exact_append(s):
    q, k, v = _exact_rotary(s)
    k_codes, k_scale = _exact_cache(s, k, s["k_pool"], s["k_scale"])
    v_codes, v_scale = _exact_cache(s, v, s["v_pool"], s["v_scale"])
    return q, k_codes, v_codes, k_scale, v_scale


def _exact_decode(s):
    B, n_q, D = s["q"].shape
    n_kv, page = s["n_kv"], s["k_pool"].shape[1]
    block, G = page // s["k_scale"].shape[1], n_q // n_kv
    out = torch.zeros(B, n_q, D, dtype=torch.float64, device=DEV)

    def stored(pool, scale, token, pages):
        where = pages[torch.div(token, page, rounding_mode="floor")].long()
        x = pool.view(torch.uint8)[where, token % page].view(F8).double()
        x *= scale[where, (token % page) // block].double()[..., None]
        return x.transpose(0, 1)  # [n_kv, n, D]

    for b, n in enumerate(s["lengths"].tolist()):
        if not n:
            continue
        token = torch.arange(n, device=DEV)
        q = s["q"][b].double().view(n_kv, G, D)
        e = q @ stored(s["k_pool"], s["k_scale"], token, s["page_table"][b]).transpose(1, 2) * D ** -0.5
        e = torch.exp(e - e.max(2, keepdim=True).values)
        e /= e.sum(2, keepdim=True)
        out[b] = (e @ stored(s["v_pool"], s["v_scale"], token, s["page_table"][b])).reshape(n_q, D)
    return out


def exact(case, seed):
    """The definition in float64."""
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "append": _exact_append, "decode": _exact_decode}[case["op"]](s)
