"""The attention operators that follow the qkv prologue, as cases to measure.

Three operators, each on the tensors that the prologue writes (bf16, heads
contiguous per token):

  prompt  causal attention over whole prompts: q [T, n_q, D], k, v [T, n_kv, D],
          several sequences of different lengths packed along T, n_q / n_kv
          query heads per key/value head;
  train   the same with its gradients: (out, dq, dk, dv) for an upstream dout;
  decode  one new token per sequence against a paged key/value pool
          [num_pages, page_size, n_kv, D]; every sequence has its own pages,
          and the batch may share a prefix that is stored once.

``run`` computes a case with elementary torch operations in float32, or with
the package's operators when ``own`` is true. ``exact`` is the definition in
float64. Head counts are those of the package's workloads (Muse Spark 128 over
16 heads of 64, Llama 3 / Qwen3 32 over 8 heads of 128, GPT-OSS 64 over 8 heads
of 64) and, in ``draw``, generic ones.
"""

import math
import random

import torch

own = False

DEV = "cuda"


# ---------------------------------------------------------------- the cases ----

def listed():
    return [
        # one long document on the Llama 3 / Qwen3 heads
        dict(name="prompt_1x16384_d128", op="prompt", n_q=32, n_kv=8, dim=128, seqs=1, tokens=16384, pad=0, mix=1),
        # a batch of prompts of uneven length, packed, on the GPT-OSS heads
        dict(name="prompt_23x8192_d64", op="prompt", n_q=64, n_kv=8, dim=64, seqs=23, tokens=8192, pad=0, mix=2),
        # many short chats in a padded buffer (rows behind the last sequence), Muse Spark heads
        dict(name="prompt_60x4001_pad_d64", op="prompt", n_q=128, n_kv=16, dim=64, seqs=60, tokens=4001, pad=95, mix=3),
        # one short question: latency
        dict(name="prompt_1x37_d128", op="prompt", n_q=32, n_kv=8, dim=128, seqs=1, tokens=37, pad=0, mix=4),
        # a training step's attention, one long sequence
        dict(name="train_1x8192_d128", op="train", n_q=32, n_kv=8, dim=128, seqs=1, tokens=8192, pad=0, mix=5),
        # a training step on packed documents, Muse Spark heads
        dict(name="train_11x4096_d64", op="train", n_q=128, n_kv=16, dim=64, seqs=11, tokens=4096, pad=0, mix=6),
        # a small training step (a test, a fine-tune on short texts), with padding rows
        dict(name="train_3x700_pad_d64", op="train", n_q=64, n_kv=8, dim=64, seqs=3, tokens=700, pad=68, mix=7),
        # one user, a long conversation
        dict(name="decode_1x131072_d128", op="decode", n_q=32, n_kv=8, dim=128, batch=1, prefix=0, low=131072,
             high=131072, page=64, mix=8),
        # a serving batch on one long system prompt
        dict(name="decode_64_on_32768_d128", op="decode", n_q=32, n_kv=8, dim=128, batch=64, prefix=32768, low=1,
             high=2048, page=64, mix=9),
        # a large serving batch of unrelated requests of uneven length
        dict(name="decode_256x4096_d64", op="decode", n_q=64, n_kv=8, dim=64, batch=256, prefix=0, low=1, high=4096,
             page=64, mix=10),
        # parallel samples of one prompt, a prefix that ends inside a page, short continuations
        dict(name="decode_8_on_1000_d64", op="decode", n_q=128, n_kv=16, dim=64, batch=8, prefix=1000, low=0,
             high=300, page=16, mix=11),
        # the first tokens of a few short requests: latency
        dict(name="decode_3x33_d64", op="decode", n_q=64, n_kv=8, dim=64, batch=3, prefix=0, low=1, high=33, page=64,
             mix=12),
    ]


def _log_int(rng, low, high):
    return min(high, max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))))))


def draw(rng):
    op = rng.choice(("prompt", "train", "decode"))
    dim = rng.choice((64, 128))
    n_kv = rng.choice((1, 2, 3, 4, 8, 16))
    n_q = n_kv * rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
    mix = rng.randrange(1 << 20)
    if op != "decode":
        most = 16384 if op == "prompt" else 8192
        most = min(most, int(most * math.sqrt(32 / n_q)))  # n_q T^2 as in the largest listed case
        tokens = _log_int(rng, 1, most)
        seqs = _log_int(rng, 1, min(64, tokens))
        pad = rng.choice((0, 0, rng.randrange(1, 200)))
        pad = min(pad, most - tokens)
        return dict(op=op, n_q=n_q, n_kv=n_kv, dim=dim, seqs=seqs, tokens=tokens, pad=pad, mix=mix)
    batch = _log_int(rng, 1, 256)
    page = rng.choice((1, 8, 16, 24, 32, 64, 100, 128, 256))
    room = 131072 * 8 * 128 // (n_kv * dim)  # pool rows of the largest listed case
    prefix = rng.choice((0, _log_int(rng, 1, min(32768, room // 2))))
    high = _log_int(rng, 1, max(1, min(131072, (room - prefix) // (2 * batch))))
    low = rng.choice((0, 1, high // 2, high))
    # the scores that the plain form holds, float32 [batch, n_q, prefix + high]
    while batch * n_q * (prefix + high) > 1 << 30:
        batch = max(1, batch // 2)
        prefix //= 2
    return dict(op=op, n_q=n_q, n_kv=n_kv, dim=dim, batch=batch, prefix=prefix, low=low, high=high, page=page, mix=mix)


def _packed_lengths(case):
    """`seqs` lengths that add up to `tokens`: uniform cuts, so they are uneven and may be zero."""
    rng = random.Random(case["mix"])
    cuts = sorted(rng.randrange(case["tokens"] + 1) for _ in range(case["seqs"] - 1))
    ends = cuts + [case["tokens"]]
    return [b - a for a, b in zip([0] + cuts, ends)]


def _own_lengths(case):
    rng = random.Random(case["mix"])
    return [rng.randint(case["low"], case["high"]) for _ in range(case["batch"])]


# --------------------------------------------------------------- the inputs ----

def _heads(g, rows, heads, dim, spread):
    """What the prologue's norm leaves: rows of unit mean square times a weight
    near one, some heads sharper than others (`spread`)."""
    x = torch.randn(rows, heads, dim, generator=g, device=DEV)
    x *= torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    x *= 0.5 + torch.rand(dim, generator=g, device=DEV)
    x *= 1.0 + spread * torch.rand(heads, 1, generator=g, device=DEV)
    return x.to(torch.bfloat16)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 1000003 + case["mix"])
    n_q, n_kv, dim = case["n_q"], case["n_kv"], case["dim"]
    s = dict(op=case["op"], n_q=n_q, n_kv=n_kv, dim=dim)
    if case["op"] != "decode":
        lengths = _packed_lengths(case)
        T = case["tokens"] + case["pad"]
        ends = [0]
        for n in lengths:
            ends.append(ends[-1] + n)
        s["cu"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
        s["q"] = _heads(g, T, n_q, dim, 1.0)
        s["k"] = _heads(g, T, n_kv, dim, 0.0)
        s["v"] = torch.randn(T, n_kv, dim, generator=g, device=DEV).to(torch.bfloat16)
        if case["op"] == "train":
            s["dout"] = torch.randn(T, n_q, dim, generator=g, device=DEV).to(torch.bfloat16)
        return s
    lengths = _own_lengths(case)
    page, prefix = case["page"], case["prefix"]
    own_pages = [-(-n // page) for n in lengths]
    prefix_pages = -(-prefix // page)
    total = prefix_pages + sum(own_pages) + 3
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    s["k_pool"] = _heads(g, total * page, n_kv, dim, 0.0).view(total, page, n_kv, dim)
    s["v_pool"] = torch.randn(total, page, n_kv, dim, generator=g, device=DEV, dtype=torch.bfloat16)
    s["q"] = _heads(g, case["batch"], n_q, dim, 1.0)
    s["prefix_pages"] = order[:prefix_pages].contiguous() if prefix else None
    s["prefix_len"] = prefix
    # each sequence's pages: a row of the table, zero past its last page
    counts = torch.tensor(own_pages, device=DEV)
    wide = max(1, max(own_pages))
    at = torch.arange(wide, device=DEV)[None, :]
    before = prefix_pages + torch.cumsum(counts, 0) - counts
    taken = order[(before[:, None] + at).clamp_(max=total - 1)]
    s["page_table"] = torch.where(at < counts[:, None], taken, torch.zeros_like(taken)).contiguous()
    s["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=DEV)
    return s


# ----------------------------------------------------------- the plain form ----

def _grouped(x, n_kv):
    """[T, n_q, D] -> float32 [n_kv, G, T, D] (query head h reads key/value head h // G)."""
    T, n, D = x.shape
    return x.float().view(T, n_kv, n // n_kv, D).permute(1, 2, 0, 3)


def _packed_weights(s):
    """Softmax weights [n_kv, G, T, T] of the packed causal mask, zero rows for
    tokens of no sequence, and the float32 operands."""
    n_kv, T = s["n_kv"], s["q"].shape[0]
    q, k, v = _grouped(s["q"], n_kv), _grouped(s["k"], n_kv), _grouped(s["v"], n_kv)
    at = torch.arange(T, device=DEV)
    which = torch.searchsorted(s["cu"].long(), at, right=True)  # 1 .. batch inside the sequences
    inside = (which >= 1) & (which < s["cu"].numel())
    mask = (which[:, None] == which[None, :]) & (at[:, None] >= at[None, :]) & inside[:, None]
    w = torch.matmul(q, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(s["dim"]))
    w.masked_fill_(~mask, float("-inf"))
    top = w.amax(-1, keepdim=True)
    w.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = w.sum(-1, keepdim=True)
    w.div_(torch.where(total > 0, total, torch.ones_like(total)))
    return w, q, k, v


def _tokens_first(x):
    """[n_kv, G, T, D] -> bf16 [T, n_kv * G, D]"""
    n_kv, G, T, D = x.shape
    return x.permute(2, 0, 1, 3).reshape(T, n_kv * G, D).to(torch.bfloat16)


def _plain_prompt(s):
    w, _, _, v = _packed_weights(s)
    return _tokens_first(torch.matmul(w, v))


def _plain_train(s):
    w, q, k, v = _packed_weights(s)
    do = _grouped(s["dout"], s["n_kv"])
    out = torch.matmul(w, v)
    dv = torch.matmul(w.transpose(-1, -2), do).sum(1, keepdim=True)
    ds = torch.matmul(do, v.transpose(-1, -2))
    ds.sub_((do * out).sum(-1, keepdim=True)).mul_(w).mul_(1.0 / math.sqrt(s["dim"]))
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(1, keepdim=True)
    return tuple(_tokens_first(x) for x in (out, dq, dk, dv))


def _rows_of(pages, count, page_size):
    """Pool rows of `count` consecutive tokens stored in `pages` [..., n]."""
    at = torch.arange(count, device=DEV)
    return pages.long()[..., at // page_size] * page_size + at % page_size


def _plain_decode(s):
    n_kv, D, page_size = s["n_kv"], s["dim"], s["k_pool"].shape[1]
    B = s["q"].shape[0]
    q = s["q"].float().view(B, n_kv, -1, D)
    k_rows, v_rows = s["k_pool"].view(-1, n_kv, D), s["v_pool"].view(-1, n_kv, D)
    wide = s["page_table"].shape[1] * page_size
    own_rows = _rows_of(s["page_table"], wide, page_size)
    k = k_rows[own_rows].float()  # [B, wide, n_kv, D]
    w = torch.einsum("bhgd,bnhd->bhgn", q, k).mul_(1.0 / math.sqrt(D))
    hidden = torch.arange(wide, device=DEV)[None, :] >= s["lengths"][:, None]
    w.masked_fill_(hidden[:, None, None, :], float("-inf"))
    if s["prefix_len"]:
        shared = _rows_of(s["prefix_pages"], s["prefix_len"], page_size)
        k = k_rows[shared].float()  # [prefix, n_kv, D]
        w = torch.cat((torch.einsum("bhgd,nhd->bhgn", q, k).mul_(1.0 / math.sqrt(D)), w), -1)
    top = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(torch.isfinite(top), top, torch.zeros_like(top))).exp_()
    total = w.sum(-1, keepdim=True)
    w.div_(torch.where(total > 0, total, torch.ones_like(total)))
    out = torch.einsum("bhgn,bnhd->bhgd", w[..., s["prefix_len"]:], v_rows[own_rows].float())
    if s["prefix_len"]:
        out += torch.einsum("bhgn,nhd->bhgd", w[..., :s["prefix_len"]], v_rows[shared].float())
    return out.reshape(B, -1, D).to(torch.bfloat16)


def run(state):
    s = state
    if own:
        from rope_qkv_prologue_gb300 import functional as F

        if s["op"] == "prompt":
            return F.attention_forward(s["q"], s["k"], s["v"], s["cu"])
        if s["op"] == "train":
            out, lse = F.attention_forward(s["q"], s["k"], s["v"], s["cu"], save_lse=True)
            return (out, *F.attention_backward(s["dout"], s["q"], s["k"], s["v"], out, lse, s["cu"]))
        return F.attention_decode(s["q"], s["k_pool"], s["v_pool"], s["page_table"], s["lengths"],
                                  s["prefix_pages"], s["prefix_len"])
    return {"prompt": _plain_prompt, "train": _plain_train, "decode": _plain_decode}[s["op"]](s)


# ------------------------------------------------------------ what it costs ----

def work(case):
    n_q, n_kv, D = case["n_q"], case["n_kv"], case["dim"]
    if case["op"] == "decode":
        lengths = _own_lengths(case)
        keys = sum(lengths)
        scored = keys + case["batch"] * case["prefix"]
        rows = keys + case["prefix"]
        return {"bytes": 4 * rows * n_kv * D + 4 * case["batch"] * n_q * D, "flops": 4 * D * n_q * scored}
    pairs = sum(n * (n + 1) // 2 for n in _packed_lengths(case))
    T = case["tokens"]
    tensor_q, tensor_k = 2 * T * n_q * D, 2 * T * n_kv * D
    if case["op"] == "prompt":  # q, k, v read, out written; two products
        return {"bytes": 2 * tensor_q + 2 * tensor_k, "flops": 4 * D * n_q * pairs}
    # q, k, v, dout read, out, dq, dk, dv written; two products forward, five backward
    return {"bytes": 4 * tensor_q + 4 * tensor_k, "flops": 14 * D * n_q * pairs}


# ------------------------------------------------- the definition in 64 bits ----

def _exact_rows(q, k, first, scale):
    """Softmax weights in float64 of query rows first, first + 1, ... of one
    sequence over its keys 0 .. first + rows - 1, each row up to itself."""
    rows, keys = q.shape[0], first + q.shape[0]
    e = (q @ k[:keys].T) * scale
    later = torch.arange(keys, device=DEV)[None, :] > first + torch.arange(rows, device=DEV)[:, None]
    e[later] = -math.inf
    e = torch.exp(e - e.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _exact_packed(s, grads):
    T, n_q, D = s["q"].shape
    G, scale, step = n_q // s["n_kv"], D ** -0.5, 4096
    out = torch.zeros(T, n_q, D, dtype=torch.float64, device=DEV)
    dq = torch.zeros_like(out)
    dk = torch.zeros(T, s["n_kv"], D, dtype=torch.float64, device=DEV)
    dv = torch.zeros_like(dk)
    ends = s["cu"].tolist()
    for a, b in zip(ends, ends[1:]):
        for h in range(n_q):
            k, v = s["k"][a:b, h // G].double(), s["v"][a:b, h // G].double()
            for r in range(0, b - a, step):
                q = s["q"][a + r:min(b, a + r + step), h].double()
                n, keys = q.shape[0], r + q.shape[0]
                p = _exact_rows(q, k, r, scale)
                here = slice(a + r, a + r + n)
                out[here, h] = p @ v[:keys]
                if grads:
                    do = s["dout"][here, h].double()
                    dv[a:a + keys, h // G] += p.T @ do
                    dp = do @ v[:keys].T
                    ds = p * (dp - (p * dp).sum(1, keepdim=True)) * scale
                    dq[here, h] = ds @ k[:keys]
                    dk[a:a + keys, h // G] += ds.T @ q
    return (out, dq, dk, dv) if grads else out


def _exact_decode(s):
    B, n_q, D = s["q"].shape
    n_kv, page_size = s["n_kv"], s["k_pool"].shape[1]
    G = n_q // n_kv
    flat_k, flat_v = s["k_pool"].flatten(0, 1), s["v_pool"].flatten(0, 1)

    def stored(pages, count):
        token = torch.arange(count, device=DEV)
        row = pages.to(torch.int64)[torch.div(token, page_size, rounding_mode="floor")] * page_size + token % page_size
        return flat_k[row].double().transpose(0, 1), flat_v[row].double().transpose(0, 1)  # [n_kv, count, D]

    shared = stored(s["prefix_pages"], s["prefix_len"]) if s["prefix_len"] else None
    out = torch.zeros(B, n_q, D, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["lengths"].tolist()):
        parts = ([shared] if shared is not None else []) + ([stored(s["page_table"][b], n)] if n else [])
        if not parts:
            continue
        q = s["q"][b].double().view(n_kv, G, D)
        e = torch.cat([q @ k.transpose(1, 2) for k, _ in parts], 2) * D ** -0.5
        e = torch.exp(e - e.max(2, keepdim=True).values)
        e = e / e.sum(2, keepdim=True)
        at = 0
        for k, v in parts:
            out[b] += (e[:, :, at:at + k.shape[1]] @ v).reshape(n_q, D)
            at += k.shape[1]
    return out


def exact(case, seed):
    """The definition in float64. None where its products (about 1.2 TFLOP/s) or
    its loop over sequences and heads would take too long."""
    w = work(case)
    if w["flops"] > 8e12:
        return None
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_decode(s)
    return _exact_packed(s, case["op"] == "train")
