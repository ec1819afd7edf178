"""Tensor-level helpers over the C ABI: they allocate outputs with torch (device
memory is PyTorch's job here) and call the library. No arithmetic happens in
Python.

The training entry point, ``QKVPrologue.apply``, mirrors the region of
"[muse_spark][perf] Split the packed qkv inside the q/k region" (Solution):
packed qkv in, contiguous q, k, v out; its backward writes the gradient of the
packed tensor in one pass.
"""

import functools

import torch

from . import _lib as C


def _layout_of(packed, n_q, n_kv, head_dim, kind):
    T = packed.shape[0]
    row = packed.reshape(T, -1) if packed.is_contiguous() else None
    if row is None:
        raise ValueError("packed must be contiguous ([T, ...] rows)")
    width = row.shape[1]
    if width != (n_q + 2 * n_kv) * head_dim:
        raise ValueError(f"packed row has {width} values, expected (n_q + 2 n_kv) * head_dim = "
                         f"{(n_q + 2 * n_kv) * head_dim}")
    return C.layout(kind, n_q, n_kv, head_dim), T


def _check_dev(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must live on a CUDA device")


def _variant(bias=None, inv_freq=None, rope_scale=1.0):
    """The qkvp_variant of the GQAttention options, or None for the plain call."""
    if bias is None and inv_freq is None and rope_scale in (None, 0.0, 1.0):
        return None
    if bias is not None:
        _check_dev(bias)
        if bias.dtype != torch.float32 or not bias.is_contiguous():
            raise ValueError("bias must be a contiguous float32 tensor")
    return C.variant(inv_freq=None if inv_freq is None else [float(f) for f in inv_freq],
                     rope_scale=0.0 if rope_scale is None else float(rope_scale), bias=bias)


def _flags(nope=False, save_pre=False, norm=True):
    return (C.QKVP_NOPE if nope else 0) | (C.QKVP_SAVE_PRE if save_pre else 0) | (0 if norm else C.QKVP_NORM_OFF)


def prologue_forward(packed, pos, w_q, w_k, n_q, n_kv, head_dim=64, kind="interleaved", eps=1e-6,
                     rope_base=500000.0, nope=False, save_pre=False, stream=None, norm=True, bias=None,
                     inv_freq=None, rope_scale=1.0):
    """Split + per-head RMSNorm + RoPE. Returns (q, k, v) or (q, k, v, q_pre, k_pre).

    The GQAttention variant options: norm=False (split -> RoPE only; w_q, w_k
    may be None), bias (float32 [(n_q + 2 n_kv) * head_dim] in the packed
    row's order, added first), inv_freq (head_dim / 2 frequencies replacing
    rope_base**(-2i/D)) and rope_scale (factor on cos and sin)."""
    _check_dev(packed, pos, w_q, w_k)
    L, T = _layout_of(packed, n_q, n_kv, head_dim, kind)
    dev = packed.device
    q = torch.empty(T, n_q, head_dim, dtype=torch.bfloat16, device=dev)
    k = torch.empty(T, n_kv, head_dim, dtype=torch.bfloat16, device=dev)
    v = torch.empty(T, n_kv, head_dim, dtype=torch.bfloat16, device=dev)
    q_pre = torch.empty_like(q) if save_pre else None
    k_pre = torch.empty_like(k) if save_pre else None
    C.qkv_prologue_fwd_ex(L, _variant(bias, inv_freq, rope_scale), T, packed, pos, w_q, w_k, eps, rope_base,
                          _flags(nope, save_pre, norm), q, k, v, q_pre, k_pre, stream)
    return (q, k, v, q_pre, k_pre) if save_pre else (q, k, v)


def prologue_backward(dq, dk, dv, q_pre, k_pre, pos, w_q, w_k, n_q, n_kv, head_dim=64,
                      kind="interleaved", eps=1e-6, rope_base=500000.0, nope=False, stream=None,
                      workspace=None, norm=True, bias=None, inv_freq=None, rope_scale=1.0):
    """Packed gradient [T, (n_q + 2 n_kv) * head_dim] and fp32 (dw_q, dw_k), plus
    the fp32 bias gradient when a bias is given: (dpacked, dw_q, dw_k[, dbias]).
    Without the norm dw_q, dw_k are None and q_pre, k_pre, w_q, w_k may be None."""
    _check_dev(dq, dk, dv, q_pre, k_pre, w_q, w_k)
    T = dq.shape[0]
    L = C.layout(kind, n_q, n_kv, head_dim)
    dev = dq.device
    V = _variant(bias, inv_freq, rope_scale)
    dpacked = torch.empty(T, (n_q + 2 * n_kv) * head_dim, dtype=torch.bfloat16, device=dev)
    dw_q = torch.empty(head_dim, dtype=torch.float32, device=dev) if norm else None
    dw_k = torch.empty(head_dim, dtype=torch.float32, device=dev) if norm else None
    dbias = torch.empty((n_q + 2 * n_kv) * head_dim, dtype=torch.float32, device=dev) if bias is not None else None
    need = C.qkv_prologue_bwd_workspace_size_ex(L, V, T)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    C.qkv_prologue_bwd_ex(L, V, T, dq, dk, dv, q_pre, k_pre, pos, w_q, w_k, eps, rope_base,
                          _flags(nope, False, norm), dpacked, dw_q, dw_k, dbias, workspace, need, stream)
    return (dpacked, dw_q, dw_k, dbias) if bias is not None else (dpacked, dw_q, dw_k)


def prologue_pool_write(packed, pos, w_q, w_k, page, offset, k_pool, v_pool, n_q, n_kv, head_dim=64,
                        kind="interleaved", eps=1e-6, rope_base=500000.0, nope=False, dev_status=None,
                        stream=None, norm=True, bias=None, inv_freq=None, rope_scale=1.0):
    """q contiguous; normed(+roped) k and raw v into the paged pools. Returns q."""
    _check_dev(packed, pos, w_q, w_k, page, offset, k_pool, v_pool)
    L, T = _layout_of(packed, n_q, n_kv, head_dim, kind)
    q = torch.empty(T, n_q, head_dim, dtype=torch.bfloat16, device=packed.device)
    C.qkv_prologue_pool_write_ex(L, _variant(bias, inv_freq, rope_scale), T, packed, pos, w_q, w_k, eps,
                                 rope_base, _flags(nope, False, norm), q, page, offset, k_pool, v_pool,
                                 k_pool.shape[0], k_pool.shape[1], dev_status, stream)
    return q


def latent_rows(rows, pos, w, eps=1e-6, rope_base=10000.0, norm_dim=512, rope_dim=64, nope=False,
                stream=None, inv_freq=None, rope_scale=1.0):
    """MLA kv latent rows normed/roped into a new contiguous [T, norm_dim + rope_dim] tensor."""
    _check_dev(rows, pos, w)
    T = rows.shape[0]
    L = C.layout("latent", norm_dim=norm_dim, rope_dim=rope_dim)
    out = torch.empty(T, norm_dim + rope_dim, dtype=torch.bfloat16, device=rows.device)
    C.qkv_prologue_fwd_ex(L, _variant(None, inv_freq, rope_scale), T, rows, pos, None, w, eps, rope_base,
                          _flags(nope), None, out, None, None, None, stream)
    return out


def latent_pool_write(rows, pos, w, page, offset, pool, eps=1e-6, rope_base=10000.0, norm_dim=512,
                      rope_dim=64, nope=False, dev_status=None, stream=None, inv_freq=None, rope_scale=1.0):
    """MLA kv latent rows normed/roped straight into pool [num_pages, page_size, 576]."""
    _check_dev(rows, pos, w, page, offset, pool)
    T = rows.shape[0]
    L = C.layout("latent", norm_dim=norm_dim, rope_dim=rope_dim)
    C.qkv_prologue_pool_write_ex(L, _variant(None, inv_freq, rope_scale), T, rows, pos, None, w, eps, rope_base,
                                 _flags(nope), None, page, offset, pool, None, pool.shape[0], pool.shape[1],
                                 dev_status, stream)


def gemm_prologue_forward(x, w_qkv, pos, w_q, w_k, n_q, n_kv, head_dim=64, kind="interleaved", eps=1e-6,
                          rope_base=500000.0, nope=False, save_pre=False, stream=None):
    """The wqkv projection with the prologue in its epilogue: x [T, hidden] bf16,
    w_qkv [(n_q + 2 n_kv) * head_dim, hidden] bf16 (rows in the layout's packed
    order) -> (q, k, v) or (q, k, v, q_pre, k_pre); the packed tensor is never
    materialised."""
    _check_dev(x, w_qkv, pos, w_q, w_k)
    if x.dim() != 2 or w_qkv.dim() != 2 or x.shape[1] != w_qkv.shape[1]:
        raise ValueError("x must be [T, hidden] and w_qkv [rows, hidden]")
    if w_qkv.shape[0] != (n_q + 2 * n_kv) * head_dim:
        raise ValueError("w_qkv must have (n_q + 2 n_kv) * head_dim rows")
    T, hidden = x.shape
    L = C.layout(kind, n_q, n_kv, head_dim)
    dev = x.device
    q = torch.empty(T, n_q, head_dim, dtype=torch.bfloat16, device=dev)
    k = torch.empty(T, n_kv, head_dim, dtype=torch.bfloat16, device=dev)
    v = torch.empty(T, n_kv, head_dim, dtype=torch.bfloat16, device=dev)
    q_pre = torch.empty_like(q) if save_pre else None
    k_pre = torch.empty_like(k) if save_pre else None
    C.qkv_prologue_gemm_fwd(L, T, hidden, x.contiguous(), w_qkv.contiguous(), pos, w_q, w_k, eps, rope_base,
                            _flags(nope, save_pre), q, k, v, q_pre, k_pre, stream)
    return (q, k, v, q_pre, k_pre) if save_pre else (q, k, v)


def per_head_newton_schulz(m, n_q, n_kv, head_dim=64, kind="interleaved", split=0, out=None, workspace=None,
                           stream=None):
    """Per-head Newton-Schulz of a fused QKV weight's update m
    [(n_q + 2 n_kv) * head_dim, in_features] bf16: every head_dim-row block
    orthogonalised on its own (Muon's quintic iteration, five steps) and scaled
    by max(1, head_dim / in_features) ** 0.5 ("[muon] Per-head Newton-Schulz for
    fused QKV projections", What this PR does). `kind` names the packing of the
    rows; the result does not depend on it. A 3-D m [count, rows, cols] (one
    update per layer) is done in one set of launches. `workspace` (a device
    tensor of at least newton_schulz_workspace_bytes bytes) is allocated here
    when not given; `split` fixes the Gram pass's CTAs per 128-row unit."""
    _check_dev(m)
    if m.dim() not in (2, 3) or m.dtype != torch.bfloat16:
        raise ValueError("m must be a bf16 [rows, cols] or [count, rows, cols] tensor")
    if m.shape[-2] != (n_q + 2 * n_kv) * head_dim:
        raise ValueError("m must have (n_q + 2 n_kv) * head_dim rows")
    m = m.contiguous()
    if out is None:
        out = torch.empty_like(m)
    L = C.layout(kind, n_q, n_kv, head_dim)
    count = 1 if m.dim() == 2 else m.shape[0]
    need = C.qkv_newton_schulz_workspace(L, m.shape[-1], split, count)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=m.device)
    nbytes = workspace.numel() * workspace.element_size()
    if m.dim() == 2:
        C.qkv_newton_schulz(L, m.shape[1], m, out, split, workspace, nbytes, stream)
    else:  # every weight of the stack in one set of launches
        C.qkv_newton_schulz_batch(L, count, m.shape[2], m, out, split, workspace, nbytes, stream)
    return out


def newton_schulz_workspace_bytes(m_shape, n_q, n_kv, head_dim=64, kind="interleaved", split=0):
    """Workspace bytes per_head_newton_schulz needs for an update of this shape."""
    count = 1 if len(m_shape) == 2 else m_shape[0]
    return C.qkv_newton_schulz_workspace(C.layout(kind, n_q, n_kv, head_dim), m_shape[-1], split, count)


def on_side_stream(side, fn, *args, **kwargs):
    """Run fn(*args, **kwargs) on CUDA stream `side`, forked from the current
    stream: `side` first waits for everything already queued on the current
    stream, and the returned event is recorded on `side` after fn's work. The
    caller joins with ``torch.cuda.current_stream().wait_event(event)`` before
    anything that reads fn's results.

    This is the drafter-layer pattern of "MLA DSpark: run each drafter layer's
    kv path beside its q path" (Description): the kv path (kv projection ->
    latent norm/RoPE -> direct pool write) forks to an aux stream after the input
    layernorm, the q path runs on the main stream, and attention joins. Works
    under CUDA graph capture (the fork and join become graph edges). Tensors made
    on the current stream and used on `side` must stay alive until the join.
    """
    main = torch.cuda.current_stream()
    side.wait_stream(main)
    with torch.cuda.stream(side):
        out = fn(*args, **kwargs)
        done = torch.cuda.Event()
        done.record(side)
    return out, done


def join(event, stream=None):
    """Make `stream` (default: the current stream) wait for `event`, the join of
    a fork made with on_side_stream or mla_kv_path_beside. Under CUDA graph
    capture this becomes a graph edge."""
    (stream or torch.cuda.current_stream()).wait_event(event)


def mla_kv_path_beside(side, pos, w, page, offset, pool, kv_rows=None, kv_proj=None, eps=1e-6,
                       rope_base=10000.0, norm_dim=512, rope_dim=64, nope=False, dev_status=None,
                       inv_freq=None, rope_scale=1.0):
    """The kv path of one MLA drafter layer on the side stream `side`, beside
    the q path on the current stream ("MLA DSpark: run each drafter layer's kv
    path beside its q path", Description): fork after the layer's input norm,
    run the kv path there, join before attention reads the pool.

    The kv path is: the kv_a rows [T, norm_dim + rope_dim] bf16 (either
    `kv_rows`, already computed, or `kv_proj()`, a callable run on `side` that
    returns them, e.g. the kv_a projection of the layer input), then the
    library's latent norm / RoPE written straight into `pool` [num_pages,
    page_size, norm_dim + rope_dim] at (page, offset) (latent_pool_write).

    Returns (kv_rows, join_event). Everything the caller queued on the current
    stream before the call is visible to the kv path; nothing on the current
    stream waits for it until the caller joins (join(join_event)) -- do that
    before anything reads `pool` or the returned rows. Inputs made on the
    current stream must stay alive until the join. Works under CUDA graph
    capture: the fork and the join become graph edges."""
    if (kv_rows is None) == (kv_proj is None):
        raise ValueError("give exactly one of kv_rows and kv_proj")

    def kv_path():
        rows = kv_proj() if kv_proj is not None else kv_rows
        latent_pool_write(rows, pos, w, page, offset, pool, eps, rope_base, norm_dim, rope_dim, nope,
                          dev_status, None, inv_freq, rope_scale)
        return rows

    return on_side_stream(side, kv_path)


@functools.lru_cache(maxsize=1024)
def _heads(n_q, n_kv, head_dim):
    """The layout struct of these heads (the library only reads it)."""
    return C.layout("sectioned", n_q, n_kv, head_dim)


@functools.lru_cache(maxsize=1024)
def _decode_workspace(n_q, n_kv, head_dim, batch, page_size, max_pages, prefix_len, device_index):
    return C.qkv_attention_decode_workspace(_heads(n_q, n_kv, head_dim), batch, page_size, max_pages, prefix_len)


def _current_stream(device):
    """The raw handle of the current stream of `device`, the current device."""
    if device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {device}, which is not the current device")
    return torch._C._cuda_getCurrentRawStream(device.index)


def _on_stream(stream, like, call, *args):
    """call(*args) with `stream` (a torch.cuda.Stream or a raw handle) as the current
    one: what it allocates is then that stream's memory, in its order. The results may
    be used on the caller's stream (after it waited), so their memory is kept for it too;
    and the arguments' memory is kept for `stream`, so that the caller may drop them
    before it has read them."""
    if not like.is_cuda:
        raise ValueError("the tensors must live on a CUDA device")
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, like.device)
    if stream.device != like.device:
        raise ValueError(f"the tensors are on {like.device}, the stream is of {stream.device}")
    for t in args:
        if isinstance(t, torch.Tensor) and t.device == like.device:  # (what lies elsewhere is refused)
            t.record_stream(stream)
    with torch.cuda.stream(stream):
        got = call(*args)
    home = torch.cuda.current_stream(like.device)
    for t in got if isinstance(got, tuple) else (got,):
        t.record_stream(home)
    return got


def _check_qkv(q, k, v):
    for t in (q, k, v):
        if t.dtype != torch.bfloat16 or t.dim() != 3 or not t.is_contiguous():
            raise ValueError("q, k and v must be contiguous bf16 [T, heads, head_dim] tensors")
    if k.shape != v.shape or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("k and v must have one shape, and q's rows and head_dim")
    if not q.is_cuda or k.device != q.device or v.device != q.device:
        raise ValueError("q, k and v must live on one CUDA device")


def _check_like(t, shape, dtype, device, name):
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {list(shape)} tensor on {device}")


def _check_offsets(cu_seqlens, device):
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be [batch + 1]")
    _check_like(cu_seqlens, cu_seqlens.shape, torch.int32, device, "cu_seqlens")
    return cu_seqlens.shape[0] - 1


def _check_workspace(workspace, device):
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")


def _check_status(dev_status, device):
    if dev_status is not None and (dev_status.dtype != torch.int32 or dev_status.numel() < 1
                                   or dev_status.device != device):
        raise ValueError(f"dev_status must be an int32 tensor on {device}")


def attention_forward(q, k, v, cu_seqlens, scale=None, save_lse=False, out=None, dev_status=None, stream=None):
    """Causal attention over packed sequences: q [T, n_q, D], k, v [T, n_kv, D]
    bf16 as prologue_forward returns them, cu_seqlens int32 [batch + 1] on the
    device (sequence s is the rows cu_seqlens[s] .. cu_seqlens[s + 1] - 1). A row
    attends all of its sequence up to itself: no sliding window, no sink.
    Returns out [T, n_q, D], or (out, lse [n_q, T] float32) with save_lse.
    scale defaults to D ** -0.5 (0 is that too). Rows of no sequence are zero in an out made
    here, and left as they are in one given (lse: -inf, in both). The work is
    queued on `stream` (default: the current one), which waits for nothing by
    itself; the arguments may be dropped as soon as the call returns."""
    if stream is not None:
        return _on_stream(stream, q, attention_forward, q, k, v, cu_seqlens, scale, save_lse, out, dev_status)
    _check_qkv(q, k, v)
    dev = q.device
    batch = _check_offsets(cu_seqlens, dev)
    _check_status(dev_status, dev)
    T, n_q, D = q.shape
    flags = 0
    if out is None:
        out = torch.empty_like(q)
        flags = C.QKVP_ZERO_REST
    else:
        _check_like(out, q.shape, torch.bfloat16, dev, "out")
    lse = None
    if save_lse:
        lse = torch.empty((n_q, T), dtype=torch.float32, device=dev)
        if not flags:
            lse.fill_(float("-inf"))
    if T == 0:  # an empty tensor has no address to pass
        return (out, lse) if save_lse else out
    C.qkv_attention_fwd(_heads(n_q, k.shape[1], D), T, batch, cu_seqlens, q, k, v, 0.0 if scale is None else scale,
                        flags, out, lse, dev_status, _current_stream(dev))
    return (out, lse) if save_lse else out


@functools.lru_cache(maxsize=1024)
def attention_backward_workspace_bytes(n_q, n_kv, head_dim, T, batch):
    """Workspace bytes attention_backward needs for T rows in `batch` sequences."""
    return C.qkv_attention_bwd_workspace(_heads(n_q, n_kv, head_dim), T, batch)


def attention_backward(dout, q, k, v, out, lse, cu_seqlens, scale=None, workspace=None, dev_status=None, stream=None):
    """Gradients (dq, dk, dv) of attention_forward(q, k, v, cu_seqlens, scale) for
    the upstream gradient dout [T, n_q, D] bf16, from the forward's out and lse.
    Rows of no sequence get zero gradients. `workspace` (a device tensor of
    attention_backward_workspace_bytes bytes) is allocated here when not given.
    The work is queued on `stream` (default: the current one), as attention_forward's."""
    if stream is not None:
        return _on_stream(stream, q, attention_backward, dout, q, k, v, out, lse, cu_seqlens, scale, workspace,
                          dev_status)
    _check_qkv(q, k, v)
    dev = q.device
    T, n_q, D = q.shape
    batch = _check_offsets(cu_seqlens, dev)
    _check_status(dev_status, dev)
    _check_like(dout, q.shape, torch.bfloat16, dev, "dout")
    _check_like(out, q.shape, torch.bfloat16, dev, "out")
    _check_like(lse, (n_q, T), torch.float32, dev, "lse")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    if T == 0:
        return dq, dk, dv
    if workspace is None:
        need = attention_backward_workspace_bytes(n_q, k.shape[1], D, T, batch)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    _check_workspace(workspace, dev)
    C.qkv_attention_bwd(_heads(n_q, k.shape[1], D), T, batch, cu_seqlens, dout, q, k, v, out, lse,
                        0.0 if scale is None else scale, C.QKVP_ZERO_REST, dq, dk, dv, dev_status, workspace,
                        workspace.numel() * workspace.element_size(), _current_stream(dev))
    return dq, dk, dv


class PackedAttention(torch.autograd.Function):
    """apply(q, k, v, cu_seqlens, scale=None) -> out: causal attention over packed
    sequences with its gradients, the step after QKVPrologue.apply. The offsets
    receive no gradient, and the gradients have none of their own. In a CUDA graph,
    capture the forward and its backward together, and let no eager autograd graph
    of the same leaves be alive then: their accumulation would wait for the stream
    of that graph, which a capture does not allow."""

    @staticmethod
    def forward(ctx, q, k, v, cu_seqlens, scale=None):
        out, lse = attention_forward(q, k, v, cu_seqlens, scale, save_lse=True)
        ctx.save_for_backward(q, k, v, out, lse, cu_seqlens)
        ctx.scale = scale
        return out

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        q, k, v, out, lse, cu_seqlens = ctx.saved_tensors
        dq, dk, dv = attention_backward(dout.contiguous(), q, k, v, out, lse, cu_seqlens, ctx.scale)
        return dq, dk, dv, None, None


def _check_pages(pages, name, device, dim):
    if pages.dim() != dim or pages.dtype != torch.int32 or pages.device != device:
        raise ValueError(f"{name} must be a {dim}-dimensional int32 tensor on {device}")
    if pages.shape[-1] > 1 and pages.stride(-1) != 1:
        raise ValueError(f"the entries of a row of {name} must be contiguous")


def attention_decode_workspace_bytes(n_q, n_kv, head_dim, batch, page_size, max_pages, prefix_len=0):
    """Workspace bytes attention_decode needs for these sizes on the current device."""
    return C.qkv_attention_decode_workspace(_heads(n_q, n_kv, head_dim), batch, page_size, max_pages, prefix_len)


def attention_decode(q, k_pool, v_pool, page_table, lengths, prefix_pages=None, prefix_len=0, scale=None,
                     save_lse=False, out=None, workspace=None, dev_status=None, stream=None):
    """Attention of one new token per sequence over a paged pool: q [B, n_q, D]
    bf16; k_pool, v_pool [num_pages, page_size, n_kv, D] as prologue_pool_write
    fills them; page_table int32 [B, max_pages] (rows may be a slice of a wider
    table) and lengths int32 [B] name each sequence's own tokens, the new one
    among them. The first prefix_len tokens of prefix_pages (int32 [n]) precede
    them in every sequence: stored once, and read once for the whole batch.
    Returns out [B, n_q, D], or (out, lse [B, n_q] float32) with save_lse.
    `workspace` (a device tensor of attention_decode_workspace_bytes bytes) is
    allocated here when not given. The work is queued on `stream` (default: the
    current one), as attention_forward's."""
    if stream is not None:
        return _on_stream(stream, q, attention_decode, q, k_pool, v_pool, page_table, lengths, prefix_pages,
                          prefix_len, scale, save_lse, out, workspace, dev_status)
    for t, n in ((q, 3), (k_pool, 4), (v_pool, 4)):
        if t.dtype != torch.bfloat16 or t.dim() != n or not t.is_contiguous():
            raise ValueError("q must be a contiguous bf16 [B, n_q, D] and the pools contiguous bf16 "
                             "[num_pages, page_size, n_kv, D] tensors")
    dev, (B, n_q, D) = q.device, q.shape
    num_pages, page_size, n_kv, _ = k_pool.shape
    if k_pool.shape != v_pool.shape or k_pool.shape[3] != D:
        raise ValueError("k_pool and v_pool must have one shape, and q's head_dim")
    if not q.is_cuda or k_pool.device != dev or v_pool.device != dev:
        raise ValueError("q and the pools must live on one CUDA device")
    _check_pages(page_table, "page_table", dev, 2)
    max_pages = page_table.shape[1]
    if page_table.shape[0] != B or (B > 1 and page_table.stride(0) < max_pages):
        raise ValueError("page_table must have a row per sequence, and the rows must not overlap")
    _check_like(lengths, (B,), torch.int32, dev, "lengths")
    _check_status(dev_status, dev)
    if prefix_len:
        if prefix_pages is None or prefix_len < 0:
            raise ValueError("a prefix needs prefix_len >= 0 and its pages")
        _check_pages(prefix_pages, "prefix_pages", dev, 1)
        if prefix_pages.shape[0] * page_size < prefix_len:
            raise ValueError("prefix_pages must hold prefix_len tokens")
    else:
        prefix_pages = None
    lse = None
    if out is None:
        out = torch.empty_like(q)
    else:
        _check_like(out, q.shape, torch.bfloat16, dev, "out")
    if save_lse:
        lse = torch.empty((B, n_q), dtype=torch.float32, device=dev)
    if B == 0:
        return (out, lse) if save_lse else out
    here = _current_stream(dev)  # before a size is asked for: it is the current device's
    if workspace is None:
        need = _decode_workspace(n_q, n_kv, D, B, page_size, max_pages, prefix_len, dev.index)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    _check_workspace(workspace, dev)
    C.qkv_attention_decode(_heads(n_q, n_kv, D), B, q, k_pool, v_pool, num_pages, page_size, page_table, max_pages,
                           page_table.stride(0) if B > 1 else max_pages, lengths, prefix_pages, prefix_len,
                           0.0 if scale is None else scale, out, lse, dev_status, workspace,
                           workspace.numel() * workspace.element_size(), here)
    return (out, lse) if save_lse else out


class QKVPrologue(torch.autograd.Function):
    """packed [T, row] -> (q, k, v); backward writes d(packed) in one pass.

    The norm weights w_q, w_k are float32 [head_dim] tensors and receive
    gradients; positions do not.
    """

    @staticmethod
    def forward(ctx, packed, pos, w_q, w_k, n_q, n_kv, head_dim, kind, eps, rope_base, nope):
        q, k, v, q_pre, k_pre = prologue_forward(packed, pos, w_q, w_k, n_q, n_kv, head_dim, kind, eps,
                                                 rope_base, nope, save_pre=True)
        ctx.save_for_backward(q_pre, k_pre, pos, w_q, w_k)
        ctx.cfg = (n_q, n_kv, head_dim, kind, eps, rope_base, nope, packed.shape)
        return q, k, v

    @staticmethod
    def backward(ctx, dq, dk, dv):
        q_pre, k_pre, pos, w_q, w_k = ctx.saved_tensors
        n_q, n_kv, head_dim, kind, eps, rope_base, nope, shape = ctx.cfg
        dq, dk, dv = (g.contiguous() for g in (dq, dk, dv))
        dpacked, dw_q, dw_k = prologue_backward(dq, dk, dv, q_pre, k_pre, pos, w_q, w_k, n_q, n_kv,
                                                head_dim, kind, eps, rope_base, nope)
        return dpacked.view(shape), None, dw_q, dw_k, None, None, None, None, None, None, None


class GQAttentionPrologue(torch.autograd.Function):
    """The GQAttention variant region (Llama 3, Qwen3, GPT-OSS): packed [T, row]
    -> (q, k, v) with the norm optional, an optional qkv bias and a caller's
    RoPE frequency table / cos-sin factor; the backward writes d(packed) in one
    pass and returns the norm-weight and bias gradients where they exist.

    apply(packed, pos, w_q, w_k, bias, n_q, n_kv, head_dim, kind, eps, rope_base,
          nope, norm, inv_freq, rope_scale); w_q / w_k / bias may be None.
    """

    @staticmethod
    def forward(ctx, packed, pos, w_q, w_k, bias, n_q, n_kv, head_dim, kind, eps, rope_base, nope, norm,
                inv_freq, rope_scale):
        out = prologue_forward(packed, pos, w_q, w_k, n_q, n_kv, head_dim, kind, eps, rope_base, nope,
                               save_pre=norm, norm=norm, bias=bias, inv_freq=inv_freq, rope_scale=rope_scale)
        q, k, v = out[:3]
        q_pre, k_pre = (out[3], out[4]) if norm else (None, None)
        ctx.save_for_backward(q_pre, k_pre, pos, w_q, w_k, bias)
        ctx.cfg = (n_q, n_kv, head_dim, kind, eps, rope_base, nope, norm, inv_freq, rope_scale, packed.shape)
        return q, k, v

    @staticmethod
    def backward(ctx, dq, dk, dv):
        q_pre, k_pre, pos, w_q, w_k, bias = ctx.saved_tensors
        n_q, n_kv, head_dim, kind, eps, rope_base, nope, norm, inv_freq, rope_scale, shape = ctx.cfg
        dq, dk, dv = (g.contiguous() for g in (dq, dk, dv))
        out = prologue_backward(dq, dk, dv, q_pre, k_pre, pos, w_q, w_k, n_q, n_kv, head_dim, kind, eps, rope_base,
                                nope, norm=norm, bias=bias, inv_freq=inv_freq, rope_scale=rope_scale)
        dbias = out[3] if bias is not None else None
        return (out[0].view(shape), None, out[1], out[2], dbias) + (None,) * 10
