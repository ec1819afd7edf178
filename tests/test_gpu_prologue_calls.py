"""What the prologue's calls accept and refuse, with and without tokens."""

import pytest
import torch

import workloads

pytestmark = pytest.mark.gpu


def test_frequencies_that_can_be_taken_once(lib, cuda):
    """An iterator of frequencies, and texts: forward and backward have the list's results."""
    n_q, n_kv, D, T = 4, 2, 64, 9
    wl = workloads.gqa_inputs(T, n_q, n_kv, D, seed=2, rope_base=1e4, with_grads=True)
    freq = [1e4 ** (-2 * i / 32) for i in range(16)]

    def step(inv_freq):
        x = wl.packed_rows().to(cuda).requires_grad_()
        out = lib.functional.GQAttentionPrologue.apply(x, wl.pos.to(cuda), None, None, None, n_q, n_kv, D, "interleaved",
                                                       wl.eps, wl.rope_base, False, False, inv_freq, 1.0, 32, True)
        torch.autograd.backward(out, [t.to(cuda) for t in (wl.dq, wl.dk, wl.dv)])
        return [*out, x.grad]

    want = step(freq)
    for other in (iter(freq), (f for f in freq), [repr(f) for f in freq], torch.tensor(freq, dtype=torch.float64)):
        assert all(torch.equal(a, b) for a, b in zip(step(other), want))


def _calls(lib, cuda, T):
    """Forward, backward, pool write and 8-bit write of T tokens, each as f(**options)."""
    F, n_q, n_kv, D = lib.functional, 4, 2, 64
    wl = workloads.gqa_inputs(max(T, 1), n_q, n_kv, D, seed=1, rope_base=1e4, with_grads=True)
    cut = lambda t: t[:T].to(cuda)  # noqa: E731
    w = (wl.w_q.to(cuda), wl.w_k.to(cuda))
    rows, pos = cut(wl.packed_rows()), cut(wl.pos)
    heads = (n_q, n_kv, D)
    slot = torch.zeros(T, dtype=torch.int32, device=cuda)
    pools = [torch.zeros(1, 16, n_kv, D, dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    codes = [torch.zeros(1, 16, n_kv, D, dtype=torch.float8_e4m3fn, device=cuda) for _ in range(2)]
    scales = [torch.ones(1, 2, n_kv, device=cuda) for _ in range(2)]
    pre = (cut(wl.dq), cut(wl.dk))
    return {
        "forward": lambda **o: F.prologue_forward(rows, pos, *w, *heads, **o),
        "backward": lambda **o: F.prologue_backward(cut(wl.dq), cut(wl.dk), cut(wl.dv), *pre, pos, *w, *heads, **o),
        "pool_write": lambda **o: F.prologue_pool_write(rows, pos, *w, slot, slot, *pools, *heads, **o),
        "pool_write8": lambda **o: F.prologue_pool_write8(rows, pos, *w, slot, slot, *codes, *scales, *heads, **o),
    }


@pytest.mark.parametrize("T", [0, 1])
@pytest.mark.parametrize("name", ["forward", "backward", "pool_write", "pool_write8"])
def test_the_same_refusals_with_and_without_tokens(lib, cuda, name, T):
    call = _calls(lib, cuda, T)[name]
    call()
    for bad in (dict(eps=-1.0), dict(rope_base=0.0), dict(rotary_dim=24), dict(rotary_dim=32, nope=True),
                dict(rope_scale=float("inf")), dict(inv_freq=[float("nan")] * 32)):
        with pytest.raises(lib.QkvpError):
            call(**bad)
    with pytest.raises(ValueError):
        call(bias=torch.zeros(8 * 64, dtype=torch.float64, device=cuda))


def test_zero_gradients_come_on_the_given_stream(lib, cuda):
    """The gradients of no tokens are zeros, written in the order of the call's stream: a graph
    that is captured on it has them."""
    call = _calls(lib, cuda, 0)["backward"]
    bias = torch.zeros(8 * 64, device=cuda)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=side, capture_error_mode="relaxed"):
        with torch.cuda.stream(other):
            got = call(stream=side, bias=bias)
    torch.cuda.synchronize()
    assert got[0].shape == (0, 8 * 64)
    for t in got[1:]:
        t.fill_(7.0)
    graph.replay()
    torch.cuda.synchronize()
    assert all(bool((t == 0).all()) for t in got[1:])
