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
