"""The norm and AdamW calls on a given stream: what they allocate, and what they leave for later."""
import pytest
import torch

import message_passing_gb300 as e3

pytestmark = pytest.mark.gpu
BLOCKS, N = [(0, 1), (1, -1)], 4096


def _calls():
    """name: (shape of the first result, a call on a given stream)"""
    x, r = torch.randn(N, 4, 64, device="cuda"), torch.randn(N, 256, device="cuda")
    _, xs = e3.irreps_norm_forward(BLOCKS, x)
    _, rs = e3.layer_norm_forward(r)
    return {"ln fwd": ((N, 256), lambda s: e3.layer_norm_forward(r, stream=s)),
            "ln bwd": ((N, 256), lambda s: e3.layer_norm_backward(r, None, rs, r, stream=s)),
            "ir fwd": ((N, 4, 64), lambda s: e3.irreps_norm_forward(BLOCKS, x, stream=s)),
            "ir bwd": ((N, 4, 64), lambda s: e3.irreps_norm_backward(BLOCKS, x, None, xs, x, stream=s))}


@pytest.mark.parametrize("name", ["ln fwd", "ln bwd", "ir fwd", "ir bwd"])
def test_results_do_not_lie_in_memory_that_the_callers_stream_still_reads(cuda, name):
    """A tensor dropped with work on it still queued gives its memory to the next allocation of the same stream;
    a call on another stream, which does not wait for that work, must not get it."""
    shape, call = _calls()[name]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    want = [t.clone() for t in call(s)]
    torch.cuda.synchronize()
    late, first = torch.empty(shape, device="cuda"), torch.full(shape, 7.0, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                      # about a tenth of a second
    late.copy_(first)
    del first
    got = call(s)
    torch.cuda.synchronize()
    assert torch.all(late == 7.0)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
