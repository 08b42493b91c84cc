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


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("how", ["given", "current"])
def test_adamw_keeps_its_buffers_for_the_streams_of_its_steps(cuda, bits, how, monkeypatch):
    """A handle that goes away after a step takes nothing with it that the step still needs: all that the kernel
    addresses is marked as used on the step's stream, once."""
    params = [torch.ones(700, device="cuda"), torch.ones(30, 10, device="cuda")]
    copies = [None, torch.ones(30, 10, dtype=torch.bfloat16, device="cuda")]
    grads = [torch.ones_like(p) for p in params]
    opt = e3.AdamW.create(params, state_bits=bits, copies=copies)
    torch.cuda.synchronize()
    marked, real = [], torch.Tensor.record_stream
    monkeypatch.setattr(torch.Tensor, "record_stream",
                        lambda t, s: (marked.append((t.data_ptr(), s.cuda_stream)), real(t, s))[1])
    s = torch.cuda.Stream()

    def step(t):
        if how == "given":
            return e3.adamw_step(opt, grads, lr=1e-2, step=t, max_norm=1.0, stream=s)
        with torch.cuda.stream(s):
            return e3.adamw_step(opt, grads, lr=1e-2, step=t, max_norm=1.0)

    step(1)
    held = [opt.plan, opt.workspace, opt.m, opt.v, opt.m_scale, opt.v_scale, *params, copies[1]]
    for t in held:
        if t is not None:
            assert (t.data_ptr(), s.cuda_stream) in marked
    marked.clear()
    step(2)
    assert all(where != s.cuda_stream for _, where in marked)
    torch.cuda.synchronize()


def test_adamw_moments_are_ready_for_any_stream(cuda):
    """create() returns when the moments it made are zero: a first step on another stream need not wait."""
    big = torch.zeros(1 << 28, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    opt = e3.AdamW.create([big])
    assert torch.cuda.current_stream().query()
    del opt
