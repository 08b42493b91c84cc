"""Tensors that a call writes by their addresses: autograd sees that they changed."""
import pytest
import torch

import message_passing_gb300 as e3

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
def test_a_backward_pass_refuses_parameters_that_a_step_changed_meanwhile(cuda, bits):
    w = torch.nn.Parameter(torch.randn(8, 8, device="cuda"))
    other = torch.nn.Parameter(torch.randn(8, 8, device="cuda"))
    copy = torch.zeros(8, 8, dtype=torch.bfloat16, device="cuda")
    opt = e3.AdamW.create([w, other], state_bits=bits, copies=[copy, None])
    x = torch.randn(4, 8, device="cuda", requires_grad=True)
    loss, kept = (x @ w).sum(), (x @ other).sum()
    versions = [t._version for t in (w, copy, other)]
    e3.adamw_step(opt, [torch.ones_like(w), None], lr=1e-2, step=1)
    assert w._version > versions[0] and copy._version > versions[1] and other._version == versions[2]
    kept.backward()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()
    versions = [t._version for t in (w, other)]
    e3.adamw_step(opt, [torch.ones_like(w), torch.ones_like(other)], lr=1e-2, step=2)
    assert w._version > versions[0] and other._version > versions[1]


def test_outputs_that_a_norm_overwrites(cuda):
    x, r = torch.randn(5, 4, 8, device="cuda"), torch.randn(5, 8, device="cuda")
    blocks = [(0, 1), (1, -1)]
    _, xs = e3.irreps_norm_forward(blocks, x)
    _, rs = e3.layer_norm_forward(r)
    for call, shape in ((lambda out: e3.layer_norm_forward(r, out=out), r.shape),
                        (lambda out: e3.layer_norm_backward(r, None, rs, r, out=out), r.shape),
                        (lambda out: e3.irreps_norm_forward(blocks, x, out=out), x.shape),
                        (lambda out: e3.irreps_norm_backward(blocks, x, None, xs, x, out=out), x.shape)):
        out = torch.zeros(shape, device="cuda")
        a = torch.ones(shape, device="cuda", requires_grad=True)
        loss = (a * out).sum()
        call(out)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            loss.backward()


def test_inference_tensors_have_no_version(cuda):
    with torch.inference_mode():
        p = torch.ones(300, device="cuda")
        out = torch.zeros(5, 8, device="cuda")
    opt = e3.AdamW.create([p])
    e3.adamw_step(opt, [torch.ones(300, device="cuda")], lr=1e-2, step=1)
    r = torch.randn(5, 8, device="cuda")
    y, _ = e3.layer_norm_forward(r, out=out)
    assert torch.equal(y, e3.layer_norm_forward(r)[0]) and float(p.max()) < 1.0


def test_parameters_that_are_views_of_one_buffer(cuda):
    """They share the buffer's version counter, also with other views of it."""
    buf = torch.zeros(1000, device="cuda")
    params = [buf[100 * i:100 * i + 60] for i in range(4)] + [torch.nn.Parameter(buf[500:600])]
    opt = e3.AdamW.create(params)
    other, grads = buf[600:], [torch.ones_like(p) for p in params]
    for step in (1, 2):
        before = [t._version for t in (*params, other, buf)]
        e3.adamw_step(opt, grads, lr=1e-2, step=step)
        assert all(t._version > v for t, v in zip((*params, other, buf), before))
