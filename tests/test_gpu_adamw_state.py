"""Moments set on an AdamW handle: what the kernel would read or write past their end is refused."""
import pytest
import torch

import message_passing_gb300 as e3

pytestmark = pytest.mark.gpu


def _opt(bits):
    params = [torch.ones(700, device="cuda"), torch.ones(30, 10, device="cuda")]
    return params, e3.AdamW.create(params, state_bits=bits, seed=3)


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_that_are_set(cuda, bits):
    """A run from restored moments is the run that they came from."""
    grads = [torch.randn(700, device="cuda"), torch.randn(30, 10, device="cuda")]
    a_params, a = _opt(bits)
    b_params, b = _opt(bits)
    e3.adamw_step(a, grads, lr=1e-2, step=1)
    for name in ("m", "v", "m_scale", "v_scale"):
        if getattr(a, name) is not None:
            setattr(b, name, getattr(a, name).clone())
    for x, y in zip(a_params, b_params):
        y.copy_(x)
    for params, opt in ((a_params, a), (b_params, b)):
        e3.adamw_step(opt, grads, lr=1e-2, step=2)
    assert all(torch.equal(x, y) for x, y in zip(a_params, b_params))
    assert torch.equal(a.m.view(torch.uint8), b.m.view(torch.uint8))


@pytest.mark.parametrize("bits", [32, 8])
def test_moments_that_are_refused(cuda, bits):
    params, opt = _opt(bits)
    m, v = opt.m, opt.v
    for name, t, err in (("m", m[:-256].clone(), ValueError), ("v", v[:100].clone(), ValueError), ("m", m.cpu(), ValueError),
                         ("m", torch.zeros(m.numel(), dtype=torch.float16, device="cuda"), TypeError), ("m", v, (TypeError, ValueError)),
                         ("v", torch.zeros(2 * v.numel(), device="cuda")[::2].to(v.dtype).view(2, -1).t(), ValueError)):
        with pytest.raises(err):
            setattr(opt, name, t)
    with pytest.raises(ValueError, match="share memory" if bits == 8 else "have no"):
        opt.m_scale = opt.v_scale if bits == 8 else torch.zeros(5, device="cuda")
    assert opt.m is m and opt.v is v
    e3.adamw_step(opt, [torch.ones_like(p) for p in params], lr=1e-2, step=1)
    assert float(opt.moments(0)[0].min()) > 0
