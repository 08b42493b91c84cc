"""AdamW's update of the parameters where single roundings decide: tiny gradients, small weight decay.

u = 2^-24. The update lr m / (1 - beta1^t) / (sqrt(v / (1 - beta2^t)) + eps), from moments rounded to fp32, takes
a root and a reciprocal within 2 u each and at most eight further roundings: 12 u of it.
"""
import numpy as np
import pytest
import torch

import message_passing_gb300 as e3
import oracle
from gpu_util import to_np
from test_gpu_adamw import U, _normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("eps", [1e-8, 1e-18, 1e-20, 1e-30])
def test_adamw_of_tiny_gradients(cuda, bits, offset, eps):
    """The second moment of gradients below 1e-17 is a subnormal number, and still what the step is divided by."""
    g = torch.logspace(-19, -15, 3000, device="cuda") * torch.sign(_normal(3000, 4))
    g = torch.cat([g.new_zeros(offset), g])[offset:]
    p = _normal(3000, 5, offset=offset)
    opt = e3.AdamW.create([p], weight_decay=0.0, state_bits=bits)
    before, zero = to_np(p), np.zeros(3000)
    e3.adamw_step(opt, [g], lr=1e-2, step=1, eps=eps)
    want, m, v = oracle.adamw.step(before, to_np(g), zero, zero, lr=1e-2, t=1, eps=eps, dtype=np.float32)
    assert np.all(v > 0) and np.any(v < 1e-38)
    size = 1e-2 * np.abs(m) / 0.1 / (np.sqrt(v.astype(np.float64) / 0.001) + eps)
    assert np.all(np.abs(to_np(p) - want) <= U * np.abs(want) + 12 * U * size)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("lr,decay", [(1e-5, 0.01), (1e-6, 0.02), (1e-3, 0.1), (0.5, 1.0), (1.0, 1.0)])
def test_adamw_decays_by_little(cuda, bits, lr, decay):
    """p (1 - lr wd) - update is rounded once, half a unit of the result, whatever lr wd is: the factor is held in
    48 bits, lr and wd in 24 each, and the parts below fp32's are added to the update first."""
    n = 20_000
    p, g = _normal(n, 5), _normal(n, 6)
    opt = e3.AdamW.create([p], weight_decay=decay, state_bits=bits)
    before, zero, wd = to_np(p), np.zeros(n), float(np.float32(decay))
    e3.adamw_step(opt, [g], lr=lr, step=1)
    want, _, _ = oracle.adamw.step(before, to_np(g), zero, zero, lr=lr, t=1, decay=wd)
    bound = U * np.abs(want) * (1 + 1e-6) + 16 * U * lr + 4 * U * lr * wd * np.abs(before)
    assert np.all(np.abs(to_np(p) - want) <= bound)


def test_adamw_clips_by_less_than_fp32_holds(cuda):
    """A max_norm of 1e-60 is one all the same: the norm comes back, and the gradients are scaled to nothing."""
    p = _normal(5000, 5)
    before, g = p.clone(), _normal(5000, 6)
    opt = e3.AdamW.create([p], weight_decay=0.0)
    norm = e3.adamw_step(opt, [g], lr=1e-2, step=1, max_norm=1e-60)
    want = np.sqrt((to_np(g) ** 2).sum())
    assert abs(float(norm) - want) <= 32 * U * want
    assert torch.equal(p, before) and float(opt.m.abs().max()) < 1e-44
