"""The norms' backward where a row's mean is large against its deviation, for the statistics it is given.

For given mu and s (fp32, taken as exact) the difference x - mu and its product with s are one rounding each,
so xh carries 2 u of itself (u = 2^-24), whatever mu is. With d = K/32 + 8, how deep a sum over K entries runs,
mean g is off by u (d + 1) max|g|, mean(g xh) by u (d + 4) max|g| (mean|xh| <= 1), and the three terms of
dx = s (g - mean g - xh mean(g xh)) by at most u s max|g| ((d + 4) + (d + 9) max|xh|).
dweight: every term dy xh is off by 2 u, and the sum of n terms by (16 + 2 sqrt(n)) u of the absolute sum.
"""
import numpy as np
import pytest
import torch

import message_passing_gb300 as e3
from gpu_util import to_np
from test_gpu_norm import B, F, U, _normal

pytestmark = pytest.mark.gpu


def _check(x, stats, w, dy, dx, dw):
    """Rows x, dy, dx [R, K], stats [R, 2], w and dw [K]."""
    x, stats, w, dy, dx, dw = (to_np(t) for t in (x, stats, w, dy, dx, dw))
    R, K = x.shape
    mu, s = stats[:, :1], stats[:, 1:]
    xh, g = (x - mu) * s, dy * w
    want = s * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    d, top, gt = K / 32 + 8, np.abs(xh).max(1, keepdims=True), np.abs(g).max(1, keepdims=True)
    assert np.all(np.abs(dx - want) <= U * s * gt * ((d + 4) + (d + 9) * top))
    assert np.all(np.abs(dw - (dy * xh).sum(0)) <= (18 + 2 * np.sqrt(R)) * U * np.abs(dy * xh).sum(0))


@pytest.mark.parametrize("mean", [1e3, 3e4])
@pytest.mark.parametrize("dyt", [F, B])
@pytest.mark.parametrize("C,stride", [(8, 8), (64, 64), (77, 77), (77, 79), (512, 512), (700, 701), (1280, 1280), (5001, 5001),
                                      (9000, 9000)])
def test_layer_norm_backward_of_a_large_mean(cuda, mean, dyt, C, stride):
    R = 64
    x = _normal(R, stride, seed=C, shift=mean)[:, :C]
    w, dy = _normal(C, seed=C + 1, scale=0.3, shift=1.0), _normal(R, C, seed=C + 2, shift=1.0, dtype=dyt)
    dy = dy + x.sub(mean).to(dyt)                       # both means of the formula are about one
    _, stats = e3.layer_norm_forward(x, w)
    dx, dw, _ = e3.layer_norm_backward(x, w, stats, dy)
    _check(x, stats, w, dy, dx, dw)


@pytest.mark.parametrize("mean", [1e3, 3e4])
@pytest.mark.parametrize("mul", [7, 8, 16, 50, 128, 200, 300])
def test_irreps_norm_backward_of_a_large_mean(cuda, mean, mul):
    blocks, N = [(0, 1), (1, -1), (2, 1)], 64
    x = _normal(N, 9, mul, seed=mul)
    x[:, 0] += mean
    w, dy = _normal(3, mul, seed=mul + 1, scale=0.3, shift=1.0), _normal(N, 9, mul, seed=mul + 2, shift=1.0)
    dy[:, 0] += x[:, 0] - mean
    _, stats = e3.irreps_norm_forward(blocks, x, w)
    dx, dw, _ = e3.irreps_norm_backward(blocks, x, w, stats, dy)
    _check(x[:, 0], stats[:, 0], w[0], dy[:, 0], dx[:, 0], dw[0])
