"""Irreps norm: bf16 features of more nodes than the thread blocks take at a time, results that begin anywhere
in memory, and infinities.

Tolerances: those of test_gpu_norm.py.
"""
import pytest
import torch

import message_passing_gb300 as e3
import oracle
from test_gpu_norm import B, BLOCKS, F, _check_norm, _ir_case, _normal

pytestmark = pytest.mark.gpu
GUARD = 7.0


@pytest.mark.parametrize("types", [(B, B, B, B), (B, F, F, F), (F, B, B, B)])
@pytest.mark.parametrize("N,blocks,mul", [(250_001, "svdf", 8), (100_003, "svd", 16), (120_001, "sv", 32), (60_007, "sv", 64),
                                          (40_009, "sv", 128), (123_457, "sv", 7), (90_001, "svd", 4), (30_011, "svd", 50)])
def test_irreps_norm_of_many_nodes_in_bf16(cuda, types, N, blocks, mul):
    """The next node's prefetch, pairs of nodes and tiles after the first, with the parameters' gradients."""
    _ir_case(BLOCKS[blocks], N, mul, *types, seed=mul)


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("mul", [7, 8, 50, 128, 200, 260])
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_irreps_norm_results_that_begin_anywhere(cuda, t, mul, offset):
    blocks, N = BLOCKS["svd"], 60
    n = N * 9 * mul
    x, dy = _normal(N, 9, mul, seed=1, dtype=t), _normal(N, 9, mul, seed=2, dtype=t)
    yw, dxw = (torch.full((n + offset + 16,), GUARD, dtype=t, device="cuda") for _ in range(2))
    y, dx = (w[offset:offset + n].view(N, 9, mul) for w in (yw, dxw))
    _, stats = e3.irreps_norm_forward(blocks, x, out=y)
    e3.irreps_norm_backward(blocks, x, None, stats, dy, out=dx)
    for w in (yw, dxw):
        assert torch.all(w[:offset] == GUARD) and torch.all(w[offset + n:] == GUARD)
    for i, (lo, hi, scalar) in enumerate(oracle.norm.spans(blocks)):
        seg = lambda a: a[:, lo:hi].reshape(N, -1)  # noqa: E731
        _check_norm(f"block {i}", seg(x), None, None, seg(y), stats[:, i], seg(dy), seg(dx), scalar)


@pytest.mark.parametrize("mul", [7, 8, 16, 50, 128, 300])
def test_irreps_norm_of_infinities(cuda, mul):
    """A block with a mean turns to NaN. One without has s = 0: NaN in the entry, zeros beside it, and NaN in all
    of the block's dx. Other blocks and nodes are as they were."""
    blocks, N = BLOCKS["svd"], 40
    x, dy = _normal(N, 9, mul, seed=1), _normal(N, 9, mul, seed=2)
    y0, stats0 = e3.irreps_norm_forward(blocks, x)
    dx0, _, _ = e3.irreps_norm_backward(blocks, x, None, stats0, dy)
    bad = x.clone()
    bad[3, 0, 2], bad[11, 2, 1], bad[20, 8, mul - 1] = float("inf"), -float("inf"), float("inf")
    y, stats = e3.irreps_norm_forward(blocks, bad)
    dx, _, _ = e3.irreps_norm_backward(blocks, bad, None, stats, dy)
    assert torch.isnan(y[3, 0]).all() and torch.isnan(dx[3, 0]).all()
    for n, rows, row, q in ((11, slice(1, 4), 2, 1), (20, slice(4, 9), 8, mul - 1)):
        assert float(stats[n, 1 if n == 11 else 2, 1]) == 0
        assert torch.isnan(y[n, row, q]) and int((y[n, rows] != 0).sum()) == 1      # NaN != 0
        assert torch.isnan(dx[n, rows]).all()
    for got, want in ((y, y0), (dx, dx0)):
        got[3, 0], got[11, 1:4], got[20, 4:9] = want[3, 0], want[11, 1:4], want[20, 4:9]
        assert torch.equal(got, want)
