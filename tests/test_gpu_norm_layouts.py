"""Layer norm rows whose inputs and outputs begin anywhere in memory, and what lies beside the outputs.

Tolerances: those of test_gpu_norm.py.
"""
import pytest
import torch

import message_passing_gb300 as e3
from test_gpu_norm import B, F, _check_norm, _check_params, _normal, to_np

pytestmark = pytest.mark.gpu
GUARD = 7.0


def _rows(n_rows, cols, stride, offset, dtype, values=None):
    """(the whole buffer, its rows): rows `stride` apart that begin `offset` entries into it, GUARD elsewhere."""
    whole = torch.full((offset + n_rows * stride + 16,), GUARD, dtype=dtype, device="cuda")
    rows = whole[offset:offset + n_rows * stride].view(n_rows, stride)[:, :cols]
    if values is not None:
        rows.copy_(values)
    return whole, rows


def _guards_stay(whole, rows, offset, stride):
    R, C = rows.shape
    keep = torch.ones_like(whole, dtype=torch.bool)
    keep[offset:offset + R * stride].view(R, stride)[:, :C] = False
    assert torch.all(whole[keep] == GUARD)


def _case(R, C, dtype, offsets, strides, seed):
    """offsets, strides: of x, y, dy, dx."""
    values = _normal(R, C, seed=seed, dtype=dtype, scale=1.3, shift=0.4), _normal(R, C, seed=seed + 1, dtype=dtype)
    (_, x), (yw, y), (_, dy), (dxw, dx) = (
        _rows(R, C, s, o, dtype, v) for s, o, v in zip(strides, offsets, (values[0], None, values[1], None)))
    w, b = _normal(C, seed=seed + 2, scale=0.3, shift=1.0), _normal(C, seed=seed + 3)
    _, stats = e3.layer_norm_forward(x, w, b, out=y)
    _, dw, db = e3.layer_norm_backward(x, w, stats, dy, out=dx)
    _guards_stay(yw, y, offsets[1], strides[1])
    _guards_stay(dxw, dx, offsets[3], strides[3])
    t, absolute = _check_norm("layer norm", x, w, b, y, stats, dy, dx, True)
    _check_params("dweight", dw, t.sum(0), absolute.sum(0), R)
    _check_params("dbias", db, to_np(dy).sum(0), abs(to_np(dy)).sum(0), R)


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("offset", [1, 2, 3, 5, 7])
@pytest.mark.parametrize("R,C,stride", [(1, 5, 5), (1, 321, 321), (1, 9001, 9001), (37, 13, 13), (64, 64, 64), (37, 321, 321),
                                        (300, 700, 703), (333, 2001, 2001), (333, 5001, 5003), (200, 9001, 9001)])
def test_layer_norm_rows_that_begin_inside_a_vector(cuda, t, offset, R, C, stride):
    """All four tensors begin equally far into a vector, the first of a buffer too."""
    _case(R, C, t, [offset] * 4, [stride] * 4, seed=C + offset)


@pytest.mark.parametrize("t", [F, B])
@pytest.mark.parametrize("offsets,gaps", [((0, 1, 0, 2), (0, 0, 0, 0)), ((3, 0, 1, 0), (1, 2, 0, 3)), ((1, 1, 1, 1), (1, 1, 1, 2)),
                                          ((0, 0, 0, 0), (5, 5, 5, 5)), ((2, 2, 2, 2), (3, 3, 7, 3)), ((0, 8, 0, 8), (8, 8, 0, 16))])
@pytest.mark.parametrize("R,C", [(37, 5), (65, 64), (300, 77), (64, 128), (37, 130), (65, 700), (33, 2050), (330, 5001), (20, 9002)])
def test_layer_norm_writes_only_its_rows_at_any_alignment(cuda, t, offsets, gaps, R, C):
    """Tensors that lie over one another in vectors, or not: entries between and beside the rows keep their values."""
    _case(R, C, t, offsets, [C + g for g in gaps], seed=C)
