"""AdamW with clipping where gradients begin anywhere in memory.

Tolerances: those of test_gpu_adamw.py.
"""
import numpy as np
import pytest
import torch

import message_passing_gb300 as e3
import oracle
from gpu_util import to_np
from test_gpu_adamw import SIZES, U, _check32, _grads, _model

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("gt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("offset", [1, 2, 3])
@pytest.mark.parametrize("max_norm", [0.37, 1e4])
def test_adamw_clips_unaligned_gradients(cuda, gt, bits, offset, max_norm):
    params = _model(SIZES)
    opt = e3.AdamW.create(params, state_bits=bits)
    grads = _grads(SIZES, 3, gt, offset)
    grads[7] = None
    want = np.sqrt(sum((to_np(g) ** 2).sum() for g in grads if g is not None))
    before = [to_np(p) for p in params]
    norm = e3.adamw_step(opt, grads, lr=1e-2, step=1, max_norm=max_norm)
    assert abs(float(norm) - want) <= 32 * U * want and np.array_equal(to_np(params[7]), before[7])
    for i, n in enumerate(SIZES):
        if grads[i] is None:
            continue
        kw = dict(lr=1e-2, t=1, decay=float(np.float32(0.01)), clip=min(1.0, max_norm / want))
        if bits == 32:
            _check32(opt, i, before[i], grads[i], np.zeros(n), np.zeros(n), clip_err=32 * U, **kw)
        else:
            p, _, _ = oracle.adamw.step(before[i], to_np(grads[i]), np.zeros(n), np.zeros(n), **kw)
            assert np.all(np.abs(to_np(params[i]) - p) <= 2 * U * np.abs(before[i]) + 80 * U * 1e-2)
