"""The norm and AdamW calls take tensors of one device only: the kernels get bare addresses."""
import os
from types import SimpleNamespace

import pytest
import torch

import message_passing_gb300 as e3


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(e3.LIB_PATH):
        from message_passing_gb300 import build
        build.build()
    return e3.load()


class _Elsewhere(torch.Tensor):
    """A host tensor that says that it lies on device 1."""

    def get_device(self):
        return 1


def away(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(_Elsewhere)


X, S, W = torch.zeros(5, 8), torch.zeros(5, 2), torch.zeros(8)
G, GS, IR = torch.zeros(5, 4, 8), torch.zeros(5, 2, 2), [(0, 1), (1, -1)]
LN, LNB, IN, INB = e3.layer_norm_forward, e3.layer_norm_backward, e3.irreps_norm_forward, e3.irreps_norm_backward


@pytest.mark.parametrize("call,match", [
    (lambda: LN(X, away(8)), "weight"),
    (lambda: LN(X, None, away(8)), "bias"),
    (lambda: LN(X, out=away(5, 8)), "y"),
    (lambda: LN(away(5, 8), W), "weight"),
    (lambda: LNB(X, away(8), S, X), "weight"),
    (lambda: LNB(X, None, away(5, 2), X), "stats"),
    (lambda: LNB(X, None, S, away(5, 8)), "dy"),
    (lambda: LNB(X, None, S, X, out=away(5, 8)), "dx"),
    (lambda: LNB(X, None, S, X, workspace=away(100_000)), "workspace"),
    (lambda: IN(IR, G, away(2, 8)), "weight"),
    (lambda: IN(IR, G, None, away(1, 8)), "bias"),
    (lambda: IN(IR, G, out=away(5, 4, 8)), "y"),
    (lambda: INB(IR, G, None, away(5, 2, 2), G), "stats"),
    (lambda: INB(IR, G, None, GS, away(5, 4, 8)), "dy"),
    (lambda: INB(IR, G, None, GS, G, out=away(5, 4, 8)), "dx"),
    (lambda: INB(IR, G, None, GS, G, workspace=away(100_000)), "workspace"),
    (lambda: e3.AdamW.create([W, away(8)]), "params"),
    (lambda: e3.AdamW.create([W], copies=[away(8, dtype=torch.bfloat16)]), "copies"),
    (lambda: e3.AdamW.create([W], state=(torch.zeros(256), away(256))), "v"),
])
def test_operands_of_another_device(call, match):
    with pytest.raises(ValueError, match=f"{match}.* is on .*expected all tensors"):
        call()


@pytest.mark.parametrize("call", [lambda ws: LNB(X, None, S, X, workspace=ws),
                                  lambda ws: INB(IR, G, None, GS, G, workspace=ws)])
def test_a_workspace_with_gaps(call):
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        call(torch.zeros(200_000)[::2])


def test_the_device_has_to_be_the_current_one(monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 100 + index, raising=False)
    device = lambda i: SimpleNamespace(type="cuda", index=i)  # noqa: E731
    assert e3._current(device(0)) == 100
    with pytest.raises(ValueError, match="current device is cuda:0"):
        e3._current(device(1))
    with pytest.raises(ValueError, match="expected device memory"):
        e3._current(torch.device("cpu"))


BUF = torch.zeros(1024)


@pytest.mark.parametrize("params,kw,names", [
    ([W, X, W], {}, "params.0. and params.2."),
    ([BUF[:100], BUF[200:300], BUF[99:120]], {}, "params.0. and params.2."),
    ([BUF[300:500], BUF[200:301]], {}, "params.1. and params.0."),
    ([W], dict(state=(BUF[:256], BUF[:256])), "m and v"),
    ([BUF[:8]], dict(state=(BUF[:256], torch.zeros(256))), "m|params"),
    ([torch.zeros(4), torch.zeros(4)], dict(copies=[torch.zeros(8, dtype=torch.bfloat16)[:4]] * 2), "copies.0. and copies.1."),
    ([BUF[:8]], dict(copies=[BUF.view(torch.bfloat16)[14:22]]), "params.0. and copies.0."),
])
def test_tensors_that_share_memory(params, kw, names):
    with pytest.raises(ValueError, match=f"({names}).* share memory"):
        e3.AdamW.create(params, **kw)


def test_neighbours_in_one_buffer_do_not_share_memory():
    """Nor do tensors without entries; these are then refused as host memory only."""
    with pytest.raises(e3.E3GBError, match="not device memory|cannot query"):
        e3.AdamW.create([BUF[100:200], BUF[:100], BUF[200:], BUF[5:5], BUF[5:5]])
