"""Rates of an AdamW step that fp32 cannot hold are refused, on the host and before any launch."""
import ctypes
import os

import pytest

import message_passing_gb300 as e3


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(e3.LIB_PATH):
        from message_passing_gb300 import build
        build.build()
    return e3.load()


@pytest.mark.parametrize("lr,beta1,word", [(1e300, 0.9, b"lr"), (-1e39, 0.9, b"lr"), (1e30, 1 - 1e-12, b"lr"),
                                           (1e30, 0.9, b"plan"), (1e-3, 1 - 1e-12, b"plan")])
def test_learning_rates_that_fp32_does_not_hold(lib, lr, beta1, word):
    """The last two are accepted: what is refused then is the plan that is missing."""
    h = ctypes.c_void_p()
    n, p, d = (ctypes.c_int64 * 1)(0), (ctypes.c_void_p * 1)(None), (ctypes.c_float * 1)(0.0)
    assert lib.e3gb_adamw_create(1, n, p, None, d, 32, ctypes.byref(h)) == e3.OK
    r, g = e3._AdamwRates(lr, beta1, 0.999, 1e-8, 0.0, 1, 0), (ctypes.c_void_p * 1)(None)
    st = lib.e3gb_adamw_step(h, None, g, 0, None, None, None, None, ctypes.byref(r), None, None, 0, None)
    assert st == e3.ERR_INVALID_ARG and word in lib.e3gb_last_error()
    lib.e3gb_adamw_destroy(h)
