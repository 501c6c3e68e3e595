"""Refusals of moe_linear_plan on the host (no GPU)."""

import ctypes
import os

import pytest

import routed_expert_ffn_gb300 as moe


@pytest.fixture(scope="module", autouse=True)
def built():
    if not os.path.exists(moe.LIB_PATH):
        from routed_expert_ffn_gb300 import build
        build.build()


def test_refusals():
    f, plan = moe.library().moe_linear_plan, moe.LinearPlan()
    d = moe.linear_desc(4, 256, 512, moe.MOE_DTYPE_BF16)
    none = moe.linear_desc(0, 256, 512, moe.MOE_DTYPE_BF16)
    odd = moe.linear_desc(4, 252, 512, moe.MOE_DTYPE_BF16)
    assert f(None, 0, ctypes.byref(plan)) == moe.MOE_ERR_INVALID_ARG
    assert f(ctypes.byref(d), 0, None) == moe.MOE_ERR_INVALID_ARG
    assert f(ctypes.byref(none), 0, ctypes.byref(plan)) == moe.MOE_ERR_INVALID_ARG
    assert f(ctypes.byref(odd), 0, ctypes.byref(plan)) == moe.MOE_ERR_UNSUPPORTED_SHAPE
