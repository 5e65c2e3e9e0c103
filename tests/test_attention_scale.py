"""Scales of the scores that 32 bits do not hold are refused (no GPU needed: before a device is looked for)."""
import ctypes
import math

import pytest

import fusion_b2b_gemm_gb300 as b2b


@pytest.mark.parametrize("kind", ["PromptAttentionPlan", "SharedPrefixAttentionPlan"])
@pytest.mark.parametrize("scale", [0.0, -1.0, math.nan, math.inf, 1e-60, 1e39, 3e38], ids=str)
def test_plans_refuse_scales_that_fp32_cannot_hold(kind, scale):
    """1e-60 is 0 in 32 bits, which would mean the default; 3e38 log2(e) is infinite."""
    pytest.importorskip("torch")
    with pytest.raises(ValueError, match="scale"):
        getattr(b2b, kind)("f16", 4, 2, 64, scale)


@pytest.mark.parametrize("scale", [3e38, 2.4e38])
def test_the_c_function_refuses_scales_infinite_times_log2e(scale):
    h = ctypes.c_void_p()
    assert b2b.b2b_attn_plan_create(ctypes.byref(h), 1, 4, 2, 64, scale) == 1
