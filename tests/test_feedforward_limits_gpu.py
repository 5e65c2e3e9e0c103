"""What feed-forward results are where 16 bits or fp32 do not hold what lies between (needs a GB300)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

b2b = pytest.importorskip("fusion_b2b_gemm_gb300")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_feedforward_gpu import E4M3, kernels, normal  # noqa: E402


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.mark.parametrize("t", [5, 300])
def test_fp16_hidden_values_out_of_range_stay_in_their_rows(t):
    """A gate and an up value of 255 (h 65025, below 65504) and of 256 (65536, an infinity), exact in fp32: sums of one term."""
    d = f = o = 64
    x = normal(1, t, d, dtype="f16")
    eye = torch.eye(64, dtype=torch.float16, device="cuda")
    plan = b2b.GatedFeedForwardPlan("f16", d, f, o)
    want = plan.run(x, eye, eye, eye)
    x[1, 7], x[3, 9] = 255, 256
    y = plan.run(x, eye, eye, eye)
    assert plan.status() == 0
    rows = torch.ones(t, dtype=torch.bool, device="cuda")
    rows[[1, 3]] = False
    assert torch.equal(y[rows], want[rows])
    # 65025 lies between fp16's 65024 and 65056; its row's other columns are as before (0 times a finite value)
    assert y[1, 7] == 65024 and y[1].isfinite().all()
    assert y[3, 9].isinf() and y[3, torch.arange(64, device="cuda") != 9].isnan().all()  # (0 times an infinity)


@pytest.mark.parametrize("rows", [5, 300])
def test_scales_are_multiplied_first(rows):
    k, n = 256, 136
    a, b = torch.ones(rows, k, device="cuda").to(E4M3), torch.ones(n, k, device="cuda").to(E4M3)
    a[0] = 0
    sa, sb = torch.ones(rows, 2, device="cuda"), torch.ones(2, 2, device="cuda")
    plan = b2b.ScaledGemmPlan("bf16", k, n)
    # the product is 1, where 2^125 times a sum of 128 is more than fp32 holds
    sa[:, 0], sb[:, 0], sa[:, 1], sb[:, 1] = 2.0 ** 125, 2.0 ** -125, 2.0 ** -120, 2.0 ** 120
    out = plan.run(a, sa, b, sb)
    assert (out[1:] == 256).all() and (out[0] == 0).all()
    sb[:, 0] = 2.0 ** 10  # 2^135: not a number that fp32 has
    out = plan.run(a, sa, b, sb)
    assert out[1:].isinf().all() and out[0].isnan().all()
    sa[:, 0], sb[:, 0] = 2.0 ** -100, 2.0 ** -100  # 2^-200: 0 in fp32
    assert (plan.run(a, sa, b, sb)[1:] == 128).all()
    assert plan.status() == 0
