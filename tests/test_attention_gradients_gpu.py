"""Attention and forward-mode differentiation: inputs with a tangent are refused (needs a GB300)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

b2b = pytest.importorskip("fusion_b2b_gemm_gb300")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))

forward_ad = torch.autograd.forward_ad


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def normal(seed, *shape):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").half()


@pytest.mark.parametrize("no_grad", [False, True])
def test_tangents_are_refused(no_grad):
    q, k, v = normal(1, 9, 4, 64), normal(2, 9, 2, 64), normal(3, 9, 2, 64)
    cu, lengths = (torch.tensor(z, dtype=torch.int32, device="cuda") for z in ([0, 9], [1, 2, 3]))
    cache = normal(4, 3, 16, 2, 64)
    prompt, shared = b2b.PromptAttentionPlan("f16", 4, 2, 64), b2b.SharedPrefixAttentionPlan("f16", 4, 2, 64)
    for plan, args, floats in ((prompt, (q, k, v, cu), 3), (shared, (q, k, v, cache, cache.clone(), lengths), 5)):
        want = plan.run(*args)
        with forward_ad.dual_level(), torch.set_grad_enabled(not no_grad):
            for i in range(floats):
                moved = list(args)
                moved[i] = forward_ad.make_dual(args[i], torch.zeros_like(args[i]))
                for kw in ({}, {"out": torch.empty_like(q)}):
                    with pytest.raises(RuntimeError, match="primals"):
                        plan.run(*moved, **kw)
                moved[i] = forward_ad.unpack_dual(moved[i]).primal
                assert torch.equal(plan.run(*moved), want)
        assert plan.status() == 0
