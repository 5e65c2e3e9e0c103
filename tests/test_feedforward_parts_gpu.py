"""Feed-forward launches whose tiles are cut along k, with the kernel that joins the parts, and plans whose flags change between
runs (needs a GB300).  Tolerances as in test_feedforward_gpu.py."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

b2b = pytest.importorskip("fusion_b2b_gemm_gb300")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_feedforward_gpu import normal, scaled, weights  # noqa: E402

PAIR = 2  # B2B_DEBUG_PAIR_KERNEL


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


# ------------------------------------------------------------------- flags
@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("first", [0, PAIR])
def test_flags_that_change_after_a_run(first, compiled):
    """Workspaces have other sizes with the other kernel: 16 tokens on 4096 / 512 are cut along k in one of them only."""
    t, d, f, o = 16, 4096, 512, 256
    x, dy, w = normal(1, t, d), normal(2, t, o), weights(3, "bf16", d, f, o)
    (a, sa), (b, sb) = scaled(1, t, d, 1), scaled(2, o, d, 128)

    def plans(flags):
        ffn, product = b2b.GatedFeedForwardPlan("bf16", d, f, o), b2b.ScaledGemmPlan("bf16", d, o)
        for p in (ffn, product):
            p.set_debug(flags)
        return ffn, product

    def calls(ffn, product):
        if not compiled:
            ffn._bound = product._bound = None
        y, kept = ffn.forward(x, *w)
        out = torch.empty_like(y)
        return [ffn.run(x, *w), ffn.run(x, *w, out=out), y, *ffn.backward(dy, x, *w, kept), product.run(a, sa, b, sb)]

    def size(p):
        return p._workspace(x, t)[2]

    fresh = {flags: plans(flags) for flags in (0, PAIR)}
    assert size(fresh[0][0]) != size(fresh[PAIR][0]) and size(fresh[0][1]) != size(fresh[PAIR][1])
    want = {flags: calls(*p) for flags, p in fresh.items()}
    ffn, product = plans(first)
    for flags in (first, PAIR - first, first):
        for p in (ffn, product):
            p.set_debug(flags)
            assert not p._workspace_sizes
        assert all(torch.equal(x, y) for x, y in zip(calls(ffn, product), want[flags]))
    assert ffn.status() == 0 and product.status() == 0
