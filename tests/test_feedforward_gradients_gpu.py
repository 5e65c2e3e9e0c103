"""What the feed-forward calls and autograd have to do with each other (needs a GB300)."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

b2b = pytest.importorskip("fusion_b2b_gemm_gb300")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_feedforward_gpu import normal, scaled, weights  # noqa: E402

forward_ad = torch.autograd.forward_ad


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def calls(t=6, d=144, f=272, o=80):
    """Each call by name, with its inputs."""
    block, eight, product = b2b.GatedFeedForwardPlan("bf16", d, f, o), b2b.ScaledFeedForwardPlan("bf16", d, f, o), b2b.ScaledGemmPlan("bf16", d, o)
    x, dy, w = normal(1, t, d), normal(2, t, o), weights(3, "bf16", d, f, o)
    kept = block.forward(x, *w)[1]
    q = [z for m in w for z in b2b.quantize_blocks(m.t().contiguous(), 128)]
    (a, sa), (b, sb) = scaled(1, t, d, 1), scaled(2, o, d, 128)
    return {
        "run": (block.run, (x, *w)),
        "forward": (lambda *z: block.forward(*z)[0], (x, *w)),
        "backward": (lambda *z: block.backward(*z, kept), (dy, x, *w)),
        "scaled": (eight.run, (x, *q)),
        "product": (product.run, (a, sa, b, sb)),
        "quantize": (b2b.quantize_blocks, (x,)),
    }


def flat(done):
    return [done] if isinstance(done, torch.Tensor) else list(done)


@pytest.mark.parametrize("no_grad", [False, True])
def test_tangents_are_refused(no_grad):
    for name, (call, inputs) in calls().items():
        want = flat(call(*inputs))
        with forward_ad.dual_level(), torch.set_grad_enabled(not no_grad):
            for i, z in enumerate(inputs):
                if z.dtype is torch.float8_e4m3fn:
                    continue
                moved = list(inputs)
                moved[i] = forward_ad.make_dual(z, torch.zeros_like(z))
                with pytest.raises(RuntimeError, match="records no gradient"):
                    call(*moved)
                moved[i] = forward_ad.unpack_dual(moved[i]).primal
                assert all(torch.equal(a.float(), b.float()) for a, b in zip(flat(call(*moved)), want)), name


def into(t=6, d=144, f=272, o=80):
    """Each call that writes into tensors it is given, with these: (call, tensors)."""
    (block, (x, *w)), (eight, served), (product, operands) = (calls(t, d, f, o)[k] for k in ("run", "scaled", "product"))
    plan, dy = block.__self__, normal(2, t, o)
    y, kept = plan.forward(x, *w)
    grads = [torch.zeros_like(z, dtype=torch.float32) for z in w]

    def new():
        return torch.zeros(t, o, dtype=torch.bfloat16, device="cuda")

    return {
        "run": (lambda z: block(x, *w, out=z), [new()]),
        "forward": (lambda z: plan.forward(x, *w, out=z), [new()]),
        "kept": (lambda z: plan.forward(x, *w, kept=z), [kept]),
        "backward": (lambda *z: plan.backward(dy, x, *w, kept, weight_grads=z), grads),
        "some": (lambda z: plan.backward(dy, x, *w, kept, weight_grads=(None, z, None)), grads[1:2]),
        "scaled": (lambda z: eight(*served, out=z), [new()]),
        "product": (lambda z: product(*operands, out=z), [new()]),
    }


def test_tensors_to_write_into_that_require_a_gradient_are_refused():
    for name, (call, given) in into().items():
        for i, z in enumerate(given):
            if not z.is_floating_point():
                continue
            leaf = z.clone().requires_grad_()
            some = given[:i] + [leaf] + given[i + 1:]
            with pytest.raises(RuntimeError, match="no_grad"):
                call(*some)
            assert torch.equal(leaf, z), name
            with torch.no_grad():
                call(*some)
            assert not torch.equal(leaf, z), name


def test_tensors_written_into_have_a_new_version():
    """What autograd saved of a tensor before a call wrote into it is not taken for its contents afterwards."""
    for name, (call, given) in into().items():
        before = [z._version for z in given]
        call(*given)
        assert all(z._version > v for z, v in zip(given, before)), name
        if given[0].is_floating_point():
            p = torch.ones_like(given[0], requires_grad=True)
            product = (given[0] * p).sum()
            call(*given)
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                product.backward()
    with torch.inference_mode():
        for call, given in into().values():
            call(*given)
