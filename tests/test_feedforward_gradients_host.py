"""Feed-forward calls whose inputs autograd follows are refused, in either mode (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")
forward_ad = torch.autograd.forward_ad

import fusion_b2b_gemm_gb300 as b2b  # noqa: E402
from fusion_b2b_gemm_gb300 import feedforward  # noqa: E402


def dual(*shape, dtype=torch.float16):
    x = torch.zeros(*shape, dtype=dtype)
    return forward_ad.make_dual(x, torch.ones_like(x))


def test_tangents_are_refused():
    with forward_ad.dual_level():
        x = dual(4, 16)
        assert not x.requires_grad
        with pytest.raises(RuntimeError, match="no gradient"):
            b2b.quantize_blocks(x)
        with torch.no_grad(), pytest.raises(RuntimeError, match="primals"):  # (no_grad leaves tangents alone)
            b2b.quantize_blocks(x)
        with pytest.raises(ValueError, match="GPU expected"):
            b2b.quantize_blocks(forward_ad.unpack_dual(x).primal)
        with torch.inference_mode(), pytest.raises(ValueError, match="GPU expected"):
            b2b.quantize_blocks(x)


def test_what_counts_as_followed():
    feedforward._load()
    plain, leaf = torch.zeros(3), torch.zeros(3, requires_grad=True)
    assert not feedforward._differentiated(plain, plain) and feedforward._differentiated(plain, leaf)
    with torch.no_grad():
        assert not feedforward._differentiated(plain, leaf)
    with forward_ad.dual_level():
        assert feedforward._differentiated(plain, dual(3))
        assert not feedforward._differentiated(plain)
