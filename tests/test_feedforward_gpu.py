"""The gated feed-forward block, its gradients and the 8-bit product (needs a GB300).

Every case is compared with the formula in 64 bits on the same inputs.  The
tolerance of each element follows from what the kernels round; a value carries
two bounds through the products:

* ``w``, a bound on what fp32 sums and functions may be off.  A sum over k in
  fp32 is in error by at most (k / 8 + 8) 2^-23 sum |a||b| (the tensor cores
  add at least eight products at a time); sigmoid and products add 2^-20 |h|.
* ``v``, the sum of the squares of independent roundings, each of at most u |x|
  (u: bf16 2^-8, fp16 2^-11; fp16 also 2^-25, half its smallest step).  By
  Hoeffding's inequality their sum exceeds 7 sqrt(v) with a probability
  below 5e-11 an element.

An output is off by at most w + 7 sqrt(v) + u |y| (+ 2^-25).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

b2b = pytest.importorskip("fusion_b2b_gemm_gb300")

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f16": 2.0 ** -25, "bf16": 0.0}
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


@pytest.fixture(params=[0, 2], ids=["chosen", "pair"], autouse=True)
def kernels(request, monkeypatch):
    """Every test twice: with the kernels that the sizes lead to, and with the one for large products everywhere."""
    if not request.param:
        return
    for cls in (b2b.GatedFeedForwardPlan, b2b.ScaledFeedForwardPlan, b2b.ScaledGemmPlan):
        def init(self, *args, _init=cls.__init__, **kwargs):
            _init(self, *args, **kwargs)
            self.set_debug(0)

        def set_debug(self, flags, _set=cls.set_debug):
            _set(self, flags | request.param)

        monkeypatch.setattr(cls, "__init__", init)
        monkeypatch.setattr(cls, "set_debug", set_debug)


def normal(seed, *shape, dtype="bf16", scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(TYPES[dtype])


class Val:
    """A matrix in 64 bits with its bounds."""

    def __init__(self, x, w=None, v=None):
        self.x = x.double()
        self.w = torch.zeros_like(self.x) if w is None else w
        self.v = torch.zeros_like(self.x) if v is None else v

    def __matmul__(self, o):
        a, b = self.x.abs(), o.x.abs()
        k = self.x.shape[1]
        w = (k / 8 + 8) * 2.0 ** -23 * (a @ b) + self.w @ b + a @ o.w + self.w @ o.w
        return Val(self.x @ o.x, w, self.v @ b.square() + a.square() @ o.v)

    def __add__(self, o):
        return Val(self.x + o.x, self.w + o.w + 2.0 ** -23 * (self.x.abs() + o.x.abs()), self.v + o.v)

    @property
    def T(self):
        return Val(self.x.T, self.w.T, self.v.T)

    def rounded(self, dtype):
        return Val(self.x, self.w, self.v + (U[dtype] * (self.x.abs() + self.w) + TINY[dtype]) ** 2)

    def check(self, got, dtype=None, what=""):
        assert got.shape == self.x.shape
        assert torch.isfinite(got).all(), what
        u, tiny = (U[dtype], TINY[dtype]) if dtype else (2.0 ** -24, 0.0)
        tol = self.w + 7 * self.v.sqrt() + u * (self.x.abs() + self.w) + tiny
        over = ((got.double() - self.x).abs() - tol).max().item() if got.numel() else 0
        assert over <= 0, f"{what}: an element is {over:.3e} beyond its tolerance"


def act(g, kind):
    """The activation and its slope, from tanh."""
    if kind == "silu":
        z, dz = g / 2, 0.5
    else:
        c = math.sqrt(2 / math.pi)
        z, dz = c * (g + 0.044715 * g ** 3), c * (1 + 0.134145 * g ** 2)
    t = torch.tanh(z)
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * dz


def gated(g, u, kind):
    """act(g) u of fp32 values; slopes of both activations are below 1.13."""
    a = act(g.x, kind)[0]
    h = a * u.x
    return Val(h, 1.13 * g.w * (u.x.abs() + u.w) + a.abs() * u.w + 2.0 ** -20 * h.abs() + 2.0 ** -126)


def weights(seed, dtype, d, f, o):
    return (normal(seed, d, f, dtype=dtype, scale=d ** -0.5), normal(seed + 1, d, f, dtype=dtype, scale=d ** -0.5),
            normal(seed + 2, f, o, dtype=dtype, scale=f ** -0.5))


def want_forward(x, wg, wu, wd, kind, dtype):
    g, u = Val(x) @ Val(wg), Val(x) @ Val(wu)
    h = gated(g, u, kind)
    return g, u, h, h.rounded(dtype) @ Val(wd)


def want_backward(dy, x, wg, wu, wd, kind, dtype):
    g, u, h, _ = want_forward(x, wg, wu, wd, kind, dtype)
    a, slope = act(g.x, kind)
    dh = Val(dy) @ Val(wd).T
    # fp32 of its own: sigmoid and its products, 2^-19 of the largest term; the slope of u(g) is at most 1 + g^2.  What
    # gate and up are off moves dG and dU by at most 1.13 of it (the activations' slopes) and 1.2 (those slopes' own).
    most = u.x.abs() * (1 + g.x.abs() * (1 if kind == "silu" else 1 + g.x.square()))
    dg_w = dh.w * (u.x * slope).abs() + dh.x.abs() * (1.13 * u.w + 1.2 * g.w * (u.x.abs() + u.w) + 2.0 ** -19 * most)
    du_w = dh.w * a.abs() + dh.x.abs() * (1.13 * g.w + 2.0 ** -19 * a.abs())
    dg, du = Val(dh.x * u.x * slope, dg_w).rounded(dtype), Val(dh.x * a, du_w).rounded(dtype)
    return dg @ Val(wg).T + du @ Val(wu).T, Val(x).T @ dg, Val(x).T @ du, h.rounded(dtype).T @ Val(dy)


def case(dtype, t, d, f, o, kind="silu", seed=0):
    x, dy = normal(seed + 10, t, d, dtype=dtype), normal(seed + 11, t, o, dtype=dtype, scale=0.5)
    w = weights(seed, dtype, d, f, o)
    plan = b2b.GatedFeedForwardPlan(dtype, d, f, o, kind)
    y = plan.run(x, *w)
    y2, kept = plan.forward(x, *w)
    grads = plan.backward(dy, x, *w, kept)
    assert plan.status() == 0
    want_forward(x, *w, kind, dtype)[3].check(y, dtype, "y")
    assert torch.equal(y, y2)
    for v, got, name in zip(want_backward(dy, x, *w, kind, dtype), grads, ("dx", "dw_gate", "dw_up", "dw_down")):
        v.check(got, dtype, name)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("sizes", [(64, 64, 64, 64), (1, 8, 8, 8), (2, 264, 136, 72), (300, 520, 392, 264)], ids=str)
def test_block_and_gradients(dtype, kind, sizes):
    case(dtype, *sizes, kind)


@pytest.mark.parametrize("tokens", [1, 7, 31, 127, 128, 129, 255, 256, 257, 513, 1000])
def test_token_counts(tokens):
    case("bf16", tokens, 256, 320, 192, seed=tokens)


@pytest.mark.parametrize("sizes", [(16, 4096, 512, 256), (40, 512, 256, 4096), (3, 72, 5000, 200), (700, 1024, 2048, 1024),
                                   (2048, 136, 264, 520)], ids=str)
def test_long_products_are_cut_along_k(sizes):
    case("f16", *sizes)


@pytest.mark.parametrize("tokens", [15, 17, 33, 48, 65, 97, 130, 200, 320, 450])
def test_tiles_of_few_rows(tokens):
    """Several tiles of 16 to 128 rows, the last of them cut short, of slices whose k is cut or not."""
    case("f16", tokens, 1032, 1416, 520, seed=tokens)
    case("bf16", tokens, 96, 3080, 1608, "gelu", seed=tokens)


# ------------------------------------------------------------------------- 8 bits
def power(e):
    """2^e for -126 <= e <= 127, by its bits (torch.ldexp goes through a pow that need not be exact)."""
    return ((e.int() + 127) << 23).view(torch.float32).double()


def grid(v):
    """v rounded to the nearest e4m3 value, ties to even."""
    e = torch.frexp(v.abs().clamp(min=2.0 ** -6))[1]  # v = m 2^e, m in [1/2, 1)
    step = power(e - 4)
    return torch.round(v / step) * step


def scale_of(top):
    """The smallest power of two s with top / s <= 448, at least 2^-126."""
    m, e = torch.frexp((top / 448).clamp(min=2.0 ** -126))
    return power(e - (m == 0.5).int())


def tops(x, block_rows):
    r, c = x.shape
    pad = torch.zeros(-(-r // block_rows) * block_rows, -(-c // 128) * 128, dtype=torch.float64, device=x.device)
    pad[:r, :c] = x.abs()
    return pad.view(pad.shape[0] // block_rows, block_rows, -1, 128).amax((1, 3))


def spread(s, block_rows, shape):
    return s.double().repeat_interleave(block_rows, 0)[:shape[0]].repeat_interleave(128, 1)[:, :shape[1]]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", [(1, 8), (3, 128), (130, 136), (257, 1000), (16, 4096)], ids=str)
def test_quantize(dtype, block_rows, shape):
    x = normal(1, *shape, dtype=dtype, scale=3)
    x[:, 0] *= 100
    x[0, :] = 0
    x[-1, : shape[1] // 2] *= 1e-4
    q, s = b2b.quantize_blocks(x, block_rows)
    want = scale_of(tops(x.double(), block_rows))
    assert (s.double() != want).sum().item() == 0
    full = spread(s, block_rows, shape)
    assert (q.double() != grid(x.double() / full)).sum().item() == 0


def test_quantize_exact_borders():
    x = torch.zeros(8, 128, dtype=torch.bfloat16, device="cuda")
    x[:, 5] = torch.tensor([448, 449.9, 3.5, 3.484375, 0, 2.0 ** -130, 1e38, -448], device="cuda").bfloat16()
    q, s = b2b.quantize_blocks(x)
    assert s[:, 0].tolist() == [1, 2, 2.0 ** -7, 2.0 ** -7, 2.0 ** -126, 2.0 ** -126, 2.0 ** 118, 1]
    assert (q.double() * s.double())[[0, 2, 7], 5].tolist() == [448, 3.5, -448]


def test_quantize_not_finite():
    x = normal(2, 4, 384)
    x[1, 130] = math.inf
    x[2, 383] = math.nan
    q, s = b2b.quantize_blocks(x)
    bad = torch.zeros(4, 3, dtype=torch.bool, device="cuda")
    bad[1, 1] = bad[2, 2] = True
    assert torch.equal(s.isnan(), bad) and torch.equal(q.float().isnan(), spread(bad.float(), 1, x.shape) != 0)


def scaled(seed, n, k, block_rows):
    """e4m3 values over their whole range with scales that are no powers of two."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q = (60 * torch.randn(n, k, generator=g, device="cuda")).clamp(-448, 448).to(E4M3)
    s = 0.001 + 0.01 * torch.rand(-(-n // block_rows), -(-k // 128), generator=g, device="cuda")
    return q, s


def want_product(a, sa, b, sb):
    return Val(a.double() * spread(sa, 1, a.shape)) @ Val(b.double() * spread(sb, 128, b.shape)).T


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("sizes", [(1, 16, 8), (64, 128, 128), (5, 2000, 136), (129, 384, 392), (300, 1040, 1368),
                                   (16, 8192, 512), (1500, 512, 3000)], ids=str)
def test_product(dtype, sizes):
    m, k, n = sizes
    (a, sa), (b, sb) = scaled(1, m, k, 1), scaled(2, n, k, 128)
    plan = b2b.ScaledGemmPlan(dtype, k, n)
    out = plan.run(a, sa, b, sb)
    assert plan.status() == 0
    want_product(a, sa, b, sb).check(out, dtype)


def ffn8_case(dtype, t, d, f, o, kind="silu", seed=0):
    x = normal(seed + 10, t, d, dtype=dtype)
    x[:, :: max(1, d // 3)] *= 10
    w = [b2b.quantize_blocks(z.t().contiguous(), 128) for z in weights(seed, dtype, d, f, o)]
    plan = b2b.ScaledFeedForwardPlan(dtype, d, f, o, kind)
    y = plan.run(x, *w[0], *w[1], *w[2])
    assert plan.status() == 0
    sx = scale_of(tops(x.double(), 1))
    xq = Val(grid(x.double() / spread(sx, 1, x.shape)) * spread(sx, 1, x.shape))
    wg, wu, wd = (Val(q.double() * spread(s, 128, q.shape)).T for q, s in w)
    h = gated(xq @ wg, xq @ wu, kind)
    # Where h may lie on either side of a border, its own or its block's largest, a value may be a step off: a sixteenth
    # of a power of two up, or the block's smallest, 2^-9 scales.
    s = spread(scale_of(tops(h.x, 1)), 1, h.x.shape)
    low, high = (spread(scale_of(tops((h.x.abs() + e * h.w).clamp(min=0), 1)), 1, h.x.shape) for e in (-1, 1))
    hq = grid(h.x / s) * s
    moved = (grid((h.x - h.w) / s) != grid((h.x + h.w) / s)) | (low != high)
    step = torch.where(moved, 2 * torch.maximum(h.x.abs() / 8, high * 2.0 ** -9), 0.0)
    (Val(hq, step) @ wd).check(y, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("sizes", [(1, 16, 16, 16), (64, 128, 128, 128), (130, 272, 400, 144), (5, 2048, 1040, 336),
                                   (700, 512, 1024, 512)], ids=str)
def test_block_in_8_bits(dtype, kind, sizes):
    ffn8_case(dtype, *sizes, kind)


@pytest.mark.parametrize("rows", [15, 17, 33, 48, 65, 97, 130, 200, 320, 1000])
def test_tiles_of_few_rows_in_8_bits(rows):
    (a, sa), (b, sb) = scaled(1, rows, 2000, 1), scaled(2, 1368, 2000, 128)
    plan = b2b.ScaledGemmPlan("f16", 2000, 1368)
    out = plan.run(a, sa, b, sb)
    assert plan.status() == 0
    want_product(a, sa, b, sb).check(out, "f16")
    ffn8_case("bf16", rows, 528, 1424, 272, seed=rows)
