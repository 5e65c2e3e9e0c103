"""Feed-forward operators where they can go wrong: strides, refusals, empty inputs, infinities, streams, captures, waits that
run out, offsets past 32 bits, and a run of them together (needs a GB300).  Tolerances as in test_feedforward_gpu.py."""
import ctypes
import gc
import math
import os
import struct
import subprocess
import sys
import time

import pytest
import torch

pytestmark = pytest.mark.gpu

b2b = pytest.importorskip("fusion_b2b_gemm_gb300")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "tests"))
from test_feedforward_gpu import (  # noqa: E402
    E4M3, TINY, TYPES, U, Val, act, kernels, normal, scaled, want_backward, want_forward, want_product, weights)

INVALID, UNSUPPORTED, ALIGNMENT, ALIAS, TIMEOUT = 1, 2, 3, 4, 7


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def setup(dtype="bf16", t=70, d=136, f=264, o=72, kind="silu", seed=0):
    x, dy = normal(seed + 10, t, d, dtype=dtype), normal(seed + 11, t, o, dtype=dtype, scale=0.5)
    return b2b.GatedFeedForwardPlan(dtype, d, f, o, kind), x, weights(seed, dtype, d, f, o), dy


def within(rows, cols, dtype, left, right, fill):
    """A matrix that is a column range of a wider buffer, and the buffer."""
    buf = torch.full((rows, left + cols + right), fill, dtype=dtype, device="cuda")
    return buf[:, left:left + cols], buf


def untouched(buf, left, cols, fill):
    assert (buf[:, :left] == fill).all() and (buf[:, left + cols:] == fill).all()


# ------------------------------------------------------------------------ strides
@pytest.mark.parametrize("t", [5, 300])
def test_column_ranges_of_wider_buffers(t):
    plan, x, w, dy = setup(t=t)
    y, kept = plan.forward(x, *w)
    grads = plan.backward(dy, x, *w, kept)
    both = torch.cat([w[0], w[1]], 1)  # one matrix for both projections
    wd = within(264, 72, torch.bfloat16, 8, 16, 7.0)[0]
    wd.copy_(w[2])
    xs = within(t, 136, torch.bfloat16, 16, 8, 7.0)[0]
    xs.copy_(x)
    ws = (both[:, :264], both[:, 264:], wd)
    out, buf = within(t, 72, torch.bfloat16, 24, 8, 5.0)
    assert plan.run(xs, *ws, out=out) is out
    assert torch.equal(out, y)
    untouched(buf, 24, 72, 5.0)
    y2, kept2 = plan.forward(xs, *ws, kept=torch.empty_like(kept))
    assert torch.equal(y2, y)
    dys = within(t, 72, torch.bfloat16, 8, 0, 2.0)[0]
    dys.copy_(dy)
    for a, b in zip(plan.backward(dys, xs, *ws, kept2), grads):
        assert torch.equal(a, b)


@pytest.mark.parametrize("rows", [3, 200])
def test_scaled_operands_in_wider_buffers(rows):
    (a, sa), (b, sb) = scaled(1, rows, 272, 1), scaled(2, 136, 272, 128)
    plan = b2b.ScaledGemmPlan("f16", 272, 136)
    want = plan.run(a, sa, b, sb)
    pa = torch.zeros(rows, 272 + 48, dtype=torch.uint8, device="cuda").view(E4M3)[:, 16:288]
    pa.copy_(a)
    pb = torch.zeros(136, 304, dtype=torch.uint8, device="cuda").view(E4M3)[:, 16:288]
    pb.copy_(b)
    out, buf = within(rows, 136, torch.float16, 8, 8, 9.0)
    plan.run(pa, sa.t().contiguous().t(), pb, sb.repeat(1, 2)[:, :3], out=out)
    assert torch.equal(out, want)
    untouched(buf, 8, 136, 9.0)
    # one scale for all rows, of stride 0
    one = sa[:1].expand(rows, 3)
    assert torch.equal(plan.run(a, one, b, sb), plan.run(a, one.contiguous(), b, sb))


# ------------------------------------------------------------------------ training
def check_grads(dtype, dy, x, w, grads, kind="silu", before=None):
    wants = want_backward(dy, x, *w, kind, dtype)
    for i, (v, got) in enumerate(zip(wants, grads)):
        if got is None:
            continue
        if before is not None and i:
            v = Val(v.x + before[i - 1].double(), v.w + 2.0 ** -23 * (v.x.abs() + before[i - 1].abs().double()), v.v)
        v.check(got, None if got.dtype == torch.float32 else dtype, f"gradient {i}")


@pytest.mark.parametrize("t", [1, 40, 700])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_weight_gradients_added_to_fp32(t, dtype):
    plan, x, w, dy = setup(dtype, t=t, d=264, f=392, o=264)
    y, kept = plan.forward(x, *w)
    g = torch.Generator(device="cuda").manual_seed(3)
    # gate's and up's gradients side by side in one buffer
    both = torch.randn(264, 2 * 392 + 4, generator=g, device="cuda")
    down = torch.randn(392, 264, generator=g, device="cuda")
    grads = both[:, :392], both[:, 392:784], down
    before = [z.clone() for z in grads]
    last = both[:, 784:].clone()
    dx, *got = plan.backward(dy, x, *w, kept, weight_grads=grads)
    assert all(a is b for a, b in zip(got, grads)) and torch.equal(both[:, 784:], last)
    check_grads(dtype, dy, x, w, (dx, *got), before=before)
    # a second microbatch on top
    middle = [z.clone() for z in grads]
    plan.backward(dy, x, *w, kept, input_grad=False, weight_grads=grads)
    check_grads(dtype, dy, x, w, (None, *grads), before=middle)


def test_gradients_left_out():
    plan, x, w, dy = setup(t=33)
    y, kept = plan.forward(x, *w)
    all_of = plan.backward(dy, x, *w, kept)
    dx, *none = plan.backward(dy, x, *w, kept, weight_grads=False)
    assert torch.equal(dx, all_of[0]) and none == [None] * 3
    none, *g = plan.backward(dy, x, *w, kept, input_grad=False)
    assert none is None and all(torch.equal(a, b) for a, b in zip(g, all_of[1:]))
    for i in range(3):
        only = [None] * 3
        only[i] = torch.zeros_like(w[i], dtype=torch.float32)
        _, *g = plan.backward(dy, x, *w, kept, input_grad=False, weight_grads=only)
        assert [z is None for z in g] == [k != i for k in range(3)]
        assert torch.equal(g[i].bfloat16(), all_of[i + 1])
    assert plan.backward(dy, x, *w, kept, input_grad=False, weight_grads=False) == (None,) * 4


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_gradients_against_differences(kind):
    """Along a random direction of each input: central differences of the formula in 64 bits.

    The gradient's error is that of want_backward's bounds.  The differences' own error is below 1e-7 of their terms (step 1e-4, third
    derivatives of order one).
    """
    g = torch.Generator(device="cuda").manual_seed(5)
    d, f, o, t = 16, 40, 24, 50

    def quarters(*shape):
        return (torch.randint(-4, 5, shape, generator=g, device="cuda") / 4).half()

    x, w, dy = quarters(t, d), (quarters(d, f), quarters(d, f), quarters(f, o)), quarters(t, o)
    plan = b2b.GatedFeedForwardPlan("f16", d, f, o, kind)
    y, kept = plan.forward(x, *w)
    grads = plan.backward(dy, x, *w, kept)
    bounds = want_backward(dy, x, *w, kind, "f16")

    def loss(i, move):
        z = [m.double() for m in (x, *w)]
        z[i] = z[i] + move
        return ((act(z[0] @ z[1], kind)[0] * (z[0] @ z[2])) @ z[3] * dy.double()).sum()

    for i, (got, b) in enumerate(zip(grads, bounds)):
        v = torch.randn(got.shape, generator=g, device="cuda").double()
        slope = (loss(i, 1e-4 * v) - loss(i, -1e-4 * v)) / 2e-4
        tol = (b.w * v.abs()).sum() + 7 * ((b.v + (U["f16"] * b.x.abs() + TINY["f16"]) ** 2) * v.square()).sum().sqrt()
        tol = tol + 1e-6 * (b.x * v).abs().sum()
        assert abs((got.double() * v).sum() - slope) <= tol


# ------------------------------------------------------- empty, infinite and NaN
def test_no_tokens():
    plan, x, w, dy = setup(t=4)
    none = x[:0]
    assert plan.run(none, *w).shape == (0, 72)
    y, kept = plan.forward(none, *w)
    assert y.shape == (0, 72) and kept.shape == (0,)
    dx, *g = plan.backward(dy[:0], none, *w, kept)
    assert dx.shape == (0, 136) and all((z == 0).all() for z in g)
    acc = [torch.ones_like(z, dtype=torch.float32) for z in w]
    plan.backward(dy[:0], none, *w, kept, weight_grads=acc)
    assert all((z == 1).all() for z in acc)
    (a, sa), (b, sb) = scaled(1, 4, 64, 1), scaled(2, 32, 64, 128)
    assert b2b.ScaledGemmPlan("bf16", 64, 32).run(a[:0], sa[:0], b, sb).shape == (0, 32)
    q, s = b2b.quantize_blocks(x[:0])
    assert q.shape == (0, 136) and s.shape == (0, 2)
    assert plan.status() == 0


@pytest.mark.parametrize("t", [6, 300])
def test_nan_and_infinity_stay_in_their_rows(t):
    plan, x, w, dy = setup(t=t)
    want = plan.run(x, *w)
    x[2, 5], x[4, 100] = math.nan, math.inf
    y, kept = plan.forward(x, *w)
    bad = torch.zeros(t, dtype=torch.bool, device="cuda")
    bad[[2, 4]] = True
    assert torch.equal(y[~bad], want[~bad]) and y[2].isnan().all() and not y[4].isfinite().all()
    dx = plan.backward(dy, x, *w, kept, weight_grads=False)[0]
    assert dx[~bad].isfinite().all() and dx[2].isnan().all()


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t", [3, 200])
def test_far_out_gates(kind, t):
    """Gates of up to +-1e6 (bf16): the activation is 0 or g, its slope 0 or 1, none of it NaN."""
    plan, x, w, dy = setup(t=t, kind=kind)
    x *= 2.0 ** 20
    y, kept = plan.forward(x, *w)
    g, u, h, want = want_forward(x, *w, kind, "bf16")
    want.check(y, "bf16", "y")
    grads = plan.backward(dy, x, *w, kept)
    for v, got in zip(want_backward(dy, x, *w, kind, "bf16"), grads):
        assert got.isfinite().all()
        v.check(got, "bf16")


@pytest.mark.parametrize("rows", [5, 300])
def test_nan_scales_and_values(rows):
    (a, sa), (b, sb) = scaled(1, rows, 384, 1), scaled(2, 296, 384, 128)
    plan = b2b.ScaledGemmPlan("bf16", 384, 296)
    want = plan.run(a, sa, b, sb)
    sa[1, 2] = math.nan
    a.view(torch.uint8)[3, 7] = 0x7f  # e4m3's NaN
    got = plan.run(a, sa, b, sb)
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[[1, 3]] = True
    assert got[bad].isnan().all() and torch.equal(got[~bad], want[~bad])
    sb[1, 0] = math.nan
    got = plan.run(a, sa, b, sb)
    assert got[:, 128:256].isnan().all() and torch.equal(got[~bad][:, :128], want[~bad][:, :128])


# ---------------------------------------------------------- streams and captures
def all_calls(t, seed=0):
    """Each operator on t rows: a call that returns tensors."""
    plan, x, w, dy = setup(t=t, seed=seed)
    eight = [b2b.quantize_blocks(z.t().contiguous(), 128) for z in weights(seed, "bf16", 144, 272, 80)]
    x8 = normal(seed + 1, t, 144)
    plan8 = b2b.ScaledFeedForwardPlan("bf16", 144, 272, 80)
    (a, sa), (b, sb) = scaled(1 + seed, t, 272, 1), scaled(2 + seed, 136, 272, 128)
    product = b2b.ScaledGemmPlan("bf16", 272, 136)
    kept = plan.forward(x, *w)[1]
    return {
        "run": lambda **k: [plan.run(x, *w, **k)],
        "forward": lambda **k: [plan.forward(x, *w, **k)[0]],
        "backward": lambda **k: list(plan.backward(dy, x, *w, kept, **k)),
        "scaled": lambda **k: [plan8.run(x8, *eight[0], *eight[1], *eight[2], **k)],
        "product": lambda **k: [product.run(a, sa, b, sb, **k)],
        "quantize": lambda **k: [z.float() for z in b2b.quantize_blocks(x8, **k)],
    }, (x, x8, a)


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("t", [3, 130, 600])
def test_streams(t):
    calls, _ = all_calls(t)
    want = {k: c() for k, c in calls.items()}
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for k, c in calls.items():
        if k != "quantize":
            assert same(c(stream=streams[0]), want[k]), k
    got = []
    for i in range(30):  # several at once
        with torch.cuda.stream(streams[i % 3]):
            got.append([c() for c in calls.values()])
    torch.cuda.synchronize()
    for g in got:
        for a, b in zip(g, want.values()):
            assert same(a, b)


def test_memory_of_a_run_on_another_stream_is_kept():
    """Inputs that the caller lets go of are not handed out anew while the run on another stream reads them."""
    plan, x, w, dy = setup(t=600, d=1024, f=2048, o=512)
    want = plan.run(x, *w)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(20):
        x2 = x.clone()
        s.wait_stream(torch.cuda.current_stream())
        y = plan.run(x2, *w, stream=s)
        del x2
        junk = torch.full_like(x, 9.0)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(y, want)
        del junk


def test_memory_of_gradients_added_on_another_stream_is_kept():
    plan, x, w, dy = setup(t=600, d=1024, f=2048, o=512)
    kept = plan.forward(x, *w)[1]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(10):
        grads = [torch.zeros_like(z, dtype=torch.float32) for z in w]
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(2_000_000)
        plan.backward(dy, x, *w, kept, weight_grads=grads, stream=s)
        del grads
        others = [torch.full_like(z, 9.0, dtype=torch.float32) for z in w]
        torch.cuda.synchronize()
        assert all((z == 9).all() for z in others)


@pytest.mark.parametrize("t", [4, 200])
def test_captured_calls_follow_their_inputs(t):
    calls, inputs = all_calls(t)
    for name, c in calls.items():
        c()
        torch.cuda.synchronize()
        graphs, outs = [], []
        for _ in range(2):  # two graphs of one pool
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
                outs.append(c())
            graphs.append(g)
        for _ in range(2):
            for z in inputs:
                z.copy_(z.float().roll(1, 0).to(z.dtype))
            want = c()
            for g, o in zip(graphs, outs):
                g.replay()
                torch.cuda.synchronize()
                assert same(o, want), name
        del graphs, outs, g
        gc.collect()


@pytest.mark.parametrize("t", [1, 60, 129, 600])
def test_equal_inputs_give_equal_bits(t):
    calls, _ = all_calls(t)
    for name, c in calls.items():
        want = c()
        for _ in range(5):
            assert same(c(), want), name


@pytest.mark.parametrize("t", [2, 150])
def test_the_way_through_python_does_the_same(t):
    plan, x, w, dy = setup(t=t)
    y, kept = plan.forward(x, *w)
    grads = plan.backward(dy, x, *w, kept)
    run = plan.run(x, *w)
    bound, plan._bound = plan._bound, None
    y2, kept2 = plan.forward(x, *w)
    assert torch.equal(y, y2) and torch.equal(run, plan.run(x, *w))
    assert same(grads, plan.backward(dy, x, *w, kept)) and same(grads, plan.backward(dy, x, *w, kept2))
    plan._bound = bound
    (a, sa), (b, sb) = scaled(1, t, 64, 1), scaled(2, 32, 64, 128)
    product = b2b.ScaledGemmPlan("bf16", 64, 32)
    want = product.run(a, sa, b, sb)
    product._bound = None
    assert torch.equal(want, product.run(a, sa, b, sb))


# ------------------------------------------------------------------ large offsets
def test_offsets_past_32_bits():
    """140,000 tokens of 16,384 hidden values: 2.3e9 elements, of which the last rows are looked at."""
    t, d, f, o = 140_000, 64, 16_384, 64
    plan, x, w, dy = setup(t=t, d=d, f=f, o=o)
    y, kept = plan.forward(x, *w)
    dx = plan.backward(dy, x, *w, kept, weight_grads=False)[0]
    assert plan.status() == 0
    rows = torch.cat([torch.arange(0, t, 9973, device="cuda"), torch.arange(t - 40, t, device="cuda")])
    del kept
    want_forward(x[rows], *w, "silu", "bf16")[3].check(y[rows], "bf16", "y")
    want_backward(dy[rows], x[rows], *w, "silu", "bf16")[0].check(dx[rows], "bf16", "dx")


# ------------------------------------------------------------- waits that run out
@pytest.mark.parametrize("t", [4, 100, 600])
def test_waits_that_run_out_are_reported(t):
    plan, x, w, dy = setup(t=t)
    y, kept = plan.forward(x, *w)
    grads = plan.backward(dy, x, *w, kept)
    (a, sa), (b, sb) = scaled(1, t, 272, 1), scaled(2, 136, 272, 128)
    product = b2b.ScaledGemmPlan("bf16", 272, 136)
    d = product.run(a, sa, b, sb)
    eight = [b2b.quantize_blocks(z.t().contiguous(), 128) for z in weights(0, "bf16", 144, 272, 80)]
    x8 = normal(1, t, 144)
    plan8 = b2b.ScaledFeedForwardPlan("bf16", 144, 272, 80)
    y8 = plan8.run(x8, *eight[0], *eight[1], *eight[2])
    assert not any(p.status() for p in (plan, product, plan8))
    again = [(plan, lambda: [plan.run(x, *w)], [y]), (plan, lambda: plan.backward(dy, x, *w, kept), grads),
             (product, lambda: [product.run(a, sa, b, sb)], [d]),
             (plan8, lambda: [plan8.run(x8, *eight[0], *eight[1], *eight[2])], [y8])]
    for p, call, want in again:
        p.set_wait_budget(5_000_000)
        p.set_debug(1)
        began = time.time()
        call()
        assert p.status() == TIMEOUT and time.time() - began < 5
        assert p.status() == 0  # (read and cleared)
        p.set_debug(0)
        p.set_wait_budget(0)
        assert same(call(), want) and p.status() == 0


# ----------------------------------------------------------------------- refusals
def refused(error, match, call):
    with pytest.raises(error, match=match):
        call()


def test_refusals_by_type_shape_and_place():
    plan, x, w, dy = setup(t=6)
    y, kept = plan.forward(x, *w)
    wg, wu, wd = w
    refused(TypeError, "x: torch.float16", lambda: plan.run(x.half(), *w))
    refused(TypeError, "w_up: torch.float32", lambda: plan.run(x, wg, wu.float(), wd))
    refused(TypeError, "x: list", lambda: plan.run([1], *w))
    refused(ValueError, "w_gate: shape", lambda: plan.run(x, wg[:, :8], wu, wd))
    refused(ValueError, "w_down: shape", lambda: plan.run(x, wg, wu, wd.t()))
    refused(ValueError, "x: shape", lambda: plan.run(x[0], *w))
    refused(ValueError, "last stride", lambda: plan.run(x, wg.t().contiguous().t(), wu, wd))
    refused(ValueError, "w_up is on cpu", lambda: plan.run(x, wg, wu.cpu(), wd))
    refused(ValueError, "out: shape", lambda: plan.run(x, *w, out=y[:3]))
    refused(TypeError, "out: torch.float32", lambda: plan.run(x, *w, out=y.float()))
    refused(ValueError, "dy: shape", lambda: plan.backward(dy[:3], x, *w, kept))
    refused(ValueError, "kept: shape", lambda: plan.backward(dy, x, *w, kept[::2]))
    refused(TypeError, "kept: torch.float32", lambda: plan.backward(dy, x, *w, kept.view(torch.float32)))
    refused(TypeError, "kept: tuple", lambda: plan.backward(dy, x, *w, (kept,)))
    refused(ValueError, "kept is on cpu", lambda: plan.backward(dy, x, *w, kept.cpu()))
    refused(b2b.B2BError, "INVALID_ARG", lambda: plan.backward(dy, x, *w, kept[:-256]))
    refused(b2b.B2BError, "INVALID_ARG", lambda: plan.forward(x, *w, kept=kept[:-256]))
    refused(b2b.B2BError, "ALIGNMENT", lambda: plan.forward(x, *w, kept=torch.cat([kept, kept])[16:]))
    refused(ValueError, "three expected", lambda: plan.backward(dy, x, *w, kept, weight_grads=(None,)))
    refused(TypeError, "gradient of w_up", lambda: plan.backward(dy, x, *w, kept, weight_grads=(None, wu.clone(), None)))
    (a, sa), (b, sb) = scaled(1, 6, 64, 1), scaled(2, 32, 64, 128)
    product = b2b.ScaledGemmPlan("bf16", 64, 32)
    refused(TypeError, "a: torch.bfloat16", lambda: product.run(a.bfloat16(), sa, b, sb))
    refused(ValueError, "a_scale: shape", lambda: product.run(a, sa[:2], b, sb))
    refused(TypeError, "b_scale: torch.float64", lambda: product.run(a, sa, b, sb.double()))
    refused(ValueError, "b_scale is on cpu", lambda: product.run(a, sa, b, sb.cpu()))
    plan.close()
    refused(b2b.B2BError, "INVALID_ARG", lambda: plan.run(x, *w))


def test_refusals_of_inputs_that_need_a_gradient():
    plan, x, w, dy = setup(t=6)
    y, kept = plan.forward(x, *w)
    p = torch.nn.Parameter(w[0])
    refused(RuntimeError, "no gradient", lambda: plan.run(x, p, *w[1:]))
    refused(RuntimeError, "no gradient", lambda: plan.forward(x, p, *w[1:]))
    refused(RuntimeError, "no gradient", lambda: plan.backward(dy.requires_grad_(), x, *w, kept))
    with torch.no_grad():
        assert torch.equal(plan.run(x, p, *w[1:]), y)


def test_refusals_by_alignment_and_overlap():
    plan, x, w, dy = setup(t=6)
    y, kept = plan.forward(x, *w)

    def code(want, call):
        with pytest.raises(b2b.B2BError) as e:
            call()
        assert e.value.code == want

    odd = within(6, 136, torch.bfloat16, 4, 4, 0.0)[0]  # 8 bytes off
    code(ALIGNMENT, lambda: plan.run(odd, *w))
    code(ALIGNMENT, lambda: plan.run(within(6, 136, torch.bfloat16, 0, 4, 0.0)[0], *w))  # rows 8 bytes off
    code(INVALID, lambda: plan.run(x[:1].expand(6, 136), *w))
    code(ALIGNMENT, lambda: plan.run(x, *w, out=within(6, 72, torch.bfloat16, 4, 4, 0.0)[0]))
    square, xs, ws, dys = setup(t=6, d=72, f=264, o=72)
    code(ALIAS, lambda: square.run(xs, *ws, out=xs))
    buf = torch.zeros(6, 144, dtype=torch.bfloat16, device="cuda")
    code(ALIAS, lambda: square.run(buf[:, :72], *ws, out=buf[:, 64:136]))
    buf[:, :72] = xs
    assert torch.equal(square.run(buf[:, :72], *ws, out=buf[:, 72:]), square.run(xs, *ws))  # side by side
    whole = torch.zeros(kept.numel() + 2 * 6 * 72, dtype=torch.uint8, device="cuda")
    code(ALIAS, lambda: plan.forward(x, *w, kept=whole, out=whole[-2 * 6 * 72 - 512:-512].view(torch.bfloat16).view(6, 72)))
    g = torch.zeros(136, 264, device="cuda")
    code(ALIAS, lambda: plan.backward(dy, x, *w, kept, weight_grads=(g, g, None)))
    (a, sa), (b, sb) = scaled(1, 6, 64, 1), scaled(2, 32, 64, 128)
    product = b2b.ScaledGemmPlan("bf16", 64, 32)
    code(ALIGNMENT, lambda: product.run(torch.zeros(6, 72, dtype=torch.uint8, device="cuda").view(E4M3)[:, :64], sa, b, sb))


def test_refusals_at_the_c_entries():
    plan, x, w, dy = setup(t=600)
    lib = b2b
    n = ctypes.c_size_t()
    assert lib.b2b_ffn_workspace(plan._h, -1, 0, ctypes.byref(n)) == INVALID
    assert lib.b2b_ffn_workspace(plan._h, 1, 3, ctypes.byref(n)) == INVALID
    assert lib.b2b_ffn_workspace(plan._h, 1 << 31, 0, ctypes.byref(n)) == UNSUPPORTED
    assert lib.b2b_ffn_workspace(plan._h, 600, 0, ctypes.byref(n)) == 0 and n.value > 0
    assert lib.b2b_ffn_plan_set_debug(plan._h, 4) == INVALID
    out = torch.zeros(600, 72, dtype=torch.bfloat16, device="cuda")
    ws = torch.zeros(n.value + 256, dtype=torch.uint8, device="cuda")

    def forward(tokens=600, kept=0, kept_bytes=0, wsp=ws.data_ptr(), size=n.value, outp=out.data_ptr()):
        args = struct.pack("15q", tokens, x.data_ptr(), 136, w[0].data_ptr(), 264, w[1].data_ptr(), 264, w[2].data_ptr(), 72, outp, 72,
                           kept, kept_bytes, wsp, size)
        return lib.b2b_ffn_forward(plan._h, args, None)

    torch.cuda.synchronize()
    assert forward() == 0
    assert forward(tokens=-1) == INVALID and forward(wsp=0) == INVALID and forward(size=n.value - 1) == INVALID
    assert forward(wsp=ws.data_ptr() + 16) == ALIGNMENT and forward(outp=0) == INVALID
    assert forward(kept=ws.data_ptr(), kept_bytes=256) == INVALID  # too little
    assert lib.b2b_ffn_kept_bytes(plan._h, -1, ctypes.byref(n)) == INVALID
    assert lib.b2b_ffn_kept_bytes(plan._h, 1, None) == INVALID
    assert lib.b2b_ffn_backward(plan._h, None, None) == INVALID
    product = b2b.ScaledGemmPlan("bf16", 64, 32)
    assert lib.b2b_ffn_workspace(product._h, 5, 1, ctypes.byref(n)) == INVALID  # (training: not of this kind)
    assert lib.b2b_ffn_forward(product._h, b"\0" * 120, None) == INVALID  # another kind of plan
    assert lib.b2b_scaled_gemm_run(plan._h, b"\0" * 120, None) == INVALID
    torch.cuda.synchronize()
    assert torch.equal(out, plan.run(x, *w))


# ------------------------------------------------------------------- run together
def test_trained_then_served_in_8_bits():
    """The example: its accumulated gradients against the formula's, its 8-bit outputs against the operator's definition."""
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import feed_forward as ex
    weights_, errors = ex.train(192, 272, 100, 2)
    assert len(errors) == 2 and all(math.isfinite(e) for e in errors)
    plan = b2b.GatedFeedForwardPlan("bf16", 192, 272)
    x, target = normal(1, 100, 192), normal(2, 100, 192)
    got, _ = ex.gradients(plan, weights_, x, target, 3)
    total = None
    for part, want in zip(x.chunk(3), target.chunk(3)):
        y, kept = plan.forward(part, *weights_)
        dy = ((y.float() - want.float()) * (2 * 100 / target.numel())).bfloat16()
        b = want_backward(dy, part, *weights_, "silu", "bf16")[1:]
        total = b if total is None else [p + q for p, q in zip(total, b)]
    for g, v in zip(got, total):
        Val(v.x / 100, v.w / 100 + 2.0 ** -22 * v.x.abs() / 100, v.v / 1e4).check(g)
    y = ex.serve(weights_, x)
    eight = [b2b.quantize_blocks(z.t().contiguous(), 128) for z in weights_]
    assert torch.equal(y, b2b.ScaledFeedForwardPlan("bf16", 192, 272).run(x, *eight[0], *eight[1], *eight[2]))


def test_block_of_quantised_products():
    """Gate, up and down as three products with what lies between them in torch: the 8-bit block in one call."""
    t, d, f, o = 200, 256, 384, 128
    x = normal(1, t, d)
    eight = [b2b.quantize_blocks(z.t().contiguous(), 128) for z in weights(0, "bf16", d, f, o)]
    xq, xs = b2b.quantize_blocks(x)
    g, u = (b2b.ScaledGemmPlan("bf16", d, f).run(xq, xs, *e) for e in eight[:2])
    # (rounded to bf16 in between, so compared with the bounds that that gives)
    h = (g.double() * torch.sigmoid(g.double()) * u.double()).bfloat16()
    hq, hs = b2b.quantize_blocks(h)
    y = b2b.ScaledGemmPlan("bf16", f, o).run(hq, hs, *eight[2])
    want_product(hq, hs, *eight[2]).check(y, "bf16")
    fused = b2b.ScaledFeedForwardPlan("bf16", d, f, o).run(x, *eight[0], *eight[1], *eight[2])
    # each h off by three bf16 roundings (3 * 2^-8) and one e4m3 step on either side (2^-3 of it, or 2^-9 of its scale)
    off = Val(h.double(), h.double().abs() * (3 * 2.0 ** -8 + 2.0 ** -3) + 2.0 ** -8 * hs.double().repeat_interleave(128, 1)[:, :f])
    (off @ Val(eight[2][0].double() * eight[2][1].double().repeat_interleave(128, 0)[:o].repeat_interleave(128, 1)[:, :f]).T).check(
        fused, "bf16")


def test_example_runs():
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", "feed_forward.py"), "--tokens", "150", "--steps", "2"],
                       capture_output=True, text=True, cwd=ROOT, timeout=300)
    assert r.returncode == 0, r.stderr
    assert "in 8 bits" in r.stdout
