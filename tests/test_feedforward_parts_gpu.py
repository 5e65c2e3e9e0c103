"""Feed-forward launches whose tiles are cut along k, with the kernel that joins the parts, and plans whose flags change between
runs (needs a GB300).  Tolerances as in test_feedforward_gpu.py."""
import ctypes
import math
import os
import struct
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

b2b = pytest.importorskip("fusion_b2b_gemm_gb300")
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
from test_feedforward_gpu import (  # noqa: E402
    E4M3, Val, gated, grid, normal, scale_of, scaled, spread, tops, want_backward, want_product, weights)

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


# ------------------------------------------------- parts of the 8-bit gate
def units(sizes, gate, kpan):
    """(tiles computed as one unit each, parts) of a launch on this GPU."""
    clusters = torch.cuda.get_device_properties(0).multi_processor_count // 2
    arr = (ctypes.c_int64 * (2 * len(sizes)))(*[v for s in sizes for v in s])
    out = (ctypes.c_int64 * 240001)()
    assert b2b.b2b_ffn_units(len(sizes), arr, gate, kpan, clusters, out, 240001) == 0
    parts = [out[6 + 6 * i] >= 0 for i in range(out[0])]
    return parts.count(False), parts.count(True)


def with_pair_kernel(plan):
    plan.set_debug(PAIR)
    return plan


def want_block_in_8_bits(x, eight, kind):
    """The block's definition in 64 bits, with the bounds of test_feedforward_gpu.py's ffn8_case."""
    sx = spread(scale_of(tops(x.double(), 1)), 1, x.shape)
    wg, wu, wd = (Val(q.double() * spread(s, 128, q.shape)).T for q, s in eight)
    xq = Val(grid(x.double() / sx) * sx)
    h = gated(xq @ wg, xq @ wu, kind)
    # a value whose bounds hold a border, its own or its block's scale's, may be a step off
    s = spread(scale_of(tops(h.x, 1)), 1, h.x.shape)
    low, high = (spread(scale_of(tops((h.x.abs() + e * h.w).clamp(min=0), 1)), 1, h.x.shape) for e in (-1, 1))
    moved = (grid((h.x - h.w) / s) != grid((h.x + h.w) / s)) | (low != high)
    step = torch.where(moved, 2 * torch.maximum(h.x.abs() / 8, high * 2.0 ** -9), 0.0)
    return Val(grid(h.x / s) * s, step) @ wd


def in_8_bits(seed, d, f, o):
    return [b2b.quantize_blocks(z.t().contiguous(), 128) for z in weights(seed, "bf16", d, f, o)]


@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("t,d,f,o,whole", [(5, 8192, 272, 336, False), (300, 8192, 400, 144, False), (2560, 4096, 1024, 272, True)])
def test_8_bit_gate_in_parts(t, d, f, o, whole, kind):
    """Every tile cut, or some of them beside whole ones; hidden columns that end inside a block."""
    one, cut = units([(t, f)], 1, d // 128)
    assert (one > 0) == whole and cut > 0
    x, eight = normal(1, t, d), in_8_bits(2, d, f, o)
    x[:, ::1001] *= 10
    x[t // 2] = 0
    plan = with_pair_kernel(b2b.ScaledFeedForwardPlan("bf16", d, f, o, kind))
    y = plan.run(x, *eight[0], *eight[1], *eight[2])
    assert plan.status() == 0
    want_block_in_8_bits(x, eight, kind).check(y, "bf16")
    assert (y[t // 2] == 0).all()
    # a NaN and an infinity make their own rows NaN, and no other
    bad = torch.zeros(t, dtype=torch.bool, device="cuda")
    for r, c, v in ((1, 5, math.nan), (t - 1, d - 1, math.inf)):
        x[r, c] = v
        bad[r] = True
    z = plan.run(x, *eight[0], *eight[1], *eight[2])
    assert z[bad].isnan().all() and torch.equal(z[~bad], y[~bad])
    assert plan.status() == 0


def test_8_bit_gate_in_parts_writes_its_rows_alone():
    """The hidden values and scales lie between other things in the workspace: what follows them stays."""
    t, d, f, o = 5, 8192, 272, 336
    x, eight = normal(1, t, d), in_8_bits(2, d, f, o)
    plan = with_pair_kernel(b2b.ScaledFeedForwardPlan("f16", d, f, o))
    x = x.half()
    n = ctypes.c_size_t()
    assert b2b.b2b_ffn_workspace(plan._h, t, 0, ctypes.byref(n)) == 0
    out = torch.empty(t, o, dtype=torch.float16, device="cuda")
    ws = torch.full((n.value + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    args = struct.pack("22q", t, x.data_ptr(), d, *(v for q, _ in eight for v in (q.data_ptr(), q.stride(0))), out.data_ptr(), o,
                       *(v for _, s in eight for v in (s.data_ptr(), *s.stride())), ws.data_ptr(), n.value)
    torch.cuda.synchronize()
    assert b2b.b2b_scaled_ffn_run(plan._h, args, None) == 0
    torch.cuda.synchronize()
    assert plan.status() == 0 and torch.equal(out, plan.run(x, *eight[0], *eight[1], *eight[2]))
    hidden, rounded = ws[:t * f], -(-t * f // 256) * 256
    assert (ws[t * f:rounded] == 0x5a).all() and (ws[n.value:] == 0x5a).all()
    at = rounded + -(-t * d // 256) * 256 + -(-4 * t * (d // 128) // 256) * 256
    blocks = -(-f // 128)
    scale = ws[at:at + 4 * t * blocks].view(torch.float32).view(blocks, t).t()
    assert (ws[at + 4 * t * blocks:at + -(-4 * t * blocks // 256) * 256] == 0x5a).all()
    # each scale is that of its block: the largest value takes more than half of e4m3's range, and no value is NaN
    h = hidden.view(E4M3).view(t, f).double()
    assert torch.isfinite(h).all() and (torch.frexp(scale)[0] == 0.5).all()
    assert ((tops(h, 1) > 208) & (tops(h, 1) <= 448)).all()


# --------------------------------------------------- parts added to fp32
def panels(t):
    return -(-t // 64)


GRADS = [(4096, 264, 392, 264, False), (8192, 264, 392, 264, False), (5000, 136, 264, 520, False), (8192, 1000, 1664, 1016, True)]


def buffers(seed, w):
    """fp32 gradients to add to, gate's and up's side by side in one buffer, down's in a wider one; and what lies beside."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    (d, f), o = w[0].shape, w[2].shape[1]
    both = torch.randn(d, 2 * f + 12, generator=g, device="cuda")
    down = torch.randn(f, o + 8, generator=g, device="cuda")
    return [both[:, :f], both[:, f:2 * f], down[:, 4:4 + o]], [both[:, 2 * f:], down[:, :4], down[:, 4 + o:]]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("t,d,f,o,whole", GRADS)
def test_parts_added_to_fp32_gradients(t, d, f, o, whole, dtype):
    one, cut = units([(d, f), (d, f), (f, o)], 0, panels(t))
    assert (one > 0) == whole and cut > 0
    x, dy, w = normal(1, t, d, dtype=dtype), normal(2, t, o, dtype=dtype, scale=0.5), weights(3, dtype, d, f, o)
    plan = b2b.GatedFeedForwardPlan(dtype, d, f, o)
    y, kept = plan.forward(x, *w)
    grads, beside = buffers(4, w)
    before, around = [z.clone() for z in grads], [z.clone() for z in beside]
    dx, *got = plan.backward(dy, x, *w, kept, weight_grads=grads)
    assert plan.status() == 0 and all(a is b for a, b in zip(got, grads))
    wants = want_backward(dy, x, *w, "silu", dtype)
    wants[0].check(dx, dtype, "dx")
    for name, v, z, b in zip(("gate", "up", "down"), wants[1:], grads, before):
        v.x = v.x + b.double()
        v.w = v.w + 2.0 ** -23 * (v.x.abs() + b.abs().double())
        v.check(z, None, name)
    assert all(torch.equal(a, b) for a, b in zip(beside, around))
    # once more on top: added once again, no more and no less
    again = [z.clone() for z in grads]
    plan.backward(dy, x, *w, kept, input_grad=False, weight_grads=grads)
    for name, v, z, a, b in zip(("gate", "up", "down"), wants[1:], grads, again, before):
        v.x = v.x - b.double() + a.double()
        v.w = v.w + 2.0 ** -22 * (v.x.abs() + a.abs().double())
        v.check(z, None, name + " again")
    assert all(torch.equal(a, b) for a, b in zip(beside, around))


@pytest.mark.parametrize("t,d,f,o,whole", [GRADS[0], GRADS[2]])
def test_parts_of_some_gradients(t, d, f, o, whole):
    """Each of the gradients, and each pair of them, left out: the others as if all were there."""
    x, dy, w = normal(1, t, d), normal(2, t, o, scale=0.5), weights(3, "bf16", d, f, o)
    plan = b2b.GatedFeedForwardPlan("bf16", d, f, o)
    y, kept = plan.forward(x, *w)
    sizes = (d, f), (d, f), (f, o)
    wants = want_backward(dy, x, *w, "silu", "bf16")[1:]
    for mask in range(1, 7):
        some = [i for i in range(3) if mask >> i & 1]
        assert units([sizes[i] for i in some], 0, panels(t))[1] > 0
        grads, beside = buffers(mask, w)
        before, around = [z.clone() for z in grads], [z.clone() for z in beside]
        got = plan.backward(dy, x, *w, kept, input_grad=False, weight_grads=[grads[i] if i in some else None for i in range(3)])
        assert got[0] is None and [z is None for z in got[1:]] == [i not in some for i in range(3)]
        for i, (v, z, b) in enumerate(zip(wants, grads, before)):
            if i in some:
                Val(v.x + b.double(), v.w + 2.0 ** -23 * (v.x.abs() + 2 * b.abs().double()), v.v).check(z, None, f"{some}: {i}")
            else:
                assert torch.equal(z, b)
        assert all(torch.equal(a, b) for a, b in zip(beside, around))
    assert plan.status() == 0


# ------------------------------------------------------------ large offsets
def test_8_bit_offsets_past_32_bits():
    """140,000 rows of 16,384 values (2.3e9): the quantiser's and the product's first and last rows, and the block's."""
    t, f, n = 140_000, 16_384, 64
    rows = torch.cat([torch.arange(0, t, 9973, device="cuda"), torch.arange(t - 40, t, device="cuda")])
    x = normal(1, t, f)
    q, s = b2b.quantize_blocks(x)
    want = scale_of(tops(x[rows].double(), 1))
    assert (s[rows].double() != want).sum().item() == 0
    assert (q.view(torch.uint8)[rows].view(E4M3).double() != grid(x[rows].double() / spread(want, 1, (len(rows), f)))).sum().item() == 0
    del x
    b, sb = scaled(2, n, f, 128)
    product = b2b.ScaledGemmPlan("bf16", f, n)
    out = product.run(q, s, b, sb)
    want_product(q.view(torch.uint8)[rows].view(E4M3), s[rows], b, sb).check(out[rows], "bf16")
    del q, s, out
    x, eight = normal(3, t, 64), in_8_bits(4, 64, f, n)
    block = b2b.ScaledFeedForwardPlan("bf16", 64, f, n)
    y = block.run(x, *eight[0], *eight[1], *eight[2])
    want_block_in_8_bits(x[rows], eight, "silu").check(y[rows], "bf16")
    assert product.status() == 0 and block.status() == 0
