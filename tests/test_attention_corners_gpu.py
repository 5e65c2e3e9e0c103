"""Corners of the attention calls: what a caller may do and seldom does (needs a GB300).

Inputs, results in 64 bits and their tolerances are those of test_attention_gpu.py.
"""
import ctypes
import math

import pytest
import torch

from test_attention_gpu import ALIAS, ALIGNMENT, TIMEOUT, Want, b2b, cumulative, ints, normal, prompt_case, want_prompt

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


# ----------------------------------------------------------------- page tables
@pytest.mark.parametrize("pages", [0, 2, 5])
@pytest.mark.parametrize("prefix", [0, 150])
def test_a_page_table_without_columns_holds_no_keys(prefix, pages):
    """No request has a page yet: lengths are clamped to the table, also where the pool has as many pages as there are
    requests (an empty tensor's address is null, as that of no table)."""
    q, k, v = normal(1, 2, 4, 64), normal(2, prefix, 2, 64), normal(3, prefix, 2, 64)
    pool, lengths = normal(4, pages, 16, 2, 64), ints([5, 9])
    plan = b2b.SharedPrefixAttentionPlan("f16", 4, 2, 64)
    want = Want(2, 4, 64)
    for b in range(2):
        want.rows(b, q[b:b + 1], k, v, [prefix], 1 / 8, "f16")
    for table in (torch.empty(2, 0, dtype=torch.int32, device="cuda"), ints([[0, 1], [1, 0]])[:, :0]):
        want.check(*plan.run(q, k, v, pool, pool, lengths, table, return_lse=True))
        out, lse = torch.full_like(q, 7.0), torch.full((2, 4), 7.0, device="cuda")
        want.check(*plan.run(q, k, v, pool, pool, lengths, table, out=out, lse=lse))
    assert plan.status() == 0


# -------------------------------------------------------------------- timeouts
def split_prompt():
    """One query over many keys, which are cut into parts: plan, arguments of a run."""
    q, k, v = normal(1, 1, 4, 64), normal(2, 5000, 2, 64), normal(3, 5000, 2, 64)
    plan = b2b.PromptAttentionPlan("f16", 4, 2, 64)
    n = ctypes.c_size_t()
    assert b2b.b2b_prompt_attention_workspace(plan._h, 1, 1, 5000, 1, ctypes.byref(n)) == 0 and n.value > 0
    want = want_prompt(q, k, v, [1], [5000], True, None, "f16")
    return plan, (q, k, v, ints([0, 1]), ints([0, 5000])), want


def split_shared():
    q, k, v = normal(1, 3, 4, 64), normal(2, 5000, 2, 64), normal(3, 5000, 2, 64)
    cache, lengths = normal(4, 3, 300, 2, 64), [300, 0, 17]
    plan = b2b.SharedPrefixAttentionPlan("f16", 4, 2, 64)
    n = ctypes.c_size_t()
    assert b2b.b2b_shared_attention_workspace(plan._h, 3, 1, 5000, 300, ctypes.byref(n)) == 0 and n.value > 0
    want = Want(3, 4, 64)
    for b, m in enumerate(lengths):
        want.rows(b, q[b:b + 1], torch.cat([k, cache[b, :m]]), torch.cat([v, cache[b, :m]]), [5000 + m], 1 / 8, "f16")
    return plan, (q, k, v, cache, cache, ints(lengths)), want


def split_many():
    """More short items than CTAs: some are claimed ahead of the one that stops."""
    q, k, v = normal(1, 300, 8, 64), normal(2, 4000, 4, 64), normal(3, 4000, 4, 64)
    cache, lengths = normal(4, 300, 64, 4, 64), [(7 * b) % 65 for b in range(300)]
    plan = b2b.SharedPrefixAttentionPlan("f16", 8, 4, 64)
    n = ctypes.c_size_t()
    assert b2b.b2b_shared_attention_workspace(plan._h, 300, 1, 4000, 64, ctypes.byref(n)) == 0 and n.value > 0
    want = Want(300, 8, 64)
    for b, m in enumerate(lengths):
        want.rows(b, q[b:b + 1], torch.cat([k, cache[b, :m]]), torch.cat([v, cache[b, :m]]), [4000 + m], 1 / 8, "f16")
    return plan, (q, k, v, cache, cache, ints(lengths)), want


@pytest.mark.parametrize("case", [split_prompt, split_shared, split_many])
def test_a_timeout_leaves_results_of_joined_parts_alone(case):
    """Parts that were not written are not joined, neither another run's that lie in the same workspace."""
    plan, args, want = case()
    first = plan.run(*args, return_lse=True)  # its parts stay in the allocator's memory
    want.check(*first)
    assert plan.status() == 0
    out, lse = torch.full_like(first[0], 7.0), torch.full_like(first[1], 7.0)
    plan.set_wait_budget(20_000_000)
    plan.set_debug(1)
    plan.run(*args, out=out, lse=lse)
    plan.set_debug(0)
    plan.set_wait_budget(0)
    good = plan.run(*args, return_lse=True)  # (before the status is read: a run of its own)
    assert plan.status() == TIMEOUT
    assert (out == 7).all() and (lse == 7).all()
    assert torch.equal(good[0], first[0]) and torch.equal(good[1], first[1])
    assert plan.status() == 0


# ------------------------------------------------------- the compiled module
def test_calls_without_the_compiled_module(monkeypatch):
    """The way through Python gives the same bits."""
    from fusion_b2b_gemm_gb300 import attention
    q, k, v, cu = normal(1, 90, 4, 64), normal(2, 90, 2, 64), normal(3, 90, 2, 64), ints([0, 31, 90])
    cache, lengths = normal(4, 9, 16, 2, 64), ints([5, 16, 0])
    calls = [("PromptAttentionPlan", (q, k, v, cu)), ("SharedPrefixAttentionPlan", (q[:9], k, v, cache[:3], cache[:3], lengths)),
             ("SharedPrefixAttentionPlan", (q[:9], k, v, cache, cache, lengths, ints([[8], [3], [-1]])))]
    want = [getattr(b2b, kind)("f16", 4, 2, 64).run(*args, return_lse=True) for kind, args in calls]
    assert attention._binding is not attention._NoBinding
    monkeypatch.setattr(attention, "_binding", attention._NoBinding)
    for (kind, args), w in zip(calls, want):
        plan = getattr(b2b, kind)("f16", 4, 2, 64)
        got = plan.run(*args, return_lse=True)
        assert torch.equal(got[0], w[0]) and torch.equal(got[1], w[1])
        assert torch.equal(plan.run(*args, stream=torch.cuda.current_stream()), w[0])
        assert plan.status() == 0


def one_long_item(queries):
    """2000 sequences of which one has 600,000 keys: its item alone takes several milliseconds."""
    n = 600_000
    nq, nk = [1] * 1999 + [queries], [1] * 1999 + [n]
    q, k, v = normal(1, sum(nq), 1, 64), normal(2, sum(nk), 1, 64), normal(3, sum(nk), 1, 64)
    plan = b2b.PromptAttentionPlan("f16", 1, 1, 64)
    size = ctypes.c_size_t()
    assert b2b.b2b_prompt_attention_workspace(plan._h, 2000, sum(nq), sum(nk), 0, ctypes.byref(size)) == 0
    assert size.value == 0  # (not cut into parts)
    args = q, k, v, cumulative(nq), cumulative(nk), False
    return plan, args


def test_a_short_budget_does_not_count_the_kernel_before():
    """A run starts while the kernel before it in the stream is finishing, and its waits count from that one's end."""
    long, args = one_long_item(128)
    q, k, v, cu = normal(4, 150, 4, 64), normal(5, 150, 2, 64), normal(6, 150, 2, 64), ints([0, 150])
    plan = b2b.PromptAttentionPlan("f16", 4, 2, 64)
    plan.set_wait_budget(1_000_000)
    plan.run(q, k, v, cu)
    assert plan.status() == 0
    start, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    long.run(*args)
    assert long.status() == 0
    start.record()
    long.run(*args)
    out = plan.run(q, k, v, cu)  # (nothing between the two, which would keep them apart)
    end.record()
    assert plan.status() == 0 and long.status() == 0
    assert start.elapsed_time(end) > 1.5  # (the budget had time to run out)
    want_prompt(q, k, v, [150], [150], True, None, "f16").check(out)


@pytest.mark.parametrize("queries", [100, 200])
def test_a_short_budget_covers_a_long_item(queries):
    """Some waits last as long as an item does, in which every single hand-over is quick."""
    plan, args = one_long_item(queries)
    want = plan.run(*args)
    assert plan.status() == 0
    plan.set_wait_budget(1_000_000)
    out = plan.run(*args)
    assert plan.status() == 0
    assert torch.equal(out, want)


# ------------------------------------------------------------------- gradients
def test_inputs_that_require_a_gradient_are_refused():
    """The results have none; without grad mode the inputs may be parameters."""
    q, k, v, cu = normal(1, 9, 4, 64), normal(2, 9, 2, 64), normal(3, 9, 2, 64), ints([0, 9])
    cache, lengths = normal(4, 3, 16, 2, 64), ints([1, 2, 3])
    prompt, shared = b2b.PromptAttentionPlan("f16", 4, 2, 64), b2b.SharedPrefixAttentionPlan("f16", 4, 2, 64)
    for plan, args, floats in ((prompt, (q, k, v, cu), 3), (shared, (q, k, v, cache, cache.clone(), lengths), 5)):
        want = plan.run(*args)
        for i in range(floats):
            leaf = args[:i] + (args[i].clone().requires_grad_(),) + args[i + 1:]
            for kw in ({}, {"out": torch.empty_like(q)}, {"stream": torch.cuda.Stream()}):
                with pytest.raises(RuntimeError, match="no_grad"):
                    plan.run(*leaf, **kw)
            with torch.no_grad():
                assert torch.equal(plan.run(*leaf), want)
        assert plan.status() == 0


# --------------------------------------------------------------------- scales
@pytest.mark.parametrize("scale", [1e-30, 1e-3, 20.0])
def test_small_and_large_scales(scale):
    prompt_case("f16", 4, 2, 64, [150], scale=scale)


# ------------------------------------------------- the C functions' own checks
def test_counts_and_lse_off_their_alignment_are_refused():
    """Arrays of 32-bit values at odd addresses: refused before anything is launched."""
    q, k, v, cu = normal(1, 9, 4, 64), normal(2, 9, 2, 64), normal(3, 9, 2, 64), ints([0, 9, 9])
    out, lse, cache = torch.empty_like(q), torch.empty(10, 4, device="cuda"), normal(4, 9, 16, 2, 64)
    lengths, table = ints([1] * 10), ints([[0]] * 10)

    def rows(t):
        return t.data_ptr(), t.stride(-3), t.stride(-2), t.stride(0) if t.dim() == 4 else 0

    prompt, shared = b2b.PromptAttentionPlan("f16", 4, 2, 64), b2b.SharedPrefixAttentionPlan("f16", 4, 2, 64)
    for at in range(3):
        for off in (1, 2, 3):
            p = [cu.data_ptr(), cu.data_ptr(), lse.data_ptr()]
            p[at] += off
            run = (ctypes.c_int64 * 25)(1, 9, 9, 1, *rows(q), *rows(k), *rows(v), *rows(out), *p, 0, 0)
            assert b2b.b2b_prompt_attention_run(prompt._h, run, None) == ALIGNMENT
            p = [lengths.data_ptr(), table.data_ptr(), lse.data_ptr()]
            p[at] += off
            run = (ctypes.c_int64 * 35)(9, 1, 9, 16, 9, 1, *rows(q), *rows(k), *rows(v), *rows(cache), *rows(cache),
                                        *rows(out), *p, 0, 0)
            assert b2b.b2b_shared_attention_run(shared._h, run, None) == ALIGNMENT
    assert prompt.status() == 0 and shared.status() == 0


# ------------------------------------------------------------------- outputs
def test_an_output_between_the_inputs_columns():
    """Output and inputs as column ranges of one buffer, in any order: their rows alternate and do not overlap."""
    n, hq, hk, d = 150, 4, 2, 64
    widths = {"q": hq, "k": hk, "v": hk, "out": hq}
    plan = b2b.PromptAttentionPlan("bf16", hq, hk, d)
    for order in ("q k v out", "out q k v", "q out k v"):
        names = order.split()
        both = normal(5, n, sum(widths.values()) * d, dtype="bf16")
        t = dict(zip(names, (x.unflatten(1, (-1, d)) for x in both.split([widths[x] * d for x in names], 1))))
        want = want_prompt(t["q"], t["k"], t["v"], [n], [n], True, None, "bf16")
        keep = {x: t[x].clone() for x in "qkv"}
        want.check(plan.run(t["q"], t["k"], t["v"], ints([0, n]), out=t["out"]))
        assert all(torch.equal(keep[x], t[x]) for x in "qkv")


def test_outputs_that_overlap_an_input_are_refused():
    n, d = 20, 64
    both = normal(6, n + 2, 16, d)
    plan = b2b.PromptAttentionPlan("f16", 4, 2, d)
    k, v = normal(2, n, 2, d), normal(3, n, 2, d)
    q = both[1:n + 1, 4:8]
    for out in (q, both[:n, 4:8], both[2:, 4:8], both[1:n + 1, 3:7], both[1:n + 1, 5:9], both[1:n + 1, 1:5],
                both[:n, 7:11], both[2:, 1:5]):
        with pytest.raises(b2b.B2BError) as e:
            plan.run(q, k, v, ints([0, n]), out=out)
        assert e.value.code == ALIAS


def test_overlaps_by_their_elements():
    """Outputs and queries anywhere in one buffer: refused where an element is in both, run where rows an equal stride
    apart have none in common."""
    import random
    r, n, hq, d = random.Random(0), 5, 2, 8
    plan = b2b.PromptAttentionPlan("f16", hq, 1, d)
    k, v, cu = normal(2, n, 1, d), normal(3, n, 1, d), ints([0, n])
    buffer, at = normal(6, 60 * d), torch.arange(60 * d)
    seen = {True: 0, False: 0}
    for _ in range(300):
        step = [r.choice([2, 3, 4, 5, 6]) for _ in range(2)]
        if r.random() < 0.7:
            step[1] = step[0]
        where = [(r.randrange(60 - (n - 1) * s - hq), s) for s in step]
        out, q = (buffer.as_strided((n, hq, d), (s * d, d, 1), o * d) for o, s in where)
        both = set.intersection(*(set(at.as_strided((n, hq, d), (s * d, d, 1), o * d).flatten().tolist()) for o, s in where))
        if both:
            with pytest.raises(b2b.B2BError) as e:
                plan.run(q, k, v, cu, out=out)
            assert e.value.code == ALIAS
        elif step[0] == step[1]:
            want = want_prompt(q.clone(), k, v, [n], [n], True, None, "f16")
            want.check(plan.run(q, k, v, cu, out=out))
        seen[bool(both)] += 1
    assert min(seen.values()) > 50


# --------------------------------------------------------------------- streams
@pytest.mark.parametrize("given", [False, True])
def test_inputs_freed_after_a_call_on_another_stream(given):
    """Memory of a call's inputs is not handed out anew before the call's stream has read it."""
    q, k, v, cu = normal(1, 4000, 4, 64), normal(2, 4000, 2, 64), normal(3, 4000, 2, 64), ints([0, 4000])
    cache, lengths = normal(4, 4000, 16, 2, 64), ints([16] * 4000)
    prompt, shared = b2b.PromptAttentionPlan("f16", 4, 2, 64), b2b.SharedPrefixAttentionPlan("f16", 4, 2, 64)
    side, busy = torch.cuda.Stream(), torch.randn(4096, 4096, device="cuda")
    for plan, args in ((prompt, (q, k, v, cu)), (shared, (q, k, v, cache, cache, lengths))):
        want = plan.run(*args)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            for _ in range(40):
                busy @ busy  # some tens of milliseconds
        kw = {"out": torch.empty_like(q)} if given else {}
        copies = [x.clone() for x in args]
        side.wait_stream(torch.cuda.current_stream())
        out = plan.run(*copies, stream=side, **kw)
        del copies
        for x in args:  # what the allocator hands out now
            y = torch.empty_like(x)
            y.fill_(math.nan if x.is_floating_point() else 0)
            del y
        fresh = [torch.empty_like(x).fill_(math.nan if x.is_floating_point() else 0) for x in args]
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        del fresh
        assert plan.status() == 0


def test_another_stream_within_a_capture():
    q, k, v, cu = normal(1, 300, 4, 64), normal(2, 300, 2, 64), normal(3, 300, 2, 64), ints([0, 120, 300])
    plan, side = b2b.PromptAttentionPlan("f16", 4, 2, 64), torch.cuda.Stream()
    want = plan.run(q, k, v, cu)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        inside = q * 1
        side.wait_stream(torch.cuda.current_stream())
        first = plan.run(inside, k, v, cu, stream=side)
        del inside
        torch.cuda.current_stream().wait_stream(side)
        second = plan.run(q, k, v, cu)
    for _ in range(3):
        first.zero_(), second.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, want) and torch.equal(second, want)
    assert plan.status() == 0


def test_rows_outside_every_sequence_are_left_alone_where_parts_are_joined():
    q, k, v = normal(1, 9, 4, 64), normal(2, 6000, 2, 64), normal(3, 6000, 2, 64)
    plan = b2b.PromptAttentionPlan("f16", 4, 2, 64)
    n = ctypes.c_size_t()
    assert b2b.b2b_prompt_attention_workspace(plan._h, 2, 9, 6000, 1, ctypes.byref(n)) == 0 and n.value > 0
    out, lse = torch.full_like(q, 5.0), torch.full((9, 4), 5.0, device="cuda")
    plan.run(q, k, v, ints([3, 5, 6]), ints([10, 3000, 5990]), out=out, lse=lse)
    assert plan.status() == 0
    for t in (out, lse):
        assert (t[:3] == 5).all() and (t[6:] == 5).all()
    want = want_prompt(q[3:6], k[10:5990], v[10:5990], [2, 1], [2990, 2990], True, None, "f16")
    want.check(out[3:6], lse[3:6])


def test_the_example_tells_the_status_that_it_saw(monkeypatch):
    """Reading the status clears it."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "shared_prompt.py")
    spec = importlib.util.spec_from_file_location("shared_prompt_status", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    answers = iter([TIMEOUT])
    monkeypatch.setattr(b2b.PromptAttentionPlan, "status", lambda self: next(answers, 0))
    with pytest.raises(RuntimeError, match=f"status {TIMEOUT}"):
        example.main(["--prompt", "50", "--answers", "2", "--tokens", "3"])
