"""Attention on packed prompts and on batches that share a prefix (needs a GB300).

Every case is compared with softmax(scale Q K^T + mask) V in 64 bits on the
same 16-bit inputs.  The tolerance of each element follows from what the
kernel rounds.  With p_j the weights (sum 1), u the unit roundoff of the
operand type (bf16 2^-8, fp16 2^-11):

* P is rounded to the operand type:            u * sum_j p_j |v_j|
* the output is rounded to it:                 u * |o|
* a score is a fp32 dot product of head_dim terms and two more fp32
  roundings, in error by at most d = (head_dim + 4) 2^-23 B with
  B = scale max_j sum |q||k_j|; a weight moves by a factor exp(+-2 d), and the
  exponential and the sums add less than 2^-20:  (2 d + 2^-20) sum_j p_j |v_j|
* fp16 weights below 2^-14 are rounded to a multiple of 2^-24 (a row's sum is
  at least 1 in the kernel's units):            2^-25 sum_j |v_j|
* fp16 outputs likewise:                        2^-25

and the logarithm of the sum is off by d + 2^-20 (1 + |lse|).
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

b2b = pytest.importorskip("fusion_b2b_gemm_gb300")

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}
INVALID, UNSUPPORTED, ALIGNMENT, ALIAS, TIMEOUT = 1, 2, 3, 4, 7


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    torch.cuda.set_device(0)


def normal(seed, *shape, dtype="f16", scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (scale * torch.randn(shape, generator=g, device="cuda")).to(TYPES[dtype])


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cumulative(n):
    c = [0]
    for x in n:
        c.append(c[-1] + x)
    return ints(c)


class Want:
    """Outputs and tolerances in 64 bits, row by row of (token, head)."""

    def __init__(self, tokens, heads, dim):
        z = dict(dtype=torch.float64, device="cuda")
        self.o, self.tol = torch.zeros(tokens, heads, dim, **z), torch.zeros(tokens, heads, dim, **z)
        self.lse, self.lse_tol = torch.full((tokens, heads), -math.inf, **z), torch.zeros(tokens, heads, **z)

    def rows(self, first, q, k, v, ends, scale, dtype):
        """Rows first.. of q [rows, hq, d] over keys k, v [keys, hk, d], row i seeing the first ends[i]."""
        rows, hq, d = q.shape
        if rows == 0 or k.shape[0] == 0:
            return
        u, to = U[dtype], slice(first, first + rows)
        ends = torch.tensor(ends, device="cuda")
        none, hidden = ends <= 0, torch.arange(k.shape[0], device="cuda") >= ends[:, None]
        for h in range(hq):
            g = h // (hq // k.shape[1])
            qh, kh, vh = q[:, h].double(), k[:, g].double(), v[:, g].double()
            x = (scale * (qh @ kh.T)).masked_fill(hidden, -math.inf)
            b = (scale * (qh.abs() @ kh.abs().T)).masked_fill(hidden, 0).amax(1)
            lse = torch.logsumexp(x, 1)
            p = torch.softmax(x, 1).masked_fill(none[:, None], 0)
            o, a, all_v = p @ vh, p @ vh.abs(), (~hidden).double() @ vh.abs()
            err = (d + 4) * 2.0 ** -23 * b
            small = 2.0 ** -25 if dtype == "f16" else 0.0
            self.o[to, h] = o
            self.tol[to, h] = (u + 2 * err + 2.0 ** -20)[:, None] * a + u * o.abs() + small * (all_v + 1)
            self.lse[to, h] = lse
            self.lse_tol[to, h] = err + 2.0 ** -20 * (1 + lse.abs())

    def check(self, out, lse=None):
        out = out.double()
        assert torch.isfinite(out).all()
        over = ((out - self.o).abs() - self.tol).max().item()
        assert over <= 0, f"an output is {over:.3e} beyond its tolerance"
        if lse is not None:
            lse = lse.double()
            none = self.lse == -math.inf
            assert torch.equal(lse == -math.inf, none)
            over = ((lse - self.lse).abs() - self.lse_tol)[~none]
            assert over.numel() == 0 or over.max().item() <= 0


def prompt_case(dtype, hq, hk, d, nq, nk=None, causal=True, scale=None, seed=0, out=None, spread=1.0):
    nk = nq if nk is None else nk
    q = normal(seed, sum(nq), hq, d, dtype=dtype, scale=spread)
    k, v = normal(seed + 1, sum(nk), hk, d, dtype=dtype), normal(seed + 2, sum(nk), hk, d, dtype=dtype)
    plan = b2b.PromptAttentionPlan(dtype, hq, hk, d, scale)
    got, lse = plan.run(q, k, v, cumulative(nq), cumulative(nk), causal=causal, return_lse=True)
    assert plan.status() == 0
    want_prompt(q, k, v, nq, nk, causal, scale, dtype).check(got, lse)
    return got


def want_prompt(q, k, v, nq, nk, causal, scale, dtype):
    w = Want(q.shape[0], q.shape[1], q.shape[2])
    scale = 1 / math.sqrt(q.shape[2]) if scale is None else scale
    a = b = 0
    for n, m in zip(nq, nk):
        ends = [m - n + i + 1 if causal else m for i in range(n)]
        w.rows(a, q[a:a + n], k[b:b + m], v[b:b + m], ends, scale, dtype)
        a, b = a + n, b + m
    return w


# --------------------------------------------------------------------- prompts
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [8, 64, 72, 96, 128])
@pytest.mark.parametrize("heads", [(2, 2), (4, 1), (6, 2)], ids=str)
def test_prompts_by_type_head_size_and_group(dtype, dim, heads):
    prompt_case(dtype, *heads, dim, [1, 37, 130, 65])


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_around_the_tile_sizes(n, causal):
    prompt_case("bf16", 2, 1, 128, [n], causal=causal, seed=n)
    prompt_case("f16", 1, 1, 64, [n, 3], causal=causal, seed=n)


@pytest.mark.parametrize("group", [3, 5, 7, 8, 12, 16, 65, 128])
def test_groups_that_do_not_fill_a_tile(group):
    prompt_case("bf16", group, 1, 64, [5, 60, 1])


def test_empty_sequences_and_rows_that_see_no_key():
    # no queries, no keys, fewer keys than queries (the first rows see none)
    prompt_case("f16", 4, 2, 64, [0, 5, 9, 0, 140, 3], [7, 0, 4, 0, 133, 3])
    prompt_case("bf16", 4, 2, 128, [300, 1], [20, 0])
    prompt_case("bf16", 4, 2, 128, [3, 2], [0, 0], causal=False)


def test_nothing_to_do():
    plan = b2b.PromptAttentionPlan("f16", 4, 2, 64)
    e = torch.empty(0, 4, 64, dtype=torch.float16, device="cuda")
    assert plan.run(e, e[:, :2], e[:, :2], ints([0])).shape == (0, 4, 64)
    assert plan.run(e, e[:, :2], e[:, :2], ints([0, 0, 0])).shape == (0, 4, 64)


@pytest.mark.parametrize("nq,nk", [([1], [5000]), ([16], [3000]), ([4, 1], [2500, 1]), ([200], [1100]), ([1] * 3, [1025, 0, 2048])])
@pytest.mark.parametrize("dtype,dim", [("f16", 64), ("bf16", 128)])
def test_few_rows_over_many_keys_are_split_and_joined(dtype, dim, nq, nk):
    prompt_case(dtype, 4, 2, dim, nq, nk, seed=3)


def test_many_sequences():
    prompt_case("f16", 2, 1, 64, [(7 * i) % 23 for i in range(100)], seed=5)


@pytest.mark.parametrize("causal", [True, False])
def test_many_sequences_of_short_and_long_keys(causal):
    """Several items of every CTA, found from where the one before was, in sequences of one to twelve key tiles."""
    lens = [(37 * i) % 90 + (700 if i % 61 == 0 else 0) for i in range(300)]
    keys = [n + (800 if i % 53 == 0 else (11 * i) % 200) for i, n in enumerate(lens)]
    prompt_case("bf16", 4, 2, 64, lens, keys, causal=causal, seed=6)


@pytest.mark.parametrize("spread", [1e-3, 8.0, 40.0])
def test_flat_and_peaked_scores(spread):
    """Scores far apart move the running maximum by far more than the rescaling threshold."""
    prompt_case("bf16", 4, 2, 128, [400], seed=7, spread=spread)


def test_scores_that_rise_along_the_keys():
    """Every tile's maximum is above the one before: the accumulators are rescaled at every tile."""
    n, d = 900, 64
    q = torch.ones(n, 2, d, device="cuda", dtype=torch.float16)
    k = (torch.arange(n, device="cuda")[:, None, None] / 64).expand(n, 1, d).to(torch.float16).contiguous()
    v = normal(1, n, 1, d)
    plan = b2b.PromptAttentionPlan("f16", 2, 1, d)
    out = plan.run(q, k, v, ints([0, n]))
    want_prompt(q, k, v, [n], [n], True, None, "f16").check(out)


def test_scale_is_used():
    prompt_case("f16", 2, 2, 64, [150], scale=0.5)


def test_strided_views_of_one_projection():
    """Queries, keys and values as views of one buffer; an output with strides of its own."""
    n, hq, hk, d = 150, 4, 2, 96
    both = normal(11, n, (hq + 2 * hk) * d, dtype="bf16")
    q, k, v = (x.unflatten(1, (-1, d)) for x in both.split([hq * d, hk * d, hk * d], 1))
    out = torch.full((hq, n + 2, d + 8), 7.0, dtype=torch.bfloat16, device="cuda")
    view = out.permute(1, 0, 2)[1:n + 1, :, :d]
    plan = b2b.PromptAttentionPlan("bf16", hq, hk, d)
    assert plan.run(q, k, v, ints([0, n]), out=view) is view
    want_prompt(q, k, v, [n], [n], True, None, "bf16").check(view)
    assert (out[:, 0] == 7).all() and (out[:, n + 1:] == 7).all() and (out[:, :, d:] == 7).all()


def test_head_major_keys():
    n, d = 140, 64
    q, k, v = normal(1, 4, n, d).permute(1, 0, 2), normal(2, 2, n, d).permute(1, 0, 2), normal(3, 2, n, d).permute(1, 0, 2)
    plan = b2b.PromptAttentionPlan("f16", 4, 2, d)
    want_prompt(q, k, v, [n], [n], True, None, "f16").check(plan.run(q, k, v, ints([0, n])))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_other_sequences_and_masked_keys_do_not_leak(bad):
    """What lies past a sequence's keys is not read into its results, whatever it is."""
    nq, nk = [70, 30, 20], [75, 40, 20]
    q, k, v = normal(1, 120, 4, 128, dtype="bf16"), normal(2, 135, 2, 128, dtype="bf16"), normal(3, 135, 2, 128, dtype="bf16")
    k[75:115], v[75:115] = bad, bad
    q[70:100] = bad
    plan = b2b.PromptAttentionPlan("bf16", 4, 2, 128)
    for causal in (True, False):
        out = plan.run(q, k, v, cumulative(nq), cumulative(nk), causal=causal)
        want = want_prompt(q[:70], k[:75], v[:75], nq[:1], nk[:1], causal, None, "bf16")
        want.check(out[:70])
        want = want_prompt(q[100:], k[115:], v[115:], nq[2:], nk[2:], causal, None, "bf16")
        want.check(out[100:])
    # a key hidden by the causal mask may hold anything; rows that see it follow it
    k[:] = normal(2, 135, 2, 128, dtype="bf16")
    k[60], q[:] = bad, normal(1, 120, 4, 128, dtype="bf16")
    out = plan.run(q, k, v, cumulative(nq), cumulative(nk))
    want_prompt(q[:55], k[:60], v[:60], [55], [60], True, None, "bf16").check(out[:55])


def test_a_nan_in_a_query_stays_in_its_rows():
    q, k, v = normal(1, 64, 2, 64), normal(2, 64, 1, 64), normal(3, 64, 1, 64)
    q[10, 1, 5] = math.nan
    out = b2b.PromptAttentionPlan("f16", 2, 1, 64).run(q, k, v, ints([0, 64]))
    assert torch.isnan(out[10, 1]).all()
    out[10, 1] = 0
    assert torch.isfinite(out).all()


def test_rows_outside_every_sequence_are_left_alone():
    q, k, v = normal(1, 20, 2, 64), normal(2, 20, 2, 64), normal(3, 20, 2, 64)
    out = torch.full_like(q, 5.0)
    plan = b2b.PromptAttentionPlan("f16", 2, 2, 64)
    plan.run(q, k, v, ints([3, 9, 15]), out=out)
    assert (out[:3] == 5).all() and (out[15:] == 5).all()
    want = want_prompt(q[3:15], k[3:15], v[3:15], [6, 6], [6, 6], True, None, "f16")
    want.check(out[3:15])


def test_offsets_outside_the_tensors_are_clamped():
    q, k, v = normal(1, 20, 2, 64), normal(2, 20, 2, 64), normal(3, 20, 2, 64)
    plan = b2b.PromptAttentionPlan("f16", 2, 2, 64)
    out = plan.run(q, k, v, ints([-4, 9, 1000]))
    want_prompt(q, k, v, [9, 11], [9, 11], True, None, "f16").check(out)
    assert plan.status() == 0


def test_equal_inputs_give_equal_bits():
    q, k, v = normal(1, 600, 8, 128), normal(2, 600, 2, 128), normal(3, 600, 2, 128)
    plan = b2b.PromptAttentionPlan("f16", 8, 2, 128)
    first = plan.run(q, k, v, ints([0, 100, 600]))
    for _ in range(5):
        assert torch.equal(first, plan.run(q, k, v, ints([0, 100, 600])))


@pytest.mark.parametrize("heads", [(7, 1), (3, 1), (28, 4)], ids=str)
def test_equal_bits_whatever_ran_before(heads):
    """Groups that leave rows of a tile without a query, and one-token requests: what an earlier launch left in shared
    memory must not show, not even in the rounding."""
    hq, hk = heads
    q, k, v = normal(1, 300, hq, 128, scale=4.0), normal(2, 900, hk, 128), normal(3, 900, hk, 128)
    prompt, shared = b2b.PromptAttentionPlan("f16", hq, hk, 128), b2b.SharedPrefixAttentionPlan("f16", hq, hk, 128)
    cache = normal(4, 20, 400, hk, 128)
    n = ints([1 + 19 * i for i in range(20)])
    calls = [lambda: prompt.run(q, k, v, ints([0, 300]), ints([0, 900])),
             lambda: shared.run(q[:20], k, v, cache, cache, n),
             lambda: shared.run(q[:40], k[:70], v[:70], cache, cache, n)]
    first = [f() for f in calls]
    for i in range(30):
        noise = normal(10 + i, 2000, hq, 128, scale=30.0)
        prompt.run(noise, noise[:, :hk], noise[:, :hk], ints([0, 2000]))
        j = i % 3
        assert torch.equal(first[j], calls[j]())


def test_side_streams_and_capture():
    """Runs on streams of their own, and a captured run that follows the offsets' contents."""
    q, k, v = normal(1, 300, 4, 64), normal(2, 300, 2, 64), normal(3, 300, 2, 64)
    plan = b2b.PromptAttentionPlan("f16", 4, 2, 64)
    cu = ints([0, 120, 300])
    want = plan.run(q, k, v, cu)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [plan.run(q, k, v, cu, stream=s) for s in streams for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(want, o) for o in outs)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = plan.run(q, k, v, cu)
    for offsets in ([0, 120, 300], [0, 1, 300], [0, 300, 300]):
        cu.copy_(ints(offsets))
        g.replay()
        torch.cuda.synchronize()
        n = [offsets[1], offsets[2] - offsets[1]]
        want_prompt(q, k, v, n, n, True, None, "f16").check(out)


# --------------------------------------------------------------- shared prefix
def shared_case(dtype, hq, hk, d, prefix, lengths, fresh=1, page=0, seed=0, room=None, fill=None, scale=None):
    batch = len(lengths)
    q = normal(seed, batch * fresh, hq, d, dtype=dtype)
    pk, pv = normal(seed + 1, prefix, hk, d, dtype=dtype), normal(seed + 2, prefix, hk, d, dtype=dtype)
    room = max(lengths + [1]) if room is None else room
    if page:
        width = -(-room // page)
        pool = batch * width + 3
        table = torch.randperm(pool, generator=torch.Generator().manual_seed(seed))[:batch * width].view(batch, width).int()
        ck, cv = normal(seed + 3, pool, page, hk, d, dtype=dtype), normal(seed + 4, pool, page, hk, d, dtype=dtype)
        own = [(ck[table[b].long().cuda()].flatten(0, 1), cv[table[b].long().cuda()].flatten(0, 1)) for b in range(batch)]
        own = [(x.clone(), y.clone()) for x, y in own]
        if fill is not None:  # rows past every length, and pages no request owns
            keep_k, keep_v = ck.clone(), cv.clone()
            ck.fill_(fill)
            cv.fill_(fill)
            for b, n in enumerate(lengths):
                for j in range(n):
                    t = int(table[b, j // page])
                    ck[t, j % page], cv[t, j % page] = keep_k[t, j % page], keep_v[t, j % page]
            for b, n in enumerate(lengths):
                table[b, -(-n // page):] = 123456789 if b % 2 else -5
        table = table.cuda()
    else:
        table = None
        ck, cv = normal(seed + 3, batch, room, hk, d, dtype=dtype), normal(seed + 4, batch, room, hk, d, dtype=dtype)
        own = [(ck[b].clone(), cv[b].clone()) for b in range(batch)]
        if fill is not None:
            for b, n in enumerate(lengths):
                ck[b, n:], cv[b, n:] = fill, fill
    plan = b2b.SharedPrefixAttentionPlan(dtype, hq, hk, d, scale)
    got, lse = plan.run(q, pk, pv, ck, cv, ints(lengths), page_table=table, return_lse=True)
    assert plan.status() == 0
    w = Want(batch * fresh, hq, d)
    s = 1 / math.sqrt(d) if scale is None else scale
    for b, n in enumerate(lengths):
        for t in range(fresh):
            e = max(0, n - fresh + 1 + t)
            keys, values = torch.cat([pk, own[b][0][:e]]), torch.cat([pv, own[b][1][:e]])
            w.rows(b * fresh + t, q[b * fresh + t][None], keys, values, [prefix + e], s, dtype)
    w.check(got, lse)
    return got


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("dim", [8, 64, 72, 96, 128])
@pytest.mark.parametrize("heads", [(2, 2), (4, 1), (6, 2)], ids=str)
@pytest.mark.parametrize("page", [0, 16])
def test_shared_prefix_by_type_head_size_and_group(dtype, dim, heads, page):
    shared_case(dtype, *heads, dim, 150, [1, 40, 130], page=page)


@pytest.mark.parametrize("prefix", [0, 1, 127, 128, 129, 1000, 3001])
@pytest.mark.parametrize("page", [0, 16, 128])
def test_prefix_lengths(prefix, page):
    shared_case("bf16", 4, 2, 128, prefix, [1, 129, 5, 260], page=page, seed=prefix)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_pages_that_end_inside_and_past_a_tile(page):
    shared_case("f16", 4, 2, 64, 70, [page - 1, page, page + 1, 2 * page + 3, 300], page=page, fill=math.nan)


@pytest.mark.parametrize("fresh", [1, 2, 5, 17, 70])
@pytest.mark.parametrize("batch", [1, 3, 40])
def test_drafted_tokens(fresh, batch):
    """Several new tokens, more than a tile's or two tiles' rows among them."""
    lengths = [fresh + (13 * b) % 50 for b in range(batch)]
    shared_case("f16", 4, 1, 64, 200 if batch < 40 else 40, lengths, fresh=fresh, seed=fresh)


@pytest.mark.parametrize("page", [0, 32])
def test_requests_without_keys_and_shorter_than_their_tokens(page):
    # length 0; fewer own keys than new tokens: the first tokens see the prefix alone, or nothing
    for prefix in (0, 33):
        shared_case("bf16", 4, 2, 64, prefix, [0, 1, 3, 200], fresh=3, page=page, room=224)


@pytest.mark.parametrize("fill", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("page", [0, 64])
def test_what_lies_past_a_length_is_not_read(fill, page):
    shared_case("bf16", 8, 2, 128, 130, [1, 64, 100, 129], page=page, room=256, fill=fill)
    shared_case("f16", 8, 2, 64, 0, [1, 64, 100, 129], page=page, room=256, fill=fill)


def test_one_request_over_a_long_cache_is_split():
    shared_case("bf16", 8, 1, 128, 0, [5003])
    shared_case("f16", 8, 2, 64, 2000, [5003, 1], page=64)


def test_lengths_beyond_the_room_are_clamped():
    q, k, v = normal(1, 2, 2, 64), normal(2, 2, 40, 2, 64), normal(3, 2, 40, 2, 64)
    plan = b2b.SharedPrefixAttentionPlan("f16", 2, 2, 64)
    none = k[0, :0]
    out = plan.run(q, none, none, k, v, ints([1000, -3]))
    w = Want(2, 2, 64)
    w.rows(0, q[:1], k[0], v[0], [40], 1 / 8, "f16")
    w.check(out)
    assert plan.status() == 0


def test_a_pool_past_32_bit_offsets():
    """Pages whose element offsets pass 2^31 and byte offsets 2^32."""
    page, hk, d = 64, 8, 128
    pool = (1 << 31) // (page * hk * d) + 40
    ck, cv = (torch.empty(pool, page, hk, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = ints([[pool - 1, 3], [pool - 30, pool - 2]])
    for i, t in enumerate(table.flatten().tolist()):
        ck[t], cv[t] = normal(i, page, hk, d, dtype="bf16"), normal(50 + i, page, hk, d, dtype="bf16")
    q, pk = normal(90, 2, 16, d, dtype="bf16"), normal(91, 30, hk, d, dtype="bf16")
    plan = b2b.SharedPrefixAttentionPlan("bf16", 16, hk, d)
    out = plan.run(q, pk, pk, ck, cv, ints([100, 128]), page_table=table)
    w = Want(2, 16, d)
    for b, n in enumerate([100, 128]):
        k, v = (torch.cat([pk, x[table[b].long()].flatten(0, 1)[:n]]) for x in (ck, cv))
        w.rows(b, q[b:b + 1], k, v, [30 + n], d ** -0.5, "bf16")
    w.check(out)


def test_shared_capture_follows_lengths_and_pages():
    q, pk, pv = normal(1, 3, 4, 64), normal(2, 100, 2, 64), normal(3, 100, 2, 64)
    ck, cv = normal(4, 12, 16, 2, 64), normal(5, 12, 16, 2, 64)
    lengths, table = ints([1, 20, 33]), ints([[0, 1, 2], [3, 4, 5], [6, 7, 8]])
    plan = b2b.SharedPrefixAttentionPlan("f16", 4, 2, 64)
    plan.run(q, pk, pv, ck, cv, lengths, page_table=table)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = plan.run(q, pk, pv, ck, cv, lengths, page_table=table)
    for n, t in (([1, 20, 33], [[0, 1, 2], [3, 4, 5], [6, 7, 8]]), ([48, 2, 34], [[11, 10, 9], [8, 4, 5], [0, 1, 2]])):
        lengths.copy_(ints(n))
        table.copy_(ints(t))
        g.replay()
        torch.cuda.synchronize()
        w = Want(3, 4, 64)
        for b in range(3):
            k, v = (torch.cat([p, c[table[b].long()].flatten(0, 1)[:n[b]]]) for p, c in ((pk, ck), (pv, cv)))
            w.rows(b, q[b:b + 1], k, v, [100 + n[b]], 1 / 8, "f16")
        w.check(out)


def test_a_prompt_and_its_answers():
    """The prompt's keys become the prefix: its last row again, as a batch of one-token requests without own keys."""
    n, hq, hk, d = 333, 8, 2, 128
    q, k, v = normal(1, n, hq, d), normal(2, n, hk, d), normal(3, n, hk, d)
    prompt = b2b.PromptAttentionPlan("f16", hq, hk, d).run(q, k, v, ints([0, n]))
    empty = torch.empty(4, 0, hk, d, dtype=torch.float16, device="cuda")
    answers = b2b.SharedPrefixAttentionPlan("f16", hq, hk, d).run(q[-1:].expand(4, hq, d).contiguous(), k, v, empty, empty,
                                                                  ints([0] * 4))
    w = Want(4, hq, d)
    for b in range(4):
        w.rows(b, q[-1:], k, v, [n], d ** -0.5, "f16")
    w.check(answers)
    w.check(prompt[-1:].expand(4, hq, d))


# ------------------------------------------------------------ failure, refusals
def test_results_given_or_made_are_the_same():
    """Calls with tensors for the results are marshalled in Python, the others by the compiled module."""
    q, k, v = (normal(i, 150, h, 72, dtype="bf16") for i, h in ((1, 6), (2, 2), (3, 2)))
    cu = cumulative([40, 0, 110])
    plan = b2b.PromptAttentionPlan("bf16", 6, 2, 72)
    for causal in (True, False):
        made = plan.run(q, k, v, cu, causal=causal, return_lse=True)
        out, lse = torch.empty_like(q), torch.empty(150, 6, device="cuda")
        given = plan.run(q, k, v, cu, cu, causal, out=out, lse=lse)
        assert given[0] is out and given[1] is lse
        assert torch.equal(made[0], out) and torch.equal(made[1], lse)
        assert torch.equal(plan.run(q, k, v, cu, causal=causal), out)
    shared = b2b.SharedPrefixAttentionPlan("bf16", 6, 2, 72)
    pool = normal(4, 12, 16, 2, 72, dtype="bf16")
    table = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    lengths = torch.tensor([3, 64, 20], dtype=torch.int32, device="cuda")
    for prefix in (0, 150):
        args = (q[:6], k[:prefix], v[:prefix], pool, pool, lengths, table)
        made = shared.run(*args, return_lse=True)
        out, lse = torch.empty_like(q[:6]), torch.empty(6, 6, device="cuda")
        shared.run(*args, out=out, lse=lse)
        assert torch.equal(made[0], out) and torch.equal(made[1], lse)
        assert torch.equal(shared.run(*args), out)
    assert plan.status() == 0 and shared.status() == 0
    plan.close()
    with pytest.raises(b2b.B2BError):
        plan.run(q, k, v, cu)


@pytest.mark.parametrize("dim", [64, 128])
def test_timeout_is_reported_and_the_plan_recovers(dim):
    q, k, v = normal(1, 200, 4, dim), normal(2, 200, 2, dim), normal(3, 200, 2, dim)
    plan = b2b.PromptAttentionPlan("f16", 4, 2, dim)
    out = torch.zeros_like(q)
    plan.set_wait_budget(20_000_000)
    plan.set_debug(1)
    plan.run(q, k, v, ints([0, 200]), out=out)
    assert plan.status() == TIMEOUT
    assert torch.all(out == 0)
    assert plan.status() == 0
    plan.set_debug(0)
    plan.set_wait_budget(0)
    plan.run(q, k, v, ints([0, 200]), out=out)
    assert plan.status() == 0
    want_prompt(q, k, v, [200], [200], True, None, "f16").check(out)


def refused(error, match, f, *args, **kw):
    with pytest.raises(error, match=match):
        f(*args, **kw)


def test_prompt_refusals():
    plan = b2b.PromptAttentionPlan("f16", 4, 2, 64)
    q, k, v, cu = normal(1, 9, 4, 64), normal(2, 9, 2, 64), normal(3, 9, 2, 64), ints([0, 9])
    refused(TypeError, "q:", plan.run, q.float(), k, v, cu)
    refused(TypeError, "v:", plan.run, q, k, v.bfloat16(), cu)
    refused(ValueError, "k:", plan.run, q, normal(2, 9, 3, 64), v, cu)
    refused(ValueError, "q:", plan.run, q[..., :32], k, v, cu)
    refused(ValueError, "v:", plan.run, q, k, v[:8], cu)
    refused(ValueError, "consecutive", plan.run, normal(1, 4, 64, 9).permute(2, 0, 1), k, v, cu)
    refused(ValueError, "q is on cpu", plan.run, q.cpu(), k, v, cu)
    refused(ValueError, "cu_q is on cpu", plan.run, q, k, v, cu.cpu())
    refused(TypeError, "cu_q", plan.run, q, k, v, cu.long())
    refused(ValueError, "cu_k", plan.run, q, k, v, cu, ints([0, 4, 9]))
    refused(ValueError, "cu_q", plan.run, q, k, v, cu[:0])
    refused(ValueError, "out:", plan.run, q, k, v, cu, out=torch.empty_like(q)[:5])
    refused(TypeError, "lse", plan.run, q, k, v, cu, lse=torch.empty(9, 4, device="cuda", dtype=torch.float16))
    refused(ValueError, "lse", plan.run, q, k, v, cu, lse=torch.empty(4, 9, device="cuda"))
    for code, args, kw in (
            (ALIAS, (q, k, v, cu), {"out": q}),
            (ALIGNMENT, (normal(1, 9, 4, 68)[..., 4:], k, v, cu), {}),
            (ALIGNMENT, (normal(1, 9, 4, 68)[..., :64], k, v, cu), {}),
            (INVALID, (q, normal(2, 9, 1, 64).expand(9, 2, 64), v, cu), {})):
        with pytest.raises(b2b.B2BError) as e:
            plan.run(*args, **kw)
        assert e.value.code == code
    plan.run(q, k, v, cu)  # and is usable afterwards
    assert plan.status() == 0


def test_shared_refusals():
    plan = b2b.SharedPrefixAttentionPlan("bf16", 4, 2, 64)
    q, p = normal(1, 4, 4, 64, dtype="bf16"), normal(2, 9, 2, 64, dtype="bf16")
    c, n = normal(3, 2, 16, 2, 64, dtype="bf16"), ints([3, 4])
    refused(ValueError, "q:", plan.run, q[:3], p, p, c, c, n)
    refused(ValueError, "prefix_v", plan.run, q, p, p[:8], c, c, n)
    refused(ValueError, "cache_k", plan.run, q, p, p, c[0], c, n)
    refused(ValueError, "cache_v", plan.run, q, p, p, c, c[:, :8], n)
    refused(ValueError, "cache_k", plan.run, q, p, p, c[:1], c[:1], n)
    refused(ValueError, "page_table", plan.run, q, p, p, c, c, n, page_table=ints([[0]]))
    refused(TypeError, "page_table", plan.run, q, p, p, c, c, n, page_table=ints([[0], [1]]).long())
    refused(TypeError, "lengths", plan.run, q, p, p, c, c, n.long())
    refused(ValueError, "cache_k is on cpu", plan.run, q, p, p, c.cpu(), c, n)
    for code, args, kw in (
            (UNSUPPORTED, (q, p, p, c[:, :12], c[:, :12], n), {"page_table": ints([[0], [1]])}),
            (UNSUPPORTED, (q, p, p, c[:, :8], c[:, :8], n), {"page_table": ints([[0], [1]])}),
            (ALIAS, (q, p, p, c, c, n), {"out": q})):
        with pytest.raises(b2b.B2BError) as e:
            plan.run(*args, **kw)
        assert e.value.code == code
    plan.run(q, p, p, c, c, n)
    assert plan.status() == 0


def test_debug_flags_are_validated():
    plan = b2b.PromptAttentionPlan("f16", 4, 2, 64)
    with pytest.raises(b2b.B2BError) as e:
        plan.set_debug(2)
    assert e.value.code == INVALID


# ------------------------------------------------------------------- together
def test_the_example_runs_both_and_they_agree():
    """Both paths round P and the output to bf16, differently where they cut the keys: each to 2^-8 of the output's
    size at most, so together within 4 x 2^-8 in norm."""
    import os
    import sys
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    try:
        import shared_prompt
    finally:
        sys.path.pop(0)
    assert shared_prompt.main(["--prompt", "333", "--answers", "5", "--tokens", "20"]) <= 4 * U["bf16"]


def test_many_short_prompts_and_requests_at_once():
    """More sequences than a warp has lanes, some empty; more requests than SMs."""
    prompt_case("bf16", 2, 1, 128, [(5 * i) % 37 for i in range(70)], [(11 * i) % 53 for i in range(70)], seed=11)
    shared_case("f16", 2, 1, 64, 70, [1 + (17 * i) % 140 for i in range(200)], page=32, seed=12)


@pytest.mark.parametrize("seed", range(12))
def test_drawn_shapes(seed):
    import random
    r = random.Random(seed)
    hq, hk = r.choice([(4, 4), (6, 2), (8, 1), (7, 1)])
    dtype, dim = r.choice(["f16", "bf16"]), r.choice([40, 64, 80, 128])
    if seed % 2:
        nq = [r.choice([0, 1, r.randint(1, 300)]) for _ in range(r.randint(1, 9))]
        nk = [max(0, n + r.randint(-3, 400)) for n in nq]
        prompt_case(dtype, hq, hk, dim, nq, nk, causal=r.random() < 0.7, seed=seed)
    else:
        fresh = r.choice([1, 1, 2, 7])
        lengths = [r.randint(0, 400) for _ in range(r.randint(1, 20))]
        shared_case(dtype, hq, hk, dim, r.choice([0, 1, 130, 900]), lengths, fresh=fresh, page=r.choice([0, 16, 64]),
                    seed=seed, fill=math.nan)
