"""Cases and plain forms of the attention operators.

Two operators, each a cascade of two GEMMs with a softmax between them,
``softmax(scale * Q K^T + mask) V``, for grouped heads (query head h reads
key/value head h // (q_heads / kv_heads)):

``prompt``
    whole prompts, packed one after the other: sequence b owns the query rows
    cu_q[b]..cu_q[b+1] and the key rows cu_k[b]..cu_k[b+1].  With ``causal``
    row i of a sequence sees its keys j <= i + (keys - queries): the last row
    sees every key, so new tokens can follow keys of an earlier call.
``shared``
    a batch of requests that share one long prefix, ``new`` tokens for each
    request: every row sees the whole prefix and, of the request's own keys
    (dense [batch][room] or in pages), those up to its own.  ``lengths`` counts
    a request's own keys, the new tokens' among them.

A row that sees no key gives zeros (and -inf as the logarithm of its sum).
``run`` computes a case in its plain form, in 32 bits with elementary torch
operations, or (``own``) through this package.
"""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _prompt(name, dtype, q_heads, kv_heads, dim, batch, shortest, longest, past_shortest=0, past_longest=0, causal=True,
            lse=False, lens=0):
    """past_*: keys of each sequence that come before its query rows' own."""
    return dict(name=name, op="prompt", dtype=dtype, q_heads=q_heads, kv_heads=kv_heads, dim=dim, batch=batch,
                shortest=shortest, longest=longest, past_shortest=past_shortest, past_longest=past_longest,
                causal=causal, lse=lse, lens=lens)


def _shared(name, dtype, q_heads, kv_heads, dim, batch, new, prefix, shortest, longest, page=0, lse=False, lens=0):
    """page: rows of a page of the requests' own keys, 0 for a dense cache."""
    return dict(name=name, op="shared", dtype=dtype, q_heads=q_heads, kv_heads=kv_heads, dim=dim, batch=batch, new=new,
                prefix=prefix, shortest=shortest, longest=longest, page=page, lse=lse, lens=lens)


def listed():
    return [
        # a chat turn of a few words, nothing else in the batch: latency
        _prompt("one short prompt", "f16", 8, 2, 64, 1, 19, 19),
        # what a server packs from its queue: prompts of one token to 700
        _prompt("ragged prompts", "bf16", 32, 8, 128, 24, 1, 700, lens=1),
        # an ordinary batch of full prompts
        _prompt("four prompts of 2048", "bf16", 32, 8, 128, 4, 2048, 2048),
        # one long document with small heads, its statistics kept for a later merge
        _prompt("one prompt of 12001", "f16", 16, 4, 64, 1, 12001, 12001, lse=True),
        # one long prompt, the largest case
        _prompt("one prompt of 8192", "bf16", 32, 8, 128, 1, 8192, 8192),
        # prompts taken in pieces: a piece of each after the keys of the earlier pieces; seven heads to a group
        _prompt("pieces after cached keys", "bf16", 28, 4, 128, 6, 200, 256, 1000, 6000, lens=2),
        # passages read in both directions by an encoder
        _prompt("passages both ways", "f16", 12, 12, 96, 16, 100, 512, causal=False, lse=True, lens=3),
        # a few samples of one short prompt: latency
        _shared("four samples", "f16", 8, 2, 64, 4, 1, 133, 1, 40, lens=4),
        # many samples of one prompt
        _shared("64 samples of 8192", "bf16", 32, 8, 128, 64, 1, 8192, 1, 512, lens=5),
        # questions about one very long document, answers in pages
        _shared("32 questions on 65521", "bf16", 32, 8, 128, 32, 1, 65521, 1, 700, page=64, lens=6),
        # drafted tokens checked five at a time
        _shared("drafts of five", "f16", 24, 3, 96, 16, 5, 4001, 5, 300, page=16, lse=True, lens=7),
        # a system prompt in front of 200 long conversations: their own keys outweigh it
        _shared("200 conversations", "bf16", 32, 8, 128, 200, 1, 1024, 100, 2000, page=32, lens=8),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        q_heads, kv_heads = rng.choice([(8, 8), (8, 2), (16, 16), (16, 4), (12, 4), (28, 4), (24, 3), (32, 8), (32, 4), (16, 1)])
        same = dict(dtype=rng.choice(["f16", "bf16", "bf16"]), q_heads=q_heads, kv_heads=kv_heads,
                    dim=rng.choice([64, 64, 80, 96, 128, 128, 128]), lse=rng.random() < 0.3, lens=rng.randrange(1 << 20))
        if rng.random() < 0.5:
            longest = _spread(rng, 1, 12001)
            past = _spread(rng, 1, 8192) if rng.random() < 0.3 else 0
            case = _prompt("", batch=_spread(rng, 1, 32), shortest=_spread(rng, 1, longest), longest=longest,
                           past_shortest=past // 4, past_longest=past, causal=rng.random() < 0.8, **same)
            plain = 4 * case["batch"] * q_heads * longest * (longest + past)
        else:
            new = rng.choice([1, 1, 1, 2, 5, 8])
            longest = _spread(rng, new, 2000)
            prefix = 0 if rng.random() < 0.1 else _spread(rng, 1, 65521)
            case = _shared("", batch=_spread(rng, 1, 256), new=new, prefix=prefix, shortest=_spread(rng, new, longest),
                           longest=longest, page=rng.choice([0, 0, 16, 32, 64, 128]), **same)
            plain = 4 * case["batch"] * q_heads * new * (prefix + longest)
        del case["name"]
        # (the plain form keeps every score of the padded batch in memory)
        if _cost(case) <= most and plain <= 16e9:
            return case


# ------------------------------------------------------------------ lengths
def _lengths(case):
    """Queries and keys (prompt), or own keys (shared), of each sequence."""
    r = random.Random(case["lens"])
    n = [r.randint(case["shortest"], case["longest"]) for _ in range(case["batch"])]
    n[r.randrange(len(n))] = case["longest"]
    if case["op"] == "shared":
        return n, None
    past = [r.randint(case["past_shortest"], case["past_longest"]) for _ in n]
    return n, [a + b for a, b in zip(n, past)]


def _seen(case):
    """Pairs of a query row and a key it sees, for one head."""
    n, keys = _lengths(case)
    if case["op"] == "shared":
        t = case["new"]
        return sum(t * case["prefix"] + sum(max(0, m - t + 1 + i) for i in range(t)) for m in n)
    if not case["causal"]:
        return sum(a * b for a, b in zip(n, keys))
    return sum(a * (b - a) + a * (a + 1) // 2 for a, b in zip(n, keys))


def work(case):
    n, keys = _lengths(case)
    d, hq, hk = case["dim"], case["q_heads"], case["kv_heads"]
    if case["op"] == "prompt":
        rows, kv = sum(n), sum(keys)
    else:
        rows, kv = case["batch"] * case["new"], case["prefix"] + sum(n)
    moved = 2 * d * (2 * rows * hq + 2 * kv * hk) + (4 * rows * hq if case["lse"] else 0)
    return {"bytes": moved, "flops": 4 * d * hq * _seen(case)}


# ------------------------------------------------------------------- inputs
def _cumulative(n):
    c = [0]
    for x in n:
        c.append(c[-1] + x)
    return torch.tensor(c, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    """Activations of unit size; a head's queries lean one way and a sequence's first key answers to it, so that it
    draws weight from every row as first tokens do."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt, d, hq, hk = TYPES[case["dtype"]], case["dim"], case["q_heads"], case["kv_heads"]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    lean = 0.5 * normal(hk, 1, d)
    n, keys = _lengths(case)
    s = {"case": case}
    if case["op"] == "prompt":
        rows, kv = sum(n), sum(keys)
        q = normal(rows, hk, hq // hk, d) + lean
        k = normal(kv, hk, d)
        first = _cumulative(keys)[:-1].long()
        k[first] = 2 * lean[:, 0]
        if rows == kv:  # one projection gives all three, side by side
            both = torch.cat([q.reshape(rows, hq * d), k.reshape(rows, hk * d), normal(rows, hk * d)], 1).to(dt)
            s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in both.split([hq * d, hk * d, hk * d], 1))
        else:
            s["q"], s["k"], s["v"] = q.reshape(rows, hq, d).to(dt), k.to(dt), normal(kv, hk, d).to(dt)
        s["cu_q"], s["cu_k"] = _cumulative(n), _cumulative(keys)
    else:
        b, t = case["batch"], case["new"]
        s["q"] = (normal(b * t, hk, hq // hk, d) + lean).reshape(b * t, hq, d).to(dt)
        k = normal(case["prefix"], hk, d)
        k[:1] = 2 * lean[:, 0]
        s["prefix_k"], s["prefix_v"] = k.to(dt), normal(case["prefix"], hk, d).to(dt)
        s["lengths"] = torch.tensor(n, dtype=torch.int32, device="cuda")
        if case["page"]:  # pages handed out in no order; entries past a request's last page stay unset
            page = case["page"]
            each = [-(-m // page) for m in n]
            pool = sum(each) + 7
            order = torch.randperm(pool, generator=g, device="cuda").to(torch.int32)
            table = torch.full((b, max(each)), -1, dtype=torch.int32)
            at = torch.tensor([0] + each).cumsum(0)
            place = torch.arange(max(each))[None] < torch.tensor(each)[:, None]
            table[place] = order.cpu()[: int(at[-1])]
            s["table"] = table.cuda()
            s["cache_k"], s["cache_v"] = normal(pool, page, hk, d).to(dt), normal(pool, page, hk, d).to(dt)
        else:
            s["table"] = None
            room = -(-case["longest"] // 64) * 64
            s["cache_k"], s["cache_v"] = normal(b, room, hk, d).to(dt), normal(b, room, hk, d).to(dt)
    if own:
        import fusion_b2b_gemm_gb300 as b2b
        kind = b2b.PromptAttentionPlan if case["op"] == "prompt" else b2b.SharedPrefixAttentionPlan
        s["plan"] = kind(case["dtype"], hq, hk, d)
    return s


# -------------------------------------------------------------- plain forms
def _attend(q, k, v, see):
    """q [b, hk, rows, d], k and v [b, hk, keys, d], see [b, 1, rows, keys]: outputs and log of sums, in 32 bits."""
    s = torch.matmul(q, k.transpose(-1, -2)).mul_(1 / math.sqrt(q.shape[-1]))
    s.masked_fill_(~see, -math.inf)
    m = s.amax(-1, keepdim=True).clamp_(min=torch.finfo(torch.float32).min)
    p = s.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v).div_(total)
    return torch.where(total > 0, o, 0.0), (total.log() + m)[..., 0].masked_fill(total[..., 0] == 0, -math.inf)


def _plain_prompt(s):
    case, cu_q, cu_k = s["case"], s["cu_q"].long(), s["cu_k"].long()
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    nq, nk = cu_q.diff(), cu_k.diff()
    lq, lk = case["longest"], max(_lengths(case)[1])
    i, j = torch.arange(lq, device="cuda"), torch.arange(lk, device="cuda")
    at_q = (cu_q[:-1, None] + i).clamp_(max=s["q"].shape[0] - 1)
    at_k = (cu_k[:-1, None] + j).clamp_(max=s["k"].shape[0] - 1)
    b, group = nq.shape[0], hq // hk
    q = s["q"].float()[at_q].view(b, lq, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * lq, d)
    k, v = (s[x].float()[at_k].transpose(1, 2) for x in "kv")
    see = (j < nk[:, None])[:, None, :].expand(b, lq, lk)
    if case["causal"]:
        see = see & (j <= i[:, None] + (nk - nq)[:, None, None])
    o, lse = _attend(q, k, v, see[:, None, None].expand(b, 1, group, lq, lk).reshape(b, 1, group * lq, lk))
    row = torch.arange(s["q"].shape[0], device="cuda")
    seq = torch.searchsorted(cu_q[1:], row, right=True)
    o = o.view(b, hq, lq, d)[seq, :, row - cu_q[seq]]
    lse = lse.view(b, hq, lq)[seq, :, row - cu_q[seq]]
    return o, lse


def _plain_shared(s):
    case = s["case"]
    b, t, hq, hk, d = case["batch"], case["new"], case["q_heads"], case["kv_heads"], case["dim"]
    group = hq // hk
    if s["table"] is None:
        k, v = s["cache_k"].float(), s["cache_v"].float()
    else:
        at = s["table"].long().clamp(min=0)
        k, v = (s[x][at].flatten(1, 2).float() for x in ("cache_k", "cache_v"))
    k, v = ((torch.cat([s[p].float().expand(b, -1, -1, -1), x], 1).transpose(1, 2)
             for p, x in (("prefix_k", k), ("prefix_v", v))))
    q = s["q"].float().view(b, t, hk, group, d).permute(0, 2, 3, 1, 4).reshape(b, hk, group * t, d)
    j = torch.arange(k.shape[2], device="cuda")
    last = case["prefix"] + s["lengths"][:, None] - t + torch.arange(t, device="cuda")
    see = (j <= last[..., None])[:, None, None].expand(b, 1, group, t, -1).reshape(b, 1, group * t, -1)
    o, lse = _attend(q, k, v, see)
    return o.view(b, hk, group, t, d).permute(0, 3, 1, 2, 4).reshape(b * t, hq, d), \
        lse.view(b, hk, group, t).permute(0, 3, 1, 2).reshape(b * t, hq)


def run(s):
    case = s["case"]
    if own:
        if case["op"] == "prompt":
            return s["plan"].run(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"], return_lse=case["lse"])
        return s["plan"].run(s["q"], s["prefix_k"], s["prefix_v"], s["cache_k"], s["cache_v"], s["lengths"],
                             page_table=s["table"], return_lse=case["lse"])
    o, lse = _plain_prompt(s) if case["op"] == "prompt" else _plain_shared(s)
    o = o.to(TYPES[case["dtype"]])
    return (o, lse) if case["lse"] else o


# ---------------------------------------------------------------- in 64 bits
def exact(case, seed):
    """Every sequence and head by itself, in 64 bits."""
    if 4 * case["dim"] * case["q_heads"] * _seen(case) > 4e12:
        return None
    s = prepare(case, seed)
    hq, hk, d = case["q_heads"], case["kv_heads"], case["dim"]
    n, keys = _lengths(case)
    o = torch.zeros(s["q"].shape[0], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["q"].shape[0], hq), -math.inf, dtype=torch.float64, device="cuda")
    row = key = 0
    for b in range(case["batch"]):
        if case["op"] == "prompt":
            rows, k, v = n[b], s["k"][key:key + keys[b]], s["v"][key:key + keys[b]]
            ends = [keys[b] - rows + i + 1 if case["causal"] else keys[b] for i in range(rows)]
            key += keys[b]
        else:
            rows = case["new"]
            if s["table"] is None:
                mine = [s[x][b, :n[b]] for x in ("cache_k", "cache_v")]
            else:
                pages = s["table"][b, : -(-n[b] // case["page"])].long()
                mine = [s[x][pages].flatten(0, 1)[:n[b]] for x in ("cache_k", "cache_v")]
            k, v = torch.cat([s["prefix_k"], mine[0]]), torch.cat([s["prefix_v"], mine[1]])
            ends = [case["prefix"] + n[b] - rows + i + 1 for i in range(rows)]
        ends = torch.tensor(ends, device="cuda")
        hidden = torch.arange(k.shape[0], device="cuda")[None] >= ends[:, None]
        for h in range(hq):
            kh, vh = k[:, h // (hq // hk)].double(), v[:, h // (hq // hk)].double()
            x = s["q"][row:row + rows, h].double() @ kh.T / math.sqrt(d)
            x.masked_fill_(hidden, -math.inf)
            some = ends > 0
            lse[row:row + rows, h] = torch.logsumexp(x, 1)
            o[row:row + rows, h][some] = torch.softmax(x[some], 1) @ vh
        row += rows
    return (o, lse) if case["lse"] else o
