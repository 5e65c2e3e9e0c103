"""Cases and plain forms of the feed-forward operators.

Four operators, a transformer block's feed-forward half in 16 and in 8 bits:

``ffn``
    the gated block, ``y = (act(x Wg) * (x Wu)) Wd``, x [tokens][width],
    Wg and Wu [width][hidden], Wd [hidden][out];
``train``
    the same with its backward pass: y and, for a given gradient of y, the
    gradients of x and of the three weights;
``product``
    a matrix product of e4m3 operands, ``D = A B^T``, A [rows][k] with a scale
    for each 128 elements of a row, B [n][k] with one for each block of 128
    x 128;
``ffn8``
    the gated block with e4m3 weights in such blocks: x and the hidden
    activations are brought to e4m3 with a scale for each 128 of a row, the
    smallest power of two that leaves no magnitude above 448.

act is silu, ``g / (1 + exp(-g))``, or gelu in its tanh form.  ``run`` computes
a case in its plain form, in 32 bits with elementary torch operations, or
(``own``) through this package.
"""
import math
import random

import torch

own = False

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
E4M3 = torch.float8_e4m3fn
BLOCK = 128


def _ffn(name, op, dtype, tokens, width, hidden, out, act="silu"):
    return dict(name=name, op=op, dtype=dtype, tokens=tokens, width=width, hidden=hidden, out=out, act=act)


def _product(name, dtype, rows, k, n):
    """dtype: of the result."""
    return dict(name=name, op="product", dtype=dtype, tokens=rows, width=k, out=n)


def listed():
    return [
        # a small model answers one request: latency
        _ffn("one token, small block", "ffn", "f16", 1, 1024, 2816, 1024),
        # one request, a large block: the weights' bytes
        _ffn("one token, large block", "ffn", "bf16", 1, 4096, 14336, 4096),
        # the running requests of a server, a token each
        _ffn("33 requests", "ffn", "f16", 33, 2048, 5632, 2048, "gelu"),
        # a full prompt
        _ffn("prompt of 4096", "ffn", "bf16", 4096, 4096, 14336, 4096),
        # a step of a small model on what is left of a batch: odd sizes throughout
        _ffn("small odd step", "train", "f16", 77, 520, 1368, 264, "gelu"),
        # an ordinary step
        _ffn("step of 2048 tokens", "train", "bf16", 2048, 2048, 5632, 2048),
        # a step of a large block, the largest case
        _ffn("step of 8192 tokens", "train", "bf16", 8192, 4096, 14336, 4096),
        # a projection for the running requests
        _product("16 rows", "bf16", 16, 4096, 14336),
        # ragged in every extent: the last block of k has 80 elements, that of n 88
        _product("ragged product", "f16", 1000, 2000, 1368),
        # a projection of a long prompt
        _product("8192 rows", "bf16", 8192, 4096, 14336),
        # one request on 8-bit weights
        _ffn("one token in 8 bits", "ffn8", "bf16", 1, 4096, 14336, 4096),
        # a prompt on 8-bit weights
        _ffn("prompt of 2048 in 8 bits", "ffn8", "bf16", 2048, 4096, 14336, 4096),
    ]


def _spread(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 250)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["ffn", "train", "product", "ffn8"])
        dtype = rng.choice(["f16", "bf16"])
        tokens = _spread(rng, 1, 8192)
        step = 16 if op in ("product", "ffn8") else 8
        width, out = (step * _spread(rng, 256 // step, 4096 // step) for _ in range(2))
        hidden = step * _spread(rng, 256 // step, 14336 // step)
        if op == "product":
            case = _product("", dtype, tokens, width, hidden)
        else:
            case = _ffn("", op, dtype, tokens, width, hidden, out, rng.choice(["silu", "gelu"]))
        del case["name"]
        if _cost(case) <= most:
            return case


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    t, d, o = case["tokens"], case["width"], case["out"]
    if case["op"] == "product":
        scales = 4 * (t * _blocks(d) + _blocks(o) * _blocks(d))
        return {"bytes": t * d + o * d + scales + 2 * t * o, "flops": 2 * t * d * o}
    f = case["hidden"]
    weights, flops = 2 * d * f + f * o, 2 * t * (2 * d * f + f * o)
    if case["op"] == "ffn8":
        scales = 4 * (2 * _blocks(d) * _blocks(f) + _blocks(f) * _blocks(o))
        return {"bytes": weights + scales + 2 * t * (d + o), "flops": flops}
    if case["op"] == "ffn":
        return {"bytes": 2 * (weights + t * (d + o)), "flops": flops}
    return {"bytes": 2 * (2 * weights + t * (2 * d + 2 * o)), "flops": 3 * flops}


# ------------------------------------------------------------------- inputs
def _quantized_weight(w):
    """e4m3 [n][k] and the scale of each block, the largest magnitude over 448."""
    n, k = w.shape
    nb, kb = _blocks(n), _blocks(k)
    padded = torch.zeros(nb * BLOCK, kb * BLOCK, device=w.device)
    padded[:n, :k] = w
    tiles = padded.view(nb, BLOCK, kb, BLOCK)
    scale = tiles.abs().amax((1, 3)) / 448
    q = (tiles / scale[:, None, :, None]).view(nb * BLOCK, kb * BLOCK)[:n, :k]
    return q.clamp(-448, 448).to(E4M3).contiguous(), scale


def prepare(case, seed):
    """Activations as a norm leaves them, of unit size with a few channels that stand out; weights of unit gain."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    t, d, o = case["tokens"], case["width"], case["out"]
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    x = normal(t, d)
    x[:, :: max(1, d // 5)] *= 8
    s = {"case": case}
    if case["op"] == "product":
        s["a"], s["a_scale"] = _quantized(x)
        s["a"] = s["a"].to(E4M3)
        s["b"], s["b_scale"] = _quantized_weight(normal(o, d) / math.sqrt(d))
    else:
        f = case["hidden"]
        s["x"] = x.to(dt)
        if case["op"] == "ffn8":
            for name, n, k in (("gate", f, d), ("up", f, d), ("down", o, f)):
                s[name], s[name + "_scale"] = _quantized_weight(normal(n, k) / math.sqrt(k))
        else:
            for name, n, k in (("gate", f, d), ("up", f, d), ("down", o, f)):
                s[name] = (normal(k, n) / math.sqrt(k)).to(dt)
        if case["op"] == "train":
            s["dy"] = (0.05 * normal(t, o)).to(dt)
    if own:
        import fusion_b2b_gemm_gb300 as b2b
        if case["op"] == "product":
            s["plan"] = b2b.ScaledGemmPlan(case["dtype"], d, o)
        elif case["op"] == "ffn8":
            s["plan"] = b2b.ScaledFeedForwardPlan(case["dtype"], d, f, o, activation=case["act"])
        else:
            s["plan"] = b2b.GatedFeedForwardPlan(case["dtype"], d, f, o, activation=case["act"])
    return s


# -------------------------------------------------------------- plain forms
def _power(e):
    """2^e for -126 <= e <= 127, by its bits."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _quantized(x):
    """Values on the e4m3 grid (in x's type) and the power-of-two scale of each 128 of a row."""
    rows, k = x.shape
    kb = _blocks(k)
    padded = torch.zeros(rows, kb * BLOCK, dtype=x.dtype, device=x.device)
    padded[:, :k] = x
    tiles = padded.view(rows, kb, BLOCK)
    m, e = torch.frexp(tiles.abs().amax(2))  # m * 2^e, m in [1/2, 1); 448 = 7/8 * 2^9
    scale = _power((e - 9 + (m > 0.875)).clamp(min=-126))
    q = (tiles / scale[..., None]).to(E4M3).to(x.dtype)
    return q.view(rows, kb * BLOCK)[:, :k], scale


def _widened(q, scale, rows_of_block, dtype=torch.float32):
    """The values that q and its scales stand for."""
    n, k = q.shape
    full = scale.to(dtype).repeat_interleave(BLOCK, 1)[:, :k]
    if rows_of_block > 1:
        full = full.repeat_interleave(rows_of_block, 0)[:n]
    return q.to(dtype) * full


def _sigmoid(x):
    return 1 / (1 + torch.exp(-x))


def _act(g, act):
    if act == "silu":
        return g * _sigmoid(g)
    return g * _sigmoid(2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g))


def _act_slope(g, act):
    if act == "silu":
        s = _sigmoid(g)
        return s + g * s * (1 - s)
    c = 2 * math.sqrt(2 / math.pi)
    s = _sigmoid(c * (g + 0.044715 * g * g * g))
    return s + g * s * (1 - s) * c * (1 + 3 * 0.044715 * g * g)


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        if op == "product":
            return s["plan"].run(s["a"], s["a_scale"], s["b"], s["b_scale"])
        if op == "ffn8":
            return s["plan"].run(s["x"], s["gate"], s["gate_scale"], s["up"], s["up_scale"], s["down"], s["down_scale"])
        if op == "ffn":
            return s["plan"].run(s["x"], s["gate"], s["up"], s["down"])
        y, saved = s["plan"].forward(s["x"], s["gate"], s["up"], s["down"])
        return (y, *s["plan"].backward(s["dy"], s["x"], s["gate"], s["up"], s["down"], saved))
    dt = TYPES[case["dtype"]]
    if op == "product":
        a, b = _widened(s["a"], s["a_scale"], 1), _widened(s["b"], s["b_scale"], BLOCK)
        return torch.matmul(a, b.T).to(dt)
    if op == "ffn8":
        wg, wu, wd = (_widened(s[w], s[w + "_scale"], BLOCK).T for w in ("gate", "up", "down"))
        x = _widened(*_quantized(s["x"].float()), 1)
        h = _act(torch.matmul(x, wg), case["act"]) * torch.matmul(x, wu)
        return torch.matmul(_widened(*_quantized(h), 1), wd).to(dt)
    x, wg, wu, wd = (s[w].float() for w in ("x", "gate", "up", "down"))
    gate, up = torch.matmul(x, wg), torch.matmul(x, wu)
    active = _act(gate, case["act"])
    h = active * up
    y = torch.matmul(h, wd).to(dt)
    if op == "ffn":
        return y
    dy = s["dy"].float()
    dh = torch.matmul(dy, wd.T)
    d_up, d_gate = dh * active, dh * up * _act_slope(gate, case["act"])
    dx = torch.matmul(d_gate, wg.T) + torch.matmul(d_up, wu.T)
    return y, *(z.to(dt) for z in (dx, torch.matmul(x.T, d_gate), torch.matmul(x.T, d_up), torch.matmul(h.T, dy)))


# ---------------------------------------------------------------- in 64 bits
def _grid(v):
    """v rounded to the nearest e4m3 value, ties to even: steps of 2^-9 up to 2^-6, then of an eighth of the power below."""
    step = _power(torch.frexp(v.abs().clamp(min=2.0 ** -6))[1] - 4).double()
    return torch.round(v / step) * step


def _exact_quantized(x):
    out = torch.empty_like(x)
    for k in range(0, x.shape[1], BLOCK):
        part = x[:, k:k + BLOCK]
        top = part.abs().amax(1, keepdim=True)
        m, e = torch.frexp(top.clamp(min=448 * 2.0 ** -126) / 448)
        scale = _power(e - (m == 0.5).int()).double()
        out[:, k:k + BLOCK] = _grid(part / scale) * scale
    return out


def _exact_blocks(q, scale, rows):
    w = q.double()
    for i in range(scale.shape[0]):
        for j in range(scale.shape[1]):
            w[i * rows:(i + 1) * rows, j * BLOCK:(j + 1) * BLOCK] *= scale[i, j].double()
    return w


def exact(case, seed):
    if work(case)["flops"] > 1.2e13:
        return None
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        a = s["a"].double().clone()
        for j in range(s["a_scale"].shape[1]):
            a[:, j * BLOCK:(j + 1) * BLOCK] *= s["a_scale"][:, j:j + 1].double()
        return a @ _exact_blocks(s["b"], s["b_scale"], BLOCK).T

    def both(g):
        """The activation and its slope, from tanh: sigmoid(2 z) = (1 + tanh z) / 2."""
        if case["act"] == "silu":
            z, dz = g / 2, 0.5
        else:
            z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
            dz = math.sqrt(2 / math.pi) * (1 + 0.134145 * g ** 2)
        t = torch.tanh(z)
        return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * dz

    if op == "ffn8":
        wg, wu, wd = (_exact_blocks(s[w], s[w + "_scale"], BLOCK) for w in ("gate", "up", "down"))
        x = _exact_quantized(s["x"].double())
        return _exact_quantized(both(x @ wg.T)[0] * (x @ wu.T)) @ wd.T
    x, wg, wu, wd = (s[w].double() for w in ("x", "gate", "up", "down"))
    gate, up = x @ wg, x @ wu
    active, slope = both(gate)
    y = (active * up) @ wd
    if op == "ffn":
        return y
    dy = s["dy"].double()
    dh = dy @ wd.T
    d_gate, d_up = dh * up * slope, dh * active
    return y, d_gate @ wg.T + d_up @ wu.T, x.T @ d_gate, x.T @ d_up, (active * up).T @ dy
