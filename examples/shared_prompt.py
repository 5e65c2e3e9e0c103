"""Several answers to one prompt: prompt attention, then attention of the batch on the shared prefix.

One attention layer of grouped heads with random weights over random token
embeddings.  The prompt is read once (``PromptAttentionPlan``); its keys and
values are the prefix that all answers share.  Each answer then grows token by
token: its own keys and values go into pages handed out from a pool, and each
step attends the prefix, read once for the batch, and the answer's own tokens
(``SharedPrefixAttentionPlan``).  At the end every answer's outputs are
computed again as one whole sequence, prompt and answer, in one call.

    python examples/shared_prompt.py [--prompt 1000] [--answers 16] [--tokens 40]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import fusion_b2b_gemm_gb300 as b2b  # noqa: E402

PAGE = 16


class Layer:
    """Projections of one attention layer; q, k and v are views of one product."""

    def __init__(self, q_heads=8, kv_heads=2, head_dim=64, vocabulary=1000, seed=0):
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        width = q_heads * head_dim
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return (torch.randn(shape, generator=g, device="cuda") / shape[-2] ** 0.5).to(torch.bfloat16)

        self.embedding = normal(vocabulary, width) * vocabulary ** 0.5
        self.qkv, self.out = normal(width, width + 2 * kv_heads * head_dim), normal(width, width)

    def project(self, tokens):
        x = self.embedding[tokens] @ self.qkv
        w = self.kv_heads * self.head_dim
        return (y.unflatten(-1, (-1, self.head_dim)) for y in x.split([self.q_heads * self.head_dim, w, w], -1))

    def next_token(self, attended):
        return ((attended.flatten(-2) @ self.out) @ self.embedding.T).argmax(-1)


def answer(layer, prompt, answers, steps):
    """Token ids [answers, steps] and the attention outputs of the answers' tokens [answers, steps, heads, dim]."""
    heads = ("bf16", layer.q_heads, layer.kv_heads, layer.head_dim)
    prompt_plan, shared_plan = b2b.PromptAttentionPlan(*heads), b2b.SharedPrefixAttentionPlan(*heads)

    q, k, v = layer.project(prompt)
    ends = torch.tensor([0, len(prompt)], dtype=torch.int32, device="cuda")
    attended = prompt_plan.run(q, k, v, ends)

    # a first token of its own for each answer: the most likely ones
    scores = (attended[-1].flatten() @ layer.out) @ layer.embedding.T
    token = scores.topk(answers).indices

    each = -(-steps // PAGE)
    table = torch.randperm(answers * each, device="cuda", dtype=torch.int32).view(answers, each)
    shape = (answers * each, PAGE, layer.kv_heads, layer.head_dim)
    pages_k, pages_v = torch.empty(shape, dtype=k.dtype, device="cuda"), torch.empty(shape, dtype=k.dtype, device="cuda")
    lengths = torch.zeros(answers, dtype=torch.int32, device="cuda")
    tokens, outputs = [], []
    for step in range(steps):
        tokens.append(token)
        nq, nk, nv = layer.project(token)
        page = table[:, step // PAGE].long()
        pages_k[page, step % PAGE], pages_v[page, step % PAGE] = nk, nv
        lengths += 1
        outputs.append(shared_plan.run(nq, k, v, pages_k, pages_v, lengths, page_table=table))
        token = layer.next_token(outputs[-1])
    for plan in (prompt_plan, shared_plan):
        status = plan.status()  # (cleared by reading it)
        if status != 0:
            raise RuntimeError(f"device status {status}")
    return torch.stack(tokens, 1), torch.stack(outputs, 1)


def again(layer, prompt, tokens):
    """The same outputs from whole sequences: prompt and answer, packed one after the other, in one call."""
    answers, steps = tokens.shape
    q, k, v = layer.project(torch.cat([prompt.expand(answers, -1), tokens], 1).flatten())
    ends = torch.arange(answers + 1, dtype=torch.int32, device="cuda") * (len(prompt) + steps)
    plan = b2b.PromptAttentionPlan("bf16", layer.q_heads, layer.kv_heads, layer.head_dim)
    out = plan.run(q, k, v, ends)
    return out.unflatten(0, (answers, -1))[:, len(prompt):]


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--prompt", type=int, default=1000)
    p.add_argument("--answers", type=int, default=16)
    p.add_argument("--tokens", type=int, default=40)
    a = p.parse_args(argv)
    layer = Layer()
    prompt = torch.randint(1000, (a.prompt,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    tokens, outputs = answer(layer, prompt, a.answers, a.tokens)
    whole = again(layer, prompt, tokens)
    off = ((outputs.float() - whole.float()).norm() / whole.float().norm()).item()
    print(f"{a.answers} answers of {a.tokens} tokens on a prompt of {a.prompt}: "
          f"token by token and as whole sequences, the outputs differ by {off:.1e} (relative norm)")
    return off


if __name__ == "__main__":
    main()
