"""Speculative decoding with a drafted chain per request, on a one-layer attention model of random
weights: cache write, tree attention, verification and cache move as a serving loop calls them.

The target is embedding + attention over the paged cache -> lm_head; the draft (the student) reads
the embedding alone.  The share of accepted first tokens is compared with 1 - tvd of the two
distributions, from the loss's own forward: the quantity the CE + TVD distillation drives.

    python examples/speculative_step.py [--cache e4m3] [--steps 4]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from distillation_ce_tvd_gb300 import binding, speculative  # noqa: E402


class Model:
    """Random weights; ``draft_logits`` see one token, ``logits`` its request's history."""

    def __init__(self, vocab, dim, q_heads, kv_heads, head_dim, gen, device):
        def w(*shape):
            return (torch.randn(shape, generator=gen, device=device) * shape[-1] ** -0.5).to(torch.bfloat16)
        self.q_heads, self.kv_heads, self.head_dim = q_heads, kv_heads, head_dim
        self.embed = w(vocab, dim) * 8
        self.w_qkv = w((q_heads + 2 * kv_heads) * head_dim, dim)
        self.w_out = w(dim, q_heads * head_dim)
        self.head = w(vocab, dim)

    def draft_logits(self, tokens):
        return binding.fct_gemm_bf16(self.embed[tokens], self.head, out_dtype=torch.bfloat16)

    def qkv(self, tokens):
        y = binding.fct_gemm_bf16(self.embed[tokens], self.w_qkv, out_dtype=torch.bfloat16)
        y = y.view(tokens.shape[0], -1, self.head_dim)
        return y.split([self.q_heads, self.kv_heads, self.kv_heads], 1)

    def logits(self, tokens, attended):
        mixed = binding.fct_gemm_bf16(attended.flatten(1), self.w_out, out_dtype=torch.bfloat16)
        return binding.fct_gemm_bf16(self.embed[tokens] + 12 * mixed, self.head, out_dtype=torch.bfloat16)


def new_cache(kind, pages, page, heads, dim, device):
    shape = (pages, page, heads, dim)
    if kind == "bf16":
        return binding.KVCache(*(torch.zeros(shape, dtype=torch.bfloat16, device=device) for _ in "kv"))
    pools = [torch.zeros(shape, dtype=torch.float8_e4m3fn, device=device) for _ in "kv"]
    scales = [torch.zeros(shape[:3], dtype=torch.uint8, device=device) for _ in "kv"]
    return binding.KVCache(*pools, *scales)


def run(batch=64, prompt=50, steps=4, drafted=4, vocab=4096, page=16, kind="bf16", seed=0,
        device="cuda:0"):
    """{"accepted": share of accepted first drafted tokens, "expected": mean 1 - tvd, "checked": how
    many, "tokens": (batch, generated) lists}."""
    gen = torch.Generator(device=device).manual_seed(seed)
    model = Model(vocab, 512, 8, 2, 64, gen, device)
    width = -(-(prompt + steps * (drafted + 1)) // page) + 1
    order = torch.randperm(batch * width, generator=gen, device=device)
    table = order.view(batch, width).to(torch.int32)
    cache = new_cache(kind, batch * width, page, 2, 64, device)
    status = torch.zeros(1, dtype=torch.int32, device=device)
    i32 = dict(dtype=torch.int32, device=device)

    # the prompts: keys and values of all but the last token, which is each request's node 0
    history = torch.randint(0, vocab, (batch, prompt), generator=gen, device=device)
    context = torch.full((batch,), prompt - 1, **i32)
    starts = torch.arange(batch + 1, device=device) * (prompt - 1)
    _, k, v = model.qkv(history[:, :-1].flatten())
    slots = speculative.node_slots(table, torch.zeros(batch, **i32), starts.to(torch.int32),
                                   batch * (prompt - 1), page)
    binding.fct_kv_cache_write(cache, k, v, slots, dev_status=status)
    last = history[:, -1]

    nodes = drafted + 1
    starts = (torch.arange(batch + 1, device=device) * nodes).to(torch.int32)
    parent = torch.arange(-1, drafted, **i32).repeat(batch)
    mask = speculative.ancestor_mask([[-1] + list(range(drafted))] * batch, device)
    workspace = torch.empty(binding.fct_tree_attention_workspace_size(batch * nodes, 8, 2, 64),
                            dtype=torch.uint8, device=device)
    made, hits, expected = [[] for _ in range(batch)], 0, 0.0
    for _ in range(steps):
        # draft: a chain of tokens, each from the student's distribution after the one before
        chain, drafts = [last], []
        for _ in range(drafted):
            drafts.append(model.draft_logits(chain[-1]))
            race = torch.empty((batch, vocab), device=device).exponential_(generator=gen)
            chain.append((torch.softmax(drafts[-1].float(), -1) / race).argmax(-1))
        tokens = torch.stack(chain, 1).flatten()
        draft = torch.stack(drafts + [drafts[-1]], 1).flatten(0, 1)  # a leaf's row is not read
        # the target on all nodes
        q, k, v = model.qkv(tokens)
        binding.fct_kv_cache_write(
            cache, k, v, speculative.node_slots(table, context, starts, batch * nodes, page),
            dev_status=status)
        attended, _ = binding.fct_tree_attention(q, cache, table, context, starts, mask,
                                                 workspace=workspace, dev_status=status)
        target = model.logits(tokens, attended)
        # verification, and the accepted path kept
        uniform = torch.rand(batch * nodes, generator=gen, device=device)
        noise = torch.empty((batch, vocab), device=device).exponential_(generator=gen)
        out, _, count, context = speculative.commit(
            [cache], table, context, target, tokens, parent, starts, uniform, noise, draft,
            max_depth=drafted, dev_status=status)
        first = torch.arange(batch, device=device) * nodes
        _, tvd, *_ = binding.fused_ce_tvd_forward(draft[first], target[first], tokens[first + 1])
        expected += float((1 - tvd).sum())
        hits += int((count > 0).sum())
        for b, (row, n) in enumerate(zip(out.tolist(), count.tolist())):
            made[b] += row[:n + 1]
        last = out.gather(1, count.long()[:, None])[:, 0]
    if status.item() != 0:
        raise RuntimeError(f"device status {status.item()}")
    n = batch * steps
    return {"accepted": hits / n, "expected": expected / n, "checked": n, "tokens": made,
            "context": context.tolist()}


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--cache", choices=("bf16", "e4m3"), default="bf16")
    ap.add_argument("--steps", type=int, default=4)
    ap.add_argument("--batch", type=int, default=64)
    a = ap.parse_args()
    r = run(batch=a.batch, steps=a.steps, kind=a.cache)
    mean = sum(map(len, r["tokens"])) / len(r["tokens"]) / a.steps
    print(f"first drafted token accepted: {r['accepted']:.3f} of {r['checked']}, 1 - tvd: "
          f"{r['expected']:.3f}; tokens per request and step: {mean:.2f}")


if __name__ == "__main__":
    main()
