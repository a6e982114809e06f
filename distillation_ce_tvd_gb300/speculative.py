"""What a speculative decoding loop needs around the library's four calls: where the drafted nodes
go in the cache, which nodes see which, and the order of the calls.

One step for a batch of requests, with a draft distilled by this package's loss:

1. draft: each request's tree of tokens below its last committed token (its node 0);
2. ``node_slots`` and ``binding.fct_kv_cache_write``: the nodes' keys and values go to the positions
   after the request's context;
3. ``binding.fct_tree_attention`` with ``ancestor_mask``: every node attends to the context and to
   the nodes above it, in every layer;
4. ``commit``: ``binding.fct_spec_verify`` on the target's logits of all nodes, and
   ``binding.fct_kv_cache_move`` of the accepted path in every layer's cache.

These are indexing helpers in torch (or plain lists), with no arithmetic of the operators in them.
"""
from __future__ import annotations

import torch

from . import binding


def ancestor_mask(parents, device, words: int | None = None) -> torch.Tensor:
    """``tree_mask`` of fct_tree_attention for one list of parents per request (indexes within the
    request, -1 for node 0): a node sees itself and the nodes above it."""
    most = max((len(p) for p in parents), default=0)
    words = words or max(1, -(-most // 64))
    rows = []
    for parent in parents:
        seen: list[int] = []
        for i, p in enumerate(parent):
            if p >= i:
                raise ValueError("a node's parent must have a lower index")
            seen.append((1 << i) | (seen[p] if p >= 0 else 0))
        for bits in seen:
            row = [(bits >> (64 * w)) & (2 ** 64 - 1) for w in range(words)]
            rows.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in row])
    return torch.tensor(rows, dtype=torch.int64, device=device).reshape(len(rows), words)


#: The slot of a node that has no place in the block table: past any pool, so that
#: fct_kv_cache_write skips the node and sets FCT_DEV_INDEX_OUT_OF_RANGE.
NO_SLOT = 2 ** 62


def node_slots(block_table: torch.Tensor, context_len: torch.Tensor, node_start: torch.Tensor,
               n_nodes: int, page_size: int) -> torch.Tensor:
    """The cache slots (page * page_size + offset) of all nodes: node i of request b is at position
    context_len[b] + i.  Nodes of no request, positions outside the table and entries without a page
    get NO_SLOT."""
    node = torch.arange(n_nodes, device=block_table.device)
    batch, width = block_table.shape
    if batch == 0 or width == 0:
        return torch.full_like(node, NO_SLOT)
    start = node_start.long()
    b = torch.searchsorted(start, node, right=True) - 1
    held = (b >= 0) & (b < batch)
    b = b.clamp(0, batch - 1)
    pos = context_len.long()[b] + node - start[b]
    held &= (pos >= 0) & (pos < width * page_size)
    page = block_table.long()[b, (pos // page_size).clamp(0, width - 1)]
    return torch.where(held & (page >= 0), page * page_size + pos % page_size, NO_SLOT)


def commit(caches, block_table, context_len, target_logits, tokens, parent, node_start, uniform,
           noise, draft_logits=None, temperature=None, *, max_depth, dev_status=None, stream=None):
    """Verify the drafted trees and keep what was accepted: (out_tokens, path, count, new
    context_len).  The accepted nodes' keys and values move behind the context in every cache of
    ``caches``; the last value of a request's out_tokens is its next node 0."""
    if stream is not None:
        return binding.on_stream(
            commit, stream, target_logits.get_device(), caches, block_table, context_len,
            target_logits, tokens, parent, node_start, uniform, noise, draft_logits, temperature,
            max_depth=max_depth, dev_status=dev_status)
    out, path, count = binding.fct_spec_verify(
        target_logits, tokens, parent, node_start, uniform, noise, draft_logits, temperature,
        max_depth=max_depth, dev_status=dev_status)
    for cache in caches:
        binding.fct_kv_cache_move(cache, block_table, context_len, path, count,
                                  dev_status=dev_status)
    has_nodes = (node_start[1:] > node_start[:-1]).to(torch.int32)
    return out, path, count, context_len + has_nodes + count
