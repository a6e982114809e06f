"""The four operators together, as a serving loop calls them."""
import importlib.util
import math
import os

import pytest
import torch

import spec_util as su
from distillation_ce_tvd_gb300 import binding, speculative

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    path = os.path.join(ROOT, "examples", "speculative_step.py")
    spec = importlib.util.spec_from_file_location("speculative_step", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_first_tokens_are_accepted_as_often_as_the_tvd_says(kind):
    r = example().run(batch=256, steps=4, kind=kind, seed=3)
    # hits are independent with probability 1 - tvd each: 4.5 standard deviations at most
    sigma = math.sqrt(0.25 / r["checked"])
    assert abs(r["accepted"] - r["expected"]) < 4.5 * sigma
    assert 0.1 < r["expected"] < 0.95           # the case says something
    for tokens, context in zip(r["tokens"], r["context"]):
        assert context == 49 + len(tokens)      # prompt of 50, its last token the first node 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_an_accepted_path_lies_behind_the_context(kind):
    # after a step the cache holds, position by position, what was written for the accepted nodes
    gen = torch.Generator(device=DEV).manual_seed(5)
    heads, dim, page, depth, V = 2, 64, 16, 4, 97
    contexts, parents = [10, 31, 0], [[-1, 0, 0, 1, 2, 4, 5], [-1, 0, 1, 1, 3], [-1]]
    table, pages = su.make_tables([c + len(p) for c, p in zip(contexts, parents)], page,
                                  torch.Generator().manual_seed(5))
    cache = example().new_cache(kind, pages, page, heads, dim, DEV)
    starts = [0]
    for p in parents:
        starts.append(starts[-1] + len(p))
    i32 = dict(dtype=torch.int32, device=DEV)
    table, ctx, st = table.to(DEV), torch.tensor(contexts, **i32), torch.tensor(starts, **i32)
    n = starts[-1]
    k = torch.randn((n, heads, dim), generator=gen, device=DEV).to(torch.bfloat16)
    slots = speculative.node_slots(table, ctx, st, n, page)
    binding.fct_kv_cache_write(cache, k, k * 2, slots)
    written = su.values_of(cache.k, cache.k_scale).reshape(-1, heads, dim)[slots.cpu()]
    target = torch.randn((n, V), generator=gen, device=DEV)
    tokens = torch.randint(0, V, (n,), generator=gen, device=DEV)
    uniform = torch.zeros(n, device=DEV)        # every first child is accepted
    noise = torch.empty((3, V), device=DEV).exponential_(generator=gen)
    parent = torch.tensor([x for p in parents for x in p], **i32)
    out, path, count, new_ctx = speculative.commit([cache], table, ctx, target, tokens, parent, st,
                                                   uniform, noise, max_depth=depth)
    assert count.tolist() == [2, 2, 0]          # 0 -> 1 -> 3, and 0 -> 1 -> 2
    assert new_ctx.tolist() == [c + 1 + x for c, x in zip(contexts, count.tolist())]
    flat = su.values_of(cache.k, cache.k_scale)
    for b in range(3):
        nodes = [0] + path[b, :int(count[b])].tolist()
        for j, node in enumerate(nodes):
            pos = contexts[b] + j
            assert torch.equal(flat[int(table[b, pos // page]), pos % page], written[starts[b] + node])


def test_masks_and_slots():
    mask = speculative.ancestor_mask([[-1, 0, 0, 2], [-1]], DEV)
    assert mask.tolist() == [[1], [3], [5], [13], [1]]
    long = speculative.ancestor_mask([[-1] + list(range(69))], DEV)
    assert long.shape == (70, 2) and long[69].tolist() == [-1, 63]
    with pytest.raises(ValueError):
        speculative.ancestor_mask([[-1, 1]], DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    slots = speculative.node_slots(torch.tensor([[7, 3], [1, -1]], **i32), torch.tensor([3, 0], **i32),
                                   torch.tensor([0, 2, 3], **i32), 3, 4)
    assert slots.tolist() == [31, 12, 4]
