"""Tree attention on the GPU against attention in 64 bits.

Tolerances: scores are fp32 sums of exact products (relative error at most head_dim * 2^-24 of
sum |q||k|, under 2e-5 here, and as much in each weight's relative error); weights are rounded to
bf16 (2^-9 each) for the second product and the output once more (2^-9 of itself).  So an output is
within (2^-9 + 1e-4) * sum w|v| + 2^-9 |out|, taken with a factor 1.25, and lse within 1e-4.
"""
import math
import random

import pytest
import torch

import spec_util as su
from distillation_ce_tvd_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def case(contexts, nodes, q_heads, heads, dim, page, dtype=torch.bfloat16, layout="nhd", tree=True,
         seed=0, words=None, spread=1.0, pad=0):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    cpu, rnd = torch.Generator().manual_seed(seed), random.Random(seed)
    table, pages = su.make_tables([c + n for c, n in zip(contexts, nodes)], page, cpu)
    k, v, ks, vs = su.make_pool(pages, page, heads, dim, dtype, gen, DEV, layout)
    starts = [0]
    for n in nodes:
        starts.append(starts[-1] + n)
    q = torch.randn((starts[-1], q_heads, dim + pad), generator=gen, device=DEV) * spread
    q = q.to(torch.bfloat16)[..., :dim]
    mask = None
    if tree:
        parents = [su.random_tree(n, rnd) if n else [] for n in nodes]
        mask = su.ancestor_masks(parents, words or max(1, -(-max(nodes) // 64)))
    return dict(q=q, k=k, v=v, ks=ks, vs=vs, table=table, page=page, contexts=contexts,
                starts=starts, mask=mask)


def run(c, **kw):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    i32 = dict(dtype=torch.int32, device=DEV)
    out, lse = binding.fct_tree_attention(
        c["q"], binding.KVCache(c["k"], c["v"], c["ks"], c["vs"]), c["table"].to(DEV),
        torch.tensor(c["contexts"], **i32), torch.tensor(c["starts"], **i32),
        None if c["mask"] is None else c["mask"].to(DEV), dev_status=st, **kw)
    return out, lse, st.item()


def check(c, scale=None, **kw):
    out, lse, st = run(c, scale=scale, **kw)
    assert st == 0
    ref, ref_lse, bound = su.attention_ref(
        c["q"], su.values_of(c["k"], c["ks"]), su.values_of(c["v"], c["vs"]), c["table"], c["page"],
        c["contexts"], c["starts"], c["mask"], scale or c["q"].shape[2] ** -0.5)
    got, got_lse = out.cpu().double(), lse.cpu().double()
    empty = ref_lse == -math.inf
    assert torch.equal(got_lse == -math.inf, empty)
    assert bool((got[empty] == 0).all())
    assert float((got_lse - ref_lse)[~empty].abs().max() if (~empty).any() else 0.0) <= 1e-4
    tol = 1.25 * ((2.0 ** -9 + 1e-4) * bound + 2.0 ** -9 * ref.abs()) + 1e-30
    worst = ((got - ref).abs() - tol).max().item()
    assert worst <= 0, worst
    return out, lse


# head_dim 64 and 128 with pages of whole 8-token rows, and what else the cache can be
LAYOUTS = [(64, 16, "nhd"), (128, 16, "nhd"), (128, 8, "hnd"), (64, 48, "pair"), (128, 128, "nhd"),
           (128, 256, "nhd"), (72, 16, "nhd"), (128, 5, "nhd"), (256, 1, "hnd"), (8, 16, "pair")]


@pytest.mark.parametrize("dtype", [torch.bfloat16, su.E4M3])
@pytest.mark.parametrize("dim,page,layout", LAYOUTS)
def test_ragged_trees_over_layouts(dtype, dim, page, layout):
    check(case([0, 1, 127, 128, 129, 300], [1, 7, 12, 1, 9, 20], 6, 2, dim, page, dtype, layout,
               seed=dim + page))


@pytest.mark.parametrize("dtype", [torch.bfloat16, su.E4M3])
@pytest.mark.parametrize("group", [1, 3, 4, 7, 8, 16, 33])
def test_single_tokens_and_head_groups(dtype, group):
    check(case([0, 1, 15, 16, 17, 255, 511], [1] * 7, 2 * group, 2, 64, 16, dtype, tree=False,
               seed=group))


@pytest.mark.parametrize("nodes", [2, 31, 32, 33, 63, 64, 65, 127, 129, 200])
def test_node_counts_around_the_tiles(nodes):
    # with 4 heads per kv head: one tile of rows, two, more; masks of one word and more
    check(case([37, 130], [nodes, max(1, nodes // 3)], 4, 1, 64, 16, seed=nodes))


@pytest.mark.parametrize("dtype", [torch.bfloat16, su.E4M3])
def test_long_contexts_split_over_the_gpu(dtype):
    check(case([20011, 5, 4096, 0], [5, 3, 1, 2], 8, 2, 128, 64, dtype, seed=4))


def test_many_rows_of_one_long_request():
    check(case([2500], [40], 16, 2, 128, 32, seed=5))


def test_chain_masks_equal_no_mask():
    c = case([70, 300], [9, 66], 4, 2, 64, 16, tree=False, seed=6)
    out, lse = check(c)
    c["mask"] = su.ancestor_masks([[-1] + list(range(8)), [-1] + list(range(65))], 2)
    out2, lse2 = check(c)
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


def test_rows_that_see_nothing():
    c = case([0, 0, 40], [5, 130, 6], 4, 2, 128, 16, seed=7)
    c["mask"][0] = 0
    c["mask"][3] = 0
    c["mask"][5:120] = 0
    c["mask"][-2] = 0          # sees its context still
    check(c)


def test_peaked_scores_and_given_scale():
    check(case([515], [9], 4, 2, 128, 16, seed=8, spread=8.0))
    check(case([515], [9], 4, 2, 64, 16, seed=9), scale=0.5)


def test_scores_that_grow_along_the_keys():
    # every tile raises the running maximum by far: the sums are rescaled each time
    c = case([1500], [3], 2, 1, 64, 16, seed=10)
    c["q"].zero_()
    c["q"][..., 0] = 8.0
    pos = torch.arange(1503)
    c["k"].zero_()
    c["k"][c["table"][0, pos // 16].long().to(DEV), (pos % 16).to(DEV), :, 0] = \
        (pos.to(DEV).float() / 4).to(torch.bfloat16)[:, None]
    check(c)


@pytest.mark.parametrize("dtype", [torch.bfloat16, su.E4M3])
@pytest.mark.parametrize("dim,page", [(128, 16), (72, 5)])
def test_what_is_not_visible_has_no_influence(dtype, dim, page):
    c = case([61, 140], [9, 12], 4, 2, dim, page, dtype, seed=11)
    out, lse = check(c)
    # slots past each request's end, pages of no request, and a node that only its own row sees
    k, v = c["k"].clone(), c["v"].clone()
    used = torch.zeros(k.shape[:2], dtype=torch.bool)
    for b, n in enumerate([70, 152]):
        pos = torch.arange(n)
        used[c["table"][b, pos // page].long(), pos % page] = True
    bad = torch.full((1,), math.nan, device=DEV).to(dtype)
    node = 61 + 8                                  # the last node of request 0: a leaf
    c["mask"][8] = 1 << 8                          # it sees itself only, no one sees it
    c["mask"][:8] &= ~(1 << 8)
    leaf = (int(c["table"][0, node // page]), node % page)
    out, lse = check(c)
    for x, value in ((c["k"], math.nan), (c["v"], math.nan)):
        raw = x.view(torch.uint8 if dtype == su.E4M3 else torch.int16)
        raw[~used.to(DEV)] = bad.view(raw.dtype).item()
        raw[leaf] = bad.view(raw.dtype).item()
    if dtype == su.E4M3:
        for s in (c["ks"], c["vs"]):
            s[~used.to(DEV)] = 255
            s[leaf] = 255
    got, got_lse, st = run(c)
    assert st == 0
    keep = torch.arange(got.shape[0]) != 8
    assert torch.equal(got[keep], out[keep]) and torch.equal(got_lse[keep], lse[keep])
    assert bool(torch.isnan(got[8]).all()) and bool(torch.isnan(got_lse[8]).all())


def test_infinite_values_reach_the_rows_that_see_them_only():
    c = case([30], [6], 2, 1, 64, 16, seed=12)
    c["mask"] = su.ancestor_masks([[-1, 0, 0, 1, 2, 3]], 1)
    pos = 30 + 2                                   # node 2: seen by itself and node 4
    c["v"][int(c["table"][0, pos // 16]), pos % 16, 0, 5] = math.inf
    out, _, st = run(c)
    assert st == 0
    hit = torch.isinf(out[..., 5]).cpu()
    assert hit.tolist() == [[i in (2, 4)] * 2 for i in range(6)]
    assert bool(torch.isfinite(out[..., :5]).all()) and bool(torch.isfinite(out[..., 6:]).all())


def test_nodes_past_the_mask_words_are_not_seen():
    c = case([10], [70], 2, 1, 64, 16, seed=13, words=2)
    two, _, _ = run(c)
    c["mask"] = c["mask"][:, :1].contiguous()
    check(c)
    c["mask"] = torch.cat([c["mask"], torch.zeros_like(c["mask"])], 1)
    check(c)


def test_strided_queries_outputs_and_no_requests():
    c = case([50, 9], [4, 3], 4, 2, 128, 16, seed=14, pad=24)      # rows of 152: not a TMA row
    out, lse = check(c)
    wide = torch.zeros((7, 6, 136), dtype=torch.bfloat16, device=DEV)
    got, _, _ = run(c, out=wide[:, 1:5, 3:131])
    assert torch.equal(got, out) and float(wide[:, 0].abs().max()) == 0.0
    c["q"] = c["q"].transpose(0, 1).contiguous().transpose(0, 1)   # heads outermost
    assert torch.equal(run(c)[0], out)
    empty = case([4], [1], 4, 2, 128, 16)
    i32 = dict(dtype=torch.int32, device=DEV)
    o, z = binding.fct_tree_attention(
        empty["q"][:0], binding.KVCache(empty["k"], empty["v"]), torch.zeros((0, 1), **i32),
        torch.zeros(0, **i32), torch.zeros(1, **i32))
    assert o.shape == (0, 4, 128) and z.shape == (0, 4)


def test_requests_without_nodes_between_others():
    check(case([50, 9, 0, 33], [3, 0, 0, 4], 4, 2, 128, 16, seed=15))


def test_repeated_calls_other_streams_and_a_kept_workspace_agree():
    c = case([3000, 77, 640], [9, 2, 30], 8, 2, 128, 16, seed=16)
    out, lse, _ = run(c)
    ws = torch.full((binding.fct_tree_attention_workspace_size(41, 8, 2, 128) + 64,), 255,
                    dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            out2, lse2, _ = run(c, workspace=ws[:-64])
    torch.cuda.synchronize()
    assert torch.equal(out, out2) and torch.equal(lse, lse2)
    assert bool((ws[-64:] == 255).all())


def test_a_page_outside_the_pool_is_reported():
    c = case([40, 40], [2, 2], 4, 2, 128, 16, seed=17)
    ref, _ = check(c)
    c["table"][0, 1] = 10 ** 6
    out, _, st = run(c)
    assert st == binding.FCT_DEV_INDEX_OUT_OF_RANGE
    assert torch.equal(out[2:], ref[2:])           # the other request is untouched
    c["table"][0, 1] = -5
    assert run(c)[2] == binding.FCT_DEV_INDEX_OUT_OF_RANGE


def test_a_length_past_the_table_is_reported():
    c = case([40, 40], [2, 2], 4, 2, 128, 16, seed=18)
    ref, _ = check(c)
    c["contexts"] = [10 ** 6, 40]
    out, _, st = run(c)
    assert st == binding.FCT_DEV_INDEX_OUT_OF_RANGE
    assert torch.equal(out[2:], ref[2:])
    c["contexts"] = [-3, 40]
    out, _, st = run(c)
    assert st == binding.FCT_DEV_INDEX_OUT_OF_RANGE
    assert torch.equal(out[2:], ref[2:])


def test_offsets_past_32_bits():
    # a pool of 2^31 + elements, of which a few pages at the end are used
    page, heads, dim = 64, 8, 128
    pages = (1 << 31) // (page * heads * dim) + 8
    c = case([200], [3], 8, 8, dim, page, seed=19)
    small_k, small_v = c["k"], c["v"]
    k = torch.zeros((pages, page, heads, dim), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    n = small_k.shape[0]
    k[-n:], v[-n:] = small_k, small_v
    ref, _ = check(c)
    c["k"], c["v"] = k, v
    c["table"] = torch.where(c["table"] >= 0, c["table"] + (pages - n), c["table"])
    assert torch.equal(run(c)[0], ref)


def test_captured_in_a_graph():
    c = case([700, 30], [4, 4], 8, 2, 128, 16, seed=20)
    i32 = dict(dtype=torch.int32, device=DEV)
    cache = binding.KVCache(c["k"], c["v"])
    args = (c["q"], cache, c["table"].to(DEV), torch.tensor(c["contexts"], **i32),
            torch.tensor(c["starts"], **i32), c["mask"].to(DEV))
    ws = torch.empty(binding.fct_tree_attention_workspace_size(8, 8, 2, 128), dtype=torch.uint8,
                     device=DEV)
    want, _ = binding.fct_tree_attention(*args, workspace=ws)
    out, lse = torch.empty_like(want), torch.empty((8, 8), device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.fct_tree_attention(*args, out=out, lse=lse, workspace=ws)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
