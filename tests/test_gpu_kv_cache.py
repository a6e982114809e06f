"""The paged cache on the GPU: values as written (bf16, e4m3 by its definition in 64 bits) and the
move of accepted paths, bit for bit."""
import math

import pytest
import torch

import spec_util as su
from distillation_ce_tvd_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def awkward(n, heads, dim, gen):
    """Rows of many sizes, and the edges of the exponent rule."""
    x = torch.randn((n, heads, dim), generator=gen, device=DEV)
    x *= torch.exp2(torch.randint(-40, 40, (n, heads, 1), generator=gen, device=DEV).float())
    flat = x.view(n * heads, dim)
    edge = [0.0, 448.0, 449.0, 448.0 * 2.0 ** 7, 1.75 * 2.0 ** -118, 1.76 * 2.0 ** -118, 2.0 ** -130,
            3.3e38, 1e-44, math.nan, math.inf, -math.inf]
    for i, value in enumerate(edge[:flat.shape[0]]):
        flat[i] *= 0.0
        flat[i, dim // 2] = value
    return x


@pytest.mark.parametrize("cache_dtype", [torch.bfloat16, su.E4M3])
@pytest.mark.parametrize("src", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("heads,dim,page,layout,fused", [
    (8, 128, 16, "nhd", True), (2, 64, 7, "hnd", False), (3, 72, 1, "pair", True),
    (1, 8, 5, "nhd", False), (5, 256, 32, "hnd", True)])
def test_write_matches_the_definition(cache_dtype, src, heads, dim, page, layout, fused):
    gen = torch.Generator(device=DEV).manual_seed(heads * dim + page)
    n, pages = 53, 53 // page + 9
    k, v, ks, vs = su.make_pool(pages, page, heads, dim, cache_dtype, gen, DEV, layout)
    before = [None if x is None else x.clone() for x in (k, v, ks, vs)]
    if fused:       # K and V side by side, as one projection gives them
        kv = torch.stack([awkward(n, heads, dim, gen), awkward(n, heads, dim, gen) * -0.5], 1).to(src)
        nk, nv = kv[:, 0], kv[:, 1]
    else:
        nk, nv = awkward(n, heads, dim, gen).to(src), (awkward(n, heads, dim, gen) * 3).to(src)
    slots = torch.randperm(pages * page, generator=gen, device=DEV)[:n]
    slots[5], slots[17] = -1, -7
    st = status()
    binding.fct_kv_cache_write(binding.KVCache(k, v, ks, vs), nk, nv, slots, dev_status=st)
    assert st.item() == 0
    kept = (slots >= 0).cpu()
    at = slots.cpu()[kept]
    for pool, scale, old, old_scale, new in ((k, ks, before[0], before[2], nk),
                                             (v, vs, before[1], before[3], nv)):
        want = old.cpu().double().reshape(pages * page, heads, dim)
        if cache_dtype == su.E4M3:
            y, byte = su.quantise_ref(new.cpu()[kept])
            want[at] = y
            ws = old_scale.cpu().reshape(pages * page, heads)
            ws[at] = byte
            assert torch.equal(scale.cpu().reshape(pages * page, heads), ws)
        else:
            want[at] = new.cpu()[kept].to(torch.bfloat16).double()
        got = pool.cpu().double().reshape(pages * page, heads, dim)
        assert torch.equal(torch.nan_to_num(got, nan=1e30), torch.nan_to_num(want, nan=1e30))


def test_write_reads_back_within_the_formats_step():
    # e4m3 has 3 mantissa bits: each value is within 2^-4 of itself, or half a subnormal step
    # (2^-10 of the scale) away
    gen = torch.Generator(device=DEV).manual_seed(3)
    k, v, ks, vs = su.make_pool(9, 16, 4, 128, su.E4M3, gen, DEV)
    new = torch.randn((130, 4, 128), generator=gen, device=DEV).to(torch.bfloat16)
    slots = torch.arange(130, device=DEV)
    binding.fct_kv_cache_write(binding.KVCache(k, v, ks, vs), new, new * 2, slots)
    for pool, byte, want in ((k, ks, new), (v, vs, new * 2)):
        got = su.values_of(pool, byte).reshape(-1, 4, 128)[:130]
        want = want.cpu().double()
        step = torch.exp2(byte.cpu().double().reshape(-1, 4)[:130] - 127).unsqueeze(-1) * 2.0 ** -10
        assert bool(((got - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, step)).all())


@pytest.mark.parametrize("n", [0, 1])
def test_write_of_no_and_one_token(n):
    gen = torch.Generator(device=DEV).manual_seed(1)
    k, v, _, _ = su.make_pool(2, 4, 2, 64, torch.bfloat16, gen, DEV)
    before = k.clone()
    new = torch.ones((n, 2, 64), device=DEV, dtype=torch.bfloat16)
    binding.fct_kv_cache_write(binding.KVCache(k, v), new, new, torch.full((n,), 6, device=DEV))
    if n:
        before[1, 2] = 1
    assert torch.equal(k, before)


def test_write_past_the_pool_is_reported_and_skipped():
    gen = torch.Generator(device=DEV).manual_seed(2)
    k, v, _, _ = su.make_pool(2, 4, 2, 64, torch.bfloat16, gen, DEV)
    before = k.clone()
    new = torch.ones((2, 2, 64), device=DEV, dtype=torch.bfloat16)
    st = status()
    binding.fct_kv_cache_write(binding.KVCache(k, v), new, new,
                               torch.tensor([8, 1 << 60], device=DEV), dev_status=st)
    assert st.item() == binding.FCT_DEV_INDEX_OUT_OF_RANGE
    assert torch.equal(k, before)


@pytest.mark.parametrize("dtype", [torch.bfloat16, su.E4M3])
@pytest.mark.parametrize("page,layout", [(16, "nhd"), (3, "hnd"), (64, "pair")])
def test_move_is_the_paths_copy(dtype, page, layout):
    gen = torch.Generator(device=DEV).manual_seed(page)
    cpu = torch.Generator().manual_seed(page)
    contexts = [0, 5, 31, 64, 200]
    # in place, far, none, two in a row, and longer than one step of the kernel's loop
    paths = [[1, 2, 3], [2, 3, 7], [], [4, 5], [1, 3, 4, 6, 7, 8, 9, 11, 12, 13, 15, 17, 18, 19, 24]]
    nodes, heads, dim, depth = 25, 3, 72, 15
    table, pages = su.make_tables([c + nodes for c in contexts], page, cpu)
    k, v, ks, vs = su.make_pool(pages, page, heads, dim, dtype, gen, DEV, layout)
    want = [None if x is None else x.cpu().clone() for x in (k, v, ks, vs)]
    old = [None if x is None else x.clone() for x in want]
    for b, path in enumerate(paths):
        for j, node in enumerate(path):
            src, dst = contexts[b] + node, contexts[b] + 1 + j
            for x, o in zip(want, old):
                if x is not None:
                    x[int(table[b, dst // page]), dst % page] = o[int(table[b, src // page]), src % page]
    path = torch.tensor([p + [-1] * (depth - len(p)) for p in paths], dtype=torch.int32, device=DEV)
    st = status()
    binding.fct_kv_cache_move(binding.KVCache(k, v, ks, vs), table.to(DEV),
                              torch.tensor(contexts, dtype=torch.int32, device=DEV), path,
                              torch.tensor([len(p) for p in paths], dtype=torch.int32, device=DEV),
                              dev_status=st)
    assert st.item() == 0
    for x, w in zip((k, v, ks, vs), want):
        if w is not None:
            assert torch.equal(x.cpu().view(torch.uint8) if x.element_size() == 1 else x.cpu(),
                               w.view(torch.uint8) if w.element_size() == 1 else w)


@pytest.mark.parametrize("path,count,kept", [
    ([3, 3, 4], 3, 1),          # not ascending: the second entry stops the move
    ([2, 1, 4], 3, 1),
    ([0, 2, 3], 3, 0),          # below its destination
    ([2, 3, 500], 3, 2),        # past the table
    ([2, 3, 4], 9, 3),          # a count past the path's length is clipped
    ([2, 3, 4], -2, 0)])
def test_move_stops_at_a_bad_entry(path, count, kept):
    gen = torch.Generator(device=DEV).manual_seed(8)
    k, v, _, _ = su.make_pool(4, 8, 1, 64, torch.bfloat16, gen, DEV)
    want = k.clone()
    flat, old = want.view(32, 64), k.clone().view(32, 64)
    for j in range(kept):
        flat[4 + 1 + j] = old[4 + path[j]]
    st = status()
    i32 = dict(dtype=torch.int32, device=DEV)
    binding.fct_kv_cache_move(binding.KVCache(k, v), torch.tensor([[0, 1, 2, 3]], **i32),
                              torch.tensor([4], **i32), torch.tensor([path], **i32),
                              torch.tensor([count], **i32), dev_status=st)
    assert st.item() == binding.FCT_DEV_INDEX_OUT_OF_RANGE
    assert torch.equal(k, want)
