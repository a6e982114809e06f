"""The speculative decoding step without a GPU: refusals of the C ABI and of the binding, and the
plain forms the GPU tests compare with."""
import ctypes
import math

import pytest
import torch

import spec_util as su
from distillation_ce_tvd_gb300 import binding

OK, INVALID, UNSUPPORTED, ALIGN = 0, 1, 2, 3
FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def cache(**kw):
    f = dict(k=FAKE, v=FAKE + (1 << 33), k_scale=None, v_scale=None, dtype=1, page_size=16,
             n_heads=2, head_dim=64, num_pages=10, page_stride=2048, slot_stride=128,
             head_stride=64, scale_page_stride=0, scale_slot_stride=0, scale_head_stride=0)
    f.update(kw)
    return ctypes.byref(binding._KvCacheStruct(*f.values()))


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(dtype=0), UNSUPPORTED),
    (dict(dtype=7), UNSUPPORTED), (dict(page_size=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(n_heads=-1), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=60), UNSUPPORTED),
    (dict(head_dim=264), UNSUPPORTED), (dict(page_stride=-2048), INVALID),
    (dict(page_stride=1 << 61), INVALID), (dict(k=FAKE + 2), ALIGN), (dict(slot_stride=124), ALIGN),
    (dict(dtype=2), INVALID), (dict(dtype=2, k_scale=FAKE, v_scale=None), INVALID),
    (dict(dtype=2, k_scale=FAKE, v_scale=FAKE, k=FAKE + 4), ALIGN),
    (dict(dtype=2, k_scale=FAKE, v_scale=FAKE, scale_head_stride=-1), INVALID)]


@pytest.mark.parametrize("change,want", BAD_CACHES)
def test_caches_are_checked(lib, change, want):
    c = cache(**change)
    assert lib.fct_kv_cache_write(FAKE, FAKE, 128, 64, 1, 4, FAKE, c, None, None) == want
    assert lib.fct_kv_cache_move(c, FAKE, 8, 8, FAKE, 1, FAKE, 4, 4, FAKE, None, None) == want
    assert lib.fct_tree_attention(FAKE, 256, 64, 5, 4, c, FAKE, 8, 8, FAKE, FAKE, 1, None, 0, 0.1,
                                  FAKE + (1 << 40), 256, 64, None, None, 0, None, None) == want


def call(f, args, **kw):
    a = list(args)
    for i, v in kw.items():
        a[int(i[1:])] = v
    return f(*a)


def test_write_arguments(lib):
    f, args = lib.fct_kv_cache_write, [FAKE, FAKE, 128, 64, 1, 4, FAKE, cache(), None, None]
    assert call(f, args, a5=0) == OK                     # no tokens
    assert call(f, args, a5=-1) == INVALID
    assert call(f, args, a7=None) == INVALID
    assert call(f, args, a4=2) == UNSUPPORTED            # an e4m3 source
    assert call(f, args, a0=None) == INVALID
    assert call(f, args, a1=None) == INVALID
    assert call(f, args, a6=None) == INVALID
    assert call(f, args, a2=-1) == INVALID
    assert call(f, args, a2=1 << 62) == INVALID
    assert call(f, args, a0=FAKE + 1) == ALIGN
    assert call(f, args, a6=FAKE + 4) == ALIGN
    assert call(f, args, a8=FAKE + 2) == ALIGN


def test_move_arguments(lib):
    f = lib.fct_kv_cache_move
    args = [cache(), FAKE, 8, 8, FAKE, 3, FAKE, 4, 4, FAKE, None, None]
    assert call(f, args, a5=0) == OK
    assert call(f, args, a8=0) == OK                     # an empty path
    assert call(f, args, a5=-1) == INVALID
    assert call(f, args, a8=-1) == INVALID
    assert call(f, args, a1=None) == INVALID
    assert call(f, args, a2=7) == INVALID                # ld < max_pages
    assert call(f, args, a3=0) == INVALID
    assert call(f, args, a4=None) == INVALID
    assert call(f, args, a6=None) == INVALID
    assert call(f, args, a7=3) == INVALID                # ld < path_len
    assert call(f, args, a9=None) == INVALID
    assert call(f, args, a5=1 << 30) == UNSUPPORTED
    assert call(f, args, a6=FAKE + 2) == ALIGN
    assert call(f, args, a10=FAKE + 1) == ALIGN


def test_attention_arguments(lib):
    f = lib.fct_tree_attention
    args = [FAKE, 256, 64, 5, 4, cache(), FAKE, 8, 8, FAKE, FAKE, 1, FAKE, 1, 0.1,
            FAKE + (1 << 40), 256, 64, None, None, 0, None, None]
    assert call(f, args, a3=0) == OK
    assert call(f, args, a11=0) == OK
    assert call(f, args, a3=-1) == INVALID
    assert call(f, args, a11=-1) == INVALID
    assert call(f, args, a4=3) == INVALID                # not a multiple of the cache's heads
    assert call(f, args, a4=0) == INVALID
    assert call(f, args, a14=math.nan) == INVALID
    assert call(f, args, a0=None) == INVALID
    assert call(f, args, a15=None) == INVALID
    assert call(f, args, a10=None) == INVALID
    assert call(f, args, a6=None) == INVALID
    assert call(f, args, a7=4) == INVALID
    assert call(f, args, a12=None) == INVALID            # words without a mask
    assert call(f, args, a13=0) == INVALID               # a mask without words
    assert call(f, args, a1=-8) == INVALID
    assert call(f, args, a15=FAKE + 64) == INVALID       # over q
    assert call(f, args, a0=FAKE + 1) == ALIGN
    assert call(f, args, a12=FAKE + 4) == ALIGN
    assert call(f, args, a18=FAKE + 2) == ALIGN
    assert lib.fct_tree_attention_workspace_size(0, 4, 2, 64) == 0
    assert lib.fct_tree_attention_workspace_size(5, 3, 2, 64) == 0
    assert lib.fct_tree_attention_workspace_size(5, 4, 2, 60) == 0


def test_verify_arguments(lib):
    f = lib.fct_spec_verify
    args = [FAKE, 100, FAKE, 100, 1, 6, 100, FAKE, FAKE, FAKE, 2, FAKE, FAKE, 100, FAKE, 3, FAKE,
            FAKE, FAKE, None, None]
    assert call(f, args, a10=0) == OK
    assert call(f, args, a10=-1) == INVALID
    assert call(f, args, a5=-1) == INVALID
    assert call(f, args, a6=0) == INVALID
    assert call(f, args, a15=-1) == INVALID
    assert call(f, args, a4=2) == UNSUPPORTED
    assert call(f, args, a6=(1 << 30) + 1, a1=1 << 31, a3=1 << 31, a13=1 << 31) == UNSUPPORTED
    for i in (0, 7, 8, 9, 11, 12, 16, 17, 18):
        assert call(f, args, **{f"a{i}": None}) == INVALID, i
    for i in (1, 3, 13):
        assert call(f, args, **{f"a{i}": 99}) == INVALID, i
    assert call(f, args, a1=1 << 62) == INVALID
    for i, off in ((0, 1), (2, 1), (7, 4), (8, 2), (9, 2), (11, 2), (12, 2), (14, 2), (16, 4),
                   (17, 2), (18, 2), (19, 2)):
        assert call(f, args, **{f"a{i}": FAKE + off}) == ALIGN, i


def test_the_cache_object_refuses_cpu_and_other_types():
    k = torch.zeros((2, 4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.KVCache(k, k)
    with pytest.raises(TypeError):
        binding.KVCache(k.half(), k.half())


def test_quantise_reference_agrees_with_the_format():
    # the arithmetic definition against the type's own rounding, where nothing saturates
    gen = torch.Generator().manual_seed(0)
    x = torch.randn((200, 16), generator=gen) * torch.exp2(torch.arange(200.) / 4 - 25)[:, None]
    y, byte = su.quantise_ref(x)
    scaled = x.double() / torch.exp2(byte.double() - 127)[:, None]
    assert float(scaled.abs().max()) <= 448.0
    assert bool((scaled.abs().amax(-1) > 224.0).all())
    assert torch.equal(y, scaled.float().to(su.E4M3).double())


def test_verify_reference_keeps_the_targets_distribution():
    # two siblings drawn from q: the chance of each first token, summed over the draws, is p
    p = torch.softmax(torch.tensor([0.3, -1.0, 0.8]).double(), 0)
    q = torch.softmax(torch.tensor([-0.2, 0.5, 0.1]).double(), 0)
    total = torch.zeros(3, dtype=torch.float64)
    for a in range(3):
        first = torch.minimum(torch.ones(()), p[a] / q[a])
        total[a] += q[a] * first
        r = (p - q).clamp(min=0)
        Z = r.sum()
        for b in range(3):
            second = torch.minimum(torch.ones(()).double(), r[b] / (Z * q[b]))
            total[b] += q[a] * (1 - first) * q[b] * second
            rest = (p - (1 + Z) * q).clamp(min=0)
            if float(rest.sum()) > 0:
                total += q[a] * (1 - first) * q[b] * (1 - second) * rest / rest.sum()
    assert torch.allclose(total, p, atol=1e-12)
