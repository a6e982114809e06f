"""Tree attention on the GPU against attention in 64 bits: weights that a few of many keys carry, a
scale of zero, values near the largest and values that are not finite.

Tolerances.  Scores: exact products summed in fp32, in fewer than 32 roundings of at most
sum |q||k| * scale, which is under 60 here, so 32 * 60 * 2^-24 = 1.2e-4 in a score and as much in its
weight's relative error, twice for numerator and sum; weights to 16 bits (2^-16).  Under
4e-4 * sum w|v| together.  The output is rounded to bf16 once: 2^-8 of itself.
"""
import math

import pytest
import torch

import spec_util as su
from distillation_ce_tvd_gb300 import binding
from test_gpu_tree_attention import case, run

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16


def close(c, scale=None):
    out, lse, st = run(c, scale=scale)
    assert st == 0
    ref, ref_lse, bound = su.attention_ref(
        c["q"], su.values_of(c["k"], c["ks"]), su.values_of(c["v"], c["vs"]), c["table"], c["page"],
        c["contexts"], c["starts"], c["mask"], c["q"].shape[2] ** -0.5 if scale is None else scale)
    worst = ((out.cpu().double() - ref).abs() - 2.0 ** -8 * ref.abs() - 4e-4 * bound).max().item()
    assert worst <= 0, worst
    assert float((lse.cpu().double() - ref_lse).abs().max()) <= 4e-4
    return out, lse


@pytest.mark.parametrize("dtype", [BF16, su.E4M3])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("nodes", [[5, 5, 3, 2], [12, 9, 16, 14], [70, 3, 33, 40]])
def test_peaked_weights_at_any_number_of_keys(dtype, dim, nodes):
    # a few keys carry the weight, so that roundings do not average out; from one tile of rows held
    # four times to two tiles, below and above 2048 keys
    close(case([1900, 2060, 4500, 9000], nodes, 8, 2, dim, 16, dtype, seed=dim + nodes[0],
               spread=4.0 if dtype == BF16 else 2.0))


@pytest.mark.parametrize("dtype", [BF16, su.E4M3])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 32), (72, 16), (128, 5)])
def test_a_scale_of_zero_gives_the_mean(dtype, dim, page):
    c = case([0, 61, 700], [3, 9, 40], 8, 2, dim, page, dtype, seed=1)
    for scale in (0.0, -0.0):
        out, lse = close(c, scale)
    seen = torch.tensor([sum(bin(w & (2 ** 64 - 1)).count("1") for w in row) for row in c["mask"].tolist()])
    ctx = torch.tensor([0] * 3 + [61] * 9 + [700] * 40)
    assert torch.allclose(lse.cpu().double(), (seen + ctx).double().log()[:, None], atol=1e-5)
    # 0 times what is not finite is not a number
    c["q"][5, 3, 7] = math.nan
    c["q"][6, 2, 0] = math.inf
    got, got_lse, st = run(c, scale=0.0)
    bad = torch.isnan(got_lse)
    assert st == 0 and bad.nonzero().tolist() == [[5, 3], [6, 2]]
    assert bool(torch.isnan(got[bad]).all()) and torch.equal(got[~bad], out[~bad])


@pytest.mark.parametrize("scale", [-0.125, 0.07])
def test_negative_scales(scale):
    close(case([0, 61, 700], [3, 9, 40], 8, 2, 64, 16, seed=2), scale)


def put(c, which, b, pos, head, d, payload, byte=None):
    """One element (or all, d = slice(None)) of a cached vector by its 8-bit payload."""
    at = (int(c["table"][b, pos // c["page"]]), pos % c["page"], head)
    c[which].view(torch.uint8)[at + (d,)] = payload
    if byte is not None:
        c[which + "s"][at] = byte


@pytest.mark.parametrize("payload", [0x7F, 0xFF])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (72, 16), (128, 5)])
def test_not_a_number_payloads_of_an_e4m3_cache(dim, page, payload):
    # the scale's byte is an ordinary one
    c = case([61, 140, 30], [9, 12, 50], 4, 2, dim, page, su.E4M3, seed=3)
    clean, clean_lse, _ = run(c)
    put(c, "v", 0, 17, 1, 5, payload)               # a value of the context: its column, its head
    put(c, "k", 1, 130, 0, 63, payload)             # a key: its head's rows
    put(c, "v", 2, 30 + 4, 0, 8, payload)           # a value of a drafted node: who sees it
    out, lse, st = run(c)
    assert st == 0
    want = torch.zeros(out.shape, dtype=torch.bool)
    want[:9, 2:, 5] = True
    want[9:21, :2] = True
    sees = [i for i in range(50) if (int(c["mask"][21 + i, 0]) >> 4) & 1]
    want[torch.tensor(sees) + 21, :2, 8] = True
    assert 1 <= len(sees) < 50
    assert torch.equal(torch.isnan(out).cpu(), want)
    assert torch.equal(out[~want.to(DEV)], clean[~want.to(DEV)])
    rows = torch.isnan(lse).cpu()
    assert rows[9:21, :2].all() and int(rows.sum()) == 24
    assert torch.equal(lse[~rows.to(DEV)], clean_lse[~rows.to(DEV)])


@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (72, 16), (128, 5)])
@pytest.mark.parametrize("byte", [247, 248, 250, 254, 255])
@pytest.mark.parametrize("nodes", [9, 80])
def test_large_scales_of_drafted_nodes_stay_with_who_sees_them(dim, page, byte, nodes):
    c = case([61], [nodes], 4, 2, dim, page, su.E4M3, seed=4)
    last = 61 + nodes - 1
    word, bit = (nodes - 1) // 64, (nodes - 1) % 64
    one = (1 << bit) - (1 << 64 if bit == 63 else 0)
    c["mask"][:-1, word] &= ~one                    # a leaf: only its own row sees it, and the context
    c["mask"][-1] = 0
    c["mask"][-1, word] = one
    put(c, "v", 0, last, 0, slice(None), 0x38)      # 1, and below 448, -448 and NaN
    clean, clean_lse, _ = run(c)
    for d, payload in ((2, 0x7E), (9, 0xFE)):
        put(c, "v", 0, last, 0, d, payload, byte)
    out, lse, st = run(c)
    assert st == 0
    assert torch.equal(out[:-1], clean[:-1]) and torch.equal(out[-1, 2:], clean[-1, 2:])
    assert torch.equal(lse, clean_lse)
    own = out[-1, :2].float().cpu()
    if byte == 255:
        assert bool(torch.isnan(own).all())
    else:                                           # 2^128 and more reads as an infinity
        assert bool((own[:, 2] == math.inf).all()) and bool((own[:, 9] == -math.inf).all())
        rest = torch.ones(dim, dtype=torch.bool)
        rest[[2, 9]] = False
        # 1 * 2^(byte - 127) counts with its weight
        assert bool((torch.isfinite(own[:, rest]) == (byte < 255)).all())
        assert bool((own[:, rest] > 1e20).all())
    put(c, "k", 0, last, 1, slice(None), 0x7E, 254)  # a key that only its own row sees
    got, got_lse, st = run(c)
    assert st == 0 and torch.equal(got[:-1], clean[:-1]) and torch.equal(got_lse[:-1], clean_lse[:-1])


@pytest.mark.parametrize("dtype", [BF16, su.E4M3])
@pytest.mark.parametrize("nodes", [3, 40])
def test_values_near_the_largest_do_not_overflow(dtype, nodes):
    # the key that holds 2^127 comes in the third tile, with a score 5 above all others': its value
    # has to be weighted with less than 1 before anything is summed
    c = case([300], [nodes], 4, 1, 64, 16, dtype, tree=False, seed=5)
    raw = [c[x].view(torch.uint8 if dtype == su.E4M3 else torch.int16) for x in "kv"]
    for x in raw:
        x.zero_()
    c["q"].zero_()
    c["q"][..., 0] = 1.0
    at = (int(c["table"][0, 299 // 16]), 299 % 16, 0)
    if dtype == su.E4M3:
        c["ks"][:], c["vs"][:] = 127, 127
        raw[0][at + (0,)], raw[1][at] = 0x4A, 0x38     # 5, and 1 with a scale of 2^127
        c["vs"][at] = 254
    else:
        c["k"][at + (0,)], c["v"][at] = 5.0, 2.0 ** 127
    out, lse, st = run(c, scale=1.0)
    assert st == 0
    others = 300 + torch.arange(nodes, dtype=torch.float64)
    want = 2.0 ** 127 * math.exp(5) / (math.exp(5) + others)
    got = out.cpu().double()
    assert float((got / want[:, None, None] - 1).abs().max()) <= 2.0 ** -8 + 1e-5
