"""Verification of drafted tokens on the GPU against the same walk in 64 bits.

Probabilities are computed in fp32 (relative error under 1e-5 for the logits used), so a request's
outputs have to equal the 64-bit walk's wherever no decision of that walk is closer than 1e-4 to
going the other way; such requests are a few in a thousand and are counted.
"""
import math
import random

import pytest
import torch

import spec_util as su
from distillation_ce_tvd_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def case(nodes, V, dtype, draft, seed, chain=False, spread=2.0, noise_gap=0.7, pad=0):
    gen, rnd = torch.Generator().manual_seed(seed), random.Random(seed)
    starts = [0]
    for n in nodes:
        starts.append(starts[-1] + n)
    parents = [([-1] + list(range(n - 1)) if chain else su.random_tree(n, rnd)) if n else []
               for n in nodes]
    N, B = starts[-1], len(nodes)
    target = torch.randn((N, V + pad), generator=gen) * spread
    dl = (target + torch.randn((N, V + pad), generator=gen) * noise_gap).to(dtype)
    target = target.to(dtype)
    tokens = torch.randint(0, V, (N,), generator=gen)
    for b in range(B):
        for i, p in enumerate(parents[b]):
            if p >= 0:
                at = starts[b] + p
                if draft:
                    w = torch.softmax(dl[at, :V].float(), 0)
                    tokens[starts[b] + i] = torch.multinomial(w, 1, generator=gen)
                else:
                    nth = parents[b][:i].count(p)
                    tokens[starts[b] + i] = target[at, :V].float().argsort(descending=True)[nth % V]
    return dict(target=target, draft=dl if draft else None, tokens=tokens, V=V, starts=starts,
                parent=torch.tensor([p for q in parents for p in q], dtype=torch.int32),
                uniform=torch.rand(N, generator=gen),
                noise=torch.empty((B, V)).exponential_(generator=gen), temperature=None)


def run(c, max_depth, **kw):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    cut = lambda x: None if x is None else x.to(DEV)[:, :c["V"]]  # noqa: E731
    got = binding.fct_spec_verify(
        cut(c["target"]), d(c["tokens"]), d(c["parent"]),
        torch.tensor(c["starts"], dtype=torch.int32, device=DEV), d(c["uniform"]), d(c["noise"]),
        cut(c["draft"]), d(c["temperature"]), max_depth=max_depth, dev_status=st, **kw)
    return [x.cpu() for x in got], st.item()


def check(c, max_depth, close=0.05):
    got, st = run(c, max_depth)
    assert st == 0
    cut = lambda x: None if x is None else x[:, :c["V"]]  # noqa: E731
    *want, margin = su.verify_ref(cut(c["target"]), cut(c["draft"]), c["tokens"],
                                  c["parent"].tolist(), c["starts"], c["uniform"], c["noise"],
                                  c["temperature"], max_depth)
    sure = torch.tensor([m > 1e-4 for m in margin])
    assert int((~sure).sum()) <= max(1, close * len(margin))
    for g, w in zip(got, want):
        assert torch.equal(g[sure], w.to(g.dtype)[sure])
    return got


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 1000, 4099, 4104, 32000])
def test_chains_with_a_drafts_distribution(dtype, V):
    got = check(case([5] * 12 + [1, 2, 8], V, dtype, True, seed=V, chain=True), 7)
    if V >= 1000:
        assert 0 < int(got[2].sum()) < 12 * 4 + 8      # some accepted, some not


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("V", [5, 500, 4104])
def test_trees(dtype, draft, V):
    # siblings: the residual after one and several rejections
    check(case([12, 20, 40, 1, 7, 33, 64, 65, 100], V, dtype, draft, seed=V + 1), 6)


def test_many_siblings_of_one_node():
    # more rejected tokens at a node than a thread keeps: 30 children over a tiny vocabulary
    c = case([31] * 8, 24, torch.float32, False, seed=5)
    c["parent"][:] = 0
    for s in c["starts"][:-1]:
        c["parent"][s] = -1
    c["uniform"][:] = 0.999
    check(c, 3, close=0.3)
    check(case([31] * 8, 6000, torch.float32, False, seed=6), 3)


def test_a_large_vocabulary():
    check(case([6, 3, 9], 151936, torch.bfloat16, True, seed=2), 5)
    check(case([6, 3, 9], 151936, torch.bfloat16, False, seed=3), 5)


@pytest.mark.parametrize("draft", [True, False])
def test_temperatures_and_greedy(draft):
    c = case([6] * 8, 777, torch.float32, draft, seed=9)
    c["temperature"] = torch.tensor([0.0, 0.3, 1.0, 2.5, 0.0, 0.7, 1.0, 0.0])
    check(c, 5, close=0.3)
    # greedy with equal largest logits: the lowest index
    c["target"][:, 300] = c["target"][:, 5] = 30.0
    c["temperature"][:] = 0.0
    c["tokens"][:] = 5
    got, _ = run(c, 5)
    assert bool((got[0][:, 0] == 5).all()) and bool((got[2] >= 1).all())
    c["tokens"][:] = 300
    got, _ = run(c, 5)
    assert bool((got[0][:, 0] == 5).all()) and bool((got[2] == 0).all())


def test_masked_logits_are_never_chosen():
    # all but a few logits -inf, whole vectors and threads' shares among them
    c = case([5] * 30, 5000, torch.float32, True, seed=10, chain=True)
    keep = torch.tensor([17, 1234, 2500, 4999])
    for x in (c["target"], c["draft"]):
        y = torch.full_like(x, -math.inf)
        y[:, keep] = x[:, keep]
        x.copy_(y)
    c["tokens"] = keep[torch.randint(0, 4, c["tokens"].shape, generator=torch.Generator().manual_seed(1))]
    got = check(c, 4, close=0.3)
    assert set(got[0].flatten().tolist()) <= set(keep.tolist()) | {-1}
    # a drafted token that the target masks is never accepted
    c["tokens"][:] = 18
    assert int(run(c, 4)[0][2].sum()) == 0


def test_the_lowest_finite_value_as_a_mask():
    c = case([4] * 10, 900, torch.bfloat16, True, seed=11, chain=True)
    low = torch.finfo(torch.bfloat16).min
    c["target"][:, 100:] = low
    c["draft"][:, 100:] = low
    c["tokens"] %= 100
    got = check(c, 3, close=0.3)
    assert int(got[0].max()) < 100


@pytest.mark.parametrize("value", [math.nan, math.inf, None])
@pytest.mark.parametrize("temperature", [1.0, 0.0])
def test_rows_without_a_distribution(value, temperature):
    c = case([3] * 4, 300, torch.float32, True, seed=12, chain=True)
    c["temperature"] = torch.full((4,), temperature)
    c["uniform"][:] = 0.0                  # every drafted token with p > 0 is accepted ...
    if temperature == 0.0:                 # ... or the largest
        for s in c["starts"][:-1]:
            c["tokens"][s + 1] = c["target"][s].argmax()
            c["tokens"][s + 2] = c["target"][s + 1].argmax()
    row = c["starts"][2] + 1               # request 2's second row
    if value is None:
        c["target"][row] = -math.inf
    else:
        c["target"][row, 211] = value
    got, st = run(c, 2)
    assert st == binding.FCT_DEV_NO_DISTRIBUTION
    assert got[2].tolist() == [2, 2, 1, 2]
    assert got[0][2].tolist()[1:] == [-1, -1]
    assert all(got[0][b, 2] >= 0 for b in (0, 1, 3))


def test_rows_that_are_not_visited_are_not_read_for_decisions():
    c = case([4] * 6, 640, torch.float32, True, seed=13, chain=True)
    c["uniform"][:] = 0.0
    want, _ = run(c, 3)
    leaf = [s + 3 for s in c["starts"][:-1]]
    c["draft"][leaf] = math.nan            # draft rows of nodes without children
    got, st = run(c, 3)
    assert st == 0 and all(torch.equal(a, b) for a, b in zip(got, want))


def test_tokens_outside_the_vocabulary_are_rejected():
    for draft in (True, False):
        c = case([2] * 3, 50, torch.float32, draft, seed=14, chain=True)
        c["uniform"][:] = 0.0
        c["tokens"][1], c["tokens"][3] = 50, -1
        got, st = run(c, 1)
        assert st == binding.FCT_DEV_TARGET_OUT_OF_RANGE
        assert got[2].tolist() == [0, 0, 1]
        assert bool((got[0][:, 0] >= 0).all())


def test_depth_limit_and_empty_requests():
    c = case([6, 0, 6], 100, torch.float32, True, seed=15, chain=True)
    c["uniform"][:] = 0.0
    check(c, 2)
    got, _ = run(c, 2)
    assert got[2].tolist() == [2, 0, 2]
    assert got[0][1].tolist() == [-1] * 3 and got[1][1].tolist() == [-1] * 2
    got, _ = run(c, 0)
    assert got[0].shape == (3, 1) and got[1].shape == (3, 0) and got[0][1, 0] == -1
    check(c, 9)


def test_equal_distributions_accept_everything():
    c = case([5] * 8, 3001, torch.bfloat16, True, seed=16, chain=True)
    c["draft"] = c["target"].clone()
    c["uniform"][:] = 1 - 2.0 ** -24
    for b in range(8):
        for i in range(1, 5):
            c["tokens"][c["starts"][b] + i] = c["target"][c["starts"][b] + i - 1].float().argmax()
    got, _ = run(c, 4)
    assert got[2].tolist() == [4] * 8


@pytest.mark.parametrize("pad", [0, 1, 3, 8])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_row_strides_and_alignment(pad, dtype):
    check(case([5] * 6, 1016, dtype, True, seed=17 + pad, pad=pad), 4)


def test_unaligned_noise_and_offset_rows():
    c = case([5] * 6, 1000, torch.bfloat16, True, seed=18)
    want = check(c, 4)
    wide = torch.empty((6, 1003))
    wide[:, 1:1001] = c["noise"]
    c["noise"] = wide
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    big_t = torch.zeros((30, 1009), dtype=torch.bfloat16, device=DEV)
    big_t[:, 3:1003] = c["target"].to(DEV)
    got = binding.fct_spec_verify(
        big_t[:, 3:1003], c["tokens"].to(DEV), c["parent"].to(DEV),
        torch.tensor(c["starts"], dtype=torch.int32, device=DEV), c["uniform"].to(DEV),
        wide.to(DEV)[:, 1:1001], c["draft"].to(DEV), max_depth=4, dev_status=st)
    assert all(torch.equal(g.cpu(), w) for g, w in zip(got, want))


@pytest.mark.parametrize("draft", [True, False])
def test_tokens_follow_the_targets_distribution(draft):
    # one drafted level with two siblings drawn from q (or the two best tokens): the first output
    # token's frequencies over 40000 independent requests against p, by chi-square with 5 degrees
    # of freedom (99.99% quantile 25.7)
    B, V = 40000, 6
    gen = torch.Generator().manual_seed(21)
    p = torch.softmax(torch.randn(V, generator=gen, dtype=torch.float64) * 1.5, 0)
    q = torch.softmax(torch.randn(V, generator=gen, dtype=torch.float64), 0)
    target = p.log().float().expand(3 * B, V).contiguous()
    dl = q.log().float().expand(3 * B, V).contiguous()
    tokens = torch.multinomial(q, 3 * B, replacement=True, generator=gen)
    if not draft:
        best = p.argsort(descending=True)
        tokens = torch.tensor([0, int(best[0]), int(best[1])]).repeat(B)
    c = dict(target=target, draft=dl if draft else None, tokens=tokens, V=V,
             starts=list(range(0, 3 * B + 1, 3)),
             parent=torch.tensor([-1, 0, 0], dtype=torch.int32).repeat(B),
             uniform=torch.rand(3 * B, generator=gen),
             noise=torch.empty((B, V)).exponential_(generator=gen), temperature=None)
    got, st = run(c, 1)
    assert st == 0
    seen = torch.bincount(got[0][:, 0], minlength=V).double()
    chi = float(((seen - B * p) ** 2 / (B * p)).sum())
    assert chi < 25.7, (chi, seen / B, p)
