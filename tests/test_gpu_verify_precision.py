"""Verification on the GPU where probabilities have to be good to a few units of 2^-20: logits far
from 0 and low temperatures, with decisions placed 1e-5 from going the other way.

A probability is 2^d / s with d = (x - max) * log2(e) / T.  Logits and their differences here are
exact in fp32; d is within 3 * 2^-24 of itself (the factor's two roundings and the product's), 4e-6
for |d| <= 24, times ln 2; the exponential and the sum add under 2e-6.  A ratio of two such
probabilities is within 1e-5.  Decisions use tokens with |d| <= 12, which halves the first part.
"""
import math

import pytest
import torch

from distillation_ce_tvd_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GAP = 1e-5


def verify(target, tokens, uniform, noise, draft, temperature, nodes):
    B = noise.shape[0]
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    d = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    out, _, count = binding.fct_spec_verify(
        d(target), d(tokens), torch.arange(-1, nodes - 1, dtype=torch.int32, device=DEV).repeat(B),
        torch.arange(0, B * nodes + 1, nodes, dtype=torch.int32, device=DEV), d(uniform), d(noise),
        d(draft), d(temperature), max_depth=nodes - 1, dev_status=st)
    assert st.item() == 0
    return out.cpu(), count.cpu()


def logits(gen, rows, V, offset):
    # multiples of 2^-10 below 2^11: exact in fp32, as are their differences
    return offset + torch.round(torch.randn((rows, V), generator=gen) * 2 * 1024) / 1024


# (offset of the target's logits, of the draft's, temperature)
SCENES = [(0.0, 0.0, 1.0), (1024.0, 0.0, 1.0), (0.0, -1024.0, 1.0), (1024.0, 1024.0, 1.0),
          (30.0, 30.0, 0.0625), (-30.0, 30.0, 0.25)]


@pytest.mark.parametrize("V", [999, 4096, 32768])
@pytest.mark.parametrize("at,dt,T", SCENES)
def test_acceptance_against_a_drafts_probability(at, dt, T, V):
    B, gen = 128, torch.Generator().manual_seed(int(at) + V)
    target = logits(gen, 2 * B, V, at)
    draft = dt + (target - at) + torch.round(torch.randn((2 * B, V), generator=gen) * 512 * T) / 1024
    p, q = (torch.softmax(x[::2].double() / T, 1) for x in (target, draft))
    # a token of some weight that the draft favours, so that p / q < 1 decides
    score = torch.where(p < 0.999 * q, q, torch.zeros_like(q))
    x = score.argmax(1)
    rows = torch.arange(B)
    ratio = p[rows, x] / q[rows, x]
    usable = (score[rows, x] > 0) & (q[rows, x] > 2.0 ** -12 * q.amax(1)) & (p[rows, x] > 2.0 ** -12 * p.amax(1))
    assert int(usable.sum()) > B // 2
    yes = torch.arange(B) % 2 == 0
    uniform = torch.zeros(2 * B)
    uniform[1::2] = (ratio * torch.where(yes, 1 - GAP, 1 + GAP)).float()
    tokens = torch.zeros(2 * B, dtype=torch.int64)
    tokens[1::2] = x
    noise = torch.empty((B, V)).exponential_(generator=gen)
    _, count = verify(target, tokens, uniform, noise, draft, torch.full((B,), T), 2)
    assert torch.equal(count[usable] == 1, yes[usable])


@pytest.mark.parametrize("V", [999, 4096, 32768])
@pytest.mark.parametrize("at,T", [(0.0, 1.0), (1024.0, 1.0), (-1024.0, 1.0), (30.0, 0.0625)])
@pytest.mark.parametrize("drafted", [False, True])
def test_the_race_for_the_next_token(at, T, V, drafted):
    # two tokens whose p / noise are 1e-5 apart, the others far behind; from a node without children,
    # and after a rejected child (which the target gives no probability)
    B, gen = 64, torch.Generator().manual_seed(int(at) + V + 1)
    n = 2 if drafted else 1
    target = logits(gen, n * B, V, at)
    target[:, 7] = -math.inf
    p = torch.softmax(target[::n].double() / T, 1)
    two = torch.topk(p, 2).indices
    two = two[:, torch.randperm(2, generator=gen)]
    rows = torch.arange(B)
    noise = torch.full((B, V), 1e6)
    first = torch.arange(B) % 2 == 0
    a, b = p[rows, two[:, 0]], p[rows, two[:, 1]]
    usable = torch.minimum(a, b) > 2.0 ** -12 * torch.maximum(a, b)
    assert int(usable.sum()) > B // 2
    noise[rows, two[:, 0]] = a.float()
    # the fp32 noise decides: the other's share is set from what it became
    ratio = noise[rows, two[:, 0]].double() / a
    noise[rows, two[:, 1]] = (b * ratio * torch.where(first, 1 + GAP, 1 - GAP)).float()
    tokens, uniform = torch.full((n * B,), 7), torch.full((n * B,), 0.5)
    out, count = verify(target, tokens, uniform, noise, None, torch.full((B,), T), n)
    assert int(count.sum()) == 0
    want = torch.where(first, two[:, 0], two[:, 1])
    assert torch.equal(out[:, 0][usable], want[usable])


def test_a_constant_on_a_row_changes_nothing():
    # the same logits and 1024 more: the same tokens, decision by decision
    B, V, nodes, gen = 64, 8192, 5, torch.Generator().manual_seed(3)
    target = logits(gen, nodes * B, V, 0.0)
    draft = target + torch.round(torch.randn((nodes * B, V), generator=gen) * 300) / 1024
    tokens = torch.zeros((B, nodes), dtype=torch.int64)
    q = torch.softmax(draft, 1)
    tokens[:, 1:] = torch.multinomial(q, 1, generator=gen).view(B, nodes)[:, :-1]
    args = (tokens.flatten(), torch.rand(nodes * B, generator=gen),
            torch.empty((B, V)).exponential_(generator=gen))
    want = verify(target, *args, draft, None, nodes)
    for a, b in ((1024.0, 0.0), (0.0, 1024.0), (-1024.0, 512.0)):
        got = verify(target + a, *args, draft + b, None, nodes)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_temperature_that_is_none_has_no_distribution():
    # not a number, and below 0: it was taken for greedy
    V, gen = 500, torch.Generator().manual_seed(5)
    target, temperature = logits(gen, 8, V, 0.0), torch.tensor([1.0, math.nan, -1.0, 0.0])
    tokens = torch.zeros(8, dtype=torch.int64)
    tokens[1::2] = target[::2].argmax(1)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out, path, count = binding.fct_spec_verify(
        target.to(DEV), tokens.to(DEV), torch.tensor([-1, 0] * 4, dtype=torch.int32, device=DEV),
        torch.arange(0, 9, 2, dtype=torch.int32, device=DEV), torch.zeros(8, device=DEV),
        torch.ones((4, V), device=DEV), None, temperature.to(DEV), max_depth=1, dev_status=st)
    assert st.item() == binding.FCT_DEV_NO_DISTRIBUTION
    assert count.tolist() == [1, 0, 0, 1] and path[:, 0].tolist() == [1, -1, -1, 1]
    assert out[1:3].tolist() == [[-1, -1]] * 2
    assert out[0, 0] == tokens[1] and out[3].tolist() == [int(tokens[7]), int(target[7].argmax())]
