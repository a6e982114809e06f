"""Verification on the GPU against the same walk in 64 bits, by the kernel's ways of reading: how many
nodes' rows are staged ahead, rows too large to be staged, and trees larger than its tables.

Probabilities are within 1e-5 of themselves for these logits (see test_gpu_verify_precision), so a
request's outputs have to equal the 64-bit walk's unless a decision of that walk is closer than 2e-5
to going the other way.
"""
import pytest
import torch

import spec_util as su
import test_gpu_verify as base
from distillation_ce_tvd_gb300 import binding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def check(c, max_depth, excluded=0.02):
    """The walk's outputs; at most the given share of the requests may be too close to decide."""
    V, st = c["V"], torch.zeros(1, dtype=torch.int32, device=DEV)
    d = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    cut = lambda x: None if x is None else x[:, :V]  # noqa: E731
    got = binding.fct_spec_verify(
        cut(d(c["target"])), d(c["tokens"]), d(c["parent"]),
        torch.tensor(c["starts"], dtype=torch.int32, device=DEV), d(c["uniform"]),
        cut(d(c["noise"])), cut(d(c["draft"])), d(c["temperature"]), max_depth=max_depth,
        dev_status=st)
    assert st.item() == 0
    *want, margin = su.verify_ref(cut(c["target"]), cut(c["draft"]), c["tokens"],
                                  c["parent"].tolist(), c["starts"], c["uniform"], cut(c["noise"]),
                                  c["temperature"], max_depth)
    sure = torch.tensor([m > 2e-5 for m in margin])
    assert int((~sure).sum()) <= excluded * len(margin)
    for g, w in zip(got, want):
        assert torch.equal(g.cpu()[sure], w.to(g.dtype)[sure])
    return want


# 64 requests leave two CTAs to each, or four where a node's rows need them: (V, nodes staged ahead
# in 216 KB of shared memory per CTA with a draft in bf16)
@pytest.mark.parametrize("V,staged", [(20000, 4), (32000, 3), (50000, 2), (100000, 1), (151936, 1)])
@pytest.mark.parametrize("chain", [False, True])
def test_nodes_staged_ahead(V, staged, chain):
    per_cta = -(-(V // 8) // (4 if V > 110592 else 2)) * 32
    assert min(4, 216 * 1024 // per_cta) == staged
    c = base.case([4] * 64 if V > 60000 else [7] * 64, V, torch.bfloat16, True, seed=V + chain, chain=chain)
    _, path, count = check(c, 5)
    # walks along the first children, and away from them
    assert 0 < int(count.sum()) < 64 * 3 and len(set(count.tolist())) > 1
    if not chain:
        assert bool((path[:, 0] > 1).any())


@pytest.mark.parametrize("dtype,V,draft", [(torch.float32, 450001, True), (torch.float32, 900003, False),
                                           (torch.bfloat16, 900003, True), (torch.bfloat16, 1800003, False)])
def test_rows_too_large_to_be_staged(dtype, V, draft):
    # 16-byte aligned rows with a ragged end
    c = base.case([6, 1, 4], V, dtype, draft, seed=V % 1000, pad=8 - V % 8)
    c["noise"] = torch.nn.functional.pad(c["noise"], (0, 8 - V % 8), value=1.0)
    check(c, 3)
    c["temperature"] = torch.tensor([0.0, 0.5, 0.0])
    check(c, 3)


@pytest.mark.parametrize("dtype,V", [(torch.float32, 600), (torch.bfloat16, 4097)])
@pytest.mark.parametrize("draft", [False, True])
def test_trees_larger_than_the_tables(dtype, V, draft):
    check(base.case([300, 257, 256, 400, 2], V, dtype, draft, seed=V), 8, excluded=0.2)


def test_a_chain_longer_than_the_tables():
    # every drafted token is accepted, up to a rejected one past the tables' end
    c = base.case([300, 5], 64, torch.float32, True, seed=9, chain=True)
    c["uniform"][:] = 0.0
    c["uniform"][290] = 1e6
    want = check(c, 299)
    assert want[2].tolist() == [289, 4]


def test_many_children_past_the_tables():
    # a root with 299 children: more rejected tokens than a thread keeps, some past the tables
    c = base.case([300], 2048, torch.float32, False, seed=10)
    c["parent"][1:] = 0
    c["tokens"][1:] = torch.randperm(2048, generator=torch.Generator().manual_seed(1))[:299]
    c["uniform"][:] = 1e6
    want = check(c, 2)
    assert int(want[2][0]) == 0
    c["uniform"][280] = 0.0
    want = check(c, 2)
    assert want[1][0, 0] == 280
