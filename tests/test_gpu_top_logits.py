"""The K largest logits of each row and the log-sum-exp of the others, against the definition."""
import math

import pytest
import torch

import top_util as tu
from distillation_ce_tvd_gb300 import binding

pytestmark = pytest.mark.gpu


def check(x, K, **kw):
    values, index, rest = (t.cpu() for t in binding.fct_top_logits(x, K, **kw))
    x = x.cpu()
    for r in range(x.shape[0]):
        v, i, m = tu.top_ref(x[r], K)
        assert index[r].tolist() == i, r
        assert values[r].tolist() == v, r
        left = -math.inf if m == -math.inf else sorted(x[r].double().tolist())[-K - 1]
        assert tu.close(float(rest[r]), m, tu.lse_tol(m, left, x.shape[1])), (r, float(rest[r]), m)
    return values, index, rest


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,K", [(1, 1), (1, 3), (7, 2), (8, 8), (33, 5), (1000, 64), (1000, 1024),
                                 (4099, 1), (4096, 200), (20000, 17), (32001, 513), (50257, 1024)])
def test_sizes(dtype, V, K):
    g = torch.Generator().manual_seed(V * 7 + K)
    x = (torch.randn(5, V, generator=g) * 3).to(dtype).cuda()
    check(x, K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_large_vocabulary(dtype):
    g = torch.Generator().manual_seed(11)
    x = (torch.randn(3, 151936, generator=g) * 3).to(dtype).cuda()
    check(x, 64)


@pytest.mark.parametrize("K", [1, 20, 300, 1024])
@pytest.mark.parametrize("order", ["rising", "falling", "equal", "steps", "late", "two"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_orders(order, K, dtype):
    V = 40001
    at = torch.arange(V, dtype=torch.float32)
    x = {"rising": at / 1000, "falling": -at / 1000, "equal": torch.full((V,), 2.5),
         "steps": (at % 37) / 4, "late": torch.where(at > V - 700, 5 + at / V, -at / V),
         "two": torch.where(at % 3 == 0, 1.0, -1.0)}[order]
    check(x.to(dtype).repeat(2, 1).cuda(), K)


@pytest.mark.parametrize("K", [64, 128, 129, 512, 513, 1024])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_many_equal_logits(dtype, K):
    """Rows of a few values: all or hundreds of times K reach the K-th, in every part of the row."""
    V = 50_021
    g = torch.Generator().manual_seed(K)
    x = torch.stack([torch.zeros(V), torch.randint(8, (V,), generator=g).float(),
                     torch.round(2 * (100 + torch.randn(V, generator=g))) / 2,
                     torch.where(torch.rand(V, generator=g) < 0.3, 1.0, torch.randn(V, generator=g))])
    x[0, 40_000:40_010] = 1.0
    check(x.to(dtype).cuda(), K)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_little_is_left_outside(dtype):
    """The rest keeps its relative precision where the list holds nearly all of the mass."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(4, 5003, generator=g) - 60
    x[:, 100:110] = torch.randn(4, 10, generator=g)
    x[1, 4000:] -= 200
    x[2, 200:] = -math.inf
    x[3, 7:100] = -math.inf
    check(x.to(dtype).cuda(), 10)
    check(x.to(dtype).cuda(), 11)


def test_zeros_of_either_sign_are_equal():
    x = torch.full((1, 600), -1.0)
    x[0, 10:400:3] = 0.0
    x[0, 11:400:3] = -0.0
    check(x.cuda(), 50)


def test_values_far_apart_and_extreme():
    x = torch.randn(2, 3001)
    x[0, 5], x[0, 77], x[0, 78] = 3e38, 1e30, -3e38
    x[1] *= 1e4
    check(x.cuda(), 9)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows_without_numbers(dtype):
    x = torch.randn(6, 777)
    x[0] = -math.inf
    x[1, 3] = math.nan
    x[2, 700] = math.inf
    x[3] = math.nan
    x[4, 5:] = -math.inf
    x = x.to(dtype).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    values, index, rest = binding.fct_top_logits(x, 20, dev_status=status)
    assert status.item() == binding.FCT_DEV_NO_DISTRIBUTION
    assert (index[0] == -1).all() and (values[0] == -math.inf).all() and rest[0] == -math.inf
    want = torch.where(x[1].isnan(), -math.inf, x[1].float()).topk(20)
    assert rest[1].isnan() and torch.equal(values[1], want.values)
    assert rest[2].isnan() and values[2, 0] == math.inf and index[2, 0] == 700
    assert rest[3].isnan() and (index[3] == -1).all()
    assert (index[4, 5:] == -1).all() and rest[4] == -math.inf
    status.zero_()
    check(x[4:6], 20, dev_status=status)
    assert status.item() == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset,pad", [(0, 3), (1, 0), (1, 8), (5, 7)])
def test_strides_and_alignment(dtype, offset, pad):
    g = torch.Generator().manual_seed(offset + pad)
    V, rows, K = 9001, 4, 33
    whole = (torch.randn(offset + rows * (V + pad), generator=g) * 3).to(dtype).cuda()
    x = whole[offset:].as_strided((rows, V), (V + pad, 1), offset)
    values = torch.full((rows, K + 2), -7.0, device="cuda")
    index = torch.full((rows, K + 5), -7, dtype=torch.int32, device="cuda")
    check(x, K, values=values[:, :K], index=index[:, 2:K + 2])
    assert (values[:, K:] == -7).all() and (index[:, :2] == -7).all() and (index[:, K + 2:] == -7).all()


def test_repeated_and_split_calls_give_the_same_bits():
    x = (torch.randn(700, 30011, device="cuda") * 2).bfloat16()
    a = binding.fct_top_logits(x, 50)
    b = binding.fct_top_logits(x, 50)
    parts = [binding.fct_top_logits(p, 50) for p in x.split([1, 399, 300])]
    for i in range(3):
        assert torch.equal(a[i], b[i])
        assert torch.equal(a[i], torch.cat([p[i] for p in parts]))


def test_streams_graphs_and_no_rows():
    x = torch.randn(16, 5000, device="cuda")
    want = binding.fct_top_logits(x, 12)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.fct_top_logits(x, 12, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    out = dict(values=torch.empty_like(want[0]), index=torch.empty_like(want[1]),
               rest_lse=torch.empty_like(want[2]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.fct_top_logits(x, 12, **out)
    x.copy_(x.flip(1).clone())
    graph.replay()
    want = binding.fct_top_logits(x, 12)
    assert all(torch.equal(p, q) for p, q in zip(want, out.values()))
    assert [t.shape[0] for t in binding.fct_top_logits(x[:0], 12)] == [0, 0, 0]
