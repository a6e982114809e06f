"""The loss against a teacher's top logits, forward, backward and in one launch, against the
definition in 64 bits."""
import math

import pytest
import torch

import top_util as tu
from distillation_ce_tvd_gb300 import binding

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16]


def cuda(*ts):
    return [None if t is None else t.cuda() for t in ts]


def all_ways(s, target, values, index, rest, gce, gtvd, status=None):
    """Statistics and gradient; the single launch and in-place gradients give the same bits."""
    ds, dt, dv, di, dr, dc, dg = cuda(s, target, values, index, rest, gce, gtvd)
    stats = binding.fused_ce_tvd_top_forward(ds, dt, dv, di, dr, dev_status=status)
    grad = binding.fused_ce_tvd_top_backward(ds, dt, dv, di, dr, *stats[2:], dc, dg,
                                             dev_status=status)
    both = binding.fused_ce_tvd_top_forward_backward(ds, dt, dv, di, dr, dc, dg, dev_status=status)
    same = lambda a, b: torch.equal(a.nan_to_num(7.7e33), b.nan_to_num(7.7e33))  # noqa: E731
    for a, b in zip((*stats, grad), both):
        assert same(a, b)
    copy = ds.clone()
    assert binding.fused_ce_tvd_top_backward(copy, dt, dv, di, dr, *stats[2:], dc, dg,
                                             inplace=True) is copy
    assert same(copy, grad)
    copy = ds.clone()
    assert same(binding.fused_ce_tvd_top_forward_backward(copy, dt, dv, di, dr, dc, dg,
                                                          inplace=True)[-1], grad)
    return [x.cpu() for x in stats], grad.cpu()


def check(s, target, values, index, rest, gce, gtvd):
    stats, grad = all_ways(s, target, values, index, rest, gce, gtvd)
    tu.check_rows(stats, grad, s, target, values, index, rest, gce, gtvd)
    return stats, grad


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rest", [True, False])
@pytest.mark.parametrize("V,K", [(1, 1), (2, 5), (9, 9), (31, 4), (501, 20), (1000, 1), (4099, 64),
                                 (20011, 300), (32000, 1024)])
def test_sizes(dtype, rest, V, K):
    check(*tu.make(6, V, K, dtype, V + K, rest))


@pytest.mark.parametrize("dtype", DTYPES)
def test_large_vocabularies(dtype):
    check(*tu.make(3, 151936, 64, dtype, 3))
    check(*tu.make(2, 300007, 33, dtype, 4, rest=False))       # rows shared by several CTAs


@pytest.mark.parametrize("dtype,V", [(torch.float32, 170_007), (torch.float32, 262_144),
                                     (torch.float32, 400_003), (torch.float32, 700_001),
                                     (torch.bfloat16, 524_289), (torch.bfloat16, 1_048_583)])
def test_rows_of_a_megabyte_and_more(dtype, V):
    """Rows shared by two, four and eight CTAs, in one launch and in two."""
    check(*tu.make(3, V, 70, dtype, V))


@pytest.mark.parametrize("dtype,V", [(torch.float32, 180_001), (torch.float32, 400_003),
                                     (torch.bfloat16, 530_003)])
def test_many_long_rows(dtype, V):
    """More rows than are in flight: the bits of calls on a few rows each, and of two launches."""
    rows, K = 170, 40
    g = torch.Generator(device="cuda").manual_seed(V)
    s = torch.randn(rows, V, generator=g, device="cuda").to(dtype)
    target = torch.randint(V, (rows,), generator=g, device="cuda")
    target[::7] = -100
    lists = binding.fct_top_logits(s.flip(0), K)
    up = torch.rand(rows, generator=g, device="cuda") / rows
    whole = binding.fused_ce_tvd_top_forward_backward(s, target, *lists, up, up)
    for a in range(0, rows, 17):
        part = [x[a:a + 17] for x in (s, target, *lists)]
        stats = binding.fused_ce_tvd_top_forward(*part)
        grad = binding.fused_ce_tvd_top_backward(*part, *stats[2:], up[a:a + 17], up[a:a + 17])
        for x, y in zip(whole, (*stats, grad)):
            assert torch.equal(x[a:a + 17], y)
    assert not any(x.isnan().any() for x in whole)


@pytest.mark.parametrize("dtype", DTYPES)
def test_peaked_students(dtype):
    """Nearly all mass inside the list, and nearly all outside."""
    s, target, values, index, rest, gce, gtvd = tu.make(8, 3001, 16, dtype, 9)
    for r in range(4):
        s[r, index[r][index[r] >= 0].long()] += 40
    for r in range(4, 8):
        s[r, index[r][index[r] >= 0].long()] -= 40
    rest[1], rest[5] = -math.inf, 90.0
    check(s, target, values, index, rest, gce, gtvd)


@pytest.mark.parametrize("dtype", DTYPES)
def test_masked_words_and_empty_lists(dtype):
    s, target, values, index, rest, gce, gtvd = tu.make(7, 999, 12, dtype, 21)
    s[0, 5:900] = -math.inf
    target[0] = 3
    s[1, index[1][index[1] >= 0].long()] = -math.inf    # the student excludes the list
    target[1] = int((s[1] > -math.inf).nonzero()[7])
    index[3] = -1                                       # nothing listed: the rest is all
    index[4] = -1
    rest[4] = -math.inf                                 # no teacher
    values[5] = -math.inf
    rest[5] = -math.inf                                 # no probability: no teacher either
    index[6, :] = -1
    values[6, :] = math.inf                             # what is not used does not matter
    stats, grad = check(s, target, values, index, rest, gce, gtvd)
    assert [float(stats[i][4]) for i in (1, 4, 5)] == [0.0, -math.inf, 0.0]


@pytest.mark.parametrize("dtype", DTYPES)
def test_a_list_of_every_word_is_the_whole_teacher(dtype):
    V = 700
    g = torch.Generator().manual_seed(2)
    s = (torch.randn(5, V, generator=g) * 2).to(dtype)
    t = (torch.randn(5, V, generator=g) * 2).to(dtype)
    target = torch.randint(V, (5,), generator=g)
    order = torch.stack([torch.randperm(V, generator=g) for _ in range(5)])
    gce, gtvd = torch.rand(5, generator=g), torch.rand(5, generator=g)
    stats, grad = check(s, target, t.float().gather(1, order), order.to(torch.int32), None, gce, gtvd)
    ce, tvd, lse, t_lse, sigma = (x.cpu() for x in binding.fused_ce_tvd_forward(
        s.cuda(), t.cuda(), target.cuda()))
    for a, b in zip(stats, (ce, tvd, lse, None, t_lse, sigma)):
        if b is not None:
            assert torch.allclose(a, b, rtol=2e-6, atol=4e-6)
    # a student that equals its teacher: no distance, and cross-entropy's gradient
    stats, grad = all_ways(s, target, s.float().gather(1, order), order.to(torch.int32), None, gce, gtvd)
    assert (stats[1] == 0).all() and (stats[5] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,pad", [(0, 3), (1, 0), (3, 8), (6, 7)])
def test_strides_and_alignment(dtype, offset, pad):
    rows, V, K = 5, 6007, 19
    s, target, values, index, rest, gce, gtvd = tu.make(rows, V, K, dtype, offset + pad)
    whole = torch.zeros(offset + rows * (V + pad) + 8, dtype=dtype, device="cuda")
    view = whole.as_strided((rows, V), (V + pad, 1), offset)
    view.copy_(s)
    wide_v = torch.full((rows, K + 3), 9.0, device="cuda")
    wide_i = torch.full((rows, K + 1), 0, dtype=torch.int32, device="cuda")
    wide_v[:, 1:K + 1], wide_i[:, :K] = values.cuda(), index.cuda()
    lists = (wide_v[:, 1:K + 1], wide_i[:, :K], rest.cuda())
    dt, dc, dg = cuda(target, gce, gtvd)
    stats = binding.fused_ce_tvd_top_forward(view, dt, *lists)
    grads = [binding.fused_ce_tvd_top_backward(view, dt, *lists, *stats[2:], dc, dg)]
    other = torch.zeros(rows * (V + 5) + 3, dtype=dtype, device="cuda").as_strided((rows, V), (V + 5, 1), 2)
    grads.append(binding.fused_ce_tvd_top_backward(view, dt, *lists, *stats[2:], dc, dg,
                                                   grad_student=other))
    grads.append(binding.fused_ce_tvd_top_forward_backward(view, dt, *lists, dc, dg)[-1])
    binding.fused_ce_tvd_top_backward(view, dt, *lists, *stats[2:], dc, dg, inplace=True)
    grads.append(view)
    for g in grads:
        assert torch.equal(g, grads[0])
    tu.check_rows([x.cpu() for x in stats], grads[0].cpu(), s, target, values, index, rest, gce, gtvd)
    used = torch.zeros_like(whole, dtype=torch.bool)
    used.as_strided((rows, V), (V + pad, 1), offset)[:] = True
    assert (whole[~used] == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_targets_and_lists_that_are_wrong(dtype):
    args = list(tu.make(8, 2000, 10, dtype, 31))
    clean, _ = all_ways(*args)
    s, target, values, index, rest, gce, gtvd = args
    target[0], target[1], target[2] = 2000, -5, -100
    index[3, 4], index[4, 0] = 2000, -2
    a, b = index[5][index[5] >= 0][:2]
    index[5][index[5] == b] = a                          # one word twice
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stats, grad = all_ways(*args, status=status)
    assert status.item() == binding.FCT_DEV_TARGET_OUT_OF_RANGE | binding.FCT_DEV_BAD_LIST
    assert stats[0][:2].isnan().all() and grad[:2].isnan().all()
    assert all(torch.equal(x[:2], y[:2]) for x, y in zip(stats[1:], clean[1:]))
    assert (grad[2] == 0).all() and all(x[2] == 0 for x in stats)
    assert all(x[3:6].isnan().all() for x in stats) and grad[3:6].isnan().all()
    assert not any(x[6:].isnan().any() for x in stats) and not grad[6:].isnan().any()
    # a list whose row is ignored is not read
    target[3:6] = -100
    status.zero_()
    target[0] = target[1] = 0
    all_ways(*args, status=status)
    assert status.item() == 0


def test_numbers_that_are_not_finite_are_seen():
    s, target, values, index, rest, gce, gtvd = tu.make(4, 800, 6, torch.float32, 8)
    s[0, 799], s[1, 0] = math.nan, math.inf
    values[3, 0], index[3, 0] = math.nan, int([v for v in range(800) if v not in index[3]][0])
    stats, grad = all_ways(s, target, values, index, rest, gce, gtvd)
    assert stats[2][:2].isnan().all() and stats[1][3].isnan() and grad[[0, 1, 3]].isnan().any(1).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradient_against_differences(dtype):
    """Central differences of the definition along random directions."""
    s, target, values, index, rest, gce, gtvd = tu.make(4, 300, 8, dtype, 77)
    target[2] = 5
    _, grad = all_ways(s, target, values, index, rest, gce, gtvd)
    g = torch.Generator().manual_seed(1)
    for r in range(4):
        def loss(x):
            w = tu.row_ref(x, int(target[r]), values[r], index[r], float(rest[r]))
            return float(gce[r]) * w["ce"] + float(gtvd[r]) * w["tvd"]
        d = torch.randn(300, generator=g).double()
        h = 1e-6
        slope = (loss(s[r].double() + h * d) - loss(s[r].double() - h * d)) / (2 * h)
        # truncation h^2, cancellation 1e-16 / h, and the kernel's rounding of each element
        tol = 1e-8 + (grad[r].double().abs() * d.abs()).sum() * (
            torch.finfo(dtype).eps / 2 + 2.0 ** -17)
        assert abs((grad[r].double() * d).sum() - slope) <= tol


@pytest.mark.parametrize("dtype", DTYPES)
def test_students_and_teachers_that_are_sure_of_one_word(dtype):
    """1 - p below what fp32 log-sum-exps near 30 resolve: the gradient of tvd is still p (1 - p) and
    the like, not p."""
    rows, V, K = 40, 2000, 8
    s, target, values, index, rest, gce, gtvd = tu.make(rows, V, K, dtype, 50)
    for r in range(rows):
        used = index[r] >= 0
        word = int(index[r][used][0])
        values[r][(index[r] == word)] = 35.0 + 0.37 * (r % 7)
        s[r, word] = 32.0 + 0.5 * (r % 9)
        if r % 3 == 0:      # the rest instead: the list is what hardly counts
            s[r, word] = -3.0
            values[r][used] = -12.0 - 0.5 * (r % 5)
            s[r, index[r][used].long()] -= 14.0
    gce = torch.zeros(rows)
    stats, grad = all_ways(s, target, values, index, rest, gce, gtvd)
    for r in range(rows):
        if target[r] == tu.IGNORE:
            continue
        # |p (sign - sigma)| <= 2 (1 - p) for the word or the rest that p is near 1 of, 2 p elsewhere
        p = torch.softmax(s[r].double(), 0)
        used = index[r][index[r] >= 0].long()
        p_rest = 1 - p[used].sum().item()
        most = max(p.max().item(), p_rest)
        left = p[used].sum().item() if p_rest == most else 1 - p.max().item()
        assert most > 0.999
        bound = 0.5 * abs(float(gtvd[r])) * 2 * (left + 2.0 ** -21)
        assert grad[r].double().abs().max().item() <= bound, (r, most)


def test_upstream_broadcast_split_and_repeated():
    s, target, values, index, rest, gce, gtvd = cuda(*tu.make(600, 5003, 40, torch.bfloat16, 6))
    one = binding.fused_ce_tvd_top_forward_backward(s, target, values, index, rest, 0.25, 0.5)
    rows = binding.fused_ce_tvd_top_forward_backward(
        s, target, values, index, rest, torch.full((600,), 0.25, device="cuda"),
        torch.tensor(0.5, device="cuda"))
    again = binding.fused_ce_tvd_top_forward_backward(s, target, values, index, rest, 0.25, 0.5)
    cut = [binding.fused_ce_tvd_top_forward_backward(s[a:b], target[a:b], values[a:b], index[a:b],
                                                     rest[a:b], 0.25, 0.5)
           for a, b in ((0, 1), (1, 400), (400, 600))]
    for i in range(7):
        assert torch.equal(one[i], rows[i]) and torch.equal(one[i], again[i])
        assert torch.equal(one[i], torch.cat([c[i] for c in cut]))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 5, 13, 2001, 131_080])
def test_rows_without_a_gradient_at_every_offset(dtype, V):
    """Rows that are ignored get 0, rows of a target outside the vocabulary NaN, and nothing else is
    written, wherever a row starts and however it ends."""
    rows = 8
    s, target, values, index, rest, gce, gtvd = cuda(*tu.make(rows, V, 3, dtype, 5))
    target[0::3], target[1::3] = -100, V
    for ld in (V + 1, V + 2):                      # 16-byte phases differ from row to row
        whole = torch.full((rows * ld + 8,), 5.0, dtype=dtype, device="cuda")
        grad = whole.as_strided((rows, V), (ld, 1), 1)
        used = torch.zeros_like(whole, dtype=torch.bool)
        used.as_strided((rows, V), (ld, 1), 1)[:] = True
        stats = binding.fused_ce_tvd_top_forward(s, target, values, index, rest)
        for call in (
                lambda: binding.fused_ce_tvd_top_backward(s, target, values, index, rest, *stats[2:],
                                                          gce, gtvd, grad_student=grad),
                lambda: binding.fused_ce_tvd_top_forward_backward(s, target, values, index, rest, gce,
                                                                  gtvd, grad_student=grad)):
            whole.fill_(5.0)
            call()
            assert (grad[0::3] == 0).all() and grad[1::3].isnan().all()
            assert not grad[2::3].isnan().any() and (whole[~used] == 5).all()


def test_streams_graphs_and_no_rows():
    s, target, values, index, rest, gce, gtvd = cuda(*tu.make(64, 4000, 16, torch.bfloat16, 16))
    want = binding.fused_ce_tvd_top_forward_backward(s, target, values, index, rest, gce, gtvd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = binding.fused_ce_tvd_top_forward_backward(s, target, values, index, rest, gce, gtvd,
                                                    stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    outs = {n: torch.empty_like(want[0]) for n in binding._TOP_STATS}
    grad = torch.empty_like(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.fused_ce_tvd_top_forward(s, target, values, index, rest, **outs)
        binding.fused_ce_tvd_top_backward(s, target, values, index, rest,
                                          *list(outs.values())[2:], gce, gtvd, grad_student=grad)
    s.copy_(s.roll(17, 1).clone())
    graph.replay()
    want = binding.fused_ce_tvd_top_forward_backward(s, target, values, index, rest, gce, gtvd)
    assert all(torch.equal(a, b) for a, b in zip(want, (*outs.values(), grad)))
    empty = binding.fused_ce_tvd_top_forward_backward(s[:0], target[:0], values[:0], index[:0],
                                                      rest[:0], 1.0, 1.0)
    assert [t.shape[0] for t in empty] == [0] * 7


def test_from_a_teachers_rows():
    """fct_top_logits' lists go straight into the loss; with all words listed it is the dense one."""
    g = torch.Generator().manual_seed(40)
    s = torch.randn(20, 1000, generator=g).cuda()
    t = (torch.randn(20, 1000, generator=g) * 2).cuda()
    target = torch.randint(1000, (20,), generator=g).cuda()
    dense = binding.fused_ce_tvd_forward(s, t, target)
    last = None
    for k in (10, 100, 1000):
        stats = binding.fused_ce_tvd_top_forward(s, target, *binding.fct_top_logits(t, k))
        assert torch.allclose(stats[0], dense[0], rtol=1e-6, atol=2e-6)
        assert (stats[1] <= dense[1] + 2e-6).all()         # merging words brings nothing apart
        assert last is None or (stats[1] >= last - 2e-6).all()
        last = stats[1]
    assert torch.allclose(last, dense[1], rtol=0, atol=2e-6)
