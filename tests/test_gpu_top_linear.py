"""The loss against a teacher's top logits, and cross-entropy alone, from hidden states and weights,
against the definition in 64 bits.

Bounds: a logit is a sum of d products; the tensor cores add 16 products at a time to a partial sum
of at most 768, dropping bits below it (48 steps of at most 2^-23 of the sum of magnitudes: a step of
the accumulator's last bit), and the partial sums are added in float32 (d / 768 steps of 2^-24).  A logit's gradient is rounded to
bfloat16 (2^-8, half a step), and enters sums over the vocabulary (d hidden) or the rows (d weight)
that the tensor cores accumulate the same way, at most n / 16 steps; the results are rounded once.
"""
import math

import pytest
import torch

import top_util as tu
from distillation_ce_tvd_gb300 import binding

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8


def make(rows, V, d, K, seed, rest=True):
    g = torch.Generator().manual_seed(seed)
    h = torch.randn(rows, d, generator=g).bfloat16()
    w = (torch.randn(V, d, generator=g) * (2.5 / math.sqrt(d))).bfloat16()
    s = h.double() @ w.double().t()
    err = (48 * 2.0 ** -23 + (d / 768 + 1) * 2.0 ** -24) * (h.double().abs() @ w.double().abs().t())
    if K:
        _, target, values, index, rests, gce, gtvd = tu.make(rows, V, K, torch.float32, seed, rest)
        t = 0.8 * s + torch.randn(rows, V, generator=g)
        for r in range(rows):                       # the list of a teacher near these logits
            used = index[r] >= 0
            n = int(used.sum())
            words = t[r].topk(n).indices
            index[r][used] = words.to(torch.int32)
            values[r][used] = t[r][words].float()
            outside = torch.ones(V, dtype=torch.bool)
            outside[words] = False
            if rests is not None:
                rests[r] = torch.logsumexp(t[r][outside], 0) if outside.any() else -math.inf
    else:
        target = torch.randint(V, (rows,), generator=g)
        if rows > 2:
            target[2] = tu.IGNORE
        gce = torch.rand(rows, generator=g)
        values, index = torch.empty(rows, 0), torch.empty(rows, 0, dtype=torch.int32)
        rests, gtvd = None, torch.zeros(rows)
    return dict(h=h, w=w, s=s, err=err, target=target, values=values, index=index, rest=rests,
                gce=gce, gtvd=gtvd, K=K)


def cuda(c):
    return {k: v.cuda() if torch.is_tensor(v) else v for k, v in c.items()}


def call(c, **kw):
    """(statistics, grad_h, grad_w) of the two calls; with K 0 the statistics are (ce, lse)."""
    x = cuda(c)
    up = dict(kw)
    status = up.pop("dev_status", None)
    if c["K"]:
        lists = (x["values"], x["index"], x["rest"])
        stats = binding.fused_linear_ce_tvd_top_forward(x["h"], x["w"], x["target"], *lists,
                                                        dev_status=status)
        grads = binding.fused_linear_ce_tvd_top_backward(
            x["h"], x["w"], x["target"], *lists, *stats[2:], x["gce"], x["gtvd"],
            dev_status=status, **up)
    else:
        stats = binding.fused_linear_ce_forward(x["h"], x["w"], x["target"], dev_status=status)
        grads = binding.fused_linear_ce_backward(x["h"], x["w"], x["target"], stats[1], x["gce"],
                                                 dev_status=status, **up)
    return [t.cpu() for t in stats], *(None if t is None else t.cpu() for t in grads)


def check(c, stats, grad_h, grad_w):
    rows, V = c["s"].shape
    G, tol = torch.zeros(rows, V, dtype=torch.float64), torch.zeros(rows, V, dtype=torch.float64)
    names = tu.NAMES if c["K"] else ("ce", "lse")
    for r in range(rows):
        want = tu.row_ref(c["s"][r], int(c["target"][r]), c["values"][r], c["index"][r],
                          None if c["rest"] is None else float(c["rest"][r]), float(c["gce"][r]),
                          float(c["gtvd"][r]), err=c["err"][r].max().item())
        for name, x in zip(names, stats):
            assert tu.close(float(x[r]), want[name], want["tol"][name]), \
                (r, name, float(x[r]), want[name], want["tol"][name])
        G[r] = want["grad"]
        tol[r] = want["tol"]["grad"] + want["grad"].abs() * HALF + 1e-38
    for got, a, n in ((grad_h, c["w"].double(), V), (grad_w, c["h"].double(), rows)):
        if got is None:
            continue
        g, t = (G, tol) if got is grad_h else (G.t(), tol.t())
        want = g @ a
        bound = (t + (n / 16 + 32) * 2.0 ** -22 * (g.abs() + t)) @ a.abs()
        bound += want.abs() * (torch.finfo(got.dtype).eps / 2) + 1e-38
        off = (got.double() - want).abs() - bound
        assert bool((off <= 0).all()), (off.max().item(), (got.double() - want).norm().item())


@pytest.mark.parametrize("K", [0, 6, 300])
@pytest.mark.parametrize("rows,V,d", [(1, 1, 8), (1, 9, 64), (5, 257, 72), (3, 1000, 520),
                                      (130, 700, 1032), (300, 513, 64), (257, 2050, 128),
                                      (16, 5003, 2048)])
def test_sizes(rows, V, d, K):
    c = make(rows, V, d, K, rows + V + d)
    check(c, *call(c))


@pytest.mark.parametrize("K,rest", [(1, True), (1024, True), (40, False)])
def test_lists(K, rest):
    c = make(20, 3001, 96, K, K, rest)
    check(c, *call(c))


@pytest.mark.parametrize("piece", [1, 256, 300, 1024, 5000])
def test_pieces_of_the_vocabulary(piece):
    c = make(70, 1801, 200, 12, 3)
    stats, gh, gw = call(c, piece_cols=piece)
    check(c, stats, gh, gw)
    _, _, whole = call(c)
    assert torch.equal(gw, whole)


def test_kinds_of_weight_gradient_and_what_is_not_wanted():
    c = make(40, 900, 136, 9, 5)
    x = cuda(c)
    stats, gh, gw = call(c, grad_w_dtype=torch.float32)
    assert gw.dtype is torch.float32
    check(c, stats, gh, gw)
    acc = torch.full((900, 136), 2.0, device="cuda")
    _, _, added = call(c, grad_w=acc, accumulate=True)
    assert added.data_ptr() != acc.data_ptr() and torch.allclose(acc.cpu() - 2.0, gw, atol=1e-6, rtol=0)
    _, none, only = call(c, want_grad_h=False, grad_w_dtype=torch.float32)
    assert none is None and torch.equal(only, gw)
    _, only, none = call(c, want_grad_w=False)
    assert none is None and torch.equal(only, gh)
    assert call(c, want_grad_h=False, want_grad_w=False)[1:] == (None, None)
    assert x["h"].shape == (40, 136)


def test_strides():
    c = make(33, 777, 56, 7, 6)
    h, w = torch.zeros(33, 72).bfloat16(), torch.zeros(777, 64).bfloat16()
    h[:, 8:64], w[:, :56] = c["h"], c["w"]
    gh, gw = torch.zeros(33, 59).bfloat16().cuda(), torch.zeros(777, 57).bfloat16().cuda()
    want = call(c)
    c2 = dict(c, h=h.cuda()[:, 8:64], w=w.cuda()[:, :56])
    got = call(c2, grad_h=gh[:, 1:57], grad_w=gw[:, :56])
    for a, b in zip((*want[0], *want[1:]), (*got[0], *got[1:])):
        assert torch.equal(a, b)
    assert (gh[:, :1] == 0).all() and (gh[:, 57:] == 0).all() and (gw[:, 56:] == 0).all()


def test_against_the_loss_on_logits():
    """Exact products: the logits are the same bits either way, and so are signs and sums to their
    rounding."""
    g = torch.Generator().manual_seed(9)
    h = torch.randint(-4, 5, (50, 64), generator=g).bfloat16().cuda()
    w = (torch.randint(-4, 5, (2000, 64), generator=g) / 16).bfloat16().cuda()
    logits = h.float() @ w.float().t()
    teacher = logits * 0.7 + torch.randn(50, 2000, generator=g).cuda()
    target = torch.randint(2000, (50,), generator=g).cuda()
    lists = binding.fct_top_logits(teacher, 30)
    a = binding.fused_linear_ce_tvd_top_forward(h, w, target, *lists)
    b = binding.fused_ce_tvd_top_forward(logits, target, *lists)
    for x, y in zip(a, b):
        assert torch.allclose(x, y, rtol=1e-6, atol=2e-6)
    gce, gtvd = torch.rand(50, device="cuda"), torch.rand(50, device="cuda")
    G = binding.fused_ce_tvd_top_backward(logits, target, *lists, *a[2:], gce, gtvd).bfloat16()
    eye = torch.eye(64, device="cuda").bfloat16()
    _, gw = binding.fused_linear_ce_tvd_top_backward(h, w, target, *lists, *a[2:], gce, gtvd,
                                                     grad_w_dtype=torch.float32)
    want = G.double().t() @ h.double()
    assert eye.shape == (64, 64) and (gw.double() - want).norm() <= 1e-5 * want.norm()


def test_wrong_targets_and_lists():
    c = make(300, 1500, 64, 8, 12)
    clean = call(c)
    c["target"][0], c["target"][1] = 1500, -3
    c["index"][5, 0], c["index"][270, 3] = 1500, -9
    used = c["index"][9][c["index"][9] >= 0]
    c["index"][9][c["index"][9] == used[1]] = used[0]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    stats, gh, gw = call(c, dev_status=status)
    assert status.item() == binding.FCT_DEV_TARGET_OUT_OF_RANGE | binding.FCT_DEV_BAD_LIST
    bad = torch.zeros(300, dtype=torch.bool)
    bad[[5, 9, 270]] = True
    assert all(x[bad].isnan().all() for x in stats) and stats[0][:2].isnan().all()
    bad[:2] = True
    for x, y in zip(stats, clean[0]):
        assert torch.equal(x[~bad], y[~bad])
    assert gh[bad].isnan().all() and torch.equal(gh[~bad], clean[1][~bad]) and gw.isnan().all()


def test_all_rows_ignored_and_no_teacher():
    c = make(40, 600, 64, 5, 13)
    c["target"][:] = tu.IGNORE
    stats, gh, gw = call(c)
    assert all((x == 0).all() for x in stats) and (gh == 0).all() and (gw == 0).all()
    c = make(6, 600, 64, 5, 14)
    c["index"][:] = -1
    c["rest"][:] = -math.inf
    check(c, *call(c))


def test_a_padded_batch():
    """Ignored rows whose hidden states and lists hold anything: no part of either gradient."""
    c = make(40, 700, 72, 6, 21)
    c["target"][25:] = tu.IGNORE
    want = call(c)
    c["h"][25:] = math.nan
    c["h"][30] = math.inf
    c["index"][25:], c["values"][25:] = 1 << 30, math.nan
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = call(c, dev_status=status)
    for a, b in zip((*want[0], *want[1:]), (*got[0], *got[1:])):
        assert torch.equal(a, b)
    assert status.item() == 0 and (got[1][25:] == 0).all()


def test_repeated_calls_streams_graphs_and_no_rows():
    c = make(150, 3000, 256, 20, 15)
    x = cuda(c)
    lists = (x["values"], x["index"], x["rest"])
    want = call(c)
    again = call(c)
    for a, b in zip((*want[0], *want[1:]), (*again[0], *again[1:])):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    stats = binding.fused_linear_ce_tvd_top_forward(x["h"], x["w"], x["target"], *lists, stream=side)
    grads = binding.fused_linear_ce_tvd_top_backward(x["h"], x["w"], x["target"], *lists, *stats[2:],
                                                     x["gce"], x["gtvd"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((*want[0], *want[1:]), (*stats, *grads)):
        assert torch.equal(a, b.cpu())
    outs = {n: torch.empty(150, device="cuda") for n in binding._TOP_STATS}
    gh, gw = torch.empty_like(x["h"]), torch.empty_like(x["w"])
    f = torch.empty(binding.fused_linear_ce_tvd_top_forward_workspace_size(150, 3000, 20),
                    dtype=torch.uint8, device="cuda")
    b = torch.empty(binding.fused_linear_ce_tvd_top_backward_workspace_size(150, 3000, 256, 20),
                    dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.fused_linear_ce_tvd_top_forward(x["h"], x["w"], x["target"], *lists, workspace=f, **outs)
        binding.fused_linear_ce_tvd_top_backward(
            x["h"], x["w"], x["target"], *lists, *list(outs.values())[2:], x["gce"], x["gtvd"],
            workspace=b, grad_h=gh, grad_w=gw)
    x["h"].mul_(0.5)
    graph.replay()
    c["h"] = c["h"] * 0.5
    want = call(c)
    for a, b in zip((*want[0], *want[1:]), (*outs.values(), gh, gw)):
        assert torch.equal(a, b.cpu())
    e, lse = binding.fused_linear_ce_forward(x["h"][:0], x["w"], x["target"][:0])
    gh, gw = binding.fused_linear_ce_backward(x["h"][:0], x["w"], x["target"][:0], lse, 1.0)
    assert e.shape == (0,) and gh.shape == (0, 256) and (gw == 0).all()
