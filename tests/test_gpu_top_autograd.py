"""Distillation from a teacher's cached top logits as a training step makes it: lists from the
teacher's rows, then the loss and its gradients through torch.autograd, on logits and from hidden
states."""
import pytest
import torch

from distillation_ce_tvd_gb300 import autograd, binding

pytestmark = pytest.mark.gpu


def reference(s, target, values, index, rest):
    """Per-row (ce, tvd) in float64, differentiable; rows of target -100 are 0."""
    live = target != -100
    logp = torch.log_softmax(s, 1)
    ce = -logp.gather(1, target.clamp(min=0)[:, None])[:, 0]
    p = logp.exp()
    q = torch.softmax(torch.cat([values.double(), rest.double()[:, None]], 1), 1)
    mine = p.gather(1, index.long())
    tvd = 0.5 * ((mine - q[:, :-1]).abs().sum(1) + (1 - mine.sum(1) - q[:, -1]).abs())
    zero = torch.zeros_like(ce)
    return torch.where(live, ce, zero), torch.where(live, tvd, zero)


def setup(rows=60, V=1200, d=64, K=24):
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    h, w = r(rows, d).bfloat16(), (r(V, d) * (2.5 / d ** 0.5)).bfloat16()
    s = h.float() @ w.float().t()
    lists = binding.fct_top_logits(0.8 * s + r(rows, V), K)
    target = lists[1][:, 0].long()
    target[4] = -100
    return h, w, s, target, lists


def near(a, b, rel):
    return (a.double() - b).norm() <= rel * b.norm()


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rows(dtype, inplace):
    _, _, s, target, lists = setup()
    s = s.to(dtype)
    x = s.clone().requires_grad_()
    y = s.double().requires_grad_()
    weight = torch.rand(60, device="cuda")
    ce, tvd = autograd.fused_ce_tvd_top_loss(x.clone() if inplace else x, target, *lists,
                                             inplace=inplace)
    (ce * weight + 2 * tvd).sum().backward()
    want = reference(y, target, *lists)
    (want[0] * weight + 2 * want[1]).sum().backward()
    assert near(ce, want[0].detach(), 1e-6) and near(tvd, want[1].detach(), 1e-5)
    # every element rounded once (half a step) after the errors of float32 exponentials
    assert near(x.grad, y.grad, torch.finfo(dtype).eps / 2 + 1e-5)


@pytest.mark.parametrize("scale", [1.0, 3.0])
def test_mean(scale):
    _, _, s, target, lists = setup()
    x, y = s.clone().requires_grad_(), s.double().requires_grad_()
    loss = autograd.fused_ce_tvd_top_mean_loss(x, target, *lists, alpha=0.5, beta=2.0)
    (scale * loss).backward()
    ce, tvd = reference(y, target, *lists)
    want = (0.5 * ce.sum() + 2.0 * tvd.sum()) / 59
    (scale * want).backward()
    assert abs(loss.item() - want.item()) <= 1e-5 * want.item()
    assert near(x.grad, y.grad, 1e-5)


@pytest.mark.parametrize("needs", [(True, True), (True, False), (False, True)])
def test_from_hidden_states(needs):
    h, w, _, target, lists = setup()
    a, b = h.clone().requires_grad_(needs[0]), w.clone().requires_grad_(needs[1])
    c, e = h.double().requires_grad_(), w.double().requires_grad_()
    ce, tvd = autograd.fused_linear_ce_tvd_top_loss(a, b, target, *lists, piece_cols=512)
    (ce + tvd).mean().backward()
    want = reference(c @ e.t(), target, *lists)
    (want[0] + want[1]).mean().backward()
    assert near(ce, want[0].detach(), 1e-5) and near(tvd, want[1].detach(), 1e-4)
    # the logits' gradient and the result are each rounded to bfloat16: 2^-8 each
    for got, ref in ((a.grad, c.grad), (b.grad, e.grad)):
        if got is not None:
            assert got.dtype is torch.bfloat16 and near(got, ref, 2 * 2.0 ** -8)
    assert (a.grad is not None, b.grad is not None) == needs


def test_cross_entropy_from_hidden_states():
    h, w, _, target, _ = setup()
    a, b = h.clone().requires_grad_(), w.clone().requires_grad_()
    c, e = h.double().requires_grad_(), w.double().requires_grad_()
    ce = autograd.fused_linear_ce_loss(a, b, target)
    ce.mean().backward()
    want = torch.nn.functional.cross_entropy(c @ e.t(), target, reduction="none")
    want.mean().backward()
    assert near(ce, want.detach(), 1e-5)
    assert near(a.grad, c.grad, 2 * 2.0 ** -8) and near(b.grad, e.grad, 2 * 2.0 ** -8)


def test_a_training_step_as_a_graph():
    """Lists, loss and gradients captured once, replayed on new data."""
    h, w, _, target, _ = setup()
    teacher = torch.randn(60, 1200, device="cuda")
    out = {}

    def step():
        lists = binding.fct_top_logits(teacher, 16)
        stats = binding.fused_linear_ce_tvd_top_forward(h, w, target, *lists)
        out["stats"] = stats
        out["grads"] = binding.fused_linear_ce_tvd_top_backward(h, w, target, *lists, *stats[2:],
                                                                1 / 60, 0.5 / 60)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    captured = dict(out)
    teacher.copy_(torch.randn(60, 1200, device="cuda"))
    h.mul_(-0.5)
    graph.replay()
    step()
    for a, b in zip((*captured["stats"], *captured["grads"]), (*out["stats"], *out["grads"])):
        assert torch.equal(a, b)


def test_a_captured_mean_loss_and_its_backward():
    """Loss and gradient by torch.autograd, captured once and replayed on new logits; the scale of
    the loss is read at the replay."""
    _, _, s, target, lists = setup()
    scale = torch.ones((), device="cuda")

    def step(x):
        loss = autograd.fused_ce_tvd_top_mean_loss(x, target, *lists, alpha=0.5, beta=2.0)
        return loss.detach(), torch.autograd.grad(loss * scale, x)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(s.clone().requires_grad_())
    torch.cuda.current_stream().wait_stream(side)
    x = s.clone().requires_grad_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, grad = step(x)
    with torch.no_grad():
        x.copy_(s.roll(1, 1))
    scale.fill_(-3.0)
    graph.replay()
    want_loss, want_grad = step(x.detach().clone().requires_grad_())
    assert torch.equal(loss, want_loss) and torch.equal(grad, want_grad)


def test_calls_on_two_streams_at_once():
    """Lists, loss and both linear calls on two streams, with workspaces of their own: the same bits
    as one after the other."""
    h, w, s, target, lists = setup(rows=300, V=5000, d=128, K=40)

    def work(x, hidden):
        top = binding.fct_top_logits(x, 40)
        both = binding.fused_ce_tvd_top_forward_backward(x, target, *lists, 1.0, 0.5)
        stats = binding.fused_linear_ce_tvd_top_forward(hidden, w, target, *lists)
        grads = binding.fused_linear_ce_tvd_top_backward(hidden, w, target, *lists, *stats[2:], 1.0,
                                                         0.5, piece_cols=2048)
        return (*top, *both, *stats, *grads)

    inputs = [(s, h), (s.flip(0).contiguous(), h.flip(0).contiguous())]
    want = [work(*x) for x in inputs]
    streams = [torch.cuda.Stream() for _ in inputs]
    torch.cuda.synchronize()
    for _ in range(4):
        got = []
        for stream, x in zip(streams, inputs):
            with torch.cuda.stream(stream):
                got.append(work(*x))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
