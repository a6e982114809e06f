"""Cases of distillation from a teacher's top logits: the selection of each row's largest logits, the
fused cross-entropy and total-variation loss against such a list, forward and backward, and the same
loss (or cross-entropy alone) from hidden states and lm_head weights without the logits.

``listed`` and ``draw`` give cases, ``prepare`` the inputs of one, ``run`` one pass (through the
library where ``own`` is true, else in elementary torch operations), ``work`` the bytes and
operations a pass cannot do without, ``exact`` its outputs in 64 bits.

The teacher of a row is a list of (vocabulary index, logit) pairs, index -1 for an unused place, and
``rest``, the log-sum-exp of all its logits outside the list (None: the list is the whole teacher).
With U the used indices, p = softmax(student) and q = softmax of (listed logits, rest):

  ce    = lse(student) - student[target]
  tvd   = (sum_{v in U} |p_v - q_v| + |p_rest - q_rest|) / 2,  p_rest = sum of p outside U
  sigma = sum_{v in U} p_v sign(p_v - q_v) + p_rest sign(p_rest - q_rest)
  grad_v = grad_ce (p_v - 1[v = target]) + grad_tvd p_v (sign_v - sigma) / 2

where sign_v is sign(p_rest - q_rest) outside U.
"""
import math

import torch

own = False

IGNORE = -100
#: Elements of one block of rows where inputs are made or 64-bit results computed.
BLOCK = 1 << 28

# ---------------------------------------------------------------- cases


def listed():
    return [
        # A handful of rows of a small vocabulary: the teacher's answers of one short sequence.
        dict(name="top_few_f32", op="top", rows=5, vocab=32000, top=8, type="f32"),
        # Caching a teacher's distributions for a training batch.
        dict(name="top_batch_bf16", op="top", rows=8192, vocab=151936, top=64, type="bf16"),
        # Long lists from a large vocabulary in 32 bits.
        dict(name="top_long_f32", op="top", rows=1003, vocab=256000, top=256, type="f32"),
        # The loss of one short sequence against a cached list: latency.
        dict(name="forward_few_bf16", op="forward", rows=37, vocab=32000, top=20, type="bf16",
             rest=True),
        # A training batch, loss and gradient by two calls (autograd's order).
        dict(name="forward_batch_bf16", op="forward", rows=8192, vocab=151936, top=64, type="bf16",
             rest=True),
        dict(name="backward_batch_bf16", op="backward", rows=8192, vocab=151936, top=64,
             type="bf16", rest=True),
        # Upstream gradients known ahead (a mean over tokens): both in one call, logits in 32 bits,
        # lists without the rest of the teacher.
        dict(name="step_long_f32", op="step", rows=1021, vocab=256000, top=256, type="f32",
             rest=False),
        # The loss of a few tokens from hidden states: bound by reading the weights.
        dict(name="linear_few", op="linear_forward", rows=16, vocab=151936, hidden=4096, top=64,
             rest=True),
        # A training batch from hidden states: the forward pass, then the backward pass of half of
        # one at a smaller hidden size.
        dict(name="linear_forward_batch", op="linear_forward", rows=8192, vocab=151936, hidden=4096,
             top=64, rest=True),
        dict(name="linear_backward_batch", op="linear_backward", rows=4096, vocab=151936,
             hidden=2048, top=64, rest=True),
        # Cross-entropy alone from hidden states, an odd number of rows.
        dict(name="linear_backward_ce", op="linear_backward", rows=1001, vocab=32000, hidden=1024,
             top=0, rest=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["top", "top", "forward", "backward", "step", "linear_forward",
                     "linear_backward"])
    vocab = _log(rng, 1000, 256000)
    top = _log(rng, 1, 256)
    if not op.startswith("linear"):
        kind = rng.choice(["bf16", "f32"])
        most = 8192 * 151936 * 2 // ((2 if kind == "bf16" else 4) * vocab)
        case = dict(op=op, rows=_log(rng, 1, min(8192, most)), vocab=vocab, top=top, type=kind)
        return case if op == "top" else dict(case, rest=rng.random() < 0.7)
    hidden = 8 * _log(rng, 8, 512)
    top = 0 if rng.random() < 0.3 else top
    passes = 1 if op == "linear_forward" else 3
    most = 8192 * 4096 * 151936 // (passes * hidden * vocab)
    return dict(op=op, rows=_log(rng, 1, min(8192, most)), vocab=vocab, hidden=hidden, top=top,
                rest=top > 0 and rng.random() < 0.7)


# ---------------------------------------------------------------- inputs

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _blocks(rows, width):
    step = max(1, BLOCK // width)
    return [(at, min(rows, at + step)) for at in range(0, rows, step)]


def _frequency(vocab, gen, dev):
    """Some words are common in every row: 8 rank^-1.1 over a shuffled vocabulary."""
    rank = torch.randperm(vocab, generator=gen, device=dev) + 1
    return 8 * rank.float() ** -1.1


def _list_of(teacher, top, with_rest):
    """The list of a block of teacher logits, and the log-sum-exp of the others."""
    values, index = teacher.topk(top, dim=1)
    rest = None
    if with_rest:
        rest = _lse(teacher.scatter(1, index, -math.inf))
    return values, index.to(torch.int32), rest


def _apart(logits, values, index, rest):
    """The loss's sigma and gradient jump where the student gives a listed word, or the words outside
    the list, exactly the teacher's probability.  A logit that comes within 1e-4 of that is moved by
    0.01, so that what is compared does not hang on the last bits of a logit."""
    used = index >= 0
    at = index.clamp(min=0).long()
    none = torch.full_like(values, -math.inf)
    lse = _lse(logits).unsqueeze(1)
    p = torch.where(used, (logits.gather(1, at) - lse).exp(), torch.zeros_like(lse))
    p_rest = 1 - p.sum(1)
    for _ in range(4):
        teacher = torch.where(used, values, none)
        t_lse = _lse(teacher if rest is None else torch.cat([teacher, rest.unsqueeze(1)], 1))
        near = (p / (teacher - t_lse.unsqueeze(1)).exp() - 1).abs() < 1e-4
        values[near] += 0.01
        if rest is not None:
            near = (p_rest / (rest - t_lse).exp() - 1).abs() < 1e-4
            rest[near] += 0.01


def _unused(values, index, gen):
    """One row in eight has a shorter list: what lies behind its end is not used, whatever its
    value."""
    rows, top = index.shape
    dev = index.device
    short = torch.rand(rows, generator=gen, device=dev) < 0.125
    count = torch.where(short, torch.randint(1, top + 1, (rows,), generator=gen, device=dev), top)
    off = torch.arange(top, device=dev) >= count.unsqueeze(1)
    index[off] = -1
    values[off] = math.nan


def _targets(rows, vocab, index, gen, dev):
    """Words that the teacher holds likely for most rows, any word for some; some rows ignored."""
    target = torch.randint(vocab, (rows,), generator=gen, device=dev)
    if index is not None:
        place = (torch.rand(rows, generator=gen, device=dev) ** 2 * index.shape[1]).long()
        likely = index.gather(1, place.unsqueeze(1)).squeeze(1).long()
        use = (torch.rand(rows, generator=gen, device=dev) < 0.9) & (likely >= 0)
        target = torch.where(use, likely, target)
    target[torch.rand(rows, generator=gen, device=dev) < 0.03] = IGNORE
    return target


def prepare(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    rows, vocab, top = case["rows"], case["vocab"], case["top"]
    state = {"case": case}
    if case["op"].startswith("linear"):
        hidden = case["hidden"]
        state["h"] = torch.randn((rows, hidden), generator=gen, device=dev, dtype=torch.bfloat16)
        w = torch.randn((vocab, hidden), generator=gen, device=dev, dtype=torch.bfloat16)
        state["w"] = w.mul_(3.5 / math.sqrt(hidden))
        logits = lambda a, b: state["h"][a:b].float() @ state["w"].float().t()  # noqa: E731
    else:
        frequency = _frequency(vocab, gen, dev)
        x = torch.empty((rows, vocab), device=dev, dtype=_DTYPE[case["type"]])
        for a, b in _blocks(rows, vocab):
            # heavy tails: a few words hold most of a row
            z = torch.randn((b - a, vocab), generator=gen, device=dev)
            x[a:b] = z * (2.2 + 0.12 * z * z) + frequency
        state["logits"] = x
        if case["op"] == "top":
            return state
        logits = lambda a, b: x[a:b].float()  # noqa: E731
    if top:
        values = torch.empty((rows, top), device=dev)
        index = torch.empty((rows, top), device=dev, dtype=torch.int32)
        rest = torch.empty(rows, device=dev) if case["rest"] else None
        for a, b in _blocks(rows, vocab):
            student = logits(a, b)
            noise = torch.randn((b - a, vocab), generator=gen, device=dev)
            values[a:b], index[a:b], r = _list_of(noise + 0.8 * student, top, case["rest"])
            _unused(values[a:b], index[a:b], gen)
            if rest is not None:
                rest[a:b] = r
            _apart(student, values[a:b], index[a:b], None if rest is None else rest[a:b])
        state |= {"values": values, "index": index, "rest": rest}
    else:
        state |= {"values": None, "index": None, "rest": None}
    state["target"] = _targets(rows, vocab, state["index"], gen, dev)
    if not case["op"].endswith("forward"):
        state["grad_ce"] = torch.rand(rows, generator=gen, device=dev) / rows
        state["grad_tvd"] = torch.rand(rows, generator=gen, device=dev) / rows
    if case["op"].endswith("backward"):
        saved = [torch.empty(rows, device=dev) for _ in range(4)]
        for a, b in _blocks(rows, vocab):
            part = {n: None if state[n] is None else state[n][a:b]
                    for n in ("values", "index", "rest", "target")}
            for to, v in zip(saved, _statistics(logits(a, b), part)[2:]):
                to[a:b] = v
        state["saved"] = saved
    return state


# ---------------------------------------------------------------- plain forms


def _lse(x):
    """Log-sum-exp of each row: a 32-bit sum, its logarithm added to the maximum in 64 bits."""
    m = x.amax(1, keepdim=True)
    m = torch.where(m > -math.inf, m, torch.zeros_like(m))
    return (x - m).exp().sum(1).double().log() + m.squeeze(1).double()


def _statistics(s, given):
    """(ce, tvd, student_lse, student_rest, teacher_lse, sigma) of 32-bit student logits.  What is
    left of the vocabulary's sums, the rows of the lists, is worked out in 64 bits: a distance of two
    nearly equal masses is small beside them."""
    target = given["target"]
    live = target != IGNORE
    lse = _lse(s)
    ce = lse - s.gather(1, target.clamp(min=0).unsqueeze(1)).squeeze(1)
    zero = torch.zeros_like(lse)
    if given["index"] is None:
        return tuple(torch.where(live, v, zero).float() for v in (ce, zero, lse, zero, zero, zero))
    values, index = given["values"], given["index"]
    used = index >= 0
    at = index.clamp(min=0).long()
    none = torch.full_like(values, -math.inf)
    mine = torch.where(used, s.gather(1, at), none)
    outside = s.clone()
    outside.scatter_reduce_(1, at, torch.where(used, none, -none), "amin")
    rest = _lse(outside)
    teacher = torch.where(used, values, none)
    t_rest = given["rest"] if given["rest"] is not None else torch.full_like(lse, -math.inf)
    t_lse = _lse(torch.cat([teacher, t_rest.unsqueeze(1)], 1))
    p = torch.cat([mine, rest.unsqueeze(1)], 1).sub(lse.unsqueeze(1)).exp()
    q = torch.cat([teacher, t_rest.unsqueeze(1)], 1).sub(t_lse.unsqueeze(1)).exp()
    tvd = (p - q).abs().sum(1) / 2
    sigma = (p * (p - q).sign()).sum(1)
    return tuple(torch.where(live, v, zero).float() for v in (ce, tvd, lse, rest, t_lse, sigma))


def _gradient(s, given, saved, grad_ce, grad_tvd):
    """The gradient in 32 bits with respect to 32-bit student logits."""
    lse, rest, t_lse, sigma = saved
    target = given["target"]
    live = (target != IGNORE).unsqueeze(1)
    p = (s - lse.unsqueeze(1)).exp()
    gce, half = grad_ce.unsqueeze(1), grad_tvd.unsqueeze(1) / 2
    if given["index"] is None:
        grad = gce * p
    else:
        values, index = given["values"], given["index"]
        used = index >= 0
        at = index.clamp(min=0).long()
        q = torch.where(used, (values - t_lse.unsqueeze(1)).exp(), torch.zeros_like(values))
        t_rest = given["rest"] if given["rest"] is not None else torch.full_like(lse, -math.inf)
        border = ((rest - lse).exp() - (t_rest - t_lse).exp()).sign().unsqueeze(1)
        mine = p.gather(1, at)
        grad = p * (gce + half * (border - sigma.unsqueeze(1)))
        more = mine * half * ((mine - q).sign() - border)
        grad.scatter_add_(1, at, torch.where(used, more, torch.zeros_like(more)))
    grad.scatter_add_(1, target.clamp(min=0).unsqueeze(1), -gce)
    return torch.where(live, grad, torch.zeros_like(grad))


def _top_plain(x, top):
    """The largest logits, the lowest index first among equal ones, and the others' log-sum-exp."""
    x = x.float() + 0.0  # -0 and +0 are equal
    bits = x.view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long() << 32  # increasing with x
    order -= torch.arange(x.shape[1], device=x.device)
    index = order.topk(top, dim=1).indices
    values = x.gather(1, index)
    return values, index.to(torch.int32), _lse(x.scatter(1, index, -math.inf)).float()


def run(state):
    case = state["case"]
    op, top = case["op"], case["top"]
    if own:
        return _run_own(state, op, top)
    if op == "top":
        return _top_plain(state["logits"], top)
    if not op.startswith("linear"):
        s = state["logits"].float()
        if op == "forward":
            return _statistics(s, state)
        if op == "backward":
            return _gradient(s, state, state["saved"], state["grad_ce"],
                             state["grad_tvd"]).to(state["logits"].dtype)
        found = _statistics(s, state)
        grad = _gradient(s, state, found[2:], state["grad_ce"], state["grad_tvd"])
        return (*found, grad.to(state["logits"].dtype))
    h, w = state["h"].float(), state["w"].float()
    s = h @ w.t()
    if op == "linear_forward":
        found = _statistics(s, state)
        return found if top else (found[0], found[2])
    grad = _gradient(s, state, state["saved"], state["grad_ce"], state["grad_tvd"])
    return (grad @ w).to(state["h"].dtype), (grad.t() @ h).to(state["w"].dtype)


def _run_own(state, op, top):
    from distillation_ce_tvd_gb300 import binding
    if op == "top":
        return binding.fct_top_logits(state["logits"], top)
    target, lists = state["target"], (state["values"], state["index"], state["rest"])
    if op == "forward":
        return binding.fused_ce_tvd_top_forward(state["logits"], target, *lists)
    if op == "backward":
        return binding.fused_ce_tvd_top_backward(state["logits"], target, *lists, *state["saved"],
                                                 state["grad_ce"], state["grad_tvd"])
    if op == "step":
        return binding.fused_ce_tvd_top_forward_backward(state["logits"], target, *lists,
                                                         state["grad_ce"], state["grad_tvd"])
    h, w = state["h"], state["w"]
    if op == "linear_forward":
        if top:
            return binding.fused_linear_ce_tvd_top_forward(h, w, target, *lists)
        return binding.fused_linear_ce_forward(h, w, target)
    if top:
        return binding.fused_linear_ce_tvd_top_backward(h, w, target, *lists, *state["saved"],
                                                        state["grad_ce"], state["grad_tvd"])
    return binding.fused_linear_ce_backward(h, w, target, state["saved"][0], state["grad_ce"])


# ---------------------------------------------------------------- work


def work(case):
    rows, vocab, top, op = case["rows"], case["vocab"], case["top"], case["op"]
    lists = rows * top * 8 + (4 * rows if op == "top" or case["rest"] else 0)
    if op == "top":
        e = 2 if case["type"] == "bf16" else 4
        return {"bytes": rows * vocab * e + lists, "flops": 3 * rows * vocab}
    scalars = {"forward": 8 + 24, "backward": 8 + 16 + 8, "step": 8 + 8 + 24}
    if not op.startswith("linear"):
        e = 2 if case["type"] == "bf16" else 4
        passes = 1 if op == "forward" else 2
        flops = {"forward": 3, "backward": 4, "step": 7}[op] * rows * vocab
        return {"bytes": passes * rows * vocab * e + lists + scalars[op] * rows, "flops": flops}
    hidden = case["hidden"]
    inputs = 2 * hidden * (rows + vocab) + lists
    product = 2 * rows * vocab * hidden
    if op == "linear_forward":
        return {"bytes": inputs + 32 * rows, "flops": product}
    return {"bytes": inputs + 32 * rows + 2 * hidden * (rows + vocab), "flops": 3 * product}


# ---------------------------------------------------------------- 64 bits


def exact(case, seed):
    state = prepare(case, seed)
    rows, vocab, top, op = case["rows"], case["vocab"], case["top"], case["op"]
    linear = op.startswith("linear")
    if linear and 2 * rows * vocab * case["hidden"] * (1 if op == "linear_forward" else 3) > 1.5e13:
        return None
    w = state["w"].double() if linear else None
    parts, grad_w = [], None
    for a, b in _blocks(rows, 2 * vocab):
        s = state["h"][a:b].double() @ w.t() if linear else state["logits"][a:b].double()
        if op == "top":
            # a stable ascending order of the negated values: equal ones stay by index
            index = torch.sort(-s, dim=1, stable=True).indices[:, :top]
            taken = torch.zeros_like(s, dtype=torch.bool).scatter_(1, index, True)
            parts.append((s.gather(1, index), index.to(torch.int32),
                          torch.logsumexp(s.masked_fill(taken, -math.inf), 1)))
            continue
        cut = {n: None if state.get(n) is None else state[n][a:b]
               for n in ("values", "index", "rest", "target", "grad_ce", "grad_tvd")}
        given = None if "saved" not in state else [v[a:b].double() for v in state["saved"]]
        found, grad = _exact_rows(s, cut, given)
        if op == "forward" or op == "linear_forward":
            parts.append(found if top else (found[0], found[2]))
        elif op == "backward":
            parts.append((grad.to(torch.float32),))
        elif op == "step":
            parts.append((*found, grad.to(torch.float32)))
        else:
            parts.append(((grad @ w).to(torch.float32),))
            more = grad.t() @ state["h"][a:b].double()
            grad_w = more if grad_w is None else grad_w.add_(more)
    out = [torch.cat(p) for p in zip(*parts)]
    if op == "linear_backward":
        return out[0], grad_w.to(torch.float32)
    return out[0] if op == "backward" else tuple(out)


def _exact_rows(s, cut, given):
    """The definition, row block by row block: statistics and, with upstream gradients, gradient.
    Where the statistics are inputs (``given``), the gradient is the formula at those."""
    n, vocab = s.shape
    target = cut["target"]
    dead = target == IGNORE
    rows = torch.arange(n, device=s.device)
    label = torch.where(dead, 0, target)
    lse = torch.logsumexp(s, 1)
    ce = lse - s[rows, label]
    # every word's teacher probability, or -1 where the list does not have it
    has_list = cut["index"] is not None
    nothing = s.new_zeros(n)
    tvd, rest, t_lse, sigma = nothing, nothing, nothing, nothing
    if has_list:
        at_row, at_col = (cut["index"] >= 0).nonzero(as_tuple=True)
        word = cut["index"][at_row, at_col].long()
        inside = torch.zeros((n, vocab), dtype=torch.bool, device=s.device)
        inside[at_row, word] = True
        logit = torch.full((n, vocab), -math.inf, dtype=torch.float64, device=s.device)
        logit[at_row, word] = cut["values"][at_row, at_col].double()
        t_rest = (cut["rest"].double() if cut["rest"] is not None
                  else torch.full((n,), -math.inf, dtype=torch.float64, device=s.device))
        t_lse = torch.logaddexp(torch.logsumexp(logit, 1), t_rest)
        rest = torch.logsumexp(s.masked_fill(inside, -math.inf), 1)

    def signs(lse, rest, t_lse):
        p = torch.exp(s - lse[:, None])
        if not has_list:
            return p, nothing, torch.zeros_like(s), nothing, nothing
        p_rest, q_rest = torch.exp(rest - lse), torch.exp(t_rest - t_lse)
        gap = p - torch.exp(logit - t_lse[:, None])
        border = torch.sign(p_rest - q_rest)
        side = torch.where(inside, torch.sign(gap), border[:, None])
        return p, p_rest, side, (gap.abs() * inside).sum(1) + (p_rest - q_rest).abs(), border

    p, p_rest, side, distance, border = signs(lse, rest, t_lse)
    if has_list:
        tvd = distance / 2
        sigma = (p * side * inside).sum(1) + p_rest * border
    found = tuple(torch.where(dead, nothing, v) for v in (ce, tvd, lse, rest, t_lse, sigma))
    if cut["grad_ce"] is None:
        return found, None
    if given is not None:
        p, _, side, _, _ = signs(*given[:3])
        sigma = given[3]
    gce, gtvd = cut["grad_ce"].double()[:, None], cut["grad_tvd"].double()[:, None]
    grad = gce * p
    if has_list:
        grad = grad + gtvd / 2 * p * (side - sigma[:, None])
    grad[rows, label] -= gce[:, 0]
    return found, grad.masked_fill(dead[:, None], 0.0)
