"""Plain 64-bit forms of distillation from a teacher's top logits, on the CPU, a row at a time, and
bounds of how far the kernels' 32-bit values may be from them.

Bounds count roundings (u = 2^-24, half a step of float32).  With `terms` the longest chain of
additions of one partial sum:

  PROB  relative error of a probability from the maximum and the sum: ex2's error (2^-22), the
        exponent's rounding (u |x - m| log2 e, times e^-|x - m| at most 0.4 u), the constant log2 e
        (2^-26 relative, the same), the division and the sum (terms u + 2^-22).
  LSE   absolute error of a log-sum-exp: u |lse| for its rounding, 2^-26 |max| for the constant,
        and the sum's relative error.
"""
import math

import torch

U = 2.0 ** -24
IGNORE = -100


def terms(V):
    return V / 512 + 32          # a thread's vectors (8 or 4 wide, two chains) and the trees above


def sum_error(V):
    return terms(V) * U + 2.0 ** -22


def lse_tol(lse, top, V):
    return U * abs(lse) + 2.0 ** -25 * abs(top) + sum_error(V) + 2.0 ** -23


def top_ref(row, K):
    """(values, index, rest) of one row: K places, -1 where there is nothing above -inf."""
    x = [float(v) for v in row.double()]
    order = sorted((i for i in range(len(x)) if x[i] > -math.inf), key=lambda i: (-x[i], i))
    pick, left = order[:K], order[K:]
    rest = -math.inf
    if left:
        m = x[left[0]]
        rest = m + math.log(math.fsum(math.exp(x[i] - m) for i in left))
    values = [x[i] for i in pick] + [-math.inf] * (K - len(pick))
    return values, pick + [-1] * (K - len(pick)), rest


def _lse(x):
    return torch.logsumexp(x, 0).item() if x.numel() else -math.inf


def row_ref(s, target, values, index, rest, gce=0.0, gtvd=0.0, err=0.0):
    """The definition for one row of float64 logits, which the kernel may see up to ``err`` off.
    Returns a dict with the statistics, the gradient, and bounds of the error of each."""
    V = s.numel()
    zero = torch.zeros(V, dtype=torch.float64)
    if target == IGNORE:
        return dict(ce=0.0, tvd=0.0, lse=0.0, rest=0.0, t_lse=0.0, sigma=0.0, grad=zero,
                    tol=dict(ce=0.0, tvd=0.0, lse=0.0, rest=0.0, t_lse=0.0, sigma=0.0, grad=zero))
    used = index >= 0
    words = index[used].long()
    t = values[used].double()
    inside = torch.zeros(V, dtype=torch.bool)
    inside[words] = True
    lse, s_rest = _lse(s), _lse(s[~inside])
    t_rest = -math.inf if rest is None else float(rest)
    t_all = torch.cat([t, torch.tensor([t_rest], dtype=torch.float64)])
    t_lse = _lse(t_all)
    p = torch.exp(s - lse)
    p_rest = math.exp(s_rest - lse)
    top_s, top_t = s.max().item(), t_all.max().item()
    tol = dict(lse=lse_tol(lse, top_s, V) + err,
               ce=lse_tol(lse, top_s, V) + U * abs(lse - s[target].item()) + 2 * err,
               rest=lse_tol(s_rest, s[~inside].max().item(), V) + err if s_rest > -math.inf else 0.0)
    prob = 2.0 ** -21 + sum_error(V) + 2 * err          # PROB
    saved = prob + 2 * lse_tol(lse, top_s, V) + 2 * err  # exp(s - lse) with the rounded lse
    if t_lse == -math.inf:
        side, sigma, tvd, flip, sigma_tol = zero, 0.0, 0.0, zero, 0.0
        tol |= dict(t_lse=0.0, tvd=0.0, sigma=0.0)
    else:
        q = torch.exp(t - t_lse)
        q_rest = math.exp(t_rest - t_lse)
        gap = p[words] - q
        tvd = 0.5 * (gap.abs().sum().item() + abs(p_rest - q_rest))
        side = torch.full((V,), float((p_rest > q_rest) - (p_rest < q_rest)), dtype=torch.float64)
        side[words] = torch.sign(gap)
        sigma = (p[words] * side[words]).sum().item() + \
            p_rest * ((p_rest > q_rest) - (p_rest < q_rest))
        # signs that the rounded values may see differently
        t_saved = prob + 2 * lse_tol(t_lse, top_t, V)
        rest_saved = 2 * tol["rest"]
        close = torch.zeros(V, dtype=torch.bool)
        rest_close = abs(p_rest - q_rest) <= (saved + rest_saved) * p_rest + t_saved * q_rest
        close[~inside] = rest_close
        close[words] = gap.abs() <= saved * p[words] + t_saved * q
        flip = 2.0 * close.double()
        flip_mass = 2 * p[words][close[words]].sum().item() + (2 * p_rest if rest_close else 0.0)
        sigma_tol = flip_mass + 2 * prob + 2 * U
        # masses of the two sides, or of what they hold inside where both are large
        tol |= dict(t_lse=lse_tol(t_lse, top_t, V), tvd=2 * prob * 1.0 + U, sigma=sigma_tol)
    grad = gce * p + 0.5 * gtvd * p * (side - sigma)
    grad_tol = p * ((abs(gce) + abs(gtvd)) * (saved + 4 * U) + 0.5 * abs(gtvd) * (flip + sigma_tol))
    grad[target] -= gce
    grad_tol[target] += 2 * U * abs(gce)
    tol["grad"] = grad_tol
    return dict(ce=lse - s[target].item(), tvd=tvd, lse=lse, rest=s_rest, t_lse=t_lse, sigma=sigma,
                grad=grad, tol=tol)


NAMES = ("ce", "tvd", "lse", "rest", "t_lse", "sigma")


def close(got, want, tol):
    if math.isnan(want) or math.isinf(want):
        return got == want or (math.isnan(got) and math.isnan(want))
    return abs(got - want) <= tol


def check_rows(stats, grad, s, target, values, index, rest, gce=None, gtvd=None):
    """Compares the kernels' six (BT,) statistics and the gradient (either may be None) with the
    definition, row by row.  Everything on the CPU, s as given to the kernel."""
    for r in range(s.shape[0]):
        want = row_ref(s[r].double(), int(target[r]), values[r], index[r],
                       None if rest is None else float(rest[r]),
                       0.0 if gce is None else float(gce[r]), 0.0 if gtvd is None else float(gtvd[r]))
        if stats is not None:
            for name, x in zip(NAMES, stats):
                assert close(float(x[r]), want[name], want["tol"][name]), \
                    (r, name, float(x[r]), want[name], want["tol"][name])
        if grad is not None:
            tol = want["tol"]["grad"] + want["grad"].abs() * torch.finfo(grad.dtype).eps / 2 + 1e-38
            off = (grad[r].double() - want["grad"]).abs() - tol
            assert bool((off <= 0).all()), (r, off.argmax().item(), off.max().item())


def make(rows, V, K, dtype, seed, rest=True, spread=3.0, device="cpu"):
    """Student logits, targets, and a teacher's list in random order with unused places."""
    g = torch.Generator().manual_seed(seed)
    s = torch.randn(rows, V, generator=g) * spread
    t = 0.8 * s + torch.randn(rows, V, generator=g)
    n = min(K, V)
    index = torch.full((rows, K), -1, dtype=torch.int32)
    values = torch.full((rows, K), math.nan)
    rests = torch.empty(rows)
    for r in range(rows):
        want = n if r % 4 else max(0, n - 3)
        words = t[r].topk(want).indices if want else torch.empty(0, dtype=torch.long)
        places = torch.randperm(K, generator=g)[:want]
        index[r, places] = words.to(torch.int32)
        values[r, places] = t[r][words]
        outside = torch.ones(V, dtype=torch.bool)
        outside[words] = False
        rests[r] = torch.logsumexp(t[r][outside], 0) if outside.any() else -math.inf
    target = torch.randint(V, (rows,), generator=g)
    if rows > 2:
        target[2] = IGNORE
    gce = torch.rand(rows, generator=g)
    gtvd = torch.rand(rows, generator=g) - 0.3
    return s.to(dtype), target, values, index, rests if rest else None, gce, gtvd
