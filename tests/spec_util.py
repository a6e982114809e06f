"""Plain 64-bit forms of the speculative decoding step, on the CPU, one request and one head at a
time, and builders of its inputs."""
import math

import torch

E4M3 = torch.float8_e4m3fn


def values_of(payload, byte=None):
    """What a cache holds, as float64 (byte 255 is NaN)."""
    x = payload.cpu().double()
    if byte is None:
        return x
    e = byte.cpu().double()
    scale = torch.where(e == 255, torch.full_like(e, math.nan), torch.exp2(e - 127))
    return x * scale.unsqueeze(-1)


def quantise_ref(x):
    """(payload values, exponent byte) of vectors (..., D) by the definition, in float64."""
    x = x.double()
    bad = ~torch.isfinite(x).all(-1)
    x = torch.where(bad.unsqueeze(-1), torch.zeros_like(x), x)
    amax = x.abs().amax(-1)
    e = torch.full_like(amax, -126.0)
    for _ in range(260):            # the smallest e >= -126 with amax <= 448 * 2^e
        e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    y = x / torch.exp2(e).unsqueeze(-1)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    y = torch.round(y / step) * step
    return y, torch.where(bad, torch.full_like(e, 255 - 127), e).add(127).to(torch.uint8)


def make_pool(pages, page, heads, dim, dtype, gen, device, layout="nhd", scale=1.0):
    """k, v (pages, page, heads, dim) and exponent bytes (None for bf16); ``layout`` hnd keeps a
    page's heads apart, pair puts K and V of a page next to each other."""
    def blank(last, dt):
        if layout == "hnd":
            return [torch.zeros((pages, heads, page) + last, dtype=dt, device=device).transpose(1, 2)
                    for _ in range(2)]
        if layout == "pair":
            both = torch.zeros((pages, 2, page, heads) + last, dtype=dt, device=device)
            return [both[:, 0], both[:, 1]]
        return [torch.zeros((pages, page, heads) + last, dtype=dt, device=device) for _ in range(2)]
    pool = blank((dim,), dtype)
    scales = blank((), torch.uint8) if dtype == E4M3 else (None, None)
    for x, s in zip(pool, scales):
        r = torch.randn((pages, page, heads, dim), generator=gen, device=device) * scale
        if dtype == E4M3:
            x.view(torch.uint8).copy_(r.to(E4M3).view(torch.uint8))
            s.copy_(torch.randint(125, 130, s.shape, generator=gen, device=device))
        else:
            x.copy_(r.to(dtype))
    return pool[0], pool[1], scales[0], scales[1]


def make_tables(lengths, page, gen, spare=2):
    """Scattered pages for requests of these lengths: (table int32 (B, width), pages in the pool)."""
    need = [-(-n // page) for n in lengths]
    total = sum(need) + spare
    order = torch.randperm(total, generator=gen).tolist()
    width = max(1, max(need))
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n] + [-1] * (width - n))
        at += n
    return torch.tensor(rows, dtype=torch.int32), total


def random_tree(n, rnd, most_children=4):
    parent, kids = [-1], [0] * n
    for i in range(1, n):
        p = rnd.randrange(i)
        while kids[p] >= most_children:
            p = rnd.randrange(i)
        kids[p] += 1
        parent.append(p)
    return parent


def ancestor_masks(parents, words):
    """(sum of nodes, words) int64 of node-or-above bits for a list of parent lists."""
    rows = []
    for parent in parents:
        seen = []
        for i, p in enumerate(parent):
            seen.append((1 << i) | (seen[p] if p >= 0 else 0))
        for v in seen:
            row = [(v >> (64 * w)) & (2 ** 64 - 1) for w in range(words)]
            rows.append([x - 2 ** 64 if x >= 2 ** 63 else x for x in row])
    return torch.tensor(rows, dtype=torch.int64)


def attention_ref(q, k, v, table, page, contexts, starts, mask, scale):
    """(out, lse, bound): float64 attention, and per output the sum of |weight| * |value|."""
    N, H, D = q.shape
    group = H // k.shape[2]
    out = torch.zeros(N, H, D, dtype=torch.float64)
    lse = torch.full((N, H), -math.inf, dtype=torch.float64)
    bound = torch.zeros(N, H, D, dtype=torch.float64)
    q = q.cpu().double()
    for b, ctx in enumerate(contexts):
        n0, n1 = starts[b], starts[b + 1]
        pos = torch.arange(ctx + n1 - n0)
        ids = table[b, pos // page].long()
        kk, vv = k[ids, pos % page], v[ids, pos % page]
        for i in range(n1 - n0):
            sees = pos < ctx
            for j in range(n1 - n0):
                if mask is None:
                    sees[ctx + j] = j <= i
                else:
                    word = int(mask[n0 + i, j // 64]) if j // 64 < mask.shape[1] else 0
                    sees[ctx + j] = bool((word >> (j % 64)) & 1)
            if not sees.any():
                continue
            for h in range(H):
                s = kk[sees][:, h // group] @ q[n0 + i, h] * scale
                m = s.max()
                w = torch.exp(s - m)
                x = vv[sees][:, h // group]
                out[n0 + i, h] = (w @ x) / w.sum()
                bound[n0 + i, h] = (w @ x.abs()) / w.sum()
                lse[n0 + i, h] = m + torch.log(w.sum())
    return out, lse, bound


def verify_ref(target, draft, tokens, parent, starts, uniform, noise, temperature, max_depth):
    """(out_tokens, path, count, margin): the walk in float64; margin is the smallest relative
    distance of a decision (a test of a child, the race's winner) from going the other way."""
    V = target.shape[1]
    toks, paths, counts, margins = [], [], [], []
    for b in range(len(starts) - 1):
        first, end = starts[b], starts[b + 1]
        T = 1.0 if temperature is None else float(temperature[b])
        at, walk, last, margin = first, [], -1, math.inf
        while end > first:
            z = target[at].double()
            kids = [c for c in range(at + 1, end)
                    if parent[c] >= 0 and first + parent[c] == at and len(walk) < max_depth]
            zq = draft[at].double() if draft is not None and kids else None

            def fine(x):
                return not bool(torch.isnan(x).any()) and not bool((x == math.inf).any()) \
                    and bool((x > -math.inf).any())
            if not fine(z) or (zq is not None and T > 0 and not fine(zq)):
                last = -1
                break
            if T > 0:
                p = torch.softmax(z / T, 0)
            else:
                p = torch.zeros(V, dtype=torch.float64)
                p[int((z == z.max()).nonzero()[0])] = 1.0
            q = torch.softmax(zq / T, 0) if zq is not None and T > 0 else None
            r, S, Z, hit = p.clone(), 0.0, 1.0, None
            for c in kids:
                x = int(tokens[c])
                inside = 0 <= x < V
                rx = float(r[x]) if inside else 0.0
                qx = (float(q[x]) if inside else 0.0) if q is not None else 1.0
                if T <= 0:
                    if rx > 0:
                        hit = c
                        break
                    continue
                left = float(uniform[c]) * Z * qx
                if inside and max(left, rx) > 0:
                    margin = min(margin, abs(left - rx) / max(left, rx))
                if left < rx:
                    hit = c
                    break
                if q is not None:
                    S += Z
                    r = (p - S * q).clamp(min=0)
                elif inside:
                    r[x] = 0.0
                Z = float(r.sum())
            if hit is not None:
                walk.append(hit)
                at = hit
                continue
            if not bool((r > 0).any()):
                r = p
            race = torch.where(r > 0, r / noise[b].double(), torch.full_like(r, -math.inf))
            last = int((race == race.max()).nonzero()[0])
            if T > 0 and V > 1 and int((r > 0).sum()) > 1:
                two = torch.topk(race, 2).values
                # the residual is a difference: its error is that of p and S q
                margin = min(margin, float((two[0] - two[1]) / two[0] * r[last] / (p[last] + 1e-300)))
            break
        toks.append([int(tokens[c]) for c in walk] + [last] + [-1] * (max_depth - len(walk)))
        if end <= first:
            toks[-1] = [-1] * (max_depth + 1)
        paths.append([c - first for c in walk] + [-1] * (max_depth - len(walk)))
        counts.append(len(walk))
        margins.append(margin)
    return (torch.tensor(toks), torch.tensor(paths, dtype=torch.int32).reshape(len(counts), max_depth),
            torch.tensor(counts, dtype=torch.int32), margins)
