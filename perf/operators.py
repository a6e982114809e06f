"""Cases of the speculative-decoding operators: the key/value cache written and compacted, attention
of drafted trees over it, and the verification of drafted tokens.

``listed`` and ``draw`` give cases, ``prepare`` the inputs of one, ``run`` one pass (through the
library where ``own`` is true, else in elementary torch operations), ``work`` the bytes and
operations a pass cannot do without, ``exact`` its outputs in 64 bits.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
PAGES_SPARE = 3

# ---------------------------------------------------------------- cases


def listed():
    return [
        # One decode step of a small batch: the new tokens' keys and values, one call per layer.
        dict(name="write_step_e4m3", op="write", tokens=67, heads=8, dim=128, page=16, cache="e4m3",
             source="bf16"),
        # A long prompt going into the cache in one call; the last page is part filled.
        dict(name="write_prompt_e4m3", op="write", tokens=16389, heads=8, dim=128, page=64,
             cache="e4m3", source="bf16"),
        # After a verified step of a few requests: the accepted path moves to the tree's front.
        dict(name="move_step_bf16", op="move", batch=3, nodes=16, depth=5, heads=8, dim=128, page=16,
             cache="bf16", context=700),
        # The same for a large batch over an 8-bit cache (payload and scales).
        dict(name="move_batch_e4m3", op="move", batch=256, nodes=32, depth=8, heads=8, dim=128,
             page=64, cache="e4m3", context=900),
        # Plain decoding, one token per request, short contexts: latency.
        dict(name="attend_token_bf16", op="attend", batch=2, nodes=1, q_heads=16, heads=8, dim=64,
             page=16, cache="bf16", context=333, context_min=61, tree="chain"),
        # A served batch, a short drafted chain each, ragged contexts.
        dict(name="attend_chain_bf16", op="attend", batch=48, nodes=5, q_heads=32, heads=8, dim=128,
             page=16, cache="bf16", context=8190, context_min=450, tree="chain"),
        # The same from an 8-bit cache, with drafted trees.
        dict(name="attend_tree_e4m3", op="attend", batch=20, nodes=27, q_heads=32, heads=8, dim=128,
             page=64, cache="e4m3", context=16300, context_min=2000, tree="tree"),
        # One request over a long document: few rows, a long axis.
        dict(name="attend_long_bf16", op="attend", batch=1, nodes=8, q_heads=32, heads=8, dim=128,
             page=128, cache="bf16", context=131071, context_min=131071, tree="tree"),
        # Wide trees and wide groups: many rows per key, bound by the products.
        dict(name="attend_wide_tree_bf16", op="attend", batch=12, nodes=64, q_heads=64, heads=8,
             dim=128, page=32, cache="bf16", context=9001, context_min=2500, tree="tree"),
        # One request, four drafted tokens, a small vocabulary: latency.
        dict(name="verify_one_f32", op="verify", batch=1, nodes=5, depth=4, vocab=32000, type="f32",
             draft=True, tree="chain"),
        # A served batch, seven drafted tokens each from a distilled draft model.
        dict(name="verify_chain_bf16", op="verify", batch=64, nodes=8, depth=7, vocab=151936,
             type="bf16", draft=True, tree="chain"),
        # Trees of the draft's best tokens, no draft distribution; some requests greedy.
        dict(name="verify_tree_bf16", op="verify", batch=24, nodes=32, depth=6, vocab=151936,
             type="bf16", draft=False, tree="tree"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "move", "attend", "attend", "attend", "verify", "verify"])
    cache = rng.choice(["bf16", "e4m3"])
    page = rng.choice([8, 16, 32, 48, 64, 128])
    dim = rng.choice([64, 128])
    heads = rng.choice([1, 2, 4, 8])
    if op == "write":
        return dict(op=op, tokens=_log(rng, 1, 16389), heads=heads, dim=dim, page=page, cache=cache,
                    source=rng.choice(["bf16", "f32"]))
    if op == "move":
        return dict(op=op, batch=_log(rng, 1, 256), nodes=_log(rng, 9, 64), depth=rng.randint(2, 8),
                    heads=heads, dim=dim, page=page, cache=cache, context=_log(rng, 1, 900))
    if op == "attend":
        nodes = _log(rng, 1, 64)
        group = rng.choice([1, 2, 3, 4, 7, 8])
        context = _log(rng, 17, 131071)
        # at most the work of the largest listed case, and at most its keys
        keys = 12 * 9001 * 8
        most = min(keys // (heads * context), 12 * 9001 * 512 * 8 // (context * nodes * group * heads))
        batch = _log(rng, 1, max(1, min(48, most)))
        return dict(op=op, batch=batch, nodes=nodes, q_heads=heads * group, heads=heads, dim=dim,
                    page=page, cache=cache, context=context,
                    context_min=rng.randint(0, max(1, context // 2)),
                    tree=rng.choice(["chain", "tree"]))
    chain = rng.random() < 0.5
    depth = rng.randint(1, 8)
    nodes = depth + 1 if chain else _log(rng, depth + 1, 40)
    vocab = _log(rng, 1000, 256000)
    batch = _log(rng, 1, max(1, min(64, 64 * 16 * 151936 // (2 * nodes * vocab))))
    return dict(op=op, batch=batch, nodes=nodes, depth=depth, vocab=vocab,
                type=rng.choice(["bf16", "f32"]), draft=chain or rng.random() < 0.5,
                tree="chain" if chain else "tree")


# ---------------------------------------------------------------- inputs

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
#: What a verified tree node's first, second, ... child takes of the target's probability.
_SHARES = (0.45, 0.2, 0.1, 0.05)


def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _node_counts(case):
    """Nodes per request: the first has all of case["nodes"], the others that or fewer (the same for
    every seed, so that the outputs' shapes are)."""
    most, rng = case["nodes"], random.Random(case["batch"] * 1009 + case["nodes"])
    least = most if case.get("tree") == "chain" else max(1, most // 2)
    return [most] + [rng.randint(least, most) for _ in range(case["batch"] - 1)]


def _parents(count, kind, depth, rng):
    """Parents (local indexes, -1 for the root) of a tree of `count` nodes, at most four children
    each and at most `depth` edges deep."""
    if kind == "chain":
        return [-1] + list(range(count - 1))
    parent, level, children = [-1], [0], [0]
    for i in range(1, count):
        # the first `depth` nodes form a chain, so that the depth is reached
        at = i - 1 if i <= depth else rng.randrange(i)
        while level[at] >= depth or children[at] >= 4:
            at = rng.randrange(i)
        parent.append(at)
        level.append(level[at] + 1)
        children.append(0)
        children[at] += 1
    return parent


def _ancestors(parent):
    """Per node the integer whose bit j says that node j is the node itself or above it."""
    seen = []
    for i, at in enumerate(parent):
        seen.append((1 << i) | (seen[at] if at >= 0 else 0))
    return seen


def _words(values, width):
    """(n, width) signed 64-bit words, lowest bits first."""
    rows = []
    for v in values:
        row = [(v >> (64 * w)) & ((1 << 64) - 1) for w in range(width)]
        rows.append([x - (1 << 64) if x >> 63 else x for x in row])
    return rows


def quantise(x):
    """e4m3 payload and exponent byte of vectors along the last dimension: the smallest power of two
    2^(byte - 127), not below 2^-126, under which no value passes 448."""
    x = x.float()
    amax = x.abs().amax(-1)
    mant, exp = torch.frexp(amax)               # amax = mant * 2^exp, mant in [0.5, 1)
    power = torch.where(mant > E4M3_MAX / 512, exp - 8, exp - 9)
    power = torch.where(amax > 0, power, torch.full_like(power, -126)).clamp_(min=-126)
    payload = torch.ldexp(x, -power.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return payload, (power + 127).to(torch.uint8)


def _dequantise(payload, byte):
    return torch.ldexp(payload.float(), (byte.to(torch.int32) - 127).unsqueeze(-1))


def _cache(case, pages, gen, dev):
    """A pool of pages holding keys and values as a model's projections give them."""
    shape = (pages, case["page"], case["heads"], case["dim"])
    state = {}
    for name in ("k", "v"):
        x = torch.randn(shape, generator=gen, device=dev, dtype=torch.bfloat16)
        if case["cache"] == "e4m3":
            state[name], state[name + "_scale"] = quantise(x)
        else:
            state[name], state[name + "_scale"] = x, None
    if own:
        from distillation_ce_tvd_gb300 import binding
        state["cache"] = binding.KVCache(state["k"], state["v"], state["k_scale"], state["v_scale"])
    return state


def _tables(case, lengths, rng, dev):
    """A block table whose pages are scattered over the pool, and the pool's size."""
    page = case["page"]
    need = [-(-n // page) for n in lengths]
    pool = list(range(sum(need) + PAGES_SPARE))
    rng.shuffle(pool)
    width = max(1, max(need))
    table, at = [], 0
    for n in need:
        table.append(pool[at:at + n] + [-1] * (width - n))
        at += n
    return torch.tensor(table, dtype=torch.int32, device=dev), len(pool)


def prepare(case, seed):
    dev = _device()
    rng = random.Random(seed)
    gen = torch.Generator(device=dev).manual_seed(seed)
    ints = lambda v, t=torch.int32: torch.tensor(v, dtype=t, device=dev)  # noqa: E731
    if case["op"] == "write":
        n, page = case["tokens"], case["page"]
        pages = -(-n // page) + PAGES_SPARE
        state = _cache(case, pages, gen, dev)
        order = torch.randperm(pages, generator=gen, device=dev)
        at = torch.arange(n, device=dev)
        state["slots"] = order[at // page] * page + at % page
        # a projection's output: keys and values side by side in one row per token
        kv = torch.randn((n, 2, case["heads"], case["dim"]), generator=gen, device=dev)
        kv *= torch.rand((n, 2, case["heads"], 1), generator=gen, device=dev) * 3 + 0.1
        kv = kv.to(_DTYPE[case["source"]])
        return {"case": case, **state, "new_k": kv[:, 0], "new_v": kv[:, 1]}
    counts = _node_counts(case)
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    depth = case.get("depth", 8)
    parents = [_parents(c, case.get("tree", "tree"), min(depth, c - 1) if c > 1 else 1, rng)
               for c in counts]
    state = {"case": case, "node_start": ints(starts)}
    if case["op"] in ("move", "attend"):
        low = case.get("context_min", case["context"])
        contexts = [case["context"]] + [rng.randint(min(low, case["context"]), case["context"])
                                        for _ in range(case["batch"] - 1)]
        table, pages = _tables(case, [c + n for c, n in zip(contexts, counts)], rng, dev)
        state |= _cache(case, pages, gen, dev)
        state |= {"block_table": table, "context_len": ints(contexts)}
    if case["op"] == "move":
        path = []
        for p in parents:
            at, walk = 0, []
            while True:  # a path from the root: a random child each time
                below = [i for i, q in enumerate(p) if q == at]
                if not below or len(walk) == depth or rng.random() < 0.2:
                    break
                at = rng.choice(below)
                walk.append(at)
            path.append(walk)
        state["path"] = ints([w + [-1] * (depth - len(w)) for w in path])
        state["count"] = ints([len(w) for w in path])
    elif case["op"] == "attend":
        q = torch.randn((starts[-1], case["q_heads"], case["dim"]), generator=gen, device=dev)
        state["q"] = (q * 2).to(torch.bfloat16)
        if case["tree"] == "tree":
            width = -(-max(counts) // 64)
            state["tree_mask"] = ints([w for p in parents for w in _words(_ancestors(p), width)],
                                      torch.int64)
        else:
            state["tree_mask"] = None
        if own:
            from distillation_ce_tvd_gb300 import binding
            state["workspace"] = torch.empty(
                binding.fct_tree_attention_workspace_size(starts[-1], case["q_heads"],
                                                          case["heads"], case["dim"]),
                dtype=torch.uint8, device=dev)
    elif case["op"] == "verify":
        state |= _verify_inputs(case, starts, parents, gen, rng, dev)
    return state


def _verify_inputs(case, starts, parents, gen, rng, dev):
    n, vocab, dtype = starts[-1], case["vocab"], _DTYPE[case["type"]]
    parent = torch.tensor([q for p in parents for q in p], dtype=torch.int32, device=dev)
    first = torch.tensor([s for s, p in zip(starts, parents) for _ in p], device=dev)
    above = (first + parent.long()).clamp_(min=0)
    target = torch.randn((n, vocab), generator=gen, device=dev) * 1.5
    tokens = torch.randint(0, vocab, (n,), generator=gen, device=dev)
    out = {}
    if case["draft"]:
        # a draft distilled from the target: its logits with an error of half a unit; each node's
        # token drawn from the draft's distribution at its parent
        draft = target + torch.randn((n, vocab), generator=gen, device=dev) * 0.5
        out["draft"] = draft.to(dtype)
        race = torch.empty((n, vocab), device=dev).exponential_(generator=gen).log_()
        drawn = (out["draft"].float()[above] - race).argmax(-1)
        tokens = torch.where(parent >= 0, drawn, tokens)
    else:
        # the draft's best tokens: they hold most of the target's probability at their parent
        out["draft"] = None
        rank, seen = [], {}
        for s, p in zip(starts, parents):
            for q in p:
                rank.append(seen.get((s, q), 0) if q >= 0 else 0)
                seen[(s, q)] = seen.get((s, q), 0) + 1
        share = torch.tensor([_SHARES[r] for r in rank], device=dev)
        rest = math.log(vocab) + 1.5 ** 2 / 2 - math.log(1 - sum(_SHARES))
        kids = (parent >= 0).nonzero()[:, 0]
        target[above[kids], tokens[kids]] = torch.log(share[kids]) + rest
    out |= {"target": target.to(dtype), "tokens": tokens, "parent": parent}
    out["widest"] = max(p.count(q) for p in parents for q in p)
    out["uniform"] = torch.rand((n,), generator=gen, device=dev)
    out["noise"] = torch.empty((case["batch"], vocab), device=dev).exponential_(generator=gen)
    heat = [rng.choice([0.7, 1.0, 1.0, 1.3]) for _ in range(case["batch"])]
    if not case["draft"]:
        heat = [0.0 if rng.random() < 0.25 else 1.0 for _ in heat]
    out["temperature"] = torch.tensor(heat, device=dev)
    return out


# ---------------------------------------------------------------- plain forms


def _plain_write(s):
    page = s["case"]["page"]
    at = (s["slots"] // page, s["slots"] % page)
    for name in ("k", "v"):
        x = s["new_" + name]
        if s["case"]["cache"] == "e4m3":
            payload, byte = quantise(x)
            s[name].view(torch.uint8)[at] = payload.view(torch.uint8)
            s[name + "_scale"][at] = byte
        else:
            s[name][at] = x.float().to(torch.bfloat16)
    return _pool(s)


def _pool(s):
    return {n: s[n] for n in ("k", "v", "k_scale", "v_scale")}


def _plain_move(s):
    page, path = s["case"]["page"], s["path"].long()
    step = torch.arange(path.shape[1], device=path.device)
    live = step < s["count"][:, None]
    start = s["context_len"].long()[:, None]
    table = s["block_table"].long()

    def slots(position):
        pages = table.gather(1, (position // page).clamp(max=table.shape[1] - 1))
        return (pages * page + position % page)[live]

    src, dst = slots(start + path.clamp(min=0)), slots((start + 1 + step).expand_as(path))
    for x in _pool(s).values():
        if x is not None:
            flat = (x.view(torch.uint8) if x.element_size() == 1 else x).flatten(0, 1)
            flat[dst] = flat[src]
    return _pool(s)


def _plain_attend(s):
    case, start = s["case"], s["node_start"].long()
    count, context = start[1:] - start[:-1], s["context_len"].long()
    dev, page, heads, dim = start.device, case["page"], case["heads"], case["dim"]
    batch, most, group = case["batch"], case["nodes"], case["q_heads"] // heads
    longest = s["block_table"].shape[1] * page
    at = torch.arange(longest, device=dev)
    held = at < (context + count)[:, None]                       # (batch, longest)
    pages = torch.where(held, s["block_table"].long()[:, at // page], 0)
    k, v = (s[n][pages, at % page] if s[n + "_scale"] is None else
            _dequantise(s[n].view(torch.uint8)[pages, at % page].view(torch.float8_e4m3fn),
                        s[n + "_scale"][pages, at % page]) for n in ("k", "v"))
    k = k.float().permute(0, 2, 3, 1)                            # (batch, heads, dim, longest)
    v = torch.where(held[:, :, None, None], v.float(), 0.0).permute(0, 2, 1, 3)
    node = torch.arange(most, device=dev)
    real = node < count[:, None]                                 # (batch, most)
    row = torch.where(real, start[:-1, None] + node, 0)
    q = s["q"][row].float().view(batch, most, heads, group, dim).permute(0, 2, 1, 3, 4)
    scores = q.reshape(batch, heads, most * group, dim) @ k * dim ** -0.5
    other = at - context[:, None]                                # node index of each key, or < 0
    if s["tree_mask"] is None:
        inside = other[:, None, :] <= node[:, None]
    else:
        words = s["tree_mask"][row].gather(
            2, (other.clamp(0, most - 1) // 64)[:, None].expand(-1, most, -1))
        inside = ((words >> (other.clamp(min=0) % 64)[:, None]) & 1).bool()
    sees = held[:, None] & ((other < 0)[:, None] | inside)       # (batch, most, longest)
    sees = sees[:, None, :, None].expand(-1, -1, -1, group, -1).reshape(batch, 1, most * group, -1)
    scores = scores.masked_fill_(~sees, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = torch.exp(scores - torch.where(top > -math.inf, top, 0.0))
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, (p @ v) / total, 0.0)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)
    each = torch.arange(s["q"].shape[0], device=dev)
    request = torch.searchsorted(start, each, right=True) - 1
    unpack = lambda x: x.view(batch, heads, most, group, -1)[  # noqa: E731
        request, :, each - start[request]].flatten(1, 2)
    return {"out": unpack(out).to(torch.bfloat16), "lse": unpack(lse)[..., 0]}


def _plain_verify(s):
    start, parent, tokens = s["node_start"].long(), s["parent"].long(), s["tokens"]
    batch, depth, n = s["case"]["batch"], s["case"]["depth"], parent.shape[0]
    dev = parent.device
    here, widest = torch.arange(n, device=dev), s["widest"]
    first = start[torch.searchsorted(start, here, right=True) - 1]
    above = torch.where(parent >= 0, first + parent, n)
    # child[i, r]: node i's r-th child in index order, or -1 (row n: the roots)
    rank = ((above[:, None] == above[None, :]) & (here[None, :] < here[:, None])).sum(-1)
    child = torch.full((n + 1, widest), -1, dtype=torch.long, device=dev)
    child[above, torch.where(parent >= 0, rank, 0)] = here
    heat = s["temperature"][:, None]

    def softmax(logits):
        z = logits.float() / torch.where(heat > 0, heat, 1.0)
        z = torch.exp(z - z.amax(-1, keepdim=True))
        return z / z.sum(-1, keepdim=True)

    def target_at(at):
        top = s["target"][at].float()
        best = torch.zeros_like(top).scatter_(1, top.argmax(-1, keepdim=True), 1.0)
        return torch.where(heat > 0, softmax(top), best)

    at, count = start[:-1].clone(), torch.zeros(batch, dtype=torch.int32, device=dev)
    path = torch.full((batch, depth), -1, dtype=torch.int32, device=dev)
    out = torch.full((batch, depth + 1), -1, dtype=torch.long, device=dev)
    going = torch.ones(batch, dtype=torch.bool, device=dev)
    left = torch.zeros((batch, s["target"].shape[1]), device=dev)   # what the last token is drawn from
    for step in range(depth + 1):
        p = target_at(at)
        q = softmax(s["draft"][at]) if s["draft"] is not None else None
        rest, mass, taken = p.clone(), torch.ones(batch, device=dev), torch.zeros(batch, device=dev)
        moved = torch.zeros(batch, dtype=torch.bool, device=dev)
        nxt = at.clone()
        for r in range(widest if step < depth else 0):
            c = child[at, r]
            asked = going & ~moved & (c >= 0)
            x = tokens[c.clamp(min=0)][:, None]
            u, rx = s["uniform"][c.clamp(min=0)], rest.gather(1, x)[:, 0]
            qx = q.gather(1, x)[:, 0] if q is not None else 1.0
            yes = asked & (u * mass * qx < rx)
            nxt, moved = torch.where(yes, c, nxt), moved | yes
            no = asked & ~yes
            if q is not None:
                taken = torch.where(no, taken + mass, taken)
                rest = torch.where(no[:, None], (p - taken[:, None] * q).clamp_(min=0), rest)
            else:
                rest = torch.where(no[:, None], rest.scatter(1, x, 0.0), rest)
            mass = torch.where(no, rest.sum(-1), mass)
        ends = going & ~moved
        left = torch.where(ends[:, None], torch.where((rest > 0).any(-1, keepdim=True), rest, p), left)
        if step < depth:
            path[:, step] = torch.where(moved, (nxt - start[:-1]).int(), -1)
            out[:, step] = torch.where(moved, tokens[nxt], -1)
        count += moved.int()
        at, going = nxt, moved
    race = torch.where(left > 0, left / s["noise"], -1.0)
    out.scatter_(1, count.long()[:, None], race.argmax(-1, keepdim=True))
    return {"tokens": out, "path": path, "count": count}


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"write": _plain_write, "move": _plain_move, "attend": _plain_attend,
                "verify": _plain_verify}[op](state)
    from distillation_ce_tvd_gb300 import binding
    if op == "write":
        binding.fct_kv_cache_write(state["cache"], state["new_k"], state["new_v"], state["slots"])
        return _pool(state)
    if op == "move":
        binding.fct_kv_cache_move(state["cache"], state["block_table"], state["context_len"],
                                  state["path"], state["count"])
        return _pool(state)
    if op == "attend":
        out, lse = binding.fct_tree_attention(state["q"], state["cache"], state["block_table"],
                                              state["context_len"], state["node_start"],
                                              state["tree_mask"], workspace=state["workspace"])
        return {"out": out, "lse": lse}
    tokens, path, count = binding.fct_spec_verify(
        state["target"], state["tokens"], state["parent"], state["node_start"], state["uniform"],
        state["noise"], state["draft"], state["temperature"], max_depth=state["case"]["depth"])
    return {"tokens": tokens, "path": path, "count": count}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    per = case.get("heads", 0) * case.get("dim", 0)
    held = 2 * per * (2 if case.get("cache") == "bf16" else 1)   # a token's key and value, bytes
    if case.get("cache") == "e4m3":
        held += 2 * case["heads"]
    if case["op"] == "write":
        source = 2 * per * (4 if case["source"] == "f32" else 2)
        return {"bytes": case["tokens"] * (source + held + 8), "flops": 2 * 2 * per * case["tokens"]}
    if case["op"] == "move":
        # a path goes on with probability 0.8 as far as the tree does: about 2.5 nodes
        moved = case["batch"] * min(2.5, case["depth"])
        return {"bytes": 2 * moved * held + case["batch"] * (case["depth"] * 4 + 8), "flops": 0}
    if case["op"] == "attend":
        batch, nodes = case["batch"], case["nodes"]
        mean = 1.0 if case["tree"] == "chain" else 0.75
        nodes = nodes if batch == 1 else max(1.0, nodes * (mean + (1 - mean) / batch))
        low = min(case["context_min"], case["context"])
        keys = (case["context"] + (batch - 1) * (case["context"] + low) / 2) + batch * nodes
        rows = nodes * case["q_heads"]
        io = batch * rows * (2 * 2 * case["dim"] + 4)
        return {"bytes": keys * held + io, "flops": 4 * rows * keys * case["dim"]}
    # verification: the rows of the visited nodes (target, and draft where there are children), and
    # one row of noise; a drafted token is accepted with probability 0.8, a tree's node goes on with
    # the sum of its children's shares
    size = 4 if case["type"] == "f32" else 2
    go = 0.8 if case["draft"] else 0.6
    visited = sum(go ** i for i in range(case["depth"] + 1))
    rows = visited + (visited - go ** case["depth"] if case["draft"] else 0)
    return {"bytes": case["batch"] * case["vocab"] * (rows * size + 4),
            "flops": case["batch"] * case["vocab"] * rows * 4}


# ---------------------------------------------------------------- 64 bits


def _wide(s, name):
    """A pool's values in 64 bits."""
    if s[name + "_scale"] is None:
        return s[name].double()
    return s[name].double() * torch.exp2(s[name + "_scale"].double() - 127)[..., None]


def _exact_write(s):
    got = {}
    page = s["case"]["page"]
    for name in ("k", "v"):
        x = s["new_" + name].double()
        pool = s[name].double().flatten(0, 1)
        if s["case"]["cache"] == "e4m3":
            amax = x.abs().amax(-1, keepdim=True)
            power = torch.ceil(torch.log2(amax / E4M3_MAX))
            power += (amax > E4M3_MAX * torch.exp2(power)).double()
            power -= (amax <= E4M3_MAX * torch.exp2(power - 1)).double()
            y = x / torch.exp2(power.clamp(min=-126))
            fine = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            y = torch.round(y / fine) * fine
            scale = s[name + "_scale"].clone().flatten(0, 1)
            scale[s["slots"]] = (power.clamp(min=-126)[..., 0] + 127).to(torch.uint8)
            got[name + "_scale"] = scale.view(-1, page, scale.shape[-1])
        else:
            y = x.to(torch.bfloat16).double()
            got[name + "_scale"] = None
        pool[s["slots"]] = y
        got[name] = pool.view(s[name].shape)
    return got


def _exact_move(s):
    got = {n: None if x is None else (x.clone() if x.dtype == torch.uint8 else x.double())
           for n, x in _pool(s).items()}
    page = s["case"]["page"]
    table, path, context = s["block_table"].tolist(), s["path"].tolist(), s["context_len"].tolist()
    for b, count in enumerate(s["count"].tolist()):
        slot = lambda i: (table[b][i // page], i % page)  # noqa: B023, E731
        for j in range(count):
            to, at = slot(context[b] + 1 + j), slot(context[b] + path[b][j])
            for x in got.values():
                if x is not None:
                    x[to] = x[at]
    return got


def _exact_attend(s):
    case, start, context = s["case"], s["node_start"].tolist(), s["context_len"].tolist()
    heads, dim, group = case["heads"], case["dim"], case["q_heads"] // case["heads"]
    outs, lses = [], []
    for b in range(case["batch"]):
        n, c = start[b + 1] - start[b], context[b]
        used = s["block_table"][b, :-(-(c + n) // case["page"])].long()
        part = {x: None if s[x] is None else s[x].view(torch.uint8)[used].view(s[x].dtype)
                for x in ("k", "v", "k_scale", "v_scale")}
        k, v = (_wide(part, x).flatten(0, 1)[:c + n] for x in ("k", "v"))
        sees = torch.zeros((n, c + n), dtype=torch.bool)
        sees[:, :c] = True
        rows = None if s["tree_mask"] is None else s["tree_mask"][start[b]:start[b + 1]].tolist()
        for i in range(n):
            for j in range(n):
                bit = j <= i if rows is None else (rows[i][j // 64] >> (j % 64)) & 1
                sees[i, c + j] = bool(bit)
        sees = sees.to(k.device)
        q = s["q"][start[b]:start[b + 1]].double()
        for h in range(case["q_heads"]):
            z = q[:, h] @ k[:, h // group].T / math.sqrt(dim)
            z[~sees] = -math.inf
            lse = torch.logsumexp(z, -1)
            w = torch.exp(z - torch.where(lse > -math.inf, lse, 0.0)[:, None])
            outs.append(w @ v[:, h // group])
            lses.append(lse)
    split = lambda xs: torch.cat([torch.stack(xs[b * case["q_heads"]:(b + 1) * case["q_heads"]], 1)  # noqa: E731
                                  for b in range(case["batch"])])
    return {"out": split(outs), "lse": split(lses)}


def _exact_verify(s):
    case, start = s["case"], s["node_start"].tolist()
    parent, tokens, uniform = s["parent"].tolist(), s["tokens"].tolist(), s["uniform"].tolist()
    heat, depth = s["temperature"].double().tolist(), case["depth"]
    got = {"tokens": [], "path": [], "count": []}
    for b in range(case["batch"]):
        at, walk = start[b], []
        while True:
            z = s["target"][at].double()
            if heat[b] > 0:
                p = torch.softmax(z / heat[b], -1)
            else:
                p = torch.zeros_like(z)
                p[z.argmax()] = 1.0
            q = None
            if s["draft"] is not None:
                q = torch.softmax(s["draft"][at].double() / (heat[b] or 1.0), -1)
            rest, nxt = p, None
            for c in range(at + 1, start[b + 1]):
                if start[b] + parent[c] != at or len(walk) == depth:
                    continue
                x, total = tokens[c], float(rest.sum())
                if uniform[c] * total * (1.0 if q is None else float(q[x])) < float(rest[x]):
                    nxt = c
                    break
                if q is None:
                    rest = rest.clone()
                    rest[x] = 0.0
                else:
                    rest = (rest - total * q).clamp(min=0)
            if nxt is None:
                break
            at = nxt
            walk.append(at)
        rest = rest if float(rest.max()) > 0 else p
        last = int((rest / s["noise"][b].double()).argmax())
        pad = [-1] * (depth - len(walk))
        got["tokens"].append([tokens[c] for c in walk] + [last] + pad)
        got["path"].append([c - start[b] for c in walk] + pad)
        got["count"].append(len(walk))
    return {n: torch.tensor(x) for n, x in got.items()}


def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _exact_write, "move": _exact_move, "attend": _exact_attend,
            "verify": _exact_verify}[case["op"]](s)
