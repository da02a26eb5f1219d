"""Decoding with trees of drafted tokens, measured: attention of a tree's nodes
over the paged 4-bit cache, the KDA recurrence over a tree, verification of the
drafted tokens against the target's probabilities, and what follows from the
accepted path: its cache entries move together, its tokens enter the states.

A request's tree has up to 64 nodes in topological order: node 0 is the last
token that is certain, node i > 0 follows node parents[i] < i.  Node i is cached
behind the context, at position cache_lens + i.

`run` computes each operator in elementary torch operations, or, where `own`
is true, through the framework's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E_MIN, E_MAX = 2, 252  # exponent bytes in use: every value is a normal bf16
EPS = 1e-6  # of the norms of q and k


def _attend(name, dtype, n_seq, nodes, fan, context, q_heads, kv_heads, dim, page, ragged):
    return {"name": name, "op": "attend", "dtype": dtype, "n_seq": n_seq, "nodes": nodes, "fan": fan, "context": context,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "ragged": ragged}


def _states(name, op, dtype, n_seq, nodes, fan, heads, ragged):
    return {"name": name, "op": op, "dtype": dtype, "n_seq": n_seq, "nodes": nodes, "fan": fan, "heads": heads,
            "ragged": ragged}


def _keep(name, dtype, n_seq, nodes, kept, context, kv_heads, dim, page):
    return {"name": name, "op": "keep", "dtype": dtype, "n_seq": n_seq, "nodes": nodes, "kept": kept, "context": context,
            "kv_heads": kv_heads, "dim": dim, "page": page, "ragged": True}


def _verify(name, dtype, n_seq, nodes, fan, vocab, draft, ragged):
    return {"name": name, "op": "verify", "dtype": dtype, "n_seq": n_seq, "nodes": nodes, "fan": fan, "vocab": vocab,
            "draft": draft, "ragged": ragged}


def listed():
    return [
        # one request's small tree: latency
        _attend("attend_one", "bf16", 1, 8, 2, 1000, 32, 8, 128, 128, False),
        # a decode step of 16 requests of mixed age, trees of up to 32 nodes
        _attend("attend_step", "bf16", 16, 32, 2, 8191, 32, 8, 128, 128, True),
        # large trees over long contexts, small heads
        _attend("attend_long", "f16", 2, 64, 3, 60000, 16, 2, 64, 32, True),
        # one request's tree through one layer's states: latency
        _states("tree_one", "tree", "f32", 1, 13, 2, 12, False),
        # a decode step's trees
        _states("tree_step", "tree", "f16", 64, 48, 3, 12, True),
        # the accepted tokens of one request enter its states
        _states("path_one", "path", "f32", 1, 13, 2, 12, False),
        # and those of a batch: chains of 1 + 7, up to 8 accepted
        _states("path_step", "path", "f16", 64, 8, 1, 12, True),
        # accepted tokens' cache entries move together
        _keep("keep_one", "bf16", 1, 16, 4, 300, 8, 128, 128),
        _keep("keep_many", "bf16", 128, 48, 8, 200, 12, 128, 16),
        # one request's chain of 1 + 7 with the draft's probabilities: latency
        _verify("verify_one", "f32", 1, 8, 1, 32768, True, False),
        # a batch of such chains, a vocabulary of odd size
        _verify("verify_chains", "f32", 64, 8, 1, 100003, True, False),
        # trees of the draft's likeliest tokens, no probabilities of the draft
        _verify("verify_trees", "bf16", 32, 64, 3, 131072, False, True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["attend", "attend", "tree", "path", "keep", "verify"])
    fan, ragged = rng.choice([1, 2, 2, 3]), rng.random() < 0.6
    if op == "attend":
        kv_heads, group = rng.choice([1, 2, 3, 4, 8, 12]), rng.choice([1, 2, 4, 5, 8])
        n_seq = _log(rng, 1, 48)
        nodes = _log(rng, 1, 64)
        c = _attend("", rng.choice(["f32", "f16", "bf16"]), n_seq, nodes, fan,
                    min(_log(rng, 1, 60000), 130000 // n_seq, 30_000_000 // (n_seq * nodes * kv_heads * group)),
                    kv_heads * group, kv_heads, rng.choice([64, 128]), rng.choice([16, 32, 64, 128, 256]), ragged)
    elif op in ("tree", "path"):
        n_seq = _log(rng, 1, 64)
        c = _states("", op, rng.choice(["f32", "f16"]), n_seq, min(_log(rng, 1, 64), 1536 // n_seq), fan,
                    rng.choice([1, 3, 8, 12]), ragged)
    elif op == "keep":
        kept = rng.randint(1, 12)
        c = _keep("", rng.choice(["f32", "f16", "bf16"]), _log(rng, 1, 128), rng.randint(2 * kept, 64), kept,
                  _log(rng, 1, 400) - 1, rng.choice([1, 2, 3, 8, 12]), rng.choice([64, 128]),
                  rng.choice([16, 32, 64, 128, 256]))
    else:
        n_seq, vocab = _log(rng, 1, 64), _log(rng, 100, 160000)
        draft = rng.random() < 0.5
        nodes = min(_log(rng, 1, 12 if draft else 64), 100_000_000 // (n_seq * vocab))
        c = _verify("", rng.choice(["f32", "f16", "bf16"]), n_seq, max(nodes, 1), fan, vocab, draft, ragged)
    del c["name"]
    return c


def _spread(most, n, ragged, least):
    """n lengths up to `most`: all equal, or evenly spread and out of order."""
    if not ragged:
        return [most] * n
    step = next(s for s in (7, 11, 13, 17, 1) if math.gcd(s, n) == 1)
    return [max(least, most * ((i * step) % n + 1) // n) for i in range(n)]


def _tree(case, s, n):
    """Parents of request s's n nodes: a chain (fan 1), or `fan` to `fan` + 1 children a node, level by level."""
    rng, fan = random.Random(1009 * s + n), case["fan"]
    return [-1] + [i - 1 if fan == 1 else rng.randint((i - 1) // (fan + 1), (i - 1) // fan) for i in range(1, n)]


def _trees(case):
    return [_tree(case, s, n) for s, n in enumerate(_spread(case["nodes"], case["n_seq"], case["ragged"], 1))]


def _depths(parents):
    depth = []
    for p in parents:
        depth.append(0 if p < 0 else depth[p] + 1)
    return depth


def _path_to(parents, node):
    path = []
    while node >= 0:
        path.append(node)
        node = parents[node]
    return path[::-1]


def _paths(case):
    """The accepted nodes of each request."""
    counts = _spread(case["nodes"], case["n_seq"], case["ragged"], 1)
    paths = []
    for s, n in enumerate(counts):
        rng = random.Random(31 * s + 7 * n)
        if case["op"] == "keep":
            # in wide trees an accepted node lies behind all that are moved in front of it
            m = max(1, min(1 + (s * 5) % case["kept"] if case["n_seq"] > 1 else case["kept"], (n + 1) // 2))
            paths.append([0] + sorted(rng.sample(range(m, n), m - 1)))
        else:
            paths.append(_path_to(_tree(case, s, n), rng.randrange(n)))
    return paths


def work(case):
    op = case["op"]
    if op in ("attend", "keep"):
        stored = case["kv_heads"] * case["dim"] * 17 // 16  # bytes of one token's keys and values
        size = 4 if case["dtype"] == "f32" else 2
    if op == "attend":
        trees, past = _trees(case), _spread(case["context"], case["n_seq"], case["ragged"], 0)
        nodes = sum(map(len, trees))
        pairs = sum(len(t) * p + sum(_depths(t)) + len(t) for t, p in zip(trees, past))
        return {"bytes": (nodes + sum(past)) * stored + 2 * size * nodes * case["q_heads"] * case["dim"] + 4 * nodes,
                "flops": 4 * case["dim"] * case["q_heads"] * pairs}
    if op == "keep":  # the tokens that move in and out, those kept read back as values
        lens = [len(p) for p in _paths(case)]
        return {"bytes": sum(n - 1 for n in lens) * 2 * stored + sum(lens) * (stored + 2 * size * case["kv_heads"] * case["dim"]),
                "flops": sum(lens) * case["kv_heads"] * case["dim"] * 2}
    if op == "verify":  # each request's last row (with the draft's) whole; probabilities of the drafted tokens
        trees = _trees(case)
        size, nodes = 4 if case["dtype"] == "f32" else 2, sum(map(len, trees))
        rows = 2 if case["draft"] else 1
        return {"bytes": len(trees) * rows * case["vocab"] * size + nodes * (rows * size + 12) + len(trees) * 12,
                "flops": len(trees) * case["vocab"] * 2 * rows}
    state = case["heads"] * 128 * 128 * (4 if case["dtype"] == "f32" else 2)
    if op == "tree":
        trees = _trees(case)
        nodes = sum(map(len, trees))
        pairs = sum(sum(_depths(t)) for t in trees)
        return {"bytes": len(trees) * state + nodes * case["heads"] * (5 * 128 + 1) * 4 + 4 * nodes,
                "flops": case["heads"] * (nodes * 4 * 128 * 128 + pairs * 10 * 128)}
    tokens = sum(map(len, _paths(case)))
    return {"bytes": 2 * case["n_seq"] * state + tokens * case["heads"] * (3 * 128 + 1) * 4,
            "flops": case["heads"] * tokens * 5 * 128 * 128}


# --------------------------------------------------------------------------
# the cache's format
# --------------------------------------------------------------------------

def _parts(pool):
    """A pool [pages, heads, P, 17 D / 16] of bytes as its key codes, value codes, key and value exponents (views)."""
    pages, heads, P, width = pool.shape
    D = width * 16 // 17
    flat = pool.view(pages, heads, P * width)
    a, b, c = P * D // 2, P * D, P * D + P * D // 32
    return (flat[..., :a].unflatten(-1, (P, D // 2)), flat[..., a:b].unflatten(-1, (P, D // 2)),
            flat[..., b:c].unflatten(-1, (P, D // 32)), flat[..., c:].unflatten(-1, (D // 32, P)))


def _values(codes, exps):
    """fp32 values of codes [..., D / 2] with exponents [..., D / 32]."""
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=codes.device)
    table = torch.cat([table, -table])
    x = torch.stack([table[(codes & 15).long()], table[(codes >> 4).long()]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, 32)) * torch.exp2(exps.float() - 127).unsqueeze(-1)).flatten(-2)


def _random_codes(shape, D, gen, dev, wide):
    """Codes and exponents of numbers like a normal's: all codes, exponents around one."""
    codes = torch.randint(0, 256, (*shape, D // 2), generator=gen, device=dev, dtype=torch.uint8)
    exps = 125 + torch.randint(0, 2, (*shape, D // 32), generator=gen, device=dev, dtype=torch.uint8)
    if wide:  # a few strong channels
        exps += 2 * (torch.rand((shape[1], 1, D // 32), generator=gen, device=dev) < 0.1).byte()
    return codes, exps


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    n = case["n_seq"]
    state = {"op": case["op"]}

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=dev)

    def fresh(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    trees = _trees(case) if case["op"] != "keep" else [
        [-1] * c for c in _spread(case["nodes"], n, case["ragged"], 1)]
    counts = [len(t) for t in trees]
    T, most = sum(counts), max(counts)
    state["cu"] = ints([0] + counts).cumsum(0).to(torch.int32)
    state["parents"] = ints([p for t in trees for p in t])
    state["rows"] = most
    # each node's request and its index there, as a program that lays out a batch has them
    state["seq"] = torch.repeat_interleave(torch.arange(n, device=dev), ints(counts).long())
    state["index"] = torch.arange(T, device=dev) - state["cu"].long()[state["seq"]]
    if case["op"] in ("path", "keep"):
        paths = _paths(case)
        lens = [len(p) for p in paths]
        wide = max(lens)
        state["path"] = ints([p + [-1] * (wide - len(p)) for p in paths])
        state["lens"], state["longest"] = ints(lens), wide
    if case["op"] in ("attend", "keep"):
        heads, D, P = case["kv_heads"], case["dim"], case["page"]
        past = _spread(case["context"], n, case["ragged"], 0)
        need = [-(-(a + b) // P) for a, b in zip(counts, past)]
        pages = sum(need) + 3
        # pages are handed out in no order; entries behind a sequence's end name no page
        order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
        table = torch.full((n, max(need) + 2), -1, dtype=torch.int32, device=dev)
        table[torch.arange(table.shape[1], device=dev).unsqueeze(0) < ints(need).unsqueeze(1)] = order[:sum(need)]
        pool = torch.empty((pages, heads, P, D * 17 // 16), dtype=torch.uint8, device=dev)
        kc, vc, ke, ve = _parts(pool)
        for at in range(0, pages, 512):
            some = min(512, pages - at)
            kc[at:at + some], ke[at:at + some] = _random_codes((some, heads, P), D, gen, dev, True)
            vc[at:at + some], e = _random_codes((some, heads, P), D, gen, dev, False)
            ve[at:at + some] = e.transpose(-1, -2)
        state.update(pool=pool, table=table, past=ints(past), most=max(a + b for a, b in zip(counts, past)))
        dtype = DTYPES[case["dtype"]]
        if case["op"] == "attend":
            state["q"] = fresh(T, case["q_heads"], D).mul_(0.4).to(dtype)
            state["out"] = torch.empty_like(state["q"])
        else:
            state["cu_kept"] = ints([0] + lens).cumsum(0).to(torch.int32)
            state["kept_seq"] = torch.repeat_interleave(torch.arange(n, device=dev), state["lens"].long())
            state["kept_at"] = torch.arange(sum(lens), device=dev) - state["cu_kept"].long()[state["kept_seq"]]
            state["k_out"] = torch.empty((sum(lens), heads, D), dtype=dtype, device=dev)
            state["v_out"] = torch.empty_like(state["k_out"])
        return state
    if case["op"] in ("tree", "path"):
        H, slots = case["heads"], 2 * n + 2
        pool = torch.empty((slots, H, 128, 128), dtype=DTYPES[case["dtype"]], device=dev)
        for at in range(0, slots, 16):
            pool[at:at + 16] = fresh(min(16, slots - at), H, 128, 128) * 0.05
        ids = torch.randperm(slots, generator=gen, device=dev).to(torch.int32)
        state.update(pool=pool, init=ids[:n].contiguous())
        state["q"], state["k"], state["v"] = fresh(T, H, 128), fresh(T, H, 128), fresh(T, H, 128)
        state["g"] = -torch.nn.functional.softplus(fresh(T, H, 128))
        state["b"] = fresh(T, H)
        if case["op"] == "tree":
            state["out"] = torch.empty_like(state["v"])
            depths = [_depths(t) for t in trees]
            # the levels of all trees: node indices, and their parents' (-1: none)
            first = state["cu"].tolist()
            flat = [(d, first[s] + i, first[s] + p if p >= 0 else -1)
                    for s, t in enumerate(trees) for i, (d, p) in enumerate(zip(depths[s], t))]
            state["levels"] = [(ints([x[1] for x in flat if x[0] == d]).long(), ints([x[2] for x in flat if x[0] == d]).long())
                               for d in range(1 + max(x[0] for x in flat))]
        else:
            # every destination differs from its source: a pass can be repeated
            state["dst"] = ids[n:2 * n].contiguous()
        return state
    # verify: the draft's logits are the target's with noise; rows of both as softmax leaves them
    V, dtype = case["vocab"], DTYPES[case["dtype"]]
    target = torch.empty((T, V), dtype=dtype, device=dev)
    draft = torch.empty_like(target) if case["draft"] else None
    ranks, seen = [], {}
    for s, t in enumerate(trees):
        for i, p in enumerate(t):
            ranks.append(seen.get((s, p), 0))
            seen[s, p] = ranks[-1] + 1
    k = min(max(ranks) + 1, V)
    picks = torch.empty((T, k), dtype=torch.int64, device=dev)
    for at in range(0, T, 256):
        rows = slice(at, min(at + 256, T))
        logits = fresh(rows.stop - at, V) * 2.5
        target[rows] = torch.softmax(logits, -1)
        logits += fresh(rows.stop - at, V) * 0.5
        if case["draft"]:
            draft[rows] = torch.softmax(logits, -1)
            picks[rows] = torch.multinomial(draft[rows].float(), k, replacement=True, generator=gen)
        else:
            picks[rows] = torch.topk(logits, k, -1).indices
    above = (state["cu"].long()[state["seq"]] + state["parents"].clamp(min=0)).long()
    tokens = picks[above, torch.tensor(ranks, device=dev).clamp(max=k - 1)].to(torch.int32)
    state.update(target=target, draft=draft, tokens=tokens, accept=torch.rand(T, generator=gen, device=dev),
                 sample=torch.rand(n, generator=gen, device=dev))
    state["path"] = torch.empty((n, most), dtype=torch.int32, device=dev)
    state["lens"] = torch.empty(n, dtype=torch.int32, device=dev)
    state["next"] = torch.empty(n, dtype=torch.int32, device=dev)
    return state


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _plain_attend(s):
    """Sequences padded to the longest, in one batch."""
    pool, q, table = s["pool"], s["q"], s["table"]
    heads, P, D = pool.shape[1], pool.shape[2], pool.shape[3] * 16 // 17
    n, group, rows = table.shape[0], q.shape[1] // heads, s["rows"]
    # which nodes each node descends from: the paths of one step, doubled until no path is longer
    above = torch.eye(rows, device=q.device).repeat(n, 1, 1)
    has = s["parents"] >= 0
    above[s["seq"][has], s["index"][has], s["parents"][has].long()] = 1
    for _ in range(max(1, (rows - 1).bit_length())):
        above = (above @ above).clamp(max=1)
    pages = table[:, :-(-s["most"] // P)].long().clamp(min=0)
    L = pages.shape[1] * P
    kc, vc, ke, ve = _parts(pool)
    keys = _values(kc[pages], ke[pages]).transpose(1, 2).reshape(n, heads, L, D)
    x = q.new_zeros((n, rows, heads, group, D), dtype=torch.float32)
    x[s["seq"], s["index"]] = q.float().unflatten(1, (heads, group))
    x = x.permute(0, 2, 1, 3, 4).reshape(n, heads, rows * group, D)
    scores = torch.matmul(x, keys.transpose(-1, -2).contiguous()) * (1 / math.sqrt(D))
    del keys
    at = torch.arange(L, device=q.device).unsqueeze(0) - s["past"].unsqueeze(1)  # [n, L]
    seen = torch.gather(above, 2, at.clamp(0, rows - 1).unsqueeze(1).expand(-1, rows, -1)) > 0
    seen = torch.where((at < 0).unsqueeze(1), True, seen & (at < rows).unsqueeze(1))
    scores = scores.view(n, heads, rows, group, L).masked_fill_(~seen[:, None, :, None], -math.inf)
    weights = torch.exp(scores - scores.amax(-1, keepdim=True))
    del scores
    total = weights.sum(-1, keepdim=True)
    values = _values(vc[pages], ve[pages].transpose(-1, -2)).transpose(1, 2).reshape(n, heads, L, D)
    o = torch.matmul(weights.view(n, heads, rows * group, L), values).view(n, heads, rows, group, D) / total
    s["out"].copy_(o.permute(0, 2, 1, 3, 4)[s["seq"], s["index"]].flatten(1, 2))
    return s["out"]


def _unit(x):
    return x / torch.sqrt((x * x).sum(-1, keepdim=True) + EPS)


def _advance(S, k, v, g, b):
    """One token's update of states S [.., 128, 128]; k of length 1."""
    S = S * torch.exp(g).unsqueeze(-1)
    u = v - torch.matmul(k.unsqueeze(-2), S).squeeze(-2)
    return S + (torch.sigmoid(b).unsqueeze(-1) * k).unsqueeze(-1) * u.unsqueeze(-2)


def _plain_tree(s):
    """Level by level; a node starts from its parent's state."""
    states = torch.empty((s["q"].shape[0], *s["pool"].shape[1:]), device=s["q"].device)
    q, k = _unit(s["q"]) * (1 / math.sqrt(128)), _unit(s["k"])
    for depth, (nodes, above) in enumerate(s["levels"]):
        start = s["pool"][s["init"].long()[s["seq"][nodes]]].float() if depth == 0 else states[above]
        new = _advance(start, k[nodes], s["v"][nodes], s["g"][nodes], s["b"][nodes])
        states[nodes] = new
        s["out"][nodes] = torch.matmul(q[nodes].unsqueeze(-2), new).squeeze(-2)
    return s["out"]


def _plain_path(s):
    S = s["pool"][s["init"].long()].float()
    k = _unit(s["k"])
    for e in range(s["longest"]):
        at = s["cu"][:-1].long() + s["path"][:, e].clamp(min=0).long()
        new = _advance(S, k[at], s["v"][at], s["g"][at], s["b"][at])
        S = torch.where((e < s["lens"]).view(-1, 1, 1, 1), new, S)
    s["pool"][s["dst"].long()] = S.to(s["pool"].dtype)
    return s["pool"][s["dst"].long()]


def _plain_keep(s):
    kc, vc, ke, ve = _parts(s["pool"])
    P, seq, at = s["pool"].shape[2], s["kept_seq"], s["kept_at"]
    past = s["past"].long()[seq]
    a, b = past + s["path"].long()[seq, at], past + at
    pa, pb, ra, rb = s["table"].long()[seq, a // P], s["table"].long()[seq, b // P], a % P, b % P
    kc[pb, :, rb], ke[pb, :, rb] = kc[pa, :, ra], ke[pa, :, ra]
    vc[pb, :, rb], ve[pb, :, :, rb] = vc[pa, :, ra], ve[pa, :, :, ra]
    s["k_out"].copy_(_values(kc[pb, :, rb], ke[pb, :, rb]))
    s["v_out"].copy_(_values(vc[pb, :, rb], ve[pb, :, :, rb]))
    return s["k_out"], s["v_out"]


def _plain_verify(s):
    """Nodes in their order, all requests at once: a node is tried if its parent is the last accepted one.  In 64 bits."""
    cu, target, draft = s["cu"].long(), s["target"], s["draft"]
    n, rows = s["lens"].shape[0], s["rows"]
    at = torch.zeros_like(s["lens"])  # the last accepted node
    length = torch.ones_like(s["lens"])
    s["path"].fill_(-1)
    s["path"][:, 0] = 0
    left = target[cu[:-1]].double()  # what is left of the last node's row
    mass = left.new_ones(n)
    every = torch.arange(n, device=cu.device)
    for i in range(1, rows):
        node = torch.minimum(cu[:-1] + i, cu[1:] - 1)
        tried = (cu[:-1] + i < cu[1:]) & (s["parents"][node] == at)
        x = s["tokens"][node].long()
        have = left[every, x]
        row = cu[:-1] + at
        need = s["accept"][node].double() * (draft[row, x].double() if draft is not None else 1.0) * mass
        yes, no = tried & (need < have), tried & (need >= have)
        if draft is not None:
            rest = (left - mass.unsqueeze(1) * draft[row].double()).clamp(min=0)
        else:
            rest = left.clone()
            rest[every, x] = 0
        rest = torch.where(no.unsqueeze(1), rest, left)
        mass = torch.where(no, rest.sum(1) if draft is not None else mass - have, mass)
        at = torch.where(yes, i, at)
        s["path"][every, torch.where(yes, length, 0)] = torch.where(yes, i, s["path"][:, 0])
        length += yes
        left = torch.where(yes.unsqueeze(1), target[node].double(), rest)
        mass = torch.where(yes, 1.0, mass)
    left = torch.where((left.sum(1) > 0).unsqueeze(1), left, target[cu[:-1] + at].double())
    sums = left.cumsum(1)
    hit = (sums > (s["sample"].double() * sums[:, -1]).unsqueeze(1)) & (left > 0)
    s["next"].copy_(hit.float().argmax(1))
    s["lens"].copy_(length)
    return s["path"], s["lens"], s["next"]


def run(state):
    s = state
    if not own:
        return {"attend": _plain_attend, "tree": _plain_tree, "path": _plain_path, "keep": _plain_keep,
                "verify": _plain_verify}[s["op"]](s)
    from kda_gated_delta_decode_amd import binding as B
    if s["op"] == "attend":
        B.kda_kv_attend_tree(s["pool"], s["table"], s["cu"], s["past"], s["parents"], s["q"], s["out"],
                             max_rows=s["rows"], max_kv_len=s["most"])
        return s["out"]
    if s["op"] == "tree":
        B.kda_decode_tree(s["pool"], s["init"], s["cu"], s["parents"], s["q"], s["k"], s["v"], s["g"], s["b"], s["out"],
                          max_nodes=s["rows"])
        return s["out"]
    if s["op"] == "path":
        B.kda_decode_path(s["pool"], s["init"], s["cu"], s["path"], s["lens"], s["k"], s["v"], s["g"], s["b"],
                          dst_slot_ids=s["dst"])
        return s["pool"][s["dst"].long()]
    if s["op"] == "keep":
        B.kda_kv_keep(s["pool"], s["table"], s["cu"], s["past"], s["path"], s["lens"])
        B.kda_kv_read(s["pool"], s["table"], s["cu_kept"], s["past"], s["k_out"], s["v_out"])
        return s["k_out"], s["v_out"]
    B.kda_verify_drafts(s["target"], s["cu"], s["parents"], s["tokens"], s["accept"], s["sample"], s["path"], s["lens"],
                        s["next"], draft=s["draft"])
    return s["path"], s["lens"], s["next"]


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------

def _exact_cached(pool, pages, at, which):
    """Keys (0) or values (1) of the tokens at places `at` of one sequence with page ids `pages`: fp64 [heads, n, D]."""
    _, heads, P, width = pool.shape
    D = width * 16 // 17
    block = pool.reshape(pool.shape[0], heads, P * width)[pages.long()[at // P]]
    c, r = torch.arange(D, device=pool.device), (at % P).view(-1, 1, 1)
    code = torch.gather(block, 2, ((which * P + r) * (D // 2) + c // 2).expand(-1, heads, -1)).int()
    code = (code >> (4 * (c % 2))) & 15
    e = P * D + (r * (D // 32) + c // 32 if which == 0 else P * D // 32 + (c // 32) * P + r)
    e = torch.gather(block, 2, e.expand(-1, heads, -1)).double()
    m, x = code & 1, (code >> 1) & 3  # mantissa and exponent of E2M1
    mag = torch.where(x > 0, (1 + 0.5 * m) * torch.exp2(x.double() - 1), 0.5 * m.double())
    return ((1 - 2 * (code >> 3)) * mag * torch.exp2(e - 127)).transpose(0, 1).contiguous()


def _exact_attend(case, s):
    q, D, past, cu = s["q"].double(), case["dim"], s["past"].tolist(), s["cu"].tolist()
    out, group = torch.empty_like(q), case["q_heads"] // case["kv_heads"]
    for i, tree in enumerate(_trees(case)):
        at = torch.arange(past[i] + len(tree), device=q.device)
        K, V = (_exact_cached(s["pool"], s["table"][i], at, w) for w in (0, 1))
        seen = torch.zeros((len(tree), len(at)), dtype=torch.bool)
        seen[:, :past[i]] = True
        for node in range(len(tree)):
            seen[node, [past[i] + j for j in _path_to(tree, node)]] = True
        seen = seen.to(q.device)
        for h in range(case["q_heads"]):
            logits = (q[cu[i]:cu[i + 1], h] / math.sqrt(D)) @ K[h // group].T
            out[cu[i]:cu[i + 1], h] = torch.softmax(logits.masked_fill(~seen, -math.inf), -1) @ V[h // group]
    return out


def _exact_step(S, k, v, g, b):
    """fp64 state [H, 128, 128] after one token, as (I - beta k k^T) diag(a) S + beta k v^T."""
    k, beta = k / (k.square().sum(-1, keepdim=True) + EPS).sqrt(), 1 / (1 + torch.exp(-b))
    M = torch.eye(128, dtype=torch.float64, device=k.device) - beta[:, None, None] * k[:, :, None] * k[:, None, :]
    return torch.bmm(M, torch.exp(g)[:, :, None] * S) + beta[:, None, None] * k[:, :, None] * v[:, None, :]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    cu = s["cu"].tolist()
    if case["op"] == "keep":
        past = s["past"].tolist()
        places = [torch.tensor([past[i] + x for x in p], device=s["pool"].device) for i, p in enumerate(_paths(case))]
        return tuple(torch.cat([_exact_cached(s["pool"], s["table"][i], at, w).transpose(0, 1)
                                for i, at in enumerate(places)]) for w in (0, 1))
    if case["op"] in ("tree", "path"):
        k, v, g, b = (s[x].double() for x in ("k", "v", "g", "b"))
        q = s["q"].double()
        q = q / (q.square().sum(-1, keepdim=True) + EPS).sqrt() / math.sqrt(128)
        outs, ends = torch.empty_like(q), []
        trees, paths = _trees(case), _paths(case) if case["op"] == "path" else None
        for r, slot in enumerate(s["init"].tolist()):
            S0 = s["pool"][slot].double()
            if case["op"] == "path":
                for node in paths[r]:
                    t = cu[r] + node
                    S0 = _exact_step(S0, k[t], v[t], g[t], b[t])
                ends.append(S0)
                continue
            states = []
            for i, p in enumerate(trees[r]):
                t = cu[r] + i
                states.append(_exact_step(S0 if p < 0 else states[p], k[t], v[t], g[t], b[t]))
                outs[t] = torch.bmm(q[t][:, None, :], states[-1])[:, 0]
        return outs if case["op"] == "tree" else torch.stack(ends)
    paths, nexts = torch.full_like(s["path"], -1), []
    for r, tree in enumerate(_trees(case)):
        way, last = [0], 0
        f, mass = s["target"][cu[r]].double(), 1.0
        for i in range(1, len(tree)):
            if tree[i] != last:
                continue
            x, t = int(s["tokens"][cu[r] + i]), float(s["accept"][cu[r] + i])
            qrow = s["draft"][cu[r] + last].double() if case["draft"] else None
            if t * mass * (float(qrow[x]) if case["draft"] else 1.0) < float(f[x]):
                way.append(i)
                last, f, mass = i, s["target"][cu[r] + i].double(), 1.0
            elif case["draft"]:
                f = torch.relu(f - mass * qrow)
                mass = float(f.sum())
            else:
                mass -= float(f[x])
                f[x] = 0
        if not float(f.sum()) > 0:
            f = s["target"][cu[r] + last].double()
        # draw: the first token at which the running sum passes the random share of the total
        sums = torch.cumsum(f, 0)
        at = int(torch.searchsorted(sums, s["sample"][r].double() * sums[-1], right=True))
        nexts.append(min(at, f.shape[0] - 1))
        paths[r, :len(way)] = torch.tensor(way, dtype=torch.int32, device=paths.device)
    return paths, (paths >= 0).sum(1).to(torch.int32), torch.tensor(nexts, dtype=torch.int32, device=paths.device)
