"""The paged 4-bit key/value cache, measured: appending with the position
rotation, reading cached tokens back, and attention over the cache.

The cache holds E2M1 values (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives)
with one power-of-two exponent byte for 32 channels.  A page of P tokens keeps,
for each head, a block of P * (D + D / 16) bytes: key codes [P][D / 2] (two
channels a byte, the even one low), value codes [P][D / 2], key exponents
[P][D / 32], value exponents [D / 32][P].

`run` computes each operator in elementary torch operations, or, where `own`
is true, through the framework's entry points.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
E_MIN, E_MAX = 2, 252  # exponent bytes in use: every value is a normal bf16


def _case(name, op, dtype, n_seq, rows, context, q_heads, kv_heads, dim, page, ragged, rot=0, interleaved=False):
    return {"name": name, "op": op, "dtype": dtype, "n_seq": n_seq, "rows": rows, "context": context,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "ragged": ragged,
            "rot": rot, "interleaved": interleaved}


def listed():
    return [
        # one decode step's new tokens of 64 requests
        _case("append_step", "append", "bf16", 64, 1, 4000, 32, 8, 128, 128, True, 128),
        # a verify step's 1 + 7 rows for 8 requests, fp32 activations, half of each head rotated
        _case("append_verify", "append", "f32", 8, 8, 500, 12, 12, 128, 16, True, 64, True),
        # a prefill batch of ragged prompts, small heads
        _case("append_prompts", "append", "f16", 32, 700, 0, 16, 2, 64, 32, True, 64),
        # one long prompt
        _case("append_long", "append", "bf16", 1, 16384, 0, 32, 8, 128, 128, False, 128),
        # a short shared prefix read back, to be moved to another cache
        _case("read_prefix", "read", "bf16", 1, 333, 0, 32, 8, 128, 128, False),
        # many sequences moved at once
        _case("read_many", "read", "f32", 24, 8192, 0, 12, 12, 128, 64, True),
        # one request, one token: latency
        _case("attend_one", "attend", "bf16", 1, 1, 1000, 32, 8, 128, 128, False),
        # one decode step of 64 requests of mixed age
        _case("attend_step", "attend", "bf16", 64, 1, 8191, 32, 8, 128, 128, True),
        # a verify step: 8 requests x (1 + 7) rows, one query head for each cached head
        _case("attend_verify", "attend", "f32", 8, 8, 4089, 12, 12, 128, 128, False),
        # one token over a very long context
        _case("attend_long", "attend", "f16", 1, 1, 131071, 64, 8, 128, 128, False),
        # a whole prompt
        _case("attend_prompt", "attend", "bf16", 1, 8192, 0, 32, 8, 128, 128, False),
        # chunks of prompts appended to cached ones, small heads
        _case("attend_chunk", "attend", "f16", 4, 700, 16000, 16, 2, 64, 32, True),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kv_heads, group = rng.choice([1, 2, 3, 4, 8, 12]), rng.choice([1, 2, 4, 5, 8])
    shape = dict(dtype=rng.choice(["f32", "f16", "bf16"]), q_heads=kv_heads * group, kv_heads=kv_heads,
                 dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64, 128, 256]), ragged=rng.random() < 0.6)
    what = rng.choice(["append", "read", "step", "prompt"])
    if what == "append":
        n_seq = _log(rng, 1, 64)
        rows = min(_log(rng, 1, 4096), 16384 // n_seq)
        rot = rng.choice([0, shape["dim"] // 2, shape["dim"]])
        c = _case("", "append", n_seq=n_seq, rows=rows, context=_log(rng, 1, 4096) - 1, rot=rot,
                  interleaved=rot > 0 and rng.random() < 0.5, **shape)
    elif what == "read":
        n_seq = _log(rng, 1, 32)
        c = _case("", "read", n_seq=n_seq, rows=min(_log(rng, 1, 8192), 65536 // n_seq), context=0, **shape)
    elif what == "step":
        n_seq = _log(rng, 1, 96)
        c = _case("", "attend", n_seq=n_seq, rows=rng.choice([1, 1, 1, 2, 3, 5, 8]),
                  context=min(_log(rng, 1, 60000), 400000 // n_seq), **shape)
    else:
        n_seq = _log(rng, 1, 16)
        pairs = 130_000_000_000 // (n_seq * shape["q_heads"] * shape["dim"])  # what the longest listed prompt has, a sequence
        rows = min(_log(rng, 9, 4000), 8000 // n_seq, math.isqrt(pairs))
        c = _case("", "attend", n_seq=n_seq, rows=rows, context=min(_log(rng, 1, 16000), pairs // rows - rows // 2), **shape)
    del c["name"]
    return c


def _spread(most, n, ragged, least):
    """n lengths up to `most`: all equal, or evenly spread and out of order."""
    if not ragged:
        return [most] * n
    step = next(s for s in (7, 11, 13, 17, 1) if math.gcd(s, n) == 1)
    return [max(least, most * ((i * step) % n + 1) // n) for i in range(n)]


def _lengths(case):
    """Each sequence's new rows and the tokens it had before them."""
    rows = _spread(case["rows"], case["n_seq"], case["ragged"] and case["rows"] > 8, 1)
    return rows, _spread(case["context"], case["n_seq"], case["ragged"], 0)


def work(case):
    rows, past = _lengths(case)
    size = 4 if case["dtype"] == "f32" else 2
    dim, tokens = case["dim"], sum(rows)
    stored = case["kv_heads"] * dim * 17 // 16  # bytes of one token's keys and values
    values = case["kv_heads"] * dim * 2
    if case["op"] == "append":  # new q, k, v and the tables in; rotated q and 4-bit k, v out; those read back as values
        return {"bytes": tokens * (size * (2 * case["q_heads"] * dim + 2 * values) + 2 * stored + 4 * case["rot"]),
                "flops": tokens * (case["q_heads"] + case["kv_heads"]) * case["rot"] * 3 + tokens * values * 2}
    if case["op"] == "read":
        return {"bytes": tokens * (stored + size * values), "flops": tokens * values}
    pairs = sum(n * p + n * (n + 1) // 2 for n, p in zip(rows, past))
    return {"bytes": sum(n + p for n, p in zip(rows, past)) * stored + 2 * size * tokens * case["q_heads"] * dim,
            "flops": 4 * dim * case["q_heads"] * pairs}


# --------------------------------------------------------------------------
# the cache's format
# --------------------------------------------------------------------------

def _parts(pool):
    """A pool [pages, heads, P, 17 D / 16] of bytes as its four arrays (views)."""
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


def _quantize(x):
    """Codes [..., D / 2] and exponents [..., D / 32] of x [..., D]."""
    x = x.unflatten(-1, (-1, 32))
    most = x.abs().amax(-1)
    exps = (torch.frexp(most)[1] - 1 - 2 + 127).clamp(E_MIN, E_MAX)
    exps = torch.where(most == 0, E_MIN, exps)
    a = x.abs() * torch.exp2((127 - exps).to(x.dtype)).unsqueeze(-1)
    # to the nearest of the eight magnitudes, a tie to the even code
    code = ((a > 0.25).byte() + (a >= 0.75).byte() + (a > 1.25).byte() + (a >= 1.75).byte()
            + (a > 2.5).byte() + (a >= 3.5).byte() + (a > 5).byte())
    code = (code + 8 * ((x < 0) & (code > 0)).byte()).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), exps.byte()


def _places(state):
    """Each new token's page, its place there and its position."""
    pos = state["past"].long()[state["seq"]] + state["index"]
    P = state["pool"].shape[2]
    return state["table"].long()[state["seq"], pos // P], pos % P, pos


def _store(pool, page, place, k, v):
    kc, vc, ke, ve = _parts(pool)
    kc[page, :, place], ke[page, :, place] = _quantize(k)
    vc[page, :, place], ve[page, :, :, place] = _quantize(v)


def _load(pool, page, place):
    kc, vc, ke, ve = _parts(pool)
    return (_values(kc[page, :, place], ke[page, :, place]), _values(vc[page, :, place], ve[page, :, :, place]))


def _rotated(x, cos, sin, interleaved):
    """x [T, H, D] turned by its tokens' angles (cos, sin [T, r / 2]) in its first r channels."""
    half = cos.shape[-1]
    if half == 0:
        return x
    cos, sin = cos.to(x.dtype).unsqueeze(1), sin.to(x.dtype).unsqueeze(1)
    r, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., :half], r[..., half:])
    c, d = a * cos - b * sin, b * cos + a * sin
    return torch.cat([torch.stack([c, d], -1).flatten(-2) if interleaved else torch.cat([c, d], -1), rest], -1)


# --------------------------------------------------------------------------
# one case
# --------------------------------------------------------------------------

def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rows, past = _lengths(case)
    n, heads, D, P = case["n_seq"], case["kv_heads"], case["dim"], case["page"]
    tokens, dtype = sum(rows), DTYPES[case["dtype"]]
    need = [-(-(a + b) // P) for a, b in zip(rows, past)]
    pages = sum(need) + 3
    # pages are handed out in no order; entries behind a sequence's end name no page
    order = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    table = torch.full((n, max(need) + 2), -1, dtype=torch.int32)
    table = table.to(dev)
    width = torch.tensor(need, device=dev)
    used = torch.arange(table.shape[1], device=dev).unsqueeze(0) < width.unsqueeze(1)
    table[used] = order[:sum(need)]
    cu = torch.tensor([0] + rows, device=dev).cumsum(0).to(torch.int32)
    lens = torch.tensor(rows, device=dev)
    state = {"op": case["op"], "table": table, "cu": cu, "past": torch.tensor(past, dtype=torch.int32, device=dev),
             "seq": torch.repeat_interleave(torch.arange(n, device=dev), lens),
             "rows": max(rows), "most": max(a + b for a, b in zip(rows, past)), "interleaved": case["interleaved"]}
    state["index"] = torch.arange(tokens, device=dev) - cu.long()[state["seq"]]
    # every page holds keys and values of other tokens: normal, with a few strong key channels
    pool = torch.empty((pages, heads, P, D * 17 // 16), dtype=torch.uint8, device=dev)
    strong = 1 + 5 * (torch.rand((heads, D), generator=gen, device=dev) < 0.05)
    kc, vc, ke, ve = _parts(pool)
    for at in range(0, pages, 512):
        some = min(512, pages - at)
        kc[at:at + some], ke[at:at + some] = _quantize(
            torch.randn((some, heads, P, D), generator=gen, device=dev) * strong.unsqueeze(1))
        c, e = _quantize(torch.randn((some, heads, P, D), generator=gen, device=dev))
        vc[at:at + some], ve[at:at + some] = c, e.transpose(-1, -2)
    state["pool"] = pool
    if case["op"] == "attend":
        state["q"] = (torch.randn((tokens, case["q_heads"], D), generator=gen, device=dev) * 1.2).to(dtype)
        state["out"] = torch.empty_like(state["q"])
        return state
    state["k_out"] = torch.empty((tokens, heads, D), dtype=dtype, device=dev)
    state["v_out"] = torch.empty_like(state["k_out"])
    if case["op"] == "append":
        # q, k and v lie side by side, as one projection leaves them
        joint = torch.randn((tokens, case["q_heads"] + 2 * heads, D), generator=gen, device=dev).to(dtype)
        state["q"], state["k"], state["v"] = joint.split([case["q_heads"], heads, heads], 1)
        state["q_out"] = torch.empty((tokens, case["q_heads"], D), dtype=dtype, device=dev)
        state["cos"] = state["sin"] = None
        if case["rot"]:
            half = case["rot"] // 2
            angle = (torch.arange(state["most"], device=dev, dtype=torch.float64).unsqueeze(1)
                     * 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half))
            state["cos"], state["sin"] = angle.cos().float(), angle.sin().float()
    return state


def _plain_append(s):
    page, place, pos = _places(s)
    if s["cos"] is None:
        cos = sin = torch.empty((pos.shape[0], 0), device=pos.device)
    else:
        cos, sin = s["cos"][pos], s["sin"][pos]
    # 64 bits decide a key next to a rounding border
    _store(s["pool"], page, place, _rotated(s["k"].double(), cos, sin, s["interleaved"]), s["v"].float())
    s["q_out"].copy_(_rotated(s["q"].float(), cos, sin, s["interleaved"]))
    return (s["q_out"],) + _plain_read(s)


def _plain_read(s):
    page, place, _ = _places(s)
    k, v = _load(s["pool"], page, place)
    s["k_out"].copy_(k)
    s["v_out"].copy_(v)
    return s["k_out"], s["v_out"]


def _plain_attend(s):
    """Sequences padded to the longest, in one batch."""
    pool, q, table = s["pool"], s["q"], s["table"]
    heads, P, D = pool.shape[1], pool.shape[2], pool.shape[3] * 16 // 17
    n, group, rows = table.shape[0], q.shape[1] // heads, s["rows"]
    pages = table[:, :-(-s["most"] // P)].long().clamp(min=0)
    L = pages.shape[1] * P
    kc, vc, ke, ve = _parts(pool)
    keys = _values(kc[pages], ke[pages]).transpose(1, 2).reshape(n, heads, L, D)
    scores = q.new_zeros((n, rows, heads, group, D), dtype=torch.float32)
    scores[s["seq"], s["index"]] = q.float().unflatten(1, (heads, group))
    scores = scores.permute(0, 2, 1, 3, 4).reshape(n, heads, rows * group, D)
    scores = torch.matmul(scores, keys.transpose(-1, -2).contiguous()) * (1 / math.sqrt(D))
    del keys
    at = s["past"].unsqueeze(1) + torch.arange(rows, device=q.device)
    hidden = torch.arange(L, device=q.device) > at.unsqueeze(-1)  # [n, rows, L]
    scores = scores.view(n, heads, rows, group, L).masked_fill_(hidden[:, None, :, None], -math.inf)
    weights = torch.exp(scores - scores.amax(-1, keepdim=True))
    del scores
    total = weights.sum(-1, keepdim=True)
    values = _values(vc[pages], ve[pages].transpose(-1, -2)).transpose(1, 2).reshape(n, heads, L, D)
    o = torch.matmul(weights.view(n, heads, rows * group, L), values).view(n, heads, rows, group, D) / total
    s["out"].copy_(o.permute(0, 2, 1, 3, 4)[s["seq"], s["index"]].flatten(1, 2))
    return s["out"]


def run(state):
    s = state
    if not own:
        return {"append": _plain_append, "read": _plain_read, "attend": _plain_attend}[s["op"]](s)
    from kda_gated_delta_decode_amd import binding as B
    if s["op"] == "attend":
        B.kda_kv_attend(s["pool"], s["table"], s["cu"], s["past"], s["q"], s["out"], max_rows=s["rows"],
                        max_kv_len=s["most"])
        return s["out"]
    if s["op"] == "append":
        B.kda_kv_append(s["pool"], s["table"], s["cu"], s["past"], s["k"], s["v"], q=s["q"], q_out=s["q_out"],
                        cos=s["cos"], sin=s["sin"], interleaved=s["interleaved"])
    B.kda_kv_read(s["pool"], s["table"], s["cu"], s["past"], s["k_out"], s["v_out"])
    return (s["q_out"], s["k_out"], s["v_out"]) if s["op"] == "append" else (s["k_out"], s["v_out"])


# --------------------------------------------------------------------------
# the definition, in 64 bits
# --------------------------------------------------------------------------

def _exact_turn(x, pos, case):
    """The rotation as a complex product, from the tables' own fp32 entries."""
    r = case["rot"]
    if r == 0:
        return x
    half = r // 2
    angle = pos.double().unsqueeze(1) * 10000.0 ** (-torch.arange(half, device=x.device, dtype=torch.float64) / half)
    turn = torch.complex(angle.cos().float().double(), angle.sin().float().double()).unsqueeze(1)
    y = x.clone()
    i = torch.arange(half, device=x.device)
    a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
    z = torch.complex(x[..., a], x[..., b]) * turn
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_stored(x):
    """The values that the format keeps of x: the nearest by distance, ties to even, block by block."""
    y = x.reshape(-1, 32)
    most = y.abs().max(1, keepdim=True).values
    unit = torch.exp2(torch.log2(torch.where(most > 0, most, 1e-300)).floor() - 2)
    unit = torch.where(unit * 4 > most, unit / 2, unit)
    unit = torch.where(unit * 8 <= most, unit * 2, unit).clamp(2.0 ** (E_MIN - 127), 2.0 ** (E_MAX - 127))
    a = (y.abs() / unit).clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.round(a / step) * step * torch.sign(y) * unit).reshape(x.shape)


def _exact_cached(pool, table, n_tokens, which):
    """One sequence's first n_tokens keys (0) or values (1), fp64 [heads, n_tokens, D]."""
    pages, heads, P, width = pool.shape
    D = width * 16 // 17
    t = torch.arange(n_tokens, device=pool.device)
    block = pool.reshape(pages, heads, P * width)[table.long()[t // P]]  # [n, heads, bytes]
    c = torch.arange(D, device=pool.device)
    code = torch.gather(block, 2, ((which * P + t % P).view(-1, 1, 1) * (D // 2) + c // 2).expand(-1, heads, -1)).int()
    code = (code >> (4 * (c % 2))) & 15
    if which == 0:
        at = P * D + (t % P).view(-1, 1, 1) * (D // 32) + c // 32
    else:
        at = P * D + P * D // 32 + (c // 32) * P + (t % P).view(-1, 1, 1)
    e = torch.gather(block, 2, at.expand(-1, heads, -1)).double()
    m, x = code & 1, (code >> 1) & 3  # mantissa and exponent of E2M1
    mag = torch.where(x > 0, (1 + 0.5 * m) * torch.exp2(x.double() - 1), 0.5 * m.double())
    return ((1 - 2 * (code >> 3)) * mag * torch.exp2(e - 127)).transpose(0, 1).contiguous()


def exact(case, seed):
    s = prepare(case, seed)
    cu, past = s["cu"].tolist(), s["past"].tolist()
    if case["op"] == "append":
        pos = s["past"].long()[s["seq"]] + s["index"]
        return (_exact_turn(s["q"].double(), pos, case), _exact_stored(_exact_turn(s["k"].double(), pos, case)),
                _exact_stored(s["v"].double()))
    if case["op"] == "read":
        return tuple(torch.cat([_exact_cached(s["pool"], s["table"][i], cu[i + 1] - cu[i], w).transpose(0, 1)
                                for i in range(case["n_seq"])]) for w in (0, 1))
    q, D, heads = s["q"].double(), case["dim"], case["kv_heads"]
    out = torch.empty_like(q)
    group = case["q_heads"] // heads
    for i in range(case["n_seq"]):
        L = past[i] + cu[i + 1] - cu[i]
        K, V = (_exact_cached(s["pool"], s["table"][i], L, w) for w in (0, 1))
        for first in range(cu[i], cu[i + 1], 1024):
            last = min(first + 1024, cu[i + 1])
            at = torch.arange(first, last, device=q.device) - cu[i] + past[i]
            seen = torch.arange(L, device=q.device) <= at.unsqueeze(1)
            for h in range(case["q_heads"]):
                logits = (q[first:last, h] / math.sqrt(D)) @ K[h // group].T
                out[first:last, h] = torch.softmax(logits.masked_fill(~seen, -math.inf), -1) @ V[h // group]
    return out
