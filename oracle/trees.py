"""Trees of drafted tokens in 64-bit NumPy, from their definitions: attention of a
tree's nodes, the KDA recurrence along every path, the verification of drafted
tokens from given random numbers, and the accepted path's cache entries.  It
shares no code with the GPU path; its own pins are in tests/test_tree_cpu.py.

Every function takes one request at a time; parents[i] is -1 or below i.
"""
from __future__ import annotations

import numpy as np


def path_to(parents, node):
    """The nodes from the root down to `node`."""
    way = []
    while node >= 0:
        way.append(node)
        node = parents[node]
    return way[::-1]


def attend(k, v, q, past, parents, scale):
    """Rows q [n, Hq, D] over cached k, v [past + n, H, D]: node i sees the context
    and its path.  Returns what kv_cache.attend does."""
    n, heads, D = q.shape
    group = heads // k.shape[1]
    out, mass, most = np.zeros(q.shape), np.zeros((n, heads)), np.zeros((n, heads))
    for i in range(n):
        seen = list(range(past)) + [past + j for j in path_to(parents, i)]
        for h in range(heads):
            kk, vv, x = k[seen, h // group], v[seen, h // group], q[i, h].astype(np.float64)
            s = kk @ x * scale
            w = np.exp(s - s.max()) if np.isfinite(s).all() else np.full(len(seen), np.nan)
            out[i, h] = w @ vv / w.sum()
            mass[i, h] = (np.abs(kk) @ np.abs(x)).max() * abs(scale)
            most[i, h] = np.abs(vv).max()
    return out, mass, most


def step(S, k, v, g, b):
    """One token's update of S [H, 128, 128]."""
    k = k / np.sqrt((k * k).sum(-1, keepdims=True) + 1e-6)
    S = np.exp(g)[..., None] * S
    u = v - np.einsum("hk,hkv->hv", k, S)
    return S + (1 / (1 + np.exp(-b)))[:, None, None] * k[..., None] * u[:, None, :]


def recurrence(S0, parents, q, k, v, g, b, scale):
    """Every node's read-out [n, H, 128] from state S0 [H, 128, 128]."""
    q, k, v, g, b = (np.asarray(x, np.float64) for x in (q, k, v, g, b))
    qn = q / np.sqrt((q * q).sum(-1, keepdims=True) + 1e-6)
    states, out = [], np.empty(v.shape)
    for i, p in enumerate(parents):
        states.append(step(np.asarray(S0, np.float64) if p < 0 else states[p], k[i], v[i], g[i], b[i]))
        out[i] = scale * np.einsum("hk,hkv->hv", qn[i], states[i])
    return out


def advance(S0, path, k, v, g, b):
    """The state after the nodes of `path`, one after the other."""
    S = np.asarray(S0, np.float64)
    for i in path:
        S = step(S, *(np.asarray(x[i], np.float64) for x in (k, v, g, b)))
    return S


def _weights(row):
    row = np.asarray(row, np.float64)
    return np.where(row > 0, row, 0.0)


def verify(target, draft, parents, tokens, accept, sample, max_path=64):
    """(path, following token) of one request: target [n, V], draft the same or
    None.  A walk by children; a node's are tried in their order."""
    n, V = len(parents), target.shape[1]
    path, f, mass = [0], _weights(target[0]).copy(), 1.0
    while len(path) < max_path:
        last = path[-1]
        f, mass, taken = _weights(target[last]).copy(), 1.0, None
        for i in [j for j in range(n) if parents[j] == last]:
            x, u = int(tokens[i]), float(accept[i])
            inside = 0 <= x < V
            have = f[x] if inside else 0.0
            q = _weights(draft[last]) if draft is not None else None
            if u * ((q[x] if inside else 0.0) if q is not None else 1.0) * mass < have:
                taken = i
                break
            if q is not None:
                f = np.maximum(f - mass * q, 0.0)
                mass = f.sum()
            else:
                mass -= have
                if inside:
                    f[x] = 0.0
        if taken is None:
            break
        path.append(taken)
        f = _weights(target[taken]).copy()
    if not f.sum() > 0:
        f = _weights(target[path[-1]])
    total = f.sum()
    if not 0 < total < np.inf:
        return path, -1
    hit = np.flatnonzero((np.cumsum(f) > float(sample) * total) & (f > 0))
    return path, int(hit[0] if hit.size else np.flatnonzero(f > 0)[-1])


def keep(tokens, past, path):
    """tokens: an array whose rows are one sequence's cached tokens, changed in
    place as the definition says: row past + path[e] becomes row past + e."""
    old = tokens.copy()
    for e, i in enumerate(path):
        tokens[past + e] = old[past + i]
