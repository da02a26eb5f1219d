"""GPU tests of the calls for trees of drafted tokens against the 64-bit oracle.

Tolerances, set before the first run.  Attention: kda_kv_attend's (derived in
test_kv_gpu.py), the kernels being the same but for the mask.  Verification and
kept cache entries: equal.  Read-outs of a tree: every number is a sum of at most
128 products of a unit vector and a column of S0, and of one term for each node
above, whose coefficients are at most 1 in size; with the norms', decays' and
gates' roundings (a few units each, one for each step of the path) a read-out of
node i, column c, is off by at most
    2 * 2^-24 * (128 + 16 len) * scale * (|S0[:, c]| + sum of |v_j[c]| on the path),
len being the path's length (the update never lengthens a column by more than
|v_j[c]|, so that bounds every number on the way too).  A stored state is off by as
much without the scale, an fp16 one by half a step more (2^-11 of it, 2^-25 at
least).
"""
import numpy as np
import pytest

import test_kv_gpu as K
from gpu_helpers import B, need_gpu, torch
from oracle import kv_cache as O
from oracle import trees as T

pytestmark = pytest.mark.gpu

dev, host, i32 = K.dev, K.host, K.i32
TYPES, HALF_STEP = K.TYPES, K.HALF_STEP


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def chain(n):
    return [i - 1 for i in range(n)]


def star(n):
    return [-1] + [0] * (n - 1) if n else []


def some_tree(n, seed, roots=1):
    """Parents anywhere before the node, the nearest likelier; the first nodes are roots."""
    rng = np.random.default_rng(seed)
    return [-1 if i < roots else int(i - 1 - min(i - 1, rng.geometric(0.3) - 1)) for i in range(n)]


# --------------------------------------------------------------------------
# attention
# --------------------------------------------------------------------------

class TreeCase(K.Case):
    def __init__(self, trees, past, **kw):
        super().__init__([len(t) for t in trees], past, **kw)
        self.trees = trees
        self.up = np.full(self.T, 77, np.int32)  # rows of no request: no parents
        for s, t in enumerate(trees):
            self.up[self.cu[s]:self.cu[s + 1]] = t
        self.d_up = dev(self.up)

    def attend(self, out=None, **kw):
        out = torch.empty(self.T, self.hq, self.D, dtype=TYPES[self.dtype], device="cuda") if out is None else out
        kw.setdefault("max_rows", max(self.rows + [0]))
        kw.setdefault("max_kv_len", max([a + b for a, b in zip(self.rows, self.past)] + [0]))
        B.kda_kv_attend_tree(self.d_pool, self.d_table, self.d_cu, self.d_past, self.d_up, self.q, out, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, scale=None, which=None, rows=None):
        scale = self.D ** -0.5 if scale is None else scale
        got, drop = host(out), 0.0 if self.dtype == "f32" else 2.0 ** -11
        for s in range(self.n) if which is None else which:
            a, b, N = self.cu[s], self.cu[s + 1], self.past[s] + self.rows[s]
            if a == b:
                continue
            k, v = O.read(self.pool, self.table[s], 0, N)
            want, mass, top = T.attend(k, v, self.hq_np[a:b], self.past[s], self.trees[s], scale)
            e = (3 * self.D + 4) * 2.0 ** -24 * mass[..., None]
            if self.dtype == "bf16":
                spread = np.abs(self.hq_np[a:b]).max(-1) * np.abs(k).sum(-1).max() * abs(scale)
                e = e + 2.0 ** -25 * spread[..., None]
            assert not (e >= 0.1).any()
            tol = top[..., None] * (2 * (2 * e + 2.0 ** -22) + 2 * (N + 64) * 2.0 ** -24 + drop)
            tol = tol + HALF_STEP[self.dtype] * (np.abs(want) + tol) + 2.0 ** -25
            ok = (np.abs(got[a:b] - want) <= tol) | (np.isnan(got[a:b]) & np.isnan(want))
            assert ok.all(), (s, np.argwhere(~ok)[:5], np.nanmax(np.abs(got[a:b] - want)))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,P,heads", [(128, 16, (4, 2)), (64, 32, (8, 1)), (128, 128, (3, 3)), (64, 256, (5, 1))])
def test_attend_tree(dtype, D, P, heads):
    trees = [some_tree(9, 1), chain(1), star(17), [], some_tree(64, 2, roots=3), chain(33), some_tree(48, 3)]
    c = TreeCase(trees, [0, 40, 15, 9, 130, 1, 63], dtype=dtype, D=D, P=P, heads=heads, seed=D + P, lead=3, trail=4).fill()
    out = torch.full((c.T, c.hq, D), 7.0, dtype=TYPES[dtype], device="cuda")
    c.check(c.attend(out))
    rest = host(out)
    assert (rest[:3] == 7).all() and (rest[c.cu[-1]:] == 7).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n", [1, 2, 5, 8, 12, 16, 17, 31, 32, 63, 64])
def test_attend_tree_sizes_and_tiles(dtype, n):
    # 2 query heads a cached head: 16-, 32- and 128-row tiles as n grows
    c = TreeCase([some_tree(n, n), some_tree(max(1, n // 2), n + 1)], [n + 3, 257], dtype=dtype, heads=(4, 2), D=64, P=64,
                 seed=n).fill()
    c.check(c.attend())


@pytest.mark.parametrize("rows,past,heads", [([8, 3], [700, 90], (4, 2)), ([1], [600], (2, 2)), ([32, 2], [400, 0], (2, 2)),
                                             ([16], [2000], (4, 4)), ([5], [3000], (8, 8)), ([40], [40], (2, 2))])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_a_small_chain_gives_the_bits_of_causal_attention(rows, past, heads, dtype):
    c = TreeCase([chain(n) for n in rows], past, dtype=dtype, heads=heads, D=128, P=32, seed=5).fill()
    want = K.Case.attend(c)
    assert torch.equal(c.attend().view(torch.uint8), want.view(torch.uint8))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("n,past,heads", [(13, 4100, (2, 2)), (64, 3000, (8, 1)), (7, 9000, (2, 1)), (20, 2500, (4, 1))])
def test_attend_tree_over_splits(dtype, n, past, heads):
    c = TreeCase([some_tree(n, n)], [past], dtype=dtype, heads=heads, D=128, P=128, seed=n).fill()
    assert B.kda_kv_attend_tree_workspace(c.d_pool, c.d_table, c.T, c.hq, n, past + n, dtype) > 0
    c.check(c.attend())


@pytest.mark.parametrize("past", [0, 1, 15, 16, 17, 30, 31, 32, 33, 62, 63, 64, 65, 127, 128, 129, 500, 511, 512, 513])
@pytest.mark.parametrize("heads", [(1, 1), (4, 1)])
def test_nodes_across_tile_and_split_borders(past, heads):
    c = TreeCase([some_tree(40, past)], [past], dtype="bf16", heads=heads, D=64, P=16, seed=past).fill()
    c.check(c.attend())


def test_sizes_of_the_launch_are_hints():
    c = TreeCase([some_tree(30, 1), some_tree(9, 2)], [300, 20], heads=(4, 2), D=64, P=16).fill()
    for kw in (dict(max_rows=1, max_kv_len=1), dict(max_rows=64, max_kv_len=0), dict(max_rows=0, max_kv_len=5)):
        c.check(c.attend(**kw))
    out = torch.empty(c.T, c.hq, c.D, device="cuda")
    B.kda_kv_attend_tree(c.d_pool, c.d_table, c.d_cu, c.d_past, c.d_up, c.q, out)
    c.check(out)


def test_a_workspace_that_is_not_needed_is_left_alone():
    # 40 nodes x 8 query heads, tiles of 128 rows, too few tokens for parts
    c = TreeCase([some_tree(40, 1), some_tree(9, 2)] * 3, [100, 20] * 3, heads=(8, 1), D=64, P=16).fill()
    assert B.kda_kv_attend_tree_workspace(c.d_pool, c.d_table, c.T, c.hq, 40, 140) == 0
    around = torch.full((4096,), 7, dtype=torch.uint8, device="cuda")
    c.check(c.attend(workspace=around[2048:2064]))
    assert bool((around == 7).all())


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("bf16", 128)])
def test_large_trees_of_many_sequences(dtype, D):
    # more sequences than a wave has lanes, of uneven sizes; some without rows
    rng = np.random.default_rng(8)
    rows = [int(x) for x in rng.integers(0, 65, 140)]
    past = [int(x) for x in rng.integers(0, 200, 140)]
    rows[3], past[3], rows[69], past[69], rows[130], past[130] = 64, 2900, 33, 1500, 17, 777
    c = TreeCase([some_tree(n, i) for i, n in enumerate(rows)], past, dtype=dtype, heads=(8, 1), D=D, P=64).fill()
    assert B.kda_kv_attend_tree_workspace(c.d_pool, c.d_table, c.T, c.hq, 64, 2964, dtype) > 0
    c.check(c.attend())


def test_large_trees_that_fill_the_chip_uncut():
    # so many tiles that none is cut, more sequences than two waves have lanes
    rng = np.random.default_rng(9)
    rows = [int(x) for x in rng.integers(0, 65, 140)]
    c = TreeCase([some_tree(n, i) for i, n in enumerate(rows)], [int(x) for x in rng.integers(0, 300, 140)], dtype="bf16",
                 heads=(16, 2), D=64, P=32).fill()
    assert B.kda_kv_attend_tree_workspace(c.d_pool, c.d_table, c.T, c.hq, 64, 364, "bf16") == 0
    c.check(c.attend(max_rows=64, max_kv_len=364))


@pytest.mark.parametrize("n", [3, 70])
@pytest.mark.parametrize("max_rows,max_kv_len", [(20, 600), (64, 100), (17, 0), (64, 1000000)])
def test_sizes_of_large_trees_are_hints(n, max_rows, max_kv_len):
    c = TreeCase([some_tree(64, i) if i % 7 == 2 else some_tree(5, i) for i in range(n)],
                 [1900 if i % 35 == 2 else 13 for i in range(n)], dtype="f16", heads=(8, 1), D=64, P=64).fill()
    c.check(c.attend(max_rows=max_rows, max_kv_len=max_kv_len))


def test_large_trees_many_of_whose_sequences_are_bad():
    rows = [64, 33, 64, 20, 64]
    c = TreeCase([some_tree(n, i) for i, n in enumerate(rows)], [2000, 40, 700, 3000, 9], heads=(8, 1), D=64, P=16).fill()
    c.d_past[1], c.d_past[3] = -1, c.table.shape[1] * 16  # no length; past the table's end
    out = c.attend()
    c.check(out, which=[0, 2, 4])
    for s in (1, 3):
        assert bool(out[c.cu[s]:c.cu[s + 1]].isnan().all())


@pytest.mark.parametrize("n,nodes,past,heads,D,dtype", [
    (25, 32, 400, (32, 8), 128, "bf16"), (15, 32, 1020, (32, 8), 128, "bf16"), (3, 48, 1960, (32, 8), 128, "f16"),
    (50, 20, 390, (16, 4), 64, "f16"), (43, 20, 390, (8, 2), 128, "f32"), (64, 10, 390, (24, 3), 64, "bf16")])
@pytest.mark.parametrize("uneven", [False, True])
def test_large_trees_whose_first_parts_have_no_place(n, nodes, past, heads, D, dtype, uneven):
    # parts of (all steps) / (places) steps, rounded up, would be more than the places
    rng = np.random.default_rng(n)
    rows, lens = [nodes] * n, [past] * n
    if uneven:
        rows = [int(x) for x in rng.integers(nodes - 2, nodes + 1, n)]
        lens = [int(x) for x in rng.integers(past - past // 40, past + 1, n)]
    c = TreeCase([some_tree(m, i) for i, m in enumerate(rows)], lens, dtype=dtype, heads=heads, D=D, P=64, seed=n).fill()
    units = np.array([-(-m * (heads[0] // heads[1]) // 128) * heads[1] for m in rows])
    steps = np.array([-(-(m + t) // 64) for m, t in zip(rows, lens)])
    most = max(a + b for a, b in zip(rows, lens))
    work = B.kda_kv_attend_tree_workspace(c.d_pool, c.d_table, c.T, c.hq, max(rows), most, dtype)
    places = (work - (n + 31) // 32 * 256) // (128 * (D + 2) * 4)
    first = max(3, -(-int((units * steps).sum()) // places))
    assert 3 <= first < 8 and (units * -(-steps // first)).sum() > places > units.sum()
    out = c.attend()
    assert bool(out.isfinite().all())
    c.check(out, which=sorted({0, 1, n // 2, n - 2, n - 1}))


@pytest.mark.parametrize("heads", [(2, 2), (8, 1)])
@pytest.mark.parametrize("past", [5, 3000])
def test_trees_that_are_none_are_nan(heads, past):
    trees = [some_tree(20, 1), chain(65), some_tree(20, 2), some_tree(8, 3), star(7), chain(70)]
    c = TreeCase(trees, [past] * 6, heads=heads, D=64, P=32).fill()
    for row, parent in ((c.cu[2] + 19, 19), (c.cu[3], 0), (c.cu[4] + 3, -2)):
        c.up[row] = parent
    c.d_up = dev(c.up)
    out = c.attend(max_rows=64)
    c.check(out, which=[0])
    assert np.isnan(host(out)[c.cu[1]:]).all()


def test_a_poisoned_node_spoils_its_descendants_alone():
    tree = [-1, 0, 0, 1, 1, 2, 5, -1]
    c = TreeCase([tree], [70], heads=(4, 2), D=128, P=16).fill()
    block = O.Block(c.pool[c.table[0, 71 // 16], 1])
    block.ke[71 % 16] = 255  # node 1, cached head 1
    c.d_pool = dev(c.pool)
    got = host(c.attend())
    for i in range(8):
        spoiled = 1 in T.path_to(tree, i)
        assert np.isnan(got[i, 2:]).all() == spoiled and np.isfinite(got[i, :2]).all()
        assert spoiled or np.isfinite(got[i]).all()
    c.pool[c.table[0, 71 // 16], 1] = 0
    # values of a token that a row does not see may be anything: infinite exponents
    # cannot be stored, the largest may
    c2 = TreeCase([[-1, 0, 0]], [3], heads=(2, 2), D=64, P=16).fill()
    O.Block(c2.pool[c2.table[0, 0], 0]).ve[:, 4] = 252
    c2.d_pool = dev(c2.pool)
    got = host(c2.attend())
    assert np.abs(got[[0, 2]]).max() < 100 and np.isfinite(got).all()


@pytest.mark.parametrize("past,page", [(40, 0), (40, 2), (2000, 3), (2000, 125)])
def test_a_missing_page_is_nan(past, page):
    c = TreeCase([some_tree(5, 1), some_tree(6, 2)], [past, past], heads=(2, 2), D=64, P=16).fill()
    c.table[1, page] = -1
    c.d_table = dev(c.table)
    got = host(c.attend())
    a, b = c.cu[1], c.cu[2]
    c.check(dev(got, TYPES["f32"]), which=[0])
    first = past // 16  # the page of node 0
    for i in range(b - a):
        seen = page < first or any((past + j) // 16 == page for j in T.path_to(c.trees[1], i))
        assert np.isnan(got[a + i]).all() == seen


@pytest.mark.parametrize("dtype,D", [("f32", 64), ("f16", 128), ("bf16", 64), ("bf16", 128)])
@pytest.mark.parametrize("past", [20, 1500])
def test_a_poisoned_node_of_a_large_tree(dtype, D, past):
    # tiles of 128 rows, in one part and in many; the node's own page holds others too
    tree = some_tree(60, 5, roots=2)
    c = TreeCase([tree], [past], dtype=dtype, heads=(8, 2), D=D, P=64).fill()
    assert T.path_to(tree, 59)[0] in (0, 1)
    at = past + 7
    O.Block(c.pool[c.table[0, at // 64], 1]).ke[at % 64] = 255  # node 7, cached head 1
    c.d_pool = dev(c.pool)
    got = host(c.attend())
    for i in range(60):
        spoiled = 7 in T.path_to(tree, i)
        assert np.isnan(got[i, 4:]).all() == spoiled and np.isfinite(got[i, :4]).all()
        assert spoiled or np.isfinite(got[i]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("past", [20, 1500])
def test_exponents_outside_fp16_in_a_large_tree(dtype, past):
    # a small key and a small value late in the context and in a node: the tiles go on in bf16
    c = TreeCase([some_tree(64, 6)], [past], dtype=dtype, heads=(8, 2), D=64, P=64).fill()
    for at in (past - 3, past + 9):
        b = O.Block(c.pool[c.table[0, at // 64], 0])
        b.ke[at % 64], b.ve[:, at % 64] = 90, 80
    c.d_pool = dev(c.pool)
    c.check(c.attend())


@pytest.mark.parametrize("D,heads", [(64, (8, 1)), (128, (16, 2))])
@pytest.mark.parametrize("past", [60, 250])
def test_weights_of_large_fp16_trees_keep_their_bits(D, heads, past):
    # Two scores, 0 and -x scale, whose values are 1 and -1: an output is (a - n w) / (a + n w)
    # for w = exp(-x scale), off by up to half of what w is, 2^-12 were it held in 11
    # bits.  A score is one exact product, rounded twice (scale is a power of two at
    # D = 64): w is off by less than 2^-20 of itself (x scale < 1), in two fp16 pieces by 2^-22
    # more, and the sums as everywhere.
    c = TreeCase([chain(10), some_tree(12, 1)], [past, past // 2], dtype="f16", heads=heads, D=D, P=64, seed=D + past)
    for s in range(2):
        n = c.past[s] + c.rows[s]
        k, v = np.zeros((n, c.h, D)), np.ones((n, c.h, D))
        less = np.arange(n) % 5 < 3
        k[less, :, 0], v[less] = -1, -1
        O.append(c.pool, c.table[s], 0, k, v)
    c.d_pool = dev(c.pool)
    c.q = torch.zeros(c.T, c.hq, D, dtype=torch.float16)
    c.q[:, :, 0] = torch.linspace(0.3, 0.69, c.T * c.hq).view(c.T, c.hq) * D ** 0.5
    c.hq_np, c.q = host(c.q), c.q.cuda()
    got = host(c.attend())
    for s in range(2):
        a, b, n = c.cu[s], c.cu[s + 1], c.past[s] + c.rows[s]
        k, v = O.read(c.pool, c.table[s], 0, n)
        want, _, top = T.attend(k, v, c.hq_np[a:b], c.past[s], c.trees[s], D ** -0.5)
        assert np.abs(want).max() < 0.25 and (top == 1).all()
        tol = 2.0 ** -20 + 2.0 ** -22 + 2 * (n + 64) * 2.0 ** -24 + HALF_STEP["f16"] * np.abs(want)
        assert (np.abs(got[a:b] - want) <= tol).all(), (s, (np.abs(got[a:b] - want) / tol).max())


def test_large_trees_in_place_with_strides_and_bad_sequences():
    c = TreeCase([some_tree(60, 1), some_tree(40, 2), some_tree(3, 3)], [900, 0, 5], heads=(8, 2), D=64, P=64, dtype="bf16",
                 seed=3).fill()
    c.d_past[1] = -1
    out = c.attend()
    c.check(out, which=[0, 2])
    assert np.isnan(host(out)[60:100]).all()
    q = c.q.contiguous()
    B.kda_kv_attend_tree(c.d_pool, c.d_table, c.d_cu, c.d_past, c.d_up, q, q, max_rows=60, max_kv_len=960)
    torch.cuda.synchronize()
    assert torch.equal(q.view(torch.int16), out.view(torch.int16))


def test_attend_tree_in_place_with_strides_and_bad_sequences():
    c = TreeCase([some_tree(7, 1), some_tree(4, 2), some_tree(3, 3)], [20, -1, 5], heads=(2, 2), D=64, P=16, dtype="f16",
                 seed=3)
    c.past = [20, 0, 5]
    c.fill()
    out = c.attend()
    c.past[1] = 0
    c.check(out, which=[0, 2])
    assert np.isnan(host(out)[7:11]).all()
    q = c.q.contiguous()
    B.kda_kv_attend_tree(c.d_pool, c.d_table, c.d_cu, c.d_past, c.d_up, q, q, max_rows=7)
    torch.cuda.synchronize()
    assert torch.equal(q.view(torch.int16), out.view(torch.int16))


def test_append_at_turns_by_positions_and_stores_by_places():
    c = K.Case([6, 3], [10, 30], dtype="f32", heads=(4, 2), D=64, P=16, seed=8)
    half, N = 16, 64
    angle = np.arange(N)[:, None] * 100.0 ** (-np.arange(half) / half)
    cos, sin = np.cos(angle).astype(np.float32), np.sin(angle).astype(np.float32)
    pos = np.array([10, 11, 11, 12, 12, 12, 30, N, -1], np.int32)  # the last two have none
    q_out = torch.zeros(c.T, c.hq, c.D, device="cuda")
    before = c.pool.copy()
    B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v, q=c.q, q_out=q_out, cos=dev(cos), sin=dev(sin),
                    positions=i32(pos))
    torch.cuda.synchronize()
    got = c.d_pool.cpu().numpy()
    want = before.copy()
    for t in range(7):
        s = 0 if t < 6 else 1
        p = c.past[s] + t - c.cu[s]
        for h in range(c.h):
            k = O.rotate(c.k_np[t, h], cos[pos[t]], sin[pos[t]], False)
            O.Block(want[c.table[s, p // 16], h]).store(p % 16, k, c.v_np[t, h])
    K.same_cache(got, want)
    turned = np.stack([O.rotate(c.hq_np[t], cos[pos[t]], sin[pos[t]], False) for t in range(7)])
    size = np.abs(c.hq_np[:7]).max()
    assert np.abs(host(q_out)[:7] - turned).max() <= 4 * 2.0 ** -24 * 2 * size
    assert np.isnan(host(q_out)[7:]).all()


def test_append_at_the_places_is_append():
    c = K.Case([5, 4], [3, 17], dtype="bf16", heads=(4, 2), D=128, P=16, seed=9)
    cos, sin = (torch.rand(40, 32, device="cuda") for _ in range(2))
    pos = i32([3, 4, 5, 6, 7, 17, 18, 19, 20])
    a, b = c.d_pool.clone(), c.d_pool.clone()
    for pool, kw in ((a, {}), (b, dict(positions=pos))):
        B.kda_kv_append(pool, c.d_table, c.d_cu, c.d_past, c.k, c.v, cos=cos, sin=sin, **kw)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    # without a rotation positions are not looked at
    B.kda_kv_append(a, c.d_table, c.d_cu, c.d_past, c.k, c.v)
    B.kda_kv_append(b, c.d_table, c.d_cu, c.d_past, c.k, c.v, positions=i32([-5] * 9))
    torch.cuda.synchronize()
    assert torch.equal(a, b)


# --------------------------------------------------------------------------
# kept entries
# --------------------------------------------------------------------------

def keep(c, paths, lens=None, width=None, **kw):
    width = width or max(len(p) for p in paths)
    table = np.full((len(paths), width), 99, np.int32)
    for s, p in enumerate(paths):
        table[s, :len(p)] = p
    lens = [len(p) for p in paths] if lens is None else lens
    B.kda_kv_keep(c.d_pool, c.d_table, c.d_cu, c.d_past, dev(table), i32(lens), **kw)
    torch.cuda.synchronize()
    return c.d_pool.cpu().numpy()


def expect(c, paths):
    """The whole pool after keeping: blocks' tokens as rows of bytes."""
    want = c.pool.copy()
    for s, path in enumerate(paths):
        for h in range(c.h):
            def rows(pool):
                blocks = [O.Block(pool[page, h]) for page in c.table[s] if page >= 0]
                return [np.concatenate(x) for x in zip(*((b.kc, b.vc, b.ke, b.ve.T) for b in blocks))], blocks
            new, blocks = rows(want)
            for x in new:
                T.keep(x, c.past[s], path)
            P = c.P
            for j, b in enumerate(blocks):
                b.kc[:], b.vc[:], b.ke[:], b.ve[:] = (new[0][j * P:(j + 1) * P], new[1][j * P:(j + 1) * P],
                                                      new[2][j * P:(j + 1) * P], new[3][j * P:(j + 1) * P].T)
    return want


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("h", [1, 3, 8])
def test_keep(D, P, h):
    paths = [[0, 2, 5, 6], [0], [], [0, 1, 2, 3], [3], list(range(0, 64, 3)), list(range(64)), list(range(5, 64)), [0, 1, 4, 5, 9, 10, 11, 12, 33]]
    rows = [9, 4, 5, 4, 4, 64, 64, 64, 40]
    c = K.Case(rows, [0, 3, 7, 14, 15, 250, 9, 60, 31], heads=(h, h), D=D, P=P, seed=h)
    assert np.array_equal(keep(c, paths), expect(c, paths))


def test_keep_leaves_bad_paths_alone():
    c = K.Case([6] * 8, [10] * 8, heads=(2, 2), D=64, P=16, seed=1)
    c.past[6] = -4
    c.d_past = i32(c.past)
    paths = [[0, 2, 2], [1, 0], [0, 6], [-1, 2], [0, 3], [0, 3], [0, 3], [2, 4]]
    lens = [3, 2, 2, 2, -1, 4, 2, 2]
    got = keep(c, paths, lens, width=3)
    assert np.array_equal(got, expect(c, [[]] * 7 + [[2, 4]]))
    # nodes behind the launch's tokens: the sequence is skipped
    got2 = keep(c, [[0]] * 7 + [[1]], [1] * 8, n_tokens=47)
    assert np.array_equal(got2, got)


def test_keep_with_missing_pages():
    c = K.Case([20, 20], [10, 10], heads=(2, 2), D=128, P=16, seed=2)
    c.table[0, 1] = -1          # node 6.. of the first
    c.table[1, 0] = c.n_pages   # nodes 0..5 of the second
    c.d_table = dev(c.table)
    got = keep(c, [[1, 8], [7, 9]])
    k0, v0 = O.Block(got[c.table[0, 0], 0]).load(11)
    assert np.isnan(k0).all() and (v0 == 0).all()
    before = O.Block(c.pool[c.table[0, 0], 0]).load(11)
    after = O.Block(got[c.table[0, 0], 0]).load(10)
    assert np.array_equal(before[0], after[0], equal_nan=True)
    same = c.pool.copy()
    same[c.table[0, 0]] = got[c.table[0, 0]]
    assert np.array_equal(got, same)


@pytest.mark.parametrize("D", [64, 128])
def test_keep_reads_a_token_before_its_place_is_poisoned(D):
    # four tokens move at once: the fourth has no page, and its place is the first one's token
    c = K.Case([40], [0], heads=(3, 3), D=D, P=16, seed=D)
    c.table[0, 1] = -1  # nodes 16..31
    c.d_table = dev(c.table)
    got = keep(c, [[3, 4, 5, 20, 33]])
    page, other = c.table[0, 0], c.table[0, 2]
    for h in range(c.h):
        new, old = O.Block(got[page, h]), O.Block(c.pool[page, h])
        for e, i in enumerate((3, 4, 5)):
            assert np.array_equal(new.load(e), old.load(i), equal_nan=True)
        k, v = new.load(3)
        assert np.isnan(k).all() and (v == 0).all()
        assert np.array_equal(new.load(4), O.Block(c.pool[other, h]).load(1), equal_nan=True)


# --------------------------------------------------------------------------
# the recurrence
# --------------------------------------------------------------------------

class States:
    def __init__(self, trees, H=2, dtype="f32", seed=0, slots=None, lead=0, trail=0, strong=False):
        rng = self.rng = np.random.default_rng(seed)
        self.trees, self.H, self.n = trees, H, len(trees)
        rows = [len(t) for t in trees]
        self.cu = np.concatenate([[lead], lead + np.cumsum(rows)]).astype(np.int32)
        self.T = int(self.cu[-1]) + trail
        self.up = np.full(self.T, 5000, np.int32)
        for r, t in enumerate(trees):
            self.up[self.cu[r]:self.cu[r + 1]] = t
        self.slots = 2 * self.n + 3 if slots is None else slots
        self.pool = torch.from_numpy((rng.standard_normal((self.slots, H, 128, 128)) * 0.3).astype(np.float32)).to(TYPES[dtype])
        self.init = rng.permutation(self.slots)[:self.n].astype(np.int32)
        f = lambda *s: rng.standard_normal(s).astype(np.float32)  # noqa: E731
        self.q, self.k, self.v = f(self.T, H, 128), f(self.T, H, 128), f(self.T, H, 128)
        self.g = -np.log1p(np.exp(f(self.T, H, 128))) * (8 if strong else 1)
        self.b = f(self.T, H)
        self.dtype = dtype

    def put(self):
        self.d = {n: dev(getattr(self, n)) for n in ("q", "k", "v", "g", "b", "cu", "up", "init")}
        self.d["pool"] = self.pool.cuda()
        return self

    def tree(self, out=None, scale=0.1, **kw):
        out = torch.full((self.T, self.H, 128), 7.0, device="cuda") if out is None else out
        kw.setdefault("max_nodes", max(len(t) for t in self.trees))
        d = self.d
        B.kda_decode_tree(d["pool"], d["init"], d["cu"], d["up"], d["q"], d["k"], d["v"], d["g"], d["b"], out, scale=scale, **kw)
        torch.cuda.synchronize()
        return out

    def span(self, r, way):
        """|S0[:, c]| + sum of |v_j[c]| over a path, [H, 128]."""
        S0 = host(self.pool[self.init[r]])
        return np.sqrt((S0 * S0).sum(1)) + np.abs(self.v[[self.cu[r] + j for j in way]].astype(np.float64)).sum(0)

    def check(self, out, scale=0.1, which=None):
        got = host(out)
        for r in range(self.n) if which is None else which:
            a, b = self.cu[r], self.cu[r + 1]
            want = T.recurrence(host(self.pool[self.init[r]]), self.trees[r], self.q[a:b], self.k[a:b], self.v[a:b],
                                self.g[a:b], self.b[a:b], scale)
            for i in range(b - a):
                way = T.path_to(self.trees[r], i)
                tol = 2.0 ** -23 * (128 + 16 * len(way)) * abs(scale) * self.span(r, way)
                bad = ~(np.abs(got[a + i] - want[i]) <= tol)
                assert not bad.any(), (r, i, np.abs(got[a + i] - want[i]).max(), tol.min())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("H", [1, 3])
@pytest.mark.parametrize("n", [1, 2, 7, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64])
def test_decode_tree(dtype, H, n):
    s = States([some_tree(n, n), star(n), chain(n), [], some_tree(max(1, n // 2), 3, roots=2)], H=H, dtype=dtype, seed=n, lead=2,
               trail=3).put()
    out = s.tree()
    s.check(out)
    rest = host(out)
    assert (rest[:2] == 7).all() and (rest[s.cu[-1]:] == 7).all()
    assert torch.equal(s.d["pool"].cpu(), s.pool)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("most", [12, 40])
def test_decode_tree_of_many_heads(dtype, most):
    # more than 128 requests x heads: whole heads
    s = States([some_tree(1 + (7 * r) % most, r) for r in range(23)], H=6, dtype=dtype, seed=most).put()
    s.check(s.tree())


@pytest.mark.parametrize("max_nodes", [5, 16, 17, 32, 33, 64, None])
def test_decode_tree_variants_agree(max_nodes):
    s = States([some_tree(5, 1), chain(4)], seed=4).put()
    s.check(s.tree(max_nodes=max_nodes))


@pytest.mark.parametrize("strong", [False, True])
def test_decode_tree_is_the_chained_step(strong):
    # 8 chained rows of kda_decode_step, whose states go to snapshot slots
    n = 8
    s = States([chain(n)] * 3, H=4, slots=40, seed=6, strong=strong).put()
    got = s.tree()
    s.check(got)
    pool, out = s.pool.cuda(), torch.empty(s.T, 4, 128, device="cuda")
    ids = [x for x in range(40) if x not in s.init][:24]
    d = s.d
    B.kda_decode_step(pool, i32(ids), d["q"], d["k"], d["v"], d["g"], d["b"], out, n_rows_per_slot=n, scale=0.1,
                      init_slot_ids=d["init"])
    torch.cuda.synchronize()
    s.check(out)


def test_decode_tree_shared_slots_and_bad_requests():
    s = States([some_tree(9, i) for i in range(7)], seed=7)
    s.init[:] = 2
    s.init[3], s.init[4] = -1, s.slots
    s.up[s.cu[5] + 4] = 4
    s.up[s.cu[6]] = 0
    s.put()
    out = s.tree()
    s.check(out, which=[0, 1, 2])
    assert np.isnan(host(out)[s.cu[3]:]).all()


@pytest.mark.parametrize("n,most", [(17, 16), (65, 64), (200, 64), (5, 4), (3, 0)])
def test_decode_tree_of_too_many_nodes_is_nan(n, most):
    s = States([chain(min(most, 3)), chain(n), chain(min(most, 2))], seed=8).put()
    out = s.tree(max_nodes=most)
    s.check(out, which=[0, 2])
    assert np.isnan(host(out)[s.cu[1]:s.cu[2]]).all()


def test_decode_tree_out_of_range_requests_are_skipped():
    s = States([chain(4)] * 4, seed=9)
    s.cu = np.array([-1, 4, 8, 12, 17], np.int32)  # the first starts before the rows, the last passes their end
    s.put()
    out = s.tree()
    s.check(out, which=[1, 2])
    got = host(out)
    assert (got[:4] == 7).all() and (got[12:] == 7).all()


def test_decode_tree_zero_vectors_and_gates():
    s = States([some_tree(12, 2)], seed=10)
    s.q[2], s.k[3], s.k[0] = 0, 0, 0
    s.b[4], s.b[5], s.b[6] = 200, -200, 0
    s.g[7], s.g[8] = 0, -200
    s.put()
    s.check(s.tree())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("decay", [-0.9, -1.5, -3.0, -40.0, -85.0])
def test_decode_tree_decays_to_nothing(dtype, decay):
    # products of decays down to 2^-126 and below, in every channel at once, and zero vectors
    s = States([chain(64), some_tree(30, 3)], seed=13, dtype=dtype)
    s.g[:] = decay
    s.q[70], s.k[71] = 0, 0
    s.put()
    s.check(s.tree())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_gates_at_infinity(dtype):
    # a decay of exactly zero, beta of exactly 0 and 1
    s = States([some_tree(20, 3), chain(6)], seed=12, dtype=dtype)
    s.g[3, 0], s.g[5, :, 7:90], s.g[21], s.g[8, 1, 4] = -np.inf, -np.inf, -np.inf, -np.finfo(np.float32).max
    s.b[4], s.b[22] = np.inf, -np.inf
    s.put()
    s.check(s.tree())
    paths = [list(range(20)), list(range(6))]
    check_path(s, run_path(s, paths), paths)


def test_decode_tree_a_bad_number_stays_on_its_paths():
    tree = [-1, 0, 0, 1, 2, -1, 5, 3]
    s = States([tree], seed=11)
    s.v[1, 0, 5] = np.nan
    s.put()
    got = host(s.tree())
    for i in range(8):
        bad = 1 in T.path_to(tree, i)
        assert np.isnan(got[i, 0, 5]) == bad
        assert np.isfinite(np.delete(got[i], 5, -1)).all() and np.isfinite(got[i, 1]).all()


@pytest.mark.parametrize("scale", [0.0, -2.0, 1e-30])
def test_decode_tree_scales(scale):
    s = States([some_tree(6, 2)], seed=12).put()
    s.check(s.tree(scale=scale), scale)


# --------------------------------------------------------------------------
# paths
# --------------------------------------------------------------------------

def run_path(s, paths, dst=None, lens=None, width=None):
    width = width or max(1, max(len(p) for p in paths))
    table = np.full((len(paths), width), -7, np.int32)
    for r, p in enumerate(paths):
        table[r, :len(p)] = p[:width]
    d = s.d
    pool = s.pool.cuda()
    B.kda_decode_path(pool, d["init"], d["cu"], dev(table), i32([len(p) for p in paths] if lens is None else lens), d["k"],
                      d["v"], d["g"], d["b"], dst_slot_ids=None if dst is None else i32(dst))
    torch.cuda.synchronize()
    return pool.cpu()


def check_path(s, pool, paths, dst=None, skip=()):
    want = s.pool.clone()
    to = s.init if dst is None else dst
    for r, path in enumerate(paths):
        if r in skip:
            continue
        a, b = s.cu[r], s.cu[r + 1]
        S = T.advance(host(s.pool[s.init[r]]), path, s.k[a:b], s.v[a:b], s.g[a:b], s.b[a:b])
        got = host(pool[to[r]])
        if not path:
            assert torch.equal(pool[to[r]], s.pool[s.init[r]])
        tol = 2.0 ** -23 * (128 + 16 * len(path)) * s.span(r, path)[:, None]
        tol = tol + (0 if s.dtype == "f32" else 2.0 ** -11 * (np.abs(S) + tol) + 2.0 ** -25)
        assert (np.abs(got - S) <= tol).all(), (r, np.abs(got - S).max())
        want[to[r]] = pool[to[r]]
    assert torch.equal(pool, want)  # nothing else is touched


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("H", [1, 5])
@pytest.mark.parametrize("elsewhere", [False, True])
def test_decode_path(dtype, H, elsewhere):
    s = States([some_tree(64, 1), chain(64), star(20), [], chain(17), some_tree(9, 2), chain(3)], H=H, dtype=dtype, seed=H,
               lead=1, trail=2).put()
    paths = [T.path_to(s.trees[0], 63), list(range(64)), [0, 19], [], list(range(17)), [0], []]
    dst = None
    if elsewhere:
        dst = [x for x in range(s.slots) if x not in s.init][:7]
        dst[2] = int(s.init[2])
    check_path(s, run_path(s, paths, dst), paths, dst)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_decode_path_of_many_heads(dtype):
    # more than 128 requests x heads: whole heads; every length around a block's end
    lens = [0, 1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 18, 31, 32, 33, 48, 49, 63, 64, 1, 6]
    s = States([chain(64)] * len(lens), H=6, dtype=dtype, seed=9).put()
    paths = [list(range(n)) for n in lens]
    check_path(s, run_path(s, paths), paths)


def test_decode_path_any_order_and_repeats():
    s = States([star(6), chain(5)], seed=3).put()
    paths = [[3, 1, 1, 5], [4, 0]]
    check_path(s, run_path(s, paths), paths)


def test_decode_path_skips_bad_requests():
    s = States([chain(4)] * 9, H=2, seed=4)
    s.init[3] = -1
    s.init[4] = s.slots
    s.put()
    free = [x for x in range(s.slots) if x not in s.init]
    dst = [int(x) for x in s.init]
    dst[3], dst[4], dst[5], dst[6] = free[0], free[1], -1, s.slots
    paths = [[0, 4], [0, -1], [0, 1], [0], [0], [0], [0], [0, 1], [0, 1, 2]]
    lens = [2, 2, 4, 1, 1, 1, 1, -1, 3]
    check_path(s, run_path(s, paths, dst, lens, width=3), paths, dst, skip=range(8))


def test_decode_path_without_nodes_copies():
    s = States([[], []], slots=6, seed=5).put()
    dst = [x for x in range(6) if x not in s.init][:2]
    pool = run_path(s, [[], []], dst)
    check_path(s, pool, [[], []], dst)


# --------------------------------------------------------------------------
# verification
# --------------------------------------------------------------------------

class Drafts:
    def __init__(self, trees, V, dtype="f32", draft=False, seed=0, sharp=3.0, stride=0, offset=0, lead=0, trail=0):
        rng = np.random.default_rng(seed)
        self.trees, self.n, self.V, self.dtype = trees, len(trees), V, dtype
        rows = [len(t) for t in trees]
        self.cu = np.concatenate([[lead], lead + np.cumsum(rows)]).astype(np.int32)
        N = self.T = int(self.cu[-1]) + trail
        self.up = np.full(N, 4000, np.int32)
        for r, t in enumerate(trees):
            self.up[self.cu[r]:self.cu[r + 1]] = t
        logits = rng.standard_normal((N, V)) * sharp
        soft = lambda x: np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
        self.target = self._rows(soft(logits), stride, offset)
        noisy = logits + rng.standard_normal((N, V))
        self.draft = self._rows(soft(noisy), stride, offset) if draft else None
        self.tokens = np.zeros(N, np.int32)
        for r, t in enumerate(trees):
            used = {}
            for i, p in enumerate(t):
                if p < 0:
                    continue
                row = self.cu[r] + p
                if draft:
                    w = soft(noisy)[row]
                    self.tokens[self.cu[r] + i] = rng.choice(V, p=w)
                else:
                    order = np.argsort(-noisy[row])
                    self.tokens[self.cu[r] + i] = order[min(used.get(p, 0), V - 1)]
                    used[p] = used.get(p, 0) + 1
        self.accept, self.sample = rng.random(N).astype(np.float32), rng.random(self.n).astype(np.float32)

    def _rows(self, x, stride, offset):
        """Device rows of the type, `stride` entries further apart than their length and shifted by `offset`."""
        n, V = x.shape
        flat = torch.zeros(n * (V + stride) + offset, dtype=TYPES[self.dtype], device="cuda")
        rows = flat[offset:].view(n, V + stride)[:, :V] if stride else flat[offset:].view(n, V)
        rows.copy_(torch.from_numpy(x).cuda().to(TYPES[self.dtype]))
        return rows

    def run(self, max_path=64, **kw):
        i = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")  # noqa: E731
        path, lens, nxt = i(self.n, max_path), i(self.n), i(self.n)
        B.kda_verify_drafts(self.target, dev(self.cu), dev(self.up), dev(self.tokens), dev(self.accept), dev(self.sample), path,
                            lens, nxt, draft=self.draft, **kw)
        torch.cuda.synchronize()
        return path.cpu().numpy(), lens.cpu().numpy(), nxt.cpu().numpy()

    def want(self, r, max_path=64):
        a, b = self.cu[r], self.cu[r + 1]
        if a == b:
            return [], -1
        return T.verify(host(self.target[a:b]), None if self.draft is None else host(self.draft[a:b]), self.trees[r],
                        self.tokens[a:b], self.accept[a:b], self.sample[r], max_path)

    def check(self, max_path=64, which=None, **kw):
        path, lens, nxt = self.run(max_path, **kw)
        for r in range(self.n) if which is None else which:
            way, x = self.want(r, max_path)
            assert lens[r] == len(way) and path[r, :len(way)].tolist() == way and (path[r, len(way):] == -1).all(), r
            assert nxt[r] == x, (r, nxt[r], x)
        return path, lens, nxt


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("draft", [False, True])
@pytest.mark.parametrize("V", [1, 2, 7, 64, 255, 257, 1000, 2049])
def test_verify(dtype, draft, V):
    trees = [chain(8), star(9), some_tree(64, V), some_tree(20, V + 1), [], chain(1), chain(2)] * 4
    Drafts(trees, V, dtype, draft, seed=V, sharp=2.0, lead=2, trail=1).check()


@pytest.mark.parametrize("V", [5000, 32768, 50021, 131072])
@pytest.mark.parametrize("draft", [False, True])
def test_verify_large_vocabularies(V, draft):
    trees = [chain(5), some_tree(7, 1), star(4)]
    d = Drafts(trees, V, "bf16" if draft else "f32", draft, seed=V, sharp=3.0)
    for seed in range(4):
        rng = np.random.default_rng(seed)
        d.accept, d.sample = rng.random(d.T).astype(np.float32), rng.random(d.n).astype(np.float32)
        d.check()


def test_verify_many_requests():
    trees = [chain(1 + i % 3) for i in range(1100)]
    Drafts(trees, 300, "f16", True, seed=1).check()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("stride,offset", [(0, 1), (1, 0), (3, 5), (8, 2)])
def test_verify_rows_of_any_alignment(dtype, stride, offset):
    Drafts([chain(4), some_tree(6, 1)] * 3, 4099, dtype, True, seed=stride, stride=stride, offset=offset).check()


def test_verify_the_given_numbers_at_borders():
    # all sums are exact: quarters
    d = Drafts([chain(2)] * 12, 4, "f32", False, seed=2)
    d.target.fill_(0.25)
    d.tokens[:] = 2
    d.accept[1::2] = [0.0, 0.2499999, 0.25, 0.5] * 3
    d.sample[:] = np.repeat([0.0, 0.25, 0.75], 4)
    d.check()
    path, lens, nxt = d.run()
    assert lens.tolist() == [2, 2, 1, 1] * 3
    # a refused token 2 leaves 0, 1, 3 of a quarter each; else a draw at 0, 1/4, 3/4
    assert nxt.tolist() == [0, 0, 0, 0, 1, 1, 0, 0, 3, 3, 3, 3]


def test_verify_every_draw_has_its_token():
    V = 97
    rng = np.random.default_rng(3)
    w = rng.integers(0, 3, V) / 256.0  # exact sums, with zeros
    total = w.sum()
    shares = (np.arange(300) / 300).astype(np.float32)
    d = Drafts([chain(1)] * 300, V, "f32", False, seed=3)
    d.target.copy_(torch.from_numpy(w).float().expand(300, V))
    d.sample[:] = shares
    nxt = d.check()[2]
    want = [int(np.flatnonzero((np.cumsum(w) > float(u) * total) & (w > 0))[0]) for u in shares]
    assert nxt.tolist() == want


def test_verify_rows_without_weight_and_bad_numbers():
    d = Drafts([chain(1)] * 8, 600, "f32", False, seed=4)
    x = torch.zeros(8, 600)
    x[0, 599] = 1e-30
    x[1] = float("nan")
    x[1, 77] = 0.5
    x[2] = -1
    x[3, 5] = float("inf")
    x[4, 0] = 0.5
    x[5, 300:] = 1e-38
    x[7] = float("nan")
    d.target.copy_(x)
    d.sample[:] = [0.99, 0.99, 0.5, 0.5, 0.9999, 0.0, 0.5, 0.5]
    nxt = d.run()[2]
    assert nxt.tolist() == [599, 77, -1, -1, 0, 300, -1, -1]


def test_verify_random_numbers_out_of_range():
    d = Drafts([chain(1)] * 4, 50, "f32", False, seed=5)
    d.sample[:] = [1.0, 2.0, -1.0, np.nan]
    nxt = d.run()[2]
    assert nxt.tolist() == [49, 49, 0, 49]  # every entry is above 0
    d = Drafts([chain(2)] * 3, 50, "f32", False, seed=5)
    d.accept[:] = 1.0
    d.target[::2, 7] = 2.0
    d.tokens[:] = 7
    assert d.run()[1].tolist() == [2, 2, 2]
    d.accept[1::2] = np.nan
    assert d.run()[1].tolist() == [1, 1, 1]


def test_verify_tokens_outside_the_vocabulary_are_refused():
    for draft in (False, True):
        d = Drafts([star(4), chain(3)], 40, "f32", draft, seed=6)
        d.tokens[:] = [0, -1, 40, 2 ** 31 - 1, 0, -2 ** 31, 3]
        d.accept[:] = 0
        path, lens, _ = d.check()
        assert lens.tolist() == [1, 1]


def test_verify_repeated_siblings():
    # a refused token has no weight left for the next child of the same token
    d = Drafts([star(6)] * 40, 12, "f32", False, seed=7, sharp=1.0)
    for r in range(40):
        d.tokens[d.cu[r]:d.cu[r + 1]] = [0, 3, 3, 5, 3, 5]
    d.check()
    d = Drafts([star(6)] * 40, 12, "f32", True, seed=8, sharp=1.0)
    for r in range(40):
        d.tokens[d.cu[r]:d.cu[r + 1]] = [0, 3, 3, 5, 3, 5]
    d.check()


@pytest.mark.parametrize("draft", [False, True])
def test_verify_nothing_left(draft):
    # the draft covers the target: what is left is drawn from the target's row
    d = Drafts([chain(2), star(3)] * 3, 5, "f32", draft, seed=9)
    d.target.copy_(torch.tensor([0.5, 0.0, 0.25, 0.0, 0.25]).expand(d.T, 5))
    if draft:
        d.draft.copy_(torch.tensor([0.5, 0.5, 0.25, 0.5, 0.25]).expand(d.T, 5))
        d.tokens[:] = 1
    else:
        d.target.copy_(torch.tensor([0.0, 0.0, 1.0, 0.0, 0.0]).expand(d.T, 5))
        d.tokens[:] = 2
    d.accept[:] = 0.99 if draft else 1.5
    d.check()


@pytest.mark.parametrize("most", [1, 2, 3, 7, 8, 64])
def test_verify_short_tables(most):
    d = Drafts([chain(8), star(3), chain(64)], 30, "f32", False, seed=10)
    d.accept[:] = 0.0
    path, lens, _ = d.check(most)
    assert lens.tolist() == [min(most, 8), min(most, 2), min(most, 64)]


def test_verify_bad_trees_and_ranges():
    d = Drafts([chain(3), chain(65), chain(3), chain(3), chain(3), chain(3)], 30, "f32", True, seed=11)
    d.up[d.cu[2]] = 0
    d.up[d.cu[3] + 1] = 1
    d.cu[6] = d.T + 1
    path, lens, nxt = d.check(which=[0, 4])
    for r in (1, 2, 3, 5):
        assert lens[r] == 0 and nxt[r] == -1 and (path[r] == -1).all()


def test_verify_without_nodes():
    z = lambda *s: torch.full(s, 7, dtype=torch.int32, device="cuda")  # noqa: E731
    path, lens, nxt = z(2, 3), z(2), z(2)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    B.kda_verify_drafts(torch.empty(0, 9, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda"), e, e, e.float(),
                        torch.zeros(2, device="cuda"), path, lens, nxt)
    torch.cuda.synchronize()
    assert (path == -1).all() and (lens == 0).all() and (nxt == -1).all()


def test_verify_offsets_pass_32_bits():
    V, stride, n = 500, 2 ** 30 + 8, 4
    flat = torch.empty(3 * stride + V, dtype=torch.bfloat16, device="cuda")
    rows = flat.as_strided((n, V), (stride, 1))
    d = Drafts([chain(4)], V, "bf16", False, seed=12)
    rows.copy_(d.target)
    d.target = rows
    d.accept[:] = 0
    assert d.check()[1][0] == 4
    d.accept[3] = 1.5
    d.check()


def test_verify_refuses_tensors_of_other_kinds():
    d = Drafts([chain(2)], 10, "f32", True, seed=1)
    d.draft = d.draft.half()
    with pytest.raises(TypeError):
        d.run()
    d.draft = d.target[:, :5]
    with pytest.raises(ValueError):
        d.run()
    d.draft = d.target.t().contiguous().t()
    with pytest.raises(ValueError):
        d.run()
    d.draft = None
    with pytest.raises(ValueError):
        d.run(workspace=torch.empty(1024, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(B.KdaError):
        d.run(workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(B.KdaError):
        d.run(max_path=65)
    d.target = d.target.double()
    with pytest.raises(B.KdaError):
        d.run()


# --------------------------------------------------------------------------
# graphs, streams, a whole step
# --------------------------------------------------------------------------

def calls(seed=0):
    """Every call on tensors of its own: name -> (launch, outputs)."""
    c = TreeCase([some_tree(20, 1), some_tree(9, 2)], [2100, 30], heads=(2, 2), D=64, P=16, seed=seed).fill()
    s = States([some_tree(20, 1), some_tree(9, 2)], seed=seed).put()
    d = Drafts([some_tree(20, 1), some_tree(9, 2)], 9000, "f32", True, seed=seed)
    out, read = torch.empty(c.T, 2, 64, device="cuda"), torch.empty(s.T, 2, 128, device="cuda")
    i = lambda *x: torch.zeros(x, dtype=torch.int32, device="cuda")  # noqa: E731
    path, lens, nxt = i(2, 20), i(2), i(2)
    ws = torch.empty(B.kda_kv_attend_tree_workspace(c.d_pool, c.d_table, c.T, 2, 20, 2120), dtype=torch.uint8, device="cuda")
    vs = torch.empty(B.kda_verify_workspace(2, d.T, 9000, 20), dtype=torch.uint8, device="cuda")
    t = [dev(x) for x in (d.cu, d.up, d.tokens, d.accept, d.sample)]
    e = s.d
    dst = i32([x for x in range(s.slots) if x not in s.init][:2])
    cache, ways, three, two = c.d_pool.clone(), i32([[0, 3, 7], [0, 4, 5]]), i32([3, 3]), i32([3, 2])

    def attend(**kw):
        B.kda_kv_attend_tree(c.d_pool, c.d_table, c.d_cu, c.d_past, c.d_up, c.q, out, max_rows=20, max_kv_len=2120,
                             workspace=ws, **kw)

    def tree(**kw):
        B.kda_decode_tree(e["pool"], e["init"], e["cu"], e["up"], e["q"], e["k"], e["v"], e["g"], e["b"], read, max_nodes=20,
                          **kw)

    def path_(**kw):
        B.kda_decode_path(e["pool"], e["init"], e["cu"], ways, two, e["k"], e["v"], e["g"], e["b"], dst_slot_ids=dst, **kw)

    def keep_(**kw):
        B.kda_kv_keep(cache, c.d_table, c.d_cu, c.d_past, ways, three, **kw)

    def verify(**kw):
        B.kda_verify_drafts(d.target, *t, path, lens, nxt, draft=d.draft, workspace=vs, **kw)

    return {"attend": (attend, [out]), "tree": (tree, [read]), "path": (path_, [e["pool"]]), "keep": (keep_, [cache]),
            "verify": (verify, [path, lens, nxt])}


@pytest.mark.parametrize("name", ["attend", "tree", "path", "keep", "verify"])
def test_graph_replays(name):
    launch, outs = calls(3)[name]
    launch()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        launch()
    for turn in range(4):
        if name not in ("keep", "path"):  # (those read what they write)
            for o in outs:
                o.fill_(turn)
        junk = torch.randn(1000, device="cuda").sum()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.isfinite(junk)
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_graphs_of_the_largest_trees(dtype):
    """The most nodes need the most shared memory; a first call may be a captured one."""
    s = States([some_tree(64, 1), some_tree(50, 2), chain(64)], H=3, dtype=dtype).put()
    c = TreeCase([some_tree(64, 1), some_tree(50, 2)], [2100, 30], dtype=dtype, heads=(16, 2), D=64, P=16).fill()
    read, out = torch.zeros(s.T, 3, 128, device="cuda"), torch.zeros(c.T, 16, 64, dtype=TYPES[dtype], device="cuda")
    ws = torch.empty(B.kda_kv_attend_tree_workspace(c.d_pool, c.d_table, c.T, 16, 64, 2164, dtype), dtype=torch.uint8,
                     device="cuda")
    assert ws.numel() > 0
    d = s.d
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.kda_decode_tree(d["pool"], d["init"], d["cu"], d["up"], d["q"], d["k"], d["v"], d["g"], d["b"], read, scale=0.1,
                          max_nodes=64)
        B.kda_kv_attend_tree(c.d_pool, c.d_table, c.d_cu, c.d_past, c.d_up, c.q, out, max_rows=64, max_kv_len=2164,
                             workspace=ws)
    for _ in range(3):
        read.zero_(), out.zero_(), ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        s.check(read)
        c.check(out)


@pytest.mark.parametrize("name", ["attend", "tree", "path", "keep", "verify"])
def test_other_streams(name):
    launch, outs = calls(4)[name]
    launch()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for o in outs if name not in ("keep", "path") else []:
        o.zero_()
    side.wait_stream(torch.cuda.current_stream())
    launch(stream=side)
    side.synchronize()
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


def test_workspaces_of_other_streams():
    c = TreeCase([some_tree(20, 1)], [2100], heads=(2, 2), D=64, P=16).fill()
    d = Drafts([some_tree(20, 1)] * 3, 9000, "f32", True)
    want, drafts = c.attend(), d.run()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = c.attend(stream=side)
    again = d.run(stream=side)
    assert torch.equal(got, want)
    for a, b in zip(drafts, again):
        assert np.array_equal(a, b)


@pytest.mark.parametrize("heads", [(2, 2), (8, 2)])
def test_caches_beyond_32_bits(heads):
    c = TreeCase([some_tree(20, 1), some_tree(64, 2)], [700, 300], heads=heads, D=128, P=256, seed=30).fill()
    want, path, lens = c.attend(), i32([[0, 4, 9], [1, 30, 63]]), i32([3, 3])
    n = 5 * 2 ** 30 // c.d_pool[0].numel()
    big = torch.zeros((n, *c.d_pool.shape[1:]), dtype=torch.uint8, device="cuda")
    big[-c.n_pages:] = c.d_pool
    small, small_table = c.d_pool, c.d_table
    c.d_pool, c.d_table = big, torch.where(small_table < 0, small_table, small_table + (n - c.n_pages))
    assert torch.equal(c.attend(), want)
    B.kda_kv_keep(small, small_table, c.d_cu, c.d_past, path, lens)
    B.kda_kv_keep(big, c.d_table, c.d_cu, c.d_past, path, lens)
    assert torch.equal(big[-c.n_pages:], small) and not bool(big[:-c.n_pages].any())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_pools_beyond_32_bits(dtype):
    s = States([some_tree(20, 1), some_tree(64, 2), chain(3)], H=3, dtype=dtype, seed=31).put()
    want, paths = s.tree(), [T.path_to(s.trees[0], 19), T.path_to(s.trees[1], 63), [0, 1]]
    moved = run_path(s, paths)
    n = 5 * 2 ** 30 // (s.pool[0].numel() * s.pool.element_size())
    pool = torch.zeros((n, *s.pool.shape[1:]), dtype=s.pool.dtype, device="cuda")
    pool[-s.slots:] = s.d["pool"]
    s.d["pool"], s.d["init"] = pool, s.d["init"] + (n - s.slots)
    assert torch.equal(s.tree(), want)
    table = np.zeros((3, 64), np.int32)
    for r, p in enumerate(paths):
        table[r, :len(p)] = p
    d = s.d
    B.kda_decode_path(pool, d["init"], d["cu"], dev(table), i32([len(p) for p in paths]), d["k"], d["v"], d["g"], d["b"])
    assert torch.equal(pool[-s.slots:].cpu(), moved) and not bool(pool[:-s.slots].any())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_a_whole_step(dtype):
    """A step over trees, then the accepted path's entries and states: the same as
    those of the accepted tokens alone, appended and decoded one after the other."""
    H, D, P, V, n_req = 2, 128, 16, 64, 3
    rng = np.random.default_rng(20)
    trees = [some_tree(14, 1), star(6), chain(9)]
    depth = [[len(T.path_to(t, i)) - 1 for i in range(len(t))] for t in trees]
    past = [37, 5, 60]
    c = TreeCase(trees, past, dtype="bf16", heads=(2 * H, H), D=D, P=P, seed=21)
    angle = np.arange(128)[:, None] * 100.0 ** (-np.arange(32) / 32)
    cos, sin = dev(np.cos(angle).astype(np.float32)), dev(np.sin(angle).astype(np.float32))
    for s in range(n_req):  # the context
        x = rng.standard_normal((past[s], H, D))
        O.append(c.pool, c.table[s], 0, x, rng.standard_normal(x.shape))
    c.d_pool = dev(c.pool)
    plain = c.d_pool.clone()
    pos = i32(np.concatenate([past[s] + np.array(depth[s]) for s in range(n_req)]))
    q_out, out = torch.empty_like(c.q.contiguous()), torch.empty_like(c.q.contiguous())
    B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v, q=c.q, q_out=q_out, cos=cos, sin=sin, positions=pos)
    B.kda_kv_attend_tree(c.d_pool, c.d_table, c.d_cu, c.d_past, c.d_up, q_out, out, max_rows=14, max_kv_len=80)
    s = States(trees, H=H, dtype=dtype, seed=22).put()
    read = s.tree()
    d = Drafts(trees, V, "f32", False, seed=23, sharp=4.0)
    i = lambda *x: torch.zeros(x, dtype=torch.int32, device="cuda")  # noqa: E731
    path, lens, nxt = i(n_req, 14), i(n_req), i(n_req)
    d.accept[:] *= 0.3
    B.kda_verify_drafts(d.target, c.d_cu, c.d_up, dev(d.tokens), dev(d.accept), dev(d.sample), path, lens, nxt)
    B.kda_kv_keep(c.d_pool, c.d_table, c.d_cu, c.d_past, path, lens)
    e = s.d
    B.kda_decode_path(e["pool"], e["init"], e["cu"], path, lens, e["k"], e["v"], e["g"], e["b"])
    torch.cuda.synchronize()
    ways = [path[r, :lens[r]].tolist() for r in range(n_req)]
    assert max(len(w) for w in ways) > 2
    for r in range(n_req):
        assert (ways[r], int(nxt[r])) == d.want(r)
    # the accepted tokens alone
    rows = [c.cu[r] + x for r, w in enumerate(ways) for x in w]
    cu = i32(np.concatenate([[0], np.cumsum([len(w) for w in ways])]))
    qa, oa = torch.empty_like(c.q[rows]), torch.empty_like(c.q[rows])
    B.kda_kv_append(plain, c.d_table, cu, c.d_past, c.k[rows].contiguous(), c.v[rows].contiguous(), q=c.q[rows].contiguous(),
                    q_out=qa, cos=cos, sin=sin)
    B.kda_kv_attend(plain, c.d_table, cu, c.d_past, qa, oa)
    T_kept = len(rows)
    ka, va, kb, vb = (torch.empty(T_kept, H, D, device="cuda") for _ in range(4))
    B.kda_kv_read(c.d_pool, c.d_table, cu, c.d_past, ka, va)
    B.kda_kv_read(plain, c.d_table, cu, c.d_past, kb, vb)
    torch.cuda.synchronize()
    assert torch.equal(ka, kb) and torch.equal(va, vb)
    assert torch.equal(qa, q_out[rows])
    # both forms are within the tolerance of the same 64-bit rows
    c.pool = c.d_pool.cpu().numpy()
    assert (out[rows].float() - oa.float()).abs().max() <= 4 * 2.0 ** -8 * out.float().abs().max()
    check_path(s, e["pool"].cpu(), ways)
    s.check(read)
