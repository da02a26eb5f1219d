"""GPU tests of the paged 4-bit key/value cache against the 64-bit oracle.

Tolerances, set before the first run.  Stored codes, exponents and values read
back are equal to the oracle's (a negative zero counts as zero; fp16 reads are
the exact value rounded once).  A turned query is two products and a sum in
fp32 and one rounding: |error| <= 3 * 2^-24 (|a| + |b|) + half a step.

Attention, for a row that sees T tokens, with mass = max_t sum_c |q_c k_tc| *
|scale| and top = max |v|:
 - a score is a sum of at most 3 D exact products in fp32, then two roundings,
   and the running maximum's subtraction another: its error is at most
   e = (3 D + 4) 2^-24 mass (in units of the natural exponent);
 - a weight is off by a factor of at most 1 + 2 e (e < 0.1), plus 2^-22 for
   exp2 and the maxima's ratios;
 - sums over T tokens and up to 4 waves and n splits add (T + 64) 2^-24;
 - in the value products 16-bit types round a weight w to fp16 (11 bits: half a
   step is 2^-11) for prompts: |sum (w' - w) v| <= 2^-11 top sum w; weights so
   small that fp16 holds them as subnormals, 2^-31 of the row's largest, are off
   by 2^-32 of it each, less than the T 2^-24 above.  For few rows less than
   2^-15 of a weight is dropped; the larger one is taken for both.
 - a bf16 query of a prompt, divided by its row's power of two, is rounded to a
   step of at most 2^-24 max|q|: its scores are off by 2^-25 max|q| sum|k| |scale|
   more (spread).
Numerator and denominator both carry these, each weighing at most top, so
  |error| <= top * (2 (2 e + 2^-22) + 2 (T + 64) 2^-24 + drop) + half a step.
"""
import numpy as np
import pytest

from gpu_helpers import B, need_gpu, torch
from oracle import kv_cache as O

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    return t.double().cpu().numpy()


def i32(x):
    return dev(np.asarray(x, np.int32))


class Case:
    """A step's tables and tensors: rows new tokens for each sequence, past
    ones before them; pages dealt out of order, unused entries -1."""

    def __init__(self, rows, past, dtype="f32", heads=(4, 2), D=128, P=16, seed=0, lead=0, trail=0, joint=True, spare=2):
        rng = np.random.default_rng(seed)
        self.rng, self.dtype, self.D, self.P = rng, dtype, D, P
        self.rows, self.past, self.n = list(rows), list(past), len(rows)
        self.hq, self.h = heads
        self.cu = np.concatenate([[lead], lead + np.cumsum(rows)]).astype(np.int32)
        self.T = int(self.cu[-1]) + trail
        need = [-(-(a + b) // P) for a, b in zip(rows, past)]
        self.n_pages = sum(need) + spare
        order = rng.permutation(self.n_pages)
        self.table = np.full((self.n, max(need + [1]) + 1), -1, np.int32)
        at = 0
        for s, m in enumerate(need):
            self.table[s, :m] = order[at:at + m]
            at += m
        self.pool = rng.integers(0, 256, B.kv_pool_shape(self.n_pages, self.h, P, D), dtype=np.uint8)
        x = torch.from_numpy(rng.standard_normal((self.T, self.hq + 2 * self.h, D)).astype(np.float32)).to(TYPES[dtype])
        self.x = x.cuda() if joint else None
        parts = x.split([self.hq, self.h, self.h], 1)
        self.q, self.k, self.v = (self.x if joint else x.cuda()).split([self.hq, self.h, self.h], 1)
        if not joint:
            self.q, self.k, self.v = (t.contiguous() for t in (self.q, self.k, self.v))
        self.hq_np, self.k_np, self.v_np = (host(t) for t in parts)
        self.d_pool, self.d_table, self.d_cu, self.d_past = dev(self.pool), dev(self.table), dev(self.cu), i32(past)

    def fill(self):
        """Every sequence's tokens, past ones included, stored by the oracle."""
        r = self.rng
        for s in range(self.n):
            k = r.standard_normal((self.past[s] + self.rows[s], self.h, self.D)) * (1 + 3 * (r.random(self.D) < 0.1))
            O.append(self.pool, self.table[s], 0, k, r.standard_normal(k.shape))
        self.d_pool = dev(self.pool)
        return self

    def attend(self, out=None, **kw):
        out = torch.empty(self.T, self.hq, self.D, dtype=TYPES[self.dtype], device="cuda") if out is None else out
        kw.setdefault("max_rows", max(self.rows + [0]))
        kw.setdefault("max_kv_len", max([a + b for a, b in zip(self.rows, self.past)] + [0]))
        B.kda_kv_attend(self.d_pool, self.d_table, self.d_cu, self.d_past, self.q, out, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out, scale=None, which=None):
        scale = self.D ** -0.5 if scale is None else scale
        got, drop = host(out), 0.0 if self.dtype == "f32" else 2.0 ** -11
        for s in range(self.n) if which is None else which:
            a, b, T = self.cu[s], self.cu[s + 1], self.past[s] + self.rows[s]
            if a == b:
                continue
            k, v = O.read(self.pool, self.table[s], 0, T)
            want, mass, top = O.attend(k, v, self.hq_np[a:b], self.past[s], scale)
            e = (3 * self.D + 4) * 2.0 ** -24 * mass[..., None]
            if self.dtype == "bf16":
                spread = np.abs(self.hq_np[a:b]).max(-1) * np.abs(k).sum(-1).max() * abs(scale)
                e = e + 2.0 ** -25 * spread[..., None]
            assert e.max() < 0.1
            tol = top[..., None] * (2 * (2 * e + 2.0 ** -22) + 2 * (T + 64) * 2.0 ** -24 + drop)
            tol = tol + HALF_STEP[self.dtype] * (np.abs(want) + tol) + 2.0 ** -25
            bad = ~(np.abs(got[a:b] - want) <= tol)
            # a value within the tolerance is past the type's largest: infinite
            bad &= ~(np.isinf(got[a:b]) & (np.sign(got[a:b]) * want + tol > float(torch.finfo(TYPES[self.dtype]).max)))
            assert not bad.any(), (s, np.argwhere(bad)[:5], np.abs(got[a:b] - want).max(), tol.min())


def same_cache(got, want):
    """Codes, exponents and the bytes nobody wrote; -0 counts as 0."""
    P, D = want.shape[2], want.shape[3] * 16 // 17
    def split(x):
        f = x.reshape(x.shape[0], x.shape[1], -1)
        c = np.stack([f[..., :P * D] & 15, f[..., :P * D] >> 4], -1)
        return np.where(c == 8, 0, c), f[..., P * D:]
    (gc, ge), (wc, we) = split(got), split(want)
    np.testing.assert_array_equal(ge, we)
    np.testing.assert_array_equal(gc, wc)


def angles(n, half):
    a = np.arange(n)[:, None] * 10000.0 ** (-np.arange(half) / half)
    return np.cos(a).astype(np.float32), np.sin(a).astype(np.float32)


# -- append -----------------------------------------------------------------

@pytest.mark.parametrize("dtype,D,P,heads,rot,inter,joint", [
    ("bf16", 128, 128, (8, 2), 128, False, True),
    ("bf16", 64, 16, (3, 1), 64, True, True),
    ("f16", 128, 32, (5, 5), 64, True, False),
    ("f16", 64, 64, (4, 2), 32, False, True),
    ("f32", 128, 16, (12, 12), 128, False, True),
    ("f32", 128, 256, (2, 2), 0, False, False),
    ("f32", 64, 16, (7, 7), 16, False, True),
])
def test_append_stores_what_the_definition_says(dtype, D, P, heads, rot, inter, joint):
    c = Case([1, 0, 5, 37, 8], [0, 9, P - 2, 3, 2 * P], dtype, heads, D, P, seed=3, lead=2, trail=3, joint=joint)
    cos, sin = angles(3 * P + 60, rot // 2) if rot else (None, None)
    q_out = torch.full((c.T, c.hq, D), -7.0, dtype=TYPES[dtype], device="cuda")
    B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v, q=c.q, q_out=q_out,
                    cos=None if cos is None else dev(cos), sin=None if sin is None else dev(sin), interleaved=inter)
    torch.cuda.synchronize()
    got_q = host(q_out)
    for s in range(c.n):
        a, b = c.cu[s], c.cu[s + 1]
        want = O.append(c.pool, c.table[s], c.past[s], c.k_np[a:b], c.v_np[a:b], c.hq_np[a:b], cos, sin, inter)
        size = np.abs(c.hq_np[a:b]).max(initial=0)
        tol = 3 * 2.0 ** -24 * 2 * size * (rot > 0) + HALF_STEP[dtype] * np.abs(want) * (rot > 0) + 2.0 ** -30
        assert (np.abs(got_q[a:b] - want) <= tol).all()
    same_cache(c.d_pool.cpu().numpy(), c.pool)           # and no other byte has changed
    assert (got_q[:2] == -7).all() and (got_q[c.cu[-1]:] == -7).all()   # rows outside the sequences


def test_append_without_queries_and_over_its_own_input():
    c = Case([3, 4], [5, 0], "f16", (4, 2), seed=4, joint=False)
    cos, sin = angles(40, 64)
    B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v)
    for s in range(2):
        O.append(c.pool, c.table[s], c.past[s], c.k_np[c.cu[s]:c.cu[s + 1]], c.v_np[c.cu[s]:c.cu[s + 1]])
    same_cache(c.d_pool.cpu().numpy(), c.pool)
    apart = torch.empty_like(c.q)
    args = (c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v)
    B.kda_kv_append(*args, q=c.q, q_out=apart, cos=dev(cos), sin=dev(sin))
    B.kda_kv_append(*args, q=c.q, q_out=c.q, cos=dev(cos), sin=dev(sin))
    assert torch.equal(apart, c.q)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_rounding_borders_and_extremes(dtype):
    # each row holds one kind of number at many scales; keys and values alike
    D, rows = 128, []
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, 6, 7, 0, 0.5, 1, 1.5, 2, 3, 4])
    for power in (-12, -4, 0, 3, 9):
        near = np.concatenate([ties, -ties, ties * (1 + 2.0 ** -7), ties * (1 - 2.0 ** -7)] * 2)
        rows.append(near * 2.0 ** power)
    rows.append(np.zeros(D))
    rows.append(np.full(D, -0.0))
    rows.append(np.full(D, float(torch.finfo(TYPES[dtype]).max)))
    rows.append(np.full(D, float(torch.finfo(TYPES[dtype]).tiny)))
    rows.append(np.full(D, float(torch.finfo(TYPES[dtype]).tiny) / 4))          # subnormal
    rows.append(np.where(np.arange(D) % 32 == 7, -3.0, 1e-6))
    x = torch.from_numpy(np.array(rows)).to(TYPES[dtype])
    n = x.shape[0]
    c = Case([n], [3], dtype, (1, 1), D, seed=5, joint=False)
    c.k = x.view(n, 1, D).cuda()
    c.v = x.flip(0).contiguous().view(n, 1, D).cuda()
    B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v)
    O.append(c.pool, c.table[0], 3, host(c.k), host(c.v))
    same_cache(c.d_pool.cpu().numpy(), c.pool)


def test_keys_turned_onto_rounding_borders():
    # (x, y) turned by 45 degrees in fp32's own cosine: sums next to ties
    # that fp32 arithmetic would round the other way now and then
    D, n = 64, 256
    rng = np.random.default_rng(6)
    c = Case([n], [0], "f32", (1, 1), D, seed=6, joint=False)
    cos = np.full((n, 32), np.float32(np.sqrt(0.5)))
    sin = np.full((n, 32), -np.float32(np.sqrt(0.5)))
    y = rng.choice([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0], (n, 1, 32))
    a = (y * np.sqrt(0.5)).astype(np.float32)
    b = ((y - a.astype(np.float64) * cos[0, 0]) / cos[0, 0]).astype(np.float32)  # a cos + b cos within an fp32 step of y
    c.k = dev(np.concatenate([a, b], -1).astype(np.float32))
    B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v, cos=dev(cos), sin=dev(sin))
    O.append(c.pool, c.table[0], 0, host(c.k), c.v_np, cos=cos, sin=sin)
    same_cache(c.d_pool.cpu().numpy(), c.pool)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("where", ["k", "v"])
def test_a_number_that_is_not_finite_poisons_its_token_and_head_only(where, value):
    c = Case([6, 5], [10, 17], "bf16", (4, 2), seed=7, joint=False)
    c.fill()
    getattr(c, where)[8, 1, 77] = value        # sequence 1, its third token, head 1
    B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v)
    for s in range(2):
        a, b = c.cu[s], c.cu[s + 1]
        O.append(c.pool, c.table[s], c.past[s], host(c.k)[a:b], host(c.v)[a:b])
    same_cache(c.d_pool.cpu().numpy(), c.pool)
    got = host(c.attend())
    nan = np.isnan(got)
    assert nan[8:, 2:].all()                              # rows that see it, the heads that read head 1
    nan[8:, 2:] = False
    assert not nan.any()
    c.check(torch.from_numpy(got).to(torch.bfloat16), which=[0])


def test_append_skips_tokens_without_a_place():
    c = Case([4, 4, 4, 4], [0, 14, 0, 0], "f32", (2, 1), seed=8)
    c.table[1, 1] = c.n_pages                              # its tokens 2.. have no page
    c.past[2] = -2                                         # negative position
    c.past[3] = c.table.shape[1] * 16 - 2                  # the table ends after two tokens
    c.table[3] = c.table[3, 0]
    c.d_table, c.d_past = dev(c.table), i32(c.past)
    want = c.pool.copy()
    q_out = torch.zeros(c.T, 2, 128, device="cuda")
    B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v, q=c.q, q_out=q_out)
    O.append(want, c.table[0], 0, c.k_np[0:4], c.v_np[0:4])
    O.append(want, c.table[1], 14, c.k_np[4:6], c.v_np[4:6])
    O.append(want, c.table[3], c.past[3], c.k_np[12:14], c.v_np[12:14])
    same_cache(c.d_pool.cpu().numpy(), want)
    bad = np.isnan(host(q_out)).all((1, 2))
    np.testing.assert_array_equal(bad, [False] * 4 + [False, False, True, True] + [True] * 4 + [False, False, True, True])
    # the angle table ends before the last token
    cos, sin = angles(3, 64)
    B.kda_kv_append(c.d_pool, c.d_table, i32([0, 4, 4, 4, 4]), c.d_past, c.k, c.v, q=c.q, q_out=q_out, cos=dev(cos),
                    sin=dev(sin))
    assert np.isnan(host(q_out)[3]).all() and np.isfinite(host(q_out)[:3]).all()


def test_many_short_sequences_are_found():
    for n in (1, 2, 15, 16, 17, 257, 1000):
        rng = np.random.default_rng(n)
        rows = rng.integers(0, 3, n)
        c = Case(rows.tolist(), rng.integers(0, 30, n).tolist(), "bf16", (1, 1), 64, seed=n, lead=1, trail=2)
        if c.T == 3:
            continue
        B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v)
        for s in range(n):
            a, b = c.cu[s], c.cu[s + 1]
            O.append(c.pool, c.table[s], c.past[s], c.k_np[a:b], c.v_np[a:b])
        same_cache(c.d_pool.cpu().numpy(), c.pool)


# -- read -------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,P", [(128, 64), (64, 16)])
def test_read_returns_the_stored_values(dtype, D, P):
    c = Case([1, 0, 70, 16], [P - 1, 4, 3, 0], dtype, (2, 3), D, P, seed=9, lead=1, trail=2).fill()
    wide = torch.full((c.T, 5, D), -7.0, dtype=TYPES[dtype], device="cuda")
    k, v = wide[:, :3], torch.full((c.T, 3, D), -7.0, dtype=TYPES[dtype], device="cuda")
    B.kda_kv_read(c.d_pool, c.d_table, c.d_cu, c.d_past, k, v)
    wk, wv = np.full((c.T, 3, D), -7.0), np.full((c.T, 3, D), -7.0)
    for s in range(c.n):
        a, b = c.cu[s], c.cu[s + 1]
        wk[a:b], wv[a:b] = O.read(c.pool, c.table[s], c.past[s], b - a)
    for got, want in ((k, wk), (v, wv)):
        assert torch.equal(got.cpu(), torch.from_numpy(want).to(TYPES[dtype]))
    assert bool((wide[:, 3:] == -7).all())
    only = torch.empty_like(v)
    only.fill_(-7)
    B.kda_kv_read(c.d_pool, c.d_table, c.d_cu, c.d_past, v_out=only)
    assert torch.equal(only, v)


def test_read_of_every_code_and_exponent():
    # exponents 0, 1, 253 and 254 are never stored, and not read here
    D = P = 128
    c = Case([128, 128], [0, 0], "f32", (1, 1), D, P, seed=10)
    for s in range(2):
        b = O.Block(c.pool[c.table[s, 0], 0])
        b.kc[:], b.vc[:] = np.random.default_rng(s).integers(0, 256, (2, P, D // 2))
        e = np.clip(np.arange(P) + 126 * s, 2, 252)
        b.ke[:], b.ve[:] = e[:, None], e[::-1]
    c.d_pool = dev(c.pool)
    for dtype in ("f32", "bf16", "f16"):
        k, v = (torch.empty(c.T, 1, D, dtype=TYPES[dtype], device="cuda") for _ in range(2))
        B.kda_kv_read(c.d_pool, c.d_table, c.d_cu, c.d_past, k, v)
        for s in range(2):
            want = O.read(c.pool, c.table[s], 0, 128)
            for got, w in zip((k, v), want):
                w = torch.from_numpy(w).to(torch.float32).to(TYPES[dtype])
                assert torch.equal(got[128 * s:128 * (s + 1)].cpu(), w), dtype


def test_read_without_a_page_is_nan():
    c = Case([20, 3], [0, 0], "bf16", (1, 2), seed=11).fill()
    c.table[0, 1] = -1
    c.d_table = dev(c.table)
    k = torch.zeros(c.T, 2, 128, dtype=torch.bfloat16, device="cuda")
    B.kda_kv_read(c.d_pool, c.d_table, c.d_cu, c.d_past, k_out=k)
    nan = torch.isnan(k).all(-1).all(-1).cpu().numpy()
    np.testing.assert_array_equal(np.flatnonzero(nan), [16, 17, 18, 19])
    assert not torch.isnan(k[:16]).any() and not torch.isnan(k[20:]).any()


# -- attention --------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D,P,heads,rows,past", [
    (128, 16, (4, 2), [1] * 8, [0, 1, 14, 15, 16, 31, 32, 33]),          # around one step
    (128, 128, (8, 1), [1, 0, 1, 1], [126, 40, 127, 128]),               # around a page, a sequence without rows
    (64, 16, (3, 3), [1, 1, 1], [255, 256, 900]),                        # several splits, one head each
    (64, 32, (10, 2), [8, 5, 1], [0, 300, 77]),                          # chained rows, a group of 5
    (128, 64, (16, 1), [3, 8], [200, 61]),                               # many rows of one cached head
    (128, 16, (2, 2), [40, 17, 1], [0, 5, 33]),                          # prompts
    (64, 256, (6, 2), [33, 70], [250, 0]),
    (128, 32, (8, 2), [150], [0]),
])
def test_attend_matches_the_definition(dtype, D, P, heads, rows, past):
    c = Case(rows, past, dtype, heads, D, P, seed=12, lead=1, trail=2).fill()
    out = torch.full((c.T, c.hq, D), -7.0, dtype=TYPES[dtype], device="cuda")
    c.attend(out)
    c.check(out)
    assert bool((out[:1] == -7).all()) and bool((out[c.cu[-1]:] == -7).all())


@pytest.mark.parametrize("dtype,D", [("f32", 128), ("bf16", 64), ("f16", 128)])
def test_attend_over_a_long_cache(dtype, D):
    c = Case([1, 2], [5000, 2047], dtype, (4, 2), D, 128, seed=13).fill()
    c.check(c.attend())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_the_hints_lay_out_the_launch_and_nothing_else(dtype):
    c = Case([1, 60, 8], [700, 0, 300], dtype, (4, 2), 128, 16, seed=14).fill()
    for rows, kv in ((60, 701), (1, 1), (0, 1), (1, 701), (60, 1), (5000, 0), (60, 10 ** 9), (3, 130)):
        c.check(c.attend(max_rows=rows, max_kv_len=kv))
    c.check(c.attend(max_rows=None))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,past,power", [([1, 2], [300, 4097], 0), ([1] * 3, [3000] * 3, 0), ([300, 40], [0, 2500], 0),
                                             ([300, 40], [0, 2500], 20)])
def test_outputs_over_the_queries(dtype, rows, past, power):
    # one split and several, prompts that start again in bf16 pieces
    c = Case(rows, past, dtype, (8, 4), 128, 32, seed=33, joint=False)
    for s in range(c.n):
        k = c.rng.standard_normal((past[s] + rows[s], 4, 128))
        O.append(c.pool, c.table[s], 0, k, c.rng.standard_normal(k.shape) * 2.0 ** power)
    c.d_pool = dev(c.pool)
    want = c.attend()
    assert torch.equal(c.attend(c.q), want)
    c.check(want)


def test_a_prompt_among_many_steps():
    # tiles of a launch with a long prompt between single tokens, sequences
    # without rows, and spare rows at both ends
    rows = [1, 0, 1, 1, 300, 1, 0, 0, 5, 1, 129, 1] + [1] * 70 + [0, 33]
    past = [(37 * i) % 90 for i in range(len(rows))]
    c = Case(rows, past, "f16", (6, 2), 64, 32, seed=30, lead=3, trail=40).fill()
    out = torch.full((c.T, 6, 64), -7.0, dtype=torch.float16, device="cuda")
    c.attend(out)
    c.check(out)
    assert bool((out[:3] == -7).all()) and bool((out[c.cu[-1]:] == -7).all())
    c.attend(out, max_rows=0)       # the same rows in small tiles
    c.check(out)


@pytest.mark.parametrize("scale", [1.0, 0.0, -0.3])
def test_any_scale(scale):
    c = Case([2, 20], [50, 3], "f16", (4, 1), 64, 16, seed=15).fill()
    c.check(c.attend(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [2, 80])
def test_a_scale_near_the_largest_number(dtype, rows):
    # scores of zero stay zero
    c = Case([rows], [50], dtype, (2, 1), 64, 16, seed=31)
    O.append(c.pool, c.table[0], 0, np.zeros((50 + rows, 1, 64)), c.rng.standard_normal((50 + rows, 1, 64)))
    c.d_pool = dev(c.pool)
    c.check(c.attend(scale=3.3e38), scale=0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [2, 80])
@pytest.mark.parametrize("scale", [0.0, 1e-43])
def test_a_scale_of_nothing_over_the_largest_scores(dtype, rows, scale):
    # scores of up to 3 * 2^125: times 0 they are 0, times 1e-43 below 2^-15
    c = Case([rows], [50], dtype, (2, 1), 64, 16, seed=39, joint=False)
    k = np.zeros((50 + rows, 1, 64))
    k[:, 0, 0] = np.arange(50 + rows) % 7 - 3
    O.append(c.pool, c.table[0], 0, k, c.rng.standard_normal(k.shape))
    c.d_pool = dev(c.pool)
    c.q.zero_()
    c.q[:, :, 0] = 2.0 ** 125
    c.hq_np = host(c.q)
    c.check(c.attend(scale=scale), scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows,past", [(2, 50), (80, 50), (2, 3000), (80, 3000)])
@pytest.mark.parametrize("what", ["largest", "all", "query"])
def test_rows_whose_largest_score_is_infinite_are_nan(dtype, rows, past, what):
    # a key whose score passes the largest fp32 in the middle of the new rows;
    # all scores below the lowest; a query with an infinity over keys that make
    # every score minus infinity.  Other scores are 0: rows before are the mean.
    c = Case([rows], [past], dtype, (2, 1), 64, 16, seed=34, joint=False)
    k = np.zeros((past + rows, 1, 64))
    first = past + rows // 2 if what == "largest" else 0    # the first token of which a row becomes NaN
    k[first if what == "largest" else slice(0, None)] = 1.0 if what == "largest" else -1.0
    O.append(c.pool, c.table[0], 0, k, c.rng.standard_normal(k.shape))
    c.d_pool = dev(c.pool)
    c.q = torch.ones_like(c.q)
    if what == "query":
        c.q[:, :, 5] = float("inf")
    got = c.attend(scale=3.3e38 if what != "query" else 0.125)
    sees = past + np.arange(rows) >= first
    np.testing.assert_array_equal(np.isnan(host(got)).all((1, 2)), sees)
    assert not np.isnan(host(got)[~sees]).any()
    c.rows, c.cu = [int((~sees).sum())], np.array([0, (~sees).sum()])
    c.hq_np = np.zeros_like(c.hq_np)
    c.check(got, scale=0.0)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [1, 50])
def test_strong_scores(dtype, rows):
    # one key far above the others, then one above that: the running maximum
    # moves, and early weights fall below fp32's smallest
    c = Case([rows], [600], dtype, (2, 1), 128, 16, seed=16).fill()
    k, v = O.read(c.pool, c.table[0], 0, 600 + rows)
    k[100] = 40.0 * np.sign(c.hq_np[0, 0])
    k[500] = 80.0 * np.sign(c.hq_np[0, 0])
    k[599] = -80.0 * np.sign(c.hq_np[0, 0])
    O.append(c.pool, c.table[0], 0, k, v)
    c.d_pool = dev(c.pool)
    scale = 128 ** -0.5
    got = host(c.attend())
    want, _, _ = O.attend(k_v := O.read(c.pool, c.table[0], 0, 600 + rows)[0], O.read(c.pool, c.table[0], 0, 600 + rows)[1],
                          c.hq_np, 600, scale)
    assert np.isfinite(got).all() and k_v.shape[0] == 600 + rows
    # mass is about 80 * sum|q| / sqrt(128) < 1000: a weight is off by at most 2 (3 * 128 + 4) 2^-24 * 1000 = 0.047
    assert np.abs(got - want).max() <= 2 * 0.047 * np.abs(v).max() + HALF_STEP[dtype] * np.abs(want).max()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_bytes_behind_a_sequence_end_do_not_matter(dtype):
    c = Case([1, 9, 37], [20, 30, 0], dtype, (4, 2), 128, 64, seed=17).fill()
    first = c.attend().clone()
    for s in range(c.n):
        end = c.past[s] + c.rows[s]
        for p in range(end, -(-end // 64) * 64):
            for h in range(2):
                b = O.Block(c.pool[c.table[s, p // 64], h])
                b.kc[p % 64], b.vc[p % 64], b.ke[p % 64], b.ve[:, p % 64] = 255, 255, 255, 255
    c.d_pool = dev(c.pool)
    assert torch.equal(first, c.attend())


@pytest.mark.parametrize("rows", [40, 8])
def test_a_missing_page_is_nan_for_the_rows_that_see_it(rows):
    c = Case([rows, 2], [30, 3], "bf16", (4, 2), 128, 16, seed=18).fill()
    page = (30 + rows) // 16 - 1 if rows == 40 else 2
    c.table[0, page] = c.n_pages + 5
    c.d_table = dev(c.table)
    got = host(c.attend())
    sees = 30 + np.arange(rows) >= 16 * page
    np.testing.assert_array_equal(np.isnan(got[:rows]).all((1, 2)), sees)
    np.testing.assert_array_equal(np.isnan(got[:rows]).any((1, 2)), sees)
    assert not np.isnan(got[rows:]).any()


def test_bad_tables():
    c = Case([2, 2, 2, 2], [10, 10, 10, 10], "f32", (2, 2), seed=19).fill()
    good = c.attend().clone()
    past = i32([10, -1, c.table.shape[1] * 16 - 1, 10])
    out = torch.full_like(good, -7.0)
    B.kda_kv_attend(c.d_pool, c.d_table, c.d_cu, past, c.q, out)
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[6:], good[6:])
    assert bool(torch.isnan(out[2:6]).all())
    # sequences whose token range leaves the tensors, or descends, are left alone
    for cu, skipped in (([0, 2, 4, 6, 9], [3]), ([-1, 2, 4, 6, 8], [0]), ([0, 2, 4, 8, 6], [3])):
        out.fill_(-7.0)
        B.kda_kv_attend(c.d_pool, c.d_table, i32(cu), i32([10, 10, 8, 10]), c.q, out)
        torch.cuda.synchronize()
        assert not torch.isnan(out).any()
        for s in range(4):
            kept = bool((out[2 * s:2 * s + 2] == -7).all())
            assert kept == (s in skipped and not (s == 3 and cu[3] == 8)), (cu, s)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("which,power", [("k", -30), ("v", -30), ("v", 40), ("k", 20), ("v", -115), ("both", -20)])
def test_exponents_that_fp16_does_not_hold(dtype, D, which, power):
    # some tokens' groups leave 2^-24 .. 49152, in one tile of a prompt or in
    # all; queries shrink with large keys, so that scores stay moderate
    c = Case([150, 2], [90, 200], dtype, (4, 2), D, 16, seed=27, joint=False)
    small = 2.0 ** (-power if which == "k" and power > 0 else 0)
    c.q = (c.q.float() * small).to(c.q.dtype)
    c.hq_np = host(c.q)
    r = c.rng
    for s in range(2):
        n = c.past[s] + c.rows[s]
        k, v = r.standard_normal((n, 2, D)), r.standard_normal((n, 2, D))
        far = slice(100, 104) if s == 0 else slice(0, n)
        if which in ("k", "both"):
            k[far, :, :32] *= 2.0 ** power
        if which in ("v", "both"):
            v[far, :, 32:] *= 2.0 ** power
        O.append(c.pool, c.table[s], 0, k, v)
    c.d_pool = dev(c.pool)
    c.check(c.attend())


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_prompts_over_zeros_and_poison(dtype):
    # rows of zeros (exponent 2) are ordinary; a poisoned token makes the rows
    # that see it NaN in its head, and no others
    c = Case([200], [20], dtype, (4, 2), 64, 32, seed=28, joint=False).fill()
    O.append(c.pool, c.table[0], 50, np.zeros((3, 2, 64)), np.zeros((3, 2, 64)))
    c.d_pool = dev(c.pool)
    c.check(c.attend())
    clean = c.attend().clone()
    bad = np.ones((1, 2, 64))
    bad[0, 1, 5] = np.inf
    O.append(c.pool, c.table[0], 130, bad, np.ones((1, 2, 64)))
    c.d_pool = dev(c.pool)
    got = host(c.attend())
    nan = np.isnan(got)
    assert nan[110:, 2:].all() and not nan[:110].any() and not nan[:, :2].any()
    k, v = (x[:, :1] for x in O.read(c.pool, c.table[0], 0, 220))      # the other head, as before
    want, _, top = O.attend(k, v, c.hq_np[:, :2], 20, 64 ** -0.5)
    assert (np.abs(got[:, :2] - want) <= 2.0 ** -8 * (top[..., None] + np.abs(want))).all()
    assert (np.abs(got[:110, 2:] - host(clean)[:110, 2:]) <= 2.0 ** -7).all()


@pytest.mark.parametrize("dtype,D", [("f16", 64), ("bf16", 128)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("past,at", [(0, 0), (0, 63), (0, 64), (0, 127), (100, 140), (100, 192), (100, 220), (100, 299),
                                     (1500, 0), (1500, 1023), (1500, 1088), (1500, 1540), (1500, 1620), (1500, 1699)])
def test_one_far_exponent_anywhere_in_a_prompt(dtype, D, which, past, at):
    # a single group that fp16 does not hold, in any tile of a split: the block
    # goes on in bf16 pieces from its pair of tiles on, and rows that see nothing
    # of that keep their bits (scores are too small to move a maximum after a
    # first tile)
    rows = 200
    c = Case([rows], [past], dtype, (2, 2), D, 64, seed=36, joint=False)
    c.q *= 2.0 ** -6
    c.hq_np = host(c.q)
    r, n = c.rng, past + rows
    k, v = r.standard_normal((n, 2, D)), r.standard_normal((n, 2, D))
    O.append(c.pool, c.table[0], 0, k, v)
    c.d_pool = dev(c.pool)
    clean = c.attend().clone()
    c.check(clean)
    (k if which == "k" else v)[at, 1, 32:64] *= 2.0 ** -30
    O.append(c.pool, c.table[0], 0, k, v)
    c.d_pool = dev(c.pool)
    got = c.attend()
    c.check(got)
    keep = max(at // 128 * 128 - past, 0)
    assert torch.equal(got[:keep], clean[:keep])
    assert torch.equal(got[:, :1], clean[:, :1])        # the other head's


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [8, 200])
@pytest.mark.parametrize("how", ["poison", "page"])
def test_rows_before_a_poisoned_token_keep_their_bits(dtype, rows, how):
    # scores so small that the running maximum moves in the first tile alone:
    # then nothing of a row depends on its tile's other rows
    past = 130
    c = Case([rows], [past], dtype, (4, 2), 64, 16, seed=35, joint=False).fill()
    c.q *= 2.0 ** -6
    clean = c.attend().clone()
    at = past + (5 if rows == 8 else 110)
    if how == "poison":
        O.append(c.pool, c.table[0], at, np.full((1, 2, 64), np.inf), np.ones((1, 2, 64)))
    else:
        at = at // 16 * 16
        c.table[0, at // 16] = c.n_pages
    c.d_pool, c.d_table = dev(c.pool), dev(c.table)
    got = c.attend()
    keep = max(at - past, 0)
    assert torch.equal(got[:keep], clean[:keep])
    assert bool(got[keep:].isnan().all())


@pytest.mark.parametrize("power", [-120, -60, -10, 10, 60])
def test_queries_of_any_size(power):
    # bf16 queries far outside fp16's range, keys inside: scores tiny or, with
    # a scale to match, ordinary
    c = Case([130], [70], "bf16", (2, 1), 128, 16, seed=29, joint=False).fill()
    c.q = (c.q.float() * 2.0 ** power).to(torch.bfloat16)
    c.q[7] = 0
    c.hq_np = host(c.q)
    scale = 128 ** -0.5 * 2.0 ** -power
    c.check(c.attend(scale=scale), scale=scale)
    if power < 0:
        c.check(c.attend())


@pytest.mark.parametrize("rows,far", [(8, False), (100, False), (100, True)])
def test_errors_lean_to_neither_side(rows, far):
    # The part of the error that goes with the result, over some 300,000 fp16
    # outputs.  Each is rounded to half a step, to either side alike, which gives
    # the slope a variance of sum step^2 want^2 / 12 / (sum want^2)^2, its root some
    # 1e-6.  Weights cut to 16 bits instead of rounded lean by 2^-17 = 8e-6.
    # A prompt whose weights p_t are rounded to fp16, by up to 2^-11 of each to either
    # side, gets sum_t p_t d_t (v_t - out) more: along out, and summed over rows and
    # heads, a variance of 2^-22 / 3 sum p_t^2 (v_t . out - out . out)^2 / (sum want^2)^2.
    n = 24 if rows == 8 else 2
    c = Case([rows] * n, [300] * n, "f16", (12, 12), 128, 16, seed=37, joint=False).fill()
    if far:  # a group that fp16 does not hold, in the first tile
        for s in range(n):
            k, v = O.read(c.pool, c.table[s], 0, 3)
            O.append(c.pool, c.table[s], 0, k, v * 2.0 ** -30)
        c.d_pool = dev(c.pool)
    got, err, want, weights = host(c.attend()), [], [], 0.0
    for s in range(n):
        k, v = O.read(c.pool, c.table[s], 0, 300 + rows)
        q = c.hq_np[s * rows:(s + 1) * rows]
        want.append(O.attend(k, v, q, 300, 128 ** -0.5)[0])
        err.append(got[s * rows:(s + 1) * rows] - want[-1])
        if rows == 100 and not far:
            p = np.matmul(q.transpose(1, 0, 2), k.transpose(1, 2, 0)) * 128 ** -0.5      # [heads, rows, tokens]
            p = np.where(np.arange(300 + rows) <= 300 + np.arange(rows)[:, None], p, -np.inf)
            p = np.exp(p - p.max(-1, keepdims=True))
            p /= p.sum(-1, keepdims=True)
            out = want[-1].transpose(1, 0, 2)
            along = np.matmul(out, v.transpose(1, 2, 0)) - (out ** 2).sum(-1, keepdims=True)
            weights += (p ** 2 * along ** 2).sum() * 2.0 ** -22 / 3
    want, err = np.concatenate(want), np.concatenate(err)
    step = np.exp2(np.maximum(np.floor(np.log2(np.abs(want) + 1e-30)), -14) - 10)
    sd = np.sqrt((step ** 2 * want ** 2).sum() / 12 + weights) / (want ** 2).sum()
    assert rows == 100 and not far or 5 * sd < 2.0 ** -17      # else the cut would not show
    assert abs((err * want).sum() / (want ** 2).sum()) <= 5 * sd


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,past", [(8, 900), (200, 0), (200, 900), (200, 3000)])
@pytest.mark.parametrize("what", ["equal scores", "random"])
def test_equal_values_come_out_as_they_are(dtype, rows, past, what):
    # All values are 1.  Both sums take the same weights (few rows: to 2^-16 of
    # them), so their quotient is 1 within (T + 64) 2^-24 + 2^-23 + 2^-16, T the tokens:
    # less than the 2^-12 to fp16's next border below 1 for T < 3500.
    # Equal scores: behind a first tile of 64 tokens, weights of 2^14 (1 + 0.45 2^-10),
    # which all lose 0.45 2^-10 when rounded to fp16, nearly a step of the output.
    c = Case([rows], [past], dtype, (2, 1), 64, 16, seed=38, joint=False).fill()
    k, _ = O.read(c.pool, c.table[0], 0, past + rows)
    scale = 0.125
    if what == "equal scores":
        c.q.zero_()
        c.q[:, :, 0] = 1
        k[:] = 0
        k[64:, :, 0] = 1
        scale = (7 + np.log2(1 + 0.45 / 1024)) * np.log(2)
    O.append(c.pool, c.table[0], 0, k, np.ones_like(k))
    c.d_pool = dev(c.pool)
    assert bool((c.attend(scale=scale) == 1).all())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows", [4, 80])
@pytest.mark.parametrize("first", [0.0, 1.0])
def test_many_weights_far_below_the_largest(dtype, rows, first):
    # One token, and 60,000 of 2^-22.5 of its weight in the same split (a prompt's
    # fp16 holds them as subnormals, 362 of 2^-24 for 362.04).  With values 1 but for
    # the first, which is 0 or 1, the result is S / (1 + S), S = 0.0101 (T 2^-22.5), or
    # 1: off by 2^-13 of S, half a step of the output (2^-8 at most) and, of sums over
    # T equal terms in fp32, T 2^-24 of S or of 1 at most.
    past = 60000
    c = Case([rows], [past], dtype, (2, 1), 64, 256, seed=40, joint=False)
    pool, one = c.d_pool, torch.zeros((past + rows, 1, 64), dtype=torch.float32, device="cuda")
    k, v = one.clone(), one + 1
    k[0, 0, 0], v[0] = 1, first
    B.kda_kv_append(pool, c.d_table, i32([0, past + rows]), i32([0]), k, v)
    c.q.zero_()
    c.q[:, :, 0] = 1
    got = host(c.attend(max_kv_len=64, scale=22.5 * np.log(2)))
    s = (past + np.arange(rows))[:, None, None] * 2.0 ** -22.5
    want = (first + s) / (1 + s)
    off = 2.0 ** -13 + 60100 * 2.0 ** -24
    assert (np.abs(got - want) <= (off * s if first == 0 else off) + HALF_STEP[dtype] * want).all()


@pytest.mark.parametrize("rows,past", [([1, 1, 1], [3000, 10, 555]), ([200, 8], [0, 900])])
def test_equal_calls_give_equal_bits(rows, past):
    c = Case(rows, past, "bf16", (8, 2), 128, 64, seed=20).fill()
    first = c.attend().clone()
    for _ in range(3):
        assert torch.equal(first, c.attend())


# -- how programs use them ---------------------------------------------------

def test_offsets_past_32_bits():
    # 5.2 GB of pages, the sequence on the last ones; queries 2^31 elements in
    n_pages = 100_000
    pool = torch.empty(B.kv_pool_shape(n_pages, 12, 32, 128), dtype=torch.uint8, device="cuda")
    assert pool.numel() > 1 << 32
    c = Case([5], [70], "bf16", (12, 12), 128, 32, seed=21).fill()
    last = torch.arange(n_pages - c.n_pages, n_pages, device="cuda")
    pool[last] = c.d_pool
    big = torch.empty((6, (1 << 29) + 8), dtype=torch.bfloat16, device="cuda")  # token stride 2^29: 5 tokens pass 2^31
    q = big[1:, :12 * 128].view(5, 12, 128)
    q.copy_(c.q)
    table = torch.where(c.d_table >= 0, c.d_table + (n_pages - c.n_pages), -1).to(torch.int32)
    out = torch.empty((5, 12, 128), dtype=torch.bfloat16, device="cuda")
    B.kda_kv_attend(pool, table, c.d_cu, c.d_past, q, out, max_rows=5, max_kv_len=75)
    assert torch.equal(out, c.attend())
    k, v = (torch.empty((5, 12, 128), device="cuda") for _ in range(2))
    B.kda_kv_append(pool, table, c.d_cu, c.d_past, c.k, c.v)
    B.kda_kv_read(pool, table, c.d_cu, c.d_past, k, v)
    O.append(c.pool, c.table[0], 70, c.k_np, c.v_np)
    for got, want in zip((k, v), O.read(c.pool, c.table[0], 70, 5)):
        np.testing.assert_array_equal(host(got), want)


@pytest.mark.parametrize("rows", [1, 80])
def test_the_last_positions(rows):
    # all of 2^31 - 4096 positions on one page of 256 equal tokens: the mean of
    # 1.5, over sums that fp32 holds exactly but for the join of the splits
    n = (1 << 31) - 4096
    c = Case([256], [0], "bf16", (1, 1), 64, 256, seed=32)
    O.append(c.pool, c.table[0], 0, np.zeros((256, 1, 64)), np.full((256, 1, 64), 1.5))
    pool = dev(c.pool)
    table = torch.full((1, n // 256), int(c.table[0, 0]), dtype=torch.int32, device="cuda")
    q = torch.ones((rows, 1, 64), dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    B.kda_kv_attend(pool, table, i32([0, rows]), i32([n - rows]), q, out, max_rows=rows)
    torch.cuda.synchronize()
    assert float((out.float() - 1.5).abs().max()) <= 2.0 ** -7  # a step of bf16
    k, v = (torch.zeros((rows, 1, 64), device="cuda") for _ in range(2))
    B.kda_kv_read(pool, table, i32([0, rows]), i32([n - rows]), k, v)
    assert bool((v == 1.5).all())
    B.kda_kv_append(pool, table, i32([0, rows]), i32([n - rows]), q, q)
    B.kda_kv_read(pool, table, i32([0, rows]), i32([n - rows]), k, v)
    assert bool((k == 1).all()) and bool((v == 1).all())
    B.kda_kv_attend(pool, table, i32([0, rows]), i32([n - rows + 1]), q, out, max_rows=rows)
    assert bool(out.isnan().all())  # one position too many


def test_other_streams_and_own_workspaces():
    c = Case([1, 1, 8], [2000, 100, 900], "f32", (4, 2), 64, 16, seed=22).fill()
    want = c.attend().clone()
    n = B.kda_kv_attend_workspace(c.d_pool, c.d_table, c.T, 4, 8, 2001, "f32")
    assert n > 0
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs, works = [], []
    for i, st in enumerate(streams):            # three calls in flight at once
        st.wait_stream(torch.cuda.current_stream())
        outs.append(torch.zeros_like(want))
        works.append(torch.empty(n, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    for st, o, w in zip(streams, outs, works):
        B.kda_kv_attend(c.d_pool, c.d_table, c.d_cu, c.d_past, c.q, o, max_rows=8, max_kv_len=2001, workspace=w,
                        stream=st)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, want)
    # a workspace of the library's choosing on a stream that is not the current one
    o = torch.zeros_like(want)
    torch.cuda.synchronize()
    B.kda_kv_attend(c.d_pool, c.d_table, c.d_cu, c.d_past, c.q, o, max_rows=8, max_kv_len=2001, stream=streams[0])
    torch.cuda.synchronize()
    assert torch.equal(o, want)
    with pytest.raises(B.KdaError):
        B.kda_kv_attend(c.d_pool, c.d_table, c.d_cu, c.d_past, c.q, o, max_rows=8, max_kv_len=2001,
                        workspace=works[0][:-16])


def test_replayed_graphs_follow_their_tables():
    # one graph holds a step: append, then attention; the tables' contents
    # move on between replays, with eager work of the same kind in between
    c = Case([1, 8, 1], [40, 33, 90], "bf16", (8, 2), 128, 16, seed=23, joint=False).fill()
    cos, sin = (dev(a) for a in angles(400, 64))
    c.table = np.arange(3 * 20, dtype=np.int32).reshape(3, 20)
    c.pool = np.zeros(B.kv_pool_shape(60, 2, 16, 128), np.uint8)
    for s in range(3):
        k = c.rng.standard_normal((c.past[s], 2, 128))
        O.append(c.pool, c.table[s], 0, k, c.rng.standard_normal(k.shape))
    pool, table, lens = dev(c.pool), dev(c.table), i32(c.past)
    q_out, out = torch.empty_like(c.q), torch.empty_like(c.q)

    def step(pool, lens, q_out, out):
        B.kda_kv_append(pool, table, c.d_cu, lens, c.k, c.v, q=c.q, q_out=q_out, cos=cos, sin=sin)
        B.kda_kv_attend(pool, table, c.d_cu, lens, q_out, out, max_rows=8, max_kv_len=320)

    step(pool.clone(), lens, q_out, out)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):                     # two graphs of the same step
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(pool, lens, q_out, out)
        graphs.append(g)
    eager, e_lens = pool.clone(), lens.clone()
    e_q, e_out = torch.empty_like(q_out), torch.empty_like(out)
    grow = i32(c.rows)
    for i in range(6):
        c.k.normal_()
        c.v.normal_()
        c.q.normal_()
        graphs[i % 2].replay()
        step(eager, e_lens, e_q, e_out)
        torch.cuda.synchronize()
        assert torch.equal(out, e_out) and torch.equal(q_out, e_q) and torch.equal(pool, eager), i
        lens += grow
        e_lens += grow


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_prompt_in_pieces_then_steps(dtype):
    """A prompt appended and attended in two pieces, single tokens after it,
    then a verify step of 1 + 7 rows that is taken back and repeated: each
    against the oracle over the cache as it stands."""
    D, P, heads = 64, 16, (6, 2)
    runs = [[70, 33], [25, 1], [1, 1], [1, 1], [8, 8], [8, 8], [1, 1]]
    keep = [1, 1, 1, 1, 0, 1, 1]            # the first verify step is rejected whole
    total = [sum(r[s] for r, k in zip(runs, keep) if k) + 8 for s in range(2)]
    cos, sin = angles(max(total), 16)
    whole = Case([0, 0], total, dtype, heads, D, P, seed=24)
    pool, table = np.zeros_like(whole.pool), whole.table
    d_pool = torch.zeros_like(whole.d_pool)
    past = [0, 0]
    for i, rows in enumerate(runs):
        c = Case(rows, past, dtype, heads, D, P, seed=100 + i)
        c.pool, c.table, c.d_pool, c.d_table = pool, table, d_pool, dev(table)
        q_out = torch.empty((c.T, c.hq, D), dtype=TYPES[dtype], device="cuda")
        B.kda_kv_append(d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v, q=c.q, q_out=q_out, cos=dev(cos), sin=dev(sin))
        for s in range(2):
            a, b = c.cu[s], c.cu[s + 1]
            O.append(pool, table[s], past[s], c.k_np[a:b], c.v_np[a:b], None, cos, sin)
        same_cache(d_pool.cpu().numpy(), pool)
        c.q, c.hq_np = q_out, host(q_out)
        c.check(c.attend())
        if keep[i]:
            past = [a + b for a, b in zip(past, rows)]


def test_a_hybrid_step_with_the_kda_layers():
    """A linear-attention layer and a cached-attention layer in turn, as a
    hybrid model steps them: the KDA decode's output rows go on as the next
    layer's queries on the same stream, without a copy in between."""
    H, n = 4, 3
    g = torch.Generator(device="cuda").manual_seed(25)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    state = 0.1 * rnd(n, H, 128, 128)
    ids = torch.arange(n, dtype=torch.int32, device="cuda")
    c = Case([1] * n, [20, 0, 63], "f32", (H, 2), 128, 16, seed=25).fill()
    kda_out = torch.empty(n, H, 128, device="cuda")
    out = torch.empty_like(kda_out)
    start = state.clone()
    x = [rnd(n, H, 128) for _ in range(4)] + [rnd(n, H)]
    B.kda_decode_step(state, ids, x[0], x[1], x[2], -x[3].abs(), x[4], kda_out)
    B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v)
    B.kda_kv_attend(c.d_pool, c.d_table, c.d_cu, c.d_past, kda_out, out, max_rows=1, max_kv_len=64)
    torch.cuda.synchronize()
    assert not torch.equal(state, start)
    for s in range(n):
        O.append(c.pool, c.table[s], c.past[s], c.k_np[s:s + 1], c.v_np[s:s + 1])
    c.q, c.hq_np = kda_out, host(kda_out)
    c.check(out)


def test_the_binding_checks_its_tensors():
    c = Case([2], [3], "f32", (2, 1), seed=26)
    out = torch.empty(2, 2, 128, device="cuda")
    call = lambda **o: B.kda_kv_attend(o.get("pool", c.d_pool), o.get("table", c.d_table), o.get("cu", c.d_cu),  # noqa: E731
                                       o.get("lens", c.d_past), o.get("q", c.q), o.get("out", out))
    call()
    for bad in (dict(pool=c.d_pool.int()), dict(pool=c.d_pool[:, :, :8]), dict(table=c.d_table.long()),
                dict(cu=c.d_cu[:1]), dict(lens=c.d_past.repeat(2)), dict(q=c.q.half()), dict(q=c.q[:, :, ::2]),
                dict(out=out[:1]), dict(out=out.double()), dict(table=c.d_table[0]), dict(q=c.q.transpose(0, 1)),
                dict(out=torch.empty(2, 3, 128, device="cuda")[:, :2])):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    with pytest.raises(ValueError):
        B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v, q=c.q)
    with pytest.raises(ValueError):
        B.kda_kv_append(c.d_pool, c.d_table, c.d_cu, c.d_past, c.k, c.v, cos=torch.zeros(9, 16, device="cuda"))
    with pytest.raises(B.KdaError):
        B.kda_kv_attend(c.d_pool, c.d_table, c.d_cu, c.d_past, c.q[:, :1].repeat(1, 1, 1).double(), out.double()[:, :1].contiguous())
    with pytest.raises(ValueError):
        B.kda_kv_read(c.d_pool, c.d_table, c.d_cu, c.d_past)
    torch.cuda.synchronize()
