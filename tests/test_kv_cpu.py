"""The paged 4-bit key/value cache without a GPU: the 64-bit oracle's pins
(format, rotation, attention), the refusals of the entry points, the host
checks of tables, sizes and workspaces."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from oracle import kv_cache as O

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
K = pytest.importorskip("kda_gated_delta_decode_amd")
from kda_gated_delta_decode_amd import binding as B  # noqa: E402

FAKE = 0x10000  # never dereferenced: the calls are refused on the host


# -- the oracle's pins ------------------------------------------------------

def test_every_code_reads_as_its_value():
    codes = np.arange(16, dtype=np.uint8).repeat(2)
    x = O.decode(codes, np.array([127 + 3], np.uint8))
    want = [0, .5, 1, 1.5, 2, 3, 4, 6]
    np.testing.assert_array_equal(x[::2], 8.0 * np.array(want + [-w for w in want]))


def test_every_value_is_its_own_encoding():
    x = np.zeros(32)
    x[:16] = O.decode(np.arange(16, dtype=np.uint8).repeat(2), np.array([127], np.uint8))[::2]
    for power in (-100, -3, 0, 5, 100):
        c, e = O.encode(x * 2.0 ** power)
        assert e[0] == 127 + power
        np.testing.assert_array_equal(O.decode(c, e), x * 2.0 ** power)


@pytest.mark.parametrize("value,code", [(0.25, 0), (0.2500001, 1), (0.75, 2), (0.7499999, 1), (1.25, 2), (1.75, 4),
                                        (2.5, 4), (2.51, 5), (3.5, 6), (5.0, 6), (5.01, 7), (7.9, 7)])
def test_rounding_is_to_nearest_with_ties_to_even(value, code):
    x = np.zeros(32)
    x[0], x[1] = 4.0, value  # a largest magnitude in [4, 8) makes the unit 1
    c, e = O.encode(x)
    assert e[0] == 127 and c[1] == code
    c, e = O.encode(-x)
    assert c[1] == (code + 8 if code else 0)


def test_rounding_error_is_at_most_half_a_step():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((200, 64)) * np.exp2(rng.integers(-20, 20, (200, 1)))
    c, e = O.encode(x)
    y = O.decode(c, e)
    unit = np.repeat(np.exp2(e - 127.0), 32, -1)
    a = np.abs(x) / unit
    half = np.where(a < 2, 0.25, np.where(a < 4, 0.5, np.where(a < 6, 1.0, 2.0)))
    assert (np.abs(x - y) <= half * unit).all()


def test_exponents_stay_in_range():
    for x, e in ((0.0, 2), (1e-300, 2), (2.0 ** -123, 2), (2.0 ** -122, 3), (2.0 ** 127, 252), (2.0 ** 128, 252)):
        assert O.encode(np.full(32, x))[1][0] == e


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_lengths_and_relative_angles(interleaved):
    rng = np.random.default_rng(1)
    half = 16
    angle = np.arange(50)[:, None] * 10000.0 ** (-np.arange(half) / half)
    cos, sin = np.cos(angle), np.sin(angle)
    q, k = rng.standard_normal(64), rng.standard_normal(64)
    turn = lambda x, p: O.rotate(x, cos[p], sin[p], interleaved)  # noqa: E731
    np.testing.assert_array_equal(turn(k, 0), k)
    np.testing.assert_array_equal(turn(k, 7)[2 * half:], k[2 * half:])
    np.testing.assert_allclose(np.linalg.norm(turn(k, 31)), np.linalg.norm(k), rtol=1e-12)
    np.testing.assert_allclose(turn(q, 40) @ turn(k, 33), turn(q, 12) @ turn(k, 5), rtol=1e-9)


def test_blocks_do_not_overlap():
    for P, D in ((16, 64), (256, 128)):
        raw = np.zeros((P, 17 * D // 16), np.uint8)
        b = O.Block(raw)
        sizes = [a.size for a in (b.kc, b.vc, b.ke, b.ve)]
        assert sum(sizes) == raw.size
        for i, a in enumerate((b.kc, b.vc, b.ke, b.ve)):
            a[:] = i + 1
        assert (np.diff(raw.reshape(-1).astype(int)) >= 0).all()


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    v = rng.standard_normal((9, 1, 64))
    q = rng.standard_normal((2, 3, 64))
    out, _, _ = O.attend(np.zeros((9, 1, 64)), v, q, 7, 0.125)      # equal keys: the mean of what is seen
    np.testing.assert_allclose(out[0], np.repeat(v[:8, 0].mean(0, keepdims=True), 3, 0), atol=1e-12)
    np.testing.assert_allclose(out[1], np.repeat(v.mean(0), 3, 0), atol=1e-12)
    out, _, _ = O.attend(rng.standard_normal((1, 1, 64)), v[:1], q[:1], 0, 0.125)  # one token: its value
    np.testing.assert_allclose(out[0], np.repeat(v[0], 3, 0), atol=1e-15)


# -- refusals ---------------------------------------------------------------

def cache(base=FAKE, n_pages=10, P=16, H=2, D=128):
    return B.kda_kv_pool(base, n_pages, P, H, D)


def append(C=None, **over):
    a = dict(table=FAKE, max_pages=4, cu=FAKE, lens=FAKE, k=FAKE, v=FAKE, ks=256, vs=256, q=FAKE, qs=512, q_out=FAKE,
             cos=FAKE, sin=FAKE, n_pos=100, rot=64, inter=0, n_seq=1, n_tokens=3, heads=4, dtype=B.KDA_BF16)
    a.update(over)
    C = cache() if C is None else C
    return B.library().kda_kv_append(ctypes.byref(C), a["table"], a["max_pages"], a["cu"], a["lens"], a["k"], a["v"],
                                     a["ks"], a["vs"], a["q"], a["qs"], a["q_out"], a["cos"], a["sin"], a["n_pos"],
                                     a["rot"], a["inter"], a["n_seq"], a["n_tokens"], a["heads"], a["dtype"], None)


def read(C=None, **over):
    a = dict(table=FAKE, max_pages=4, cu=FAKE, first=FAKE, k=FAKE, v=FAKE, ks=256, vs=256, n_seq=1, n_tokens=3,
             dtype=B.KDA_F16)
    a.update(over)
    C = cache() if C is None else C
    return B.library().kda_kv_read(ctypes.byref(C), a["table"], a["max_pages"], a["cu"], a["first"], a["k"], a["v"],
                                   a["ks"], a["vs"], a["n_seq"], a["n_tokens"], a["dtype"], None)


def attend(C=None, **over):
    a = dict(table=FAKE, max_pages=4, cu=FAKE, lens=FAKE, q=FAKE, qs=512, out=FAKE, n_seq=1, n_tokens=3, max_rows=3,
             max_kv=64, heads=4, dtype=B.KDA_F32, scale=0.1, ws=FAKE, ws_bytes=1 << 30)
    a.update(over)
    C = cache() if C is None else C
    return B.library().kda_kv_attend(ctypes.byref(C), a["table"], a["max_pages"], a["cu"], a["lens"], a["q"], a["qs"],
                                     a["out"], a["n_seq"], a["n_tokens"], a["max_rows"], a["max_kv"], a["heads"],
                                     a["dtype"], a["scale"], a["ws"], a["ws_bytes"], None)


@pytest.mark.parametrize("call", [append, read, attend])
def test_what_every_entry_point_refuses(call):
    lib = B.library()
    assert lib.kda_kv_pool_bytes(10, 16, 2, 128) == 10 * 2 * 16 * 136
    assert call(cache(base=None)) == B.KDA_ERR_NULL
    for bad in (dict(P=8), dict(P=48), dict(P=512), dict(D=32), dict(D=96), dict(D=256), dict(H=0), dict(H=4097),
                dict(n_pages=0)):
        assert call(cache(**bad)) == B.KDA_ERR_SHAPE, bad
    assert call(n_seq=-1) == B.KDA_ERR_ARG
    assert call(n_tokens=-1) == B.KDA_ERR_ARG
    assert call(n_tokens=1 << 31) == B.KDA_ERR_ARG
    assert call(max_pages=0) == B.KDA_ERR_ARG
    assert call(max_pages=1 << 27) == B.KDA_ERR_ARG          # 2^31 positions
    assert call(max_pages=(1 << 27) - 255) == B.KDA_ERR_ARG  # 16 more than 2^31 - 4096
    assert call(max_pages=(1 << 27) - 256, n_tokens=0) == B.KDA_OK
    for dtype in (3, 99, -1):
        assert call(dtype=dtype) == B.KDA_ERR_DTYPE_REFUSED
    for name in ("table", "cu"):
        assert call(**{name: None}) == B.KDA_ERR_NULL
        assert call(**{name: FAKE + 2}) == B.KDA_ERR_ALIGN
    assert call(cache(base=FAKE + 8)) == B.KDA_ERR_ALIGN
    # nothing to do is no error, whatever the pointers
    assert call(n_seq=0, table=None, cu=None) == B.KDA_OK
    assert call(n_tokens=0, table=None, cu=None) == B.KDA_OK


def test_append_refusals():
    for name in ("lens", "k", "v", "q", "q_out", "cos", "sin"):
        assert append(**{name: None}) == B.KDA_ERR_NULL, name
    for name in ("k", "v", "q", "q_out", "cos", "sin"):
        assert append(**{name: FAKE + 4}) == B.KDA_ERR_ALIGN, name
    assert append(rot=144) == B.KDA_ERR_SHAPE
    assert append(rot=24) == B.KDA_ERR_SHAPE
    assert append(rot=-16) == B.KDA_ERR_SHAPE
    assert append(inter=2) == B.KDA_ERR_ARG
    assert append(heads=-1) == B.KDA_ERR_ARG
    assert append(n_pos=-1) == B.KDA_ERR_ARG
    for name, short, odd in (("ks", 248, 260), ("vs", 248, 260), ("qs", 504, 516)):
        assert append(**{name: short}) == B.KDA_ERR_ARG      # rows would overlap
        assert append(**{name: odd}) == B.KDA_ERR_ALIGN      # rows not 16-byte aligned
        assert append(**{name: -512}) == B.KDA_ERR_ARG


def test_read_refusals():
    assert read(first=None) == B.KDA_ERR_NULL
    assert read(k=None, v=None) == B.KDA_ERR_NULL
    for name in ("k", "v"):
        assert read(**{name: FAKE + 8}) == B.KDA_ERR_ALIGN
    for name in ("ks", "vs"):
        assert read(**{name: 255}) == B.KDA_ERR_ARG
        assert read(**{name: 257}) == B.KDA_ERR_ALIGN


def test_attend_refusals():
    for name in ("lens", "q", "out"):
        assert attend(**{name: None}) == B.KDA_ERR_NULL, name
    for name in ("q", "out", "ws"):
        assert attend(**{name: FAKE + 4}) == B.KDA_ERR_ALIGN, name
    for heads in (0, -2, 3, 65536 * 2):
        assert attend(heads=heads) == B.KDA_ERR_SHAPE
    assert attend(max_rows=-1) == B.KDA_ERR_ARG
    assert attend(max_kv=-1) == B.KDA_ERR_ARG
    for scale in (float("nan"), float("inf")):
        assert attend(scale=scale) == B.KDA_ERR_ARG
    assert attend(qs=511) == B.KDA_ERR_ARG
    assert attend(qs=514) == B.KDA_ERR_ALIGN
    assert attend(n_tokens=1 << 30) == B.KDA_ERR_ARG          # n_tokens * q_heads / H
    # a long cache is split, and the split needs its workspace
    need = B.library().kda_kv_attend_workspace(ctypes.byref(cache()), 1000, 1, 3, 3, 16000, 4, B.KDA_F32)
    assert need > 0
    assert attend(max_pages=1000, max_kv=16000, ws=None, ws_bytes=0) == B.KDA_ERR_NULL
    assert attend(max_pages=1000, max_kv=16000, ws_bytes=need - 1) == B.KDA_ERR_ARG


def test_workspace_sizes():
    lib = B.library()
    size = lambda **o: lib.kda_kv_attend_workspace(  # noqa: E731
        ctypes.byref(o.get("C", cache(H=8))), o.get("max_pages", 100000), o.get("n_seq", 1), o.get("n_tokens", 1),
        o.get("rows", 1), o.get("kv", 0), o.get("heads", 32), o.get("dtype", B.KDA_BF16))
    assert size(kv=100) == 0                                  # one split
    assert size(kv=100000) % (32 * 130 * 4) == 0 and size(kv=100000) > 0
    assert size(kv=0) >= size(kv=100000)                      # 0: all that the table covers
    assert size(C=cache(P=17)) == 0 and size(heads=31) == 0 and size(rows=-1) == 0
    assert size(n_seq=4096, n_tokens=4096, kv=4096) == 0      # enough sequences fill the chip by themselves


def test_no_workspace_for_what_the_attention_refuses():
    # by type, heads, rows or workgroups; and a size for what it takes
    for over in (dict(dtype=3), dict(dtype=-1), dict(heads=65536), dict(heads=65536 * 2), dict(n_tokens=1 << 28),
                 dict(n_tokens=0), dict(n_seq=0), dict(n_seq=1 << 22, n_tokens=1 << 22, H=1)):
        C = cache(H=over.get("H", 2))
        kw = dict(max_pages=1000, max_kv=16000, heads=4, dtype=B.KDA_F32, n_seq=1, n_tokens=3, max_rows=3)
        kw.update({k: v for k, v in over.items() if k != "H"})
        need = B.library().kda_kv_attend_workspace(ctypes.byref(C), kw["max_pages"], kw["n_seq"], kw["n_tokens"],
                                                   kw["max_rows"], kw["max_kv"], kw["heads"], kw["dtype"])
        assert need == 0, over
        rc = attend(C, qs=65536 * 2 * 128, ws=None, ws_bytes=0, **kw)
        assert (rc == B.KDA_OK) == (kw["n_seq"] * kw["n_tokens"] == 0), over
    assert B.library().kda_kv_attend_workspace(ctypes.byref(cache()), 1000, 1, 3, 3, 16000, 4, B.KDA_F32) > 0


# -- host tables ------------------------------------------------------------

def valid(table, cu, lens, n_tokens, **pool):
    return B.kda_kv_validate(cache(**pool), np.array(table), cu, lens, n_tokens)


def test_validate():
    ok = dict(table=[[1, 2, -1], [3, 9, -1]], cu=[0, 3, 4], lens=[15, 30], n_tokens=5)
    assert valid(**ok) == B.KDA_OK
    assert valid([[1, 2, -1], [3, 10, -1]], [0, 3, 4], [15, 30], 5) == B.KDA_ERR_SLOT    # no such page
    assert valid([[1, -1, 4], [3, 9, -1]], [0, 3, 4], [15, 30], 5) == B.KDA_ERR_SLOT     # a page is missing
    assert valid([[1, 9, -1], [3, 9, -1]], [0, 3, 4], [15, 30], 5) == B.KDA_ERR_SLOT     # two write one page
    assert valid([[1, 1, -1], [3, 9, -1]], [0, 3, 4], [15, 30], 5) == B.KDA_ERR_SLOT     # one page at two places
    assert valid([[1, 2, -1], [1, 9, -1]], [0, 3, 4], [15, 30], 5) == B.KDA_ERR_SLOT     # read here, written there
    assert valid([[1, 2, -1], [1, 9, -1]], [0, 3, 4], [16, 30], 5) == B.KDA_OK           # a shared full page
    assert valid([[1, 2, 0], [3, 9, 0]], [0, 3, 6], [15, 30], 5) == B.KDA_ERR_ARG        # more tokens than there are
    assert valid([[1, 2, 0], [3, 9, 0]], [0, 3, 2], [15, 30], 5) == B.KDA_ERR_ARG
    assert valid([[1, 2, 0], [3, 9, 0]], [-1, 3, 4], [15, 30], 5) == B.KDA_ERR_ARG
    assert valid([[1, 2, 0], [3, 9, 0]], [0, 3, 4], [-1, 30], 5) == B.KDA_ERR_ARG
    assert valid([[1, 2, 0], [3, 9, 0]], [0, 3, 4], [15, 48], 5) == B.KDA_ERR_ARG        # behind the table
    assert valid([[1, 2, 0], [3, 9, 0]], [0, 3, 3], [15, 48], 5) == B.KDA_OK             # full, and nothing new


def test_pool_sizes():
    assert B.kda_kv_pool_bytes(7, 128, 8, 128) == 7 * 8 * 128 * 136
    assert B.kda_kv_pool_bytes(7, 128, 8, 64) == 7 * 8 * 128 * 68
    for bad in ((7, 100, 8, 128), (7, 128, 8, 96), (-1, 128, 8, 128), (7, 128, -8, 128)):
        assert B.kda_kv_pool_bytes(*bad) == 0
    assert B.kda_kv_pool_bytes(100000, 256, 4096, 128) == 100000 * 256 * 4096 * 136      # past 32 bits
    assert np.prod(K.kv_pool_shape(7, 8, 128, 64)) == B.kda_kv_pool_bytes(7, 128, 8, 64)


def test_no_size_for_shapes_that_are_refused():
    for shape in ((7, 128, 4097, 128), (7, 128, 0, 128), (0, 128, 8, 128), (7, 128, 1 << 30, 64)):
        assert B.kda_kv_pool_bytes(*shape) == 0, shape
    assert B.kda_kv_pool_bytes((1 << 31) - 1, 256, 4096, 128) == ((1 << 31) - 1) * 256 * 4096 * 136


def test_the_binding_refuses_what_is_not_on_a_gpu():
    torch = pytest.importorskip("torch")
    pool = torch.zeros(K.kv_pool_shape(2, 1, 16, 64), dtype=torch.uint8)
    t = torch.zeros((1, 2), dtype=torch.int32)
    x = torch.zeros((1, 1, 64))
    with pytest.raises(TypeError):
        K.kda_kv_append(pool, t, t[0], t[0, :1], x, x)
    with pytest.raises(TypeError):
        K.kda_kv_attend(pool, t, t[0], t[0, :1], x, x)
    with pytest.raises(TypeError):
        K.kda_kv_read(pool, t, t[0], t[0, :1], x, x)


def test_host_half_under_asan_ubsan(tmp_path):
    """The host checks alone (no HIP runtime), with random tables against a
    restatement of the rules."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src = tmp_path / "check.cpp"
    src.write_text(r'''
#include <cstdio>
#include <cstdlib>
#include <map>
#include <vector>
#include "kda_kv.h"
using namespace kda;
int main() {
  srand(7);
  char dummy[16];
  int seen[3] = {0, 0, 0};
  for (int it = 0; it < 20000; ++it) {
    const int n = rand() % 4, pages = 2 + rand() % 9, P = 16, mp = 1 + rand() % 4;
    kda_kv_pool kv{dummy, pages, P, 2, 64};
    std::vector<int> table(n * mp), cu{0}, lens;
    for (int& t : table) t = rand() % (pages + (rand() % 6 == 0)) - (rand() % 12 == 0);
    for (int s = 0; s < n; ++s) {
      cu.push_back(cu.back() + rand() % 20);
      lens.push_back(rand() % (mp * P) - (rand() % 40 == 0));
    }
    int want = KDA_OK;
    for (int s = 0; s < n && want == KDA_OK; ++s)
      if (lens[s] < 0 || lens[s] + cu[s + 1] - cu[s] > mp * P) want = KDA_ERR_ARG;
    if (want == KDA_OK) {
      std::map<int, int> uses, writes;
      for (int s = 0; s < n; ++s) {
        const int end = lens[s] + cu[s + 1] - cu[s];
        for (int i = 0; i * P < end; ++i) {
          const int page = table[s * mp + i];
          if (page < 0 || page >= pages) want = KDA_ERR_SLOT;
          ++uses[page];
          if (cu[s + 1] > cu[s] && (i + 1) * P > lens[s]) ++writes[page];
        }
      }
      for (auto& w : writes)
        if (uses[w.first] > 1) want = KDA_ERR_SLOT;
    }
    const int got = kda_kv_validate(&kv, table.data(), mp, cu.data(), lens.data(), n, cu.back());
    if (got != want) { std::printf("case %d: %d, not %d\n", it, got, want); return 1; }
    ++seen[want == KDA_OK ? 0 : want == KDA_ERR_SLOT ? 1 : 2];
  }
  if (!seen[0] || !seen[1] || !seen[2]) { std::printf("one sided\n"); return 1; }
  for (int it = 0; it < 20000; ++it) {
    // a plan covers its rows and its cache, in whole steps
    const int H = 1 + rand() % 16, G = 1 + rand() % 9, n_seq = 1 + rand() % 200, rows = 1 + rand() % 5000;
    const int64_t kv = 1 + rand() % 200000;
    const kda_dtype dt = static_cast<kda_dtype>(rand() % 3);
    const KvPlan p = kv_plan(H, rand() % 2 ? 64 : 128, n_seq, static_cast<int64_t>(n_seq) * rows, rows, kv, H * G, dt);
    const int64_t tiles = p.tile_rows == 128 ? p.slots : p.row_tiles;
    if (tiles * p.tile_rows < static_cast<int64_t>(rows) * G ||
        static_cast<int64_t>(p.n_splits) * p.chunk + p.chunk / 8 < kv ||  // (the last split may be longer)
        p.chunk % 32 != 0 || p.n_splits < 1 ||
        (p.n_splits > 1 && static_cast<int64_t>(p.n_splits - 1) * p.chunk >= kv)) {
      std::printf("plan %d: %d x %d rows, %d x %d tokens\n", it, p.row_tiles, p.tile_rows, p.n_splits, p.chunk);
      return 1;
    }
  }
  // slots hold every sequence's tiles, one after the other
  for (int it = 0; it < 20000; ++it) {
    const int G = 1 + rand() % 9, n = 1 + rand() % 6, spare = rand() % 3 * 50;
    int64_t cu = rand() % 30, next = 0;
    int64_t ends[6];
    for (int s = 0; s < n; ++s) {
      const int64_t first = cu * G / 128 + s, rows = rand() % 4 ? rand() % 700 : rand() % 3;
      if (first < next) { std::printf("slots of %d overlap\n", s); return 1; }
      next = first + (rows * G + 127) / 128;
      ends[s] = cu += rows;
    }
    const KvPlan p = kv_plan(1, 64, n, ends[n - 1] + spare, 1000, 5000, G, KDA_F32);
    if (p.tile_rows == 128 && next > p.slots) { std::printf("%d slots, not %d\n", p.slots, (int)next); return 1; }
  }
  std::printf("kv host checks ok\n");
  return 0;
}
''')
    exe = tmp_path / "check"
    csrc = os.path.join(ROOT, "kda_gated_delta_decode_amd", "csrc")
    b = subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=address,undefined", "-fno-sanitize-recover=all", "-g",
                        "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", csrc, str(src),
                        os.path.join(csrc, "kda_kv_host.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert b.returncode == 0, b.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "kv host checks ok" in r.stdout, r.stdout + r.stderr


def test_validate_without_host_memory(tmp_path):
    """The table check's own memory runs out: an error, and no exception
    through the C entry."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    src = tmp_path / "oom.cpp"
    src.write_text(r'''
#include <cstdio>
#include <cstdlib>
#include <new>
#include "kda_kv.h"
static int left = 1 << 30;
void* operator new(size_t n) {
  if (left-- <= 0) throw std::bad_alloc();
  return std::malloc(n);
}
void operator delete(void* p) noexcept { std::free(p); }
void operator delete(void* p, size_t) noexcept { std::free(p); }
int main() {
  char dummy[16];
  kda_kv_pool kv{dummy, 64, 16, 2, 64};
  int table[64], cu[2] = {0, 64 * 16}, lens[1] = {0};
  for (int i = 0; i < 64; ++i) table[i] = i;
  if (kda_kv_validate(&kv, table, 64, cu, lens, 1, 64 * 16) != KDA_OK) return 1;
  for (int n = 0; n < 40; ++n) {
    left = n;
    if (kda_kv_validate(&kv, table, 64, cu, lens, 1, 64 * 16) != KDA_ERR_ARG) return 2;
  }
  std::printf("no exception\n");
  return 0;
}
''')
    exe = tmp_path / "oom"
    csrc = os.path.join(ROOT, "kda_gated_delta_decode_amd", "csrc")
    b = subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"),
                        "-I", csrc, str(src), os.path.join(csrc, "kda_kv_host.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    assert b.returncode == 0, b.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "no exception" in r.stdout, (r.returncode, r.stdout + r.stderr)
