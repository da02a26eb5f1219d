"""CPU tests of the calls for trees of drafted tokens: the oracle's own pins, every
refusal of the entry points (no HIP call happens before one), the host checks
under the sanitizers, and the binding's checks of its arguments."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

from kda_gated_delta_decode_amd import binding as B
from oracle import kv_cache, trees

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # an aligned address that is never dereferenced


# --------------------------------------------------------------------------
# the oracle
# --------------------------------------------------------------------------

def test_oracle_chain_attention_is_causal_attention():
    rng = np.random.default_rng(0)
    k, v, q = rng.standard_normal((9, 2, 64)), rng.standard_normal((9, 2, 64)), rng.standard_normal((5, 4, 64))
    got = trees.attend(k, v, q, 4, [-1, 0, 1, 2, 3], 0.2)
    want = kv_cache.attend(k, v, q, 4, 0.2)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


def test_oracle_siblings_do_not_see_each_other():
    rng = np.random.default_rng(1)
    k, v, q = rng.standard_normal((5, 1, 64)), rng.standard_normal((5, 1, 64)), rng.standard_normal((3, 1, 64))
    a = trees.attend(k, v, q, 2, [-1, 0, 0], 0.2)[0]
    k[3], v[3] = 100, 100  # node 1
    b = trees.attend(k, v, q, 2, [-1, 0, 0], 0.2)[0]
    assert np.array_equal(a[[0, 2]], b[[0, 2]]) and not np.array_equal(a[1], b[1])


def test_oracle_recurrence_closed_forms():
    # from a zero state, one node: o = scale beta (qn . kn) v
    rng = np.random.default_rng(2)
    q, k, v = (rng.standard_normal((3, 2, 128)) for _ in range(3))
    g, b = -np.abs(rng.standard_normal((3, 2, 128))), rng.standard_normal((3, 2))
    out = trees.recurrence(np.zeros((2, 128, 128)), [-1, -1, 0], q, k, v, g, b, 0.5)
    unit = lambda x: x / np.sqrt((x * x).sum(-1, keepdims=True) + 1e-6)  # noqa: E731
    beta = 1 / (1 + np.exp(-b))
    for i in (0, 1):
        want = 0.5 * beta[i][:, None] * (unit(q[i]) * unit(k[i])).sum(-1, keepdims=True) * v[i]
        assert np.allclose(out[i], want, rtol=1e-12, atol=1e-14)
    # the third follows the first: its path's state, read out
    S = trees.advance(np.zeros((2, 128, 128)), [0, 2], k, v, g, b)
    assert np.allclose(out[2], 0.5 * np.einsum("hk,hkv->hv", unit(q[2]), S), rtol=1e-12, atol=1e-14)


def test_oracle_verification_preserves_the_target():
    # every outcome of a small case, weighted by the share of random numbers that
    # leads to it, gives the target's distribution back: one drafted token from q
    # and the token that replaces it
    p, q = np.array([0.5, 0.125, 0.25, 0.125]), np.array([0.25, 0.5, 0.125, 0.125])
    target, draft = np.stack([p, p]), np.stack([q, q])
    steps = (np.arange(64) + 0.5) / 64
    got = np.zeros(4)
    for x in range(4):
        for u in steps:
            for s in steps:
                path, nxt = trees.verify(target, draft, [-1, 0], [0, x], [0, u], s)
                got[x if len(path) == 2 else nxt] += q[x] / 64 / 64
    # acceptance borders (1 and 0.25) lie between two steps, so the shares are
    # exact; what replaces a refused token is drawn with shares 2/3 and 1/3, which
    # 64 midpoints hold to half a step, with a probability of 0.375
    assert np.allclose(got, p, rtol=0, atol=0.375 / 128)


def test_oracle_verification_of_chosen_children_preserves_the_target():
    p = np.array([0.5, 0.125, 0.25, 0.125])
    target = np.stack([p, p, p])
    steps = (np.arange(48) + 0.5) / 48
    got = np.zeros(4)
    for u in steps:
        for w in steps:
            for s in steps:
                path, nxt = trees.verify(target, None, [-1, 0, 0], [0, 2, 1], [0, u, w], s)
                got[nxt if len(path) == 1 else {1: 2, 2: 1}[path[1]]] += 48.0 ** -3
    # borders of u M < p (1/4, 1/6) lie between two steps; the last draw's at 0.8,
    # held to half a step, with a probability of 0.625
    assert np.allclose(got, p, rtol=0, atol=0.625 / 96)


def test_oracle_verification_edges():
    one = np.array([[0.0, 1.0, 0.0], [0.0, 0.0, 0.0], [np.nan, -1.0, np.inf]])
    assert trees.verify(one, None, [-1, 0, 1], [0, 1, 1], [0, 0.999, 0], 0.0) == ([0, 1], -1)
    assert trees.verify(one[:1], None, [-1], [0], [0], 0.99) == ([0], 1)
    assert trees.verify(one[2:], None, [-1], [0], [0], 0.5) == ([0], -1)
    # q is p: every draw of it is accepted; nothing is left otherwise
    p = np.array([[0.25, 0.75], [0.5, 0.5]])
    assert trees.verify(p, p, [-1, 0], [0, 0], [0, 0.999], 0.6) == ([0, 1], 1)
    # a residual of nothing is drawn from the row itself
    q = np.array([[0.5, 1.0], [0.5, 0.5]])
    assert trees.verify(p, q, [-1, 0], [0, 1], [0, 0.9], 0.3) == ([0], 1)


def test_oracle_keep():
    x = np.arange(10)
    trees.keep(x, 2, [0, 1, 3, 6])
    assert x.tolist() == [0, 1, 2, 3, 5, 8, 6, 7, 8, 9]


# --------------------------------------------------------------------------
# refusals
# --------------------------------------------------------------------------

def pool(n_slots=8, H=12, K=128, V=128, dtype=B.KDA_F32, base=FAKE):
    return B.kda_pool(ctypes.c_void_p(base), n_slots, H, K, V, dtype)


def cache(n_pages=8, P=16, H=2, D=128, base=FAKE):
    return B.kda_kv_pool(ctypes.c_void_p(base), n_pages, P, H, D)


def tree_call(P=None, n_req=2, n_tokens=8, max_nodes=8, dtype=B.KDA_F32, scale=0.1, **ptr):
    P = pool(dtype=dtype) if P is None else P
    p = [ptr.get(n, FAKE) for n in ("init", "cu", "parents", "q", "k", "v", "g", "b", "out")]
    return B.library().kda_decode_tree(ctypes.byref(P), *p, n_req, n_tokens, max_nodes, dtype, scale, None)


def path_call(P=None, n_req=2, n_tokens=8, max_path=8, dtype=B.KDA_F32, **ptr):
    P = pool(dtype=dtype) if P is None else P
    p = {n: ptr.get(n, FAKE) for n in ("init", "dst", "cu", "path", "lens", "k", "v", "g", "b")}
    return B.library().kda_decode_path(ctypes.byref(P), p["init"], p["dst"], p["cu"], p["path"], max_path, p["lens"],
                                       p["k"], p["v"], p["g"], p["b"], n_req, n_tokens, dtype, None)


@pytest.mark.parametrize("call", [tree_call, path_call])
def test_state_refusals(call):
    assert call(P=pool(base=0)) == B.KDA_ERR_NULL
    assert call(dtype=B.KDA_BF16) == B.KDA_ERR_DTYPE_REFUSED
    assert call(P=pool(dtype=B.KDA_F16)) == B.KDA_ERR_DTYPE_MISMATCH
    for P in (pool(H=0), pool(K=64), pool(V=64), pool(n_slots=0), pool(H=16385)):
        assert call(P=P) == B.KDA_ERR_SHAPE
    assert call(n_req=-1) == B.KDA_ERR_ARG
    assert call(n_tokens=-1) == B.KDA_ERR_ARG
    assert call(n_tokens=2 ** 31) == B.KDA_ERR_ARG
    assert call(n_req=0, k=0, cu=0) == B.KDA_OK
    for name in ("init", "cu", "k", "v", "g", "b"):
        assert call(**{name: 0}) == B.KDA_ERR_NULL, name
    for name in ("k", "v", "g"):
        assert call(**{name: FAKE + 4}) == B.KDA_ERR_ALIGN, name
    for name in ("init", "cu", "b"):
        assert call(**{name: FAKE + 2}) == B.KDA_ERR_ALIGN, name
    assert call(P=pool(base=FAKE + 8)) == B.KDA_ERR_ALIGN


def test_tree_refusals():
    assert tree_call(max_nodes=65) == B.KDA_ERR_ROWS
    assert tree_call(max_nodes=-1) == B.KDA_ERR_ROWS
    assert tree_call(n_tokens=0, q=0) == B.KDA_OK
    for name in ("parents", "q", "out"):
        assert tree_call(**{name: 0}) == B.KDA_ERR_NULL, name
        assert tree_call(**{name: FAKE + 2}) == B.KDA_ERR_ALIGN, name
    assert tree_call(scale=float("inf")) == B.KDA_ERR_ARG
    assert tree_call(scale=float("nan")) == B.KDA_ERR_ARG
    # (more requests than slots may share them; threads must be countable)
    assert tree_call(P=pool(H=16384), n_req=2 ** 20) == B.KDA_ERR_ARG


def test_path_refusals():
    for n in (0, -1, 65):
        assert path_call(max_path=n) == B.KDA_ERR_ROWS
    assert path_call(n_req=9) == B.KDA_ERR_SLOT
    for name in ("path", "lens"):
        assert path_call(**{name: 0}) == B.KDA_ERR_NULL, name
        assert path_call(**{name: FAKE + 2}) == B.KDA_ERR_ALIGN, name
    assert path_call(dst=FAKE + 2) == B.KDA_ERR_ALIGN
    assert path_call(P=pool(n_slots=2 ** 20, H=16384), n_req=2 ** 20) == B.KDA_ERR_ARG


def verify_call(n_req=2, n_tokens=8, vocab=100, max_path=8, dtype=B.KDA_F32, strides=(100, 100), ws=None, bytes_=1 << 20,
                **ptr):
    names = ("target", "draft", "cu", "parents", "tokens", "accept", "sample", "path", "lens", "next")
    p = {n: ptr.get(n, FAKE) for n in names}
    return B.library().kda_verify_drafts(p["target"], strides[0], p["draft"], strides[1], p["cu"], p["parents"], p["tokens"],
                                         p["accept"], p["sample"], p["path"], max_path, p["lens"], p["next"], n_req,
                                         n_tokens, vocab, dtype, FAKE if ws is None else ws, bytes_, None)


def test_verify_refusals():
    assert verify_call(dtype=7) == B.KDA_ERR_DTYPE_REFUSED
    for kw in (dict(n_req=-1), dict(n_tokens=-1), dict(n_tokens=2 ** 31), dict(vocab=0), dict(vocab=-5)):
        assert verify_call(**kw) == B.KDA_ERR_ARG, kw
    for n in (0, -1, 65):
        assert verify_call(max_path=n) == B.KDA_ERR_ROWS
    assert verify_call(n_req=0, target=0, cu=0) == B.KDA_OK
    for name in ("target", "cu", "parents", "tokens", "accept", "sample", "path", "lens", "next"):
        assert verify_call(**{name: 0}) == B.KDA_ERR_NULL, name
        assert verify_call(**{name: FAKE + 2}) == B.KDA_ERR_ALIGN, name
    assert verify_call(draft=FAKE + 2) == B.KDA_ERR_ALIGN
    for dtype in (B.KDA_F16, B.KDA_BF16):  # rows at any multiple of their type
        assert verify_call(dtype=dtype, target=FAKE + 1) == B.KDA_ERR_ALIGN
        assert verify_call(dtype=dtype, target=FAKE + 2, ws=0) == B.KDA_ERR_NULL
    assert verify_call(strides=(99, 100)) == B.KDA_ERR_ARG
    assert verify_call(strides=(100, 99)) == B.KDA_ERR_ARG
    need = B.kda_verify_workspace(2, 8, 100, 8)
    assert need > 0
    assert verify_call(ws=0) == B.KDA_ERR_NULL
    assert verify_call(bytes_=need - 1) == B.KDA_ERR_ARG
    assert verify_call(ws=FAKE + 4) == B.KDA_ERR_ALIGN
    for kw in (dict(n_req=0), dict(n_req=-1), dict(vocab=0), dict(max_path=0), dict(max_path=65), dict(n_tokens=-1),
               dict(dtype=9)):
        a = dict(n_req=2, n_tokens=8, vocab=100, max_path=8, dtype=B.KDA_F32)
        a.update(kw)
        assert B.kda_verify_workspace(**a) == 0, kw
    assert verify_call(n_req=2 ** 31 - 1, bytes_=2 ** 62) == B.KDA_ERR_ARG


def attend_tree_call(C=None, n_seq=2, n_tokens=8, max_rows=8, q_heads=4, dtype=B.KDA_F32, scale=0.1, stride=512, **ptr):
    C = cache() if C is None else C
    p = {n: ptr.get(n, FAKE) for n in ("table", "cu", "lens", "parents", "q", "out", "ws")}
    return B.library().kda_kv_attend_tree(ctypes.byref(C), p["table"], 8, p["cu"], p["lens"], p["parents"], p["q"], stride,
                                          p["out"], n_seq, n_tokens, max_rows, 0, q_heads, dtype, scale, p["ws"], 1 << 30,
                                          None)


def test_attend_tree_refusals():
    call = attend_tree_call
    assert call(C=cache(base=0)) == B.KDA_ERR_NULL
    assert call(C=cache(P=24)) == B.KDA_ERR_SHAPE
    assert call(n_seq=-1) == B.KDA_ERR_ARG
    assert call(dtype=7) == B.KDA_ERR_DTYPE_REFUSED
    assert call(q_heads=3) == B.KDA_ERR_SHAPE
    assert call(max_rows=-1) == B.KDA_ERR_ARG
    assert call(max_rows=65) == B.KDA_ERR_ROWS
    assert call(scale=float("inf")) == B.KDA_ERR_ARG
    assert call(n_seq=0, q=0) == B.KDA_OK
    assert call(n_tokens=0, q=0) == B.KDA_OK
    for name in ("table", "cu", "lens", "parents", "q", "out"):
        assert call(**{name: 0}) == B.KDA_ERR_NULL, name
        assert call(**{name: FAKE + 2}) == B.KDA_ERR_ALIGN, name
    assert call(stride=511) == B.KDA_ERR_ARG


def keep_call(C=None, n_seq=2, n_tokens=8, max_path=8, **ptr):
    C = cache() if C is None else C
    p = {n: ptr.get(n, FAKE) for n in ("table", "cu", "lens", "path", "path_lens")}
    return B.library().kda_kv_keep(ctypes.byref(C), p["table"], 8, p["cu"], p["lens"], p["path"], max_path,
                                   p["path_lens"], n_seq, n_tokens, None)


def test_keep_refusals():
    assert keep_call(C=cache(base=0)) == B.KDA_ERR_NULL
    assert keep_call(C=cache(D=96)) == B.KDA_ERR_SHAPE
    assert keep_call(n_seq=-1) == B.KDA_ERR_ARG
    for n in (0, -1, 65):
        assert keep_call(max_path=n) == B.KDA_ERR_ROWS
    assert keep_call(n_seq=0, path=0) == B.KDA_OK
    for name in ("table", "cu", "lens", "path", "path_lens"):
        assert keep_call(**{name: 0}) == B.KDA_ERR_NULL, name
        assert keep_call(**{name: FAKE + 2}) == B.KDA_ERR_ALIGN, name
    assert keep_call(C=cache(base=FAKE + 8)) == B.KDA_ERR_ALIGN


def append_at_call(rot=64, positions=FAKE, n_positions=10):
    C = cache()
    return B.library().kda_kv_append_at(ctypes.byref(C), FAKE, 8, FAKE, FAKE, FAKE, 0, 256, 256, 0, 0, 0, FAKE, FAKE,
                                        positions, n_positions, rot, 0, 2, 8, 0, B.KDA_F32, None)


def test_append_at_refusals():
    assert append_at_call() == B.KDA_ERR_NULL  # no values
    C = cache()
    call = lambda positions: B.library().kda_kv_append_at(  # noqa: E731
        ctypes.byref(C), FAKE, 8, FAKE, FAKE, FAKE, FAKE, 256, 256, 0, 0, 0, FAKE, FAKE, positions, 10, 64, 0, 2, 8, 0,
        B.KDA_F32, None)
    assert call(FAKE + 2) == B.KDA_ERR_ALIGN


@pytest.mark.parametrize("cu,parents,code", [
    ([0, 3, 3, 5], [-1, 0, 0, -1, 0], "KDA_OK"),
    ([0, 2], [-1, -1], "KDA_OK"),
    ([1, 3], [9, -1, 0, 9], "KDA_OK"),
    ([0], [], "KDA_OK"),
    ([0, 0], [], "KDA_OK"),
    ([0, 2], [-1, 1], "KDA_ERR_ARG"),
    ([0, 2], [0, 0], "KDA_ERR_ARG"),
    ([0, 2], [-1, -2], "KDA_ERR_ARG"),
    ([0, 3, 2], [-1, 0, 0], "KDA_ERR_ARG"),
    ([-1, 2], [-1, 0], "KDA_ERR_ARG"),
    ([0, 3], [-1, 0], "KDA_ERR_ARG"),
    ([0, 64], [-1] * 64, "KDA_OK"),
    ([0, 65], [-1] * 65, "KDA_ERR_ROWS"),
])
def test_tree_validate(cu, parents, code):
    assert B.kda_tree_validate(cu, parents) == getattr(B, code)


def test_tree_validate_nulls_and_counts():
    f = B.library().kda_tree_validate
    one = np.array([0, 1], np.int32)
    assert f(None, None, 0, 0) == B.KDA_OK
    assert f(None, one.ctypes.data, 1, 1) == B.KDA_ERR_NULL
    assert f(one.ctypes.data, None, 1, 1) == B.KDA_ERR_NULL
    assert f(one.ctypes.data, None, -1, 1) == B.KDA_ERR_ARG
    assert f(one.ctypes.data, None, 1, -1) == B.KDA_ERR_ARG
    with pytest.raises(ValueError):
        B.kda_tree_validate([0, 3], [-1, 0], n_tokens=3)


HOST_MAIN = r"""
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "kda_decode.h"
#include "kda_tree.h"
// a row's runs cover every entry once, and none is empty
static void plan(int32_t vocab) {
  const kda::VerifyPlan p = kda::verify_plan(vocab);
  const int64_t covered = (int64_t)p.runs * p.run;
  if (p.runs < 1 || p.runs > 64 || p.run < 1 || covered < vocab || covered - p.run >= vocab) {
    std::printf("plan %d: %d x %d\n", vocab, p.runs, p.run);
    std::exit(1);
  }
}
int main() {
  for (int32_t v : {1, 2, 255, 256, 257, 4095, 4096, 4097, 8193, 32768, 50021, 100003, 131072, 999983, 2147483392, 2147483647}) plan(v);
  std::srand(1);
  for (int i = 0; i < 20000; ++i) plan(1 + std::rand() % 300000);
  // parents of a table that ends where the nodes end
  for (int n = 0; n <= 64; ++n) {
    std::vector<int32_t> cu = {0, n}, parents(n);
    for (int i = 0; i < n; ++i) parents[i] = i - 1;
    if (kda_tree_validate(cu.data(), parents.data(), 1, n) != KDA_OK) return 1;
    if (n > 0) {
      parents[n - 1] = n - 1;
      if (kda_tree_validate(cu.data(), parents.data(), 1, n) != KDA_ERR_ARG) return 1;
    }
  }
  std::puts("tree host checks ok");
  return 0;
}
"""


def test_host_half_under_asan_ubsan(tmp_path):
    if not shutil.which("g++"):
        pytest.skip("no g++")
    csrc = os.path.join(ROOT, "kda_gated_delta_decode_amd", "csrc")
    src, exe = tmp_path / "main.cpp", tmp_path / "tree_host"
    src.write_text(HOST_MAIN)
    b = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", csrc, str(src),
                        os.path.join(csrc, "kda_tree_host.cpp"), os.path.join(csrc, "kda_host.cpp"), "-o", str(exe)],
                       capture_output=True, text=True)
    assert b.returncode == 0, b.stdout + b.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and "tree host checks ok" in r.stdout, r.stdout + r.stderr


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    z = torch.zeros
    i = z(3, dtype=torch.int32)
    rows = [z(2, 1, 128) for _ in range(4)]
    with pytest.raises(TypeError):
        B.kda_decode_tree(z(2, 1, 128, 128), i[:2], i, i[:2], *rows, z(2, 1), z(2, 1, 128))
    with pytest.raises(TypeError):
        B.kda_decode_path(z(2, 1, 128, 128), i[:2], i, z(2, 2, dtype=torch.int32), i[:2], *rows[:3], z(2, 1))
    with pytest.raises(TypeError):
        B.kda_verify_drafts(z(2, 5), i, i[:2], i[:2], z(2), z(2), z(2, 2, dtype=torch.int32), i[:2], i[:2])
    with pytest.raises(TypeError):
        B.kda_kv_keep(z(B.kv_pool_shape(2, 1, 16, 64), dtype=torch.uint8), z(2, 2, dtype=torch.int32), i, i[:2],
                      z(2, 2, dtype=torch.int32), i[:2])
    with pytest.raises(TypeError):
        B.kda_kv_attend_tree(z(B.kv_pool_shape(2, 1, 16, 64), dtype=torch.uint8), z(2, 2, dtype=torch.int32), i, i[:2],
                             i[:2], z(2, 1, 64), z(2, 1, 64))


def test_constants_and_exports():
    assert B.KDA_MAX_NODES == 64
    import kda_gated_delta_decode_amd as pkg
    for name in ("kda_decode_tree", "kda_decode_path", "kda_kv_attend_tree", "kda_kv_keep", "kda_verify_drafts",
                 "kda_verify_workspace", "kda_tree_validate"):
        assert getattr(pkg, name) is getattr(B, name)


PLAN_MAIN = r"""
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <vector>
#include "kda_kv.h"
struct Tree { int rows; int64_t past; };
static int64_t cut_launches = 0, first_did_not_fit = 0;
static std::mt19937 rng(1);
static int pick(int lo, int hi) { return lo + static_cast<int>(rng() % static_cast<uint32_t>(hi - lo + 1)); }
static int spread(int lo, int hi) {  // over the logarithm
  return std::min(hi, static_cast<int>(lo * std::pow(static_cast<double>(hi + 1) / lo, rng() % 4096 / 4096.0)));
}
// The kernel's choice for these trees under a launch planned with the given sizes:
// found in few rounds, every part with a place, every tile's steps covered once.
static void launch(const std::vector<Tree>& trees, int H, int group, int D, kda_dtype dtype, int max_rows, int64_t max_kv_len) {
  const int n = static_cast<int>(trees.size());
  kda_kv_pool kv{};
  kv.H = H;
  kv.D = D;
  kv.page_tokens = 64;
  const int64_t cover = 1ll << 31;
  const kda::KvTreePlan plan = kda::kv_tree_plan(&kv, n, max_rows, group, cover, max_kv_len, dtype);
  std::vector<int> units(n), steps(n);
  float all_steps = 0.0f, all_units = 0.0f;
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    units[i] = trees[i].rows == 0 ? 0 : (trees[i].rows * group + 127) / 128 * H;
    steps[i] = static_cast<int>((trees[i].past + trees[i].rows + 63) / 64);
    all_steps += static_cast<float>(units[i]) * static_cast<float>(steps[i]);
    all_units += static_cast<float>(units[i]);
    tiles += units[i];
  }
  const auto fail = [&](const char* what, int each) {
    std::printf("%s: %d trees, %d x %d heads of %d, type %d, rows %d (%d), tokens %lld (%lld), places %d, each %d\n", what, n,
                H, group, D, static_cast<int>(dtype), trees[0].rows, max_rows, static_cast<long long>(trees[0].past),
                static_cast<long long>(max_kv_len), plan.places, each);
    std::exit(1);
  };
  int rounds = 0;
  const int each = kda::kv_tree_each(all_steps, all_units, plan.places, n <= 64, [&](int e) {
    if (++rounds > 200) fail("does not end", e);
    float parts = 0.0f;
    for (int i = 0; i < n; ++i) parts += static_cast<float>(units[i]) * static_cast<float>(kda::kv_tree_parts(steps[i], e));
    return parts;
  });
  first_did_not_fit += rounds > 1;
  int64_t parts = 0;
  for (int i = 0; i < n; ++i) {
    if (units[i] == 0) continue;
    const int k = kda::kv_tree_parts(steps[i], each), len = kda::kv_tree_parts(steps[i], k);
    if (k < 1 || static_cast<int64_t>(k) * len < steps[i] || len > each) fail("steps left out", each);
    parts += static_cast<int64_t>(units[i]) * k;
  }
  // uncut: a block for every tile; cut: a place for every part, and a block
  if (each != INT32_MAX) {
    ++cut_launches;
    if (parts > plan.places) fail("parts without a place", each);
  } else if (parts != tiles) {
    fail("cut without places", each);
  }
  if (parts > plan.blocks) fail("parts without a block", each);
}
int main() {
  const int heads[][2] = {{8, 4}, {2, 8}, {4, 5}, {1, 8}, {8, 2}, {12, 3}, {1, 128}, {64, 2}, {96, 8}};
  for (const auto& h : heads)
    for (int n = 1; n <= 64; ++n)
      for (int nodes : {9, 17, 25, 32, 33, 48, 64})
        for (int past : {0, 129, 161, 200, 257, 300, 400, 512, 650, 700, 967, 1000, 1100, 1500, 1900, 2500, 4000, 9000, 60000}) {
          if (nodes * h[1] <= 64) continue;
          // all alike, then of uneven lengths and sizes below these
          std::vector<Tree> trees(n, Tree{nodes, past});
          for (int uneven = 0; uneven < 2; ++uneven) {
            for (Tree& t : trees)
              if (uneven) t = {pick(0, nodes), spread(1, past + 1) - 1};
            launch(trees, h[0], h[1], 128, KDA_BF16, nodes, past + nodes);
            launch(trees, h[0], h[1], 128, KDA_F32, nodes, past + nodes);
          }
        }
  for (int i = 0; i < 300000; ++i) {  // any number of requests, hints that need not hold
    const int n = spread(1, 700), H = spread(1, 96), group = spread(1, 64);
    const int long_one = rng() % 4 == 0 ? 2000000000 : 70000;
    std::vector<Tree> trees(n);
    for (Tree& t : trees) t = {pick(0, 64), spread(1, long_one) - 1};
    if (rng() % 3 == 0) trees.assign(n, trees[0]);
    launch(trees, H, group, rng() % 2 ? 64 : 128, rng() % 2 ? KDA_F16 : KDA_F32, pick(0, 64), rng() % 3 == 0 ? 0 : spread(1, long_one));
  }
  if (cut_launches < 100000 || first_did_not_fit < 10000) {
    std::printf("%lld, %lld\n", static_cast<long long>(cut_launches), static_cast<long long>(first_did_not_fit));
    return 1;
  }
  std::puts("tree plans ok");
  return 0;
}
"""


def test_parts_of_large_trees_are_found_and_have_places(tmp_path):
    # the choice that every block of the attention makes for itself, over the sizes it meets
    if not shutil.which("g++"):
        pytest.skip("no g++")
    csrc = os.path.join(ROOT, "kda_gated_delta_decode_amd", "csrc")
    src, exe = tmp_path / "main.cpp", tmp_path / "tree_plan"
    src.write_text(PLAN_MAIN)
    b = subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fsanitize=address,undefined", "-fno-sanitize-recover=all",
                        "-Wall", "-Wextra", "-Werror", "-I", os.path.join(ROOT, "include"), "-I", csrc, str(src),
                        os.path.join(csrc, "kda_kv_host.cpp"), "-o", str(exe)], capture_output=True, text=True)
    assert b.returncode == 0, b.stdout + b.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "tree plans ok" in r.stdout, r.stdout + r.stderr
