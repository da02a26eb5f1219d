// kda_tree.hip -- the KDA recurrence over trees of drafted tokens on gfx950, and
// the accepted path's way into the states.
//
// A node's state is S_i = (I - beta_i k_i k_i^T) diag(a_i) S_parent + beta_i k_i
// v_i^T.  Along a path that unrolls to sums over the nodes above i: with A_i the
// product of the decays of i's path, and a_(j..i) that of the decays below j,
//   u_i = v_i - S0^T (A_i k_i) - sum_j (a_(j..i) k_i . k_j) beta_j u_j
//   o_i = scale (S0^T (A_i q_i) + sum_j (a_(j..i) q_i . k_j) beta_j u_j)
// (the last sum includes j = i, where a is 1).  So one product of all nodes' 2 n
// vectors with S0 on the matrix cores, and a sparse triangular solve per value
// column; S0 is read once and no node's state is ever formed.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "kda_decode.h"
#include "kda_device.h"
#include "kda_tree_device.h"

namespace kda {
namespace {

// sum over 16 lanes, in each of them
__device__ __forceinline__ float sum16(float x) { return sum_xor8(sum_xor4(sum_xor2(sum_xor1(x)))); }

// the larger of 16 lanes' x >= 0, in each of them
__device__ __forceinline__ float max16(float x) {
  x = fmaxf(x, dpp<kDppQuadXor1>(x));
  x = fmaxf(x, dpp<kDppQuadXor2>(x));
  x = fmaxf(x, dpp<kDppQuadXor3>(dpp<kDppRowHalfMirror>(x)));
  return fmaxf(x, dpp<kDppRowRor8>(x));
}

// e^x for x below 88, within 2 units of the last place (0 below 2^-126): 2^t, with
// what rounding x log2(e) to t lost put back.  (Of an infinite t nothing is left to put.)
__device__ __forceinline__ float exp_near(float x) {
  x = x < -104.0f ? -104.0f : x;
  const float t = x * 1.44269504f;
  const float lost = fmaf(x, 1.44269504f, -t) + x * 1.92596299e-8f;
  const float y = __builtin_amdgcn_exp2f(t);
  return fmaf(y, lost * 0.693147181f, y);
}

template <int DT>
using Stored = std::conditional_t<DT == KDA_F32, float, _Float16>;

constexpr int kLd = 132;  // floats between rows in LDS: neighbouring rows start 4 banks apart

// ---------------------------------------------------------------------------
// Trees
// ---------------------------------------------------------------------------

// A row of the left operand, its 128 numbers held by 16 lanes (channels 4 l16.. and
// 64 + 4 l16..).  HALF: in two fp16 pieces of 11 bits, after division by the row's
// power of two, the second one 2^11 times larger so that it is no subnormal: 22
// bits of every number down to 2^-14 of the row's largest, 2^-36 of that below;
// what the pieces miss is less than the products' own fp32 sums round away.
template <bool HALF>
__device__ __forceinline__ void put_row(float* row, float* size, const float (&w)[8]) {
  const int l16 = threadIdx.x % 16;
  if constexpr (HALF) {
    float most = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) most = fmaxf(most, fabsf(w[e]));
    most = max16(most);
    int ex = __float_as_int(most) >> 23;
    ex = ex < 12 ? 12 : ex > 253 ? 253 : ex;  // (2^11 over the power of two is finite)
    const float down = __int_as_float((254 - ex) << 23), up = 2048.0f * down;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      h4 hi, lo;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        hi[e] = static_cast<_Float16>(w[4 * p + e] * down);
        lo[e] = static_cast<_Float16>(fmaf(static_cast<float>(hi[e]), -2048.0f, w[4 * p + e] * up));
      }
      *reinterpret_cast<h4*>(reinterpret_cast<_Float16*>(row) + 64 * p + 4 * l16) = hi;
      *reinterpret_cast<h4*>(reinterpret_cast<_Float16*>(row) + 128 + 64 * p + 4 * l16) = lo;
    }
    if (l16 == 0) *size = __int_as_float(ex << 23);
  } else {
#pragma unroll
    for (int p = 0; p < 2; ++p)
      *reinterpret_cast<f4*>(row + 64 * p + 4 * l16) = f4{w[4 * p], w[4 * p + 1], w[4 * p + 2], w[4 * p + 3]};
  }
}

// 16 rows of the left operand times the wave's 16 columns of the state; a lane gets
// rows 4 (lane / 16) + e of column lane % 16.
template <bool HALF, typename T, int N, int RUN>
__device__ __forceinline__ f4 product(const float* rows, const float* sizes, const T (&S)[N][RUN]) {
  const int lane = threadIdx.x % 64, quarter = lane / 16;
  f4 hi = {0, 0, 0, 0};
  if constexpr (HALF) {
    f4 lo = {0, 0, 0, 0};
    const _Float16* from = reinterpret_cast<const _Float16*>(rows + (lane % 16) * kLd) + 8 * quarter;
#pragma unroll
    for (int kk = 0; kk < N; ++kk) {
      h8 s;
#pragma unroll
      for (int j = 0; j < 8; ++j) s[j] = S[kk][j];
      hi = __builtin_amdgcn_mfma_f32_16x16x32_f16(*reinterpret_cast<const h8*>(from + 32 * kk), s, hi, 0, 0, 0);
      lo = __builtin_amdgcn_mfma_f32_16x16x32_f16(*reinterpret_cast<const h8*>(from + 128 + 32 * kk), s, lo, 0, 0, 0);
    }
    const f4 size = *reinterpret_cast<const f4*>(sizes + 4 * quarter);
#pragma unroll
    for (int e = 0; e < 4; ++e) hi[e] = fmaf(lo[e], 0x1p-11f, hi[e]) * size[e];
  } else {
    const float* from = rows + (lane % 16) * kLd + 4 * quarter;
#pragma unroll
    for (int kk = 0; kk < N; ++kk) {
      const f4 x = *reinterpret_cast<const f4*>(from + 16 * kk);
#pragma unroll
      for (int e = 0; e < 4; ++e) hi = __builtin_amdgcn_mfma_f32_16x16x4f32(x[e], S[kk][e], hi, 0, 0, 0);
    }
  }
  return hi;
}

// What a node takes from a node above it: a k_i . k_j and a q_i . k_j.
using Pair = f2;

constexpr int kTreeThreads = 512;

// Node i's pairs start at a multiple of 4, behind those of the nodes before it, of
// which node m has at most m.
KDA_HD constexpr int first_pair(int i) {
  return i < 1 ? 0 : 4 * ((i - 1) / 4 + 1) * (2 * ((i - 1) / 4) + (i - 1) % 4);
}
// LDS for nb nodes: keys and decays, then the decayed vectors as operands, then
// right-hand sides (which become beta u) and the queries' products; pairs, and
// their j.
constexpr int tree_rows_bytes(int nb) { return 2 * nb * kLd * 4; }
constexpr int tree_lds_bytes(int nb) { return tree_rows_bytes(nb) + 9 * first_pair(nb + 1); }

// A workgroup for a request and head; nb: its places for nodes, a multiple of 16.
// Sixteen lanes a node up to the products, 32 PER nodes in all; there a wave has 16
// value columns, in the solve 64 and four nodes.  COLS 64: a workgroup has half a
// head's columns, and half its waves the keys' products, half the queries'.
// Bound by its phases, each of which waits for the one before it (loads, the pairs up
// the tree, products, the solve level by level): two workgroups a compute unit run
// them beside each other, up to 48 nodes (with more, 89 KB of LDS leave room for one: 64
// trees of 48 nodes 39 us, of 56 57).  The state comes in 32-byte pieces of fp16, 64 of
// fp32, in front of the rest.  64 ragged trees of up to 48 nodes, 12 heads, fp16 states: 30.9
// us, 72 MB, 2.3 TB/s of the 6.5 that a streaming copy reaches (26.8 with all of it in the
// caches; 87 one node after the other); fp32 states 43.9; one tree of 13 nodes, fp32, 7.8.
template <int DT, int PER, int COLS>
__global__ __launch_bounds__(kTreeThreads, 4) void kda_tree_kernel(TreeArgs a, int nb) {
  constexpr int GROUPS = kTreeThreads / 16;
  constexpr int TILES = 2 * PER;  // of 16 nodes
  constexpr bool HALF = DT == KDA_F16;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  float* x_sh = reinterpret_cast<float*>(lds);
  Pair* pair_sh = reinterpret_cast<Pair*>(lds + tree_rows_bytes(nb));
  uint8_t* from_sh = reinterpret_cast<uint8_t*>(pair_sh + first_pair(nb + 1));
  __shared__ uint64_t path_sh[64];
  __shared__ __attribute__((aligned(16))) float size_sh[128];  // HALF: the operand's rows' powers of two
  // nodes level by level (those with as many above them): beta, q_i . k_i, i, the
  // place of its pairs
  __shared__ f4 node_sh[64];

  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  constexpr int PARTS = 128 / COLS;
  const int c0 = blockIdx.x % PARTS * COLS, h = blockIdx.x / PARTS % a.H, r = blockIdx.x / PARTS / a.H;
  const int slot = a.init_ids[r];
  const Nodes t = nodes_of(a.cu, r, a.n_tokens);
  if (t.n == 0) return;
  const int64_t step = static_cast<int64_t>(a.H) * 128;              // between nodes
  const int64_t row0 = t.n0 * step + static_cast<int64_t>(h) * 128;  // node 0's
  const bool fits = t.n <= a.max_nodes, placed = slot >= 0 && slot < a.n_slots;
  const int n = fits ? t.n : 0;

  // -- everything is asked for before anything is waited for: parents, gates,
  // nodes (channels 4 l16.. and 64 + 4 l16.. of a lane), the state
  const int parent = lane < n ? a.parents[t.n0 + lane] : -1;
  const float gate = lane < n ? a.b[(t.n0 + lane) * a.H + h] : 0.0f;
  const int l16 = tid % 16;
  f4 x[PER][2], y[PER][2], z[PER][2];
  // a wave's four nodes of a share; without one of the tree it passes it by
  const auto has = [&](int m) __attribute__((always_inline)) { return 4 * wave + GROUPS * m < n; };
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    if (!has(m)) break;
    const int i = tid / 16 + GROUPS * m;
    const int64_t at = row0 + (i < n ? i : 0) * step + 4 * l16;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      x[m][p] = *reinterpret_cast<const f4*>(a.k + at + 64 * p);
      y[m][p] = *reinterpret_cast<const f4*>(a.q + at + 64 * p);
      z[m][p] = *reinterpret_cast<const f4*>(a.g + at + 64 * p);
    }
  }
  // the wave's 16 columns, one a lane: as they go into the products, rows 16 kk + 4
  // quarter + j of fp32, 32 kk + 8 quarter + j of fp16
  const int quarter = lane / 16, col = 16 * (wave % (COLS / 16)) + lane % 16;
  const bool keys = COLS == 128 || wave < 4, queries = COLS == 128 || wave >= 4;  // this wave's products
  const Stored<DT>* S0 =
      static_cast<const Stored<DT>*>(a.pool) + (static_cast<int64_t>(placed ? slot : 0) * a.H + h) * 128 * 128 + c0 + col;
  constexpr int RUN = HALF ? 8 : 4;
  Stored<DT> S[128 / (4 * RUN)][RUN];
#pragma unroll
  for (int kk = 0; kk < 128 / (4 * RUN); ++kk)
#pragma unroll
    for (int j = 0; j < RUN; ++j) S[kk][j] = S0[(4 * RUN * kk + RUN * quarter + j) * 128];
  __builtin_amdgcn_sched_barrier(0);

  bool bad;
  const uint64_t above = tree_paths(parent, n, &bad);
  if (!fits || bad || !placed) {
    for (int64_t i = tid; i < static_cast<int64_t>(t.n) * COLS; i += kTreeThreads)
      a.out[row0 + i / COLS * step + c0 + i % COLS] = __builtin_nanf("");
    return;
  }
  const int depth_of = lane < n ? __popcll(above) - 1 : -1;
  const float beta = 1.0f / (1.0f + expf(-gate));
  if (wave == 0) path_sh[lane] = above;
  int rank = 0;  // of lane's node, among the levels
  for (int level = 0, before = 0; before < n; ++level) {
    const uint64_t same = __ballot(depth_of == level);
    if (depth_of == level) rank = before + __builtin_amdgcn_mbcnt_hi(same >> 32, __builtin_amdgcn_mbcnt_lo(same, 0));
    before += __popcll(same);
  }

  // -- lengths, decays
  float wk[PER][8], wq[PER][8];
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    if (!has(m)) break;
    const int i = tid / 16 + GROUPS * m;
    float kk = 0.0f, qq = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      kk = fmaf(x[m][e / 4][e % 4], x[m][e / 4][e % 4], kk);
      qq = fmaf(y[m][e / 4][e % 4], y[m][e / 4][e % 4], qq);
    }
    const float kn = __builtin_amdgcn_rsqf(sum16(kk) + 1e-6f), qn = __builtin_amdgcn_rsqf(sum16(qq) + 1e-6f);
    float dot = 0.0f;
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[m][p][e] *= kn;
        y[m][p][e] *= qn;
        z[m][p][e] = exp_near(z[m][p][e]);
        dot = fmaf(x[m][p][e], y[m][p][e], dot);
        wk[m][4 * p + e] = x[m][p][e] * z[m][p][e];
        wq[m][4 * p + e] = y[m][p][e] * z[m][p][e];
      }
    dot = sum16(dot);
    const int place = __shfl(rank, i % 64);
    const float mine = __shfl(beta, i % 64);
    if (i < n) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        *reinterpret_cast<f4*>(x_sh + i * kLd + 64 * p + 4 * l16) = x[m][p];
        *reinterpret_cast<f4*>(x_sh + (nb + i) * kLd + 64 * p + 4 * l16) = z[m][p];
      }
      if (l16 == 0) node_sh[place] = f4{mine, dot, __int_as_float(i), __int_as_float(first_pair(i))};
    }
  }
  __syncthreads();

  // -- up the tree: at each node above, the products with its key, then its decay.
  // A path's nodes are the bits of a word, the lowest node the highest bit.
  uint64_t way[PER];
  int at[PER];
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    const int i = tid / 16 + GROUPS * m;
    way[m] = i < n ? path_sh[i] & ~(1ull << i) : 0;
    at[m] = first_pair(i);
  }
  for (;;) {
    uint64_t any = 0;
#pragma unroll
    for (int m = 0; m < PER; ++m) any |= way[m];
    if (__ballot(any != 0) == 0) break;
#pragma unroll
    for (int m = 0; m < PER; ++m) {
      if (!has(m)) break;
      const int j = way[m] == 0 ? 0 : 63 - __builtin_clzll(way[m]);
      f4 key[2], dec[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        key[p] = *reinterpret_cast<const f4*>(x_sh + j * kLd + 64 * p + 4 * l16);
        dec[p] = *reinterpret_cast<const f4*>(x_sh + (nb + j) * kLd + 64 * p + 4 * l16);
      }
      f2 c = {0.0f, 0.0f}, d = {0.0f, 0.0f};
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c[e % 2] = fmaf(wk[m][e], key[e / 4][e % 4], c[e % 2]);
        d[e % 2] = fmaf(wq[m][e], key[e / 4][e % 4], d[e % 2]);
      }
      const float cs = sum16(c[0] + c[1]), ds = sum16(d[0] + d[1]);
      if (way[m] != 0) {
        if (l16 == 0) {
          pair_sh[at[m]] = Pair{cs, ds};
          from_sh[at[m]] = static_cast<uint8_t>(j);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          wk[m][e] *= dec[e / 4][e % 4];
          wq[m][e] *= dec[e / 4][e % 4];
        }
        way[m] &= ~(1ull << j);
        ++at[m];
      }
    }
  }
  // (pairs come in fours: nothing of the node's own row behind the last)
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    const int i = tid / 16 + GROUPS * m, none = -at[m] & 3;
    if (i < n && l16 < none) {
      pair_sh[at[m] + l16] = Pair{0.0f, 0.0f};
      from_sh[at[m] + l16] = static_cast<uint8_t>(i);
    }
  }
  __syncthreads();
  // -- the decayed vectors as rows of the left operand: 16 nodes' keys, then their
  // queries (what lies in rows of no node comes out in rows of no node)
  const int tiles = (n + 15) / 16;
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    const int i = tid / 16 + GROUPS * m;
    if (has(m)) {
      const int to = 32 * (i / 16) + i % 16;
      put_row<HALF>(x_sh + to * kLd, size_sh + to, wk[m]);
      put_row<HALF>(x_sh + (to + 16) * kLd, size_sh + to + 16, wq[m]);
    }
  }
  // (the values are on their way while the products run)
  float v[TILES][4];
#pragma unroll
  for (int m = 0; m < TILES; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * m + 4 * quarter + e;
      if (keys) v[m][e] = a.v[row0 + (i < n ? i : 0) * step + c0 + col];
    }
  __syncthreads();

  // -- products with the state: a lane gets its column of nodes 4 quarter + e of a tile
  f4 pk[TILES], pq[TILES];
#pragma unroll
  for (int m = 0; m < TILES; ++m)
    if (m < tiles) {
      if (keys) pk[m] = product<HALF>(x_sh + 32 * m * kLd, size_sh + 32 * m, S);
      if (queries) pq[m] = product<HALF>(x_sh + (32 * m + 16) * kLd, size_sh + 32 * m + 16, S);
    }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < TILES; ++m)
    if (m < tiles)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * m + 4 * quarter + e;
        if (keys) x_sh[i * kLd + col] = v[m][e] - pk[m][e];
        if (queries) x_sh[(nb + i) * kLd + col] = pq[m][e];
      }

  // -- the solve and the read-outs, level after level.  A wave takes 64 columns, four a
  // lane, and each quarter of it a node, so eight waves take 16 (32) nodes of a level
  // at once; up to four nodes below level 4 have a wave's quarters share each one's sum.
  __syncthreads();
  const int c4 = 64 * (wave % (COLS / 64)) + 4 * (lane % 16), team = wave / (COLS / 64);
  constexpr int TURN = 4 * (kTreeThreads / 64) / (COLS / 64);
  char* const out = reinterpret_cast<char*>(a.out + row0 + c0 + c4);
  const uint32_t out_step = static_cast<uint32_t>(4 * step);  // (64 of them are less than 2^30)
  float* const x_col = x_sh + c4;
  const auto solve = [&](int level, int at, bool some, int part, auto share) __attribute__((always_inline)) {
    constexpr bool SHARE = decltype(share)::value;
    const f4 node = node_sh[at];
    float* row = x_col + __float_as_int(node[2]) * kLd;
    int pairs = __float_as_int(node[3]) + 4 * part;
    f4 u = *reinterpret_cast<const f4*>(row), o = *reinterpret_cast<const f4*>(row + nb * kLd);
    if (SHARE && part > 0) u = o = f4{0, 0, 0, 0};
    const auto quad = [&]() __attribute__((always_inline)) {
      const uint32_t from = *reinterpret_cast<const uint32_t*>(from_sh + pairs);
      const f4 p0 = *reinterpret_cast<const f4*>(pair_sh + pairs), p1 = *reinterpret_cast<const f4*>(pair_sh + pairs + 2);
      f4 y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) y[q] = *reinterpret_cast<const f4*>(x_col + ((from >> (8 * q)) & 0xFF) * kLd);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float c = q < 2 ? p0[2 * (q % 2)] : p1[2 * (q % 2)], d = q < 2 ? p0[2 * (q % 2) + 1] : p1[2 * (q % 2) + 1];
          u[k] = fmaf(-c, y[q][k], u[k]);
          o[k] = fmaf(d, y[q][k], o[k]);
        }
    };
    if constexpr (SHARE) {
      for (int e = 4 * part; e < level; e += 16, pairs += 16) quad();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        u[k] = sum_xor32(sum_xor16(u[k]));
        o[k] = sum_xor32(sum_xor16(o[k]));
      }
    } else {
      for (int e = 0; e < level; e += 4, pairs += 4) quad();
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      u[k] *= node[0];
      o[k] = a.scale * fmaf(node[1], u[k], o[k]);
    }
    if (some) {
      *reinterpret_cast<f4*>(row) = u;
      *reinterpret_cast<f4*>(out + __float_as_int(node[2]) * out_step) = o;
    }
  };
  for (int level = 0, place = 0; place < n; ++level) {
    if (level > 0) __syncthreads();
    const int end = place + __popcll(__ballot(depth_of == level));
    if (level > 4 && end - place <= 4) {
      if (place + team < end) solve(level, place + team, quarter == 0, quarter, std::true_type{});
    } else {
      for (int at = place + 4 * team; at < end; at += TURN) {
        const bool some = at + quarter < end;
        solve(level, some ? at + quarter : at, some, 0, std::false_type{});
      }
    }
    place = end;
  }
}

// ---------------------------------------------------------------------------
// Paths
// ---------------------------------------------------------------------------

// A workgroup for a request and head: 32 value columns a wave, 16 bytes of them
// and R key rows a lane, so that a node's column sums stay inside the wave and the
// nodes follow each other without a barrier.  The nodes' keys, decays and values
// are staged sixteen at a time.  A batch is bound by its one round of workgroups, which
// load, compute and store in step (64 paths of up to 8 nodes, 12 heads, fp16: 15.7 us, 3.4
// TB/s, reading and writing; kda_decode_step moves these states in 9.4), one path by
// latency (5.1).
// Nodes eight at a time, states updated by matrix products: 41 -> 36 us for up to 20
// nodes of fp16 states, but fp32 47 -> 59 and 8 nodes no faster; not taken.
template <int DT>
__global__ __launch_bounds__(256) void kda_path_kernel(PathArgs a) {
  using T = Stored<DT>;
  constexpr int C = 16 / static_cast<int>(sizeof(T));  // columns a lane
  constexpr int LPR = 32 / C;                          // lanes of a state row
  constexpr int R = 128 * LPR / 64;                    // rows a lane
  constexpr int STAGE = 16;
  using Vec = T __attribute__((ext_vector_type(C)));
  __shared__ __attribute__((aligned(16))) float k_sh[STAGE][128];
  __shared__ __attribute__((aligned(16))) float a_sh[STAGE][128];
  __shared__ __attribute__((aligned(16))) float v_sh[STAGE][128];
  __shared__ float b_sh[STAGE];

  const int tid = threadIdx.x, lane = tid % 64, wave = tid / 64;
  const int h = blockIdx.x % a.H, r = blockIdx.x / a.H;
  const int from = a.init_ids[r], to = a.dst_ids[r], len = a.lens[r];
  const Nodes t = nodes_of(a.cu, r, a.n_tokens);
  const int node = lane < len && lane < a.max_path ? a.path[static_cast<int64_t>(r) * a.max_path + lane] : 0;
  const bool bad = len < 0 || len > a.max_path || from < 0 || from >= a.n_slots || to < 0 || to >= a.n_slots;
  if (bad || __ballot(lane < len && (node < 0 || node >= t.n)) != 0) return;

  const int col = 32 * wave + C * (lane % LPR), row = R * (lane / LPR);
  const int64_t block = static_cast<int64_t>(128) * 128, place = static_cast<int64_t>(row) * 128 + col;
  const T* src = static_cast<const T*>(a.pool) + (static_cast<int64_t>(from) * a.H + h) * block + place;
  T* dst = static_cast<T*>(a.pool) + (static_cast<int64_t>(to) * a.H + h) * block + place;
  Vec raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i] = __builtin_nontemporal_load(reinterpret_cast<const Vec*>(src + i * 128));
  float S[R][C];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int c = 0; c < C; ++c) S[i][c] = static_cast<float>(raw[i][c]);

  for (int e0 = 0; e0 < len; e0 += STAGE) {
    if (e0 > 0) __syncthreads();
    {
      const int e = e0 + tid / 16, l16 = tid % 16;
      const int which = __shfl(node, e % 64);
      if (e < len) {
        const int64_t at = ((t.n0 + which) * a.H + h) * 128 + 4 * l16;
        f4 x[2], z[2];
        float kk = 0.0f;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          x[p] = *reinterpret_cast<const f4*>(a.k + at + 64 * p);
          z[p] = *reinterpret_cast<const f4*>(a.g + at + 64 * p);
          *reinterpret_cast<f4*>(&v_sh[tid / 16][4 * l16 + 64 * p]) = *reinterpret_cast<const f4*>(a.v + at + 64 * p);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) kk = fmaf(x[i / 4][i % 4], x[i / 4][i % 4], kk);
        const float kn = __builtin_amdgcn_rsqf(sum16(kk) + 1e-6f);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[p][i] *= kn;
            z[p][i] = exp_near(z[p][i]);
          }
          *reinterpret_cast<f4*>(&k_sh[tid / 16][4 * l16 + 64 * p]) = x[p];
          *reinterpret_cast<f4*>(&a_sh[tid / 16][4 * l16 + 64 * p]) = z[p];
        }
        if (l16 == 0) b_sh[tid / 16] = 1.0f / (1.0f + expf(-a.b[(t.n0 + which) * a.H + h]));
      }
    }
    __syncthreads();
    const int some = len - e0 < STAGE ? len - e0 : STAGE;
    for (int e = 0; e < some; ++e) {
      float w[C] = {};
#pragma unroll
      for (int i = 0; i < R; i += 4) {
        const f4 dec = *reinterpret_cast<const f4*>(&a_sh[e][row + i]);
        const f4 key = *reinterpret_cast<const f4*>(&k_sh[e][row + i]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < C; ++c) {
            S[i + j][c] *= dec[j];
            w[c] = fmaf(key[j], S[i + j][c], w[c]);
          }
      }
      const float b = b_sh[e];
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if constexpr (LPR == 4) w[c] = sum_xor4(w[c]);
        w[c] = sum_xor32(sum_xor16(sum_xor8(w[c])));
        w[c] = b * (v_sh[e][col + c] - w[c]);
      }
#pragma unroll
      for (int i = 0; i < R; i += 4) {
        const f4 key = *reinterpret_cast<const f4*>(&k_sh[e][row + i]);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < C; ++c) S[i + j][c] = fmaf(key[j], w[c], S[i + j][c]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i) {
    Vec x;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float y = S[i][c];
      asm volatile("" : "+v"(y));  // the last multiply-add and the narrowing stay two roundings
      x[c] = static_cast<T>(y);
    }
    __builtin_nontemporal_store(x, reinterpret_cast<Vec*>(dst + i * 128));
  }
}

int status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH; }
bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int DT>
hipError_t launch_tree(const TreeArgs& a, hipStream_t st) {
  const int nb = a.max_nodes < 1 ? 16 : (a.max_nodes + 15) / 16 * 16;
  const int64_t units = static_cast<int64_t>(a.n_req) * a.H;
  const auto launch = [&](auto kernel, int parts) {
    // (more than 64 KiB of LDS has to be asked for)
    hipError_t e = hipSuccess;
    if (tree_lds_bytes(nb) > 65536)
      e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                              tree_lds_bytes(nb));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(units * parts)), dim3(kTreeThreads), tree_lds_bytes(nb), st, a,
                       nb);
    return hipGetLastError();
  };
  // Half heads where whole ones would leave half the chip idle (13 nodes, fp32, 12 units
  // of a request and head: 8.3 -> 7.5 us; 24 nodes, 120 units, 11.3 -> 10.4; 144 units
  // 12.4 -> 13.4, 768 of fp16 27.4 -> 35.8).  Up to 32 nodes a node has one turn's registers
  // (24 nodes, 480 units, fp16: 14.9 us, 15.3 with the larger form).
  const bool half = units <= 128;
  if (nb <= 32) return half ? launch(kda_tree_kernel<DT, 1, 64>, 2) : launch(kda_tree_kernel<DT, 1, 128>, 1);
  return half ? launch(kda_tree_kernel<DT, 2, 64>, 2) : launch(kda_tree_kernel<DT, 2, 128>, 1);
}

// threads of a launch stay below 2^32 for the widest workgroup
bool grid_fits(int32_t n_req, int32_t H) { return static_cast<int64_t>(n_req) * H <= INT32_MAX / 512; }

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int kda_decode_tree(const kda_pool* pool, const int32_t* init_slot_ids, const int32_t* cu_seqlens,
                               const int32_t* parents, const float* q, const float* k, const float* v,
                               const float* g, const float* b, float* out, int32_t n_req, int64_t n_tokens,
                               int32_t max_nodes, kda_dtype state_dtype, float scale, void* stream) {
  const int rc = tree_check(pool, n_req, n_tokens, state_dtype);
  if (rc != KDA_OK) return rc;
  if (max_nodes < 0 || max_nodes > kMaxNodes) return KDA_ERR_ROWS;
  if (n_req == 0 || n_tokens == 0) return KDA_OK;
  if (init_slot_ids == nullptr || cu_seqlens == nullptr || parents == nullptr || q == nullptr || k == nullptr ||
      v == nullptr || g == nullptr || b == nullptr || out == nullptr)
    return KDA_ERR_NULL;
  if (!std::isfinite(scale) || !grid_fits(n_req, pool->H)) return KDA_ERR_ARG;
  if (!aligned(pool->base, 16) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 16) ||
      !aligned(out, 16) || !aligned(b, 4) || !aligned(init_slot_ids, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(parents, 4))
    return KDA_ERR_ALIGN;
  TreeArgs a;
  a.pool = pool->base;
  a.init_ids = init_slot_ids;
  a.cu = cu_seqlens;
  a.parents = parents;
  a.q = q;
  a.k = k;
  a.v = v;
  a.g = g;
  a.b = b;
  a.out = out;
  a.n_tokens = n_tokens;
  a.n_req = n_req;
  a.H = pool->H;
  a.n_slots = pool->n_slots;
  a.max_nodes = max_nodes;
  a.scale = scale;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return status(state_dtype == KDA_F32 ? launch_tree<KDA_F32>(a, st) : launch_tree<KDA_F16>(a, st));
}

extern "C" int kda_decode_path(const kda_pool* pool, const int32_t* init_slot_ids, const int32_t* dst_slot_ids,
                               const int32_t* cu_seqlens, const int32_t* path, int32_t max_path,
                               const int32_t* path_lens, const float* k, const float* v, const float* g,
                               const float* b, int32_t n_req, int64_t n_tokens, kda_dtype state_dtype,
                               void* stream) {
  const int rc = tree_check(pool, n_req, n_tokens, state_dtype);
  if (rc != KDA_OK) return rc;
  if (max_path < 1 || max_path > kMaxNodes) return KDA_ERR_ROWS;
  if (n_req > pool->n_slots) return KDA_ERR_SLOT;
  if (n_req == 0) return KDA_OK;
  if (init_slot_ids == nullptr || cu_seqlens == nullptr || path == nullptr || path_lens == nullptr) return KDA_ERR_NULL;
  if (n_tokens > 0 && (k == nullptr || v == nullptr || g == nullptr || b == nullptr)) return KDA_ERR_NULL;
  if (!grid_fits(n_req, pool->H)) return KDA_ERR_ARG;
  if (!aligned(pool->base, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(g, 16) || !aligned(b, 4) ||
      !aligned(init_slot_ids, 4) || !aligned(dst_slot_ids, 4) || !aligned(cu_seqlens, 4) || !aligned(path, 4) ||
      !aligned(path_lens, 4))
    return KDA_ERR_ALIGN;
  PathArgs a;
  a.pool = pool->base;
  a.init_ids = init_slot_ids;
  a.dst_ids = dst_slot_ids != nullptr ? dst_slot_ids : init_slot_ids;
  a.cu = cu_seqlens;
  a.path = path;
  a.lens = path_lens;
  a.k = k;
  a.v = v;
  a.g = g;
  a.b = b;
  a.n_tokens = n_tokens;
  a.n_req = n_req;
  a.H = pool->H;
  a.n_slots = pool->n_slots;
  a.max_path = max_path;
  const auto kernel = state_dtype == KDA_F32 ? kda_path_kernel<KDA_F32> : kda_path_kernel<KDA_F16>;
  hipLaunchKernelGGL(kernel, dim3(static_cast<uint32_t>(n_req) * pool->H), dim3(256), 0,
                     static_cast<hipStream_t>(stream), a);
  return status(hipGetLastError());
}
