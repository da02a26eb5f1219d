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

using f16v = float __attribute__((ext_vector_type(16)));

// sum over 16 lanes, in each of them
__device__ __forceinline__ float sum16(float x) { return sum_xor8(sum_xor4(sum_xor2(sum_xor1(x)))); }

template <int DT>
using Stored = std::conditional_t<DT == KDA_F32, float, _Float16>;

constexpr int kLd = 132;  // floats between rows in LDS: neighbouring rows start 4 banks apart

// ---------------------------------------------------------------------------
// Trees
// ---------------------------------------------------------------------------

// What node i takes from a node on its path.
struct Pair {
  float c, d;  // a k_i . k_j and a q_i . k_j
  int row;     // j's place in LDS
  int pad;
};

template <int NB>
constexpr int tree_threads() { return NB == 64 ? 512 : 256; }

// A workgroup for a request and head, up to NB nodes.
template <int DT, int NB>
__global__ __launch_bounds__(tree_threads<NB>()) void kda_tree_kernel(TreeArgs a) {
  constexpr int NT = tree_threads<NB>(), NW = NT / 64;
  constexpr int GROUPS = NT / 16, PER = NB / GROUPS;  // 16 lanes a node, PER nodes each
  constexpr int SETS = NW / 4;                        // waves that share 32 columns
  constexpr int TILES = NB / 16 / SETS;               // 16-node tiles of a wave
  constexpr int SOLVE = NT / 128;                     // lanes of a column in the solve
  constexpr int PAIRS = NB * (NB + 1) / 2;
  // first the keys (rows 0..NB) and decays; then the 2 NB decayed vectors; then
  // a row of right-hand sides for each node, which become beta u
  __shared__ __attribute__((aligned(16))) float x_sh[2 * NB * kLd];
  __shared__ __attribute__((aligned(16))) Pair pair_sh[PAIRS];
  __shared__ int parent_sh[64];

  const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
  const int h = blockIdx.x % a.H, r = blockIdx.x / a.H;
  const Nodes t = nodes_of(a.cu, r, a.n_tokens);
  if (t.n == 0) return;
  const int slot = a.init_ids[r];
  const int64_t step = static_cast<int64_t>(a.H) * 128;           // between nodes
  const int64_t row0 = t.n0 * step + static_cast<int64_t>(h) * 128;  // node 0's
  const bool fits = t.n <= NB && t.n <= a.max_nodes;
  const int n = fits ? t.n : 0;
  const int parent = lane < n ? a.parents[t.n0 + lane] : -1;
  bool bad;
  const uint64_t above = tree_paths(parent, n, &bad);
  if (!fits || bad || slot < 0 || slot >= a.n_slots) {
    for (int64_t i = tid; i < static_cast<int64_t>(t.n) * 128; i += NT)
      a.out[row0 + i / 128 * step + i % 128] = __builtin_nanf("");
    return;
  }
  // places of the nodes' pairs: lane i has node i's first, and their number
  const int count = lane < n ? __popcll(above) : 0;
  int first = count;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const int y = __shfl_up(first, m);
    first = lane >= m ? first + y : first;
  }
  first -= count;
  if (wave == 0) parent_sh[lane] = parent;
  const float beta = lane < n ? 1.0f / (1.0f + expf(-a.b[(t.n0 + lane) * a.H + h])) : 0.0f;

  // -- the state's columns 32 (wave % 4).., one a lane: rows 8 kk + 4 half + j
  const int half = lane / 32, col = 32 * (wave % 4) + lane % 32;
  const Stored<DT>* S0 = static_cast<const Stored<DT>*>(a.pool) + (static_cast<int64_t>(slot) * a.H + h) * 128 * 128;
  float S[64];
#pragma unroll
  for (int i = 0; i < 64; ++i) S[i] = static_cast<float>(S0[(8 * (i / 4) + 4 * half + i % 4) * 128 + col]);

  // -- nodes: 16 lanes each, channels 4 l16.. and 64 + 4 l16..
  const int l16 = tid % 16;
  float wk[PER][8], wq[PER][8];
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    const int i = tid / 16 + GROUPS * m;
    const int64_t at = row0 + (i < n ? i : 0) * step + 4 * l16;
    f4 x[2], y[2], z[2];
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      x[p] = *reinterpret_cast<const f4*>(a.k + at + 64 * p);
      y[p] = *reinterpret_cast<const f4*>(a.q + at + 64 * p);
      z[p] = *reinterpret_cast<const f4*>(a.g + at + 64 * p);
    }
    float kk = 0.0f, qq = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      kk = fmaf(x[e / 4][e % 4], x[e / 4][e % 4], kk);
      qq = fmaf(y[e / 4][e % 4], y[e / 4][e % 4], qq);
    }
    const float kn = 1.0f / sqrtf(sum16(kk) + 1e-6f), qn = 1.0f / sqrtf(sum16(qq) + 1e-6f);
    float dot = 0.0f;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      f4 dec;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[p][e] *= kn;
        y[p][e] *= qn;
        dec[e] = expf(z[p][e]);
        dot = fmaf(x[p][e], y[p][e], dot);
        wk[m][4 * p + e] = x[p][e] * dec[e];
        wq[m][4 * p + e] = y[p][e] * dec[e];
      }
      *reinterpret_cast<f4*>(x_sh + i * kLd + 64 * p + 4 * l16) = x[p];
      *reinterpret_cast<f4*>(x_sh + (NB + i) * kLd + 64 * p + 4 * l16) = dec;
    }
    dot = sum16(dot);
    const int at_pair = __shfl(first, i % 64);
    if (l16 == 0 && i < n) pair_sh[at_pair] = Pair{0.0f, dot, i * kLd, 0};
  }
  __syncthreads();

  // -- up the tree: at each node above, the products with its key, then its decay
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    const int i = tid / 16 + GROUPS * m;
    int at_pair = __shfl(first, i % 64) + 1;
    int j = i < n ? parent_sh[i] : -1;
    while (__ballot(j >= 0) != 0) {
      const int from = j < 0 ? 0 : j;
      float c = 0.0f, d = 0.0f;
      f4 key[2], dec[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        key[p] = *reinterpret_cast<const f4*>(x_sh + from * kLd + 64 * p + 4 * l16);
        dec[p] = *reinterpret_cast<const f4*>(x_sh + (NB + from) * kLd + 64 * p + 4 * l16);
      }
      const int next = parent_sh[from];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        c = fmaf(wk[m][e], key[e / 4][e % 4], c);
        d = fmaf(wq[m][e], key[e / 4][e % 4], d);
      }
      c = sum16(c);
      d = sum16(d);
      if (j >= 0) {
        if (l16 == 0) pair_sh[at_pair] = Pair{c, d, j * kLd, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          wk[m][e] *= dec[e / 4][e % 4];
          wq[m][e] *= dec[e / 4][e % 4];
        }
      }
      ++at_pair;
      j = j < 0 ? -1 : next;
    }
  }
  __syncthreads();
  // -- the decayed vectors as rows of the left operand: 32 of a tile, 16 nodes'
  // keys, then their queries
#pragma unroll
  for (int m = 0; m < PER; ++m) {
    const int i = tid / 16 + GROUPS * m;
    float* to = x_sh + (32 * (i / 16) + i % 16) * kLd + 4 * l16;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const bool some = i < n;
      f4 x, y;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = some ? wk[m][4 * p + e] : 0.0f, y[e] = some ? wq[m][4 * p + e] : 0.0f;
      *reinterpret_cast<f4*>(to + 64 * p) = x;
      *reinterpret_cast<f4*>(to + 16 * kLd + 64 * p) = y;
    }
  }
  __syncthreads();

  // -- products with the state.  Result e of a lane: row 8 (e / 4) + 4 half + e % 4
  // of the tile, so e < 8 is a node's key and e + 8 its query.
  const int set = wave / 4;
  f16v acc[TILES];
#pragma unroll
  for (int m = 0; m < TILES; ++m) {
    const int tile = SETS * m + set;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[m][e] = 0.0f;
    if (16 * tile < n) {
      const float* from = x_sh + (32 * tile + lane % 32) * kLd + 4 * half;
#pragma unroll
      for (int kk = 0; kk < 16; ++kk) {
        const f4 w = *reinterpret_cast<const f4*>(from + 8 * kk);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[m] = __builtin_amdgcn_mfma_f32_32x32x2f32(w[e], S[4 * kk + e], acc[m], 0, 0, 0);
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int m = 0; m < TILES; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = 16 * (SETS * m + set) + 8 * (e / 4) + 4 * half + e % 4;
      if (i < n) x_sh[i * kLd + col] = a.v[row0 + i * step + col] - acc[m][e];
    }
  __syncthreads();

  // -- the solve: SOLVE lanes a column share a node's sum, node after node
  {
    constexpr int COLS = 64 / SOLVE;
    const int mine = COLS * wave + lane % COLS, part = lane / COLS;
    for (int i = 0; i < n; ++i) {
      const int at = __builtin_amdgcn_readlane(first, i), end = at + __builtin_amdgcn_readlane(count, i);
      float s = 0.0f;
      for (int e = at + 1 + part; e < end; e += SOLVE) s = fmaf(pair_sh[e].c, x_sh[pair_sh[e].row + mine], s);
      if constexpr (SOLVE == 4) s = sum_xor16(s);
      s = sum_xor32(s);
      const float b = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(beta), i));
      const float u = b * (x_sh[i * kLd + mine] - s);
      if (part == 0) x_sh[i * kLd + mine] = u;
    }
  }
  __syncthreads();

  // -- read-outs
#pragma unroll
  for (int m = 0; m < TILES; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = 16 * (SETS * m + set) + 8 * (e / 4) + 4 * half + e % 4;
      const int at = __shfl(first, i % 64), end = at + __shfl(count, i % 64);
      if (i < n) {
        float s = acc[m][8 + e];
        for (int p = at; p < end; ++p) s = fmaf(pair_sh[p].d, x_sh[pair_sh[p].row + col], s);
        a.out[row0 + i * step + col] = a.scale * s;
      }
    }
}

// ---------------------------------------------------------------------------
// Paths
// ---------------------------------------------------------------------------

// A workgroup for a request and head: 32 value columns a wave, 16 bytes of them
// and R key rows a lane, so that a node's column sums stay inside the wave and the
// nodes follow each other without a barrier.  The nodes' keys, decays and values
// are staged sixteen at a time.
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
        const float kn = 1.0f / sqrtf(sum16(kk) + 1e-6f);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x[p][i] *= kn;
            z[p][i] = expf(z[p][i]);
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
  const dim3 grid(static_cast<uint32_t>(a.n_req) * a.H);
  if (a.max_nodes <= 16)
    hipLaunchKernelGGL((kda_tree_kernel<DT, 16>), grid, dim3(tree_threads<16>()), 0, st, a);
  else if (a.max_nodes <= 32)
    hipLaunchKernelGGL((kda_tree_kernel<DT, 32>), grid, dim3(tree_threads<32>()), 0, st, a);
  else
    hipLaunchKernelGGL((kda_tree_kernel<DT, 64>), grid, dim3(tree_threads<64>()), 0, st, a);
  return hipGetLastError();
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
  const dim3 grid(static_cast<uint32_t>(n_req) * pool->H);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (state_dtype == KDA_F32)
    hipLaunchKernelGGL((kda_path_kernel<KDA_F32>), grid, dim3(256), 0, st, a);
  else
    hipLaunchKernelGGL((kda_path_kernel<KDA_F16>), grid, dim3(256), 0, st, a);
  return status(hipGetLastError());
}
