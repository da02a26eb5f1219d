// kda_verify.hip -- verification of drafted tokens on gfx950: rejection sampling
// along a tree from given random numbers.
//
// The walk needs single probabilities, two of them for a node, and the last row is
// summed and searched for the following token.  With a draft, a refused child that has
// a later sibling also needs the sum of what is left of its parent's row.  All of it
// is fp64: the chip adds doubles at half the rate of floats, far faster than the rows
// arrive, and a sum of a hundred thousand fp32 numbers is then off by less than 1e-13
// of itself, so that a draw is decided by the numbers and not by the order they are
// added in.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "kda_decode.h"
#include "kda_tree_device.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kVec = 8;  // entries a thread loads at once

template <int DT>
using Entry = std::conditional_t<DT == KDA_F32, float, uint16_t>;

// an entry as a weight: above 0, or 0
template <int DT>
__device__ __forceinline__ double weight(Entry<DT> e) {
  float x;
  if constexpr (DT == KDA_F32)
    x = e;
  else if constexpr (DT == KDA_F16)
    x = static_cast<float>(__builtin_bit_cast(_Float16, e));
  else
    x = __uint_as_float(static_cast<uint32_t>(e) << 16);
  return x > 0.0f ? static_cast<double>(x) : 0.0;
}

template <int DT>
__device__ __forceinline__ const Entry<DT>* row_of(const void* base, int64_t row, int64_t stride) {
  return static_cast<const Entry<DT>*>(base) + row * stride;
}

// kVec entries of a row of `vocab`, from `at` on; WHOLE: the row has as many
template <int DT, bool WHOLE>
__device__ __forceinline__ void load_run(const Entry<DT>* row, int64_t at, int vocab, Entry<DT> (&e)[kVec]) {
  if constexpr (WHOLE) {
    __builtin_memcpy(e, row + at, sizeof(e));
  } else {
#pragma unroll
    for (int i = 0; i < kVec; ++i) e[i] = at + i < vocab ? row[at + i] : Entry<DT>{};
  }
}

__device__ __forceinline__ double lane_double(double x, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// a wave's sum, the same in every lane
__device__ __forceinline__ double wave_sum(double x) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) x += __shfl_xor(x, m);
  return x;
}

// the same sum, in the same order, in every thread
__device__ __forceinline__ double block_sum(double x, double* sh) {
  x = wave_sum(x);
  if (threadIdx.x % 64 == 0) sh[threadIdx.x / 64] = x;
  __syncthreads();
  double s = 0.0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) s += sh[w];
  __syncthreads();
  return s;
}

// The weights that are left of a row after `tries` refusals: of entries
// [x0, x0 + N).  mass: M of refusal j in lane j, with a draft; without one
// `tokens` are the refused ones, lane by lane in `refused`.
template <int DT, bool DRAFT>
struct Left {
  const Entry<DT>* p;
  const Entry<DT>* q;
  int vocab, tries;
  double mass;
  int token;
  uint64_t refused;

  // kVec entries as they lie, of which those from x on count: at the end of a run
  // they begin before x
  struct Raw {
    Entry<DT> p[kVec], q[DRAFT ? kVec : 1];
    int64_t at;
    int skip;
  };
  // (nothing here depends on the row: the loads of a thread do not wait for each other)
  template <bool WHOLE, bool TRIED>
  __device__ __forceinline__ void load(int64_t x, int64_t end, Raw& raw) const {
    const int64_t last = end > kVec ? end - kVec : 0;
    raw.at = x < last ? x : last;
    raw.skip = x - raw.at < kVec ? static_cast<int>(x - raw.at) : kVec;
    load_run<DT, WHOLE>(p, raw.at, vocab, raw.p);
    if constexpr (TRIED && DRAFT) load_run<DT, WHOLE>(q, raw.at, vocab, raw.q);
  }
  // and what is left of them
  template <bool TRIED>
  __device__ __forceinline__ void weights(const Raw& raw, double (&f)[kVec]) const {
#pragma unroll
    for (int i = 0; i < kVec; ++i) f[i] = weight<DT>(raw.p[i]);
    if constexpr (TRIED && DRAFT) {
      for (int j = 0; j < tries; ++j) {
        const double m = lane_double(mass, j);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const double d = f[i] - m * weight<DT>(raw.q[i]);
          f[i] = d > 0.0 ? d : 0.0;
        }
      }
    } else if constexpr (TRIED) {
      for (uint64_t r = refused; r != 0; r &= r - 1) {
        const int64_t at = __builtin_amdgcn_readlane(token, __builtin_ctzll(r)) - raw.at;
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] = at == i ? 0.0 : f[i];
      }
    }
    if (__ballot(raw.skip != 0) != 0) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) f[i] = i < raw.skip ? 0.0 : f[i];
    }
  }

  // f(whole, tried) with constants for this row
  template <typename F>
  __device__ __forceinline__ auto as(F f) const {
    if (vocab < kVec) return f(std::false_type{}, std::true_type{});
    return tries > 0 ? f(std::true_type{}, std::true_type{}) : f(std::true_type{}, std::false_type{});
  }

  // a thread's share of the sum of entries [x0, x1), `threads` of them on it: four
  // loads in flight, the rest one by one
  __device__ __forceinline__ double share(int64_t x0, int64_t x1, int thread, int threads) const {
    return as([&](auto whole, auto tried) __attribute__((always_inline)) {
      constexpr bool WHOLE = decltype(whole)::value, TRIED = decltype(tried)::value;
      const int turn = threads * kVec;
      int64_t at = x0;
      double s = 0.0;
      const auto add = [&](auto ahead) __attribute__((always_inline)) {
        constexpr int AHEAD = decltype(ahead)::value;
        Raw raw[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) load<WHOLE, TRIED>(at + thread * kVec + i * turn, x1, raw[i]);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
          double f[kVec];
          weights<TRIED>(raw[i], f);
          s += ((f[0] + f[1]) + (f[2] + f[3])) + ((f[4] + f[5]) + (f[6] + f[7]));
        }
        at += AHEAD * turn;
      };
      if constexpr (WHOLE)
        while (at + 3 * turn < x1) add(std::integral_constant<int, 4>{});
      while (at < x1) add(std::integral_constant<int, 1>{});
      return s;
    });
  }
};

// A wave for each run of each request's last row.  All walk, so that none waits
// for another: lane i of every wave holds node i, the walk reads lanes.  Bound by HBM
// for many rows (64 chains of up to 8 over 100003 tokens, fp32, with a draft: 12.3 us for
// 51 MB, 4.2 TB/s), else by the loads that follow from each other: tables, the nodes'
// probabilities, the row (32 trees over 131072, bf16: 8.3; one request: 4.4).  Where trees
// have a draft, by the residual sums, which every workgroup of a request forms for
// itself over whole rows, all refusals of that node once more for each (fp32, 131072
// tokens: 8 trees of 12 nodes 83 us with the draw, 8 chains 11.6; all children of a node
// refused, 11 of them 0.47 ms, 63 10.7 ms).
template <int DT, bool DRAFT>
__global__ __launch_bounds__(kThreads) void kda_verify_walk_kernel(VerifyArgs a) {
  __shared__ double sh[kWaves];
  const int lane = threadIdx.x % 64;
  const int blocks = (a.runs + kWaves - 1) / kWaves;  // of a request
  const int r = blockIdx.x / blocks, run = blockIdx.x % blocks * kWaves + threadIdx.x / 64;
  const bool writes = run == 0;
  const Nodes t = nodes_of(a.cu, r, a.n_tokens);
  bool bad = t.n == 0 || t.n > kMaxNodes;
  const int n = bad ? 0 : t.n;
  const int parent = lane < n ? a.parents[t.n0 + lane] : -1;
  bad |= __ballot(lane < n && (parent < -1 || parent >= lane)) != 0;
  if (bad) {
    if (writes) {
      if (lane < a.max_path) a.path[static_cast<int64_t>(r) * a.max_path + lane] = -1;
      if (lane == 0) {
        a.lens[r] = 0;
        a.stops[r].last = -1;
      }
    }
    return;
  }
  const int token = lane < n ? a.tokens[t.n0 + lane] : -1;
  const float u = lane < n ? a.accept[t.n0 + lane] : 0.0f;
  double p = 0.0, q = 0.0;
  if (parent >= 0 && token >= 0 && token < a.vocab) {
    p = weight<DT>(row_of<DT>(a.target, t.n0 + parent, a.target_stride)[token]);
    if constexpr (DRAFT) q = weight<DT>(row_of<DT>(a.draft, t.n0 + parent, a.draft_stride)[token]);
  }

  Left<DT, DRAFT> left;
  left.vocab = a.vocab;
  left.token = token;
  left.mass = 0.0;
  int last = 0, length = 1;
  int way = lane == 0 ? 0 : -1;  // lane e: entry e of the path
  left.refused = 0;
  left.tries = 0;
  double mass = 1.0;
  uint64_t kids = __ballot(parent == 0);
  while (kids != 0 && length < a.max_path) {
    const int i = __builtin_ctzll(kids);
    kids &= kids - 1;
    const int x = __builtin_amdgcn_readlane(token, i);
    const double pu = lane_double(p, i), qu = lane_double(q, i);
    const double uu = static_cast<double>(__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(u), i)));
    double have = pu;
    if constexpr (DRAFT) {
      for (int j = 0; j < left.tries; ++j) {
        const double d = have - lane_double(left.mass, j) * qu;
        have = d > 0.0 ? d : 0.0;
      }
    } else {
      if ((__ballot(token == x) & left.refused) != 0) have = 0.0;
    }
    const bool yes = DRAFT ? uu * qu * mass < have : uu * mass < have;
    if (yes) {
      last = i;
      way = lane == length ? i : way;
      ++length;
      left.refused = 0;
      left.tries = 0;
      mass = 1.0;
      kids = __ballot(parent == i);
    } else {
      left.refused |= 1ull << i;
      if constexpr (DRAFT) {
        left.mass = lane == left.tries ? mass : left.mass;
        ++left.tries;
        if (kids != 0) {  // the next child's M: a sum of the whole row
          left.p = row_of<DT>(a.target, t.n0 + last, a.target_stride);
          left.q = row_of<DT>(a.draft, t.n0 + last, a.draft_stride);
          mass = block_sum(left.share(0, a.vocab, threadIdx.x, kThreads), sh);
        }
      } else {
        ++left.tries;
        mass -= have;
      }
    }
  }
  left.p = row_of<DT>(a.target, t.n0 + last, a.target_stride);
  left.q = DRAFT ? row_of<DT>(a.draft, t.n0 + last, a.draft_stride) : nullptr;
  if (writes) {
    if (lane < a.max_path) a.path[static_cast<int64_t>(r) * a.max_path + lane] = way;
    VerifyStop* s = a.stops + r;
    s->mass[lane] = left.mass;
    if (lane == 0) {
      a.lens[r] = length;
      s->refused = left.refused;
      s->last = last;
      s->tries = left.tries;
    }
  }
  if (run >= a.runs) return;
  const int64_t x0 = static_cast<int64_t>(run) * a.run;
  const int64_t x1 = x0 + a.run < a.vocab ? x0 + a.run : a.vocab;
  const double s = wave_sum(left.share(x0, x1, lane, 64));
  if (lane == 0) a.sums[static_cast<int64_t>(r) * a.runs + run] = s;
}

// running sum over the lanes of a wave
__device__ __forceinline__ double wave_scan(double x) {
  const int lane = threadIdx.x % 64;
#pragma unroll
  for (int m = 1; m < 64; m *= 2) {
    const double y = __shfl_up(x, m);
    x = lane >= m ? x + y : x;
  }
  return x;
}

// The first entry of [x0, x1) above 0 at which `before` and the running sum
// exceed `target`; if none does, the last one above 0; -1 if there is none.  By all
// threads, 2048 entries at a time.
template <typename L>
__device__ int search(const L& left, int64_t x0, int64_t x1, double before, double target, double* sh, int* found) {
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  if (threadIdx.x == 0) found[0] = INT32_MAX, found[1] = -1;
  for (int64_t at = x0; at < x1; at += kThreads * kVec) {
    double w[kVec], s = 0.0;
    typename L::Raw raw;
    left.as([&](auto whole, auto tried) __attribute__((always_inline)) {
      left.template load<decltype(whole)::value, decltype(tried)::value>(at + threadIdx.x * kVec, x1, raw);
      left.template weights<decltype(tried)::value>(raw, w);
    });
    const int mine = static_cast<int>(raw.at);
#pragma unroll
    for (int j = 0; j < kVec; ++j) s += w[j];
    const double upto = wave_scan(s);
    if (lane == 63) sh[wave] = upto;
    __syncthreads();
    double base = before, all = 0.0;
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
      base += v < wave ? sh[v] : 0.0;
      all += sh[v];
    }
    // Looked through by every thread that may hold the border.  (base + upto is
    // one order of the sum, the running one another: it is taken on either's word.)
    double run = base + (upto - s);
    if (s > 0.0) {
      int hit = INT32_MAX, top = -1;
      const bool near = base + upto > target || run + s > target;
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        run += w[j];
        top = w[j] > 0.0 ? mine + j : top;
        hit = w[j] > 0.0 && run > target && hit == INT32_MAX ? mine + j : hit;
      }
      if (near) atomicMin(&found[0], hit == INT32_MAX ? top : hit);
      atomicMax(&found[1], top);
    }
    __syncthreads();
    if (found[0] != INT32_MAX) break;
    before += all;
    __syncthreads();
  }
  return found[0] != INT32_MAX ? found[0] : found[1];
}

// A workgroup a request: the runs' sums, a lane each, say which run holds the following
// token; that run is searched.  Bound by latency (3.4 to 5.0 us).
template <int DT, bool DRAFT>
__global__ __launch_bounds__(kThreads) void kda_verify_draw_kernel(VerifyArgs a) {
  __shared__ double sh[kWaves];
  __shared__ int found[2];
  const int lane = threadIdx.x % 64;
  const int r = blockIdx.x;
  const VerifyStop* stop = a.stops + r;
  const int last = stop->last;
  if (last < 0) {
    if (threadIdx.x == 0) a.next[r] = -1;
    return;
  }
  const int64_t n0 = a.cu[r], row = n0 + last;
  Left<DT, DRAFT> left;
  left.p = row_of<DT>(a.target, row, a.target_stride);
  left.q = DRAFT ? row_of<DT>(a.draft, row, a.draft_stride) : nullptr;
  left.vocab = a.vocab;
  left.tries = stop->tries;
  left.refused = stop->refused;
  left.mass = stop->mass[lane];
  left.token = (left.refused >> lane & 1) != 0 ? a.tokens[n0 + lane] : -1;
  const double part = lane < a.runs ? a.sums[static_cast<int64_t>(r) * a.runs + lane] : 0.0;
  const double upto = wave_scan(part);
  double total = lane_double(upto, 63);
  const double u = static_cast<double>(a.sample[r]);
  int64_t x0 = 0, x1 = a.vocab;
  double before = 0.0;
  if (total > 0.0) {
    // the first run that passes the border; the last with weight if none does
    uint64_t over = __ballot(part > 0.0 && upto > u * total);
    if (over == 0) over = 1ull << (63 - __builtin_clzll(__ballot(part > 0.0)));
    const int at = __builtin_ctzll(over);
    before = at == 0 ? 0.0 : lane_double(upto, at - 1);
    x0 = static_cast<int64_t>(at) * a.run;
    x1 = x0 + a.run < a.vocab ? x0 + a.run : a.vocab;
  } else {
    // nothing is left: the target's row itself
    left.tries = 0;
    left.refused = 0;
    total = block_sum(left.share(0, a.vocab, threadIdx.x, kThreads), sh);
  }
  int x = -1;
  if (total > 0.0 && total < __builtin_huge_val()) x = search(left, x0, x1, before, u * total, sh, found);
  if (threadIdx.x == 0) a.next[r] = x;
}

int status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH; }
bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <int DT, bool DRAFT>
hipError_t launch(const VerifyArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((kda_verify_walk_kernel<DT, DRAFT>), dim3(static_cast<uint32_t>(a.n_req) * ((a.runs + kWaves - 1) / kWaves)),
                     dim3(kThreads), 0, st, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((kda_verify_draw_kernel<DT, DRAFT>), dim3(a.n_req), dim3(kThreads), 0, st, a);
  return hipGetLastError();
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int kda_verify_drafts(const void* target, int64_t target_stride, const void* draft, int64_t draft_stride,
                                 const int32_t* cu_seqlens, const int32_t* parents, const int32_t* tokens,
                                 const float* accept_rand, const float* sample_rand, int32_t* path,
                                 int32_t max_path, int32_t* path_lens, int32_t* next_tokens, int32_t n_req,
                                 int64_t n_tokens, int32_t vocab, kda_dtype dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const int rc = verify_check(n_req, n_tokens, vocab, max_path, dtype);
  if (rc != KDA_OK) return rc;
  if (n_req == 0) return KDA_OK;
  if (cu_seqlens == nullptr || sample_rand == nullptr || path == nullptr || path_lens == nullptr ||
      next_tokens == nullptr)
    return KDA_ERR_NULL;
  if (n_tokens > 0 && (target == nullptr || parents == nullptr || tokens == nullptr || accept_rand == nullptr))
    return KDA_ERR_NULL;
  if (target_stride < vocab || (draft != nullptr && draft_stride < vocab)) return KDA_ERR_ARG;
  const VerifyPlan p = verify_plan(vocab);
  if (static_cast<int64_t>(n_req) * ((p.runs + kWaves - 1) / kWaves) > INT32_MAX / kThreads) return KDA_ERR_ARG;
  const unsigned size = dtype == KDA_F32 ? 4 : 2;
  if (!aligned(target, size) || !aligned(draft, size) || !aligned(cu_seqlens, 4) || !aligned(parents, 4) ||
      !aligned(tokens, 4) || !aligned(accept_rand, 4) || !aligned(sample_rand, 4) || !aligned(path, 4) ||
      !aligned(path_lens, 4) || !aligned(next_tokens, 4) || !aligned(workspace, 8))
    return KDA_ERR_ALIGN;
  const size_t need = kda_verify_workspace(n_req, n_tokens, vocab, max_path, dtype);
  if (need > 0 && workspace == nullptr) return KDA_ERR_NULL;
  if (need > workspace_bytes) return KDA_ERR_ARG;
  VerifyArgs a;
  a.target = target;
  a.draft = draft;
  a.cu = cu_seqlens;
  a.parents = parents;
  a.tokens = tokens;
  a.accept = accept_rand;
  a.sample = sample_rand;
  a.path = path;
  a.lens = path_lens;
  a.next = next_tokens;
  a.stops = static_cast<VerifyStop*>(workspace);
  a.sums = reinterpret_cast<double*>(a.stops + n_req);
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.n_tokens = n_tokens;
  a.n_req = n_req;
  a.vocab = vocab;
  a.max_path = max_path;
  a.runs = p.runs;
  a.run = p.run;
  hipStream_t st = static_cast<hipStream_t>(stream);
  switch (dtype) {
    case KDA_F32: return status(draft ? launch<KDA_F32, true>(a, st) : launch<KDA_F32, false>(a, st));
    case KDA_F16: return status(draft ? launch<KDA_F16, true>(a, st) : launch<KDA_F16, false>(a, st));
    default: return status(draft ? launch<KDA_BF16, true>(a, st) : launch<KDA_BF16, false>(a, st));
  }
}
