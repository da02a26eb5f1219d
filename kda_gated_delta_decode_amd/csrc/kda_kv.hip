// kda_kv.hip -- the paged 4-bit key/value cache on gfx950: appending keys and
// values with the position rotation, reading them back, and attention.
//
// The cache's format is OCP microscaling MXFP4: E2M1 codes with one E8M0
// exponent for 32 channels, 4.25 bits a value.  Two properties carry the
// kernels.  v_cvt_scalef32_pk_bf16_fp4 turns two codes and their exponent
// into two bf16 in one instruction, and every such value is exact in bf16
// (exponent bytes 2..252), so the matrix cores take the cache without a
// rounding; queries and weights enter as 1..3 bf16 pieces whose sum is the
// fp32, fp16 or bf16 number.
#include <hip/hip_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>
#include <utility>

#include "kda_decode.h"
#include "kda_device.h"
#include "kda_kv.h"

namespace kda {
namespace {

using bf2 = __bf16 __attribute__((ext_vector_type(2)));
using bf8 = __bf16 __attribute__((ext_vector_type(8)));
using f16v = float __attribute__((ext_vector_type(16)));
using h2 = _Float16 __attribute__((ext_vector_type(2)));
using u16x2 = uint16_t __attribute__((ext_vector_type(2)));
using u2 = uint32_t __attribute__((ext_vector_type(2)));
using u4 = uint32_t __attribute__((ext_vector_type(4)));

// Loads of uniform addresses through the scalar cache, apart from the vector
// loads' counter: a page id can be waited for while cache rows are in flight.
using const_i32 = const int32_t __attribute__((address_space(4)));

// A launch's arguments where they lie.
using kernel_args = const KvAttendArgs __attribute__((address_space(4)))*;

template <int DT>
constexpr int elem_bytes() { return DT == KDA_F32 ? 4 : 2; }

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
// NaN if either is (one instruction, without fmaxf's quieting of its operands)
__device__ __forceinline__ float max_nan(float x, float y) { return __builtin_elementwise_maximum(x, y); }
__device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
// the upper (lower) halves of a and b as one register, a's first
__device__ __forceinline__ uint32_t pack_hi(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x07060302); }
__device__ __forceinline__ uint32_t pack_lo(uint32_t a, uint32_t b) { return __builtin_amdgcn_perm(b, a, 0x05040100); }
// two E2M1 codes (byte SEL of c) times 2^(e - 127), scale = e << 23, as two bf16
template <int SEL>
__device__ __forceinline__ uint32_t dequant2(uint32_t c, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, SEL));
}
__device__ __forceinline__ float exp_scale(uint32_t e) { return __uint_as_float(e << 23); }

template <int DT>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&x)[8]) {
  if constexpr (DT == KDA_F32) {
    const f4* s = reinterpret_cast<const f4*>(static_cast<const float*>(p) + at);
    const f4 a = s[0], b = s[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = a[e], x[e + 4] = b[e];
  } else if constexpr (DT == KDA_F16) {
    const h8 a = *reinterpret_cast<const h8*>(static_cast<const _Float16*>(p) + at);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(a[e]);
  } else {
    const u4 a = *reinterpret_cast<const u4*>(static_cast<const uint16_t*>(p) + at);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(a[e] << 16);
      x[2 * e + 1] = __uint_as_float(a[e] & 0xFFFF0000u);
    }
  }
}

// rounds to nearest even, once
template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&x)[8]) {
  if constexpr (DT == KDA_F32) {
    f4* d = reinterpret_cast<f4*>(static_cast<float*>(p) + at);
    d[0] = f4{x[0], x[1], x[2], x[3]};
    d[1] = f4{x[4], x[5], x[6], x[7]};
  } else if constexpr (DT == KDA_F16) {
    h8 a;
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = static_cast<_Float16>(x[e]);
    *reinterpret_cast<h8*>(static_cast<_Float16*>(p) + at) = a;
  } else {
    bf8 a;
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = static_cast<__bf16>(x[e]);
    *reinterpret_cast<bf8*>(static_cast<__bf16*>(p) + at) = a;
  }
}

template <int DT>
__device__ __forceinline__ void store4(void* p, int64_t at, f4 x) {
  if constexpr (DT == KDA_F32) {
    *reinterpret_cast<f4*>(static_cast<float*>(p) + at) = x;
  } else if constexpr (DT == KDA_F16) {
    *reinterpret_cast<h4*>(static_cast<_Float16*>(p) + at) =
        h4{static_cast<_Float16>(x[0]), static_cast<_Float16>(x[1]), static_cast<_Float16>(x[2]), static_cast<_Float16>(x[3])};
  } else {
    using bf4 = __bf16 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<bf4*>(static_cast<__bf16*>(p) + at) =
        bf4{static_cast<__bf16>(x[0]), static_cast<__bf16>(x[1]), static_cast<__bf16>(x[2]), static_cast<__bf16>(x[3])};
  }
}

template <int DT>
__device__ __forceinline__ void store_channels(void* p, int64_t at, const float (&x)[8]) { store8<DT>(p, at, x); }
template <int DT>
__device__ __forceinline__ void store_channels(void* p, int64_t at, const float (&x)[4]) {
  store4<DT>(p, at, f4{x[0], x[1], x[2], x[3]});
}

// ---------------------------------------------------------------------------
// Which sequence a token belongs to, and where the cache keeps it
// ---------------------------------------------------------------------------

enum Place { kOutside = 0, kBad = 1, kPlaced = 2 };

struct TokenPlace {
  int what;          // a Place
  int32_t pos;       // position in its sequence
  uint8_t* block;    // head 0's block of its page
  int32_t row;       // its token row there
};

// W lanes (one token each group of W) search cu together: each round splits
// the range in W and keeps the part that holds the token, so 16 lanes need
// one round of loads for up to 16 sequences and two for 256.
template <int W>
__device__ __forceinline__ TokenPlace find_token(const KvTables& t, int64_t token, int n_positions) {
  const int lane = threadIdx.x % 64, li = lane % W;
  const uint64_t mask = ((1ull << W) - 1) << (lane - li);
  TokenPlace r{kOutside, 0, t.base, 0};
  int lo = 0, hi = t.n_seq;
  if (token < t.n_tokens) {
    while (hi - lo > 1) {
      const int step = (hi - lo + W - 1) / W;
      const int i = lo + step * (li + 1);
      const bool before = i < hi && t.cu[i] <= token;
      lo += step * __popcll(__ballot(before) & mask);
      hi = lo + step < hi ? lo + step : hi;
    }
    const int64_t first = t.cu[lo], end = t.cu[lo + 1], past = t.past[lo];
    if (first >= 0 && token >= first && token < end) {
      const int64_t pos = past + (token - first);
      r.what = kBad;
      if (past >= 0 && pos < n_positions && (pos >> t.log_p) < t.max_pages) {
        const int32_t page = t.page_table[static_cast<int64_t>(lo) * t.max_pages + (pos >> t.log_p)];
        if (page >= 0 && page < t.n_pages) {
          r.what = kPlaced;
          r.pos = static_cast<int32_t>(pos);
          r.block = t.base + page * t.page_bytes;
          r.row = static_cast<int32_t>(pos) & (t.P - 1);
        }
      }
    }
  }
  return r;
}

// ---------------------------------------------------------------------------
// Append
// ---------------------------------------------------------------------------

// maximum over the 4 lanes that hold one exponent's 32 channels
__device__ __forceinline__ int quad_max(int x) {
  int y = __builtin_amdgcn_mov_dpp(x, kDppQuadXor1, 0xF, 0xF, true);
  x = x > y ? x : y;
  y = __builtin_amdgcn_mov_dpp(x, kDppQuadXor2, 0xF, 0xF, true);
  return x > y ? x : y;
}

__device__ __forceinline__ int clamp_exp(int e) { return e < kKvMinExp ? kKvMinExp : e > kKvMaxExp ? kKvMaxExp : e; }

// 8 values already divided by their power of two: rounded to E2M1 (nearest,
// ties to even, saturating at 6)
__device__ __forceinline__ uint32_t quant8(const float (&a)[8]) {
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[0], a[1], 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[2], a[3], 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[4], a[5], 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, a[6], a[7], 1.0f, 3);
  return c;
}

// A double as the fp32 of 20 mantissa bits whose lowest of 23 is set when any
// later bit was: E2M1's rounding borders have at most two mantissa bits, so
// rounding this number gives what rounding the double would.
__device__ __forceinline__ float sticky_float(double d) {
  const uint64_t b = __builtin_bit_cast(uint64_t, d);
  const uint32_t hi = static_cast<uint32_t>(b >> 32), lo = static_cast<uint32_t>(b);
  const uint32_t mag = hi & 0x7FFFFFFFu;
  const uint32_t f = ((mag - (896u << 20)) << 3) | (lo != 0 ? 1u : 0u);
  return __uint_as_float((mag < (897u << 20) ? 0u : f) | (hi & 0x80000000u));
}

// 8 channels as they lie in memory
template <int DT>
struct Raw8 {
  static constexpr int N = DT == KDA_F32 ? 2 : 1;
  u4 w[N];

  template <bool STREAM>
  __device__ __forceinline__ void load(const void* p, int64_t at) {
    const u4* s = reinterpret_cast<const u4*>(static_cast<const uint8_t*>(p) + at * elem_bytes<DT>());
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (STREAM)
        w[i] = __builtin_nontemporal_load(s + i);
      else
        w[i] = s[i];
    }
  }
  template <bool STREAM>
  __device__ __forceinline__ void store(void* p, int64_t at) const {
    u4* d = reinterpret_cast<u4*>(static_cast<uint8_t*>(p) + at * elem_bytes<DT>());
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if constexpr (STREAM)
        __builtin_nontemporal_store(w[i], d + i);
      else
        d[i] = w[i];
    }
  }
  // those of another lane
  __device__ __forceinline__ Raw8 of(int lane) const {
    Raw8 r;
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) r.w[i][e] = __builtin_amdgcn_ds_bpermute(4 * lane, w[i][e]);
    return r;
  }
  // rounded to nearest even, once
  __device__ __forceinline__ void set(const float (&x)[8]) {
    if constexpr (DT == KDA_F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e / 4][e % 4] = bits(x[e]);
    } else {
      using T = std::conditional_t<DT == KDA_F16, _Float16, __bf16>;
      T __attribute__((ext_vector_type(8))) y;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = static_cast<T>(x[e]);
      w[0] = __builtin_bit_cast(u4, y);
    }
  }
  __device__ __forceinline__ void numbers(float (&x)[8]) const {
    if constexpr (DT == KDA_F32) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e / 4][e % 4]);
    } else if constexpr (DT == KDA_F16) {
      const h8 a = __builtin_bit_cast(h8, w[0]);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = static_cast<float>(a[e]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(w[0][e] << 16);
        x[2 * e + 1] = __uint_as_float(w[0][e] & 0xFFFF0000u);
      }
    }
  }
};

// One group of D / 8 lanes takes one token and walks over its units (cached
// heads, then query heads), 8 channels a lane: the token's place and its
// angles are looked up once, and a pair's other half, when another lane holds
// it, comes from that lane.  Neighbouring groups take neighbouring tokens of
// the same unit, so a wave writes 256 contiguous bytes of codes.  Queries are
// most of the bytes: four heads' loads are in flight together.  STREAM: inputs
// that the caches cannot hold anyway pass them by.  Bound by HBM (32 query and 8
// cached heads in bf16, 16384 tokens: 353 MB in 80 us, 4.4 TB/s), for few tokens
// by the chain sequence -> page -> angles of loads (64 tokens: 4 us).
template <int DT, int D, bool STREAM>
__global__ __launch_bounds__(256) void kda_kv_append_kernel(KvAppendArgs a) {
  constexpr int W = D / 8, AT_ONCE = 4;
  const int li = threadIdx.x % W;
  const int64_t tile = blockIdx.x / a.unit_blocks;
  const int ub = blockIdx.x % a.unit_blocks;
  const int64_t token = tile * (256 / W) + threadIdx.x / W;
  const int u0 = ub * a.units_per_block;
  const int u1 = u0 + a.units_per_block < a.units ? u0 + a.units_per_block : a.units;
  const TokenPlace at = find_token<W>(a.t, token, a.n_positions);
  if (at.what == kOutside) return;

  // out[e] = x[e] * cs[e] + partner[e] * sn[e]
  const int c0 = 8 * li, lane = threadIdx.x % 64;
  const bool turned = c0 < 2 * a.half && at.what == kPlaced;
  float cs[8], sn[8];
  int other = lane;  // the lane of the pairs' other halves
  if (turned) {
    if (a.interleaved) {
      const f4 c = *reinterpret_cast<const f4*>(a.cos + static_cast<int64_t>(at.pos) * a.half + c0 / 2);
      const f4 s = *reinterpret_cast<const f4*>(a.sin + static_cast<int64_t>(at.pos) * a.half + c0 / 2);
#pragma unroll
      for (int e = 0; e < 8; ++e) cs[e] = c[e / 2], sn[e] = e % 2 ? s[e / 2] : -s[e / 2];
    } else {
      const bool first = c0 < a.half;
      const int64_t row = static_cast<int64_t>(at.pos) * a.half + (first ? c0 : c0 - a.half);
      load8<KDA_F32>(a.cos, row, cs);
      load8<KDA_F32>(a.sin, row, sn);
      other = first ? lane + a.half / 8 : lane - a.half / 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) sn[e] = first ? -sn[e] : sn[e];
    }
  }
  // x and its partners; every lane takes part
  auto pairs = [&](const Raw8<DT>& r, float (&x)[8], float (&p)[8]) __attribute__((always_inline)) {
    r.numbers(x);
    if (a.half == 0) return;
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = x[e ^ 1];
    } else {
      r.of(other).numbers(p);
    }
  };
  const int block_bytes = kv_block_bytes(a.t.P, D);
  const uint64_t mine = ((1ull << W) - 1) << (lane - li);

  int u = u0;
  for (; u < u1 && u < a.t.H; ++u) {
    Raw8<DT> rk;
    float x[8], p[8], v[8];
    rk.template load<STREAM>(a.k, token * a.k_stride + u * D + c0);
    // (values without the hint: 8192 fp32 tokens 85 us, with it 96)
    load8<DT>(a.v, token * a.v_stride + u * D + c0, v);
    pairs(rk, x, p);
    // the keys' rotation and scaling in 64 bits: a code next to a rounding
    // border comes out as the definition has it
    double y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = static_cast<double>(x[e]);
    if (turned) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        y[e] = y[e] * static_cast<double>(cs[e]) + static_cast<double>(p[e]) * static_cast<double>(sn[e]);
    }
    int ek = 0, ev = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int k = static_cast<int>(__builtin_bit_cast(uint64_t, y[e]) >> 52) & 0x7FF;
      const int w = static_cast<int>(bits(v[e]) >> 23) & 0xFF;
      ek = ek > k ? ek : k;
      ev = ev > w ? ev : w;
    }
    ek = quad_max(ek);
    ev = quad_max(ev);
    const bool poison = (__ballot(ek == 0x7FF || ev == 0xFF) & mine) != 0;
    const int kb = clamp_exp(ek - 1023 - 2 + 127), vb = clamp_exp(ev - 2);
    const double km = __builtin_bit_cast(double, static_cast<uint64_t>(1023 + 127 - kb) << 52);
    const float vm = exp_scale(254 - vb);
    float ka[8], va[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      ka[e] = sticky_float(y[e] * km);
      va[e] = v[e] * vm;
    }
    if (at.what != kPlaced) continue;
    uint8_t* block = at.block + static_cast<int64_t>(u) * block_bytes;
    const int code = at.row * (D / 2) + 4 * li;
    *reinterpret_cast<uint32_t*>(block + code) = poison ? 0 : quant8(ka);
    *reinterpret_cast<uint32_t*>(block + kv_value_codes(a.t.P, D) + code) = poison ? 0 : quant8(va);
    if (li % 4 == 0) {
      block[kv_key_exps(a.t.P, D) + at.row * (D / kKvGroup) + li / 4] = static_cast<uint8_t>(poison ? kKvPoison : kb);
      block[kv_value_exps(a.t.P, D) + (li / 4) * a.t.P + at.row] = static_cast<uint8_t>(poison ? kKvMinExp : vb);
    }
  }
  for (; u < u1; u += AT_ONCE) {
    Raw8<DT> r[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i)
      if (u + i < u1) r[i].template load<STREAM>(a.q, token * a.q_stride + (u + i - a.t.H) * D + c0);
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      if (u + i >= u1) break;
      float x[8], p[8];
      pairs(r[i], x, p);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        x[e] = at.what == kBad ? __builtin_nanf("") : turned ? x[e] * cs[e] + p[e] * sn[e] : x[e];
      r[i].set(x);
      r[i].template store<STREAM>(a.q_out, (token * a.q_heads + u + i - a.t.H) * D + c0);
    }
  }
}

// ---------------------------------------------------------------------------
// Read back
// ---------------------------------------------------------------------------

// Channels a lane takes: 16 bytes of them, so that a store instruction writes
// whole lines (8 fp32 channels, two stores 16 bytes apart: 403 us instead of 348
// for 102392 tokens of 12 heads).
template <int DT>
constexpr int kv_read_channels() { return DT == KDA_F32 ? 4 : 8; }

// the codes of a lane's channels, as numbers
template <int DT>
__device__ __forceinline__ void store_codes(void* p, int64_t at, uint32_t c, uint32_t e) {
  const float s = exp_scale(e);
  const bool nan = e == kKvPoison;
  if constexpr (DT == KDA_BF16) {
    u4 o = {dequant2<0>(c, s), dequant2<1>(c, s), dequant2<2>(c, s), dequant2<3>(c, s)};
    if (nan) o = u4{0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u, 0x7FC07FC0u};
    *reinterpret_cast<u4*>(static_cast<uint16_t*>(p) + at) = o;
  } else {
    const f2 y0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 0);
    const f2 y1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 1);
    const float none = __builtin_nanf("");
    if constexpr (DT == KDA_F32) {
      store4<DT>(p, at, nan ? f4{none, none, none, none} : f4{y0[0], y0[1], y1[0], y1[1]});
    } else {
      const f2 y2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 2);
      const f2 y3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, s, 3);
      float x[8] = {y0[0], y0[1], y1[0], y1[1], y2[0], y2[1], y3[0], y3[1]};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = nan ? none : x[i];
      store8<DT>(p, at, x);
    }
  }
}

// Groups of lanes as in the append, one token each.  Bound by HBM, mostly by
// what is written: 1.43 GB in 348 us, 4.1 TB/s (torch's copy of 4 GiB: 4.7).
template <int DT, int D>
__global__ __launch_bounds__(256) void kda_kv_read_kernel(KvReadArgs a) {
  constexpr int CH = kv_read_channels<DT>(), W = D / CH;
  using Codes = std::conditional_t<CH == 4, uint16_t, uint32_t>;
  const int li = threadIdx.x % W;
  const int64_t tile = blockIdx.x / a.head_blocks;
  const int hb = blockIdx.x % a.head_blocks;
  const int64_t token = tile * (256 / W) + threadIdx.x / W;
  const int h0 = hb * a.heads_per_block;
  const int h1 = h0 + a.heads_per_block < a.t.H ? h0 + a.heads_per_block : a.t.H;
  const TokenPlace at = find_token<W>(a.t, token, INT32_MAX);
  if (at.what == kOutside) return;
  const int block_bytes = kv_block_bytes(a.t.P, D);
  const int code = at.row * (D / 2) + CH / 2 * li, grp = CH * li / kKvGroup;
  const int k_exp = kv_key_exps(a.t.P, D) + at.row * (D / kKvGroup) + grp;
  const int v_exp = kv_value_exps(a.t.P, D) + grp * a.t.P + at.row;
  for (int h = h0; h < h1; ++h) {
    // a token without a page reads page 0, and is NaN
    const uint8_t* block = at.block + static_cast<int64_t>(h) * block_bytes;
    const uint32_t kc = *reinterpret_cast<const Codes*>(block + code);
    const uint32_t vc = *reinterpret_cast<const Codes*>(block + kv_value_codes(a.t.P, D) + code);
    uint32_t ke = block[k_exp], ve = block[v_exp];
    if (at.what == kBad) ke = ve = kKvPoison;
    if (a.k_out != nullptr) store_codes<DT>(a.k_out, token * a.k_stride + h * D + CH * li, kc, ke);
    if (a.v_out != nullptr) store_codes<DT>(a.v_out, token * a.v_stride + h * D + CH * li, vc, ve);
  }
}

// ---------------------------------------------------------------------------
// Attention: one sequence's rows
// ---------------------------------------------------------------------------

// A sequence as the attention kernels see it.
struct Seq {
  int64_t n0;    // its first token's index
  int rows;      // its tokens in this launch
  int past;      // tokens cached before them
  bool skip;     // nothing is written for it
  bool bad;      // its rows are set to NaN
};

__device__ __forceinline__ Seq seq_of(const KvTables& t, int s) {
  const_i32* cu = (const_i32*)t.cu;
  const_i32* len = (const_i32*)t.past;
  const int64_t n0 = cu[s], n1 = cu[s + 1];
  Seq q;
  q.past = len[s];
  q.n0 = n0;
  q.skip = n0 < 0 || n1 <= n0 || n1 > t.n_tokens;
  q.rows = q.skip ? 0 : static_cast<int>(n1 - n0);
  q.bad = q.past < 0 || static_cast<int64_t>(q.past) + q.rows > (static_cast<int64_t>(t.max_pages) << t.log_p);
  return q;
}

// Splits of a tile whose last row sees `vis` tokens; the last split takes what
// the launch had no blocks for.
__device__ __forceinline__ int kv_splits(int vis, const KvAttendArgs& a) {
  const int n = static_cast<int>((static_cast<uint32_t>(vis) + a.chunk - 1) / static_cast<uint32_t>(a.chunk));
  return n < a.n_splits ? n : a.n_splits;
}

// Tiles of 128 rows lie in slots, sequence s's from slot
// floor(cu[s] group / 128) + s on: no fewer slots than tiles, and n_tokens group
// / 128 + n_seq of them in all, however the rows are spread over sequences.
constexpr int kTileRows = 128;
struct TileAt {
  int s, tile;  // tile < 0: none
};
__device__ __forceinline__ TileAt tile_of_slot(const KvAttendArgs& a, int slot) {
  const int lane = threadIdx.x % 64;
  int lo = 0, hi = a.t.n_seq;
  while (hi - lo > 1) {  // 64 lanes search together, as find_token
    const int step = (hi - lo + 63) / 64;
    const int i = lo + step * (lane + 1);
    const bool before = i < hi && static_cast<int64_t>(a.t.cu[i]) * a.group / kTileRows + i <= slot;
    lo += step * __popcll(__ballot(before));
    hi = lo + step < hi ? lo + step : hi;
  }
  lo = __builtin_amdgcn_readfirstlane(lo);
  const int64_t first = static_cast<int64_t>(a.t.cu[lo]) * a.group / kTileRows + lo;
  return {lo, first > slot ? -1 : static_cast<int>(slot - first)};
}

// bf16 pieces that represent a type's numbers exactly: 24, 11 or 8
// significant bits, 8 a piece.
template <int DT>
constexpr int q_pieces() { return DT == KDA_F32 ? 3 : DT == KDA_F16 ? 2 : 1; }
// Softmax weights are fp32.  fp32 outputs take all 24 bits of them; for 16-bit
// outputs the second of two pieces is rounded to nearest, which is off by at most
// 2^-16 of a weight, a 32nd of fp16's half step, to either side.
template <int DT>
constexpr int w_pieces() { return DT == KDA_F32 ? 3 : 2; }

// Splits pairs of numbers into N packed bf16 pieces by truncation: what is
// left after each piece is exact, and 3 pieces hold all of an fp32.
template <int N>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&out)[N]) {
#pragma unroll
  for (int p = 0; p < N; ++p) {
    out[p] = pack_hi(bits(x), bits(y));
    x -= __uint_as_float(bits(x) & 0xFFFF0000u);
    y -= __uint_as_float(bits(y) & 0xFFFF0000u);
  }
}

// two weights as their pieces
template <int N>
__device__ __forceinline__ void split_weights(float x, float y, uint32_t (&out)[N]) {
  if constexpr (N == 2) {
    out[0] = pack_hi(bits(x), bits(y));
    x -= __uint_as_float(bits(x) & 0xFFFF0000u);
    y -= __uint_as_float(bits(y) & 0xFFFF0000u);
    out[1] = __builtin_bit_cast(uint32_t, bf2{static_cast<__bf16>(x), static_cast<__bf16>(y)});
  } else {
    split_pair<N>(x, y, out);
  }
}

// 8 channels of a query as its bf16 pieces; sign is 1 or -1
template <int DT>
__device__ __forceinline__ void load_query(const void* q, int64_t at, float sign, u4 (&out)[q_pieces<DT>()]) {
  if constexpr (DT == KDA_BF16) {
    out[0] = *reinterpret_cast<const u4*>(static_cast<const uint16_t*>(q) + at);
    const uint32_t flip = sign < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) out[0][e] ^= flip;
  } else {
    float x[8];
    load8<DT>(q, at, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t w[q_pieces<DT>()];
      split_pair<q_pieces<DT>()>(x[2 * e] * sign, x[2 * e + 1] * sign, w);
#pragma unroll
      for (int p = 0; p < q_pieces<DT>(); ++p) out[p][e] = w[p];
    }
  }
}

__device__ __forceinline__ f4 mfma16(u4 a, u4 b, f4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}

__device__ __forceinline__ float max_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(bits(x), bits(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(bits(x), bits(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Waves a SIMD: three in 168 registers hide more of a step's latency than two
// (64 ragged requests at up to 8192 tokens: 85 -> 81 us; four would spill); with
// two row tiles two (32 rows of 8 requests at 4097 tokens: 28 -> 26 us).  Eight
// waves a workgroup are for launches that leave most of the chip idle: two.
template <int NT, int NW>
constexpr int kv_rows_waves() { return NT == 1 && NW == 4 ? 3 : 2; }

// Few rows: 16 * NT rows of one sequence and cached head against one split of
// its tokens, over NW waves.
//
// S^T = K Q^T and O^T = V^T P^T in 16x16x32 products, so that the weights go
// from the first product's result registers straight into the second's right
// operand: lane l holds query row l % 16, and its tokens 4j + r (j = l / 16)
// of two 16-token tiles are the 8 contraction slots of the second product.
// Which channel (or token) sits in which contraction slot is free as long as
// both operands agree, and it is chosen so that every lane reads whole
// contiguous pieces of the cache as it lies: a quarter of a key row (16 bytes
// and one exponent at D = 128), and D / 16 channels of 8 value rows.
// The waves take the split's 32-token steps in turn, each with its own
// maximum and sum, and join in LDS.  Bound by HBM: the next step's keys are
// loaded as soon as the scores have used this step's, its values likewise, so
// one set of registers keeps loads in flight all the time.  64 requests of 4096
// tokens, 12 cached heads in bf16: 427 MB in 81 us, 5.2 TB/s of the 6.5 that a
// streaming copy reaches; 8 requests of 8 rows: 53 MB in 15 us.
template <int DT, int D, int NT, int NW>
__global__ __launch_bounds__(64 * NW, (kv_rows_waves<NT, NW>())) void kda_kv_rows_kernel(KvAttendArgs a) {
  constexpr int NQ = q_pieces<DT>(), NP = w_pieces<DT>();
  constexpr int M = D / 32;   // products over the channels
  constexpr int C = D / 16;   // channels of a lane in the second product, and its row tiles
  constexpr int R = 16 * NT;
  constexpr int LD = D + 4;
  __shared__ float o_sh[NW][R][LD];
  __shared__ float ml_sh[NW][R][2];

  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int i16 = lane % 16, j = lane / 16;
  // block -> (split, sequence, cached head, row tile).  Row tiles, which read
  // the same tokens, are neighbours on one XCD; with one of them the heads go
  // round the XCDs, so each has a like share of every sequence.
  const int id = a.row_tiles > 1 ? tile_of_block(blockIdx.x, gridDim.x) : blockIdx.x;
  const int rt0 = id % a.row_tiles, unit = (id / a.row_tiles) % (a.t.n_seq * a.t.H);
  const int sp = id / a.row_tiles / (a.t.n_seq * a.t.H);
  const int h = unit % a.t.H, s = unit / a.t.H;
  const int t0 = sp * a.chunk;
  // Page ids of this wave's next 32 steps, two tiles each, loaded at once: a
  // lookup is then a register read, with no load in front of the rows'.  They
  // are asked for before the sequence's length is known.
  const int32_t* table = a.t.page_table + static_cast<int64_t>(s) * a.t.max_pages;
  auto load_pages = [&](int from) __attribute__((always_inline)) {
    const int64_t at = (static_cast<int64_t>(from) + 32 * NW * (lane / 2) + 16 * (lane % 2)) >> a.t.log_p;
    return at < a.t.max_pages ? table[at] : -1;
  };
  const int pages0 = load_pages(t0 + 32 * wave);
  const Seq q = seq_of(a.t, s);
  if (q.skip) return;
  const int all_rows = q.rows * a.group;

  const int block_bytes = kv_block_bytes(a.t.P, D);
  const uint8_t* head0 = a.t.base + static_cast<int64_t>(h) * block_bytes;
  // the lane's places in a block, from a tile's first token row
  const uint32_t k_off = i16 * (D / 2) + j * (D / 8);
  const uint32_t v_off = 4 * j * (D / 2) + i16 * (D / 32);
  const uint32_t ve_off = (i16 * C / kKvGroup) * a.t.P + 4 * j;

  // Tiles beyond those the launch has blocks for are walked by the same blocks.
  for (int row0 = rt0 * R; row0 < all_rows; row0 += a.row_tiles * R) {
    const int last_row = (row0 + R < all_rows ? row0 + R : all_rows) - 1;
    const int vis = q.past + last_row / a.group + 1;  // tokens the last row sees
    const int splits = q.bad ? 1 : kv_splits(vis, a);
    if (sp >= splits) continue;
    const int t1 = q.bad ? 0 : sp == splits - 1 ? vis : t0 + a.chunk;
    const int first_limit = q.past + row0 / a.group;  // the last token every row sees

    // this lane's query row of each tile, and the last token it sees
    u4 qf[NT][NQ][M];
    int limit[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int row = row0 + 16 * n + i16;
      const int r = row <= last_row ? row : last_row;
      const int tok = r / a.group, g = r - tok * a.group;
      limit[n] = row <= last_row ? q.past + tok : -1;
      const int64_t at = (q.n0 + tok) * a.q_stride + (static_cast<int64_t>(h) * a.group + g) * D + j * (D / 4);
#pragma unroll
      for (int m = 0; m < M; ++m) {
        u4 x[NQ];
        load_query<DT>(a.q, at + 8 * m, a.sign, x);
#pragma unroll
        for (int p = 0; p < NQ; ++p) qf[n][p][m] = x[p];
      }
    }

    f4 o[NT][C];
    float mx[NT], sum[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      mx[n] = -INFINITY;
      sum[n] = 0.0f;
#pragma unroll
      for (int m = 0; m < C; ++m) o[n][m] = f4{0, 0, 0, 0};
    }

    uint32_t kc[2][M], ke[2];  // keys: token i16 of two 16-token tiles, D / 4 channels of it
    uint32_t vc[8], ve[2];     // values: D / 16 channels of tokens 4j + r of both tiles
    int tb = t0 + 32 * wave, step = 0;
    int pages = pages0;
    int kp[2], vp[2];  // pages of the keys and values in flight; -1: no such page, or no token left
    auto load_keys = [&](int t) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int page = __builtin_amdgcn_readlane(pages, 2 * (step % 32) + b);
        kp[b] = t + 16 * b < t1 && page < a.t.n_pages ? page : -1;
        const uint8_t* blk = head0 + (kp[b] < 0 ? 0 : kp[b]) * a.t.page_bytes;
        const uint32_t row = (t + 16 * b) & (a.t.P - 1);
        const uint8_t* at = blk + row * (D / 2);
        if constexpr (D == 128) {
          const u4 x = *reinterpret_cast<const u4*>(at + k_off);
#pragma unroll
          for (int m = 0; m < M; ++m) kc[b][m] = x[m];
        } else {
          const u2 x = *reinterpret_cast<const u2*>(at + k_off);
#pragma unroll
          for (int m = 0; m < M; ++m) kc[b][m] = x[m];
        }
        ke[b] = (blk + kv_key_exps(a.t.P, D) + row * (D / kKvGroup))[k_off / 16];  // 16 bytes of codes an exponent
      }
    };
    auto load_values = [&](int t) __attribute__((always_inline)) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        vp[b] = kp[b];
        const uint8_t* blk = head0 + (vp[b] < 0 ? 0 : vp[b]) * a.t.page_bytes;
        const uint32_t row = (t + 16 * b) & (a.t.P - 1);
        const uint8_t* at = blk + kv_value_codes(a.t.P, D) + row * (D / 2);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (D == 128)
            vc[4 * b + r] = *reinterpret_cast<const uint32_t*>(at + v_off + r * (D / 2));
          else
            vc[4 * b + r] = *reinterpret_cast<const uint16_t*>(at + v_off + r * (D / 2));
        }
        ve[b] = *reinterpret_cast<const uint32_t*>(blk + kv_value_exps(a.t.P, D) + row + ve_off);
      }
    };

    if (tb < t1) {
      load_keys(tb);
      load_values(tb);
    }
    for (; tb < t1; tb += 32 * NW) {
      // -- scores of 32 tokens
      f4 sc[NT][2];
#pragma unroll
      for (int b = 0; b < 2; ++b) {
#pragma unroll
        for (int n = 0; n < NT; ++n) sc[n][b] = f4{0, 0, 0, 0};
        const float ks = exp_scale(ke[b]);
#pragma unroll
        for (int m = 0; m < M; ++m) {
          u4 kf = {dequant2<0>(kc[b][m], ks), dequant2<1>(kc[b][m], ks), dequant2<2>(kc[b][m], ks),
                   dequant2<3>(kc[b][m], ks)};
          // a poisoned key, or no page: scores NaN, seen where the mask lets them
          if (m == 0) kf[0] |= ke[b] == kKvPoison || kp[b] < 0 ? ~0u : 0u;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int p = 0; p < NQ; ++p) sc[n][b] = mfma16(kf, qf[n][p][m], sc[n][b]);
          if constexpr (NQ == 3) __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (tb + 32 * NW < t1) {
        if (++step % 32 == 0) pages = load_pages(tb + 32 * NW);
        load_keys(tb + 32 * NW);
      }
      __builtin_amdgcn_sched_barrier(0);  // here and below: fewer registers alive
      // -- tokens behind a row's own; values there, or of no page, may be
      // anything, and become zeros
      const bool tail = tb + 31 > first_limit || vp[0] < 0 || vp[1] < 0;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int b = 0; b < 2; ++b) sc[n][b] *= a.scale;
      if (tail) {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int t = tb + 16 * b + 4 * j + r;
#pragma unroll
            for (int n = 0; n < NT; ++n) sc[n][b][r] = t > limit[n] ? -INFINITY : sc[n][b][r];
            const bool none = t >= t1 || vp[b] < 0;
            vc[4 * b + r] = none ? 0 : vc[4 * b + r];
            ve[b] = none ? (ve[b] & ~(0xFFu << (8 * r))) | (127u << (8 * r)) : ve[b];
          }
      }
      // -- weights: the running maximum is moved only when a score passes it
      // by 8 (weights then stay below 2^8, and the sums keep their 24 bits)
      u4 pf[NT][NP];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float best = fmaxf(fmaxf(fmaxf(sc[n][0][0], sc[n][0][1]), fmaxf(sc[n][0][2], sc[n][0][3])),
                           fmaxf(fmaxf(sc[n][1][0], sc[n][1][1]), fmaxf(sc[n][1][2], sc[n][1][3])));
        if (__ballot(best > mx[n] + 8.0f) != 0) {
          best = fmaxf(max_xor32(max_xor16(best)), mx[n]);
          const float keep = mx[n] == best ? 1.0f : exp2_hw(mx[n] - best);
          mx[n] = best;
          sum[n] *= keep;
#pragma unroll
          for (int m = 0; m < C; ++m) o[n][m] *= keep;
        }
        const float base = mx[n] == -INFINITY ? 0.0f : mx[n];
        float w[8];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int r = 0; r < 4; ++r) w[4 * b + r] = exp2_hw(sc[n][b][r] - base);
        sum[n] += ((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7]));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t t[NP];
          split_weights<NP>(w[2 * e], w[2 * e + 1], t);
#pragma unroll
          for (int p = 0; p < NP; ++p) pf[n][p][e] = t[p];
        }
      }
      __builtin_amdgcn_sched_barrier(0);
      // -- values: two channels of the 8 tokens at a time
      auto channels = [&](auto pick) __attribute__((always_inline)) {
        constexpr int c = decltype(pick)::value;
        uint32_t x[8];
#pragma unroll
        for (int t = 0; t < 8; ++t) x[t] = dequant2<c>(vc[t], exp_scale((ve[t / 4] >> (8 * (t % 4))) & 0xFF));
        const u4 even = {pack_lo(x[0], x[1]), pack_lo(x[2], x[3]), pack_lo(x[4], x[5]), pack_lo(x[6], x[7])};
        const u4 odd = {pack_hi(x[0], x[1]), pack_hi(x[2], x[3]), pack_hi(x[4], x[5]), pack_hi(x[6], x[7])};
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            o[n][2 * c] = mfma16(even, pf[n][p], o[n][2 * c]);
            o[n][2 * c + 1] = mfma16(odd, pf[n][p], o[n][2 * c + 1]);
          }
        __builtin_amdgcn_sched_barrier(0);
      };
      channels(std::integral_constant<int, 0>{});
      channels(std::integral_constant<int, 1>{});
      if constexpr (C == 8) {
        channels(std::integral_constant<int, 2>{});
        channels(std::integral_constant<int, 3>{});
      }
      if (tb + 32 * NW < t1) load_values(tb + 32 * NW);
    }

    // -- join the waves: row n of a tile, channels C (4j + r) + m.  The lane's
    // place is derived from an opaque thread id: hoisted out of the loop over
    // tiles, these addresses would be spilled over the steps.
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int e16 = tid % 16, ej = tid % 64 / 16;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float total = sum_xor32(sum_xor16(sum[n]));
      if (ej == 0) {
        ml_sh[wave][16 * n + e16][0] = mx[n];
        ml_sh[wave][16 * n + e16][1] = total;
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int m = 0; m < C; m += 4)
          *reinterpret_cast<f4*>(&o_sh[wave][16 * n + e16][C * (4 * ej + r) + m]) =
              f4{o[n][m][r], o[n][m + 1][r], o[n][m + 2][r], o[n][m + 3][r]};
    }
    __syncthreads();
    constexpr int PER = D / 8;  // threads of a row, 8 channels each
    for (int it = tid; it < R * PER; it += 64 * NW) {
      const int r = it / PER, c = 8 * (it % PER), row = row0 + r;
      if (row > last_row) continue;
      float top = -INFINITY;
#pragma unroll
      for (int w = 0; w < NW; ++w) top = fmaxf(top, ml_sh[w][r][0]);
      float acc[8] = {}, total = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float m = ml_sh[w][r][0];
        const float f = m == -INFINITY ? (top == -INFINITY ? 1.0f : 0.0f) : exp2_hw(m - top);
        // a wave without a finite maximum holds zeros, or NaN from a page
        // that does not exist or a poisoned key
        total += m == -INFINITY ? ml_sh[w][r][1] : ml_sh[w][r][1] * f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(o_sh[w][r][c + e], f, acc[e]);
      }
      const int tok = row / a.group, g = row - tok * a.group;
      const int64_t at = (q.n0 + tok) * a.q_heads + static_cast<int64_t>(h) * a.group + g;
      if (splits == 1) {
        // every row sees its own token: a sum of zero means that its largest
        // score is infinite, and 0 / 0 makes the row NaN, as a bad sequence's are
        const float inv = q.bad ? __builtin_nanf("") : 1.0f / total;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= inv;
        store8<DT>(a.out, at * D + c, acc);
      } else {
        const int64_t slot = static_cast<int64_t>(sp) * a.t.n_tokens * a.q_heads + at;
        store8<KDA_F32>(a.part, slot * D + c, acc);
        if (c == 0) {
          a.part_ml[2 * slot] = top;
          a.part_ml[2 * slot + 1] = total;
        }
      }
    }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Attention: prompts
// ---------------------------------------------------------------------------

// f(0), f(1), .. with constants
template <typename F, int... I>
__device__ __forceinline__ void each_of(F f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}

// in bf16, or in fp16
template <bool HALF>
__device__ __forceinline__ f16v mfma32(u4 a, u4 b, f16v c) {
  if constexpr (HALF)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(h8, a), __builtin_bit_cast(h8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf8, a), __builtin_bit_cast(bf8, b), c, 0, 0, 0);
}

template <bool HALF, int SEL>
__device__ __forceinline__ uint32_t dequant2_as(uint32_t c, float scale) {
  if constexpr (HALF)
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(c, scale, SEL));
  else
    return dequant2<SEL>(c, scale);
}

// Exponent bytes whose values fp16 holds exactly: 0.5 * 2^-23 = 2^-24 to
// 6 * 2^13 = 49152; and kKvMinExp, which 32 zeros have (and numbers below 2^-122).
constexpr int kHalfMinExp = 104, kHalfMaxExp = 140;

// The largest exponent byte of those seen, and the smallest but kKvMinExp.
struct ExpRange {
  u16x2 top = {0, 0}, low = {0xFFFF, 0xFFFF};
  __device__ __forceinline__ void take2(uint32_t e) {  // two bytes, in bits 0..7 and 16..23
    const u16x2 x = __builtin_bit_cast(u16x2, e);
    top = __builtin_elementwise_max(top, x);
    low = __builtin_elementwise_min(low, static_cast<u16x2>(x - static_cast<uint16_t>(kKvMinExp + 1)));
  }
  __device__ __forceinline__ bool in_half() const {
    constexpr uint16_t least = kHalfMinExp - (kKvMinExp + 1), most = kHalfMaxExp;
    const u16x2 over = __builtin_elementwise_sub_sat(top, u16x2{most, most});
    const u16x2 under = __builtin_elementwise_sub_sat(u16x2{least, least}, low);
    return __builtin_bit_cast(uint32_t, over | under) == 0;
  }
};

// Many rows: 128 rows of one sequence and cached head (32 a wave) against one
// split of its tokens, 64 of them at a time.
//
// The products are the rows kernel's, S^T = K Q^T and O^T = V^T P^T, here as
// 32x32x16: weights go from the first result's registers into the second
// product without leaving the lane.  The tile's codes are turned into bf16
// once for the four waves: each thread takes D / 4 channels of a key and
// D / 16 channels of 4 values, and writes keys as rows of tokens and values as
// rows of channels, so every operand is one 16-byte LDS read.  Rows are 16
// bytes longer than their data: 16 rows in turn then start on different
// 16-byte pieces of the 256 bytes that LDS serves at once.
// A wave's matrix and vector work overlap: the scores of the next tile are
// multiplied while this one's weights are formed, and the codes of later
// tiles are turned while the values are multiplied.  Keys are therefore
// staged one tile further ahead than values; one barrier a tile.  Step i reads
// key buffer (i + 1) % 2 and value buffer i % 2 and writes the two others, which
// were last read before the barrier that ends step i - 1; the first tile's scores
// have a barrier of their own.
//
// 16-bit types take everything in fp16 first: E2M1 times 2^(e - 127) is exact
// there for e in 104..140, an fp16 query is itself, a bf16 query divided by its
// row's power of two loses at most 2^-25 of the row's largest channel, and
// weights, at most 2^15, keep 11 bits down to 2^-21 of the largest, in both sums
// alike: fp16 chunks are off by 2.45e-4 of their norm, 2.06e-4 with a second fp16
// piece of each weight, which takes 207 us instead of 152 (8192 fp16 rows 737
// instead of 529); bf16 outputs do not show it.  One product for each operand
// then does what two or three bf16 pieces do.  The exponents are looked at
// before their tiles are added, two tiles at a time: a block that
// meets another one goes on from there in bf16 pieces, with the sums that it has
// (8192 bf16 rows with one such token near the front: 720 us, fp16 820; near the
// end 530).  Poisoned keys are NaN in fp16 too.
//
// Bound by how much of the vector work two waves a SIMD hide behind the products
// (the matrix cores are busy 48% of the cycles, waves wait 25% of theirs): 8192 bf16
// rows of 32 query heads 536 us, 1026 TFLOP/s of the 1211 that a large bf16 matrix
// product reaches (829 us with two bf16 pieces for a weight, one tile after the
// other).
template <int DT, int D>
__global__ __launch_bounds__(256, DT == KDA_F32 ? 1 : 2) void kda_kv_tiles_kernel(KvAttendArgs a) {
  constexpr int KT = 64;            // tokens of a tile
  constexpr int KS = D / 16;        // products over the channels
  constexpr int CB = D / 32;        // 32-channel blocks
  constexpr int VC = D / 16;        // channels of a thread's values
  constexpr int R = kTileRows;
  constexpr int KROW = 2 * D + 16, VROW = 2 * KT + 16;  // LDS bytes of a token's key, of a channel's values
  constexpr int KBUF = KT * KROW, VBUF = D * VROW;
  __shared__ __attribute__((aligned(16))) char k_sh[2 * KBUF];
  __shared__ __attribute__((aligned(16))) char v_sh[2 * VBUF];
  // whether a wave met an exponent that fp16 does not hold
  __shared__ __attribute__((aligned(4))) uint8_t far_sh[4];

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // A sequence's last tiles see the most tokens and go first.  Heads go round
  // the XCDs: with 8 of them each stays on one, and in its L2.
  const int h = blockIdx.x % a.t.H, turn = blockIdx.x / a.t.H;
  const int sp = turn % a.n_splits;
  const TileAt mine = tile_of_slot(a, a.slots - 1 - turn / a.n_splits);
  if (mine.tile < 0) return;
  const int s = mine.s;
  const Seq q = seq_of(a.t, s);
  if (q.skip) return;
  const int all_rows = q.rows * a.group;
  if (mine.tile >= (all_rows + R - 1) / R) return;
  const int row0 = mine.tile * R;
  const int block_bytes = kv_block_bytes(a.t.P, D);
  const uint8_t* head0 = a.t.base + static_cast<int64_t>(h) * block_bytes;
  const_i32* table = (const_i32*)(a.t.page_table + static_cast<int64_t>(s) * a.t.max_pages);

  const int last_row = (row0 + R < all_rows ? row0 + R : all_rows) - 1;
  const int vis = q.past + last_row / a.group + 1;
  const int splits = q.bad ? 1 : kv_splits(vis, a);
  if (sp >= splits) return;
  const int t0 = q.bad ? 0 : sp * a.chunk;
  const int t1 = q.bad ? 0 : sp == splits - 1 ? vis : t0 + a.chunk;
  const int w_first = q.past + (row0 + 32 * wave) / a.group;  // the last token all of the wave's rows see

  // Weights of 16-bit types are taken 2^7 times larger, at most 2^15: fp16 has
  // room for smaller ones then.
  constexpr float UP = DT == KDA_F32 ? 0.0f : 7.0f;
  f16v zero;
#pragma unroll
  for (int e = 0; e < 16; ++e) zero[e] = 0.0f;
  f16v o[CB];
#pragma unroll
  for (int c = 0; c < CB; ++c) o[c] = zero;
  float mx = -INFINITY, sum = 0.0f;

  // Adds the tokens from `from` on; with HALF in fp16, up to a tile that does not
  // fit.  Returns the first token that is left.
  auto attend = [&](auto in_half, int from) __attribute__((always_inline)) {
  constexpr bool HALF = decltype(in_half)::value;
  constexpr int NQ = HALF ? 1 : q_pieces<DT>(), NP = HALF ? 1 : w_pieces<DT>();
  // 16-bit types in bf16 keep two pieces of weights (fp16: of queries too), and
  // have no registers for a second tile's scores
  constexpr bool PIPED = HALF || DT == KDA_F32;
  // The lane's places, from an opaque thread id: those of the one form kept over
  // the other's steps would be spilled.
  int tid = threadIdx.x;
  asm volatile("" : "+v"(tid));
  const int lane = tid % 64, i32 = lane % 32, half = lane / 32;
  // -- a thread's share of a tile's codes: key kt, channels D / 4 kj..; values
  // 4 vt .. 4 vt + 3, channels VC vo..  A wave's 16 tokens lie on one page.
  const int kt = tid / 4, kj = tid % 4, vt = 4 * wave + lane % 4, vo = lane / 4;
  // Values' row 16 n + vo holds channel VC vo + n: the channels that a lane
  // ends up with are then neighbours.  4 tokens are half a 16-byte piece: a
  // lane's 8 tokens in the product are 4 half .. + 3 and 8 + 4 half .. + 3 of 16.
  const int k_to = kt * KROW + 16 * kj * (D / 32);
  const int v_to = vo * VROW + 16 * (2 * (vt / 4) + vt % 2) + 8 * ((vt / 2) % 2);
  const int k_at = i32 * KROW + 16 * half, v_at = i32 * VROW + 16 * half;
  // and in a block, from the first token row of the wave's 16
  const uint32_t k_off = kt % 16 * (D / 2) + kj * (D / 8);
  const uint32_t v_off = 4 * (lane % 4) * (D / 2) + vo * (VC / 2);
  const uint32_t ve_off = (vo * VC / kKvGroup) * a.t.P + 4 * (lane % 4);

  const int row = row0 + 32 * wave + i32;
  const int r_in = row <= last_row ? row : last_row;
  const int tok = r_in / a.group, g = r_in - tok * a.group;
  const int limit = row <= last_row ? q.past + tok : -1;
  float scale = a.scale;
  u4 qf[NQ][KS];
  kernel_args args0 = (kernel_args)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(args0));
  const int64_t q_at = (q.n0 + tok) * args0->q_stride + (static_cast<int64_t>(h) * args0->group + g) * D + 8 * half;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    if constexpr (HALF && DT == KDA_F16) {
      qf[0][ks] = *reinterpret_cast<const u4*>(static_cast<const uint16_t*>(args0->q) + q_at + 16 * ks);
      const uint32_t flip = args0->sign < 0.0f ? 0x80008000u : 0u;
#pragma unroll
      for (int k = 0; k < 4; ++k) qf[0][ks][k] ^= flip;
    } else {
      u4 x[q_pieces<DT>()];
      load_query<DT>(args0->q, q_at + 16 * ks, args0->sign, x);
#pragma unroll
      for (int p = 0; p < NQ; ++p) qf[p][ks] = x[p];
    }
  }
  if constexpr (HALF && DT == KDA_BF16) {
    // the row's largest exponent, from both lanes that hold it
    u16x2 top = {0, 0};
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, qf[0][ks][k] & 0x7FFF7FFFu));
    int ex = (top[0] > top[1] ? top[0] : top[1]) >> 7;
    const auto both = __builtin_amdgcn_permlane32_swap(ex, ex, false, false);
    ex = static_cast<int>(both[0] > both[1] ? both[0] : both[1]);
    ex = ex == 0 ? 127 : ex < 253 ? ex : 253;
    const float down = exp_scale(254 - ex);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t w = qf[0][ks][k];
        const h2 y = {static_cast<_Float16>(__uint_as_float(w << 16) * down),
                      static_cast<_Float16>(__uint_as_float(w & 0xFFFF0000u) * down)};
        qf[0][ks][k] = __builtin_bit_cast(uint32_t, y);
      }
    scale = fminf(fmaxf(scale * exp_scale(ex), 0x1p-149f), FLT_MAX);  // as a.scale
  }
  ExpRange seen;

  // The codes in flight; HALF: and the exponents of the next tile's values, from
  // every second step's key load, whose block they are in.
  uint32_t kc[D / 32], ke, vc[4], ve, ve_next;
  auto page_of = [&](int tb) __attribute__((always_inline)) {
    const int t = tb + 16 * wave;
    const int page = t < t1 ? table[t >> a.t.log_p] : -1;
    return page < a.t.n_pages ? page : -1;
  };
  auto load_keys = [&](int tb, auto with_values) __attribute__((always_inline)) {
    const int page = page_of(tb);
    if constexpr (decltype(with_values)::value) ve_next = 0x7F7F7F7Fu;
    if (page >= 0) {
      const uint8_t* blk = head0 + page * a.t.page_bytes;
      const uint32_t r = (tb + 16 * wave) & (a.t.P - 1);
      const uint8_t* at = blk + r * (D / 2);
      if constexpr (D == 128) {
        const u4 x = *reinterpret_cast<const u4*>(at + k_off);
#pragma unroll
        for (int m = 0; m < 4; ++m) kc[m] = x[m];
      } else {
        const u2 x = *reinterpret_cast<const u2*>(at + k_off);
        kc[0] = x[0], kc[1] = x[1];
      }
      ke = (blk + kv_key_exps(a.t.P, D) + r * (D / kKvGroup))[k_off / 16];  // 16 bytes of codes an exponent
      if constexpr (decltype(with_values)::value)
        ve_next = *reinterpret_cast<const uint32_t*>(blk + kv_value_exps(a.t.P, D) + r + ve_off);
    } else {
      ke = kKvPoison;  // scores NaN, seen only where the mask lets them
#pragma unroll
      for (int m = 0; m < D / 32; ++m) kc[m] = 0;
    }
  };
  auto load_values = [&](int tb, auto with_exps) __attribute__((always_inline)) {
    const int page = page_of(tb);
    if constexpr (!decltype(with_exps)::value) ve = ve_next;
    if (page >= 0) {
      const uint8_t* blk = head0 + page * a.t.page_bytes;
      const uint32_t r = (tb + 16 * wave) & (a.t.P - 1);
      const uint8_t* at = blk + kv_value_codes(a.t.P, D) + r * (D / 2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (D == 128)
          vc[e] = *reinterpret_cast<const uint32_t*>(at + v_off + e * (D / 2));
        else
          vc[e] = *reinterpret_cast<const uint16_t*>(at + v_off + e * (D / 2));
      }
      if constexpr (decltype(with_exps)::value)
        ve = *reinterpret_cast<const uint32_t*>(blk + kv_value_exps(a.t.P, D) + r + ve_off);
    } else {
      if constexpr (decltype(with_exps)::value) ve = 0x7F7F7F7Fu;
#pragma unroll
      for (int e = 0; e < 4; ++e) vc[e] = 0;
    }
  };
  // dword m of the codes of the key in tile tb
  auto stage_key = [&](int buf, int m, int tb) __attribute__((always_inline)) {
    const float ks = exp_scale(ke);
    u4 x = {dequant2_as<HALF, 0>(kc[m], ks), dequant2_as<HALF, 1>(kc[m], ks), dequant2_as<HALF, 2>(kc[m], ks),
            dequant2_as<HALF, 3>(kc[m], ks)};
    if (m == 0) {
      const bool poison = ke == kKvPoison;  // NaN in either type
      if constexpr (HALF) seen.take2((tb + kt < t1 && !poison ? ke : 127u) * 0x10001u);
      x[0] |= poison ? ~0u : 0u;
    }
    *reinterpret_cast<u4*>(k_sh + buf * KBUF + k_to + 16 * m) = x;
  };
  // values behind the last token may be anything: zeros
  auto end_exps = [&](int tb, uint32_t& exps, auto zero_code) __attribute__((always_inline)) {
    if (tb + KT > t1) {
      int id = threadIdx.x;  // (as above: kept for this alone, vt was spilled)
      asm volatile("" : "+v"(id));
      const int t = tb + 16 * wave + 4 * (id % 4);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (t + e >= t1) {
          zero_code(e);
          exps = (exps & ~(0xFFu << (8 * e))) | (127u << (8 * e));
        }
    }
  };
  auto end_values = [&](int tb) __attribute__((always_inline)) { end_exps(tb, ve, [&](int e) { vc[e] = 0; }); };
  auto see = [&](uint32_t exps) __attribute__((always_inline)) {
    seen.take2(exps & 0x00FF00FFu);
    seen.take2((exps >> 8) & 0x00FF00FFu);
  };
  // channels 2 c2 and 2 c2 + 1 of the 4 values
  auto stage_value = [&](int buf, auto pick) __attribute__((always_inline)) {
    constexpr int c2 = decltype(pick)::value;
    uint32_t x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = dequant2_as<HALF, c2>(vc[e], exp_scale((ve >> (8 * e)) & 0xFF));
    *reinterpret_cast<u2*>(v_sh + buf * VBUF + 32 * c2 * VROW + v_to) = u2{pack_lo(x[0], x[1]), pack_lo(x[2], x[3])};
    *reinterpret_cast<u2*>(v_sh + buf * VBUF + (32 * c2 + 16) * VROW + v_to) =
        u2{pack_hi(x[0], x[1]), pack_hi(x[2], x[3])};
  };
  // product i of a tile's scores: channels 16 (i / 2).., tokens 32 (i % 2)..
  auto key_piece = [&](int buf, int i) __attribute__((always_inline)) {
    const int ks = i / 2, b = i % 2;
    return *reinterpret_cast<const u4*>(k_sh + buf * KBUF + k_at + 32 * ks + 32 * b * KROW);
  };
  auto score = [&](int i, u4 kf, f16v (&out)[2]) __attribute__((always_inline)) {
#pragma unroll
    for (int p = 0; p < NQ; ++p) out[i % 2] = mfma32<HALF>(kf, qf[p][i / 2], i / 2 == 0 && p == 0 ? zero : out[i % 2]);
  };
  // product i of the outputs: tokens 16 (i / CB).., rows 32 (i % CB)..
  auto value_piece = [&](int buf, int i) __attribute__((always_inline)) {
    return *reinterpret_cast<const u4*>(v_sh + buf * VBUF + v_at + 32 * (i / CB) + 32 * (i % CB) * VROW);
  };
  f16v sc0[2], sc1[2];  // scores of tiles in turn

  if constexpr (HALF) far_sh[wave] = 0;
  constexpr std::true_type yes{};
  constexpr std::false_type no{};
  load_keys(from, no);
  load_values(from, yes);
#pragma unroll
  for (int m = 0; m < D / 32; ++m) stage_key(0, m, from);
  load_keys(from + KT, no);
  end_values(from);
  if constexpr (HALF) see(ve);
  stage_value(0, std::integral_constant<int, 0>{});
  stage_value(0, std::integral_constant<int, 1>{});
  if constexpr (D == 128) {
    stage_value(0, std::integral_constant<int, 2>{});
    stage_value(0, std::integral_constant<int, 3>{});
  }
  load_values(from + KT, yes);
#pragma unroll
  for (int m = 0; m < D / 32; ++m) stage_key(1, m, from + KT);
  load_keys(from + 2 * KT, no);
  if constexpr (HALF) {
    end_values(from + KT);
    see(ve);
  }
  // A wave that met a far exponent says so before an odd step's barrier, and the
  // block turns away behind it (the even step's barrier lies between that look
  // and the next odd step's word).
  auto report = [&]() __attribute__((always_inline)) {
    if (__ballot(!seen.in_half()) != 0) far_sh[wave] = 1;
    seen = ExpRange{};
  };
  if constexpr (HALF) report();
  __syncthreads();
  if constexpr (PIPED) {
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) score(i, key_piece(0, i), sc0);
    __syncthreads();  // all waves have these keys: the first step writes over them
  }
  auto top_score = [&](const f16v (&x)[2]) __attribute__((always_inline)) {
    float y = -INFINITY;
#pragma unroll
    for (int e = 0; e < 16; ++e) y = max_nan(y, max_nan(x[0][e], x[1][e]));
    return y;
  };
  float best = PIPED ? top_score(sc0) : 0.0f;
  // Even steps look at what the block has met: their own and the next step's
  // values, and their next tile's keys (keys of the next step's next tile are
  // used in the step after that one).  False: nothing is added.
  auto step = [&](int tb, auto which, f16v (&sc)[2], f16v (&next)[2]) __attribute__((always_inline)) {
    constexpr int buf = decltype(which)::value;
    if constexpr (HALF && buf == 0) {
      if (__builtin_amdgcn_readfirstlane(*reinterpret_cast<const uint32_t*>(far_sh)) != 0) return false;
    }
    if constexpr (!PIPED) {
#pragma unroll
      for (int i = 0; i < 2 * KS; ++i) {
        score(i, key_piece(buf, i), sc);
        __builtin_amdgcn_sched_barrier(0);
      }
      best = top_score(sc);
      __syncthreads();  // this buffer's next keys are written below
    }
    if (tb + KT - 1 > w_first) {
      const int left = limit - tb - 4 * half;  // the last of the lane's tokens its row sees
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int e = 0; e < 16; ++e) sc[b][e] = 32 * b + 8 * (e / 4) + e % 4 > left ? -INFINITY : sc[b][e];
      best = top_score(sc);
    }
    // the running maximum moves only when a score passes it by 8
    if (__ballot(best * scale > mx + 8.0f) != 0) {
      const float to = fmaxf(max_xor32(best * scale), mx);
      const float keep = mx == to ? 1.0f : exp2_hw(mx - to);
      mx = to;
      sum *= keep;
#pragma unroll
      for (int c = 0; c < CB; ++c) o[c] *= keep;
    }
    end_values(tb + KT);
    const float base = (mx == -INFINITY ? 0.0f : -mx) + UP;
    // -- this tile's weights, the next one's scores: after each product the
    // vector work that fits beside it, operands read AHEAD products early
    constexpr int AHEAD = 2;
    u4 pf[4][NP], ring[AHEAD + 1];
    if constexpr (PIPED) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) ring[i] = key_piece(buf ^ 1, i);
    }
#pragma unroll
    for (int i = 0; i < 2 * KS; ++i) {
      if constexpr (PIPED) {
        if (i + AHEAD < 2 * KS) ring[(i + AHEAD) % (AHEAD + 1)] = key_piece(buf ^ 1, i + AHEAD);
        score(i, ring[i % (AHEAD + 1)], next);
      }
      constexpr int EACH = 16 / KS;  // weights beside a product
#pragma unroll
      for (int k = EACH * i; k < EACH * (i + 1); k += 2) {
        const int b = k / 16, e = k % 16;
        const float w0 = exp2_hw(fmaf(sc[b][e], scale, base)), w1 = exp2_hw(fmaf(sc[b][e + 1], scale, base));
        uint32_t x[NP];
        if constexpr (HALF) {
          // the sum takes the weights as they are multiplied: what their
          // rounding has in common falls out of the quotient
          const h2 w = {static_cast<_Float16>(w0), static_cast<_Float16>(w1)};
          sum = __builtin_amdgcn_fdot2(w, h2{1, 1}, sum, false);
          x[0] = __builtin_bit_cast(uint32_t, w);
        } else {
          sum += w0 + w1;
          split_weights<NP>(w0, w1, x);
        }
#pragma unroll
        for (int p = 0; p < NP; ++p) pf[2 * b + e / 8][p][(e % 8) / 2] = x[p];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // -- this tile's values; later tiles' codes; the next scores' maximum
    best = -INFINITY;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) ring[i] = value_piece(buf, i);
    auto output = [&](auto at) __attribute__((always_inline)) {
      constexpr int i = decltype(at)::value, G = 4 * CB, E = 32 / G;
      if (i + AHEAD < G) ring[(i + AHEAD) % (AHEAD + 1)] = value_piece(buf, i + AHEAD);
#pragma unroll
      for (int p = 0; p < NP; ++p) o[i % CB] = mfma32<HALF>(ring[i % (AHEAD + 1)], pf[i / CB][p], o[i % CB]);
      if constexpr (i % 4 == 0) stage_key(buf, i / 4, tb + 2 * KT);
      if constexpr (i % 4 == 2) stage_value(buf ^ 1, std::integral_constant<int, i / 4>{});
      if constexpr (PIPED) {
#pragma unroll
        for (int k = E * i; k < E * (i + 1); ++k) best = max_nan(best, next[k % 2][k / 2]);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    each_of(output, std::make_integer_sequence<int, 4 * CB>{});
    if constexpr (HALF && buf == 1) {
      see(ve);
      end_exps(tb + 2 * KT, ve_next, [](int) {});
      see(ve_next);
      report();
    }
    load_keys(tb + 3 * KT, std::integral_constant<bool, HALF && buf == 0>{});
    load_values(tb + 2 * KT, std::integral_constant<bool, !HALF || buf == 0>{});
    __syncthreads();
    return true;
  };
  for (int tb = from; tb < t1; tb += 2 * KT) {
    if (!step(tb, std::integral_constant<int, 0>{}, sc0, sc1)) return tb;
    if (tb + KT >= t1) break;
    if constexpr (PIPED) {
      if (!step(tb + KT, std::integral_constant<int, 1>{}, sc1, sc0)) return tb + KT;
    } else {
      if (!step(tb + KT, std::integral_constant<int, 1>{}, sc0, sc1)) return tb + KT;
    }
  }
  return t1;
  };
  if constexpr (DT == KDA_F32) {
    attend(std::false_type{}, t0);
  } else {
    const int left = attend(std::true_type{}, t0);
    if (left < t1) attend(std::false_type{}, left);
  }

  // The lane's row and the arguments once more, from an opaque thread id and
  // address: kept from above, they would be spilled over the steps.
  int again = threadIdx.x;
  kernel_args args = (kernel_args)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+v"(again), "+s"(args));
  // -- rows out: element e of block c is row 8 (e / 4) + 4 half + e % 4 of
  // 32 c.., channel 2 c + e / 8 of the VC at VC (row % 16)
  sum = sum_xor32(sum);
  const int out_half = again % 64 / 32, out_row = row0 + 32 * wave + again % 32;
  if (out_row <= last_row) {
    const int ot = out_row / args->group, og = out_row - ot * args->group;
    const int64_t at = (q.n0 + ot) * args->q_heads + static_cast<int64_t>(h) * args->group + og;
    const int64_t slot = static_cast<int64_t>(sp) * args->t.n_tokens * args->q_heads + at;
    const float inv = splits > 1 ? 1.0f : q.bad ? __builtin_nanf("") : 1.0f / sum;  // sum 0: NaN, as above
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int64_t c0 = VC * (8 * (e / 4) + 4 * out_half + e % 4);
      float x[VC];
#pragma unroll
      for (int n = 0; n < VC; ++n) x[n] = o[n / 2][8 * (n % 2) + e] * inv;
      if (splits == 1)
        store_channels<DT>(args->out, at * D + c0, x);
      else
        store_channels<KDA_F32>(args->part, slot * D + c0, x);
    }
    if (splits > 1 && out_half == 0) {
      args->part_ml[2 * slot] = mx - UP;
      args->part_ml[2 * slot + 1] = sum;
    }
  }
}

// Joins the splits of rows, D / 8 lanes across a row's channels.  Few splits:
// the lanes take theirs one after the other, four loads in flight, and a block
// takes 256 / (D / 8) rows.  MANY: a row has a whole block, splits lie across
// its lane groups, each with a maximum and sum of its own, so that no load
// waits for another split's.  Bound by latency: sequence, then partial rows (4.8
// us for the 768 rows of 64 requests and 12 heads).
template <int DT, int D, bool MANY, bool TILES>
__global__ __launch_bounds__(256) void kda_kv_join_kernel(KvAttendArgs a, int tile_rows) {
  constexpr int PER = D / 8, W = MANY ? 4 : 1;      // lanes of a row's channels, waves of a row
  constexpr int ROWS = MANY ? 1 : 256 / PER;
  constexpr int G = MANY ? 256 / PER : 1;           // splits taken at once
  __shared__ float part_sh[W][PER][10];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int c = 8 * (lane % PER), grp = MANY ? threadIdx.x / PER : 0;
  const int slices = (tile_rows + ROWS - 1) / ROWS;
  const int id = blockIdx.x;
  const int r = (id % slices) * ROWS + (MANY ? 0 : threadIdx.x / PER);
  // TILES: the tiles kernel's slots; else a.row_tiles tiles for each sequence
  const int tiles = TILES ? a.slots : a.row_tiles;
  const int h = id / slices / tiles % a.t.H;
  int rt0 = id / slices % tiles, s = id / slices / tiles / a.t.H;
  if constexpr (TILES) {
    const TileAt mine = tile_of_slot(a, rt0);
    if (mine.tile < 0) return;
    rt0 = mine.tile, s = mine.s;
  }
  const Seq q = seq_of(a.t, s);
  if (q.skip || q.bad || r >= tile_rows) return;
  const int all_rows = q.rows * a.group;
  const int64_t stride = a.t.n_tokens * a.q_heads;
  for (int64_t row0 = static_cast<int64_t>(rt0) * tile_rows + r; row0 < all_rows;
       row0 += TILES ? all_rows : a.row_tiles * tile_rows) {
    const int row = static_cast<int>(row0);
    const int end = row - r + tile_rows;  // of the tile
    const int splits = kv_splits(q.past + ((end < all_rows ? end : all_rows) - 1) / a.group + 1, a);
    if (splits <= 1) continue;  // written already
    const int tok = row / a.group, g = row - tok * a.group;
    const int64_t at = (q.n0 + tok) * a.q_heads + static_cast<int64_t>(h) * a.group + g;
    float acc[8] = {}, total = 0.0f, top = -INFINITY;
    // (m, l, x) joins this lane's; a side without a finite maximum holds
    // zeros, or NaN from a page that does not exist or a poisoned key
    auto join = [&](float m, float l, const float (&x)[8]) __attribute__((always_inline)) {
      const float to = fmaxf(top, m);
      const float f = top == to ? 1.0f : exp2_hw(top - to), y = m == to ? 1.0f : exp2_hw(m - to);
      top = to;
      total = fmaf(total, f, l * y);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(acc[e], f, x[e] * y);
    };
#pragma unroll 4
    for (int i = grp; i < splits; i += G) {
      const int64_t slot = i * stride + at;
      float x[8];
      load8<KDA_F32>(a.part, slot * D + c, x);
      join(a.part_ml[2 * slot], a.part_ml[2 * slot + 1], x);
    }
    if constexpr (MANY) {
#pragma unroll
      for (int m = PER; m < 64; m *= 2) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __shfl_xor(acc[e], m);
        const float om = __shfl_xor(top, m), ol = __shfl_xor(total, m);
        join(om, ol, x);
      }
      if (lane < PER) {
        part_sh[wave][lane][8] = top;
        part_sh[wave][lane][9] = total;
#pragma unroll
        for (int e = 0; e < 8; ++e) part_sh[wave][lane][e] = acc[e];
      }
      __syncthreads();
      if (threadIdx.x < PER) {
#pragma unroll
        for (int w = 1; w < W; ++w) {
          float x[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = part_sh[w][lane][e];
          join(part_sh[w][lane][8], part_sh[w][lane][9], x);
        }
      }
      __syncthreads();
    }
    const float inv = 1.0f / total;  // (a sum of zero: NaN, as above)
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= inv;
    if (!MANY || threadIdx.x < PER) store8<DT>(a.out, at * D + c, acc);
  }
}

// ---------------------------------------------------------------------------
// Launches
// ---------------------------------------------------------------------------

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

KvTables make_tables(const kda_kv_pool* kv, const int32_t* page_table, int32_t max_pages, const int32_t* cu,
                     const int32_t* past, int32_t n_seq, int64_t n_tokens) {
  KvTables t;
  t.base = static_cast<uint8_t*>(kv->base);
  t.page_table = page_table;
  t.cu = cu;
  t.past = past;
  t.page_bytes = static_cast<int64_t>(kv->H) * kv_block_bytes(kv->page_tokens, kv->D);
  t.n_tokens = n_tokens;
  t.n_pages = kv->n_pages;
  t.max_pages = max_pages;
  t.n_seq = n_seq;
  t.H = kv->H;
  t.P = kv->page_tokens;
  t.log_p = 31 - __builtin_clz(static_cast<unsigned>(kv->page_tokens));
  return t;
}

int status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_LAUNCH; }

// f(integral_constant<dtype>, integral_constant<D>)
template <typename F>
hipError_t by_type(kda_dtype dt, int D, F f) {
  auto with_d = [&](auto t) {
    return D == 128 ? f(t, std::integral_constant<int, 128>{}) : f(t, std::integral_constant<int, 64>{});
  };
  switch (dt) {
    case KDA_F32: return with_d(std::integral_constant<int, KDA_F32>{});
    case KDA_F16: return with_d(std::integral_constant<int, KDA_F16>{});
    default: return with_d(std::integral_constant<int, KDA_BF16>{});
  }
}

// A block takes 256 / (D / 8) tokens; with few of them the heads are dealt to
// more blocks, down to one head each.
int heads_a_block(int64_t token_tiles, int heads) {
  const int64_t most = (4096 + token_tiles - 1) / token_tiles;  // blocks wanted a token tile
  int64_t n = (heads + most - 1) / most;
  return static_cast<int>(n < 1 ? 1 : n);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" int kda_kv_append(const kda_kv_pool* kv, const int32_t* page_table, int32_t max_pages,
                             const int32_t* cu_seqlens, const int32_t* cache_lens, const void* k, const void* v,
                             int64_t k_stride, int64_t v_stride, const void* q, int64_t q_stride, void* q_out,
                             const float* cos, const float* sin, int32_t n_positions, int32_t rot_dim,
                             int32_t interleaved, int32_t n_seq, int64_t n_tokens, int32_t q_heads,
                             kda_dtype dtype, void* stream) {
  const int rc = kv_check(kv, max_pages, n_seq, n_tokens);
  if (rc != KDA_OK) return rc;
  const int size = kv_type_bytes(dtype);
  if (size == 0) return KDA_ERR_DTYPE_REFUSED;
  if (q_heads < 0 || q_heads > 65535 || n_positions < 0 || (interleaved != 0 && interleaved != 1)) return KDA_ERR_ARG;
  if (rot_dim < 0 || rot_dim > kv->D || rot_dim % 16 != 0) return KDA_ERR_SHAPE;
  if (n_seq == 0 || n_tokens == 0) return KDA_OK;
  if (page_table == nullptr || cu_seqlens == nullptr || cache_lens == nullptr || k == nullptr || v == nullptr)
    return KDA_ERR_NULL;
  if (q_heads > 0 && (q == nullptr || q_out == nullptr)) return KDA_ERR_NULL;
  if (rot_dim > 0 && (cos == nullptr || sin == nullptr)) return KDA_ERR_NULL;
  const int64_t kv_row = static_cast<int64_t>(kv->H) * kv->D, q_row = static_cast<int64_t>(q_heads) * kv->D;
  if (k_stride < kv_row || v_stride < kv_row || (q_heads > 0 && q_stride < q_row)) return KDA_ERR_ARG;
  if (!aligned(kv->base, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) ||
      !aligned(cos, 16) || !aligned(sin, 16) || !aligned(page_table, 4) || !aligned(cu_seqlens, 4) ||
      !aligned(cache_lens, 4) || k_stride * size % 16 != 0 || v_stride * size % 16 != 0 ||
      (q_heads > 0 && q_stride * size % 16 != 0))
    return KDA_ERR_ALIGN;
  KvAppendArgs a;
  a.t = make_tables(kv, page_table, max_pages, cu_seqlens, cache_lens, n_seq, n_tokens);
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  a.cos = cos;
  a.sin = sin;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.n_positions = rot_dim > 0 ? n_positions : INT32_MAX;
  a.half = rot_dim / 2;
  a.interleaved = interleaved;
  a.q_heads = q_heads;
  a.units = kv->H + q_heads;
  const int64_t tiles = (n_tokens + 256 / (kv->D / 8) - 1) / (256 / (kv->D / 8));
  a.units_per_block = heads_a_block(tiles, a.units);
  a.unit_blocks = (a.units + a.units_per_block - 1) / a.units_per_block;
  if (tiles * a.unit_blocks > kKvMaxBlocks) return KDA_ERR_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return status(by_type(dtype, kv->D, [&](auto t, auto d) {
    constexpr int DT = decltype(t)::value, D = decltype(d)::value;
    const dim3 grid(static_cast<uint32_t>(tiles * a.unit_blocks));
    // From 96 MiB of inputs on loads and stores pass the caches by (32 query and
    // 8 cached heads in bf16: 8192 tokens 63 -> 58 us, 32768 188 -> 166; 4096, which
    // the last-level cache still holds from the projection before, 28.7 -> 30.7).
    if ((kv_row * 2 + q_row) * size * n_tokens >= (96ll << 20))
      hipLaunchKernelGGL((kda_kv_append_kernel<DT, D, true>), grid, dim3(256), 0, st, a);
    else
      hipLaunchKernelGGL((kda_kv_append_kernel<DT, D, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
  }));
}

extern "C" int kda_kv_read(const kda_kv_pool* kv, const int32_t* page_table, int32_t max_pages,
                           const int32_t* cu_seqlens, const int32_t* first, void* k_out, void* v_out,
                           int64_t k_stride, int64_t v_stride, int32_t n_seq, int64_t n_tokens, kda_dtype dtype,
                           void* stream) {
  const int rc = kv_check(kv, max_pages, n_seq, n_tokens);
  if (rc != KDA_OK) return rc;
  const int size = kv_type_bytes(dtype);
  if (size == 0) return KDA_ERR_DTYPE_REFUSED;
  if (n_seq == 0 || n_tokens == 0) return KDA_OK;
  if (page_table == nullptr || cu_seqlens == nullptr || first == nullptr || (k_out == nullptr && v_out == nullptr))
    return KDA_ERR_NULL;
  const int64_t row = static_cast<int64_t>(kv->H) * kv->D;
  if ((k_out != nullptr && k_stride < row) || (v_out != nullptr && v_stride < row)) return KDA_ERR_ARG;
  if (!aligned(kv->base, 16) || !aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(page_table, 4) ||
      !aligned(cu_seqlens, 4) || !aligned(first, 4) || (k_out != nullptr && k_stride * size % 16 != 0) ||
      (v_out != nullptr && v_stride * size % 16 != 0))
    return KDA_ERR_ALIGN;
  KvReadArgs a;
  a.t = make_tables(kv, page_table, max_pages, cu_seqlens, first, n_seq, n_tokens);
  a.k_out = k_out;
  a.v_out = v_out;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  const int per = 256 / (kv->D / (dtype == KDA_F32 ? 4 : 8));  // tokens a block
  const int64_t tiles = (n_tokens + per - 1) / per;
  a.heads_per_block = heads_a_block(tiles, kv->H);
  a.head_blocks = (kv->H + a.heads_per_block - 1) / a.heads_per_block;
  if (tiles * a.head_blocks > kKvMaxBlocks) return KDA_ERR_ARG;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return status(by_type(dtype, kv->D, [&](auto t, auto d) {
    hipLaunchKernelGGL((kda_kv_read_kernel<decltype(t)::value, decltype(d)::value>),
                       dim3(static_cast<uint32_t>(tiles * a.head_blocks)), dim3(256), 0, st, a);
    return hipGetLastError();
  }));
}

extern "C" int kda_kv_attend(const kda_kv_pool* kv, const int32_t* page_table, int32_t max_pages,
                             const int32_t* cu_seqlens, const int32_t* cache_lens, const void* q,
                             int64_t q_stride, void* out, int32_t n_seq, int64_t n_tokens, int32_t max_rows,
                             int64_t max_kv_len, int32_t q_heads, kda_dtype dtype, float scale, void* workspace,
                             size_t workspace_bytes, void* stream) {
  int rc = kv_check(kv, max_pages, n_seq, n_tokens);
  if (rc == KDA_OK) rc = kv_check_attend(kv, n_tokens, max_rows, max_kv_len, q_heads, dtype);
  if (rc != KDA_OK) return rc;
  if (!std::isfinite(scale)) return KDA_ERR_ARG;
  const int size = kv_type_bytes(dtype);
  if (n_seq == 0 || n_tokens == 0) return KDA_OK;
  if (page_table == nullptr || cu_seqlens == nullptr || cache_lens == nullptr || q == nullptr || out == nullptr)
    return KDA_ERR_NULL;
  if (q_stride < static_cast<int64_t>(q_heads) * kv->D) return KDA_ERR_ARG;
  if (!aligned(kv->base, 16) || !aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 16) ||
      !aligned(page_table, 4) || !aligned(cu_seqlens, 4) || !aligned(cache_lens, 4) || q_stride * size % 16 != 0)
    return KDA_ERR_ALIGN;
  const size_t need = kda_kv_attend_workspace(kv, max_pages, n_seq, n_tokens, max_rows, max_kv_len, q_heads, dtype);
  if (need > 0 && workspace == nullptr) return KDA_ERR_NULL;
  if (need > workspace_bytes) return KDA_ERR_ARG;
  const int64_t cover = static_cast<int64_t>(max_pages) * kv->page_tokens;
  const KvPlan p = kv_plan(kv->H, kv->D, n_seq, n_tokens, max_rows,
                           max_kv_len > 0 && max_kv_len < cover ? max_kv_len : cover, q_heads, dtype);
  KvAttendArgs a;
  a.t = make_tables(kv, page_table, max_pages, cu_seqlens, cache_lens, n_seq, n_tokens);
  a.q = q;
  a.out = out;
  a.q_stride = q_stride;
  a.q_heads = q_heads;
  a.group = q_heads / kv->H;
  a.chunk = p.chunk;
  a.n_splits = p.n_splits;
  a.row_tiles = p.row_tiles;
  a.slots = p.slots;
  // Above zero, so that a masked score (-infinity) times it is what it was
  // (2^-149 times any score leaves its weight 1), and finite, so that a score of
  // zero is.
  a.scale = std::fmin(std::fmax(std::fabs(scale) * 1.44269504088896340736f, 0x1p-149f), FLT_MAX);
  a.sign = scale < 0.0f ? -1.0f : 1.0f;
  a.part = static_cast<float*>(workspace);
  a.part_ml = a.part == nullptr ? nullptr : a.part + static_cast<int64_t>(p.n_splits) * n_tokens * q_heads * kv->D;
  const int64_t tiles = kv_tiles(p, n_seq, kv->H);
  if (tiles * p.n_splits > kKvMaxBlocks) return KDA_ERR_ARG;  // (many splits: few tiles, so the join's blocks fit too)
  hipStream_t st = static_cast<hipStream_t>(stream);
  return status(by_type(dtype, kv->D, [&](auto t, auto d) {
    constexpr int DT = decltype(t)::value, D = decltype(d)::value;
    const dim3 grid(static_cast<uint32_t>(tiles * p.n_splits));
    if (p.tile_rows == kTileRows)
      hipLaunchKernelGGL((kda_kv_tiles_kernel<DT, D>), grid, dim3(256), 0, st, a);
    else if (p.waves == 8)
      hipLaunchKernelGGL((kda_kv_rows_kernel<DT, D, 1, 8>), grid, dim3(512), 0, st, a);
    else if (DT == KDA_F32 || p.tile_rows == 16)
      hipLaunchKernelGGL((kda_kv_rows_kernel<DT, D, 1, 4>), grid, dim3(256), 0, st, a);
    else if constexpr (DT != KDA_F32)
      hipLaunchKernelGGL((kda_kv_rows_kernel<DT, D, 2, 4>), grid, dim3(256), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && p.n_splits > 1) {
      // up to 8 splits a row in two rounds of loads, more side by side
      constexpr int rows = 256 / (D / 8);
      const bool many = p.n_splits > 8, in_slots = p.tile_rows == kTileRows;
      const dim3 joins(static_cast<uint32_t>(tiles * (many ? p.tile_rows : (p.tile_rows + rows - 1) / rows)));
      if (many && in_slots)
        hipLaunchKernelGGL((kda_kv_join_kernel<DT, D, true, true>), joins, dim3(256), 0, st, a, p.tile_rows);
      else if (many)
        hipLaunchKernelGGL((kda_kv_join_kernel<DT, D, true, false>), joins, dim3(256), 0, st, a, p.tile_rows);
      else if (in_slots)
        hipLaunchKernelGGL((kda_kv_join_kernel<DT, D, false, true>), joins, dim3(256), 0, st, a, p.tile_rows);
      else
        hipLaunchKernelGGL((kda_kv_join_kernel<DT, D, false, false>), joins, dim3(256), 0, st, a, p.tile_rows);
      e = hipGetLastError();
    }
    return e;
  }));
}
