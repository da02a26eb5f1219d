// kda_kv.h -- the paged 4-bit key/value cache: block layout, argument structs
// and launch-shape rules shared by the host checks (kda_kv_host.cpp) and the
// gfx950 kernels (kda_kv.hip).  Internal header.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kda_decode.h"
#include "kda_launch.h"

namespace kda {

constexpr int kKvGroup = 32;      // channels that share one exponent byte
constexpr int kKvMinExp = 2;      // exponent bytes stored: every value a normal bf16,
constexpr int kKvMaxExp = 252;    //   and 6 * 2^(252 - 127) finite
constexpr int kKvPoison = 255;    // key exponent of a token whose key or value was not finite
constexpr int kKvMaxHeads = 4096;
// Positions stay so far below 2^31 that a kernel's look ahead in int32 cannot pass it.
constexpr int64_t kKvMaxPositions = (1ll << 31) - 4096;
constexpr int64_t kKvMaxBlocks = INT32_MAX / 512;  // a launch's threads stay below 2^31

// Bytes of one (page, head) block of P tokens of D channels: key codes
// [P][D/2], value codes [P][D/2], key exponents [P][D/32], value exponents
// [D/32][P].
KDA_HD constexpr int kv_block_bytes(int P, int D) { return P * D + P * D / 16; }
KDA_HD constexpr int kv_value_codes(int P, int D) { return P * D / 2; }
KDA_HD constexpr int kv_key_exps(int P, int D) { return P * D; }
KDA_HD constexpr int kv_value_exps(int P, int D) { return P * D + P * D / kKvGroup; }

// The cache and the tables that place a launch's tokens in it.
struct KvTables {
  uint8_t* base;
  const int32_t* page_table;  // [n_seq][max_pages]
  const int32_t* cu;          // [n_seq + 1]
  const int32_t* past;        // [n_seq]: tokens before the launch's first one
  int64_t page_bytes;         // all heads of one page
  int64_t n_tokens;
  int32_t n_pages, max_pages, n_seq;
  int32_t H;                  // cached heads
  int32_t log_p;              // log2 of tokens a page
  int32_t P;
};

struct KvAppendArgs {
  KvTables t;
  const void* q;
  const void* k;
  const void* v;
  void* q_out;
  const float* cos;
  const float* sin;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  int32_t n_positions, half, interleaved, q_heads;
  int32_t units, units_per_block, unit_blocks;  // units: cached heads, then query heads
};

struct KvReadArgs {
  KvTables t;
  void* k_out;
  void* v_out;
  int64_t k_stride, v_stride;
  int32_t heads_per_block, head_blocks;
};

struct KvAttendArgs {
  KvTables t;
  const void* q;
  void* out;
  float* part;     // workspace: [n_splits][n_tokens * q_heads][D] sums, then
  float* part_ml;  //   [n_splits][n_tokens * q_heads][2] maxima and sums of weights
  int64_t q_stride;
  int32_t q_heads, group;       // group: query heads of one cached head
  int32_t chunk, n_splits;      // tokens a split covers
  int32_t row_tiles;            // tiles of rows a sequence is given blocks for
  int32_t slots;                // 128-row tiles: places for all sequences' tiles
  float scale;                  // |scale| * log2(e)
  float sign;                   // of scale: queries are multiplied by it
};

// How kda_kv_attend takes a launch.
struct KvPlan {
  int32_t tile_rows;  // rows (tokens x query heads of one cached head) a workgroup takes
  int32_t row_tiles;  // as in KvAttendArgs
  int32_t slots;
  int32_t chunk;
  int32_t n_splits;
  int32_t waves;      // of a workgroup
};

// Tiles of rows of a plan, over sequences and cached heads: a workgroup for each
// and every split.
inline int64_t kv_tiles(const KvPlan& p, int32_t n_seq, int32_t H) {
  return (p.slots > 0 ? p.slots : static_cast<int64_t>(n_seq) * p.row_tiles) * H;
}

KvPlan kv_plan(int32_t H, int32_t D, int32_t n_seq, int64_t n_tokens, int32_t max_rows,
               int64_t max_kv_len, int32_t q_heads, kda_dtype dtype);

// Checks shared by the entry points, in the documented order.
int kv_check(const kda_kv_pool* kv, int32_t max_pages, int32_t n_seq, int64_t n_tokens);

// What the attention asks of its numbers, and the bytes of an element (0: no type).
int kv_type_bytes(kda_dtype dtype);
int kv_check_attend(const kda_kv_pool* kv, int64_t n_tokens, int32_t max_rows, int64_t max_kv_len, int32_t q_heads,
                    kda_dtype dtype);

}  // namespace kda
