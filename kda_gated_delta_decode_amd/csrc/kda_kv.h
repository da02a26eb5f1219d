// kda_kv.h -- the paged 4-bit key/value cache: block layout, argument structs
// and launch-shape rules shared by the host checks (kda_kv_host.cpp) and the
// gfx950 kernels (kda_kv.hip).  Internal header.
#pragma once

#include <math.h>
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
  const int32_t* positions;  // nullable: the rows of cos and sin, apart from the places
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

struct KvKeepArgs {
  KvTables t;
  const int32_t* path;  // [n_seq][max_path]
  const int32_t* lens;  // [n_seq]
  int32_t max_path;
};

struct KvAttendArgs {
  KvTables t;
  const void* q;
  void* out;
  float* part;     // workspace: [n_splits][n_tokens * q_heads][D] sums, then
  float* part_ml;  //   [n_splits][n_tokens * q_heads][2] maxima and sums of weights
  int64_t q_stride;
  int32_t q_heads, group;       // group: query heads of one cached head
  int32_t chunk, n_splits;      // tokens a split covers (large trees: n_splits places)
  int32_t row_tiles;            // tiles of rows a sequence is given blocks for
  int32_t slots;                // 128-row tiles: places for all sequences' tiles
  float scale;                  // |scale| * log2(e)
  float sign;                   // of scale: queries are multiplied by it
  const int32_t* parents;       // trees: [n_tokens]
  int32_t most_rows;            // trees: KDA_MAX_NODES; else no bound
  int64_t* starts;              // large trees, workspace: a sequence's first part, and parts of a tile above bit 32
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

// Large trees (more than 64 rows of a sequence and cached head): tiles are cut in parts
// of at least kKvTreeSteps 64-token steps, as many as there are places for.  (bf16, 32
// nodes, 32 / 8 heads: on 1000 tokens 16.0 us with 3 steps, 17.5 with 4, 18.8 with 8, on
// 4000 21.3, 20.6, and 26 with 12; with 2 16.3 and 23.2.)
constexpr int kKvTreeSteps = 3;
struct KvTreePlan {
  int32_t places;       // of 128 rows in the workspace; 0: no tile is cut
  int64_t blocks;
  int32_t row_tiles;    // tiles of a sequence that the join has blocks for
  bool many;            // some tiles may have many parts: the join takes them side by side
  int64_t join_blocks;
};
KvTreePlan kv_tree_plan(const kda_kv_pool* kv, int32_t n_seq, int32_t max_rows, int32_t group, int64_t cover,
                        int64_t max_kv_len, kda_dtype dtype);
// A tile of `steps` steps in parts of at most `each`.
KDA_HD inline int kv_tree_parts(int steps, int each) {
  return static_cast<int>((static_cast<uint32_t>(steps) + each - 1) / static_cast<uint32_t>(each));
}
// The most steps of a part, such that all parts find a place (INT32_MAX: no tile is
// cut).  steps, units: tiles (times cached heads) and their steps, of all sequences;
// parts(each): how many parts that makes, asked only where `one`.  one: the first
// length from steps / places on that fits, an eighth longer from one to the next
// (one step below 8, where an eighth is none); it is found, for parts that hold
// whole tiles are as many as units.  Else a length that is sure to fit: parts are at
// most steps / each + units.
template <typename PARTS>
KDA_HD inline int kv_tree_each(float steps, float units, int32_t places, bool one, const PARTS& parts) {
  const float room = static_cast<float>(places);
  if (places <= 0 || units >= room) return INT32_MAX;
  float x = one ? steps / room : 1.001f * steps / (room - units) + 1.0f;
  x = fmaxf(x, static_cast<float>(kKvTreeSteps));
  int each = x < 0x1p30f ? static_cast<int>(ceilf(x)) : 1 << 30;
  while (one && each < (1 << 30) && parts(each) > room) each += each < 8 ? 1 : each / 8;
  return each;
}
// Workspace: where each sequence's parts begin and how many a tile has, then the
// places, then their rows' maxima and sums.
inline int64_t kv_tree_head_bytes(int32_t n_seq) { return (static_cast<int64_t>(n_seq) + 31) / 32 * 32 * 8; }

// Checks shared by the entry points, in the documented order.
int kv_check(const kda_kv_pool* kv, int32_t max_pages, int32_t n_seq, int64_t n_tokens);

// What the attention asks of its numbers, and the bytes of an element (0: no type).
int kv_type_bytes(kda_dtype dtype);
int kv_check_attend(const kda_kv_pool* kv, int64_t n_tokens, int32_t max_rows, int64_t max_kv_len, int32_t q_heads,
                    kda_dtype dtype);

}  // namespace kda
