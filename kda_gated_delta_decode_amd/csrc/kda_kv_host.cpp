// kda_kv_host.cpp -- host half of the paged 4-bit key/value cache: argument
// checks, sizes, table validation and the split of an attention launch.
// Makes no HIP call, so every refusal can be exercised without a GPU.
#include <cstdint>
#include <new>
#include <unordered_map>

#include "kda_kv.h"

namespace kda {

static bool kv_shape_ok(int32_t n_pages, int32_t P, int32_t H, int32_t D) {
  return (D == 64 || D == 128) && (P == 16 || P == 32 || P == 64 || P == 128 || P == 256) && H >= 1 &&
         H <= kKvMaxHeads && n_pages >= 1;
}

int kv_check(const kda_kv_pool* kv, int32_t max_pages, int32_t n_seq, int64_t n_tokens) {
  if (kv == nullptr || kv->base == nullptr) return KDA_ERR_NULL;
  if (!kv_shape_ok(kv->n_pages, kv->page_tokens, kv->H, kv->D)) return KDA_ERR_SHAPE;
  if (n_seq < 0 || n_tokens < 0 || n_tokens > INT32_MAX || max_pages < 1) return KDA_ERR_ARG;
  if (static_cast<int64_t>(max_pages) * kv->page_tokens > kKvMaxPositions) return KDA_ERR_ARG;
  return KDA_OK;
}

int kv_type_bytes(kda_dtype dtype) {
  return dtype == KDA_F32 ? 4 : dtype == KDA_F16 || dtype == KDA_BF16 ? 2 : 0;
}

int kv_check_attend(const kda_kv_pool* kv, int64_t n_tokens, int32_t max_rows, int64_t max_kv_len, int32_t q_heads,
                    kda_dtype dtype) {
  if (kv_type_bytes(dtype) == 0) return KDA_ERR_DTYPE_REFUSED;
  if (q_heads < 1 || q_heads > 65535 || q_heads % kv->H != 0) return KDA_ERR_SHAPE;
  if (max_rows < 0 || max_kv_len < 0) return KDA_ERR_ARG;
  // a row index is token * group + head within the group
  if (n_tokens * (q_heads / kv->H) > INT32_MAX / 4) return KDA_ERR_ARG;
  return KDA_OK;
}

KvPlan kv_plan(int32_t H, int32_t D, int32_t n_seq, int64_t n_tokens, int32_t max_rows,
               int64_t max_kv_len, int32_t q_heads, kda_dtype dtype) {
  (void)D;  // one plan for both: its figures are of D = 128, those of four prompt chunks of D = 64
  KvPlan p;
  const int64_t rows = static_cast<int64_t>(max_rows < n_tokens ? max_rows : n_tokens) * (q_heads / H);
  // 128-row tiles share a tile's turned codes through LDS; below that every
  // wave turns its own.  17 to 32 rows of a 16-bit type share them in one wave
  // (32 rows of 8 requests at 4097 tokens: 26.4 us against 28.9 in 16-row
  // tiles); fp32's registers do not reach (36.7 against 34.4), and 33 to 64 rows
  // are faster as more workgroups of 16 (64 rows: 38 us, 46 in 32s, 40 in
  // 128s; 96 rows: 95, and 76 in 128s).
  p.tile_rows = rows > 64 ? 128 : rows > 16 && rows <= 32 && dtype != KDA_F32 ? 32 : 16;
  const int64_t row_tiles = rows < 1 ? 1 : (rows + p.tile_rows - 1) / p.tile_rows;
  p.row_tiles = static_cast<int32_t>(row_tiles);
  int64_t units = (n_seq < 1 ? 1 : n_seq) * row_tiles * H;
  p.slots = 0;
  if (p.tile_rows == 128) {
    // as many slots as any spread of the rows over the sequences may need
    const int64_t slots = n_tokens * (q_heads / H) / 128 + n_seq;
    p.slots = slots > INT32_MAX ? INT32_MAX : static_cast<int32_t>(slots);
    if (n_seq > 1) units = static_cast<int64_t>(p.slots) * H;
  }
  const auto per = [](int64_t x, int64_t n) { return (x + n - 1) / n; };
  // n splits of a cache, none shorter than `least`
  const auto chunk_of = [&](int64_t blocks, int64_t least) {
    const int64_t n = blocks / units;
    const int64_t c = per(max_kv_len, n < 1 ? 1 : n);
    return c < least ? least : c;
  };
  int64_t chunk;
  p.waves = 4;
  if (p.tile_rows == 16 && units <= 256 && max_kv_len <= 512) {
    // Small: eight waves take at most two steps each, and no second launch
    // joins splits (one token at 256, 512: 5.6, 6.8 us against 7.5, 7.6; at
    // 1001 it would be 9.5 against 8.1).
    p.waves = 8;
    chunk = max_kv_len;
  } else if (p.tile_rows < 128) {
    // Few rows.  768 workgroups are resident at once (three a compute unit).
    // One sequence: its splits are all alike, and one round of them is best
    // (131072 tokens, 8 cached heads: 38 us; 39.5 with 1024, 43 with 1536).
    // Several: their lengths differ, and twice as many leave less of the chip
    // idle at the end (64 ragged requests: 75 us; 81 with 768, 77 with 2048).
    // A split costs as much as some 200 tokens, so none is shorter than 512
    // (8 requests of 4097: 27 us; 31 with 384) unless the chip would stay empty.
    chunk = chunk_of(n_seq > 1 ? 1536 : 768, 512);
    if (per(max_kv_len, chunk) * units < 256) chunk = chunk_of(256, 128);
  } else {
    // Many rows, two workgroups a compute unit: one round of them for one
    // sequence (512 rows on 15000 tokens: 165 us; 190, 220 for 1024, 1536), at least
    // one for several, whose rows and lengths differ (4 chunks of up to 700 rows
    // on up to 16000 tokens, 226 slots: 3 splits 174 us, 2 or 4 some 210).
    // From 1024 tokens a split, whose first steps fill the pipeline and whose rows
    // are joined (2 chunks of 262 rows on 4400 tokens: 36 us, 45 with 512; 512
    // fp32 rows on 4000: 62 and 83).
    chunk = n_seq > 1 ? chunk_of(per(512, units) * units, 1024) : chunk_of(512, 1024);
  }
  chunk = per(chunk, 128) * 128;
  if (chunk < 128) chunk = 128;
  p.chunk = static_cast<int32_t>(chunk);
  // Of several sequences a rest of up to an eighth goes to the split before it
  // (8 requests of 8 rows at 4097 tokens: fp32, 12 heads 24.0 -> 22.7 us, 32 query
  // heads 34.8 -> 30.0); one sequence's splits all run at once, and a longer one
  // would end last (131072 tokens: 36.8 -> 37.4 us).
  p.n_splits = static_cast<int32_t>(per(max_kv_len - (n_seq > 1 ? chunk / 8 : 0), chunk));
  if (p.n_splits < 1) p.n_splits = 1;
  return p;
}

}  // namespace kda

using namespace kda;

extern "C" {

size_t kda_kv_pool_bytes(int32_t n_pages, int32_t page_tokens, int32_t H, int32_t D) {
  if (!kv_shape_ok(n_pages, page_tokens, H, D)) return 0;
  return static_cast<size_t>(n_pages) * H * kv_block_bytes(page_tokens, D);
}

size_t kda_kv_attend_workspace(const kda_kv_pool* kv, int32_t max_pages, int32_t n_seq, int64_t n_tokens,
                               int32_t max_rows, int64_t max_kv_len, int32_t q_heads, kda_dtype dtype) {
  if (kv_check(kv, max_pages, n_seq, n_tokens) != KDA_OK) return 0;
  if (kv_check_attend(kv, n_tokens, max_rows, max_kv_len, q_heads, dtype) != KDA_OK) return 0;
  if (n_seq == 0 || n_tokens == 0) return 0;
  const int64_t cover = static_cast<int64_t>(max_pages) * kv->page_tokens;
  const KvPlan p = kv_plan(kv->H, kv->D, n_seq, n_tokens, max_rows,
                           max_kv_len > 0 && max_kv_len < cover ? max_kv_len : cover, q_heads, dtype);
  if (p.n_splits == 1 || kv_tiles(p, n_seq, kv->H) * p.n_splits > kKvMaxBlocks) return 0;
  return static_cast<size_t>(p.n_splits) * n_tokens * q_heads * (kv->D + 2) * sizeof(float);
}

int kda_kv_validate(const kda_kv_pool* kv, const int32_t* page_table_host, int32_t max_pages,
                    const int32_t* cu_seqlens_host, const int32_t* cache_lens_host, int32_t n_seq,
                    int64_t n_tokens) {
  const int rc = kv_check(kv, max_pages, n_seq, n_tokens);
  if (rc != KDA_OK) return rc;
  if (n_seq == 0) return KDA_OK;
  if (page_table_host == nullptr || cu_seqlens_host == nullptr || cache_lens_host == nullptr)
    return KDA_ERR_NULL;
  if (cu_seqlens_host[0] < 0) return KDA_ERR_ARG;
  const int64_t cover = static_cast<int64_t>(max_pages) * kv->page_tokens;
  for (int32_t s = 0; s < n_seq; ++s) {
    if (cu_seqlens_host[s + 1] < cu_seqlens_host[s] || cu_seqlens_host[s + 1] > n_tokens) return KDA_ERR_ARG;
    if (cache_lens_host[s] < 0) return KDA_ERR_ARG;
    if (static_cast<int64_t>(cache_lens_host[s]) + cu_seqlens_host[s + 1] - cu_seqlens_host[s] > cover)
      return KDA_ERR_ARG;
  }
  try {
    // pages that hold a sequence's tokens exist; a page that takes new tokens
    // belongs to that sequence alone (pages before it may be shared)
    std::unordered_map<int32_t, int64_t> writer;  // page -> s * max_pages + index
    for (int pass = 0; pass < 2; ++pass)
      for (int32_t s = 0; s < n_seq; ++s) {
        const int32_t n = cu_seqlens_host[s + 1] - cu_seqlens_host[s];
        const int64_t used = (static_cast<int64_t>(cache_lens_host[s]) + n + kv->page_tokens - 1) / kv->page_tokens;
        const int64_t first_new = cache_lens_host[s] / kv->page_tokens;
        for (int64_t i = 0; i < used; ++i) {
          const int64_t at = static_cast<int64_t>(s) * max_pages + i;
          const int32_t page = page_table_host[at];
          if (page < 0 || page >= kv->n_pages) return KDA_ERR_SLOT;
          const bool written = n > 0 && i >= first_new;
          if (pass == 0 && written && !writer.emplace(page, at).second) return KDA_ERR_SLOT;
          if (pass == 1) {
            const auto it = writer.find(page);
            if (it != writer.end() && it->second != at) return KDA_ERR_SLOT;
          }
        }
      }
  } catch (const std::bad_alloc&) {  // `writer` has one entry a written page
    return KDA_ERR_ARG;
  }
  return KDA_OK;
}

}  // extern "C"
