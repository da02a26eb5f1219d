// kda_tree.h -- trees of drafted tokens: argument structs and host checks, shared
// by kda_tree_host.cpp, the recurrence (kda_tree.hip), the verification
// (kda_verify.hip) and the cache (kda_kv.hip).  Internal header.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kda_decode.h"
#include "kda_launch.h"

namespace kda {

constexpr int kMaxNodes = KDA_MAX_NODES;  // a node for each lane of a wave
constexpr int kMaxTreeHeads = 16384;      // rows of one request stay below 2^31 bytes apart

struct TreeArgs {
  const void* pool;
  const int32_t* init_ids;
  const int32_t* cu;       // [n_req + 1]
  const int32_t* parents;  // [n_tokens]
  const float* q;
  const float* k;
  const float* v;
  const float* g;
  const float* b;
  float* out;
  int64_t n_tokens;
  int32_t n_req, H, n_slots;
  int32_t max_nodes;
  float scale;
};

struct PathArgs {
  void* pool;
  const int32_t* init_ids;
  const int32_t* dst_ids;
  const int32_t* cu;
  const int32_t* path;  // [n_req][max_path]
  const int32_t* lens;  // [n_req]
  const float* k;
  const float* v;
  const float* g;
  const float* b;
  int64_t n_tokens;
  int32_t n_req, H, n_slots, max_path;
};

// Where a request's walk ended: what its last row's weights are made of.
struct VerifyStop {
  uint64_t refused;        // nodes tried there and refused, as bits
  int32_t last;            // the last accepted node; -1: the request has no walk
  int32_t tries;           // refused nodes
  double mass[KDA_MAX_NODES];  // with a draft: M at each try
};

struct VerifyArgs {
  const void* target;
  const void* draft;       // nullable
  const int32_t* cu;
  const int32_t* parents;
  const int32_t* tokens;
  const float* accept;     // [n_tokens]
  const float* sample;     // [n_req]
  int32_t* path;           // [n_req][max_path]
  int32_t* lens;
  int32_t* next;
  VerifyStop* stops;       // workspace: [n_req], then
  double* sums;            //   [n_req][runs]
  int64_t target_stride, draft_stride;  // elements between rows
  int64_t n_tokens;
  int32_t n_req, vocab, max_path;
  int32_t runs, run;       // runs of a row, entries of a run
};

// How a row of `vocab` probabilities is dealt to waves.
struct VerifyPlan {
  int32_t runs, run;
};
VerifyPlan verify_plan(int32_t vocab);

// Checks shared by kda_decode_tree and kda_decode_path, up to the counts.
int tree_check(const kda_pool* pool, int32_t n_req, int64_t n_tokens, kda_dtype state_dtype);
int verify_check(int32_t n_req, int64_t n_tokens, int32_t vocab, int32_t max_path, kda_dtype dtype);

}  // namespace kda
