// kda_tree_host.cpp -- host half of the calls for trees of drafted tokens:
// argument checks, table validation and the split of a verification launch.
// Makes no HIP call, so every refusal can be exercised without a GPU.
#include <cstdint>

#include "kda_internal.h"
#include "kda_tree.h"

namespace kda {

int tree_check(const kda_pool* pool, int32_t n_req, int64_t n_tokens, kda_dtype state_dtype) {
  // (n_req may exceed the slots here: trees only read them)
  const int rc = check_common(pool, 0, 1, state_dtype);
  if (rc != KDA_OK) return rc;
  if (pool->H > kMaxTreeHeads) return KDA_ERR_SHAPE;
  if (n_req < 0 || n_tokens < 0 || n_tokens > INT32_MAX) return KDA_ERR_ARG;
  return KDA_OK;
}

int verify_check(int32_t n_req, int64_t n_tokens, int32_t vocab, int32_t max_path, kda_dtype dtype) {
  if (dtype != KDA_F32 && dtype != KDA_F16 && dtype != KDA_BF16) return KDA_ERR_DTYPE_REFUSED;
  if (n_req < 0 || n_tokens < 0 || n_tokens > INT32_MAX || vocab < 1) return KDA_ERR_ARG;
  if (max_path < 1 || max_path > kMaxNodes) return KDA_ERR_ROWS;
  return KDA_OK;
}

VerifyPlan verify_plan(int32_t vocab) {
  // At most 64 runs, a lane each where they are searched; of whole loads of a wave.  (One
  // chain over 32768: 7.0 us, 7.9 with runs of 2048, 11.4 of 8192.)
  const int64_t each = (static_cast<int64_t>(vocab) + 63) / 64, run = (each + 511) / 512 * 512;
  return {static_cast<int32_t>((vocab + run - 1) / run), static_cast<int32_t>(run)};
}

}  // namespace kda

using namespace kda;

extern "C" {

int kda_tree_validate(const int32_t* cu_seqlens_host, const int32_t* parents_host, int32_t n_req,
                      int64_t n_tokens) {
  if (n_req < 0 || n_tokens < 0 || n_tokens > INT32_MAX) return KDA_ERR_ARG;
  if (n_req == 0) return KDA_OK;
  if (cu_seqlens_host == nullptr || (n_tokens > 0 && parents_host == nullptr)) return KDA_ERR_NULL;
  if (cu_seqlens_host[0] < 0) return KDA_ERR_ARG;
  for (int32_t r = 0; r < n_req; ++r) {
    const int32_t n0 = cu_seqlens_host[r], n1 = cu_seqlens_host[r + 1];
    if (n1 < n0 || n1 > n_tokens) return KDA_ERR_ARG;
    if (n1 - n0 > kMaxNodes) return KDA_ERR_ROWS;
    for (int32_t i = 0; i < n1 - n0; ++i)
      if (parents_host[n0 + i] < -1 || parents_host[n0 + i] >= i) return KDA_ERR_ARG;
  }
  return KDA_OK;
}

size_t kda_verify_workspace(int32_t n_req, int64_t n_tokens, int32_t vocab, int32_t max_path, kda_dtype dtype) {
  if (verify_check(n_req, n_tokens, vocab, max_path, dtype) != KDA_OK || n_req == 0) return 0;
  const VerifyPlan p = verify_plan(vocab);
  return static_cast<size_t>(n_req) * (sizeof(VerifyStop) + p.runs * sizeof(double));
}

}  // extern "C"
