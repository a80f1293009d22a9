// moe_bf16_gemm: products of bf16 activations with unquantised bf16 expert weights over the
// align's blocks (moe_block_gemm.h holds the kernels).
#include "moe_block_gemm.h"

using namespace moe;

extern "C" int moe_bf16_gemm(const uint16_t* A, int64_t a_rows, int64_t lda, const uint16_t* W, const uint16_t* bias,
                             int32_t E, int32_t N, int32_t K, uint16_t* C, int64_t ldc,
                             const int32_t* sorted_token_ids, const int32_t* expert_ids,
                             const int32_t* num_tokens_post_padded, const int32_t* slot_local_ids, int64_t numel,
                             int32_t top_k, int32_t block_m, int64_t expected_slots, hipStream_t stream) {
  const char* fn = "moe_bf16_gemm";
  int rc = check_block_gemm<Bf16Type>(fn, A, a_rows, lda, W, E, N, K, bias, C, ldc, numel, top_k, block_m);
  if (rc) return rc;
  if (numel == 0) return ok();
  MOE_REQUIRE(sorted_token_ids && expert_ids && num_tokens_post_padded, MOE_EINVAL, "%s: null pointer", fn);
  int64_t cap = 0, cap_blocks = 0;
  rc = moe_align_capacity(numel, 1, E, block_m, &cap, &cap_blocks);
  if (rc) return rc;
  const BlockGemmArgs a{reinterpret_cast<const uint8_t*>(A), lda * 2, reinterpret_cast<const uint8_t*>(W), nullptr, 0,
                        nullptr, bias, C, ldc, sorted_token_ids, expert_ids, num_tokens_post_padded, (int32_t)numel,
                        top_k, block_m, N, K * 2, E, 0, 0, 0, 0, slot_local_ids,
                        expected_slots > 0 ? std::min(expected_slots, numel) : numel};
  return launch_block_gemm<Bf16Type>(fn, a, cap_blocks, stream);
}
