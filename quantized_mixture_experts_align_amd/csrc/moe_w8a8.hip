// moe_w8a8_gemm / moe_w8a8_linear: products of e4m3fn operands with one fp32 scale for each row and
// 128 columns of the activations and for each 128 x 128 block of the weights, grouped over the
// align's blocks or dense (moe_block_gemm.h holds the kernels).
#include "moe_block_gemm.h"

using namespace moe;

static int w8a8(const char* fn, bool dense, const uint8_t* A, int64_t a_rows, int64_t lda, const float* a_scales,
                int64_t ld_as, const uint8_t* W, const float* w_scales, const uint16_t* bias, int32_t E, int32_t N,
                int32_t K, uint16_t* C, int64_t ldc, const int32_t* sorted, const int32_t* eids, const int32_t* ntpp,
                int64_t numel, int32_t top_k, int32_t block_m, int64_t expected, hipStream_t stream) {
  int rc = check_block_gemm<Fp8Type>(fn, A, a_rows, lda, W, E, N, K, bias, C, ldc, numel, top_k, block_m);
  if (rc) return rc;
  const int32_t G = (K + kScaleBlock - 1) / kScaleBlock;
  MOE_REQUIRE(ld_as >= G, MOE_EINVAL, "%s: ld_scales=%lld below the %d groups of K=%d", fn, (long long)ld_as, G, K);
  if (numel == 0) return ok();
  MOE_REQUIRE(a_scales && w_scales && (dense || (sorted && eids && ntpp)), MOE_EINVAL, "%s: null pointer", fn);
  MOE_REQUIRE((((uintptr_t)a_scales | (uintptr_t)w_scales) & 3) == 0, MOE_EUNSUPPORTED, "%s: misaligned scales", fn);
  int64_t cap = 0, cap_blocks = (numel + block_m - 1) / block_m;
  if (!dense) {
    rc = moe_align_capacity(numel, 1, E, block_m, &cap, &cap_blocks);
    if (rc) return rc;
  }
  const BlockGemmArgs a{A, lda, W, a_scales, ld_as, w_scales, bias, C, ldc, dense ? nullptr : sorted, eids, ntpp,
                        (int32_t)numel, top_k, block_m, N, K, E, 0, 0, 0, 0, nullptr,
                        expected > 0 ? std::min(expected, numel) : numel};
  return launch_block_gemm<Fp8Type>(fn, a, cap_blocks, stream);
}

extern "C" int moe_w8a8_gemm(const uint8_t* A, int64_t a_rows, int64_t lda, const float* a_scales, int64_t ld_scales,
                             const uint8_t* W, const float* w_scales, const uint16_t* bias, int32_t E, int32_t N,
                             int32_t K, uint16_t* C, int64_t ldc, const int32_t* sorted_token_ids,
                             const int32_t* expert_ids, const int32_t* num_tokens_post_padded, int64_t numel,
                             int32_t top_k, int32_t block_m, int64_t expected_slots, hipStream_t stream) {
  return w8a8("moe_w8a8_gemm", false, A, a_rows, lda, a_scales, ld_scales, W, w_scales, bias, E, N, K, C, ldc,
              sorted_token_ids, expert_ids, num_tokens_post_padded, numel, top_k, block_m, expected_slots, stream);
}

extern "C" int moe_w8a8_linear(const uint8_t* A, int64_t M, int64_t lda, const float* a_scales, int64_t ld_scales,
                               const uint8_t* W, const float* w_scales, const uint16_t* bias, int32_t N, int32_t K,
                               uint16_t* C, int64_t ldc, hipStream_t stream) {
  return w8a8("moe_w8a8_linear", true, A, M, lda, a_scales, ld_scales, W, w_scales, bias, 1, N, K, C, ldc, nullptr,
              nullptr, nullptr, M, 1, M <= 16 ? 16 : (M <= 32 ? 32 : (M <= 64 ? 64 : 256)), M, stream);
}
