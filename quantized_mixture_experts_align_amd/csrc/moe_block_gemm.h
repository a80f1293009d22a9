// Grouped products with row-major weights of 8 or 16 bits a value (not part of the ABI):
//     C[s, n] = bf16( sum_k A[row(s), k] * W[e, n, k]  (+ bias[e, n]) )
// over the align's blocks (s a slot, row(s) = s / top_k), or over consecutive blocks of rows of one
// dense product.  Bf16 operands multiply directly; e4m3fn operands carry one fp32 scale for each
// row and 128 columns of A and one for each 128 x 128 block of W, applied to the fp32 partial sum
// of every 128 columns: acc += (sa * sb) * sum_128.
//
// Both types are handled in steps of 128 bytes of K per row, and a wave's MFMA operand of a step
// is 16 rows x 128 bytes: lane l holds row l % 16, bytes 16 (l / 16) + 0..15 and the same 64
// further on.  For bf16 these are the operands of two v_mfma_f32_16x16x32_bf16, for e4m3fn the
// two halves of one v_mfma_f32_16x16x128_f8f6f4 (which k a lane's bytes stand for does not matter
// as long as both operands agree).  Weights are the A operand (rows = output features),
// activations the B operand (columns = slots), so a lane ends with four consecutive output
// features of one slot.
#pragma once

#include "moe_gemm_mfma.h"

namespace moe {

constexpr int kStepBytes = 128;  // of K, per row and step
constexpr int kScaleBlock = 128;

struct BlockGemmArgs {
  const uint8_t* A;
  int64_t lda;            // bytes between rows of A
  const uint8_t* W;       // [E, N, Kb] bytes
  const float* sa;        // e4m3fn: [rows, ld_sa], one for each 128 columns
  int64_t ld_sa;
  const float* sb;        // e4m3fn: [E, ceil(N / 128), ceil(K / 128)]
  const uint16_t* bias;   // bf16 [E, N] or null
  uint16_t* C;
  int64_t ldc;
  const int32_t* sorted;  // null: dense, block b holds rows b * block_m ..., expert 0
  const int32_t* eids;
  const int32_t* ntpp;
  int32_t numel, top_k, block_m, N, Kb, E;
  int32_t group_m;        // tile kernel: align blocks per XCD workgroup group
};

struct Fp8Type {
  static constexpr bool kScaled = true;
  static constexpr int kBytes = 1;
};
struct Bf16Type {
  static constexpr bool kScaled = false;
  static constexpr int kBytes = 2;
};

typedef __attribute__((ext_vector_type(8))) int32_t i32x8_t;

// One step's operand of a wave: 16 rows x 128 bytes.
struct Frag {
  u32x4_t lo, hi;
};

// What lies past K reads as zero (in both operands, so that no NaN pattern behind a row's end
// meets a zero).
static __device__ const u32x4_t g_zero16 = {0u, 0u, 0u, 0u};

// acc + the step's product (bf16), or the step's product alone (e4m3fn, scaled by the caller)
__device__ __forceinline__ f32x4_t mfma_step(Bf16Type, const Frag& w, const Frag& x, f32x4_t acc) {
  acc = mfma(w.lo, x.lo, acc);
  return mfma(w.hi, x.hi, acc);
}
__device__ __forceinline__ f32x4_t mfma_step(Fp8Type, const Frag& w, const Frag& x) {
  const i32x8_t a = __builtin_shufflevector(__builtin_bit_cast(__attribute__((ext_vector_type(4))) int32_t, w.lo),
                                            __builtin_bit_cast(__attribute__((ext_vector_type(4))) int32_t, w.hi), 0, 1,
                                            2, 3, 4, 5, 6, 7);
  const i32x8_t b = __builtin_shufflevector(__builtin_bit_cast(__attribute__((ext_vector_type(4))) int32_t, x.lo),
                                            __builtin_bit_cast(__attribute__((ext_vector_type(4))) int32_t, x.hi), 0, 1,
                                            2, 3, 4, 5, 6, 7);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// The slot at position p of block b, or -1 for padding.
__device__ __forceinline__ int slot_of(const BlockGemmArgs& a, int b, int p) {
  if (p >= a.block_m) return -1;
  const int64_t at = (int64_t)b * a.block_m + p;
  const int64_t s = a.sorted ? a.sorted[at] : at;
  return s >= 0 && s < a.numel ? (int)s : -1;
}

// ---------------------------------------------------------------------------- few rows
// Workgroup = 16 slots of a block x NG 16-row weight tiles, K split over its KS waves, operands
// straight from memory to registers in chunks of kChunk steps, partial sums joined through LDS in
// wave order.  For blocks of at most 16 slots the cost is the stream of weights, of which each
// wave has NG * 2 * kChunk 16-byte loads a lane in flight.
template <typename T, int NG, int KS>
__global__ __launch_bounds__(64 * KS) void block_gemm_stream_kernel(BlockGemmArgs a) {
  constexpr int kChunk = 4;
  __shared__ f32x4_t part[KS][NG][64];
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int strips = (a.N + 16 * NG - 1) / (16 * NG), subs = (a.block_m + 15) / 16;
  const int strip = blockIdx.x % strips, rest = blockIdx.x / strips;
  const int b = rest / subs, sub = rest - b * subs;
  int e = 0;
  if (a.sorted) {
    if ((int64_t)b * a.block_m >= *a.ntpp) return;
    e = a.eids[b];
    if (e < 0 || e >= a.E) return;
  }
  const int slot = slot_of(a, b, sub * 16 + (lane & 15));
  if (__ballot(slot >= 0) == 0) return;  // (the same in every wave)

  const int KT = (a.Kb + kStepBytes - 1) / kStepBytes;
  const int kt0 = KT * w / KS, kt1 = KT * (w + 1) / KS;
  const int koff = 16 * (lane >> 4);
  const int64_t row = slot >= 0 ? slot / a.top_k : 0;
  const uint8_t* xp = a.A + row * a.lda + koff;
  const uint8_t* wp[NG];
  const float* sbp[NG];
  const float* sap = nullptr;
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int n = min((strip * NG + g) * 16 + (lane & 15), a.N - 1);
    wp[g] = a.W + ((int64_t)e * a.N + n) * a.Kb + koff;
    if constexpr (T::kScaled)
      sbp[g] = a.sb + ((int64_t)e * ((a.N + kScaleBlock - 1) / kScaleBlock) + n / kScaleBlock) * KT;
  }
  if constexpr (T::kScaled) sap = a.sa + row * a.ld_sa;
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(&g_zero16);

  f32x4_t acc[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int c = kt0; c < kt1; c += kChunk) {
    Frag x[kChunk], wt[kChunk][NG];
    float sa[kChunk], sb[kChunk][NG];
#pragma unroll
    for (int u = 0; u < kChunk; ++u) {
      const int kt = min(c + u, kt1 - 1);  // (past the wave's last step: loaded again, not used)
      const int64_t k0 = (int64_t)kt * kStepBytes;
      const bool lo = k0 + koff < a.Kb && slot >= 0, hi = k0 + koff + 64 < a.Kb && slot >= 0;
      const bool wlo = k0 + koff < a.Kb, whi = k0 + koff + 64 < a.Kb;
      x[u].lo = *reinterpret_cast<const u32x4_t*>(lo ? xp + k0 : zero);
      x[u].hi = *reinterpret_cast<const u32x4_t*>(hi ? xp + k0 + 64 : zero);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        wt[u][g].lo = *reinterpret_cast<const u32x4_t*>(wlo ? wp[g] + k0 : zero);
        wt[u][g].hi = *reinterpret_cast<const u32x4_t*>(whi ? wp[g] + k0 + 64 : zero);
        if constexpr (T::kScaled) sb[u][g] = sbp[g][kt];
      }
      if constexpr (T::kScaled) sa[u] = sap[kt];
    }
#pragma unroll
    for (int u = 0; u < kChunk; ++u) {
      if (c + u >= kt1) break;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if constexpr (T::kScaled) {
          const f32x4_t t = mfma_step(T{}, wt[u][g], x[u]);
          // (the scale of the weight block belongs to the tile's rows: lane l's row of the operand
          // and the rows of its result lie in one 16-row tile, hence in one block)
          const float s = sa[u] * sb[u][g];
#pragma unroll
          for (int q = 0; q < 4; ++q) acc[g][q] = fmaf(t[q], s, acc[g][q]);
        } else {
          acc[g] = mfma_step(T{}, wt[u][g], x[u], acc[g]);
        }
      }
    }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g) part[w][g][lane] = acc[g];
  __syncthreads();
  for (int g = w; g < NG; g += KS) {
    f32x4_t v = part[0][g][lane];
#pragma unroll
    for (int i = 1; i < KS; ++i) v += part[i][g][lane];
    const int n0 = (strip * NG + g) * 16 + 4 * (lane >> 4);
    if (n0 < a.N && slot >= 0) {  // (N is a multiple of 8: four columns are in or out together)
      if (a.bias) {
        const u32x2_t bb = *reinterpret_cast<const u32x2_t*>(a.bias + (int64_t)e * a.N + n0);
        v[0] += bf16_lo(bb[0]); v[1] += bf16_hi(bb[0]); v[2] += bf16_lo(bb[1]); v[3] += bf16_hi(bb[1]);
      }
      *reinterpret_cast<u32x2_t*>(a.C + (int64_t)slot * a.ldc + n0) =
          u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
  }
}

template <typename T>
static int launch_block_gemm(const char* fn, const BlockGemmArgs& a, int64_t cap_blocks, hipStream_t st) {
  constexpr int NG = 2, KS = 4;
  const int64_t grid = (int64_t)((a.N + 16 * NG - 1) / (16 * NG)) * cap_blocks * ((a.block_m + 15) / 16);
  MOE_REQUIRE(grid < (1ll << 31), MOE_EUNSUPPORTED, "%s: grid too large", fn);
  hipLaunchKernelGGL((block_gemm_stream_kernel<T, NG, KS>), dim3((unsigned)grid), dim3(64 * KS), 0, st, a);
  return check_launch(fn);
}

// Checks shared by the products over the align's blocks (A and W of T::kBytes a value).
template <typename T>
static int check_block_gemm(const char* fn, const void* A, int64_t a_rows, int64_t lda, const void* W, int32_t E,
                            int32_t N, int32_t K, const uint16_t* bias, const void* C, int64_t ldc, int64_t numel,
                            int32_t top_k, int32_t block_m) {
  constexpr int kStep = 16 / T::kBytes;
  MOE_REQUIRE(E >= 1 && N >= 1 && K >= 1, MOE_EINVAL, "%s: E=%d N=%d K=%d", fn, E, N, K);
  MOE_REQUIRE(E <= 512, MOE_EUNSUPPORTED, "%s: %d experts (at most 512)", fn, E);
  MOE_REQUIRE(N % 8 == 0 && K % kStep == 0 && N <= (1 << 24) && K <= (1 << 24), MOE_EUNSUPPORTED,
              "%s: N=%d must be a multiple of 8 and K=%d of %d (both at most 2^24)", fn, N, K, kStep);
  MOE_REQUIRE(numel >= 0 && top_k >= 1 && block_m >= 1 && block_m <= 256, MOE_EINVAL,
              "%s: numel=%lld top_k=%d block_m=%d (1..256)", fn, (long long)numel, top_k, block_m);
  MOE_REQUIRE(numel < (1 << 30), MOE_EUNSUPPORTED, "%s: numel=%lld", fn, (long long)numel);
  MOE_REQUIRE(a_rows >= (numel + top_k - 1) / top_k, MOE_EINVAL, "%s: A has %lld rows, slots need %lld", fn,
              (long long)a_rows, (long long)((numel + top_k - 1) / top_k));
  MOE_REQUIRE(lda >= K && lda % kStep == 0 && ldc >= N && ldc % 4 == 0, MOE_EINVAL,
              "%s: lda=%lld (>= K=%d, multiple of %d) ldc=%lld (>= N=%d, multiple of 4)", fn, (long long)lda, K, kStep,
              (long long)ldc, N);
  if (numel == 0) return MOE_OK;
  MOE_REQUIRE(A && W && C, MOE_EINVAL, "%s: null pointer", fn);
  MOE_REQUIRE(((uintptr_t)A & 15) == 0 && ((uintptr_t)W & 15) == 0 && ((uintptr_t)C & 7) == 0 &&
                  ((uintptr_t)bias & 7) == 0,
              MOE_EUNSUPPORTED, "%s: misaligned pointer (A and W 16 B, C and bias 8 B)", fn);
  return MOE_OK;
}

}  // namespace moe
