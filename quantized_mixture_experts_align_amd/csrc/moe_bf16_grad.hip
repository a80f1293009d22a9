// Gradients of moe_bf16_gemm, C[s, n] = sum_k A[s / top_k, k] W[e(s), n, k] + bias[e(s), n]:
//   moe_bf16_gemm_dgrad   dA[r, k] = sum over the live slots s of row r, sum_n dC[s, n] W[e(s), n, k]
//   moe_bf16_gemm_wgrad   dW[e, n, k] = sum over the slots s of e of dC[s, n] A[s / top_k, k]
//                         dbias[e, n] = sum over the slots s of e of dC[s, n]
// Both products reduce over an index whose values are rows in memory (n of W; the slots of dC and
// A), while an MFMA operand wants eight consecutive values of it in one lane.  The tiles are staged
// in LDS as they lie in memory and read with ds_read_b64_tr_b16: within 16 lanes that together read
// four rows of 16 values, lane i receives column i.
//
// Sums run in fp32 in a fixed order (no atomics).
#include <algorithm>

#include "moe_block_gemm.h"

namespace moe {

struct GradArgs {
  const uint16_t* dC;
  int64_t ld_dc;
  const uint16_t* A;   // wgrad
  int64_t lda;
  const uint16_t* W;   // dgrad: [E, N, K]
  void* dX;            // dgrad: a row for each slot (bf16, or fp32 to be summed over a row's slots)
  int64_t ld_dx;
  void* dW;            // wgrad: [E, N, K]
  void* dbias;         // wgrad: [E, N] or null
  const int32_t* sorted;
  const int32_t* eids;
  const int32_t* ntpp;
  int32_t numel, top_k, block_m, N, K, E;
};

typedef __attribute__((ext_vector_type(4))) int16_t s16x4_t;

// Lane i of each 16-lane group reads 8 bytes at its own address; it receives the i-th value of each
// of the four rows that lanes 0-3, 4-7, 8-11 and 12-15 hold.
__device__ __forceinline__ u32x2_t lds_read_tr(const uint8_t* p) {
  const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p);
  return __builtin_bit_cast(u32x2_t, v);
}

// The transposed operand of 16 columns at byte column `col` of a staged tile [32][pitch bytes]:
// lane l gets column l % 16, rows 8 (l / 16) + 0..7.
__device__ __forceinline__ u32x4_t tr_frag(const uint8_t* tile, int pitch, int col, int lane) {
  const uint8_t* p = tile + (8 * (lane >> 4) + ((lane & 15) >> 2)) * pitch + col + (lane & 3) * 8;
  const u32x2_t lo = lds_read_tr(p), hi = lds_read_tr(p + 4 * pitch);
  return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
}

// dX[s, k] of 64 slots of a block x 64 columns k: wave w holds columns 16 w .. 16 w + 15.
template <typename OUT>
__global__ __launch_bounds__(256) void dgrad_kernel(GradArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t ws[32 * 128];     // 32 rows n x 64 columns k
  __shared__ __attribute__((aligned(16))) uint8_t cs[64 * 64];      // 64 slots x 32 columns n
  __shared__ int s_slot[64];
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const int strips = (a.K + 63) / 64, subs = (a.block_m + 63) / 64;
  const int strip = blockIdx.x % strips, rest = blockIdx.x / strips;
  const int b = rest / subs, sub = rest - b * subs;
  if ((int64_t)b * a.block_m >= *a.ntpp) return;
  const int e = a.eids[b];
  if (e < 0 || e >= a.E) return;
  if (tid < 64) {
    const int p = sub * 64 + tid;
    const int s = p < a.block_m ? a.sorted[(int64_t)b * a.block_m + p] : -1;
    s_slot[tid] = s >= 0 && s < a.numel ? s : -1;
  }
  __syncthreads();
  f32x4_t acc[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) acc[h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int n0 = 0; n0 < a.N; n0 += 32) {
    {
      const int r = tid >> 3, k = strip * 64 + (tid & 7) * 8;   // 32 rows x 8 chunks of 8 columns
      u32x4_t v = {0u, 0u, 0u, 0u};
      if (n0 + r < a.N && k < a.K) v = *reinterpret_cast<const u32x4_t*>(a.W + ((int64_t)e * a.N + n0 + r) * a.K + k);
      *reinterpret_cast<u32x4_t*>(ws + r * 128 + (tid & 7) * 16) = v;
      const int q = tid >> 2, n = n0 + (tid & 3) * 8, s = s_slot[q];  // 64 slots x 4 chunks
      u32x4_t c = {0u, 0u, 0u, 0u};
      if (s >= 0 && n < a.N) c = *reinterpret_cast<const u32x4_t*>(a.dC + (int64_t)s * a.ld_dc + n);
      *reinterpret_cast<u32x4_t*>(cs + q * 64 + (tid & 3) * 16) = c;
    }
    __syncthreads();
    const u32x4_t wf = tr_frag(ws, 128, w * 32, lane);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const u32x4_t cf = *reinterpret_cast<const u32x4_t*>(cs + (h * 16 + (lane & 15)) * 64 + (lane >> 4) * 16);
      acc[h] = mfma(wf, cf, acc[h]);
    }
    __syncthreads();
  }
  const int k0 = strip * 64 + w * 16 + 4 * (lane >> 4);
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int s = s_slot[h * 16 + (lane & 15)];
    if (s < 0 || k0 >= a.K) continue;
    OUT* o = static_cast<OUT*>(a.dX) + (int64_t)s * a.ld_dx + k0;
    if constexpr (sizeof(OUT) == 4) *reinterpret_cast<f32x4_t*>(o) = acc[h];
    else *reinterpret_cast<u32x2_t*>(o) = u32x2_t{pack_bf16x2(acc[h][0], acc[h][1]), pack_bf16x2(acc[h][2], acc[h][3])};
  }
}

// [first, last) of the sorted entries of expert e: the align lists the experts' blocks in rising
// order, so counting the live blocks of lower and of equal experts gives its range.  Every thread
// of the workgroup calls it; `red` holds two ints for each wave.
__device__ __forceinline__ void expert_range(const int32_t* eids, const int32_t* ntpp, int block_m, int e, int* red,
                                             int64_t* first, int64_t* last) {
  const int nb = *ntpp / block_m, lane = threadIdx.x & 63;
  int lower = 0, equal = 0;
  for (int i = threadIdx.x; i < nb; i += blockDim.x) {
    const int v = eids[i];
    lower += v < e;
    equal += v == e;
  }
  for (int d = 32; d >= 1; d >>= 1) {
    lower += __shfl_xor(lower, d);
    equal += __shfl_xor(equal, d);
  }
  if (lane == 0) {
    red[2 * (threadIdx.x >> 6)] = lower;
    red[2 * (threadIdx.x >> 6) + 1] = equal;
  }
  __syncthreads();
  lower = equal = 0;
  for (int i = 0; i < (int)(blockDim.x >> 6); ++i) {
    lower += red[2 * i];
    equal += red[2 * i + 1];
  }
  *first = (int64_t)lower * block_m;
  *last = *first + (int64_t)equal * block_m;
}

// dW[e, n, k] of 64 rows n x 64 columns k: wave w holds columns 16 w .. 16 w + 15.
template <typename OUT>
__global__ __launch_bounds__(256) void wgrad_kernel(GradArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t xs[32 * 128];  // 32 slots x 64 columns k of A
  __shared__ __attribute__((aligned(16))) uint8_t cs[32 * 128];  // 32 slots x 64 columns n of dC
  __shared__ int red[8];
  const int tid = threadIdx.x, w = tid >> 6, lane = tid & 63;
  const int ks = (a.K + 63) / 64, ns = (a.N + 63) / 64;
  const int kt = blockIdx.x % ks, rest = blockIdx.x / ks, nt = rest % ns, e = rest / ns;
  int64_t first, last;
  expert_range(a.eids, a.ntpp, a.block_m, e, red, &first, &last);
  f32x4_t acc[4];
#pragma unroll
  for (int h = 0; h < 4; ++h) acc[h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int r = tid >> 3, c8 = (tid & 7) * 8;
  for (int64_t p = first; p < last; p += 32) {
    const int s = p + r < last ? a.sorted[p + r] : -1;
    const bool live = s >= 0 && s < a.numel;
    u32x4_t x = {0u, 0u, 0u, 0u}, c = x;
    if (live && kt * 64 + c8 < a.K)
      x = *reinterpret_cast<const u32x4_t*>(a.A + (int64_t)(s / a.top_k) * a.lda + kt * 64 + c8);
    if (live && nt * 64 + c8 < a.N)
      c = *reinterpret_cast<const u32x4_t*>(a.dC + (int64_t)s * a.ld_dc + nt * 64 + c8);
    *reinterpret_cast<u32x4_t*>(xs + r * 128 + c8 * 2) = x;
    *reinterpret_cast<u32x4_t*>(cs + r * 128 + c8 * 2) = c;
    __syncthreads();
    const u32x4_t xf = tr_frag(xs, 128, w * 32, lane);
#pragma unroll
    for (int h = 0; h < 4; ++h) acc[h] = mfma(xf, tr_frag(cs, 128, h * 32, lane), acc[h]);
    __syncthreads();
  }
  const int k0 = kt * 64 + w * 16 + 4 * (lane >> 4);
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const int n = nt * 64 + h * 16 + (lane & 15);
    if (n >= a.N || k0 >= a.K) continue;
    OUT* o = static_cast<OUT*>(a.dW) + ((int64_t)e * a.N + n) * a.K + k0;
    if constexpr (sizeof(OUT) == 4) *reinterpret_cast<f32x4_t*>(o) = acc[h];
    else *reinterpret_cast<u32x2_t*>(o) = u32x2_t{pack_bf16x2(acc[h][0], acc[h][1]), pack_bf16x2(acc[h][2], acc[h][3])};
  }
}

// dbias[e, n] of 128 columns: 16 chunks of eight columns x 16 rows at a time, joined in row order.
template <typename OUT>
__global__ __launch_bounds__(256) void bias_grad_kernel(GradArgs a) {
  __shared__ int red[8];
  __shared__ float part[16][128];
  const int tid = threadIdx.x, r = tid >> 4, c8 = (tid & 15) * 8;
  const int ns = (a.N + 127) / 128, nt = blockIdx.x % ns, e = blockIdx.x / ns;
  int64_t first, last;
  expert_range(a.eids, a.ntpp, a.block_m, e, red, &first, &last);
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.f;
  const int n = nt * 128 + c8;
  for (int64_t p = first + r; p < last; p += 16) {
    const int s = a.sorted[p];
    if (s < 0 || s >= a.numel || n >= a.N) continue;
    const u32x4_t c = *reinterpret_cast<const u32x4_t*>(a.dC + (int64_t)s * a.ld_dc + n);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] += bf16_lo(c[j]);
      v[2 * j + 1] += bf16_hi(c[j]);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) part[r][c8 + j] = v[j];
  __syncthreads();
  if (tid < 128 && nt * 128 + tid < a.N) {
    float t = 0.f;
    for (int i = 0; i < 16; ++i) t += part[i][tid];
    const int64_t at = (int64_t)e * a.N + nt * 128 + tid;
    if constexpr (sizeof(OUT) == 4) static_cast<float*>(a.dbias)[at] = t;
    else static_cast<uint16_t*>(a.dbias)[at] = f32_to_bf16(t);
  }
}

// dst[r, :] = sum over the live slots of row r, in slot order (fp32, one rounding), of src[slot, :]
__global__ __launch_bounds__(256) void sum_slots_kernel(const float* __restrict__ src, const int32_t* __restrict__ live,
                                                        int32_t top_k, int32_t K, uint16_t* __restrict__ dst,
                                                        int64_t ld_dst) {
  const int64_t r = blockIdx.x;
  for (int c = threadIdx.x * 4; c < K; c += 256 * 4) {
    f32x4_t v = {0.f, 0.f, 0.f, 0.f};
    for (int i = 0; i < top_k; ++i) {
      const int64_t s = r * top_k + i;
      if (live[s] >= 0) v += *reinterpret_cast<const f32x4_t*>(src + s * K + c);
    }
    *reinterpret_cast<u32x2_t*>(dst + r * ld_dst + c) = u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
}

// zeros in the rows of dropped slots (the others are not touched)
__global__ __launch_bounds__(256) void zero_dead_kernel(const int32_t* __restrict__ live, int64_t rows, int32_t K,
                                                        uint16_t* __restrict__ dst, int64_t ld) {
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    if (live[r] >= 0) continue;
    for (int c = threadIdx.x * 8; c < K; c += 256 * 8)
      *reinterpret_cast<u32x4_t*>(dst + r * ld + c) = u32x4_t{0u, 0u, 0u, 0u};
  }
}

static int zero_dead(const char* fn, const int32_t* live, int64_t rows, int32_t K, uint16_t* dst, int64_t ld,
                     hipStream_t st) {
  hipLaunchKernelGGL(zero_dead_kernel, dim3((unsigned)std::min<int64_t>(rows, 4096)), dim3(256), 0, st, live, rows, K,
                     dst, ld);
  return check_launch(fn);
}

static int check_grad(const char* fn, const void* dC, int64_t ld_dc, int32_t E, int32_t N, int32_t K, int64_t numel,
                      int32_t top_k, int32_t block_m) {
  MOE_REQUIRE(E >= 1 && N >= 1 && K >= 1, MOE_EINVAL, "%s: E=%d N=%d K=%d", fn, E, N, K);
  MOE_REQUIRE(E <= 512, MOE_EUNSUPPORTED, "%s: %d experts (at most 512)", fn, E);
  MOE_REQUIRE(N % 8 == 0 && K % 8 == 0 && N <= (1 << 20) && K <= (1 << 20), MOE_EUNSUPPORTED,
              "%s: N=%d and K=%d must be multiples of 8 (at most 2^20)", fn, N, K);
  MOE_REQUIRE(numel >= 0 && top_k >= 1 && block_m >= 1 && block_m <= 256, MOE_EINVAL,
              "%s: numel=%lld top_k=%d block_m=%d (1..256)", fn, (long long)numel, top_k, block_m);
  MOE_REQUIRE(numel < (1 << 30), MOE_EUNSUPPORTED, "%s: numel=%lld", fn, (long long)numel);
  MOE_REQUIRE(numel % top_k == 0, MOE_EINVAL, "%s: %lld slots are no whole rows of %d", fn, (long long)numel, top_k);
  MOE_REQUIRE(ld_dc >= N && ld_dc % 8 == 0, MOE_EINVAL, "%s: ld_dc=%lld (>= N=%d, multiple of 8)", fn,
              (long long)ld_dc, N);
  MOE_REQUIRE(numel == 0 || dC, MOE_EINVAL, "%s: null pointer", fn);
  MOE_REQUIRE(((uintptr_t)dC & 15) == 0, MOE_EUNSUPPORTED, "%s: misaligned pointer (16 B)", fn);
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_zero_dropped_rows(const int32_t* slot_local_ids, int64_t rows, int32_t N, uint16_t* C, int64_t ldc,
                                     hipStream_t stream) {
  const char* fn = "moe_zero_dropped_rows";
  MOE_REQUIRE(rows >= 0 && N >= 1, MOE_EINVAL, "%s: rows=%lld N=%d", fn, (long long)rows, N);
  MOE_REQUIRE(N % 8 == 0 && ldc >= N && ldc % 8 == 0, MOE_EUNSUPPORTED,
              "%s: N=%d and ldc=%lld must be multiples of 8, ldc >= N", fn, N, (long long)ldc);
  if (rows == 0) return ok();
  MOE_REQUIRE(slot_local_ids && C, MOE_EINVAL, "%s: null pointer", fn);
  MOE_REQUIRE(((uintptr_t)C & 15) == 0, MOE_EUNSUPPORTED, "%s: misaligned pointer (16 B)", fn);
  return zero_dead(fn, slot_local_ids, rows, N, C, ldc, stream);
}

extern "C" int moe_bf16_gemm_dgrad(const uint16_t* dC, int64_t ld_dc, const uint16_t* W, int32_t E, int32_t N,
                                   int32_t K, uint16_t* dA, int64_t ld_da, const int32_t* sorted_token_ids,
                                   const int32_t* expert_ids, const int32_t* num_tokens_post_padded,
                                   const int32_t* slot_local_ids, int64_t numel, int32_t top_k, int32_t block_m,
                                   float* work, int64_t work_elems, hipStream_t stream) {
  const char* fn = "moe_bf16_gemm_dgrad";
  int rc = check_grad(fn, dC, ld_dc, E, N, K, numel, top_k, block_m);
  if (rc) return rc;
  MOE_REQUIRE(ld_da >= K && ld_da % 8 == 0, MOE_EINVAL, "%s: ld_da=%lld (>= K=%d, multiple of 8)", fn,
              (long long)ld_da, K);
  MOE_REQUIRE(top_k == 1 || work_elems >= numel * K, MOE_ESIZE, "%s: workspace of %lld values, need %lld", fn,
              (long long)work_elems, (long long)(numel * K));
  if (numel == 0) return ok();
  MOE_REQUIRE(W && dA && sorted_token_ids && expert_ids && num_tokens_post_padded && slot_local_ids &&
                  (top_k == 1 || work),
              MOE_EINVAL, "%s: null pointer", fn);
  MOE_REQUIRE((((uintptr_t)W | (uintptr_t)dA | (uintptr_t)work) & 15) == 0, MOE_EUNSUPPORTED,
              "%s: misaligned pointer (16 B)", fn);
  int64_t cap = 0, cap_blocks = 0;
  rc = moe_align_capacity(numel, 1, E, block_m, &cap, &cap_blocks);
  if (rc) return rc;
  const GradArgs a{dC, ld_dc, nullptr, 0, W, top_k == 1 ? static_cast<void*>(dA) : work, top_k == 1 ? ld_da : (int64_t)K, nullptr, nullptr,
                   sorted_token_ids, expert_ids, num_tokens_post_padded, (int32_t)numel, top_k, block_m, N, K, E};
  const int64_t grid = (int64_t)((K + 63) / 64) * cap_blocks * ((block_m + 63) / 64);
  MOE_REQUIRE(grid < (1ll << 31), MOE_EUNSUPPORTED, "%s: grid too large", fn);
  if (top_k == 1) hipLaunchKernelGGL(dgrad_kernel<uint16_t>, dim3((unsigned)grid), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(dgrad_kernel<float>, dim3((unsigned)grid), dim3(256), 0, stream, a);
  rc = check_launch(fn);
  if (rc) return rc;
  if (top_k == 1) return zero_dead(fn, slot_local_ids, numel, K, dA, ld_da, stream);
  hipLaunchKernelGGL(sum_slots_kernel, dim3((unsigned)(numel / top_k)), dim3(256), 0, stream, work,
                     slot_local_ids, top_k, K, dA, ld_da);
  return check_launch(fn);
}

extern "C" int moe_bf16_gemm_wgrad(const uint16_t* dC, int64_t ld_dc, const uint16_t* A, int64_t a_rows, int64_t lda,
                                   int32_t E, int32_t N, int32_t K, void* dW, void* dbias, int32_t out_f32,
                                   const int32_t* sorted_token_ids, const int32_t* expert_ids,
                                   const int32_t* num_tokens_post_padded, int64_t numel, int32_t top_k,
                                   int32_t block_m, hipStream_t stream) {
  const char* fn = "moe_bf16_gemm_wgrad";
  int rc = check_grad(fn, dC, ld_dc, E, N, K, numel, top_k, block_m);
  if (rc) return rc;
  MOE_REQUIRE(a_rows >= numel / top_k, MOE_EINVAL, "%s: A has %lld rows, slots need %lld", fn, (long long)a_rows,
              (long long)(numel / top_k));
  MOE_REQUIRE(lda >= K && lda % 8 == 0, MOE_EINVAL, "%s: lda=%lld (>= K=%d, multiple of 8)", fn, (long long)lda, K);
  MOE_REQUIRE(dW && num_tokens_post_padded && (numel == 0 || (A && sorted_token_ids && expert_ids)), MOE_EINVAL,
              "%s: null pointer", fn);
  MOE_REQUIRE((((uintptr_t)A | (uintptr_t)dW) & 15) == 0 && ((uintptr_t)dbias & 3) == 0, MOE_EUNSUPPORTED,
              "%s: misaligned pointer (A and dW 16 B, dbias 4 B)", fn);
  const GradArgs a{dC, ld_dc, A, lda, nullptr, nullptr, 0, dW, dbias, sorted_token_ids, expert_ids,
                   num_tokens_post_padded, (int32_t)numel, top_k, block_m, N, K, E};
  const int64_t grid = (int64_t)((K + 63) / 64) * ((N + 63) / 64) * E;
  MOE_REQUIRE(grid < (1ll << 31), MOE_EUNSUPPORTED, "%s: grid too large", fn);
  if (out_f32) hipLaunchKernelGGL(wgrad_kernel<float>, dim3((unsigned)grid), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(wgrad_kernel<uint16_t>, dim3((unsigned)grid), dim3(256), 0, stream, a);
  rc = check_launch(fn);
  if (rc || !dbias) return rc;
  const unsigned gb = (unsigned)((int64_t)((N + 127) / 128) * E);
  if (out_f32) hipLaunchKernelGGL(bias_grad_kernel<float>, dim3(gb), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL(bias_grad_kernel<uint16_t>, dim3(gb), dim3(256), 0, stream, a);
  return check_launch(fn);
}
