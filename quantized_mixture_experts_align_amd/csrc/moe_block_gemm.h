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

typedef __attribute__((ext_vector_type(4))) int32_t i32x4_t;
typedef __attribute__((ext_vector_type(8))) int32_t i32x8_t;

// One step's operand of a wave, 16 rows x 128 bytes: two 16-byte loads a lane side by side in eight
// consecutive registers, as the e4m3fn instruction wants them.
typedef i32x8_t Frag;
__device__ __forceinline__ Frag frag_of(u32x4_t lo, u32x4_t hi) {
  return __builtin_shufflevector(__builtin_bit_cast(i32x4_t, lo), __builtin_bit_cast(i32x4_t, hi), 0, 1, 2, 3, 4, 5, 6,
                                 7);
}
__device__ __forceinline__ u32x4_t frag_lo(const Frag& f) {
  return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(f, f, 0, 1, 2, 3));
}
__device__ __forceinline__ u32x4_t frag_hi(const Frag& f) {
  return __builtin_bit_cast(u32x4_t, __builtin_shufflevector(f, f, 4, 5, 6, 7));
}
__device__ __forceinline__ Frag load_frag(const uint8_t* lo, const uint8_t* hi) {
  return frag_of(*reinterpret_cast<const u32x4_t*>(lo), *reinterpret_cast<const u32x4_t*>(hi));
}

// What lies past K reads as zero (in both operands, so that no NaN pattern behind a row's end
// meets a zero).
static __device__ const u32x4_t g_zero16 = {0u, 0u, 0u, 0u};

// acc + the step's product (bf16), or the step's product alone (e4m3fn, scaled by the caller)
__device__ __forceinline__ f32x4_t mfma_step(Bf16Type, const Frag& w, const Frag& x, f32x4_t acc) {
  acc = mfma(frag_lo(w), frag_lo(x), acc);
  return mfma(frag_hi(w), frag_hi(x), acc);
}
// (The instruction adds the products of eight consecutive k on the exponent of the largest, cut 13
// places below it, and these sums in fp32: the matrix core's own precision for 8-bit operands,
// measured 2^-19 rms and 2^-16 at most of the sum of the products' magnitudes.)
__device__ __forceinline__ f32x4_t mfma_step(Fp8Type, const Frag& w, const Frag& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
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
  const int strips = (a.N + 16 * NG - 1) / (16 * NG);
  const int strip = blockIdx.x % strips, b = blockIdx.x / strips;
  int e = 0;
  if (a.sorted) {
    if ((int64_t)b * a.block_m >= *a.ntpp) return;
    e = a.eids[b];
    if (e < 0 || e >= a.E) return;
  }
  const int slot = slot_of(a, b, lane & 15);
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
      x[u] = load_frag(lo ? xp + k0 : zero, hi ? xp + k0 + 64 : zero);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        wt[u][g] = load_frag(wlo ? wp[g] + k0 : zero, whi ? wp[g] + k0 + 64 : zero);
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

// ---------------------------------------------------------------------------- blocks of rows
// The outputs of a wave's NG 16-column tiles (columns n0 ..) for up to MG 16-row groups, of which the
// first lg are live.  acc[g][h] holds, in lane l, columns 4 (l / 16) + 0..3 of tile g of row l % 16
// of group h.  bf16 rows go through the wave's own part of LDS (idle: every wave has passed the last
// step's barrier), so that a store instruction covers whole segments of 32 * NG bytes of a row with
// 16 bytes a lane.  row_ptr(r) is where row r starts, or null.
template <int NG, int MG, typename OUT, typename RowPtr>
__device__ __forceinline__ void store_tiles(const f32x4_t (&acc)[NG][MG], int lg, uint8_t* smem, int smem_bytes, int w,
                                            int lane, int n0, int N, bool wide, RowPtr row_ptr) {
  if constexpr (sizeof(OUT) == 4) {
#pragma unroll
    for (int h = 0; h < MG; ++h) {
      if (h >= lg) break;
      OUT* row = row_ptr(h * 16 + (lane & 15));
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int n = n0 + g * 16 + 4 * (lane >> 4);
        if (row && n < N) *reinterpret_cast<f32x4_t*>(row + n) = acc[g][h];
      }
    }
  } else {
    auto pack = [&](int g, int h) {
      return u32x2_t{pack_bf16x2(acc[g][h][0], acc[g][h][1]), pack_bf16x2(acc[g][h][2], acc[g][h][3])};
    };
    if (!wide) {  // rows that are not 16-byte aligned
#pragma unroll
      for (int h = 0; h < MG; ++h) {
        if (h >= lg) break;
        OUT* row = row_ptr(h * 16 + (lane & 15));
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int n = n0 + g * 16 + 4 * (lane >> 4);
          if (row && n < N) *reinterpret_cast<u32x2_t*>(row + n) = pack(g, h);
        }
      }
      return;
    }
    constexpr int PITCH = 32 * NG + 16;     // bytes per staged row (padded against bank conflicts)
    constexpr int CHUNKS = 2 * NG, RPI = 64 / CHUNKS;  // 16-byte pieces of a row, rows per instruction
    uint8_t* wl = smem + w * (16 * PITCH);
    const int j = lane % CHUNKS;
#pragma unroll
    for (int h = 0; h < MG; ++h) {
      if (h >= lg) break;
#pragma unroll
      for (int g = 0; g < NG; ++g)
        *reinterpret_cast<u32x2_t*>(wl + (lane & 15) * PITCH + g * 32 + 8 * (lane >> 4)) = pack(g, h);
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
      for (int r0 = 0; r0 < 16; r0 += RPI) {
        const int r = r0 + lane / CHUNKS;
        OUT* row = row_ptr(h * 16 + r);
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(wl + r * PITCH + 16 * j);
        if (row && n0 + 8 * j < N) *reinterpret_cast<u32x4_t*>(row + n0 + 8 * j) = v;
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
      __builtin_amdgcn_wave_barrier();
      __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    }
  }
}

// Live 16-row groups of a block whose slots are in s_slot[BM] (live rows come first).
template <int BM>
__device__ __forceinline__ int live_groups(const int* s_slot, int lane) {
  const uint64_t m0 = __ballot(lane < BM && s_slot[lane < BM ? lane : 0] >= 0);
  const uint64_t m1 = BM > 64 ? __ballot(s_slot[BM > 64 ? 64 + lane : 0] >= 0) : 0ull;
  const int last = m1 ? 127 - __clzll((long long)m1) : (m0 ? 63 - __clzll((long long)m0) : -1);
  return __builtin_amdgcn_readfirstlane((last + 16) >> 4);
}

// Direct global -> LDS load of 16 (or 4) bytes per lane from the lane's own 64-bit address to
// lds + lane * BYTES; waited for with wait_vm<> (as dma_to_lds).
template <int BYTES>
__device__ __forceinline__ void dma_from(const uint8_t* p, uint32_t lds) {
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(lds);
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(m0), "v"(p) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(m0), "v"(p) : "memory", "m0");
}

// Workgroup = 4 waves over up to 16 * MG rows of one block x 64 * NG weight rows; wave w owns NG
// 16-row tiles and all the rows.  The waves share the activations, so these go through LDS (two
// stages, written by direct loads in operand order: a ds_read_b128 per lane and half operand); a
// weight tile is used by one wave only and goes straight to its registers, one step ahead.  With all
// of them in LDS a step of 128 rows would move 144 KB through it, more than its 128 bytes a clock
// allow beside the MFMAs; without the weights it is 80 KB.
template <typename T, int MG, int NG>
__global__ __launch_bounds__(256, 2) void block_gemm_tile_kernel(BlockGemmArgs a) {
  constexpr int BM = 16 * MG;
  constexpr int XL = MG / 2;                       // activation loads per thread and step
  constexpr int XB = 2 * MG * 1024;                // bytes of activations per step
  constexpr int STAGE = XB + (T::kScaled ? BM * 4 : 0);
  constexpr int EPI = 4 * 16 * (32 * NG + 16);
  constexpr int SMEM = 2 * STAGE > EPI ? 2 * STAGE : EPI;
  __shared__ __attribute__((aligned(16))) uint8_t smem[SMEM];
  __shared__ int s_slot[BM];
  const uint32_t smem_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;

  const int strips = (a.N + 64 * NG - 1) / (64 * NG), subs = (a.block_m + BM - 1) / BM;
  int mb, strip;
  grouped_block(strips, a.group_m, mb, strip);
  const int b = mb / subs, sub = mb - b * subs;
  int e = 0;
  if (a.sorted) {
    if ((int64_t)b * a.block_m >= *a.ntpp) return;
    e = a.eids[b];
    if (e < 0 || e >= a.E) return;
  }
  if (tid < BM) s_slot[tid] = slot_of(a, b, sub * BM + tid);
  __syncthreads();
  const int lg = live_groups<BM>(s_slot, lane);
  if (lg == 0) return;  // (uniform over the workgroup)

  const int KT = (a.Kb + kStepBytes - 1) / kStepBytes;
  const bool ragged = a.Kb % kStepBytes != 0;
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(&g_zero16);

  // activations: load l of wave w is operand half i of group g, i * MG + g = 4 l + w
  const uint8_t* xp[XL];
#pragma unroll
  for (int l = 0; l < XL; ++l) {
    const int i = (4 * l + w) / MG, g = (4 * l + w) % MG;
    const int s = s_slot[g * 16 + (lane & 15)];
    xp[l] = a.A + (int64_t)(s >= 0 ? s / a.top_k : 0) * a.lda + i * 64 + 16 * (lane >> 4);
  }
  // scales of the rows, staged [row % 16][group]
  const uint8_t* sp = nullptr;
  if constexpr (T::kScaled) {
    const int p = (w * 64 + lane) % BM, s = s_slot[(p % MG) * 16 + p / MG];
    sp = reinterpret_cast<const uint8_t*>(a.sa + (int64_t)(s >= 0 ? s / a.top_k : 0) * a.ld_sa);
  }
  auto issue_x = [&](auto partial, int kt, int stage) __attribute__((always_inline)) {
    const uint32_t st = smem_lds + (uint32_t)(stage * STAGE);
    const bool tail = ragged && kt == KT - 1;
#pragma unroll
    for (int l = 0; l < XL; ++l) {
      const int i = (4 * l + w) / MG, g = (4 * l + w) % MG;
      if (decltype(partial)::value && g >= lg) continue;  // all padding: never read
      const uint8_t* p = xp[l] + (int64_t)kt * kStepBytes;
      if (tail && kt * kStepBytes + i * 64 + 16 * (lane >> 4) >= a.Kb) p = zero;
      dma_from<16>(p, st + (uint32_t)(4 * l + w) * 1024);
    }
    if constexpr (T::kScaled) {
      if (w * 64 < BM) {
        if (BM >= 64 || lane < BM) dma_from<4>(sp + (int64_t)kt * 4, st + XB + (uint32_t)(w * 256));
      }
    }
  };
  // weights: rows n0 .. n0 + 16 NG - 1 of the expert (clamped at the N edge, not stored)
  const int n0 = (strip * 4 + w) * 16 * NG;
  const int nbase = min(n0, a.N - 1);
  const uint8_t* wbase = uniform_ptr(a.W + ((int64_t)e * a.N + nbase) * a.Kb);
  uint32_t woff[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g)
    woff[g] = (uint32_t)(min(n0 + g * 16 + (lane & 15), a.N - 1) - nbase) * (uint32_t)a.Kb + 16u * (lane >> 4);
  auto load_w = [&](int kt, Frag (&f)[NG]) __attribute__((always_inline)) {
    const uint8_t* p = wbase + (int64_t)kt * kStepBytes;
    if (ragged && kt == KT - 1) {
      const int k = kt * kStepBytes + 16 * (lane >> 4);
#pragma unroll
      for (int g = 0; g < NG; ++g)
        f[g] = load_frag(k < a.Kb ? p + woff[g] : zero, k + 64 < a.Kb ? p + woff[g] + 64 : zero);
    } else {
#pragma unroll
      for (int g = 0; g < NG; ++g) f[g] = load_frag(p + woff[g], p + woff[g] + 64);
    }
  };
  const float* sbp = nullptr;
  if constexpr (T::kScaled)  // (16 NG rows from a multiple of 16 NG: one block of 128)
    sbp = a.sb + ((int64_t)e * ((a.N + kScaleBlock - 1) / kScaleBlock) + nbase / kScaleBlock) * KT;

  f32x4_t acc[NG][MG];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int h = 0; h < MG; ++h) acc[g][h] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  auto read_x = [&](const uint8_t* st, int h) __attribute__((always_inline)) {
    return load_frag(st + h * 1024 + lane * 16, st + (MG + h) * 1024 + lane * 16);
  };
  auto read_s = [&](const uint8_t* st, int h) __attribute__((always_inline)) {
    return T::kScaled ? reinterpret_cast<const float*>(st + XB)[(lane & 15) * MG + h] : 0.f;
  };
  // One step's products.  An expert's last block (PARTIAL) skips its all-padding groups.
  auto compute = [&](auto partial, const uint8_t* st, const Frag (&wf)[NG], float sb) __attribute__((always_inline)) {
    constexpr bool PARTIAL = decltype(partial)::value;
    if constexpr (T::kScaled) {
      // The scaled sum of a product is taken two MFMAs after it, so that one wave keeps the matrix
      // core and the vector unit busy together; the scheduling barriers hold that order (left to
      // itself the compiler gathers the products first, which spills).
      f32x4_t t[3];
      float sv[3];
      auto take = [&](int i) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[i % NG][i / NG][q] = fmaf(t[i % 3][q], sv[i % 3], acc[i % NG][i / NG][q]);
        asm volatile("" : "+v"(acc[i % NG][i / NG]));  // taken here (not sunk into the next step's blocks)
      };
      Frag x = read_x(st, 0);
      float sc = read_s(st, 0);
#pragma unroll
      for (int h = 0; h < MG; ++h) {
        if (PARTIAL && h >= lg) continue;
        const Frag xn = h + 1 < MG ? read_x(st, h + 1) : x;
        const float sn = h + 1 < MG ? read_s(st, h + 1) : 0.f;
        const float s = sc * sb;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int i = h * NG + g;
          t[i % 3] = mfma_step(T{}, wf[g], x);
          sv[i % 3] = s;
          if (PARTIAL ? g >= 2 : i >= 2) take(i - 2);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (PARTIAL || h + 1 == MG) {
          take(h * NG + NG - 2);
          take(h * NG + NG - 1);
        }
        x = xn;
        sc = sn;
      }
    } else {
#pragma unroll
      for (int h = 0; h < MG; ++h) {
        if (PARTIAL && h >= lg) continue;
        const Frag x = read_x(st, h);
#pragma unroll
        for (int g = 0; g < NG; ++g) acc[g][h] = mfma_step(T{}, wf[g], x, acc[g][h]);
      }
    }
  };

  // One step: the next step's operands are requested first (the weights before the direct loads, so
  // that the wait the compiler puts before a weight's first use counts nothing but weights), and
  // have all landed when the step's closing barrier is passed.
  Frag wa[NG], wb[NG];
  float sba = 0.f, sbb = 0.f;
  auto landed = [&](Frag (&f)[NG]) __attribute__((always_inline)) {
    wait_vm<0>();
#pragma unroll
    for (int g = 0; g < NG; ++g) asm volatile("" : "+v"(f[g]));
    block_barrier();
  };
  auto step = [&](auto partial, int kt, int stage, const Frag (&cur)[NG], Frag (&next)[NG], float sc,
                  float& sn) __attribute__((always_inline)) {
    const int kn = min(kt + 1, KT - 1);  // (past the end the last step again, not used)
    load_w(kn, next);
    if constexpr (T::kScaled) sn = sbp[kn];
    issue_x(partial, kn, stage ^ 1);
    compute(partial, smem + stage * STAGE, cur, sc);
    landed(next);
  };
  auto k_loop = [&](auto partial) __attribute__((always_inline)) {
    int kt = 0;
    for (; kt + 1 < KT; kt += 2) {
      step(partial, kt, 0, wa, wb, sba, sbb);
      step(partial, kt + 1, 1, wb, wa, sbb, sba);
    }
    if (kt < KT) step(partial, kt, 0, wa, wb, sba, sbb);
  };
  load_w(0, wa);
  if constexpr (T::kScaled) sba = sbp[0];
  issue_x(std::true_type{}, 0, 0);
  landed(wa);
  if (lg == MG) k_loop(std::false_type{});
  else k_loop(std::true_type{});

  if (a.bias) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int n = n0 + g * 16 + 4 * (lane >> 4);
      if (n >= a.N) continue;
      const u32x2_t bb = *reinterpret_cast<const u32x2_t*>(a.bias + (int64_t)e * a.N + n);
      const f32x4_t bv = {bf16_lo(bb[0]), bf16_hi(bb[0]), bf16_lo(bb[1]), bf16_hi(bb[1])};
#pragma unroll
      for (int h = 0; h < MG; ++h) acc[g][h] += bv;
    }
  }
  const bool wide = ((uintptr_t)a.C & 15) == 0 && (a.ldc & 7) == 0;
  store_tiles<NG, MG, uint16_t>(acc, lg, smem, SMEM, w, lane, n0, a.N, wide, [&](int r) -> uint16_t* {
    const int s = s_slot[r];
    return s >= 0 ? a.C + (int64_t)s * a.ldc : nullptr;
  });
}

template <typename T, int MG>
static int launch_tile(const char* fn, BlockGemmArgs a, int64_t cap_blocks, hipStream_t st) {
  constexpr int NG = 4;
  a.group_m = default_group_m(a.Kb / T::kBytes, a.block_m);
  const int64_t grid = (int64_t)((a.N + 64 * NG - 1) / (64 * NG)) * cap_blocks * ((a.block_m + 16 * MG - 1) / (16 * MG));
  MOE_REQUIRE(grid < (1ll << 31), MOE_EUNSUPPORTED, "%s: grid too large", fn);
  hipLaunchKernelGGL((block_gemm_tile_kernel<T, MG, NG>), dim3((unsigned)grid), dim3(256), 0, st, a);
  return check_launch(fn);
}

template <typename T>
static int launch_block_gemm(const char* fn, const BlockGemmArgs& a, int64_t cap_blocks, hipStream_t st) {
  if (a.block_m > 64) return launch_tile<T, 8>(fn, a, cap_blocks, st);
  if (a.block_m > 32) return launch_tile<T, 4>(fn, a, cap_blocks, st);
  if (a.block_m > 16) return launch_tile<T, 2>(fn, a, cap_blocks, st);
  constexpr int NG = 2, KS = 4;
  const int64_t grid = (int64_t)((a.N + 16 * NG - 1) / (16 * NG)) * cap_blocks;
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
