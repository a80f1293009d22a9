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
  void* C;
  int64_t ldc;
  const int32_t* sorted;  // null: dense, block b holds rows b * block_m ..., expert 0
  const int32_t* eids;
  const int32_t* ntpp;
  int32_t numel, top_k, block_m, N, Kb, E;
  int32_t tiles, group_m, group_n;  // tile kernel: tiles of rows; tiles and strips of an XCD's unit
  int32_t cap_blocks;     // most blocks the align can have made
  const int32_t* live;    // set: rows of C whose slot is dropped (live[slot] < 0) are zeroed, else left alone
  int64_t expected;       // live slots to expect: chooses the launch, hence the order of sums, and nothing else
};

struct Fp8Type {
  static constexpr bool kScaled = true, kTrans = false;
  static constexpr int kBytes = 1;
  typedef uint16_t Out;
};
struct Bf16Type {
  static constexpr bool kScaled = false, kTrans = false;
  static constexpr int kBytes = 2;
  typedef uint16_t Out;
};
// The product's gradient: the reduction runs over the rows of W, C[s, n] = sum_k A[s, k] W[e, k, n] with
// W [E, Kb / 2, N] (N: the columns of C).  OUT: bf16 or fp32 rows.
template <typename OUT>
struct Bf16TransType : Bf16Type {
  static constexpr bool kTrans = true;
  typedef OUT Out;
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
__device__ __forceinline__ f32x4_t mfma_step(const Bf16Type&, const Frag& w, const Frag& x, f32x4_t acc) {
  acc = mfma(frag_lo(w), frag_lo(x), acc);
  return mfma(frag_hi(w), frag_hi(x), acc);
}
// (The instruction adds the products of eight consecutive k on the exponent of the largest, cut 13
// places below it, and these sums in fp32: the matrix core's own precision for 8-bit operands,
// measured 2^-19 rms and 2^-16 at most of the sum of the products' magnitudes.)
__device__ __forceinline__ f32x4_t mfma_step(Fp8Type, const Frag& w, const Frag& x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

// The slot of sorted entry `at` (dense: row `at`), or -1 for padding.
__device__ __forceinline__ int slot_at(const BlockGemmArgs& a, int64_t at) {
  const int64_t s = a.sorted ? a.sorted[at] : at;
  return s >= 0 && s < a.numel ? (int)s : -1;
}

// A launch counts its threads in 32 bits.
inline bool launchable(int64_t grid, int threads) { return grid * threads < (1ll << 32); }

// Zeros in the rows of dropped slots, shared by all the workgroups of a launch: rows blockIdx.x, +
// gridDim.x, ..., of which `mine` holds the flags of the first 64 (asked for when the workgroup starts,
// as drop_flags, so that its end does not wait for them).
__device__ __forceinline__ int drop_flags(const BlockGemmArgs& a, int64_t first) {
  const int64_t r = first + (int64_t)gridDim.x * (threadIdx.x & 63);
  return a.live && r < a.numel ? a.live[r] : 0;
}
template <typename OUT>
__device__ __forceinline__ void zero_dropped(const BlockGemmArgs& a, int mine) {
  if (!a.live) return;
  for (int64_t first = blockIdx.x;;) {
    for (uint64_t dead = __ballot(mine < 0); dead; dead &= dead - 1) {
      OUT* row = static_cast<OUT*>(a.C) + (first + (int64_t)gridDim.x * __builtin_ctzll(dead)) * a.ldc;
      for (int c = threadIdx.x * 4; c < a.N; c += blockDim.x * 4) {
        if constexpr (sizeof(OUT) == 4) *reinterpret_cast<f32x4_t*>(row + c) = f32x4_t{0.f, 0.f, 0.f, 0.f};
        else *reinterpret_cast<u32x2_t*>(row + c) = u32x2_t{0u, 0u};
      }
    }
    first += (int64_t)gridDim.x * 64;
    if (first >= a.numel) break;
    mine = drop_flags(a, first);
  }
}

// ---------------------------------------------------------------------------- few rows
// Workgroup = up to 16 slots of a block (MB = 2: of two consecutive blocks of one expert) x NG 16-row
// weight tiles, K split over its KS waves, operands straight from memory to registers in chunks of
// kChunk steps, partial sums joined through LDS in wave order.  The cost is the stream of weights (64 tokens
// of 8 choices on 32 of 256 experts, N = 8192, K = 4096: 876 MB in 147 - 150 us, 5.8 - 6.0 TB/s).
template <typename T, int NG, int KS, int MB>
__device__ __forceinline__ void gemm_stream(const BlockGemmArgs& a, f32x4_t (&part)[KS][NG * MB][64]) {
  constexpr int kChunk = 4;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int strips = (a.N + 16 * NG - 1) / (16 * NG);
  const int strip = blockIdx.x % strips, b = blockIdx.x / strips;
  int e = 0, blocks = 1;
  if (a.sorted) {
    const int nb = *a.ntpp / a.block_m;
    e = a.eids[b];
    if constexpr (MB == 2) {
      // the expert's blocks in front of b, and whether the next one is its too
      const int next = b + 1 < a.cap_blocks ? a.eids[b + 1] : -1;
      int before = 0;
      for (;;) {
        const int i = b - 1 - before - lane;
        const uint64_t other = __ballot(i < 0 || a.eids[i < 0 ? 0 : i] != e);
        if (other) {
          before += __builtin_ctzll(other);
          break;
        }
        before += 64;
      }
      if (before & 1) return;  // (the block in front takes this one along)
      blocks = next == e && b + 1 < nb ? 2 : 1;
    }
    if (b >= nb || e < 0 || e >= a.E) return;
  }
  const int KT = (a.Kb + kStepBytes - 1) / kStepBytes;
  const int kt0 = KT * w / KS, kt1 = KT * (w + 1) / KS;
  const int koff = 16 * (lane >> 4);
  int slot[MB];
  const uint8_t* xp[MB];
  const float* sap[MB];
#pragma unroll
  for (int m = 0; m < MB; ++m) {
    slot[m] = (lane & 15) < a.block_m && m < blocks ? slot_at(a, (int64_t)(b + m) * a.block_m + (lane & 15)) : -1;
    const int64_t row = slot[m] >= 0 ? slot[m] / a.top_k : 0;
    xp[m] = a.A + row * a.lda + koff;
    if constexpr (T::kScaled) sap[m] = a.sa + row * a.ld_sa;
  }
  const uint8_t* wp[NG];
  const float* sbp[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const int n = min((strip * NG + g) * 16 + (lane & 15), a.N - 1);
    wp[g] = a.W + ((int64_t)e * a.N + n) * a.Kb + koff;
    if constexpr (T::kScaled)
      sbp[g] = a.sb + ((int64_t)e * ((a.N + kScaleBlock - 1) / kScaleBlock) + n / kScaleBlock) * KT;
  }
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(&g_zero16);

  f32x4_t acc[NG][MB];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int m = 0; m < MB; ++m) acc[g][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int c = kt0; c < kt1; c += kChunk) {
    Frag x[kChunk][MB], wt[kChunk][NG];
    float sa[kChunk][MB], sb[kChunk][NG];
#pragma unroll
    for (int u = 0; u < kChunk; ++u) {
      const int kt = min(c + u, kt1 - 1);  // (past the wave's last step: loaded again, not used)
      const int64_t k0 = (int64_t)kt * kStepBytes;
      const bool lo = k0 + koff < a.Kb, hi = k0 + koff + 64 < a.Kb;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        wt[u][g] = load_frag(lo ? wp[g] + k0 : zero, hi ? wp[g] + k0 + 64 : zero);
        if constexpr (T::kScaled) sb[u][g] = sbp[g][kt];
      }
#pragma unroll
      for (int m = 0; m < MB; ++m) {
        x[u][m] = load_frag(lo && slot[m] >= 0 ? xp[m] + k0 : zero, hi && slot[m] >= 0 ? xp[m] + k0 + 64 : zero);
        if constexpr (T::kScaled) sa[u][m] = sap[m][kt];
      }
    }
    // (eight waves: all of a chunk's loads in flight; with more workgroups a CU the compiler's order, which
    // keeps fewer registers and more of them resident, is the faster one)
    if constexpr (KS == 8) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < kChunk; ++u) {
      if (c + u >= kt1) break;
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int m = 0; m < MB; ++m) {
          if constexpr (T::kScaled) {
            const f32x4_t t = mfma_step(T{}, wt[u][g], x[u][m]);
            // (the scale of the weight block belongs to the tile's rows: lane l's row of the operand
            // and the rows of its result lie in one 16-row tile, hence in one block)
            const float s = sa[u][m] * sb[u][g];
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[g][m][q] = fmaf(t[q], s, acc[g][m][q]);
          } else {
            acc[g][m] = mfma_step(T{}, wt[u][g], x[u][m], acc[g][m]);
          }
        }
    }
  }
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int m = 0; m < MB; ++m) part[w][g * MB + m][lane] = acc[g][m];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NG * MB; ++i) {
    if (i % KS != w) continue;
    const int g = i / MB, m = i % MB;
    f32x4_t v = part[0][i][lane];
#pragma unroll
    for (int k = 1; k < KS; ++k) v += part[k][i][lane];
    const int n0 = (strip * NG + g) * 16 + 4 * (lane >> 4);
    if (n0 < a.N && slot[m] >= 0) {  // (N is a multiple of 8: four columns are in or out together)
      if (a.bias) {
        const u32x2_t bb = *reinterpret_cast<const u32x2_t*>(a.bias + (int64_t)e * a.N + n0);
        v[0] += bf16_lo(bb[0]); v[1] += bf16_hi(bb[0]); v[2] += bf16_lo(bb[1]); v[3] += bf16_hi(bb[1]);
      }
      *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(a.C) + (int64_t)slot[m] * a.ldc + n0) =
          u32x2_t{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
  }
}

template <typename T, int NG, int KS, int MB>
__global__ __launch_bounds__(64 * KS) void block_gemm_stream_kernel(BlockGemmArgs a) {
  __shared__ f32x4_t part[KS][NG * MB][64];
  const int flags = T::kScaled ? 0 : drop_flags(a, blockIdx.x);
  gemm_stream<T, NG, KS, MB>(a, part);
  if constexpr (!T::kScaled) zero_dropped<uint16_t>(a, flags);
}

template <typename T, int NG, int KS, int MB>
static int launch_stream(const char* fn, BlockGemmArgs a, int64_t cap_blocks, hipStream_t st) {
  a.cap_blocks = (int32_t)cap_blocks;
  const int64_t grid = (int64_t)((a.N + 16 * NG - 1) / (16 * NG)) * cap_blocks;
  MOE_REQUIRE(launchable(grid, 64 * KS), MOE_EUNSUPPORTED, "%s: grid too large", fn);
  hipLaunchKernelGGL((block_gemm_stream_kernel<T, NG, KS, MB>), dim3((unsigned)grid), dim3(64 * KS), 0, st, a);
  return check_launch(fn);
}

// ---------------------------------------------------------------------------- blocks of rows
// The outputs of a wave's NG 16-column tiles (columns n0 ..) for up to MG 16-row groups, of which the
// first lg are live.  acc[g][h] holds, in lane l, columns 4 (l / 16) + 0..3 of tile g of row l % 16
// of group h.  bf16 rows go through the wave's own part of LDS (idle: every wave has passed the last
// step's barrier), so that a store instruction covers whole segments of 32 * NG bytes of a row with
// 16 bytes a lane.  row_ptr(r) is where row r starts, or null.  The stores pass the L2 by: what a tile
// writes would push the operands that the XCD's workgroups share out of it (weight gradients of 32 experts,
// N = K = 4096: 588 -> 508 us; Zipf prefill of 4096 tokens 914 -> 887, of 1024 in bf16 600 -> 584).
template <int NG, int MG, typename OUT, typename RowPtr>
__device__ __forceinline__ void store_tiles(const f32x4_t (&acc)[NG][MG], int lg, uint8_t* smem, int w, int lane,
                                            int n0, int N, bool wide, RowPtr row_ptr) {
  if constexpr (sizeof(OUT) == 4) {
#pragma unroll
    for (int h = 0; h < MG; ++h) {
      if (h >= lg) break;
      OUT* row = row_ptr(h * 16 + (lane & 15));
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const int n = n0 + g * 16 + 4 * (lane >> 4);
        if (row && n < N) __builtin_nontemporal_store(acc[g][h], reinterpret_cast<f32x4_t*>(row + n));
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
        if (RPI > 16 && r >= 16) continue;  // (one tile: 32 rows' worth of lanes, 16 rows)
        OUT* row = row_ptr(h * 16 + r);
        const u32x4_t v = *reinterpret_cast<const u32x4_t*>(wl + r * PITCH + 16 * j);
        if (row && n0 + 8 * j < N) __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(row + n0 + 8 * j));
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
  int last = -1;
#pragma unroll
  for (int r = 0; r < BM; r += 64) {
    const uint64_t m = __ballot(r + lane < BM && s_slot[r + lane < BM ? r + lane : 0] >= 0);
    if (m) last = r + 63 - __clzll((long long)m);
  }
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

// ---------------------------------------------------------------------------- transposed operands
// A tile whose rows are the reduction index, as it lies in memory, staged [rows][16 bytes * kPieces] with
// the pairs of 16-byte pieces of a row (16 values) at place pair ^ trans_swizzle(row).  An operand of 16
// columns is read with ds_read_b64_tr_b16: within 16 lanes that together read four rows of 16 values,
// lane i receives column i, so two of them give a lane the eight consecutive rows that an MFMA wants.
// The swizzle keeps the rows that 32 lanes read together, 8 j + r for j = 0, 1 and r = 0..3, in
// different banks (rows of 128 bytes have four pairs, and two rows then share a bank).
__device__ __forceinline__ int trans_swizzle(int row, int pitch) {
  return ((row & 3) | ((row >> 1) & 4)) & (pitch / 32 - 1);
}

typedef __attribute__((ext_vector_type(4))) int16_t s16x4_t;
__device__ __forceinline__ u32x2_t lds_read_tr(const uint8_t* p) {
  const s16x4_t v = __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4_t*)p);
  return __builtin_bit_cast(u32x2_t, v);
}
// Where lane l begins to read pair `pair` of the staged rows: row 8 (l / 16) + (l % 16) / 4, the lane's
// 8 bytes of the pair.  (The swizzle is the same for that row plus 4 and plus any multiple of 16.)
__device__ __forceinline__ int trans_lane(int pair, int pitch, int lane) {
  const int row = 8 * (lane >> 4) + ((lane & 15) >> 2);
  return row * pitch + ((pair ^ trans_swizzle(row, pitch)) << 5) + (lane & 3) * 8;
}
// The operand of 32 rows from `tile` on.
__device__ __forceinline__ u32x4_t trans_operand(const uint8_t* tile, int lane_off, int pitch) {
  const u32x2_t lo = lds_read_tr(tile + lane_off), hi = lds_read_tr(tile + lane_off + 4 * pitch);
  return u32x4_t{lo[0], lo[1], hi[0], hi[1]};
}

// ---------------------------------------------------------------------------- blocks of rows, the kernel
// Launch index -> (tile of rows, strip of weight rows).  A unit of group_m tiles x group_n strips runs
// on one XCD, so that its workgroups share activations and weights in that XCD's L2; the units go
// round the XCDs, strips first, so that the eight that run side by side share tiles of rows.
__host__ __device__ inline void unit_tile(int P, int strips, int group_m, int group_n, int& mb, int& strip) {
  const int U = group_m * group_n, across = (strips + group_n - 1) / group_n;
  const int j = P / kXcds, u = j / U * kXcds + P % kXcds, r = j % U;
  mb = u / across * group_m + r % group_m;
  strip = u % across * group_n + r / group_m;
}

// The units for `tiles` x `strips` workgroups, and the launch's size.  4 x 8, a workgroup for each CU of an
// XCD, or smaller ones where eight XCDs would share these unevenly: the first shape whose fullest XCD has
// within a sixteenth of the least.  Strips are split evenly.
// (Measured on the Zipf prefill product: units of 1 x all strips, 2 x 16 and 4 x 8 1076, 1024, 999 us.
// 4608 slots on 8 experts, 26 x 8 workgroups: in units of 4 x 6, hence 4 x 2 at the edge, which go to every
// other XCD, K = 512 and 2048 take 36 and 91 us, in units of 4 x 4 21 and 51.)
static int64_t choose_units(int64_t tiles, int64_t strips, int32_t* group_m, int32_t* group_n) {
  int64_t gm[6], gn[6], load[6], best = INT64_MAX;
  for (int i = 0; i < 6; ++i) {
    gm[i] = std::min<int64_t>(tiles, 4 >> (i / 2));
    const int64_t across = (strips + 7) / 8 << (i % 2);
    gn[i] = (strips + across - 1) / across;
    const int64_t units = ((tiles + gm[i] - 1) / gm[i]) * ((strips + gn[i] - 1) / gn[i]);
    load[i] = (units + kXcds - 1) / kXcds * gm[i] * gn[i];
    best = std::min(best, load[i]);
  }
  int i = 0;
  while (load[i] > best + best / 16) ++i;
  *group_m = (int32_t)gm[i];
  *group_n = (int32_t)gn[i];
  return load[i] * kXcds;
}

// A tile of BM entries made of several blocks: an expert's blocks follow each other, and the ones whose
// number within the expert is a multiple of BM / block_m start a tile.  Gives tile t's first block, its
// expert and its entries (0 behind the last tile), each wave for itself with 64 blocks at a time.  (The
// tiles are counted here, by each workgroup for itself, so that no launch has to come before and the
// live tiles lie side by side for the XCDs.)
__device__ __forceinline__ int merged_tile(const BlockGemmArgs& a, int nb, int BM, int t, int* block, int* expert) {
  const int lane = threadIdx.x & 63, per = BM / a.block_m;
  int from = 0;  // where the current expert's blocks begin
  for (int base = 0; base < nb; base += 64) {
    const int i = base + lane;
    const int e = i < nb ? a.eids[i] : -1, prev = i > 0 && i <= nb ? a.eids[i - 1] : -2;
    const uint64_t begins = __ballot(e != prev);
    const uint64_t upto = begins & (~0ull >> (63 - lane));
    const int mine = upto ? base + 63 - __clzll((long long)upto) : from;
    uint64_t starts = __ballot(e >= 0 && e < a.E && (i - mine) % per == 0);
    const int n = __popcll(starts);
    if (t < n) {
      for (; t > 0; --t) starts &= starts - 1;
      const int l = __builtin_ctzll(starts);
      *block = base + l;
      *expert = __builtin_amdgcn_readlane(e, l);
      int blocks = 1;
      while (blocks < per && base + l + blocks < nb && a.eids[base + l + blocks] == *expert) ++blocks;
      return blocks * a.block_m;
    }
    t -= n;
    if (begins) from = base + 63 - __clzll((long long)begins);
  }
  return 0;
}

// Workgroup = WM x WN waves over BM = 16 * MG * WM rows of one block x BN = 16 * NG * WN weight rows;
// wave (wm, wn) owns MG 16-row groups and NG 16-row weight tiles.
//
// Both operands go through LDS, kStages steps deep, written by direct global -> LDS loads.  A staged
// row is its 128 bytes of the step in eight 16-byte pieces, piece p at place p ^ (row & 7): the eight
// lanes that load a row then ask for one whole cache line (an operand loaded straight to registers
// has its adjacent lanes in different rows, a cache line each: 64 address cycles a load instead of
// 16, which held the first form of this kernel to a third of the speed), and the eight lanes that a
// ds_read_b128 serves at once, eight rows of the same piece, hit different banks.
//
// Step kt + kStages - 1 is requested when step kt starts.  The step's closing wait and barrier come
// before the products of its last row group, whose operands are in registers by then: the first
// operands of the next step are read from LDS behind those products.
template <typename T, int MG, int NG, int WM, int WN, int kStages>
struct TileShape {
  static constexpr int WAVES = WM * WN, BM = 16 * MG * WM, BN = 16 * NG * WN;
  static constexpr int XI = BM / 8 / WAVES, WI = BN / 8 / WAVES;   // direct loads per wave and step, 1 KB each
  static_assert(MG >= 2, "a step's loads are asked for in its row groups but the last");
  static_assert(XI * 8 * WAVES == BM && WI * 8 * WAVES == BN, "the waves share the staged rows evenly");
  static constexpr int SR = BM / WAVES, SP = SR + 4;  // rows whose scales a wave loads; its place for them
  static constexpr int XB = BM * kStepBytes, WB = BN * kStepBytes;
  static constexpr int STAGE = XB + WB + (T::kScaled ? WAVES * SP * 4 : 0);
  static constexpr int BYTES = kStages * STAGE;
  static_assert(BYTES >= WAVES * 16 * (32 * NG + 16), "the epilogue's staging fits");
};

template <typename T, int MG, int NG, int WM, int WN, int kStages, bool kMerge>
constexpr int tile_bytes() {
  constexpr int full = TileShape<T, MG, NG, WM, WN, kStages>::BYTES;
  if constexpr (kMerge && MG >= 4) {
    constexpr int half = TileShape<T, MG / 2, NG, WM, WN, kStages + 1>::BYTES;
    return half > full ? half : full;
  }
  return full;
}

// One tile: the `rows` sorted entries from `first` on, of expert e, and strip `strip` of its weights.
template <typename T, int MG, int NG, int WM, int WN, int kStages>
__device__ __forceinline__ void gemm_tile(const BlockGemmArgs& a, uint8_t* smem, int* s_slot, int64_t first, int rows,
                                          int e, int strip) {
  typedef TileShape<T, MG, NG, WM, WN, kStages> Shape;
  constexpr int BM = Shape::BM, BN = Shape::BN, XI = Shape::XI, WI = Shape::WI, SR = Shape::SR, SP = Shape::SP;
  constexpr int XB = Shape::XB, WB = Shape::WB, STAGE = Shape::STAGE;
  constexpr int LOADS = XI + WI + (T::kScaled ? 1 : 0);
  constexpr int SPREAD = kStages > 2 && MG > 2 ? MG - 1 : (MG > 2 ? 2 : 1);  // row groups over which the loads are spread
  const uint32_t smem_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = w / WN, wn = w % WN;

  int xs[XI], ss = -1;
#pragma unroll
  for (int l = 0; l < XI; ++l) {
    const int r = (w * XI + l) * 8 + (lane >> 3);
    xs[l] = r < rows ? slot_at(a, first + r) : -1;
  }
  if (T::kScaled && lane % SR + w * SR < rows) ss = slot_at(a, first + w * SR + lane % SR);
  const int KT = (a.Kb + kStepBytes - 1) / kStepBytes;
  const bool ragged = a.Kb % kStepBytes != 0;
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(&g_zero16);
  const int piece = ((lane & 7) ^ (lane >> 3)) * 16;  // (a load's rows start at a multiple of eight)

  const uint8_t* xp[XI];
#pragma unroll
  for (int l = 0; l < XI; ++l) xp[l] = a.A + (int64_t)(xs[l] >= 0 ? xs[l] / a.top_k : 0) * a.lda + piece;
  const int nw = strip * BN;  // the strip's weight rows, or columns (clamped at the N edge, not stored)
  // Trans: 64 rows of the reduction a step, PW bytes of each; a load brings RW of them
  constexpr int PW = BN * 2, RW = 1024 / PW;
  const int64_t wpitch = T::kTrans ? (int64_t)a.N * 2 : a.Kb;
  const uint8_t* wbase = uniform_ptr(T::kTrans ? a.W + (int64_t)e * (a.Kb / 2) * wpitch + nw * 2
                                               : a.W + ((int64_t)e * a.N + nw) * a.Kb);
  const int64_t wstep = T::kTrans ? (kStepBytes / 2) * wpitch : kStepBytes;
  uint32_t woff[WI];
  int wrow[WI];  // Trans: the row of the reduction that this lane loads
#pragma unroll
  for (int l = 0; l < WI; ++l) {
    if constexpr (T::kTrans) {
      wrow[l] = (w * WI + l) * RW + lane / (64 / RW);
      const int place = lane % (64 / RW), col = ((place >> 1) ^ trans_swizzle(wrow[l], PW)) * 16 + (place & 1) * 8;
      woff[l] = (uint32_t)(wrow[l] * wpitch) + (nw + col < a.N ? (uint32_t)col * 2 : 0u);
    } else {
      woff[l] = (uint32_t)min((w * WI + l) * 8 + (lane >> 3), a.N - 1 - nw) * (uint32_t)a.Kb + (uint32_t)piece;
    }
  }
  const int n0 = nw + wn * 16 * NG;
  // scales: lane l < SR brings that of row w * SR + l, lane SR that of the wave's own weight rows (16 NG
  // rows from a multiple of 16 NG lie in one block of 128).  All of it by direct loads: an ordinary
  // load in the loop would be waited for with every direct load in flight.
  const float* sp = nullptr;
  if constexpr (T::kScaled)
    sp = lane < SR ? a.sa + (int64_t)(ss >= 0 ? ss / a.top_k : 0) * a.ld_sa
                   : a.sb + ((int64_t)e * ((a.N + kScaleBlock - 1) / kScaleBlock) + min(n0, a.N - 1) / kScaleBlock) * KT;
  int lg = 0;  // (set below)
  // Loads first .. last - 1 of step kt's (past the end the last step's again, not used: every step has the
  // same count of loads).
  auto issue = [&](int kt, int stage, int first, int last) __attribute__((always_inline)) {
    const uint32_t st = smem_lds + (uint32_t)(stage * STAGE);
    kt = min(kt, KT - 1);
    auto load = [&](int l) __attribute__((always_inline)) {
      if (l < XI) dma_from<16>(xp[l] + (int64_t)kt * kStepBytes, st + (uint32_t)(w * XI + l) * 1024);
      else dma_to_lds<16>(wbase + kt * wstep, woff[l - XI], st + XB + (uint32_t)(w * WI + l - XI) * 1024);
    };
    if (ragged && kt == KT - 1) {
      // What lies behind K is zero in both operands (a NaN pattern there must not meet a zero).
      const bool in_row = kt * kStepBytes + piece < a.Kb;
#pragma unroll
      for (int l = 0; l < XI + WI; ++l) {
        if (l < first || l >= last) continue;
        const uint8_t* p = l < XI ? xp[l] + (int64_t)kt * kStepBytes : wbase + kt * wstep + woff[l - XI];
        const bool in = T::kTrans && l >= XI ? kt * (kStepBytes / 2) + wrow[l - XI] < a.Kb / 2 : in_row;
        dma_from<16>(in ? p : zero,
                     st + (l < XI ? (uint32_t)(w * XI + l) * 1024 : XB + (uint32_t)(w * WI + l - XI) * 1024));
      }
    } else {
#pragma unroll
      for (int l = 0; l < XI + WI; ++l)
        if (l >= first && l < last) load(l);
    }
    if constexpr (T::kScaled) {
      if (last == LOADS && lane <= SR)
        dma_from<4>(reinterpret_cast<const uint8_t*>(sp + kt), st + XB + WB + (uint32_t)(w * SP) * 4);
    }
  };

  f32x4_t acc[NG][MG];
#pragma unroll
  for (int g = 0; g < NG; ++g)
#pragma unroll
    for (int h = 0; h < MG; ++h) acc[g][h] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // the operand of the 16 staged rows at `rows`
  int trans_off[NG];
#pragma unroll
  for (int g = 0; g < NG; ++g) trans_off[g] = trans_lane(wn * NG + g, PW, lane);
  const int lo = (lane & 15) * kStepBytes + (((lane >> 4) ^ (lane & 7)) * 16);
  const int hi = (lane & 15) * kStepBytes + (((4 + (lane >> 4)) ^ (lane & 7)) * 16);
  auto read = [&](const uint8_t* rows) __attribute__((always_inline)) { return load_frag(rows + lo, rows + hi); };
  auto read_x = [&](const uint8_t* st, int h) __attribute__((always_inline)) {
    return read(st + (h * WM + wm) * 16 * kStepBytes);
  };
  auto read_s = [&](const uint8_t* st, int h) __attribute__((always_inline)) {
    const int r = (h * WM + wm) * 16 + (lane & 15);
    return T::kScaled ? reinterpret_cast<const float*>(st + XB + WB)[r / SR * SP + r % SR] : 0.f;
  };
  auto read_sb = [&](const uint8_t* st) __attribute__((always_inline)) {
    return T::kScaled ? reinterpret_cast<const float*>(st + XB + WB)[w * SP + SR] : 0.f;
  };
  auto read_w = [&](const uint8_t* st, int g) __attribute__((always_inline)) {
    if constexpr (T::kTrans)
      return frag_of(trans_operand(st + XB, trans_off[g], PW), trans_operand(st + XB + 32 * PW, trans_off[g], PW));
    else
      return read(st + XB + (wn * NG + g) * 16 * kStepBytes);
  };
  // A product of e4m3fn operands is scaled into the sum DIST products later, across row groups and steps,
  // so that one wave keeps the matrix core and the vector unit busy together and does not stand
  // for the product's latency (16 passes).  acc += t * s for the product before the last DIST:
  constexpr int DIST = !T::kScaled ? 1 : (NG * MG > 16 || NG * MG < 4 ? 2 : 4);
  f32x4_t t[DIST];
  float ts[DIST];
#pragma unroll
  for (int i = 0; i < DIST; ++i) {
    t[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    ts[i] = 0.f;
  }
  auto take = [&](int i, const f32x4_t& v, float s) __attribute__((always_inline)) {  // i: number of the product
    f32x4_t& c = acc[i % NG][i / NG];
#pragma unroll
    for (int q = 0; q < 4; ++q) c[q] = fmaf(v[q], s, c[q]);
    asm volatile("" : "+v"(c));  // taken here: the compiler else sinks it into later blocks
  };
  constexpr int P = NG * MG;  // products of a step
  static_assert(P % DIST == 0, "a step ends where the ring of products began");
  Frag wf[NG], x0;            // this step's weights, and its first row group
  float s0 = 0.f, sb = 0.f;   // scales: of that row group, of the weights
  // Products of row group h; where `next` is given (the last group of a step) each weight tile's place
  // takes the next step's behind its last product.
  auto products = [&](auto partial, const Frag& x, float s, int h, const uint8_t* next) __attribute__((always_inline)) {
    constexpr bool PARTIAL = decltype(partial)::value;
    if constexpr (T::kScaled) {
      if constexpr (!PARTIAL) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int i = h * NG + g;
          const f32x4_t now = mfma_step(T{}, wf[g], x);
          __builtin_amdgcn_sched_barrier(0);
          if (next) wf[g] = read_w(next, g);
          take((i + P - DIST) % P, t[i % DIST], ts[i % DIST]);
          t[i % DIST] = now;
          ts[i % DIST] = s;
          __builtin_amdgcn_sched_barrier(0);
        }
        return;
      } else if (h < lg) {  // (an expert's last tile: each group for itself)
        f32x4_t v[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) v[g] = mfma_step(T{}, wf[g], x);
#pragma unroll
        for (int g = 0; g < NG; ++g) take(h * NG + g, v[g], s);
      }
    } else if (!PARTIAL || h < lg) {
#pragma unroll
      for (int g = 0; g < NG; ++g) acc[g][h] = mfma_step(T{}, wf[g], x, acc[g][h]);
    }
    if (next) {
#pragma unroll
      for (int g = 0; g < NG; ++g) wf[g] = read_w(next, g);
    }
  };
  auto step = [&](auto partial, int kt, int stage) __attribute__((always_inline)) {
    const uint8_t* st = smem + stage * STAGE;
    const uint8_t* next = smem + (stage + 1 == kStages ? 0 : stage + 1) * STAGE;
    const int target = stage == 0 ? kStages - 1 : stage - 1;
    Frag x = x0;
    float s = s0;
#pragma unroll
    for (int h = 0; h + 1 < MG; ++h) {
      // the loads are spread over the row groups: a wave that issues them all at once waits for the
      // address unit, which takes 16 clocks for each and is shared by the CU
      if (h < SPREAD) issue(kt + kStages - 1, target, LOADS * h / SPREAD, LOADS * (h + 1) / SPREAD);
      const Frag xn = read_x(st, h + 1);
      const float sn = read_s(st, h + 1);
      products(partial, x, s * sb, h, nullptr);
      x = xn;
      s = sn;
    }
    wait_vm<(kStages - 2) * LOADS>();
    block_barrier();
    x0 = read_x(next, 0);
    s0 = read_s(next, 0);
    const float sbn = read_sb(next);
    products(partial, x, s * sb, MG - 1, next);
    sb = sbn;
  };
  auto k_loop = [&](auto partial) __attribute__((always_inline)) {
    for (int kt = 0, stage = 0; kt < KT; ++kt) {
      step(partial, kt, stage);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s, s, 0, LOADS);
  if (tid < BM) s_slot[tid] = tid < rows ? slot_at(a, first + tid) : -1;
  wait_vm<0>();  // (the first steps: the slots' load stands behind them)
  block_barrier();
  const int live = live_groups<BM>(s_slot, lane);
  // The 16-row groups go to the WM wave rows in turn, so that they share a partly filled tile evenly: of
  // this wave's groups h (group h * WM + wm of the tile) the first lg are live.
  lg = (live - wm + WM - 1) / WM;
  if (live == 0) return;  // (uniform over the workgroup, and nothing is in flight)
#pragma unroll
  for (int g = 0; g < NG; ++g) wf[g] = read_w(smem, g);
  x0 = read_x(smem, 0);
  s0 = read_s(smem, 0);
  sb = read_sb(smem);
  if (lg >= MG) k_loop(std::false_type{});
  else k_loop(std::true_type{});
  if constexpr (T::kScaled) {
#pragma unroll
    for (int i = P - DIST; i < P; ++i) take(i, t[i % DIST], ts[i % DIST]);
  }
  wait_vm<0>();     // the loads past the end have landed and every wave has read its last operands:
  block_barrier();  // the stages are free for the epilogue

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
  typedef typename T::Out Out;
  const bool wide = ((uintptr_t)a.C & 15) == 0 && (a.ldc & 7) == 0;
  store_tiles<NG, MG, Out>(acc, lg, smem, w, lane, n0, a.N, wide, [&](int r) -> Out* {
    const int s = s_slot[((r >> 4) * WM + wm) * 16 + (r & 15)];
    return s >= 0 ? static_cast<Out*>(a.C) + (int64_t)s * a.ldc : nullptr;
  });
}

// A workgroup is alone on its CU (or one of two), so its start is not hidden: what says which rows it works
// on is asked for at once (entries behind the live blocks exist, so no load waits for the block count),
// and the first steps' operands before the tile's rows are counted.  (two waves a SIMD: one workgroup of
// eight waves a CU, or two of four.)
//
// With kMerge a tile of BM rows is made of several blocks of an expert, and an expert's last tile of 64 rows
// and more that holds no more than half of them runs in the shape of half the rows with a stage more: a step
// of a half filled tile costs nearly what a full one's does.
template <typename T, int MG, int NG, int WM, int WN, int kStages, bool kMerge>
__global__ __launch_bounds__(64 * WM * WN, 2) void block_gemm_tile_kernel(BlockGemmArgs a) {
  constexpr int BM = 16 * MG * WM, BN = 16 * NG * WN;
  __shared__ __attribute__((aligned(128))) uint8_t smem[tile_bytes<T, MG, NG, WM, WN, kStages, kMerge>()];
  __shared__ int s_slot[BM];
  const int flags = T::kScaled ? 0 : drop_flags(a, blockIdx.x);
  auto work = [&]() __attribute__((always_inline)) {
    const int strips = (a.N + BN - 1) / BN, subs = (a.block_m + BM - 1) / BM;
    int mb, strip;
    unit_tile(blockIdx.x, strips, a.group_m, a.group_n, mb, strip);
    if (mb >= a.tiles || strip >= strips) return;
    if constexpr (kMerge) {
      const int nb = min(*a.ntpp / a.block_m, a.cap_blocks), per = BM / a.block_m;
      if (mb * per >= nb + min(a.E, nb) * (per - 1)) return;  // (more tiles than these blocks can make)
      int b = 0, e = 0;
      const int rows = merged_tile(a, nb, BM, mb, &b, &e);
      if (rows == 0) return;
      const int64_t first = (int64_t)b * a.block_m;
      if constexpr (MG >= 4) {
        if (rows <= BM / 2) return gemm_tile<T, MG / 2, NG, WM, WN, kStages + 1>(a, smem, s_slot, first, rows, e, strip);
      }
      gemm_tile<T, MG, NG, WM, WN, kStages>(a, smem, s_slot, first, rows, e, strip);
    } else {
      const int b = mb / subs, sub = mb - b * subs;
      int e = 0;
      if (a.sorted) {
        const int nb = *a.ntpp / a.block_m;
        e = a.eids[b];
        if (b >= nb || e < 0 || e >= a.E) return;
      }
      gemm_tile<T, MG, NG, WM, WN, kStages>(a, smem, s_slot, (int64_t)b * a.block_m + sub * BM,
                                            min(a.block_m - sub * BM, BM), e, strip);
    }
  };
  work();
  if constexpr (!T::kScaled) zero_dropped<typename T::Out>(a, flags);
}

// Most tiles of BM rows that the blocks can make (an expert's last tile may hold fewer blocks).
static int64_t merged_tiles(const BlockGemmArgs& a, int64_t cap_blocks, int BM) {
  const int64_t per = BM / a.block_m, experts = std::min<int64_t>(a.E, a.numel);
  return std::min(cap_blocks, (cap_blocks + experts * (per - 1)) / per);
}

template <typename T, int MG, int NG, int WM, int WN, int kStages, bool kMerge = false>
static int launch_tile(const char* fn, BlockGemmArgs a, int64_t cap_blocks, hipStream_t st) {
  constexpr int BM = 16 * MG * WM, BN = 16 * NG * WN;
  a.cap_blocks = (int32_t)cap_blocks;
  const int64_t tiles = kMerge ? merged_tiles(a, cap_blocks, BM) : cap_blocks * ((a.block_m + BM - 1) / BM);
  const int64_t grid = choose_units(tiles, (a.N + BN - 1) / BN, &a.group_m, &a.group_n);
  a.tiles = (int32_t)tiles;
  MOE_REQUIRE(launchable(grid, 64 * WM * WN), MOE_EUNSUPPORTED, "%s: grid too large", fn);  // (tiles <= grid)
  hipLaunchKernelGGL((block_gemm_tile_kernel<T, MG, NG, WM, WN, kStages, kMerge>), dim3((unsigned)grid),
                     dim3(64 * WM * WN), 0, st, a);
  return check_launch(fn);
}

// The kernel for a call.  Blocks of at most 16 rows stream their weights (block_gemm_stream_kernel).  For
// the others the tile shape with the least rounds of resident workgroups (half way between the whole
// number and the fraction: later ones start as earlier ones end) x time of one, for KT steps of 128 bytes
// of K (fitted to dense e4m3fn products of 8 to 56 steps; bf16's have the same proportions):
//   256 x 256, one a CU    10.4 + 1.68 KT us        128 x 128, two a CU   5.7 + 1.18 KT us
//   128 x 256, one a CU     6.4 + 1.07 KT us         64 x 64, two a CU    2.8 + 0.51 KT us
//    64 x 256, one a CU     3.6 + 0.90 KT us
// and 4 us more for finding the tile's expert and rows.  (Dense products fit 0.70 KT for 64 x 256; 0.90 picks
// better among routed ones.)  The rows of routed experts are taken as spread evenly, each expert ending
// half way through a tile.  Over 253 drawn calls of all three products the shape chosen takes 4 % more than
// the best of the five on average, 14 % at nine in ten: experts' sizes are not known here.  256-row tiles are
// made of an expert's 128-row blocks, counted in the kernel (2 us more), where the batch has 128 slots an
// expert (1024 Zipf tokens of 8 choices on 32 of 256 experts: 618 us with 128 rows, 604 with 256; 4096 of
// them 975 and 908).
// Blocks of 17 to 32 rows run the 64-row shapes with half the rows, weighed by the 64-row ones' figures, counts and
// residency (not fitted apart: up to twice as many tiles run, and LDS would hold three and two a CU).  K is split
// over waves up to 16 rows only, so 17 to some 500 dense rows along a long K leave CUs idle (N = 4096, K = 7168: 16
// rows 13 us, 17 to 256 21 - 27, 512 43).
template <typename T>
static int launch_block_gemm(const char* fn, const BlockGemmArgs& a, int64_t cap_blocks, hipStream_t st) {
  const int64_t cus = device_cu_count(), KT = (a.Kb + kStepBytes - 1) / kStepBytes;
  constexpr int64_t kMaxMerged = 4096;  // blocks that every workgroup counts through, 64 at a time
  // 16-row blocks from 12 slots an expert, when experts have more than one often enough, and enough experts for
  // every CU: two blocks in a 32-row tile, weights through LDS as whole cache lines.  With most rows live the
  // streamed form's loads, 16 rows an instruction, are what takes the time, unless K is long (16 slots each on
  // 128 experts, N = K = 2880: 245 and 221 us; on 64, N = 1024, K = 2048: 35 and 24; on 32, N = 8192, K = 4096: 209
  // and 223 us, and with 2 live slots each where 16 were expected 149 and 206).  The rows gradient takes 365 us
  // for the first of these, in blocks one by one 405.
  if (a.block_m == 16 && a.sorted && cap_blocks <= kMaxMerged && a.expected >= 12ll * a.E &&
      (int64_t)a.E * ((a.N + 127) / 128) >= cus && (T::kTrans || KT < 28))
    return launch_tile<T, 2, 2, 1, 4, 3, true>(fn, a, cap_blocks, st);
  if constexpr (!T::kTrans) {
    if (a.block_m <= 16) {
      // One tile a workgroup where two would leave CUs without one, with eight waves along a long K (a dense row,
      // N = 4096: K = 7168 two tiles and four waves 11.3, one and four 11.4, one and eight 9.7 us; K = 512 3.8,
      // 3.4, 5.0 us), and for bf16 rows of 6 KB and more while experts have one block (20 slots on 8 experts,
      // N = K = 4096: 52, 56, 44 us; e4m3 ones of 7 KB, 32 slots on 32 experts, 115 and 129 us for the first and
      // the last).  Else two tiles and four waves, and from four slots an expert four tiles, which read the rows of
      // A half as often, and two blocks of an expert together where it has them (K = 4096, N = 8192, 32 experts,
      // 2, 4, 8 slots each: 162, 181, 197 and 163, 182, 189 us; Zipf, 8 slots: 211 and 188 us).
      const int64_t n = (int64_t)((a.N + 31) / 32) * (a.sorted ? std::min<int64_t>(cap_blocks, a.expected) : cap_blocks);
      if (n < cus ? KT >= 24 : !T::kScaled && KT >= 48 && a.expected < 12ll * a.E)
        return launch_stream<T, 1, 8, 1>(fn, a, cap_blocks, st);
      if (n < cus) return launch_stream<T, 1, 4, 1>(fn, a, cap_blocks, st);
      if (a.sorted && a.expected >= 4ll * a.E) return launch_stream<T, 4, 4, 2>(fn, a, cap_blocks, st);
      return launch_stream<T, 2, 4, 1>(fn, a, cap_blocks, st);
    }
  }
  const bool merge = a.sorted && a.block_m == 128 && cap_blocks <= kMaxMerged && a.expected >= 128ll * a.E;
  auto cost = [&](int BM, int BN, int per_cu, double fixed, double step) {
    const int64_t tiles = a.sorted ? std::min(cap_blocks * ((a.block_m + BM - 1) / BM),
                                              a.expected / BM + (std::min<int64_t>(a.E, a.expected) + 1) / 2)
                                   : ((int64_t)a.numel + BM - 1) / BM;
    const int64_t n = tiles * ((a.N + BN - 1) / BN);
    const double exact = std::max(1.0, (double)n / (double)(cus * per_cu));
    const double whole = (double)((n + cus * per_cu - 1) / (cus * per_cu));
    return (exact + whole) / 2 * (fixed + (a.sorted ? 4.0 : 0.0) + step * (double)KT);
  };
  const double small = cost(64, 64, 2, 2.8, 0.51), flat = cost(64, 256, 1, 3.6, 0.90);
  if (a.block_m <= 32) {  // (at most 32 rows: the 64-row tiles' shapes with half the rows)
    if (small < flat) return launch_tile<T, 2, 1, 1, 4, 4>(fn, a, cap_blocks, st);
    return launch_tile<T, 2, 4, 1, 4, 2>(fn, a, cap_blocks, st);
  }
  const double never = 1e30;
  const bool rows128 = a.block_m > 64, rows256 = merge || !a.sorted || a.block_m == 256;
  const double low = rows128 ? cost(128, 128, 2, 5.7, 1.18) : never;
  const double mid = rows128 ? cost(128, 256, 1, 6.4, 1.07) : never;
  const double big = rows256 ? cost(256, 256, 1, merge ? 12.4 : 10.4, 1.68) : never;
  const double best = std::min({small, flat, low, mid, big});
  if (big == best) {
    if (merge) return launch_tile<T, 8, 4, 2, 4, 2, true>(fn, a, cap_blocks, st);
    return launch_tile<T, 8, 4, 2, 4, 2>(fn, a, cap_blocks, st);
  }
  if (mid == best) return launch_tile<T, 4, 4, 2, 4, 3>(fn, a, cap_blocks, st);
  if (low == best) return launch_tile<T, 4, 4, 2, 2, 2>(fn, a, cap_blocks, st);
  if (flat == best) return launch_tile<T, 2, 4, 2, 4, 3>(fn, a, cap_blocks, st);
  return launch_tile<T, 2, 2, 2, 2, 4>(fn, a, cap_blocks, st);
}

// Checks shared by the products over the align's blocks (A and W of T::kBytes a value).
template <typename T>
static int check_block_gemm(const char* fn, const void* A, int64_t a_rows, int64_t lda, const void* W, int32_t E,
                            int32_t N, int32_t K, const uint16_t* bias, const void* C, int64_t ldc, int64_t numel,
                            int32_t top_k, int32_t block_m) {
  constexpr int kStep = 16 / T::kBytes;
  MOE_REQUIRE(E >= 1 && N >= 1 && K >= 1, MOE_EINVAL, "%s: E=%d N=%d K=%d", fn, E, N, K);
  MOE_REQUIRE(E <= 512, MOE_EUNSUPPORTED, "%s: %d experts (at most 512)", fn, E);
  MOE_REQUIRE(N % 8 == 0 && K % kStep == 0 && N <= (1 << 20) && K <= (1 << 20), MOE_EUNSUPPORTED,
              "%s: N=%d must be a multiple of 8 and K=%d of %d (both at most 2^20)", fn, N, K, kStep);
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
