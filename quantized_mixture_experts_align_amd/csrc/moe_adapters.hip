// moe_adapters_add: low-rank adapters of many requests beside a shared projection,
//     out[m] = base[m] + scale[a] * B_a (A_a x[m / top_k])      (a the adapter of row m)
// over the align blocks of the rows' adapters.
//
// Two launches, or for few rows and short K one.  The first makes t = A_a x in fp32 (K split over waves, and over workgroups
// where there are few rows), the second adds B_a t to the rows.  Between them t is not rounded to bf16: the matrix core gets it as
// two bf16 halves, hi + lo, side by side along its K of 32 (16 ranks each), so the product of both costs no more
// than a rank padded to 32 would.
//
// Bound: memory -- x is read once, base read and out written once, the adapters' rows once where rows are few.  8179 rows,
// most of them with one of 6 adapters of rank 64, K = N = 4096: 22 us (83 MB fetched, 4.0 TB/s) and 35 us (91 MB fetched, 67
// written, 4.5 TB/s); 57 rows of as many adapters of rank 16, K 4096, N 8192: 5.4 and 7.5 us; one row of K 7168, N 4096
// in one launch 8.2 (loads that wait for each other, and what one CU takes in).
//
// An infinity in B meets the lower halves too, 0 or of either sign: its column may be NaN where the sum is infinite.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "moe_internal.h"

namespace moe {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;

constexpr int kAdMaxRank = 256;
constexpr int kAdRankTile = 64;    // ranks of a workgroup of the first launch
constexpr int kAdMaxSplits = 32;
constexpr int kAdMaxAdapters = 512;
// Workgroups that the two launches are split up to (8179 rows of rank 64 and 4096 columns: 256, 512, 768 of the first 32,
// 24.5, 28 us; 512, 768, 1024, 1536 of the second 37, 40, 41, 45 us).
constexpr int kAdGroups = 512, kAdStrips = 512;
constexpr int kFewGroups = 256;  // of the one launch: one a CU, which its registers fill

struct AdapterArgs {
  const uint16_t* x;
  int64_t ldx;
  const uint16_t *A, *B;
  const float* scales;
  const int32_t* ranks;
  int32_t L, r, N, K;
  const uint16_t* base;
  int64_t ldb;
  uint16_t* out;
  int64_t ldo;
  const int32_t *sorted, *adapters, *padded, *local;
  int64_t numel;
  int32_t top_k, block_m, per, splits;  // per: row tiles of an align block
  int64_t row_blocks;
  float* t;  // [splits][numel][r]
  bool over_x;  // out may hold rows of x
};

__device__ __forceinline__ int adapter_rank(const AdapterArgs& a, int ad) {
  return a.ranks ? min(max(a.ranks[ad], 0), a.r) : a.r;
}
// A row tile: its adapter (-1: nothing to do), the sorted position of its first row, its rows.  All of what it needs is
// asked for at once; what stands behind the live blocks is looked at, never used.
struct RowTile {
  int adapter;
  int64_t at;
  int n;
};
__device__ __forceinline__ RowTile row_tile(const AdapterArgs& a, int tile, int rows) {
  const int b = tile / a.per, sub = tile - b * a.per;
  RowTile w;
  w.at = (int64_t)b * a.block_m + sub * rows;
  w.n = min(rows, a.block_m - sub * rows);
  const int ad = a.adapters[b], end = *a.padded;
  w.adapter = (int64_t)b * a.block_m < end && ad < a.L ? ad : -1;
  return w;
}
// The slot of the tile's row i, -1 for padding.
__device__ __forceinline__ int slot_of(const AdapterArgs& a, const RowTile& w, int i) {
  const int s = a.sorted[w.at + min(i, w.n - 1)];
  return i < w.n && s >= 0 && s < a.numel ? s : -1;
}
// Orders a wave's own LDS accesses (the hardware keeps them in order, the compiler has to).
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// t[split][m][j] = sum over the split's k of A[a, j, k] x[m / top_k, k].  MT x RT tiles of 16 rows x 16 ranks.  A
// wave takes 64 k of every row (a line) at a time, the four waves' turns lie side by side and their sums meet in LDS.
//
// Operands pass through a place in LDS of the wave's own, so that the main loop has no barrier: eight adjacent lanes load
// a line of one row (straight to the operand's registers adjacent lanes lie in different rows, and a load takes 64 address
// cycles in the place of 16), piece p of row i stands at p ^ (i & 7).  The next UN turns' loads are in flight while
// these are multiplied (two such sets took no less time, and beside 64 sums they spill).
template <int MT, int RT, int UN>
__global__ __launch_bounds__(256, 2) void adapters_inner_kernel(AdapterArgs a) {
  constexpr int ROWS = 16 * (MT + RT), LOADS = ROWS / 8;  // staged rows of a turn, loads of 8 rows
  constexpr int STAGE = 4 * UN * ROWS * 128, RED = 3 * MT * RT * 1024;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
  __shared__ __attribute__((aligned(128))) uint8_t smem[STAGE > RED ? STAGE : RED];
  const int tile = blockIdx.x / a.splits, split = blockIdx.x - tile * a.splits;
  const RowTile w = row_tile(a, tile, 16 * MT);
  int row_slot[2 * MT], slot[MT];
#pragma unroll
  for (int q = 0; q < 2 * MT; ++q) row_slot[q] = slot_of(a, w, q * 8 + (lane >> 3));
#pragma unroll
  for (int m = 0; m < MT; ++m) slot[m] = slot_of(a, w, m * 16 + l16);
  if (w.adapter < 0) return;
  const int rank = adapter_rank(a, w.adapter), r0 = (int)blockIdx.y * kAdRankTile, piece = lane & 7;
  if (r0 >= rank && r0 > 0) return;
  const uint16_t* xp[2 * MT];
#pragma unroll
  for (int q = 0; q < 2 * MT; ++q)  // (a padding entry's product is not stored)
    xp[q] = a.x + (int64_t)(max(row_slot[q], 0) / a.top_k) * a.ldx;
  // (rows of A behind the adapter's own rank are read as they are: the second launch takes none of their sums)
  const uint16_t* Aa = a.A + (int64_t)w.adapter * a.r * a.K;
  uint32_t ar[2 * RT];
#pragma unroll
  for (int q = 0; q < 2 * RT; ++q) {
    const int j = r0 + q * 8 + (lane >> 3);
    ar[q] = (uint32_t)(j < a.r ? j : 0) * (uint32_t)a.K;
  }
  const int turns = (a.K + 255) >> 8;  // of the four waves
  const int lo = (int)((int64_t)turns * split / a.splits), hi = (int)((int64_t)turns * (split + 1) / a.splits);
  u32x4_t v[UN][LOADS];
  auto load = [&](int turn) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      const int k = (turn + u) * 256 + wv * 64 + piece * 8;
      const uint32_t kk = k < a.K ? k : 0;  // (no branch around a load: what lies behind K is read elsewhere)
#pragma unroll
      for (int q = 0; q < 2 * MT; ++q) v[u][q] = *reinterpret_cast<const u32x4_t*>(xp[q] + kk);
#pragma unroll
      for (int q = 0; q < 2 * RT; ++q) v[u][2 * MT + q] = *reinterpret_cast<const u32x4_t*>(Aa + ar[q] + kk);
    }
  };
  f32x4_t acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint8_t* stage = smem + wv * (UN * ROWS * 128);
  uint8_t* mine = stage + (lane >> 3) * 128 + (piece ^ (lane >> 3)) * 16;
  load(lo);
  for (int turn = lo; turn < hi; turn += UN) {
#pragma unroll
    for (int u = 0; u < UN; ++u) {
      // what lies behind K or the split is 0 in both operands (masked here: at the load it would be waited for there)
      const int t = turn + u;
      if (t >= hi || t * 256 + 256 > a.K) {
        const uint32_t keep = t < hi && t * 256 + wv * 64 + piece * 8 < a.K ? ~0u : 0u;
#pragma unroll
        for (int q = 0; q < LOADS; ++q) v[u][q] = v[u][q] & keep;
      }
#pragma unroll
      for (int q = 0; q < LOADS; ++q) *reinterpret_cast<u32x4_t*>(mine + (u * ROWS + q * 8) * 128) = v[u][q];
    }
    if (turn + UN < hi) load(turn + UN);
    wave_lds_fence();
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* at = stage + u * ROWS * 128 + l16 * 128 + ((4 * h + g) ^ (l16 & 7)) * 16;
        bf16x8_t xf[MT];
#pragma unroll
        for (int m = 0; m < MT; ++m) xf[m] = *reinterpret_cast<const bf16x8_t*>(at + m * 2048);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const bf16x8_t af = *reinterpret_cast<const bf16x8_t*>(at + (MT + j) * 2048);
#pragma unroll
          for (int m = 0; m < MT; ++m) acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af, xf[m], acc[m][j], 0, 0, 0);
        }
      }
    wave_lds_fence();
  }
  __syncthreads();
  f32x4_t* red = reinterpret_cast<f32x4_t*>(smem);
  if (wv > 0)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < RT; ++j) red[((wv - 1) * MT * RT + m * RT + j) * 64 + lane] = acc[m][j];
  __syncthreads();
  if (wv > 0) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (slot[m] < 0) continue;
    float* row = a.t + ((int64_t)split * a.numel + slot[m]) * a.r + r0;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const f32x4_t* o = red + (m * RT + j) * 64 + lane;
      const f32x4_t t = (acc[m][j] + o[0]) + (o[MT * RT * 64] + o[2 * MT * RT * 64]);
      const int c = j * 16 + g * 4;
      if (r0 + c < a.r) *reinterpret_cast<f32x4_t*>(row + c) = t;
    }
  }
}

// Rows of no adapter: out = base.
__device__ __forceinline__ void copy_rows(const AdapterArgs& a, int64_t first, int64_t step) {
  const int chunks = a.N >> 3;
  for (int64_t m = first; m < a.numel; m += step) {
    if (a.local[m] >= 0 && a.local[m] < a.L) continue;
    for (int c = threadIdx.x & 63; c < chunks; c += 64)
      *reinterpret_cast<u32x4_t*>(a.out + m * a.ldo + c * 8) = *reinterpret_cast<const u32x4_t*>(a.base + m * a.ldb + c * 8);
  }
}

// Columns of out for a row tile: base + B t, t in LDS as the matrix core takes it: for each 16 rows and 16 ranks, lane groups 0
// and 1 the upper halves of ranks 0..7 and 8..15, groups 2 and 3 the lower ones.  A wave makes 64 columns at a time.  Their
// columns of B (64 r values in a row, or 64 ranks of each at a time) and the sums pass through places in LDS of the wave's
// own, so that all loads and stores are of whole lines by adjacent lanes; the next columns' are in flight while these are made.
// FR: 16-rank parts of t (r <= 16 FR).
template <int MT, int FR>
struct Columns {
  static constexpr int RT = FR < 4 ? FR : 4;     // 16-rank parts that are staged at a time
  static constexpr int NL = 2 * RT;              // loads of them
  static constexpr bool LINES = RT == 4;         // staged rows of eight pieces (8 ranks each), piece p of row i at p ^ (i & 7);
                                                 // else of r / 8, as they lie in memory
  static constexpr int PITCH = 68;               // values between staged rows of sums
  static constexpr int FRAG = MT * FR * 1024, BS = 64 * RT * 32, SUMS = 16 * PITCH * 4, OWN = BS > SUMS ? BS : SUMS;
  const AdapterArgs& a;
  const uint16_t* Ba;    // the adapter's B
  const uint16_t* frag;  // [MT][parts][64][8]
  uint8_t* bs;           // the wave's own OWN bytes
  int lane, rank;
  int slot[MT][2];  // of the rows that this lane loads and stores
  u32x4_t base[MT][2], bv[NL];

  // (No branches around loads, and none of them left out: columns behind N are read again and not stored.  The waits count
  // what is in flight, and would else count on none of it.)
  __device__ __forceinline__ void load_base(int n0, int m, int h) {
    base[m][h] = *reinterpret_cast<const u32x4_t*>(a.base + (int64_t)max(slot[m][h], 0) * a.ldb +
                                                   min((uint32_t)(n0 + (lane & 7) * 8), (uint32_t)a.N - 8));
  }
  __device__ __forceinline__ void load_b(int n0, int c0) {
    const uint32_t last_b = (uint32_t)a.N * (uint32_t)a.r - 8;
#pragma unroll
    for (int q = 0; q < NL; ++q) {
      const uint32_t i = q * 64 + lane;  // piece of the staged ones
      uint32_t at;
      if constexpr (LINES) {
        const uint32_t row = i >> 3, j = c0 * 16 + ((i & 7) ^ (row & 7)) * 8;
        at = min((uint32_t)n0 + row, (uint32_t)a.N - 1) * (uint32_t)a.r + (j < (uint32_t)a.r ? j : 0);
      } else {
        at = min((uint32_t)n0 * (uint32_t)a.r + i * 8, last_b);
      }
      bv[q] = *reinterpret_cast<const u32x4_t*>(Ba + at);
    }
  }
  __device__ __forceinline__ void load(int n0) {
    load_b(n0, 0);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int h = 0; h < 2; ++h) load_base(n0, m, h);
  }
  // The columns n0, n0 + step, ..., of which the first have been asked for.
  __device__ __forceinline__ void add(int n0, int step) {
    const int l16 = lane & 15, g = lane >> 4, col = (lane & 7) * 8, pieces = a.r / 8, RK = (rank + 15) >> 4;
    float* sums = reinterpret_cast<float*>(bs);
    for (; n0 < a.N; n0 += step) {
      f32x4_t acc[MT][4];
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int u = 0; u < 4; ++u) acc[m][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
      for (int c0 = 0; c0 < (FR <= 4 ? 1 : RK); c0 += RT) {
        if (c0) load_b(n0, c0);
#pragma unroll
        for (int q = 0; q < NL; ++q)
          if (LINES || q * 64 + lane < 64 * pieces) *reinterpret_cast<u32x4_t*>(bs + (q * 64 + lane) * 16) = bv[q];
        if (FR <= 4 || c0 + RT >= RK) load_b(n0 + step, 0);
        wave_lds_fence();
#pragma unroll
        for (int c = 0; c < RT; ++c) {
          if (c0 + c >= RK) continue;
          const int pc = 2 * c + (g & 1), left = rank - (c0 + c) * 16 - (g & 1) * 8;
          uint32_t keep[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) keep[j] = 2 * j + 1 < left ? ~0u : (2 * j < left ? 0xFFFFu : 0u);
          bf16x8_t bf[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int row = u * 16 + l16, at = LINES ? row * 8 + (pc ^ (row & 7)) : row * pieces + min(pc, pieces - 1);
            const u32x4_t r = *reinterpret_cast<const u32x4_t*>(bs + at * 16);  // (values behind the adapter's own rank as 0)
            bf[u] = __builtin_bit_cast(bf16x8_t, u32x4_t{r[0] & keep[0], r[1] & keep[1], r[2] & keep[2], r[3] & keep[3]});
          }
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const bf16x8_t tv = *reinterpret_cast<const bf16x8_t*>(frag + ((int64_t)(m * RK + c0 + c) * 64 + lane) * 8);
#pragma unroll
            for (int u = 0; u < 4; ++u) acc[m][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[u], tv, acc[m][u], 0, 0, 0);
          }
        }
        wave_lds_fence();
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int u = 0; u < 4; ++u) *reinterpret_cast<f32x4_t*>(sums + l16 * PITCH + u * 16 + g * 4) = acc[m][u];
        wave_lds_fence();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float* o = sums + (h * 8 + (lane >> 3)) * PITCH + col;
          const f32x4_t p = *reinterpret_cast<const f32x4_t*>(o), q = *reinterpret_cast<const f32x4_t*>(o + 4);
          const u32x4_t b = base[m][h];
          // (past the L2, which keeps the operands: 62 -> 56 us for both launches on 8179 rows of 4096 columns)
          if (slot[m][h] >= 0 && n0 + col < a.N)
            __builtin_nontemporal_store(
                u32x4_t{pack_bf16x2(bf16_lo(b[0]) + p[0], bf16_hi(b[0]) + p[1]), pack_bf16x2(bf16_lo(b[1]) + p[2], bf16_hi(b[1]) + p[3]),
                        pack_bf16x2(bf16_lo(b[2]) + q[0], bf16_hi(b[2]) + q[1]), pack_bf16x2(bf16_lo(b[3]) + q[2], bf16_hi(b[3]) + q[3])},
                reinterpret_cast<u32x4_t*>(a.out + (int64_t)slot[m][h] * a.ldo + n0 + col));
          load_base(n0 + step, m, h);
        }
        wave_lds_fence();
      }
    }
  }
};
// Two values of t, scaled, and their lower halves.
__device__ __forceinline__ void halves(float p, float q, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16x2(p, q);
  const float dp = p - bf16_lo(hi), dq = q - bf16_hi(hi);  // (an infinity has no lower half)
  lo = pack_bf16x2(fabsf(dp) < INFINITY ? dp : 0.0f, fabsf(dq) < INFINITY ? dq : 0.0f);
}

// out[m, n] = base[m, n] + sum_j B[a, n, j] scale[a] t[m, j].
template <int MT, int FR>
__global__ __launch_bounds__(256, 2) void adapters_outer_kernel(AdapterArgs a, int strips) {
  using Cols = Columns<MT, FR>;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  __shared__ __attribute__((aligned(128))) uint8_t smem[Cols::FRAG + 4 * Cols::OWN];
  const int first = (int)a.row_blocks * strips;
  if ((int)blockIdx.x >= first) {
    copy_rows(a, (int64_t)(blockIdx.x - first) * 4 + wv, (int64_t)(gridDim.x - first) * 4);
    return;
  }
  const int tile_row = blockIdx.x / strips, strip = blockIdx.x - tile_row * strips;
  uint16_t* frag = reinterpret_cast<uint16_t*>(smem);
  const RowTile w = row_tile(a, tile_row, 16 * MT);
  int slot[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) slot[m][h] = slot_of(a, w, m * 16 + h * 8 + (lane >> 3));
  if (w.adapter < 0) return;
  const int rank = adapter_rank(a, w.adapter), RK = (rank + 15) >> 4;
  const float scale = a.scales ? a.scales[w.adapter] : 1.0f;
  Cols cols{a, a.B + (int64_t)w.adapter * a.N * a.r, frag, smem + Cols::FRAG + wv * Cols::OWN, lane, rank};
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int h = 0; h < 2; ++h) cols.slot[m][h] = slot[m][h];
  const int n0 = (strip * 4 + wv) * 64;
  cols.load(n0);
  // t: eight ranks of a row for each P adjacent threads, which share the splits
  const int items = MT * RK * 32;
  int P = 1;
  while (P * 2 * items <= 256 && P < a.splits) P *= 2;
  const int part = threadIdx.x & (P - 1);
  for (int i = threadIdx.x / P; i < items; i += 256 / P) {
    const int l = i & 15, half = (i >> 4) & 1, tile = i >> 5, m = tile / RK, c = tile - m * RK;
    const int s = slot_of(a, w, m * 16 + l), j0 = c * 16 + half * 8;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    if (s >= 0 && j0 < rank) {
      const float* q = a.t + (int64_t)s * a.r + j0;
#pragma unroll 4
      for (int p = part; p < a.splits; p += P) {
        const float4 x = *reinterpret_cast<const float4*>(q + (int64_t)p * a.numel * a.r);
        const float4 y = *reinterpret_cast<const float4*>(q + (int64_t)p * a.numel * a.r + 4);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
    }
    for (int d = P / 2; d >= 1; d >>= 1)
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] += __shfl_xor(v[j], d);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      halves(j0 + 2 * j < rank ? v[2 * j] * scale : 0.0f, j0 + 2 * j + 1 < rank ? v[2 * j + 1] * scale : 0.0f, hi[j], lo[j]);
    uint16_t* d = frag + (int64_t)tile * 512 + (half * 16 + l) * 8;
    if (part == 0) *reinterpret_cast<u32x4_t*>(d) = u32x4_t{hi[0], hi[1], hi[2], hi[3]};
    if (part == P - 1) *reinterpret_cast<u32x4_t*>(d + 256) = u32x4_t{lo[0], lo[1], lo[2], lo[3]};
  }
  __syncthreads();
  cols.add(n0, strips * 256);
}

// Both products in one launch, for tiles of 16 rows and r <= 16 RT: every workgroup of a tile makes all of t for itself.  Its
// eight waves take 64 k of every row in turn, UN turns' loads in flight a wave, through the wave's own LDS as above.
constexpr int kFewWaves = 8;
template <int RT, int UN>
__global__ __launch_bounds__(kFewWaves * 64) void adapters_few_kernel(AdapterArgs a, int strips) {
  using Cols = Columns<1, RT>;
  constexpr int W = kFewWaves, ROWS = 16 * (1 + RT), LOADS = ROWS / 8;
  constexpr int STAGE = ROWS * 128, PLACE = STAGE > Cols::OWN ? STAGE : Cols::OWN;  // a wave's (the sums need RT * 1024)
  const int lane = threadIdx.x & 63, wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l16 = lane & 15, g = lane >> 4, piece = lane & 7;
  __shared__ __attribute__((aligned(128))) uint8_t smem[Cols::FRAG + W * PLACE];
  const int first = (int)a.row_blocks * strips;
  if ((int)blockIdx.x >= first) {
    copy_rows(a, (int64_t)(blockIdx.x - first) * W + wv, (int64_t)(gridDim.x - first) * W);
    return;
  }
  const int tile = blockIdx.x / strips, strip = blockIdx.x - tile * strips;
  const RowTile w = row_tile(a, tile, 16);
  const int slot[2] = {slot_of(a, w, lane >> 3), slot_of(a, w, 8 + (lane >> 3))};
  if (w.adapter < 0) return;
  const int rank = adapter_rank(a, w.adapter);
  const float scale = a.scales ? a.scales[w.adapter] : 1.0f;
  uint16_t* frag = reinterpret_cast<uint16_t*>(smem);
  uint8_t* place = smem + Cols::FRAG + wv * PLACE;
  Cols cols{a, a.B + (int64_t)w.adapter * a.N * a.r, frag, place, lane, rank, {{slot[0], slot[1]}}};
  const int n0 = (strip * W + wv) * 64;
  cols.load(n0);
  const uint16_t* from[LOADS];  // (a padding entry's product is not stored, nor what stands behind the adapter's own rank used)
#pragma unroll
  for (int q = 0; q < 2; ++q) from[q] = a.x + (int64_t)(max(slot[q], 0) / a.top_k) * a.ldx;
#pragma unroll
  for (int q = 0; q < 2 * RT; ++q) {
    const int j = q * 8 + (lane >> 3);
    from[2 + q] = a.A + (int64_t)w.adapter * a.r * a.K + (uint32_t)(j < a.r ? j : 0) * (uint32_t)a.K;
  }
  f32x4_t acc[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  uint8_t* mine = place + (lane >> 3) * 128 + (piece ^ (lane >> 3)) * 16;
  const int turns = (a.K + 63) >> 6;
  // (X: loads of rows of x.  A tile of 8 rows or fewer leaves the second out: half of what a single row's tile would load were copies of it.)
  auto product = [&](auto x_loads) __attribute__((always_inline)) {
    constexpr int X = decltype(x_loads)::value;
    u32x4_t v[UN][LOADS];
    auto load = [&](int turn, int u) __attribute__((always_inline)) {
      const int k = turn * 64 + piece * 8;
      const uint32_t kk = k < a.K ? k : 0;  // (what lies behind K is read elsewhere; its product is masked)
#pragma unroll
      for (int q = 0; q < LOADS; ++q)
        if (q < X || q >= 2) v[u][q] = *reinterpret_cast<const u32x4_t*>(from[q] + kk);
    };
    auto multiply = [&](int turn, int u) __attribute__((always_inline)) {
      const uint32_t keep = turn * 64 + piece * 8 < a.K ? ~0u : 0u;
#pragma unroll
      for (int q = 0; q < LOADS; ++q)
        if (q < X || q >= 2) *reinterpret_cast<u32x4_t*>(mine + q * 1024) = v[u][q] & keep;
      wave_lds_fence();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint8_t* at = place + l16 * 128 + ((4 * h + g) ^ (l16 & 7)) * 16;
        const bf16x8_t xf = *reinterpret_cast<const bf16x8_t*>(at);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const bf16x8_t af = *reinterpret_cast<const bf16x8_t*>(at + (1 + j) * 2048);
          acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af, xf, acc[j], 0, 0, 0);
        }
      }
      wave_lds_fence();
    };
    int turn = wv;
    for (; turn + (UN - 1) * W < turns; turn += UN * W) {
#pragma unroll
      for (int u = 0; u < UN; ++u) load(turn + u * W, u);
#pragma unroll
      for (int u = 0; u < UN; ++u) multiply(turn + u * W, u);
    }
#pragma unroll
    for (int u = 0; u < UN - 1; ++u)
      if (turn + u * W < turns) load(turn + u * W, u);
#pragma unroll
    for (int u = 0; u < UN - 1; ++u)
      if (turn + u * W < turns) multiply(turn + u * W, u);
  };
  if (__any(slot[1] >= 0)) product(std::integral_constant<int, 2>{});
  else product(std::integral_constant<int, 1>{});
  __syncthreads();
  f32x4_t* red = reinterpret_cast<f32x4_t*>(smem + Cols::FRAG);
#pragma unroll
  for (int j = 0; j < RT; ++j) red[(wv * RT + j) * 64 + lane] = acc[j];
  __syncthreads();
  // ranks 4 g .. 4 g + 3 of a part for a row, each to its place among the halves
  if (wv < RT) {
    f32x4_t t = red[wv * 64 + lane];
#pragma unroll
    for (int i = 1; i < W; ++i) t += red[(i * RT + wv) * 64 + lane];
    const int c = wv * 16 + g * 4;
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      halves(c + 2 * j < rank ? t[2 * j] * scale : 0.0f, c + 2 * j + 1 < rank ? t[2 * j + 1] * scale : 0.0f, hi[j], lo[j]);
    uint16_t* d = frag + wv * 512 + ((g >> 1) * 16 + l16) * 8 + (g & 1) * 4;
    *reinterpret_cast<uint2*>(d) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(d + 256) = make_uint2(lo[0], lo[1]);
  }
  __syncthreads();
  cols.add(n0, strips * W * 64);
}

// Rows of a workgroup's tile, row tiles of the batch (at most), and splits of K: about 512 workgroups, each with a turn
// of its four waves (256 k) or more.
static int adapter_rows(int block_m) { return block_m <= 16 ? 16 : block_m <= 32 ? 32 : 64; }
static int64_t adapter_row_blocks(int64_t numel, int L, int block_m, int* per) {
  const int64_t rows = numel + std::min<int64_t>(L, numel) * (block_m - 1);
  *per = (block_m + adapter_rows(block_m) - 1) / adapter_rows(block_m);
  return (rows + block_m - 1) / block_m * *per;
}
static int adapter_splits(int64_t row_blocks, int r, int K) {
  const int64_t groups = std::max<int64_t>(1, row_blocks * ((r + kAdRankTile - 1) / kAdRankTile));
  const int64_t by_k = (K + 255) / 256;
  return (int)std::max<int64_t>(1, std::min<int64_t>({kAdGroups / groups, by_k, kAdMaxSplits}));
}

// Whether matrices of rows may share memory: their spans meet, and they are not different columns of the same rows.
static bool rows_meet(const uint16_t* p, int64_t rows, int64_t ld, int32_t cols, const uint16_t* q, int64_t rows_q, int64_t ld_q,
                      int32_t cols_q) {
  const uintptr_t p0 = (uintptr_t)p, p1 = p0 + ((rows - 1) * ld + cols) * 2, q0 = (uintptr_t)q,
                  q1 = q0 + ((rows_q - 1) * ld_q + cols_q) * 2;
  if (p1 <= q0 || q1 <= p0) return false;
  if (ld != ld_q) return true;
  const uintptr_t row = (uintptr_t)ld * 2, d = (p0 <= q0 ? q0 - p0 : row - (p0 - q0) % row) % row;  // q's columns behind p's
  return !(d >= (uintptr_t)cols * 2 && d + (uintptr_t)cols_q * 2 <= row);
}

static int adapter_sizes(const char* fn, int64_t numel, int32_t L, int32_t r, int32_t N, int32_t K, int32_t block_m) {
  MOE_REQUIRE(numel >= 0 && L >= 1 && r >= 1 && N >= 1 && K >= 1 && block_m >= 1 && block_m <= 256, MOE_EINVAL,
              "%s: numel=%lld L=%d r=%d N=%d K=%d block_m=%d", fn, (long long)numel, L, r, N, K, block_m);
  MOE_REQUIRE(r % 8 == 0 && r <= kAdMaxRank && N % 8 == 0 && K % 8 == 0, MOE_EUNSUPPORTED,
              "%s: r=%d (at most %d), N=%d and K=%d must be multiples of 8", fn, r, kAdMaxRank, N, K);
  MOE_REQUIRE((int64_t)std::max(N, K) * r < (1ll << 30), MOE_EUNSUPPORTED, "%s: N=%d K=%d r=%d: an adapter of 2^30 values or more",
              fn, N, K, r);
  MOE_REQUIRE(L <= kAdMaxAdapters, MOE_EUNSUPPORTED, "%s: %d adapters (at most %d)", fn, L, kAdMaxAdapters);
  MOE_REQUIRE(numel < (1ll << 31) - 256 * kAdMaxAdapters, MOE_EUNSUPPORTED, "%s: numel=%lld too large", fn, (long long)numel);
  return MOE_OK;
}

template <int MT, int RT, int FR, int UN>
static void launch_adapters(const AdapterArgs& a, int64_t copies, hipStream_t st) {
  // (splits and strips of a row tile side by side: what runs at once then takes whole rows.  One slice of every row at a
  // time, 1 KB in 8, left most memory channels idle)
  const dim3 gi((unsigned)(a.row_blocks * a.splits), (unsigned)((a.r + kAdRankTile - 1) / kAdRankTile));
  hipLaunchKernelGGL((adapters_inner_kernel<MT, RT, UN>), gi, dim3(256), 0, st, a);
  const int64_t strips = std::max<int64_t>(1, std::min<int64_t>((a.N + 255) / 256, (kAdStrips + a.row_blocks - 1) / a.row_blocks));
  hipLaunchKernelGGL((adapters_outer_kernel<MT, FR>), dim3((unsigned)(a.row_blocks * strips + copies)), dim3(256), 0, st, a,
                     (int)strips);
}
// Where one launch is right, and the better.  Right: a workgroup that stores its columns must not store over x, which the tile's
// other workgroups may still be reading (two launches are done with x before the first store).  Better: the workgroups
// of a row tile each make all of its t, at some 110 GB/s, so few tiles and short rows of A.  Against two launches, replayed from a
// graph, N 4096, one row of rank 16: K 512 4.2 us against 6.7, 2048 5.3 and 7.1, 4096 6.5 and 7.4, 6144 7.7 and 7.8, 7168 8.2 and 8.0, 8184 8.6 and
// 7.2, 14336 12.3 and 7.2; of rank 32: 2048 6.7 and 7.9, 4096 8.4 and 7.9, 8184 12.0 and 8.5.  16 rows of 8 adapters, rank 16: 4096 6.6 and 7.5;
// rank 32: 2048 6.8 and 8.0, 4096 9.8 and 8.1.  64 of 64, K 512: rank 16 5.1 and 8.1, rank 32 8.4 and 10.8; 256 of 256: 11.0 and 14.5, 15.7
// and 18.8.  A call that is not captured saves the second launch's 3 us of host time besides, and for a single tile the bound goes by
// that: replays would change to two launches at K 6144 (rank 32: between 2048 and 4096).
static bool few_rows(const AdapterArgs& a) {
  const int64_t values = (int64_t)(a.r <= 16 ? 16 : 32) * a.K;
  return !a.over_x && a.r <= 32 && (a.row_blocks == 1 ? values < (1 << 17) : a.row_blocks <= 16 ? values <= (1 << 16) : a.K <= 512);
}
template <int RT, int UN>
static void launch_few(const AdapterArgs& a, int64_t copies, hipStream_t st) {
  constexpr int COLS = kFewWaves * 64;
  const int64_t strips = std::max<int64_t>(1, std::min<int64_t>((a.N + COLS - 1) / COLS, (kFewGroups + a.row_blocks - 1) / a.row_blocks));
  hipLaunchKernelGGL((adapters_few_kernel<RT, UN>), dim3((unsigned)(a.row_blocks * strips + copies)), dim3(kFewWaves * 64), 0, st, a,
                     (int)strips);
}
template <int MT>
static void launch_adapters(const AdapterArgs& a, int64_t copies, hipStream_t st) {
  if (MT == 1 && few_rows(a)) {
    if (a.r <= 16) launch_few<1, 8>(a, copies, st);
    else launch_few<2, 6>(a, copies, st);
    return;
  }
  constexpr int UN = MT == 1 ? 2 : 1;
  if (a.r <= 16) launch_adapters<MT, 1, 1, UN>(a, copies, st);
  else if (a.r <= 32) launch_adapters<MT, 2, 2, UN>(a, copies, st);
  else if (a.r <= 64) launch_adapters<MT, 4, 4, UN>(a, copies, st);
  else launch_adapters<MT, 4, 16, UN>(a, copies, st);
}

}  // namespace moe

using namespace moe;

extern "C" int moe_adapters_workspace(int64_t numel, int32_t L, int32_t r, int32_t K, int32_t block_m, int64_t* elems) {
  MOE_REQUIRE(elems, MOE_EINVAL, "moe_adapters_workspace: null pointer");
  const int rc = adapter_sizes("moe_adapters_workspace", numel, L, r, 8, K, block_m);
  if (rc) return rc;
  int per;
  const int64_t blocks = adapter_row_blocks(numel, L, block_m, &per);
  *elems = adapter_splits(blocks, r, K) * numel * r;
  return ok();
}

extern "C" int moe_adapters_add(const uint16_t* base, int64_t ld_base, const uint16_t* x, int64_t x_rows, int64_t ld_x,
                                const uint16_t* A, const uint16_t* B, const float* scales, const int32_t* ranks,
                                int32_t L, int32_t r, int32_t N, int32_t K, uint16_t* out, int64_t ld_out,
                                const int32_t* sorted_token_ids, const int32_t* adapter_ids,
                                const int32_t* num_tokens_post_padded, const int32_t* slot_local_ids, int64_t numel,
                                int32_t top_k, int32_t block_m, float* work, int64_t work_elems, hipStream_t stream) {
  const int rc = adapter_sizes("moe_adapters_add", numel, L, r, N, K, block_m);
  if (rc) return rc;
  MOE_REQUIRE(top_k >= 1 && x_rows >= 0 && x_rows * top_k >= numel, MOE_EINVAL,
              "moe_adapters_add: %lld rows of x, top_k=%d, for %lld slots", (long long)x_rows, top_k, (long long)numel);
  MOE_REQUIRE(ld_x >= K && ld_base >= N && ld_out >= N, MOE_EINVAL, "moe_adapters_add: leading dimensions %lld, %lld, %lld",
              (long long)ld_x, (long long)ld_base, (long long)ld_out);
  MOE_REQUIRE(ld_x % 8 == 0 && ld_base % 8 == 0 && ld_out % 8 == 0, MOE_EUNSUPPORTED,
              "moe_adapters_add: leading dimensions %lld, %lld, %lld must be multiples of 8", (long long)ld_x,
              (long long)ld_base, (long long)ld_out);
  if (numel == 0) return ok();
  const bool in_place = out == base;
  MOE_REQUIRE(base && x && A && B && out && sorted_token_ids && adapter_ids && num_tokens_post_padded && work, MOE_EINVAL,
              "moe_adapters_add: null pointer");
  MOE_REQUIRE(in_place || slot_local_ids, MOE_EINVAL, "moe_adapters_add: slot_local_ids is needed unless out is base");
  if (in_place) {
    MOE_REQUIRE(ld_out == ld_base, MOE_EINVAL, "moe_adapters_add: out is base with another leading dimension");
  } else {
    MOE_REQUIRE(!rows_meet(out, numel, ld_out, N, base, numel, ld_base, N), MOE_EINVAL, "moe_adapters_add: out overlaps base");
  }
  MOE_REQUIRE((((uintptr_t)base | (uintptr_t)x | (uintptr_t)A | (uintptr_t)B | (uintptr_t)out | (uintptr_t)work) & 15) == 0 &&
                  (((uintptr_t)scales | (uintptr_t)ranks | (uintptr_t)sorted_token_ids | (uintptr_t)adapter_ids |
                    (uintptr_t)num_tokens_post_padded | (uintptr_t)slot_local_ids) & 3) == 0,
              MOE_EUNSUPPORTED, "moe_adapters_add: bf16 tensors and the workspace must be 16-byte aligned, the others 4");
  AdapterArgs a{x, ld_x, A, B, scales, ranks, L, r, N, K, base, ld_base, out, ld_out, sorted_token_ids, adapter_ids,
                num_tokens_post_padded, slot_local_ids, numel, top_k, block_m, 1, 1, 0, work,
                rows_meet(out, numel, ld_out, N, x, (numel + top_k - 1) / top_k, ld_x, K)};
  a.row_blocks = adapter_row_blocks(numel, L, block_m, &a.per);
  a.splits = adapter_splits(a.row_blocks, r, K);
  MOE_REQUIRE(work_elems >= a.splits * numel * r, MOE_ESIZE, "moe_adapters_add: workspace of %lld values, need %lld",
              (long long)work_elems, (long long)(a.splits * numel * r));
  MOE_REQUIRE(a.row_blocks < (1ll << 22) / ((r + kAdRankTile - 1) / kAdRankTile), MOE_EUNSUPPORTED,
              "moe_adapters_add: %lld row tiles", (long long)a.row_blocks);
  const int64_t copies = in_place ? 0 : std::min<int64_t>((numel + 3) / 4, 512);
  const int rows = adapter_rows(block_m);
  if (rows == 16) launch_adapters<1>(a, copies, stream);
  else if (rows == 32) launch_adapters<2>(a, copies, stream);
  else launch_adapters<4>(a, copies, stream);
  return check_launch("moe_adapters_add");
}
