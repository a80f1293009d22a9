// moe_adapters_add: low-rank adapters of many requests beside a shared projection,
//     out[m] = base[m] + scale[a] * B_a (A_a x[m / top_k])      (a the adapter of row m)
// over the align blocks of the rows' adapters.
//
// Two launches.  The first makes t = A_a x in fp32 (K split over waves, and over workgroups where there are
// few rows), the second adds B_a t to the rows.  Between them t is not rounded to bf16: the matrix core gets it as
// two bf16 halves, hi + lo, side by side along its K of 32 (16 ranks each), so the product of both costs no more
// than a rank padded to 32 would.
//
// Bound: memory -- x is read once, base read and out written once, the adapters' rows once where rows are few.
#include <algorithm>
#include <cmath>

#include "moe_internal.h"

namespace moe {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;

constexpr int kAdMaxRank = 256;
constexpr int kAdRankTile = 64;    // ranks of a workgroup of the first launch
constexpr int kAdMaxSplits = 32;
constexpr int kAdMaxAdapters = 512;

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
};

__device__ __forceinline__ int adapter_rank(const AdapterArgs& a, int ad) {
  return a.ranks ? min(max(a.ranks[ad], 0), a.r) : a.r;
}
// The row tile's adapter (-1: nothing to do) and the sorted position of its first row; `n` rows of the block
// from there.
__device__ __forceinline__ int row_tile(const AdapterArgs& a, int tile, int rows, int64_t& at, int& n) {
  const int b = tile / a.per, sub = tile - b * a.per;
  at = (int64_t)b * a.block_m + sub * rows;
  n = min(rows, a.block_m - sub * rows);
  if ((int64_t)b * a.block_m >= *a.padded) return -1;
  const int ad = a.adapters[b];
  return ad < a.L ? ad : -1;
}
__device__ __forceinline__ uint4 zero4() { return make_uint4(0u, 0u, 0u, 0u); }

// t[split][m][j] = sum over the split's k of A[a, j, k] x[m / top_k, k].  MT x RT tiles of 16 rows x 16 ranks;
// the four waves take every fourth step of 32 k and their sums meet in LDS.
template <int MT, int RT>
__global__ __launch_bounds__(256) void adapters_inner_kernel(AdapterArgs a) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
  __shared__ f32x4_t red[3][MT * RT][64];
  int64_t at;
  int n;
  const int ad = row_tile(a, blockIdx.x, 16 * MT, at, n);
  if (ad < 0) return;
  const int rank = adapter_rank(a, ad), r0 = blockIdx.z * kAdRankTile;
  if (r0 >= rank && r0 > 0) return;
  const uint16_t* xr[MT];
  int slot[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = m * 16 + l16;
    const int s = i < n ? a.sorted[at + i] : -1;
    slot[m] = s >= 0 && s < a.numel ? s : -1;
    xr[m] = a.x + (int64_t)(max(slot[m], 0) / a.top_k) * a.ldx;  // (a padding entry's product is not stored)
  }
  const uint16_t* ar[RT];
  bool on[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int row = r0 + j * 16 + l16;
    on[j] = row < rank;
    ar[j] = a.A + ((int64_t)ad * a.r + (on[j] ? row : 0)) * a.K;
  }
  f32x4_t acc[MT][RT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[m][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int steps = (a.K + 31) >> 5;
  const int lo = (int)((int64_t)steps * blockIdx.y / a.splits), hi = (int)((int64_t)steps * (blockIdx.y + 1) / a.splits);
  for (int s = lo + wv; s < hi; s += 4) {
    const int k = s * 32 + g * 8;
    const bool in = k < a.K;
    uint4 xv[MT], av[RT];
#pragma unroll
    for (int m = 0; m < MT; ++m) xv[m] = in ? *reinterpret_cast<const uint4*>(xr[m] + k) : zero4();
#pragma unroll
    for (int j = 0; j < RT; ++j) av[j] = in && on[j] ? *reinterpret_cast<const uint4*>(ar[j] + k) : zero4();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < RT; ++j)
        acc[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, av[j]),
                                                            __builtin_bit_cast(bf16x8_t, xv[m]), acc[m][j], 0, 0, 0);
  }
  if (wv > 0)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int j = 0; j < RT; ++j) red[wv - 1][m * RT + j][lane] = acc[m][j];
  __syncthreads();
  if (wv > 0) return;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (slot[m] < 0) continue;
    float* row = a.t + ((int64_t)blockIdx.y * a.numel + slot[m]) * a.r + r0;
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const f32x4_t v = (acc[m][j] + red[0][m * RT + j][lane]) + (red[1][m * RT + j][lane] + red[2][m * RT + j][lane]);
      const int c = j * 16 + g * 4;
      if (r0 + c < a.r) *reinterpret_cast<f32x4_t*>(row + c) = v;
    }
  }
}

// Rows of no adapter: out = base.
__device__ __forceinline__ void copy_rows(const AdapterArgs& a, int64_t first, int64_t step) {
  const int chunks = a.N >> 3;
  for (int64_t m = first; m < a.numel; m += step) {
    if (a.local[m] >= 0 && a.local[m] < a.L) continue;
    for (int c = threadIdx.x & 63; c < chunks; c += 64)
      *reinterpret_cast<uint4*>(a.out + m * a.ldo + c * 8) = *reinterpret_cast<const uint4*>(a.base + m * a.ldb + c * 8);
  }
}

// out[m, n] = base[m, n] + sum_j B[a, n, j] scale[a] t[m, j].  The tile's t stands in LDS as the matrix core takes it:
// for each 16 rows and 16 ranks, lane groups 0 and 1 the upper halves of ranks 0..7 and 8..15, groups 2 and 3 the
// lower ones.  A wave makes 64 columns at a time; the 16 rows of B of tile u are n = 16 (i / 4) + 4 u + i % 4, so that a
// lane ends with 16 consecutive columns of one row.
template <int MT>
__global__ __launch_bounds__(256) void adapters_outer_kernel(AdapterArgs a) {
  extern __shared__ uint16_t frag[];  // [MT][r / 16][64][8]
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, l16 = lane & 15, g = lane >> 4;
  if ((int64_t)blockIdx.x >= a.row_blocks) {
    const int64_t b = (int64_t)(blockIdx.x - a.row_blocks) * gridDim.y + blockIdx.y;
    copy_rows(a, b * 4 + wv, (int64_t)(gridDim.x - a.row_blocks) * gridDim.y * 4);
    return;
  }
  int64_t at;
  int n;
  const int ad = row_tile(a, blockIdx.x, 16 * MT, at, n);
  if (ad < 0) return;
  const int rank = adapter_rank(a, ad), RK = (rank + 15) >> 4;
  const float scale = a.scales ? a.scales[ad] : 1.0f;
  for (int i = threadIdx.x; i < MT * RK * 32; i += 256) {  // eight ranks of one row
    const int l = i & 15, half = (i >> 4) & 1, tile = i >> 5, m = tile / RK, c = tile - m * RK;
    const int pos = m * 16 + l, s = pos < n ? a.sorted[at + pos] : -1, j0 = c * 16 + half * 8;
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
    if (s >= 0 && s < a.numel && j0 < a.r)
      for (int p = 0; p < a.splits; ++p) {
        const float4* q = reinterpret_cast<const float4*>(a.t + ((int64_t)p * a.numel + s) * a.r + j0);
        const float4 u = q[0], w = q[1];
        v[0] += u.x; v[1] += u.y; v[2] += u.z; v[3] += u.w;
        v[4] += w.x; v[5] += w.y; v[6] += w.z; v[7] += w.w;
      }
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float p = j0 + 2 * j < rank ? v[2 * j] * scale : 0.0f, q = j0 + 2 * j + 1 < rank ? v[2 * j + 1] * scale : 0.0f;
      hi[j] = pack_bf16x2(p, q);
      const float dp = p - bf16_lo(hi[j]), dq = q - bf16_hi(hi[j]);  // (an infinity has no lower half)
      lo[j] = pack_bf16x2(fabsf(dp) < INFINITY ? dp : 0.0f, fabsf(dq) < INFINITY ? dq : 0.0f);
    }
    uint16_t* d = frag + (int64_t)tile * 512 + (half * 16 + l) * 8;
    *reinterpret_cast<uint4*>(d) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(d + 256) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  __syncthreads();
  int slot[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int i = m * 16 + l16, s = i < n ? a.sorted[at + i] : -1;
    slot[m] = s >= 0 && s < a.numel ? s : -1;
  }
  const uint16_t* Ba = a.B + (int64_t)ad * a.N * a.r;
  for (int n0 = (blockIdx.y * 4 + wv) * 64; n0 < a.N; n0 += gridDim.y * 256) {
    f32x4_t acc[MT][4];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int u = 0; u < 4; ++u) acc[m][u] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < RK; ++c) {
      const int j0 = c * 16 + (g & 1) * 8;
      uint4 bv[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int col = n0 + 16 * (l16 >> 2) + 4 * u + (l16 & 3);
        bv[u] = zero4();
        if (col < a.N && j0 < rank) {
          bv[u] = *reinterpret_cast<const uint4*>(Ba + (int64_t)col * a.r + j0);
          const int left = rank - j0;  // (values behind the adapter's own rank are not used)
          if (left < 8) {
            uint32_t w[4] = {bv[u].x, bv[u].y, bv[u].z, bv[u].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = 2 * j + 1 < left ? w[j] : (2 * j < left ? w[j] & 0xFFFFu : 0u);
            bv[u] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const bf16x8_t tv = *reinterpret_cast<const bf16x8_t*>(frag + ((int64_t)(m * RK + c) * 64 + lane) * 8);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          acc[m][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, bv[u]), tv, acc[m][u], 0, 0, 0);
      }
    }
    const int col = n0 + 16 * g;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (slot[m] < 0) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (col + 8 * h >= a.N) continue;
        const uint4 b = *reinterpret_cast<const uint4*>(a.base + (int64_t)slot[m] * a.ldb + col + 8 * h);
        const f32x4_t p = acc[m][2 * h], q = acc[m][2 * h + 1];
        *reinterpret_cast<uint4*>(a.out + (int64_t)slot[m] * a.ldo + col + 8 * h) =
            make_uint4(pack_bf16x2(bf16_lo(b.x) + p[0], bf16_hi(b.x) + p[1]), pack_bf16x2(bf16_lo(b.y) + p[2], bf16_hi(b.y) + p[3]),
                       pack_bf16x2(bf16_lo(b.z) + q[0], bf16_hi(b.z) + q[1]), pack_bf16x2(bf16_lo(b.w) + q[2], bf16_hi(b.w) + q[3]));
      }
    }
  }
}

// Rows of a workgroup's tile, row tiles of the batch (at most), and splits of K: about 512 workgroups, each with eight
// steps of 32 k or more.
static int adapter_rows(int block_m) { return block_m <= 16 ? 16 : block_m <= 32 ? 32 : 64; }
static int64_t adapter_row_blocks(int64_t numel, int L, int block_m, int* per) {
  const int64_t blocks = (numel + std::min<int64_t>(L, numel) * (block_m - 1)) / block_m +
                         ((numel + std::min<int64_t>(L, numel) * (block_m - 1)) % block_m != 0);
  *per = (block_m + adapter_rows(block_m) - 1) / adapter_rows(block_m);
  return blocks * *per;
}
static int adapter_splits(int64_t row_blocks, int r, int K) {
  const int64_t groups = std::max<int64_t>(1, row_blocks * ((r + kAdRankTile - 1) / kAdRankTile));
  const int64_t by_k = std::max(1, (K + 31) / 32 / 8);
  return (int)std::max<int64_t>(1, std::min<int64_t>({512 / groups, by_k, kAdMaxSplits}));
}

static int adapter_sizes(const char* fn, int64_t numel, int32_t L, int32_t r, int32_t N, int32_t K, int32_t block_m) {
  MOE_REQUIRE(numel >= 0 && L >= 1 && r >= 1 && N >= 1 && K >= 1 && block_m >= 1 && block_m <= 256, MOE_EINVAL,
              "%s: numel=%lld L=%d r=%d N=%d K=%d block_m=%d", fn, (long long)numel, L, r, N, K, block_m);
  MOE_REQUIRE(r % 8 == 0 && r <= kAdMaxRank && N % 8 == 0 && K % 8 == 0, MOE_EUNSUPPORTED,
              "%s: r=%d (at most %d), N=%d and K=%d must be multiples of 8", fn, r, kAdMaxRank, N, K);
  MOE_REQUIRE(L <= kAdMaxAdapters, MOE_EUNSUPPORTED, "%s: %d adapters (at most %d)", fn, L, kAdMaxAdapters);
  MOE_REQUIRE(numel < (1ll << 31) - 256 * kAdMaxAdapters, MOE_EUNSUPPORTED, "%s: numel=%lld too large", fn, (long long)numel);
  return MOE_OK;
}

template <int MT>
static void launch_adapters(const AdapterArgs& a, int64_t copies, hipStream_t st) {
  const dim3 gi((unsigned)a.row_blocks, (unsigned)a.splits, (unsigned)((a.r + kAdRankTile - 1) / kAdRankTile));
  if (a.r <= 16) hipLaunchKernelGGL((adapters_inner_kernel<MT, 1>), gi, dim3(256), 0, st, a);
  else if (a.r <= 32) hipLaunchKernelGGL((adapters_inner_kernel<MT, 2>), gi, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((adapters_inner_kernel<MT, 4>), gi, dim3(256), 0, st, a);
  const int64_t strips = (a.N + 255) / 256;
  const int64_t y = std::max<int64_t>(1, std::min<int64_t>(strips, (1024 + a.row_blocks - 1) / a.row_blocks));
  hipLaunchKernelGGL((adapters_outer_kernel<MT>), dim3((unsigned)(a.row_blocks + copies), (unsigned)y), dim3(256),
                     (size_t)MT * ((a.r + 15) / 16) * 1024, st, a);
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
    const uintptr_t b0 = (uintptr_t)base, b1 = b0 + ((numel - 1) * ld_base + N) * 2, o0 = (uintptr_t)out,
                    o1 = o0 + ((numel - 1) * ld_out + N) * 2;
    MOE_REQUIRE(o1 <= b0 || b1 <= o0, MOE_EINVAL, "moe_adapters_add: out overlaps base");
  }
  MOE_REQUIRE((((uintptr_t)base | (uintptr_t)x | (uintptr_t)A | (uintptr_t)B | (uintptr_t)out | (uintptr_t)work) & 15) == 0 &&
                  (((uintptr_t)scales | (uintptr_t)ranks | (uintptr_t)sorted_token_ids | (uintptr_t)adapter_ids |
                    (uintptr_t)num_tokens_post_padded | (uintptr_t)slot_local_ids) & 3) == 0,
              MOE_EUNSUPPORTED, "moe_adapters_add: bf16 tensors and the workspace must be 16-byte aligned, the others 4");
  AdapterArgs a{x, ld_x, A, B, scales, ranks, L, r, N, K, base, ld_base, out, ld_out, sorted_token_ids, adapter_ids,
                num_tokens_post_padded, slot_local_ids, numel, top_k, block_m, 1, 1, 0, work};
  a.row_blocks = adapter_row_blocks(numel, L, block_m, &a.per);
  a.splits = adapter_splits(a.row_blocks, r, K);
  MOE_REQUIRE(work_elems >= a.splits * numel * r, MOE_ESIZE, "moe_adapters_add: workspace of %lld values, need %lld",
              (long long)work_elems, (long long)(a.splits * numel * r));
  MOE_REQUIRE(a.row_blocks < (1ll << 22) / ((r + kAdRankTile - 1) / kAdRankTile), MOE_EUNSUPPORTED,
              "moe_adapters_add: %lld row tiles", (long long)a.row_blocks);
  const int64_t copies = in_place ? 0 : std::min<int64_t>((numel + 3) / 4, 256);
  const int rows = adapter_rows(block_m);
  if (rows == 16) launch_adapters<1>(a, copies, stream);
  else if (rows == 32) launch_adapters<2>(a, copies, stream);
  else launch_adapters<4>(a, copies, stream);
  return check_launch("moe_adapters_add");
}
