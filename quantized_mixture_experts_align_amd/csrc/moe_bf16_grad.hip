// Gradients of moe_bf16_gemm, C[s, n] = sum_k A[s / top_k, k] W[e(s), n, k] + bias[e(s), n]:
//   moe_bf16_gemm_dgrad   dA[r, k] = sum over the live slots s of row r, sum_n dC[s, n] W[e(s), n, k]
//   moe_bf16_gemm_wgrad   dW[e, n, k] = sum over the slots s of e of dC[s, n] A[s / top_k, k]
//                         dbias[e, n] = sum over the slots s of e of dC[s, n]
// Both products reduce over an index whose values are rows in memory (n of W; the slots of dC and
// A), while an MFMA operand wants eight consecutive values of it in one lane: the tiles are staged
// in LDS as they lie in memory and read transposed (moe_block_gemm.h, which also holds the kernel of
// the first one: the product with the weights as the transposed operand).
//
// Sums run in fp32 in a fixed order (no atomics).
#include <algorithm>

#include "moe_block_gemm.h"

namespace moe {

struct GradArgs {
  const uint16_t* dC;
  int64_t ld_dc;
  const uint16_t* A;
  int64_t lda;
  void* dW;            // [E, N, K], or null: only dbias, from one strip of columns whose product is not stored
  void* dbias;         // [E, N] or null
  const int32_t* sorted;
  const int32_t* eids;
  const int32_t* ntpp;
  int32_t numel, top_k, block_m, N, K, E;
  int32_t cap_blocks;  // most blocks the align can have made
  int32_t group_m, group_n, positions;
  uint32_t div_mul, div_shift;  // s / top_k for 0 <= s < 2^31 (top_k > 1)
  __device__ __forceinline__ uint32_t row_of(uint32_t s) const {
    return top_k == 1 ? s : __umulhi(s, div_mul) >> div_shift;
  }
};

constexpr int kMaxExperts = 512;

// dW[e, n, k] of BM = 16 * MG * WM rows n x BN = 16 * NG * WN columns k, reduced over the expert's slots in
// steps of 64: the slots' rows of dC (BM columns of each) and of A (BN columns) go through LDS as they lie
// in memory, two steps deep, and both operands are read transposed.  Wave (wm, wn) owns MG 16-row
// groups of n and NG 16-column tiles of k.
//
// An expert has few steps (8 at 512 slots), so a workgroup stays for many tiles and asks for the next one's
// first rows before it stores what it has (32 experts, 11646 slots, N = K = 4096: 553 -> 533 us).  That
// product needs 283 us of the matrix cores at the rate of a large library product and writes 1.1 GB, 210 us.
// Of a tile's 17 us on average 6.2 steps take 12.8, the stores 2.9, the rest 1.4; where no cache holds the
// operands yet (a GB of other data read in front) steps and stores take 14.5 and 4.3.
//
// The rows are gathered, so a step's loads need its slots' numbers: these come by direct loads two steps
// ahead, those of a tile's first two steps while the tile in front of it runs.  An expert's slots fill its
// blocks from the front, so its steps end with the first that begins with padding, and only the last one
// can lack rows; they are zero in both operands.
template <typename OUT, int MG, int NG, int WM, int WN>
__global__ __launch_bounds__(64 * WM * WN, 2) void wgrad_kernel(GradArgs a) {
  constexpr int WAVES = WM * WN, BM = 16 * MG * WM, BN = 16 * NG * WN, ROWS = 64;
  constexpr int PC = BM * 2, PX = BN * 2;                       // bytes of a staged row of dC and of A
  constexpr int CI = ROWS * PC / 1024 / WAVES, XI = ROWS * PX / 1024 / WAVES;  // loads per wave and step
  constexpr int RC = 1024 / PC, RX = 1024 / PX;                 // rows that a load brings
  static_assert(CI * 1024 * WAVES == ROWS * PC && XI * 1024 * WAVES == ROWS * PX, "the waves share the rows evenly");
  constexpr int CB = ROWS * PC, STAGE = CB + ROWS * PX;
  constexpr int OWN = MG / WN;                                  // row groups of dbias that a wave sums
  static_assert(OWN * WN == MG, "the waves share the row groups evenly");
  __shared__ __attribute__((aligned(128))) uint8_t smem[2 * STAGE];
  __shared__ __attribute__((aligned(16))) uint8_t s_out[WAVES * 16 * (32 * NG + 16)];
  __shared__ __attribute__((aligned(16))) int s_ids[2][2][ROWS];  // of a tile (in turn) and step (in turn)
  __shared__ int s_begin[kMaxExperts + 1];                        // blocks of the experts in front of e
  const uint32_t smem_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem;
  const uint32_t ids_lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) int*)&s_ids[0][0][0];
  const int tid = threadIdx.x, w = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int wm = w / WN, wn = w % WN;
  const int ks = a.dW ? (a.K + BN - 1) / BN : 1, ns = (a.N + BM - 1) / BM;
  const uint8_t* zero = reinterpret_cast<const uint8_t*>(&g_zero16);

  // The align lists the experts' blocks in rising order, so the counts of their blocks give their ranges.
  const int nb = min(*a.ntpp / a.block_m, a.cap_blocks);
  for (int i = tid; i <= a.E; i += 64 * WAVES) s_begin[i] = 0;
  __syncthreads();
  for (int i = tid; i < nb; i += 64 * WAVES) {
    const int e = a.eids[i];
    if (e >= 0 && e < a.E) atomicAdd(&s_begin[e + 1], 1);
  }
  __syncthreads();
  if (w == 0) {
    int sum = 0;
    for (int i = 0; i <= a.E; i += 64) {
      int v = i + lane <= a.E ? s_begin[i + lane] : 0;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int below = __shfl_up(v, d);
        v += lane >= d ? below : 0;
      }
      v += sum;
      if (i + lane <= a.E) s_begin[i + lane] = v;
      sum = __shfl(v, 63);
    }
  }
  __syncthreads();

  struct Tile {
    int e, n0, k0, rows;  // rows: entries of the expert, with the padding
    int64_t first;
  };
  auto find = [&](int& at, Tile& t) __attribute__((always_inline)) {  // the first tile from position `at` on
    for (; at < a.positions; at += gridDim.x) {
      int en, kt0;
      unit_tile(at, ks, a.group_m, a.group_n, en, kt0);
      if (kt0 >= ks || en >= ns * a.E) continue;
      t.e = en / ns;
      t.n0 = (en - t.e * ns) * BM;
      t.k0 = kt0 * BN;
      const int begin = __builtin_amdgcn_readfirstlane(s_begin[t.e]);
      t.first = (int64_t)begin * a.block_m;
      t.rows = (__builtin_amdgcn_readfirstlane(s_begin[t.e + 1]) - begin) * a.block_m;
      return true;
    }
    return false;
  };
  // the slot numbers of a tile's step kt (behind the last entry the last one again), loaded by one wave
  auto issue_ids = [&](const Tile& t, int kt, int turn) __attribute__((always_inline)) {
    if (t.rows == 0) return;
    const int64_t at = t.first + min(kt * ROWS + lane, t.rows - 1);
    dma_from<4>(reinterpret_cast<const uint8_t*>(a.sorted + at), ids_lds + (uint32_t)(turn * 2 + (kt & 1)) * ROWS * 4);
  };
  auto exists = [&](const Tile& t, int kt, int turn) __attribute__((always_inline)) {
    if (kt * ROWS >= t.rows) return false;
    return (uint32_t)__builtin_amdgcn_readfirstlane(s_ids[turn][kt & 1][0]) < (uint32_t)a.numel;
  };
  // byte offsets in a row (a column behind the edge reads the tile's first, not stored)
  uint32_t ccol[CI], xcol[XI];
  auto crow = [&](int l) __attribute__((always_inline)) { return (w * CI + l) * RC + lane / (64 / RC); };
  auto xrow = [&](int l) __attribute__((always_inline)) { return (w * XI + l) * RX + lane / (64 / RX); };
  auto columns = [&](const Tile& t) __attribute__((always_inline)) {
#pragma unroll
    for (int l = 0; l < CI; ++l) {
      const int place = lane % (64 / RC);
      const int col = t.n0 + ((place >> 1) ^ trans_swizzle(crow(l), PC)) * 16 + (place & 1) * 8;
      ccol[l] = 2u * (uint32_t)(col < a.N ? col : t.n0);
    }
#pragma unroll
    for (int l = 0; l < XI; ++l) {
      const int place = lane % (64 / RX);
      const int col = t.k0 + ((place >> 1) ^ trans_swizzle(xrow(l), PX)) * 16 + (place & 1) * 8;
      xcol[l] = 2u * (uint32_t)(col < a.K ? col : t.k0);
    }
  };
  auto issue = [&](const Tile& t, int kt, int turn, int stage, int from, int to) __attribute__((always_inline)) {
    const uint32_t st = smem_lds + (uint32_t)(stage * STAGE);
    const int* ids = s_ids[turn][kt & 1];
    const int left = t.rows - kt * ROWS;
#pragma unroll
    for (int l = 0; l < CI + XI; ++l) {
      if (l < from || l >= to) continue;
      const int r = l < CI ? crow(l) : xrow(l - CI);
      const uint32_t id = (uint32_t)ids[r];
      const bool in = r < left && id < (uint32_t)a.numel;
      const uint32_t s = in ? id : 0u;
      const uint8_t* p;
      if (l < CI) p = reinterpret_cast<const uint8_t*>(a.dC) + (int64_t)s * (a.ld_dc * 2) + ccol[l];
      else p = reinterpret_cast<const uint8_t*>(a.A) + (int64_t)a.row_of(s) * (a.lda * 2) + xcol[l - CI];
      dma_from<16>(in ? p : zero,
                   st + (l < CI ? (uint32_t)(w * CI + l) * 1024 : CB + (uint32_t)(w * XI + l - CI) * 1024));
    }
  };

  int coff[MG], xoff[NG];
#pragma unroll
  for (int h = 0; h < MG; ++h) coff[h] = trans_lane(wm * MG + h, PC, lane);
#pragma unroll
  for (int g = 0; g < NG; ++g) xoff[g] = trans_lane(wn * NG + g, PX, lane);
  auto read_x = [&](const uint8_t* st, int sub, int g) __attribute__((always_inline)) {
    return trans_operand(st + CB + sub * 32 * PX, xoff[g], PX);
  };
  auto read_c = [&](const uint8_t* st, int sub, int h) __attribute__((always_inline)) {
    return trans_operand(st + sub * 32 * PC, coff[h], PC);
  };

  int at = blockIdx.x, turn = 0;
  Tile t;
  if (!find(at, t)) return;
  if (w < 2) issue_ids(t, w, 0);
  wait_vm<0>();
  block_barrier();
  bool more = exists(t, 0, 0);
  columns(t);
  if (more) issue(t, 0, 0, 0, 0, CI + XI);
  wait_vm<0>();
  block_barrier();
  for (;;) {
    Tile after;
    at += gridDim.x;
    const bool last = !find(at, after);
    if (!last && w < 2) issue_ids(after, w, turn ^ 1);
    f32x4_t acc[NG][MG];
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < MG; ++h) acc[g][h] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // dbias is the same reduction with ones in the place of A: the first tile of columns takes it along, the
    // WN waves of the same rows MG / WN row groups each.
    const bool ones = a.dbias && t.k0 == 0;
    f32x4_t accb[OWN];
#pragma unroll
    for (int i = 0; i < OWN; ++i) accb[i] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const u32x4_t one = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
    if (more) {
      u32x4_t xf[2][NG], cf[2];
#pragma unroll
      for (int sub = 0; sub < 2; ++sub) {
#pragma unroll
        for (int g = 0; g < NG; ++g) xf[sub][g] = read_x(smem, sub, g);
        cf[sub] = read_c(smem, sub, 0);
      }
      for (int kt = 0; more; ++kt) {
        const uint8_t* st = smem + (kt & 1) * STAGE;
        const uint8_t* next = smem + (~kt & 1) * STAGE;
        more = exists(t, kt + 1, turn);
#pragma unroll
        for (int h = 0; h < MG; ++h) {
          u32x4_t cn[2];
          if (h + 1 < MG) {
            if (h < 2 && more)
              issue(t, kt + 1, turn, ~kt & 1, (CI + XI) * h / 2, (CI + XI) * (h + 1) / 2);
            if (h == 1 && more && w == 0) issue_ids(t, kt + 2, turn);
            cn[0] = read_c(st, 0, h + 1);
            cn[1] = read_c(st, 1, h + 1);
          } else {  // the next step's operands are read behind the last group's products (not used after the last step)
            wait_vm<0>();
            block_barrier();
            cn[0] = read_c(next, 0, 0);
            cn[1] = read_c(next, 1, 0);
          }
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              acc[g][h] = mfma(xf[sub][g], cf[sub], acc[g][h]);
              if (h + 1 == MG) xf[sub][g] = read_x(next, sub, g);
            }
          if (ones && h / OWN == wn) {
            accb[h % OWN] = mfma(one, cf[0], accb[h % OWN]);
            accb[h % OWN] = mfma(one, cf[1], accb[h % OWN]);
          }
          __builtin_amdgcn_sched_barrier(0);
          cf[0] = cn[0];
          cf[1] = cn[1];
        }
      }
    } else {
      wait_vm<0>();
      block_barrier();
    }
    // Every wave has passed the last step's barrier: its stage is free, and the other holds nothing.
    if (!last) {
      more = exists(after, 0, turn ^ 1);
      columns(after);
      if (more) issue(after, 0, turn ^ 1, 0, 0, CI + XI);
    }
    if (ones && lane < 16) {  // (every row of the product is the sum; lane l < 16 holds row 0 of column l)
#pragma unroll
      for (int i = 0; i < OWN; ++i) {
        const int n = t.n0 + (wm * MG + wn * OWN + i) * 16 + lane;
        if (n >= a.N) continue;
        const int64_t to = (int64_t)t.e * a.N + n;
        if constexpr (sizeof(OUT) == 4) static_cast<float*>(a.dbias)[to] = accb[i][0];
        else static_cast<uint16_t*>(a.dbias)[to] = f32_to_bf16(accb[i][0]);
      }
    }
    store_tiles<NG, MG, OUT>(acc, MG, s_out, w, lane, t.k0 + wn * 16 * NG, a.K, true, [&](int r) -> OUT* {
      const int n = t.n0 + wm * 16 * MG + r;
      return n < a.N && a.dW ? static_cast<OUT*>(a.dW) + ((int64_t)t.e * a.N + n) * a.K : nullptr;
    });
    if (last) break;
    wait_vm<0>();
    block_barrier();
    t = after;
    turn ^= 1;
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

template <typename OUT, int MG, int NG, int WM, int WN>
static int launch_wgrad_tile(const char* fn, GradArgs a, int per_cu, hipStream_t st) {
  constexpr int BM = 16 * MG * WM, BN = 16 * NG * WN;
  const int64_t tiles = (int64_t)((a.N + BM - 1) / BM) * a.E, strips = a.dW ? (a.K + BN - 1) / BN : 1;
  const int64_t positions = choose_units(tiles, strips, &a.group_m, &a.group_n);
  MOE_REQUIRE(positions < (1ll << 30), MOE_EUNSUPPORTED, "%s: grid too large", fn);
  a.positions = (int32_t)positions;
  const int64_t grid = std::min<int64_t>(positions, (device_cu_count() * per_cu + kXcds - 1) / kXcds * kXcds);
  hipLaunchKernelGGL((wgrad_kernel<OUT, MG, NG, WM, WN>), dim3((unsigned)grid), dim3(64 * WM * WN), 0, st, a);
  return check_launch(fn);
}

// 256 x 256 tiles, or 128 x 128 where these leave CUs without work (8192 slots on 8 experts, N = K = 4096: 303
// and 382 us; 4608 slots on 8 experts, N = 2048: K = 1024, 256 of the larger tiles, 29 and 36 us, K = 512, 128 of
// them, 27 and 20 us).
template <typename OUT>
static int launch_wgrad(const char* fn, const GradArgs& a, hipStream_t st) {
  if ((int64_t)((a.N + 255) / 256) * (a.dW ? (a.K + 255) / 256 : 1) * a.E >= device_cu_count())
    return launch_wgrad_tile<OUT, 8, 4, 2, 4>(fn, a, 1, st);
  return launch_wgrad_tile<OUT, 4, 2, 2, 4>(fn, a, 2, st);
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

extern "C" int moe_bf16_gemm_dgrad(const uint16_t* dC, int64_t ld_dc, const uint16_t* W, int32_t E, int32_t N,
                                   int32_t K, uint16_t* dA, int64_t ld_da, const int32_t* sorted_token_ids,
                                   const int32_t* expert_ids, const int32_t* num_tokens_post_padded,
                                   const int32_t* slot_local_ids, int64_t numel, int32_t top_k, int32_t block_m,
                                   int64_t expected_slots, float* work, int64_t work_elems, hipStream_t stream) {
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
  MOE_REQUIRE(top_k == 1 || launchable(numel / top_k, 256), MOE_EUNSUPPORTED, "%s: grid too large", fn);
  int64_t cap = 0, cap_blocks = 0;
  rc = moe_align_capacity(numel, 1, E, block_m, &cap, &cap_blocks);
  if (rc) return rc;
  const BlockGemmArgs a{reinterpret_cast<const uint8_t*>(dC), ld_dc * 2, reinterpret_cast<const uint8_t*>(W), nullptr,
                        0, nullptr, nullptr, top_k == 1 ? static_cast<void*>(dA) : work,
                        top_k == 1 ? ld_da : (int64_t)K, sorted_token_ids, expert_ids, num_tokens_post_padded,
                        (int32_t)numel, 1, block_m, K, N * 2, E, 0, 0, 0, 0, top_k == 1 ? slot_local_ids : nullptr,
                        expected_slots > 0 ? std::min(expected_slots, numel) : numel};
  rc = top_k == 1 ? launch_block_gemm<Bf16TransType<uint16_t>>(fn, a, cap_blocks, stream)
                  : launch_block_gemm<Bf16TransType<float>>(fn, a, cap_blocks, stream);
  if (rc || top_k == 1) return rc;  // (rows of dropped slots are zeroed by the same launch)
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
  // The bias alone: one strip of columns, with dC in the place of A too (the bias's sums are the same).  The backward
  // pass of 32 experts, 11666 slots, N = K = 4096 takes 79 us, 610 with the weights' gradient.
  if (!dW) {
    A = dC;
    a_rows = numel;
    lda = ld_dc;
    K = N;
    top_k = 1;
  }
  MOE_REQUIRE(a_rows >= numel / top_k, MOE_EINVAL, "%s: A has %lld rows, slots need %lld", fn, (long long)a_rows,
              (long long)(numel / top_k));
  MOE_REQUIRE(lda >= K && lda % 8 == 0, MOE_EINVAL, "%s: lda=%lld (>= K=%d, multiple of 8)", fn, (long long)lda, K);
  MOE_REQUIRE((dW || dbias) && num_tokens_post_padded && (numel == 0 || (A && sorted_token_ids && expert_ids)),
              MOE_EINVAL, "%s: null pointer", fn);
  MOE_REQUIRE((((uintptr_t)A | (uintptr_t)dW) & 15) == 0 && ((uintptr_t)dbias & 3) == 0, MOE_EUNSUPPORTED,
              "%s: misaligned pointer (A and dW 16 B, dbias 4 B)", fn);
  int64_t cap = 0, cap_blocks = 0;
  rc = moe_align_capacity(numel, 1, E, block_m, &cap, &cap_blocks);
  if (rc) return rc;
  GradArgs a{dC, ld_dc, A, lda, dW, dbias, sorted_token_ids, expert_ids, num_tokens_post_padded, (int32_t)numel, top_k,
             block_m, N, K, E, (int32_t)cap_blocks, 0, 0, 0, 0, 0};
  if (top_k > 1) {  // ceil(2^(32 + shift) / top_k): exact for numerators below 2^31
    while ((2u << a.div_shift) < (uint32_t)top_k) ++a.div_shift;
    a.div_mul = (uint32_t)(((1ull << (32 + a.div_shift)) + top_k - 1) / (uint64_t)top_k);
  }
  return out_f32 ? launch_wgrad<float>(fn, a, stream) : launch_wgrad<uint16_t>(fn, a, stream);
}
