// moe_combine_grad: gradients of the top-k weighted combine, without and with the post-expert RMSNorm.
//
//   out = c sum_s g_s y_s:      dy_s = c g_s dout,  dg_s = c <dout, y_s>
//   with a norm weight n:       z = y n,  r = (mean z^2 + eps)^-1/2,  out = c sum_s g_s r_s z_s,  d = <dout, z>
//       dg_s = c r d,   dz = c g r (dout - (r^2 d / H) z),   dy = dz n,   dn = sum over the live slots of dz y
// Dead slots: dy = 0, dg = 0, what their y holds is not used.  fp32 throughout, each result rounded once.
//
// Bound: memory (every live row of y is read once, every row of dy written once): 4096 tokens of 8 rows of 4096 columns
// with the norm take 96 us, 5.1 TB/s of operands, and 4.6 for dn; with one pass in LDS and a second read (the general
// kernel) 233 + 17.  2304 tokens of 2 rows of 512 take 4.3 us, mostly the launch.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "moe_internal.h"

namespace moe {

constexpr int kCgThreads = 256;
constexpr int kCgMaxTopK = 16;
constexpr int kCgParts = 512;      // workgroups that leave partial sums of dn, at most (4096 x 8 x 4096: 256 take 112 us in the
                                   // place of 96; 1024 no fewer, and dn 7.2 in the place of 4.6)
constexpr int kCgGrid = 1 << 20;    // workgroups at most (2^32 threads are a launch's limit); they stay for more tokens
constexpr int kCgMaxNormH = 12288; // columns of dn: 48 KB of LDS, so that three workgroups stand on a CU

struct CombineGradArgs {
  const uint16_t* y;
  const float* gw;
  const int32_t* local;
  const uint16_t* nw;
  float eps, rsf;
  int64_t M;
  int32_t k, H;
  const uint16_t* dout;
  int64_t ldd;
  uint16_t* dy;
  float* dg;
  float* part;  // [workgroups][H], or NULL
};

__device__ __forceinline__ void unpack8(const uint4& r, float (&v)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_lo(w[j]);
    v[2 * j + 1] = bf16_hi(w[j]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// A workgroup a token (or, with partial sums of dn, every gridDim.x-th one): the slots' sums first, then
// the rows of dy, for which y and dout are read again.  The general form, for top_k > 8 and rows beyond 8192 columns.
template <bool NORM>
__global__ __launch_bounds__(kCgThreads) void combine_grad_kernel(CombineGradArgs a) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int chunks = a.H >> 3;
  extern __shared__ float dn[];  // [H] (with partial sums)
  __shared__ float red[kCgThreads / 64][2 * kCgMaxTopK];
  __shared__ float f0[kCgMaxTopK], f1[kCgMaxTopK];
  if (a.part)
    for (int c = tid; c < chunks; c += kCgThreads)  // (a thread's own columns throughout)
#pragma unroll
      for (int j = 0; j < 8; ++j) dn[c * 8 + j] = 0.0f;
  for (int64_t t = blockIdx.x; t < a.M; t += gridDim.x) {
    uint32_t live = 0;
    for (int s = 0; s < a.k; ++s)
      if (a.local[t * a.k + s] >= 0) live |= 1u << s;
    const uint16_t* go = a.dout + t * a.ldd;
    for (int s = 0; s < a.k; ++s) {
      float dot = 0.0f, ss = 0.0f;
      if ((live >> s) & 1)
        for (int c = tid; c < chunks; c += kCgThreads) {
          float yv[8], gv[8], nv[8];
          unpack8(*reinterpret_cast<const uint4*>(a.y + (t * a.k + s) * (int64_t)a.H + c * 8), yv);
          unpack8(*reinterpret_cast<const uint4*>(go + c * 8), gv);
          if (NORM) unpack8(*reinterpret_cast<const uint4*>(a.nw + c * 8), nv);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float z = NORM ? yv[j] * nv[j] : yv[j];
            dot = fmaf(gv[j], z, dot);
            if (NORM) ss = fmaf(z, z, ss);
          }
        }
      for (int d = 32; d >= 1; d >>= 1) {
        dot += __shfl_xor(dot, d);
        if (NORM) ss += __shfl_xor(ss, d);
      }
      if (lane == 0) {
        red[wv][2 * s] = dot;
        red[wv][2 * s + 1] = ss;
      }
    }
    __syncthreads();
    if (tid < a.k) {
      float dot = 0.0f, ss = 0.0f;
      for (int i = 0; i < kCgThreads / 64; ++i) {
        dot += red[i][2 * tid];
        ss += red[i][2 * tid + 1];
      }
      const bool on = (live >> tid) & 1;
      const float g = on ? a.gw[t * a.k + tid] : 0.0f;
      const float r = NORM ? 1.0f / sqrtf(ss / (float)a.H + a.eps) : 1.0f;
      f0[tid] = a.rsf * g * r;
      f1[tid] = NORM ? r * r * dot / (float)a.H : 0.0f;
      if (a.dg) a.dg[t * a.k + tid] = on ? a.rsf * r * dot : 0.0f;
    }
    __syncthreads();
    if (a.dy || a.part)
      for (int s = 0; s < a.k; ++s) {
        const bool on = (live >> s) & 1;
        const float p = f0[s], q = f1[s];
        for (int c = tid; c < chunks; c += kCgThreads) {
          float o[8];
          const int64_t at = (t * a.k + s) * (int64_t)a.H + c * 8;
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = 0.0f;
          if (on) {
            float yv[8], gv[8], nv[8];
            unpack8(*reinterpret_cast<const uint4*>(go + c * 8), gv);
            if (NORM) {
              unpack8(*reinterpret_cast<const uint4*>(a.y + at), yv);
              unpack8(*reinterpret_cast<const uint4*>(a.nw + c * 8), nv);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              if (NORM) {
                const float dz = p * (gv[j] - q * (yv[j] * nv[j]));
                o[j] = dz * nv[j];
                if (a.part) dn[c * 8 + j] = fmaf(dz, yv[j], dn[c * 8 + j]);
              } else {
                o[j] = p * gv[j];
              }
            }
          }
          if (a.dy) *reinterpret_cast<uint4*>(a.dy + at) = pack8(o);
        }
      }
    __syncthreads();  // red, f0, f1
  }
  if (a.part)
    for (int c = tid; c < chunks; c += kCgThreads)
#pragma unroll
      for (int j = 0; j < 8; ++j) a.part[(int64_t)blockIdx.x * a.H + c * 8 + j] = dn[c * 8 + j];
}

// ---------------------------------------------------------------------------- one pass in registers
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;

// Sums of N values (a power of two) over the 64 lanes.  Halves of two values change places, then quarters, so that one
// register goes on with both sums: N + N / 2 exchanges and 4 N / 4 rotations in the place of 6 N.  Lane 16 r then holds in
// v[i] the sum of value 4 i + 2 (r & 1) + (r >> 1) (N >= 4), 2 (r & 1) of N = 2 in its first bit r >> 1, ...
template <int N>
__device__ __forceinline__ void wave_sums(float (&v)[N]) {
#pragma unroll
  for (int i = 0; i < (N + 1) / 2; ++i) {
    const uint32_t a = __float_as_uint(v[N > 1 ? 2 * i : 0]), b = __float_as_uint(v[N > 1 ? 2 * i + 1 : 0]);
    const u32x2_t s = __builtin_amdgcn_permlane32_swap(a, b, false, false);
    v[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  constexpr int N2 = (N + 1) / 2;
#pragma unroll
  for (int i = 0; i < (N2 + 1) / 2; ++i) {
    const uint32_t a = __float_as_uint(v[N2 > 1 ? 2 * i : 0]), b = __float_as_uint(v[N2 > 1 ? 2 * i + 1 : 0]);
    const u32x2_t s = __builtin_amdgcn_permlane16_swap(a, b, false, false);
    v[i] = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  constexpr int N4 = (N2 + 1) / 2;
#pragma unroll
  for (int i = 0; i < N4; ++i) {
    v[i] += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v[i]), 0x128, 0xf, 0xf, false));
    v[i] += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v[i]), 0x124, 0xf, 0xf, false));
    v[i] += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v[i]), 0x122, 0xf, 0xf, false));
    v[i] += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v[i]), 0x121, 0xf, 0xf, false));
  }
}

// For top_k <= TK and rows of at most CP * blockDim.x chunks of 8 columns: a token's operands are asked for at once (with
// `spec` before its flags are known; what dead rows hold is never used) and stay in registers between the sums and the
// rows of dy.  Every wave makes the slots' factors of the workgroup's sums for itself, and tokens alternate between two
// places for the sums, so that a token costs one barrier.
template <bool NORM, int TK, int CP>
__global__ __launch_bounds__(512) void combine_grad1_kernel(CombineGradArgs a, int spec) {
  constexpr int N = NORM ? 2 * TK : TK, N4 = N >= 4 ? N / 4 : 1;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, T = blockDim.x, W = T / 64;
  const int chunks = a.H >> 3;
  __shared__ float red[2][8][N];
  float dn[NORM ? CP : 1][8];
#pragma unroll
  for (int c = 0; c < (NORM ? CP : 1); ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) dn[c][j] = 0.0f;
  uint4 nv[CP];
#pragma unroll
  for (int c = 0; c < CP; ++c) {
    nv[c] = make_uint4(0u, 0u, 0u, 0u);
    if (NORM && tid + c * T < chunks) nv[c] = *reinterpret_cast<const uint4*>(a.nw + (tid + c * T) * 8);
  }
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.M; t += gridDim.x, turn ^= 1) {
    uint32_t live = 0;
    float g[TK];
#pragma unroll
    for (int s = 0; s < TK; ++s) {
      g[s] = 0.0f;
      if (s < a.k) {
        g[s] = a.gw[t * a.k + s];
        if (a.local[t * a.k + s] >= 0) live |= 1u << s;
      }
    }
    uint4 y[TK][CP], go[CP];
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.0f;
#pragma unroll
    for (int c = 0; c < CP; ++c) {
      const int col = tid + c * T;
      go[c] = make_uint4(0u, 0u, 0u, 0u);
      if (col < chunks) go[c] = *reinterpret_cast<const uint4*>(a.dout + t * a.ldd + col * 8);
#pragma unroll
      for (int s = 0; s < TK; ++s) {
        y[s][c] = make_uint4(0u, 0u, 0u, 0u);
        if (s < a.k && col < chunks && (spec || ((live >> s) & 1)))
          y[s][c] = *reinterpret_cast<const uint4*>(a.y + (t * a.k + s) * (int64_t)a.H + col * 8);
      }
    }
#pragma unroll
    for (int c = 0; c < CP; ++c) {
      float gv[8], n8[8];
      unpack8(go[c], gv);
      if (NORM) unpack8(nv[c], n8);
#pragma unroll
      for (int s = 0; s < TK; ++s) {
        if (!((live >> s) & 1)) continue;
        float yv[8];
        unpack8(y[s][c], yv);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float z = NORM ? yv[j] * n8[j] : yv[j];
          sum[s] = fmaf(gv[j], z, sum[s]);
          if constexpr (NORM) sum[TK + s] = fmaf(z, z, sum[TK + s]);
        }
      }
    }
    wave_sums<N>(sum);
    if ((lane & 15) == 0) {
      const int r = lane >> 4;
#pragma unroll
      for (int i = 0; i < N4; ++i) {
        const int at = N >= 4 ? 4 * i + 2 * (r & 1) + (r >> 1) : r >> 1;
        if (at < N) red[turn][wv][at] = sum[i];
      }
    }
    __syncthreads();
    // lane s: the factors of slot s
    const int sl = lane < TK ? lane : 0;
    float dot = 0.0f, ss = 0.0f, gs = 0.0f;
    for (int i = 0; i < W; ++i) {
      dot += red[turn][i][sl];
      if constexpr (NORM) ss += red[turn][i][TK + sl];
    }
#pragma unroll
    for (int s = 0; s < TK; ++s) gs = sl == s ? g[s] : gs;
    const bool on = (live >> sl) & 1;
    const float r = NORM ? 1.0f / sqrtf(ss / (float)a.H + a.eps) : 1.0f;
    const float f0 = on ? a.rsf * gs * r : 0.0f, f1 = NORM && on ? r * r * dot / (float)a.H : 0.0f;
    if (a.dg && wv == 0 && lane < a.k) a.dg[t * a.k + lane] = on ? a.rsf * r * dot : 0.0f;
    if (!a.dy && !a.part) continue;
    float p[TK], q[TK];  // (read from their lanes here, where all are active)
#pragma unroll
    for (int s = 0; s < TK; ++s) {
      p[s] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f0), s));
      q[s] = NORM ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(f1), s)) : 0.0f;
    }
#pragma unroll
    for (int c = 0; c < CP; ++c) {
      const int col = tid + c * T;
      if (col >= chunks) break;
      float gv[8], n8[8];
      unpack8(go[c], gv);
      if (NORM) unpack8(nv[c], n8);
#pragma unroll
      for (int s = 0; s < TK; ++s) {
        if (s >= a.k) break;
        uint4 o = make_uint4(0u, 0u, 0u, 0u);
        if ((live >> s) & 1) {
          float dv[8];
          if constexpr (NORM) {
            float yv[8];
            unpack8(y[s][c], yv);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float dz = p[s] * fmaf(-q[s], yv[j] * n8[j], gv[j]);
              dv[j] = dz * n8[j];
              dn[c][j] = fmaf(dz, yv[j], dn[c][j]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) dv[j] = p[s] * gv[j];
          }
          o = pack8(dv);
        }
        // (past the L2: the dirty lines of 268 MB else kept the step's next kernel waiting, 4096 x 8 x 4096 with its
        // forward 146 against 160 us)
        if (a.dy)
          __builtin_nontemporal_store(u32x4_t{o.x, o.y, o.z, o.w},
                                      reinterpret_cast<u32x4_t*>(a.dy + (t * a.k + s) * (int64_t)a.H + col * 8));
      }
    }
  }
  if constexpr (NORM) {
    if (a.part) {
#pragma unroll
      for (int c = 0; c < CP; ++c) {
        const int col = tid + c * T;
        if (col >= chunks) break;
        float4* o = reinterpret_cast<float4*>(a.part + (int64_t)blockIdx.x * a.H + col * 8);
        o[0] = make_float4(dn[c][0], dn[c][1], dn[c][2], dn[c][3]);
        o[1] = make_float4(dn[c][4], dn[c][5], dn[c][6], dn[c][7]);
      }
    }
  }
}

template <bool NORM>
static void launch_combine_grad1(const CombineGradArgs& a, unsigned grid, int T, int CP, int spec, hipStream_t st) {
  auto go = [&](auto tk) {
    constexpr int TK = decltype(tk)::value;
    if (CP == 1) hipLaunchKernelGGL((combine_grad1_kernel<NORM, TK, 1>), dim3(grid), dim3(T), 0, st, a, spec);
    else hipLaunchKernelGGL((combine_grad1_kernel<NORM, TK, 2>), dim3(grid), dim3(T), 0, st, a, spec);
  };
  if (a.k <= 2) go(std::integral_constant<int, 2>{});
  else if (a.k <= 4) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 8>{});
}

// The workgroups' partial sums of dn: 32 columns a workgroup, four to a thread and 32 threads to a column's rows, sixteen
// loads of each in flight.
__global__ __launch_bounds__(256) void combine_dnorm_kernel(const float* part, int parts, int32_t H, uint16_t* dn) {
  const int col = (threadIdx.x & 7) * 4, row = threadIdx.x >> 3, c = blockIdx.x * 32 + col;
  __shared__ float red[32][33];
  if (parts == 0) {  // no tokens
    if (threadIdx.x < 32 && blockIdx.x * 32 + threadIdx.x < H) dn[blockIdx.x * 32 + threadIdx.x] = 0;
    return;
  }
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  float4 v[kCgParts / 32];
#pragma unroll
  for (int i = 0; i < kCgParts / 32; ++i)  // (H is a multiple of 8: four columns are there or none)
    v[i] = *reinterpret_cast<const float4*>(part + (int64_t)min(row + i * 32, parts - 1) * H + min(c, H - 4));
#pragma unroll
  for (int i = 0; i < kCgParts / 32; ++i)
    if (row + i * 32 < parts) {
      s[0] += v[i].x;
      s[1] += v[i].y;
      s[2] += v[i].z;
      s[3] += v[i].w;
    }
#pragma unroll
  for (int j = 0; j < 4; ++j) red[row][col + j] = s[j];
  __syncthreads();
  const int o = threadIdx.x >> 3, sub = threadIdx.x & 7;  // eight threads a column
  float r = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) r += red[sub * 4 + i][o];
  for (int d = 4; d >= 1; d >>= 1) r += __shfl_xor(r, d);
  if (sub == 0 && blockIdx.x * 32 + o < H) dn[blockIdx.x * 32 + o] = f32_to_bf16(r);
}

static int64_t combine_parts(int64_t M) { return std::min<int64_t>(M, kCgParts); }

}  // namespace moe

using namespace moe;

extern "C" int moe_combine_grad_workspace(int64_t M, int32_t H, int64_t* elems) {
  MOE_REQUIRE(elems, MOE_EINVAL, "moe_combine_grad_workspace: null pointer");
  MOE_REQUIRE(M >= 0 && H >= 1, MOE_EINVAL, "moe_combine_grad_workspace: M=%lld H=%d", (long long)M, H);
  *elems = combine_parts(M) * H;
  return ok();
}

extern "C" int moe_combine_grad(const uint16_t* y, const float* topk_weights, const int32_t* slot_local_ids,
                                const uint16_t* norm_w, float eps, float routed_scaling_factor, int64_t M,
                                int32_t top_k, int32_t H, const uint16_t* d_out, int64_t ld_dout, uint16_t* dy,
                                float* d_weights, uint16_t* d_norm_w, float* work, int64_t work_elems,
                                hipStream_t stream) {
  MOE_REQUIRE(M >= 0 && top_k >= 1 && top_k <= kCgMaxTopK, MOE_EUNSUPPORTED,
              "moe_combine_grad: M=%lld top_k=%d (top_k must be 1..%d)", (long long)M, top_k, kCgMaxTopK);
  MOE_REQUIRE(H >= 8 && H % 8 == 0, MOE_EUNSUPPORTED, "moe_combine_grad: H=%d must be a multiple of 8", H);
  MOE_REQUIRE(M < (1ll << 24), MOE_EUNSUPPORTED, "moe_combine_grad: M=%lld: 2^24 tokens or more", (long long)M);
  MOE_REQUIRE(ld_dout >= H, MOE_EINVAL, "moe_combine_grad: ld_dout=%lld < H=%d", (long long)ld_dout, H);
  MOE_REQUIRE(ld_dout % 8 == 0, MOE_EUNSUPPORTED, "moe_combine_grad: ld_dout=%lld must be a multiple of 8", (long long)ld_dout);
  MOE_REQUIRE(!d_norm_w || norm_w, MOE_EINVAL, "moe_combine_grad: d_norm_w without norm_w");
  MOE_REQUIRE(!d_norm_w || H <= kCgMaxNormH, MOE_EUNSUPPORTED, "moe_combine_grad: d_norm_w of %d columns (at most %d)", H, kCgMaxNormH);
  if (M == 0 && !d_norm_w) return ok();
  MOE_REQUIRE(dy || d_weights || d_norm_w, MOE_EINVAL, "moe_combine_grad: no gradient asked for");
  MOE_REQUIRE(M == 0 || (y && topk_weights && slot_local_ids && d_out), MOE_EINVAL, "moe_combine_grad: null pointer");
  MOE_REQUIRE((((uintptr_t)y | (uintptr_t)d_out | (uintptr_t)dy | (uintptr_t)norm_w | (uintptr_t)work) & 15) == 0 && ((uintptr_t)d_norm_w & 1) == 0 &&
                  (((uintptr_t)topk_weights | (uintptr_t)slot_local_ids | (uintptr_t)d_weights) & 3) == 0,
              MOE_EUNSUPPORTED, "moe_combine_grad: bf16 tensors and the workspace must be 16-byte aligned, the others 4");
  const int64_t parts = combine_parts(M);
  if (d_norm_w)
    MOE_REQUIRE((work && work_elems >= parts * H) || parts == 0, MOE_ESIZE, "moe_combine_grad: workspace of %lld values, need %lld",
                (long long)work_elems, (long long)(parts * H));
  const CombineGradArgs a{y, topk_weights, slot_local_ids, norm_w, eps, routed_scaling_factor, M, top_k, H, d_out, ld_dout,
                          dy, d_weights, d_norm_w ? work : nullptr};
  if (M > 0) {
    const unsigned grid = (unsigned)(d_norm_w ? parts : std::min<int64_t>(M, kCgGrid));
    const size_t lds = d_norm_w ? (size_t)H * 4 : 0;
    const int chunks = H / 8;
    if (top_k <= 8 && chunks <= 1024) {  // (what two chunks a thread and eight slots hold in registers)
      const int T = std::min(512, (chunks + 63) / 64 * 64), CP = (chunks + T - 1) / T, spec = M <= 256;
      if (norm_w) launch_combine_grad1<true>(a, grid, T, CP, spec, stream);
      else launch_combine_grad1<false>(a, grid, T, CP, spec, stream);
    } else if (norm_w) hipLaunchKernelGGL(combine_grad_kernel<true>, dim3(grid), dim3(kCgThreads), lds, stream, a);
    else hipLaunchKernelGGL(combine_grad_kernel<false>, dim3(grid), dim3(kCgThreads), lds, stream, a);
  }
  if (d_norm_w)
    hipLaunchKernelGGL(combine_dnorm_kernel, dim3((H + 31) / 32), dim3(256), 0, stream, work, (int)parts, H, d_norm_w);
  return check_launch("moe_combine_grad");
}
