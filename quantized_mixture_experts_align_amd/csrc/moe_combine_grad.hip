// moe_combine_grad: gradients of the top-k weighted combine, without and with the post-expert RMSNorm.
//
//   out = c sum_s g_s y_s:      dy_s = c g_s dout,  dg_s = c <dout, y_s>
//   with a norm weight n:       z = y n,  r = (mean z^2 + eps)^-1/2,  out = c sum_s g_s r_s z_s,  d = <dout, z>
//       dg_s = c r d,   dz = c g r (dout - (r^2 d / H) z),   dy = dz n,   dn = sum over the live slots of dz y
// Dead slots: dy = 0, dg = 0, their y is not read.  fp32 throughout, each result rounded once.
//
// Bound: memory (every live row of y is read once, every row of dy written once).
#include <algorithm>
#include <cmath>

#include "moe_internal.h"

namespace moe {

constexpr int kCgThreads = 256;
constexpr int kCgMaxTopK = 16;
constexpr int kCgParts = 512;      // workgroups that leave partial sums of dn, at most
constexpr int kCgMaxNormH = 12288; // columns whose dn a workgroup can hold in LDS

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
// the rows of dy, for which y and dout are read again.
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

// The workgroups' partial sums of dn: 32 columns a workgroup, eight threads to a column.
__global__ __launch_bounds__(256) void combine_dnorm_kernel(const float* part, int parts, int32_t H, uint16_t* dn) {
  const int col = threadIdx.x & 31, row = threadIdx.x >> 5, c = blockIdx.x * 32 + col;
  __shared__ float red[8][33];
  float s = 0.0f;
  if (c < H)
    for (int p = row; p < parts; p += 8) s += part[(int64_t)p * H + c];
  red[row][col] = s;
  __syncthreads();
  if (row == 0 && c < H) {
    s = 0.0f;
    for (int i = 0; i < 8; ++i) s += red[i][col];
    dn[c] = f32_to_bf16(s);
  }
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
  MOE_REQUIRE((((uintptr_t)y | (uintptr_t)d_out | (uintptr_t)dy | (uintptr_t)norm_w) & 15) == 0 && ((uintptr_t)d_norm_w & 1) == 0 &&
                  (((uintptr_t)topk_weights | (uintptr_t)slot_local_ids | (uintptr_t)d_weights | (uintptr_t)work) & 3) == 0,
              MOE_EUNSUPPORTED, "moe_combine_grad: bf16 tensors must be 16-byte aligned, the others 4");
  const int64_t parts = combine_parts(M);
  if (d_norm_w)
    MOE_REQUIRE((work && work_elems >= parts * H) || parts == 0, MOE_ESIZE, "moe_combine_grad: workspace of %lld values, need %lld",
                (long long)work_elems, (long long)(parts * H));
  const CombineGradArgs a{y, topk_weights, slot_local_ids, norm_w, eps, routed_scaling_factor, M, top_k, H, d_out, ld_dout,
                          dy, d_weights, d_norm_w ? work : nullptr};
  if (M > 0) {
    const unsigned grid = (unsigned)(d_norm_w ? parts : M);
    const size_t lds = d_norm_w ? (size_t)H * 4 : 0;
    if (norm_w) hipLaunchKernelGGL(combine_grad_kernel<true>, dim3(grid), dim3(kCgThreads), lds, stream, a);
    else hipLaunchKernelGGL(combine_grad_kernel<false>, dim3(grid), dim3(kCgThreads), lds, stream, a);
  }
  if (d_norm_w)
    hipLaunchKernelGGL(combine_dnorm_kernel, dim3((H + 31) / 32), dim3(256), 0, stream, work, (int)parts, H, d_norm_w);
  return check_launch("moe_combine_grad");
}
