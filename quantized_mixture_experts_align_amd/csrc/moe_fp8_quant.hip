// moe_fp8_quant / moe_act_fp8_quant: bf16 rows to e4m3fn codes with one fp32 scale for each row
// and group of 128 columns, optionally with the expert activation applied on the way.
//
// For a group v[0..127] (v = x, or act(h) in fp32):
//     top = max |v| (NaN not counted, at least 2^-110),  scale = top / 448,
//     code = e4m3( v * fl(448 / top) )       (round to nearest even; |v * ..| stays below the
// point that rounds past 448, so the hardware convert needs no clamp, and a NaN stays a NaN).
// The floor keeps both 448 / top and the scale normal numbers.  An infinity makes the scale
// infinite and its own code NaN: the group's dequantised values are then NaN throughout.
// (The activations' sigmoid takes the hardware's exponential and reciprocal, each good to about an ulp, though its
// result is not rounded to bf16 here: of 134 million codes 158 fall beyond a rounding point, of the plain form's 156.)
//
// Bound: memory (2 bytes in -- 4 gated -- and 1 + 1/32 out per column, no reuse).  Sixteen lanes
// share a group, eight columns (one 16-byte load) each, so the maximum is four lane exchanges and
// a wave covers four consecutive groups; codes leave as 8 bytes a lane.
#include <algorithm>

#include "moe_internal.h"

namespace moe {

constexpr int kQuantGroup = 128;
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 0x1p-110f;

struct QuantArgs {
  const uint16_t* x;
  int64_t ldx;
  uint8_t* codes;
  int64_t ldc;
  float* scales;
  int64_t lds;
  const int32_t* live;
  int32_t K, G, total;  // columns out, groups per row, groups of all rows
};

struct NoAct {
  float alpha, limit;
};
// Relu2 and SwigluAlpha with comparisons in the place of fminf and fmaxf, which return the other operand
// for a NaN: here it stays one and becomes a NaN code.
struct Relu2Nan {
  float alpha, limit;
  __device__ __forceinline__ float operator()(float h) const {
    const float r = h < 0.0f ? 0.0f : h;
    return r * r;
  }
};
struct SwigluNan {
  float alpha, limit;
  __device__ __forceinline__ float operator()(float g, float u) const {
    g = g > limit ? limit : g;
    u = u < -limit ? -limit : u;
    u = u > limit ? limit : u;
    return g * sigmoid_f(alpha * g) * (u + 1.0f);
  }
};
template <typename ACT> struct is_gated { static constexpr bool value = true; };
template <> struct is_gated<NoAct> { static constexpr bool value = false; };
template <> struct is_gated<Relu2Nan> { static constexpr bool value = false; };

template <typename ACT>
__global__ __launch_bounds__(256) void fp8_quant_kernel(QuantArgs a, ACT act) {
  const int sub = threadIdx.x & 15;
  const uint32_t step = gridDim.x * 16u;
  for (uint32_t q = blockIdx.x * 16u + (threadIdx.x >> 4); q < (uint32_t)a.total; q += step) {
    const uint32_t row = q / (uint32_t)a.G;
    const int g = (int)(q - row * (uint32_t)a.G);
    if (a.live && a.live[row] < 0) continue;  // (the same for the group's sixteen lanes)
    const int col = g * kQuantGroup + sub * 8;
    const bool in = col < a.K;
    float v[8];
    const uint16_t* p = a.x + (int64_t)row * a.ldx + col;
    uint4 r = make_uint4(0u, 0u, 0u, 0u), s = r;
    if (in) {
      r = *reinterpret_cast<const uint4*>(p);
      if constexpr (is_gated<ACT>::value) s = *reinterpret_cast<const uint4*>(p + a.K);
    }
    const uint32_t rr[4] = {r.x, r.y, r.z, r.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (is_gated<ACT>::value) {
        v[2 * j] = act(bf16_lo(rr[j]), bf16_lo(ss[j]));
        v[2 * j + 1] = act(bf16_hi(rr[j]), bf16_hi(ss[j]));
      } else if constexpr (std::is_same<ACT, NoAct>::value) {
        v[2 * j] = bf16_lo(rr[j]);
        v[2 * j + 1] = bf16_hi(rr[j]);
      } else {
        v[2 * j] = act(bf16_lo(rr[j]));
        v[2 * j + 1] = act(bf16_hi(rr[j]));
      }
    }
    float top = kAmaxFloor;
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, in ? fabsf(v[j]) : 0.f);  // fmaxf passes a NaN over
#pragma unroll
    for (int d = 8; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float inv = __fdiv_rn(kE4m3Max, top);
    if (in) {
      int lo = 0, hi = 0;
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[0] * inv, v[1] * inv, lo, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(v[2] * inv, v[3] * inv, lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[4] * inv, v[5] * inv, hi, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(v[6] * inv, v[7] * inv, hi, true);
      *reinterpret_cast<uint2*>(a.codes + (int64_t)row * a.ldc + col) = make_uint2((uint32_t)lo, (uint32_t)hi);
    }
    if (sub == 0) a.scales[(int64_t)row * a.lds + g] = __fdiv_rn(top, kE4m3Max);
  }
}

template <typename ACT>
static int launch_quant(const char* what, const QuantArgs& a, ACT act, hipStream_t st) {
  const int64_t blocks = std::min<int64_t>(((int64_t)a.total + 15) / 16, 8192);
  hipLaunchKernelGGL((fp8_quant_kernel<ACT>), dim3((unsigned)blocks), dim3(256), 0, st, a, act);
  return check_launch(what);
}

// Shared argument checks; *empty is set when there is nothing to do.
static int quant_args(const char* fn, const uint16_t* x, int64_t ld_x, int64_t cols, int64_t R, int32_t K,
                      const int32_t* live, uint8_t* codes, int64_t ld_codes, float* scales, int64_t ld_scales,
                      QuantArgs* a, bool* empty) {
  MOE_REQUIRE(R >= 0 && K >= 1, MOE_EINVAL, "%s: R=%lld K=%d", fn, (long long)R, K);
  MOE_REQUIRE(K % 8 == 0, MOE_EUNSUPPORTED, "%s: K=%d must be a multiple of 8", fn, K);
  const int32_t G = (K + kQuantGroup - 1) / kQuantGroup;
  MOE_REQUIRE(ld_x >= cols && ld_codes >= K && ld_scales >= G, MOE_EINVAL,
              "%s: leading dimensions %lld (>= %lld), %lld (>= %d), %lld (>= %d)", fn, (long long)ld_x,
              (long long)cols, (long long)ld_codes, K, (long long)ld_scales, G);
  MOE_REQUIRE(ld_x % 8 == 0 && ld_codes % 8 == 0, MOE_EUNSUPPORTED,
              "%s: ld_x=%lld and ld_codes=%lld must be multiples of 8", fn, (long long)ld_x, (long long)ld_codes);
  MOE_REQUIRE(R < (1ll << 31) / G, MOE_EUNSUPPORTED, "%s: %lld rows of %d groups: 2^31 groups or more", fn,
              (long long)R, G);
  *empty = R == 0;
  if (R == 0) return ok();
  MOE_REQUIRE(x && codes && scales, MOE_EINVAL, "%s: null pointer", fn);
  MOE_REQUIRE(((uintptr_t)x & 15) == 0 && ((uintptr_t)codes & 7) == 0 && ((uintptr_t)scales & 3) == 0 &&
                  ((uintptr_t)live & 3) == 0,
              MOE_EUNSUPPORTED, "%s: misaligned pointer (x 16 B, codes 8 B, scales and ids 4 B)", fn);
  *a = QuantArgs{x, ld_x, codes, ld_codes, scales, ld_scales, live, K, G, (int32_t)(R * G)};
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_fp8_quant(const uint16_t* x, int64_t ld_x, int64_t R, int32_t K, const int32_t* slot_local_ids,
                             uint8_t* codes, int64_t ld_codes, float* scales, int64_t ld_scales,
                             hipStream_t stream) {
  QuantArgs a;
  bool empty = false;
  const int rc = quant_args("moe_fp8_quant", x, ld_x, K, R, K, slot_local_ids, codes, ld_codes, scales, ld_scales,
                            &a, &empty);
  if (rc || empty) return rc;
  return launch_quant("moe_fp8_quant", a, NoAct{0.f, 0.f}, stream);
}

extern "C" int moe_act_fp8_quant(moe_act_kind kind, const uint16_t* h, int64_t ld_h, int64_t R, int32_t I,
                                 const int32_t* slot_local_ids, float alpha, float limit, uint8_t* codes,
                                 int64_t ld_codes, float* scales, int64_t ld_scales, hipStream_t stream) {
  MOE_REQUIRE(kind == MOE_ACT_SILU_MUL || kind == MOE_ACT_SWIGLU_ALPHA || kind == MOE_ACT_RELU2, MOE_EINVAL,
              "moe_act_fp8_quant: unknown activation %d", (int)kind);
  QuantArgs a;
  bool empty = false;
  const int rc = quant_args("moe_act_fp8_quant", h, ld_h, kind == MOE_ACT_RELU2 ? (int64_t)I : 2 * (int64_t)I, R, I,
                            slot_local_ids, codes, ld_codes, scales, ld_scales, &a, &empty);
  if (rc || empty) return rc;
  if (kind == MOE_ACT_SILU_MUL) return launch_quant("moe_act_fp8_quant", a, SiluMul{alpha, limit}, stream);
  if (kind == MOE_ACT_RELU2) return launch_quant("moe_act_fp8_quant", a, Relu2Nan{alpha, limit}, stream);
  return launch_quant("moe_act_fp8_quant", a, SwigluNan{alpha, limit}, stream);
}
