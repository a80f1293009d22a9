// moe_router: the top_k experts of every token with their weights, the experts' counts and the balance
// loss of the batch in the same pass; moe_router_grad: the gradient of the logits from both.
//
// A token's logits lie in a group of LANES lanes, V consecutive experts in each, so that a lane's index
// order is the experts' and sums over tokens stay in the lane that holds the expert.  Selection is exact:
// keys are the logits themselves (the scores grow with them), or with a bias the scores in 64 bits, and
// carry the expert's index in their low bits, so that no two are equal and ties fall to the lowest index.
//
// Bound: memory for large batches (each logit is read once forward, once backward), the launch for small.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "moe_internal.h"

namespace moe {

constexpr int kRouterMaxExperts = 1024;
constexpr int kRouterMaxTopK = 16;
constexpr int kRouterParts = 256;  // workgroups that leave partial sums, at most

struct RouterArgs {
  const void* logits;
  int64_t ld, M;
  int32_t E, k, sigmoid, renorm;
  float scale;
  const float* bias;
  const int32_t* live;
  int32_t* ids;
  float* weights;
  // partial sums of every workgroup: probabilities [parts][E], counts [parts][E], tokens [parts]
  float* part_sum;
  int32_t* part_count;
  int32_t* part_tokens;
  int32_t* arrived;
};

struct RouterGradArgs {
  const void* logits;
  int64_t ld, M;
  int32_t E, k, sigmoid, renorm;
  float scale;
  const int32_t* live;
  const int32_t* ids;
  const float* dw;
  const int32_t* counts;
  const int32_t* tokens;
  const float* d_means;
  const float* d_balance;
  void* dx;
  int64_t ld_d;
};

// exp(x) for x <= 0 (no NaN): exp2 of the product with log2(e), whose rounding error is carried along.
__device__ __forceinline__ float exp_neg(float x) {
  constexpr float kL = 0x1.715476p+0f, kLo = 0x1.4ae0cp-26f, kLn2 = 0x1.62e430p-1f;
  x = fmaxf(x, -104.0f);  // (below it exp is under 2^-149)
  const float t = x * kL, r = fmaf(x, kL, -t) + x * kLo, e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, r * kLn2, e);
}

template <int LANES>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
  for (int d = LANES / 2; d >= 1; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
template <int LANES, typename T>
__device__ __forceinline__ T group_sum(T v) {
#pragma unroll
  for (int d = LANES / 2; d >= 1; d >>= 1) v += __shfl_xor(v, d);
  return v;
}
template <int LANES>
__device__ __forceinline__ uint64_t group_max_u64(uint64_t v) {
#pragma unroll
  for (int d = LANES / 2; d >= 1; d >>= 1) {
    const uint64_t o = __shfl_xor((unsigned long long)v, d);
    v = o > v ? o : v;
  }
  return v;
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
  if constexpr (std::is_same<T, float>::value) return *p;
  else return bf16_to_f32(*p);
}
// V consecutive logits; those at or past E read as -inf.  `wide`: rows are 16-byte aligned and E a multiple
// of the values in 16 bytes.
template <typename T, int V>
__device__ __forceinline__ void load_logits(const T* row, int first, int E, bool wide, float (&x)[V]) {
  constexpr int kPer = 16 / (int)sizeof(T);
  if constexpr (V >= kPer) {
    if (wide) {
#pragma unroll
      for (int c = 0; c < V; c += kPer) {
        uint4 r = make_uint4(0u, 0u, 0u, 0u);
        const bool in = first + c < E;
        if (in) r = *reinterpret_cast<const uint4*>(row + first + c);
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          float v;
          if constexpr (kPer == 4) v = __uint_as_float(w[j]);
          else v = (j & 1) ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
          x[c + j] = in ? v : -INFINITY;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = first + j < E ? load_logit(row + first + j) : -INFINITY;
}

// Order-preserving bits (-0 as +0).
__device__ __forceinline__ uint32_t sortable(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u >> 31) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t sortable(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// 1 / (1 + exp(-x)) (no NaN) times exp(-shift), for shift = min(0, the largest x at hand): sums of such
// values never vanish, so that their ratios stay exact however negative the logits are.
__device__ __forceinline__ float sigmoid_shifted(float x, float shift) {
  const float z = exp_neg(-fabsf(x));
  const float num = x >= 0.0f ? 1.0f : (shift == 0.0f ? z : exp_neg(x - shift));
  return num * __builtin_amdgcn_rcpf(1.0f + z);
}

template <typename T, int LANES, int V, bool BIAS, bool STATS>
__global__ __launch_bounds__(256) void router_kernel(RouterArgs a, int wide) {
  constexpr int G = 64 / LANES;  // tokens of a wave at a time
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, sub = lane & (LANES - 1), grp = lane / LANES;
  const int first = sub * V;
  __shared__ float lsum[STATS ? 4 : 1][STATS ? LANES * V : 1];
  __shared__ int lcount[STATS ? LANES * V : 1];
  __shared__ int ltokens;
  float psum[V];
  int tokens = 0;
  if constexpr (STATS) {
    if (threadIdx.x == 0) ltokens = 0;
    for (int e = threadIdx.x; e < LANES * V; e += 256) lcount[e] = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) psum[j] = 0.0f;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.arrived = 0;  // (for the launch that follows)
    __syncthreads();
  }
  const int64_t step = (int64_t)gridDim.x * 4 * G;
  for (int64_t t0 = ((int64_t)blockIdx.x * 4 + wv) * G; t0 < a.M; t0 += step) {
    const int64_t t = t0 + grp;
    const bool in = t < a.M;
    const bool live = in && (!a.live || a.live[t] >= 0);
    const T* row = reinterpret_cast<const T*>(a.logits) + (in ? t : 0) * a.ld;
    float x[V];
    if (live) load_logits<T, V>(row, first, a.E, wide, x);
    else {
#pragma unroll
      for (int j = 0; j < V; ++j) x[j] = -INFINITY;
    }
    bool bad = false;  // a NaN, or an infinite logit under a softmax: the row's weights are NaN
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      bad = bad || x[j] != x[j] || (!a.sigmoid && x[j] == INFINITY);
      m = fmaxf(m, x[j]);
    }
    const uint64_t any = __ballot(bad);
    bad = (any >> (grp * LANES)) & (LANES == 64 ? ~0ull : (1ull << (LANES & 63)) - 1);
    m = group_max<LANES>(m);
    if (m == -INFINITY) m = 0.0f;
    uint64_t key[V];
    if constexpr (BIAS) {
      double s[V], total = 0.0;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s[j] = a.sigmoid ? 1.0 / (1.0 + exp(-(double)x[j])) : exp((double)x[j] - (double)m);
        total += s[j];
      }
      if (!a.sigmoid) total = group_sum<LANES>(total);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        key[j] = 0;
        if (first + j < a.E) {
          const float b = a.bias[first + j];
          const double v = (a.sigmoid ? s[j] : s[j] / total) + (double)b;
          // (the key's lowest 10 of 53 places give way to the index)
          if (x[j] > -INFINITY && b > -INFINITY)
            key[j] = (sortable(v) & ~1023ull) | (uint64_t)(1023 - (first + j));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j)
        key[j] = x[j] > -INFINITY ? ((uint64_t)sortable(x[j]) << 32) | (uint32_t)(1023 - (first + j)) : 0;
    }
    // the largest key k times; lane j of the group keeps the j-th
    int mine = -1;
    for (int j = 0; j < a.k; ++j) {
      uint64_t best = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) best = key[i] > best ? key[i] : best;
      best = group_max_u64<LANES>(best);
#pragma unroll
      for (int i = 0; i < V; ++i) key[i] = key[i] == best ? 0 : key[i];
      if (sub == j && best) mine = 1023 - (int)(best & 1023);
    }
    const bool has = mine >= 0;
    const float xj = has ? load_logit(row + mine) : -INFINITY;
    float w = 0.0f, total = 0.0f, u[V];
    if (STATS || (!a.renorm && !a.sigmoid)) {  // every expert's share
      const float shift = fminf(m, 0.0f);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        u[j] = a.sigmoid ? sigmoid_shifted(x[j], shift) : exp_neg(x[j] - m);
        if (!(x[j] > -INFINITY)) u[j] = 0.0f;
        total += u[j];
      }
      total = group_sum<LANES>(total);
    }
    if (a.renorm) {
      const float mc = group_max<LANES>(xj);
      if (has) w = a.sigmoid ? sigmoid_shifted(xj, fminf(mc, 0.0f)) : exp_neg(xj - mc);
      const float sum = group_sum<LANES>(w);
      if (has) w = a.scale * (w / sum);
    } else if (has) {
      w = a.scale * (a.sigmoid ? sigmoid_shifted(xj, 0.0f) : exp_neg(xj - m) / total);
    }
    if (bad && has) w = NAN;
    if (in && sub < a.k) {
      a.ids[t * a.k + sub] = mine;
      a.weights[t * a.k + sub] = w;
    }
    if constexpr (STATS) {
      const float inv = bad ? NAN : (total > 0.0f ? 1.0f / total : 0.0f);
#pragma unroll
      for (int j = 0; j < V; ++j) psum[j] = live ? fmaf(u[j], inv, psum[j]) : psum[j];
      if (has) atomicAdd(&lcount[mine], 1);
      tokens += live && sub == 0;
    }
  }
  if constexpr (STATS) {
    if (tokens) atomicAdd(&ltokens, tokens);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float v = psum[j];
#pragma unroll
      for (int d = LANES; d < 64; d <<= 1) v += __shfl_xor(v, d);
      if (grp == 0) lsum[wv][first + j] = v;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += 256) {
      a.part_sum[(int64_t)blockIdx.x * a.E + e] = (lsum[0][e] + lsum[1][e]) + (lsum[2][e] + lsum[3][e]);
      a.part_count[(int64_t)blockIdx.x * a.E + e] = lcount[e];
    }
    if (threadIdx.x == 0) a.part_tokens[blockIdx.x] = ltokens;
  }
}

// The workgroups' partial sums to counts, mean probabilities and the loss.  A workgroup takes 16 experts; the
// last one to finish adds the experts' shares of the loss up, in their order.
__global__ __launch_bounds__(256) void router_stats_kernel(const float* part_sum, const int32_t* part_count,
                                                           const int32_t* part_tokens, int parts, int E,
                                                           int32_t* counts, float* means, float* balance,
                                                           int32_t* tokens, int32_t* arrived) {
  const int tid = threadIdx.x, col = tid & 15, row = tid >> 4, e = blockIdx.x * 16 + col;
  __shared__ double dsum[16][17];
  __shared__ int icount[16][17];
  __shared__ int red[4];
  __shared__ double dred[4];
  __shared__ int last;
  double s = 0.0;
  int n = 0, tok = 0;
  if (e < E)
    for (int p = row; p < parts; p += 16) {
      s += (double)part_sum[(int64_t)p * E + e];
      n += part_count[(int64_t)p * E + e];
    }
  for (int p = tid; p < parts; p += 256) tok += part_tokens[p];
  for (int d = 32; d >= 1; d >>= 1) tok += __shfl_xor(tok, d);
  if ((tid & 63) == 0) red[tid >> 6] = tok;
  dsum[row][col] = s;
  icount[row][col] = n;
  __syncthreads();
  tok = red[0] + red[1] + red[2] + red[3];
  if (row == 0 && e < E) {
    s = 0.0;
    n = 0;
    for (int i = 0; i < 16; ++i) {
      s += dsum[i][col];
      n += icount[i][col];
    }
    __hip_atomic_store(&counts[e], n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(&means[e], tok ? (float)(s / (double)tok) : 0.0f, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  if (blockIdx.x == 0 && tid == 0) *tokens = tok;
  __threadfence();
  __syncthreads();
  if (tid == 0) last = atomicAdd(arrived, 1) == (int)gridDim.x - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  double loss = 0.0;
  int all = 0;
  for (int i = tid; i < E; i += 256) {
    const int c = __hip_atomic_load(&counts[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const float p = __hip_atomic_load(&means[i], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    loss += (double)c * (double)p;
    all += c;
  }
  for (int d = 32; d >= 1; d >>= 1) {
    loss += __shfl_xor(loss, d);
    all += __shfl_xor(all, d);
  }
  __syncthreads();  // (red is read above)
  if ((tid & 63) == 0) {
    dred[tid >> 6] = loss;
    red[tid >> 6] = all;
  }
  __syncthreads();
  if (tid == 0) {
    loss = (dred[0] + dred[1]) + (dred[2] + dred[3]);
    all = red[0] + red[1] + red[2] + red[3];
    *balance = (float)((double)E * loss / (double)(all > 0 ? all : 1));
  }
}

// dx = the router's gradient + the balance loss's, one write of the row.  With q the probabilities, h the
// chosen shares (w = scale * h) and a_e = (d_means[e] + d_balance * E * n_e / sum n) / tokens:
//   loss      q_e (a_e - sum a q), times 1 - s_e for sigmoid scores
//   weights   renormalised: scale * h_j (dw_j - sum dw h), times 1 - s_j for sigmoid scores
//             softmax: scale * p_e ([e chosen] dw_e - sum dw p);  sigmoid: scale * s_j (1 - s_j) dw_j
// The chosen entries reach the lanes that hold their experts through LDS.
template <typename T, int LANES, int V>
__global__ __launch_bounds__(256) void router_grad_kernel(RouterGradArgs a, int wide) {
  constexpr int G = 64 / LANES;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, sub = lane & (LANES - 1), grp = lane / LANES;
  const int first = sub * V;
  __shared__ float chosen[4][64 * V];
  __shared__ int red[4];
  const bool loss = a.d_balance || a.d_means;
  float coef[V];
  if (loss) {
    int all = 0;
    for (int e = threadIdx.x; e < a.E; e += 256) all += a.counts[e];
    for (int d = 32; d >= 1; d >>= 1) all += __shfl_xor(all, d);
    if (lane == 0) red[wv] = all;
    __syncthreads();
    all = red[0] + red[1] + red[2] + red[3];
    const float tokens = (float)max(*a.tokens, 1);
    const float share = a.d_balance ? *a.d_balance * ((float)a.E / (float)max(all, 1)) : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      coef[j] = 0.0f;
      if (first + j < a.E)
        coef[j] = ((a.d_means ? a.d_means[first + j] : 0.0f) + share * (float)a.counts[first + j]) / tokens;
    }
  }
  const int64_t t = ((int64_t)blockIdx.x * 4 + wv) * G + grp;
  const bool in = t < a.M;
  const bool live = in && (!a.live || a.live[t] >= 0);
  const T* row = reinterpret_cast<const T*>(a.logits) + (in ? t : 0) * a.ld;
  float x[V];
  if (live) load_logits<T, V>(row, first, a.E, wide & 1, x);
  else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = -INFINITY;
  }
  bool bad = false;
  float m = -INFINITY;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    bad = bad || x[j] != x[j] || (!a.sigmoid && x[j] == INFINITY);
    m = fmaxf(m, x[j]);
  }
  const uint64_t any = __ballot(bad);
  bad = (any >> (grp * LANES)) & (LANES == 64 ? ~0ull : (1ull << (LANES & 63)) - 1);
  m = group_max<LANES>(m);
  if (m == -INFINITY) m = 0.0f;
  float q[V], total = 0.0f, aq = 0.0f;
  const bool dense = loss || (!a.renorm && !a.sigmoid);
  const float shift = fminf(m, 0.0f);
  if (dense) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      q[j] = a.sigmoid ? sigmoid_shifted(x[j], shift) : exp_neg(x[j] - m);
      if (!(x[j] > -INFINITY)) q[j] = 0.0f;
      total += q[j];
    }
    total = group_sum<LANES>(total);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) q[j] *= inv;
    if (loss) {
#pragma unroll
      for (int j = 0; j < V; ++j) aq = fmaf(coef[j], q[j], aq);
      aq = group_sum<LANES>(aq);
    }
  }
  // the chosen entries: lane j holds the j-th
  float* mine = chosen[wv] + grp * LANES * V;
#pragma unroll
  for (int j = 0; j < V; ++j) mine[first + j] = 0.0f;
  float rest = 0.0f;  // scale * sum dw p of a softmax over all experts
  if (a.dw) {
    int id = -1;
    float dw = 0.0f, h = 0.0f, slope = 1.0f;
    if (live && sub < a.k) {
      id = a.ids[t * a.k + sub];
      dw = a.dw[t * a.k + sub];
      if (id >= a.E) id = -1;
    }
    const float xj = id >= 0 ? load_logit(row + id) : -INFINITY;
    const bool has = xj > -INFINITY;
    if (a.renorm) {
      const float mc = group_max<LANES>(xj);
      if (has) h = a.sigmoid ? sigmoid_shifted(xj, fminf(mc, 0.0f)) : exp_neg(xj - mc);
      const float sum = group_sum<LANES>(h);
      if (has) h /= sum;
    } else if (has) {
      h = a.sigmoid ? sigmoid_shifted(xj, 0.0f) : exp_neg(xj - m) / total;
    }
    if (has && a.sigmoid) slope = sigmoid_shifted(-xj, 0.0f);
    const float dot = group_sum<LANES>(has ? dw * h : 0.0f);
    float d = 0.0f;
    if (has) d = a.scale * h * slope * (a.renorm ? dw - dot : dw);
    if (!a.renorm && !a.sigmoid) rest = a.scale * dot;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (has) atomicAdd(&mine[id], d);
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (!in) return;
  float out[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float v = mine[first + j];
    if (dense) {
      float g = loss ? coef[j] - aq : 0.0f;
      if (a.sigmoid) g *= sigmoid_shifted(-fmaxf(x[j], -104.0f), 0.0f);
      v = fmaf(q[j], g - rest, v);
    }
    out[j] = bad ? NAN : v;
  }
  T* o = reinterpret_cast<T*>(a.dx) + t * a.ld_d;
  constexpr int kPer = 16 / (int)sizeof(T);
  if constexpr (V >= kPer) {
    if (wide & 2) {
#pragma unroll
      for (int c = 0; c < V; c += kPer) {
        if (first + c >= a.E) break;
        uint4 r;
        if constexpr (kPer == 4)
          r = make_uint4(__float_as_uint(out[c]), __float_as_uint(out[c + 1]), __float_as_uint(out[c + 2]),
                         __float_as_uint(out[c + 3]));
        else
          r = make_uint4(pack_bf16x2(out[c], out[c + 1]), pack_bf16x2(out[c + 2], out[c + 3]),
                         pack_bf16x2(out[c + 4], out[c + 5]), pack_bf16x2(out[c + 6], out[c + 7]));
        *reinterpret_cast<uint4*>(o + first + c) = r;
      }
      return;
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j)
    if (first + j < a.E) {
      if constexpr (std::is_same<T, float>::value) o[first + j] = out[j];
      else o[first + j] = f32_to_bf16(out[j]);
    }
}

// f(lanes, values a lane) of the layout that holds E experts.
template <typename F>
static void router_layout(int E, F f) {
  using std::integral_constant;
  if (E <= 64) f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (E <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else if (E <= 256) f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else if (E <= 512) f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
  else f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}
static int router_group(int E) { return E <= 256 ? 16 : E <= 512 ? 32 : 64; }
// tokens of a workgroup at a time, and the workgroups that leave partial sums
static int64_t router_blocks(int64_t M, int E) {
  const int64_t per = 4 * (64 / router_group(E));
  return (M + per - 1) / per;
}
static int64_t router_parts(int64_t M, int E) {
  return std::max<int64_t>(1, std::min<int64_t>(router_blocks(M, E), kRouterParts));
}

template <typename T>
static void launch_router(const RouterArgs& a, unsigned grid, bool stats, int wide, hipStream_t st) {
  router_layout(a.E, [&](auto lanes, auto v) {
    constexpr int LN = decltype(lanes)::value, V = decltype(v)::value;
    if (a.bias && stats) hipLaunchKernelGGL((router_kernel<T, LN, V, true, true>), dim3(grid), dim3(256), 0, st, a, wide);
    else if (a.bias) hipLaunchKernelGGL((router_kernel<T, LN, V, true, false>), dim3(grid), dim3(256), 0, st, a, wide);
    else if (stats) hipLaunchKernelGGL((router_kernel<T, LN, V, false, true>), dim3(grid), dim3(256), 0, st, a, wide);
    else hipLaunchKernelGGL((router_kernel<T, LN, V, false, false>), dim3(grid), dim3(256), 0, st, a, wide);
  });
}

static bool wide_rows(const void* p, int64_t ld, int E, bool f32) {
  const int per = f32 ? 4 : 8;
  return ((uintptr_t)p & 15) == 0 && ld % per == 0 && E % per == 0;
}

static int router_checks(const char* fn, int64_t M, int32_t E, int64_t ld, int score, int32_t top_k) {
  MOE_REQUIRE(score == MOE_SCORE_SOFTMAX || score == MOE_SCORE_SIGMOID, MOE_EINVAL, "%s: unknown score %d", fn, score);
  MOE_REQUIRE(M >= 0 && E >= 1 && top_k >= 1 && top_k <= E && ld >= E, MOE_EINVAL, "%s: M=%lld E=%d top_k=%d ld=%lld",
              fn, (long long)M, E, top_k, (long long)ld);
  MOE_REQUIRE(E <= kRouterMaxExperts && top_k <= kRouterMaxTopK, MOE_EUNSUPPORTED, "%s: E=%d (at most %d), top_k=%d (at most %d)",
              fn, E, kRouterMaxExperts, top_k, kRouterMaxTopK);
  MOE_REQUIRE(M <= (1ll << 25), MOE_EUNSUPPORTED, "%s: M=%lld: more than 2^25 tokens", fn, (long long)M);
  return MOE_OK;
}

}  // namespace moe

using namespace moe;

extern "C" int moe_router_workspace(int64_t M, int32_t E, int64_t* bytes) {
  MOE_REQUIRE(bytes, MOE_EINVAL, "moe_router_workspace: null pointer");
  MOE_REQUIRE(M >= 0 && E >= 1 && E <= kRouterMaxExperts, MOE_EINVAL, "moe_router_workspace: M=%lld E=%d", (long long)M, E);
  *bytes = 16 + router_parts(M, E) * (8 * (int64_t)E + 4);
  return ok();
}

extern "C" int moe_router(const void* logits, int32_t logits_f32, int64_t ld, int64_t M, int32_t E, const float* bias,
                          const int32_t* live, moe_score_kind score, int32_t top_k, int32_t renormalise, float scale,
                          int32_t* topk_ids, float* topk_weights, int32_t* counts, float* means, float* balance,
                          int32_t* tokens, void* work, int64_t work_bytes, hipStream_t stream) {
  const int rc = router_checks("moe_router", M, E, ld, (int)score, top_k);
  if (rc) return rc;
  const bool stats = counts || means || balance || tokens;
  const int64_t parts = router_parts(M, E);
  if (stats) {
    MOE_REQUIRE(counts && means && balance && tokens && work, MOE_EINVAL,
                "moe_router: counts, means, balance and tokens go together, with a workspace");
    MOE_REQUIRE(work_bytes >= 16 + parts * (8 * (int64_t)E + 4), MOE_ESIZE, "moe_router: workspace of %lld bytes, need %lld",
                (long long)work_bytes, (long long)(16 + parts * (8 * (int64_t)E + 4)));
    MOE_REQUIRE(((uintptr_t)work & 3) == 0 && ((uintptr_t)counts & 3) == 0 && ((uintptr_t)means & 3) == 0,
                MOE_EUNSUPPORTED, "moe_router: counts, means and the workspace must be 4-byte aligned");
  }
  if (M == 0 && !stats) return ok();
  MOE_REQUIRE(M == 0 || (logits && topk_ids && topk_weights), MOE_EINVAL, "moe_router: null pointer");
  const int bytes = logits_f32 ? 4 : 2;
  MOE_REQUIRE((uintptr_t)logits % bytes == 0 && ((uintptr_t)topk_ids & 3) == 0 && ((uintptr_t)topk_weights & 3) == 0 &&
                  ((uintptr_t)bias & 3) == 0 && ((uintptr_t)live & 3) == 0,
              MOE_EUNSUPPORTED, "moe_router: misaligned pointer");
  RouterArgs a{logits, ld, M, E, top_k, score == MOE_SCORE_SIGMOID, renormalise != 0, scale, bias, live, topk_ids,
               topk_weights, nullptr, nullptr, nullptr, nullptr};
  if (stats) {
    a.arrived = (int32_t*)work;
    a.part_tokens = a.arrived + 4;
    a.part_sum = (float*)(a.part_tokens + parts);
    a.part_count = (int32_t*)(a.part_sum + parts * E);
  }
  const bool wide = wide_rows(logits, ld, E, logits_f32);
  const unsigned grid = (unsigned)std::max<int64_t>(1, stats ? parts : router_blocks(M, E));
  if (logits_f32) launch_router<float>(a, grid, stats, wide, stream);
  else launch_router<uint16_t>(a, grid, stats, wide, stream);
  if (stats)
    hipLaunchKernelGGL(router_stats_kernel, dim3((E + 15) / 16), dim3(256), 0, stream, a.part_sum, a.part_count,
                       a.part_tokens, (int)parts, E, counts, means, balance, tokens, a.arrived);
  return check_launch("moe_router");
}

extern "C" int moe_router_grad(const void* logits, int32_t logits_f32, int64_t ld, int64_t M, int32_t E,
                               const int32_t* live, moe_score_kind score, int32_t top_k, int32_t renormalise, float scale,
                               const int32_t* topk_ids, const float* d_weights, const int32_t* counts,
                               const int32_t* tokens, const float* d_means, const float* d_balance, void* d_logits,
                               int64_t ld_d, hipStream_t stream) {
  const int rc = router_checks("moe_router_grad", M, E, ld, (int)score, top_k);
  if (rc) return rc;
  MOE_REQUIRE(ld_d >= E, MOE_EINVAL, "moe_router_grad: ld_d=%lld", (long long)ld_d);
  MOE_REQUIRE(!(d_means || d_balance) || (counts && tokens), MOE_EINVAL,
              "moe_router_grad: the loss's gradient needs counts and tokens");
  if (M == 0) return ok();
  MOE_REQUIRE(logits && d_logits && (topk_ids || !d_weights), MOE_EINVAL, "moe_router_grad: null pointer");
  const int bytes = logits_f32 ? 4 : 2;
  MOE_REQUIRE((uintptr_t)logits % bytes == 0 && (uintptr_t)d_logits % bytes == 0 && ((uintptr_t)topk_ids & 3) == 0 &&
                  ((uintptr_t)d_weights & 3) == 0 && ((uintptr_t)counts & 3) == 0 && ((uintptr_t)live & 3) == 0 &&
                  ((uintptr_t)tokens & 3) == 0 && ((uintptr_t)d_means & 3) == 0 && ((uintptr_t)d_balance & 3) == 0,
              MOE_EUNSUPPORTED, "moe_router_grad: misaligned pointer");
  const RouterGradArgs a{logits, ld, M, E, top_k, score == MOE_SCORE_SIGMOID, renormalise != 0, scale, live, topk_ids,
                         d_weights, counts, tokens, d_means, d_balance, d_logits, ld_d};
  const int wide = wide_rows(logits, ld, E, logits_f32) | (wide_rows(d_logits, ld_d, E, logits_f32) << 1);
  const unsigned grid = (unsigned)router_blocks(M, E);
  router_layout(E, [&](auto lanes, auto v) {
    constexpr int LN = decltype(lanes)::value, V = decltype(v)::value;
    if (logits_f32) hipLaunchKernelGGL((router_grad_kernel<float, LN, V>), dim3(grid), dim3(256), 0, stream, a, wide);
    else hipLaunchKernelGGL((router_grad_kernel<uint16_t, LN, V>), dim3(grid), dim3(256), 0, stream, a, wide);
  });
  return check_launch("moe_router_grad");
}
