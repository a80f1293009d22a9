// moe_router: the top_k experts of every token with their weights, the experts' counts and the balance
// loss of the batch in the same pass; moe_router_grad: the gradient of the logits from both.
//
// A token's logits lie in a group of LANES lanes, V in each, in chunks of four consecutive experts, adjacent lanes
// adjacent chunks (one load a chunk and lane where rows are aligned; the same places, and so the same bits of every
// result, where they are not).  Sums over tokens stay in the lane that holds the expert, so the statistics cost one
// exchange per workgroup.
//
// Selection is exact: the logits themselves are ordered (the scores grow with them), or with a bias the scores in 64
// bits; ties fall to the lower index.  Keys of 32 bits carry the expert's index in their low places, so they are
// unique: a lane sorts its own by a network, then lists of the eight largest are merged across the lanes
// (no loads, no branches; taking the largest of the group k times, with a dependent exchange each, took 47 us in the place of 20).
// bf16 logits fit such a key whole.  fp32 logits and biased scores do not: they are cut to steps of 2^-19 and 2^-23
// (E <= 256) below the row's largest, and a wave in which two of the k + 1 largest stand closer than the keys' errors
// orders the candidates again by keys of 64 bits, and where scores are equal in all of those by the index.
//
// Bound: the launch for small batches (1 token 3.5 us, 64 tokens 3.0 us), vector instructions for large ones: 32768 x 256
// bf16 sigmoid + bias, top 8, take 17 us (842 instructions a wave of 4 tokens, 88 % of the time issuing; the 19 MB
// alone would take 3.7), 11 without the bias, 24 with biases of 0 (in most waves two scores are equal).  The gradient of
// 32765 x 129 fp32 takes 14 to 16 us (its 30 MB 6).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "moe_internal.h"

namespace moe {

constexpr int kRouterMaxExperts = 1024;
constexpr int kRouterMaxTopK = 16;
constexpr int kRouterParts = 256;      // workgroups that leave partial sums, at most
constexpr int kRouterThreads = 256;    // without statistics
constexpr int kRouterStatThreads = 512;

// What the statistics' launches pass on in the workspace's first bytes.
struct RouterTotals {
  uint64_t loss;      // sum of n_e P_e in units of 2^-60 tokens * top_k: an integer, so that its order does not matter
  uint32_t slots;     // sum of n_e
  uint32_t arrived;   // workgroups, in the upper half those whose share of the loss is NaN
};

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
  RouterTotals* totals;
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

// v of the lane n places further round in its row of 16 lanes.
template <int N>
__device__ __forceinline__ uint32_t row_turn(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x120 + N, 0xf, 0xf, false);
}
// Reductions over a group of LANES lanes, the same bits in each of them.
template <int LANES, typename F>
__device__ __forceinline__ uint32_t group_reduce(uint32_t v, F f) {
  v = f(v, row_turn<8>(v));
  v = f(v, row_turn<4>(v));
  v = f(v, row_turn<2>(v));
  v = f(v, row_turn<1>(v));
  if constexpr (LANES >= 32) v = f(v, (uint32_t)__shfl_xor((int)v, 16));
  if constexpr (LANES >= 64) v = f(v, (uint32_t)__shfl_xor((int)v, 32));
  return v;
}
template <int LANES>
__device__ __forceinline__ float group_max(float v) {
  return __uint_as_float(group_reduce<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int LANES>
__device__ __forceinline__ float group_sum(float v) {
  return __uint_as_float(group_reduce<LANES>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  return group_reduce<LANES>(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int LANES>
__device__ __forceinline__ bool group_any(bool b, int grp) {
  const uint64_t m = __ballot(b);
  return (m >> (grp * LANES)) & (LANES == 64 ? ~0ull : (1ull << (LANES & 63)) - 1);
}

template <typename T>
__device__ __forceinline__ float load_logit(const T* p) {
  if constexpr (std::is_same<T, float>::value) return *p;
  else return bf16_to_f32(*p);
}
// The expert of a lane's j-th logit, and the lane and place of an expert.
template <int LANES>
__device__ __forceinline__ int expert_of(int sub, int j) { return ((j / 4) * LANES + sub) * 4 + j % 4; }
template <int LANES>
__device__ __forceinline__ void place_of(int expert, int& sub, int& j) {
  const uint32_t e = (uint32_t)expert;
  sub = (int)((e / 4) % LANES);
  j = (int)(e / (4 * LANES) * 4 + e % 4);
}
// Experts j * LANES + sub, adjacent in a group, in LDS of [V][64]: the first's place for this lane, and the others' behind it.
__device__ __forceinline__ int turned_place(uint32_t sub, uint32_t lane) { return (int)((sub & 3) * 64 + (lane - sub) + (sub >> 2)); }
template <int LANES>
__device__ __forceinline__ constexpr int turned_step(int j) { return (j / 4) * 256 + (j % 4) * (LANES / 4); }

// A lane's logits (or biases, T float).  wide: rows aligned for loads of four, E a multiple of 4.  No branches around the loads: they would be waited for one by one,
// so lanes without an expert read one that is there.
// Other rows are read 16 adjacent logits a group and load, and change lanes through LDS ([V][64] of the wave, `lane`
// this one's): in the places above, four loads would each touch every line (fp32, 32765 x 129: the gradient 18.8 us against 16.3).
template <typename T, int LANES, int V>
__device__ __forceinline__ void load_logits(const T* row, int sub, int E, bool wide, float* lds, int lane, float (&x)[V]) {
  if (wide) {
#pragma unroll
    for (int c = 0; c < V; c += 4) {
      const int e = expert_of<LANES>(sub, c);
      const T* p = row + (e < E ? e : 0);
      if constexpr (std::is_same<T, float>::value) {
        const float4 r = *reinterpret_cast<const float4*>(p);
        x[c] = r.x; x[c + 1] = r.y; x[c + 2] = r.z; x[c + 3] = r.w;
      } else {
        const uint2 r = *reinterpret_cast<const uint2*>(p);
        x[c] = bf16_lo(r.x); x[c + 1] = bf16_hi(r.x); x[c + 2] = bf16_lo(r.y); x[c + 3] = bf16_hi(r.y);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = load_logit(row + min(j * LANES + sub, E - 1));
    float* to = lds + turned_place(sub, lane);
#pragma unroll
    for (int j = 0; j < V; ++j) to[turned_step<LANES>(j)] = x[j];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = lds[j * 64 + lane];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  }
}
// Those at or past `end` are -inf.
template <int LANES, int V>
__device__ __forceinline__ void mask_logits(int sub, int end, float (&x)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = expert_of<LANES>(sub, j) < end ? x[j] : -INFINITY;
}

// Order-preserving bits (-0 as +0), never 0 for a value above -inf; and back.
__device__ __forceinline__ uint32_t sortable(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unsortable(uint32_t u) {
  return __uint_as_float(u ^ ((uint32_t)((int32_t)~u >> 31) | 0x80000000u));
}
__device__ __forceinline__ uint64_t sortable(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v + 0.0);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}

// 1 / (1 + exp(-x)) (no NaN) times exp(-shift), for shift = min(0, the largest x at hand): sums of such
// values never vanish, so that their ratios stay exact however negative the logits are.  (No branches: unrolled over
// a lane's logits they cost more than the second exponential.)
__device__ __forceinline__ float sigmoid_shifted(float x, float shift) {
  return exp_neg(fminf(x, 0.0f) - shift) * __builtin_amdgcn_rcpf(1.0f + exp_neg(-fabsf(x)));
}

// Every expert's share of the row's sum before the division by it, and that sum (m: the row's largest logit).
template <int LANES, int V>
__device__ __forceinline__ float row_shares(const float (&x)[V], int sigmoid, float m, float (&u)[V]) {
  float total = 0.0f;
  if (sigmoid && __any(m < 0.0f)) {
    const float shift = fminf(m, 0.0f);
#pragma unroll
    for (int j = 0; j < V; ++j) u[j] = sigmoid_shifted(x[j], shift);
  } else if (sigmoid) {  // (the same values with one exponential)
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float z = exp_neg(-fabsf(x[j]));
      u[j] = (x[j] >= 0.0f ? 1.0f : z) * __builtin_amdgcn_rcpf(1.0f + z);
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) u[j] = exp_neg(x[j] - m);
  }
#pragma unroll
  for (int j = 0; j < V; ++j) {
    u[j] = x[j] > -INFINITY ? u[j] : 0.0f;
    total += u[j];
  }
  return group_sum<LANES>(total);
}

// The row's largest logit (0 for a row of -inf), and whether its weights are NaN: a NaN, or an infinite logit under a
// softmax.  (The maximum that hands a NaN on: one instruction for two logits and both answers.)
template <int LANES, int V>
__device__ __forceinline__ float row_max(const float (&x)[V], int sigmoid, int grp, bool& bad) {
  float m = x[0];
#pragma unroll
  for (int j = 1; j < V; ++j) m = __builtin_elementwise_maximum(m, x[j]);
  bad = group_any<LANES>(m != m || (!sigmoid && m == INFINITY), grp);
  m = group_max<LANES>(m);  // (passes a lane's NaN over)
  return m > -INFINITY ? m : 0.0f;
}

// Falling order by odd-even merging (comparators that are known at compile time; V need not be a power of two).
template <int V>
__device__ __forceinline__ void sort_falling(uint32_t (&v)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int q = p; q >= 1; q /= 2)
#pragma unroll
      for (int j = q % p; j < V - q; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i) {
          const int a = i + j, b = i + j + q;
          if (b < V && a / (2 * p) == b / (2 * p)) {
            const uint32_t hi = v[a] > v[b] ? v[a] : v[b], lo = v[a] > v[b] ? v[b] : v[a];
            v[a] = hi;
            v[b] = lo;
          }
        }
}

// One merge of falling lists of eight: the eight largest of a lane's and its partner's, and the largest of those left.
template <typename F>
__device__ __forceinline__ void merge_lists(uint32_t (&v)[8], uint32_t& left, F partner) {
  uint32_t o[8], w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = partner(v[7 - i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w[i] = max(v[i], o[i]);
    left = max(left, min(v[i], o[i]));
  }
#pragma unroll
  for (int q = 4; q >= 1; q /= 2)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (!(i & q)) {
        const uint32_t hi = max(w[i], w[i + q]), lo = min(w[i], w[i + q]);
        w[i] = hi;
        w[i + q] = lo;
      }
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = w[i];
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, false);
}
// The largest keys of a group: lane j < 8 gets the j-th, lane 8 the ninth (0: none).
template <int LANES, int V>
__device__ __forceinline__ uint32_t nine_largest(uint32_t (&key)[V], int sub) {
  sort_falling<V>(key);
  uint32_t v[8], left = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = i < V ? key[i < V ? i : 0] : 0;
  if constexpr (V > 8) left = key[8];
  merge_lists(v, left, dpp<0xB1>);   // lanes 1 apart
  merge_lists(v, left, dpp<0x4E>);   // 2
  merge_lists(v, left, dpp<0x141>);  // the other four of eight, mirrored
  merge_lists(v, left, dpp<0x140>);  // the other eight of sixteen
  if constexpr (LANES >= 32) merge_lists(v, left, [](uint32_t x) { return (uint32_t)__shfl_xor((int)x, 16); });
  if constexpr (LANES >= 64) merge_lists(v, left, [](uint32_t x) { return (uint32_t)__shfl_xor((int)x, 32); });
  left = group_max<LANES>(left);
  const bool b0 = sub & 1, b1 = sub & 2, b2 = sub & 4;
  const uint32_t a0 = b0 ? v[1] : v[0], a1 = b0 ? v[3] : v[2], a2 = b0 ? v[5] : v[4], a3 = b0 ? v[7] : v[6];
  const uint32_t c0 = b1 ? a1 : a0, c1 = b1 ? a3 : a2;
  const uint32_t r = b2 ? c1 : c0;
  return sub < 8 ? r : (sub == 8 ? left : 0);
}

// A biased score in fp32 (a sigmoid's exponential may overflow: the score is then 0).
__device__ __forceinline__ float biased(float x, float b, int sigmoid, float m, float inv) {
  constexpr float kL = 0x1.715476p+0f;
  if (sigmoid) return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -kL)) + b;
  return fmaf(__builtin_amdgcn_exp2f((x - m) * kL), inv, b);
}

// exp in 64 bits, to a few units in the last place: exp(x) = 2^n exp(r), |r| <= ln(2) / 2, by the series of exp(r)
// (0.35^15 / 15! is below 2^-62), with 14! times its coefficients, which are whole.  A loop without tables: the library's
// function, around a path that is seldom taken, took 206 registers a lane in the place of 173.
__device__ __forceinline__ double exp_wide(double x) {
  x = fmin(fmax(x, -1000.0), 1000.0);
  const double n = rint(x * 0x1.71547652b82fep+0);
  const double r = fma(n, -0x1.abc9e3b39803fp-56, fma(n, -0x1.62e42fefa39efp-1, x));
  double p = 1.0, c = 1.0;
#pragma unroll 1
  for (double i = 14.0; i > 0.5; i -= 1.0) {
    c *= i;
    p = fma(p, r, c);
  }
  return ldexp(p / 87178291200.0, (int)n);
}

// The 64-bit key of an expert (0: not eligible): its logit with the index behind it, or its biased score, whole (equal
// scores go by the index all the same).
template <bool BIAS>
__device__ __forceinline__ uint64_t wide_key(float x, float b, int e, int sigmoid, float m, double total) {
  if (!(x > -INFINITY)) return 0;
  if (!BIAS) return ((uint64_t)sortable(x) << 32) | (uint32_t)(1023 - e);
  if (!(b > -INFINITY) || (!sigmoid && x == INFINITY)) return 0;  // (an infinite logit's softmax is NaN, the others' beside it 0)
  const double z = exp_wide(sigmoid ? -(double)x : (double)x - (double)m);
  const double s = sigmoid ? 1.0 / (1.0 + z) : total > 0.0 ? z / total : 0.0;
  return sortable(s + (double)b);
}
// A row's sum of exponentials in 64 bits.
template <typename T, int LANES, int V>
__device__ __forceinline__ double wide_total(const T* row, int E, int sub, float m) {
  double total = 0.0;
#pragma unroll 1
  for (int j = 0; j < V; ++j) {
    const int e = expert_of<LANES>(sub, j);
    if (e < E) total += exp_wide((double)load_logit(row + e) - (double)m);
  }
#pragma unroll
  for (int d = LANES / 2; d >= 1; d >>= 1) total += __shfl_xor(total, d);
  return total;
}
// The selection over 64-bit keys of all experts, for top_k > 8 and rows with more candidates than lanes: it reads the
// row again and keeps its keys in LDS ([V][64] of the wave).  E = 0: none.
template <typename T, int LANES, int V, bool BIAS>
__device__ __forceinline__ int select_wide(const T* row, const float* bias, int E, int k, int sigmoid, int lane, float m,
                                           uint64_t* keys) {
  const int sub = lane & (LANES - 1);
  const double total = BIAS && !sigmoid ? wide_total<T, LANES, V>(row, E, sub, m) : 1.0;
#pragma unroll 1
  for (int j = 0; j < V; ++j) {
    const int e = expert_of<LANES>(sub, j);
    uint64_t key = 0;
    if (e < E) key = wide_key<BIAS>(load_logit(row + e), BIAS ? bias[e] : 0.0f, e, sigmoid, m, total);
    keys[j * 64 + lane] = key;  // (a lane reads its own alone)
  }
  int mine = -1;
#pragma unroll 1
  for (int j = 0; j < k; ++j) {
    uint64_t best = 0;
    int at = 0;  // (a lane's experts rise with i: the first of equal keys is the lower one)
#pragma unroll 4
    for (int i = 0; i < V; ++i) {
      const uint64_t key = keys[i * 64 + lane];
      at = key > best ? i : at;
      best = key > best ? key : best;
    }
    const uint32_t hi = group_max<LANES>((uint32_t)(best >> 32));
    const bool top = (uint32_t)(best >> 32) == hi;
    const uint32_t lo = group_max<LANES>(top ? (uint32_t)best : 0u);
    const int e = expert_of<LANES>(sub, at);
    const uint32_t first = group_max<LANES>(top && (uint32_t)best == lo && (hi | lo) ? (uint32_t)(kRouterMaxExperts - e) : 0u);
    const int won = kRouterMaxExperts - (int)first;
    if (sub == j && first) mine = won;
    if (first && e == won) keys[at * 64 + lane] = 0;
  }
  return mine;
}

// 32-bit keys cut from values that do not fit: steps of a range below the row's largest (the scores differ by
// at most 1; lower values share the last step, a near tie), then the index.  0 for -inf and NaN.
template <int IB, bool BIAS>
struct Cut {
  static constexpr float kTop = (float)((1u << (32 - IB)) - 256), kStep = kTop / (BIAS ? 2.0f : 32.0f);
  static __device__ __forceinline__ uint32_t key(float v, bool eligible, float off, int index) {
    const uint32_t q = (uint32_t)__builtin_amdgcn_fmed3f(fmaf(v, kStep, off), 1.0f, (float)((1u << (32 - IB)) - 1));
    const uint32_t keep = (eligible & (v > -INFINITY)) ? ~0u : 0u;  // (a mask: a choice of the whole would become a branch)
    return ((q << IB) | (uint32_t)index) & keep;
  }
};

// LDS of a wave for the candidates of a near tie: their number in each group, experts, logits, biases and 64-bit keys,
// and the choice.
struct NearTie {
  int32_t n[4];
  int32_t expert[64];
  float logit[64], bias[64];
  uint64_t key[64];
  int32_t choice[64];
};

template <typename T, int LANES, int V, bool BIAS, bool STATS>
__global__ __launch_bounds__(STATS ? kRouterStatThreads : kRouterThreads) void router_kernel(RouterArgs a, int wide) {
  constexpr int G = 64 / LANES;  // tokens of a wave at a time
  constexpr int W = (STATS ? kRouterStatThreads : kRouterThreads) / 64;
  constexpr bool EXACT = !BIAS && !std::is_same<T, float>::value;
  constexpr int IB = LANES * V <= 256 ? 8 : LANES * V <= 512 ? 9 : 10, LAST = (1 << IB) - 1;  // a key's index
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, place = lane & (LANES - 1), grp = lane / LANES;
  __shared__ int lcount[STATS ? LANES * V : 1];
  __shared__ int ltokens;
  __shared__ NearTie ties[EXACT ? 1 : W];
  __shared__ uint64_t lkeys[W][V * 64];
  float psum[V];
  int tokens = 0;
  if constexpr (STATS) {
    if (threadIdx.x == 0) ltokens = 0;
    for (int e = threadIdx.x; e < LANES * V; e += W * 64) lcount[e] = 0;
#pragma unroll
    for (int j = 0; j < V; ++j) psum[j] = 0.0f;
    if (blockIdx.x == 0 && threadIdx.x == 0) *a.totals = RouterTotals{0, 0, 0};  // (for the launch that follows)
    __syncthreads();
  }
  const int64_t step = (int64_t)gridDim.x * W * G;
  for (int64_t t0 = ((int64_t)blockIdx.x * W + wv) * G; t0 < a.M; t0 += step) {
    int sub = place;
    asm("" : "+v"(sub));  // (addresses are made anew for each token: kept over the loop they cost 80 registers)
    const int64_t t = t0 + grp;
    const bool in = t < a.M;
    const int32_t mark = a.live ? a.live[in ? t : 0] : 0;
    const T* row = reinterpret_cast<const T*>(a.logits) + (in ? t : 0) * a.ld;
    float x[V], b[V];
    load_logits<T, LANES, V>(row, sub, a.E, wide & 1, reinterpret_cast<float*>(lkeys[wv]), lane, x);
    const bool live = in && mark >= 0;
    if (a.E < LANES * V || __any(!live)) mask_logits<LANES, V>(sub, live ? a.E : 0, x);
    if constexpr (BIAS) load_logits<float, LANES, V>(a.bias, sub, a.E, wide & 4, reinterpret_cast<float*>(lkeys[wv]), lane, b);
    bool bad;
    float m = row_max<LANES, V>(x, a.sigmoid, grp, bad);
    if (BIAS && !a.sigmoid && __any(bad)) {  // (the largest beside a NaN of the same lane: biased scores depend on it)
      m = x[0];
#pragma unroll
      for (int j = 1; j < V; ++j) m = fmaxf(m, x[j]);
      m = group_max<LANES>(m);
      m = m > -INFINITY ? m : 0.0f;
    }
    float total = 0.0f, u[V];  // every expert's share, where it is needed
    if (STATS || (!a.sigmoid && (BIAS || !a.renorm))) total = row_shares<LANES, V>(x, a.sigmoid, m, u);
    // the choice: lane j of the group keeps the j-th
    float xj = -INFINITY;
    int mine = -1;
    bool wide_keys = a.k > 8;
    if (!wide_keys) {
      uint32_t key[V];
      float* stash = reinterpret_cast<float*>(lkeys[wv]) + lane;
      float off = 0.0f, inv = 0.0f;
      int tol = 4;  // steps that two keys' difference can be off by: the cut, and a rounding of what is cut
      if constexpr (EXACT) {
#pragma unroll
        for (int j = 0; j < V; ++j)
          key[j] = x[j] > -INFINITY ? (sortable(x[j]) & 0xFFFF0000u) | (uint32_t)(LAST - expert_of<LANES>(sub, j)) : 0;
      } else {
        float v[V], top = -INFINITY;
        if constexpr (BIAS) {
          inv = total > 0.0f ? __builtin_amdgcn_rcpf(total) : 0.0f;
          if (a.sigmoid) {
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = biased(x[j], b[j], 1, m, inv);
          } else {
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = biased(x[j], b[j], 0, m, inv);
          }
#pragma unroll
          for (int j = 0; j < V; ++j) top = fmaxf(top, v[j]);  // (of -inf logits too: it only places the range)
          top = group_max<LANES>(top);
          // A sigmoid is off by less than 5 * 2^-24 (its exponential by |x| 1.5 * 2^-24 and a unit, of which at most
          // 1.1 * 2^-24 remains, the sum and the reciprocal by a unit each), 2.5 steps of 2^-23; the sum
          // with the bias by half a step for each unit of `top`, the cut by two.  A softmax's row sum adds less
          // than 26 * 2^-24 that all scores share.
          tol = (a.sigmoid ? 12 : 28) + (int)fminf(2.0f * fabsf(top), 1e6f);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) v[j] = x[j];
          top = m;
        }
        off = Cut<IB, BIAS>::kTop - top * Cut<IB, BIAS>::kStep;  // (the same rounding for all of the row)
#pragma unroll
        for (int j = 0; j < V; ++j) key[j] = Cut<IB, BIAS>::key(v[j], !BIAS || x[j] > -INFINITY, off, LAST - expert_of<LANES>(sub, j));
        // (the sorting leaves no registers: logits and biases are looked up again here)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          stash[j * 64] = x[j];
          if constexpr (BIAS) stash[(V + j) * 64] = b[j];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
      const uint32_t got = nine_largest<LANES, V>(key, sub);
      const int e = LAST - (int)(got & LAST);
      mine = got && sub < a.k ? e : -1;
      if constexpr (EXACT) {
        if (mine >= 0) xj = unsortable((got & 0xFFFF0000u) | (got >> 31 ? 0u : 0xFFFFu));
      } else {
        int es, ej;
        place_of<LANES>(got ? e : 0, es, ej);
        const float xe = stash[ej * 64 + es - sub], be = BIAS ? stash[(V + ej) * 64 + es - sub] : 0.0f;
        if (mine >= 0) xj = xe;
        // neighbours that are closer than their errors, and not equal throughout (the key behind the last may hide others)
        const uint32_t after = dpp<0x101>(got);
        const bool equal = xe == __uint_as_float(dpp<0x101>(__float_as_uint(xe))) &&
                           be == __uint_as_float(dpp<0x101>(__float_as_uint(be))) && sub + 1 < a.k;
        const bool near = mine >= 0 && after && (int)((got >> IB) - (after >> IB)) <= tol && !equal;
        if (__any(near)) {
          NearTie& lt = ties[wv];
          const uint32_t kth = (uint32_t)__shfl((int)got, grp * LANES + a.k - 1) >> IB;
          const uint32_t least = kth > 2u * (uint32_t)tol ? (kth - 2u * (uint32_t)tol) << IB : 1u;
          lt.n[grp] = 0;
          lt.choice[lane] = -1;
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll 4
          for (int j = 0; j < V; ++j) {
            const int c = expert_of<LANES>(sub, j);
            const float y = stash[j * 64], z = BIAS ? stash[(V + j) * 64] : 0.0f;
            const float v = BIAS ? biased(y, z, a.sigmoid, m, inv) : y;
            if (Cut<IB, BIAS>::key(v, !BIAS || y > -INFINITY, off, LAST - c) >= least) {
              const int at = atomicAdd(&lt.n[grp], 1);
              if (at < LANES) {
                lt.expert[grp * LANES + at] = c;
                lt.logit[grp * LANES + at] = y;
                lt.bias[grp * LANES + at] = z;
              }
            }
          }
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
          const int n = lt.n[grp];
          if (__any(n > LANES)) wide_keys = true;
          else {
            const double sum = BIAS && !a.sigmoid ? wide_total<T, LANES, V>(row, live ? a.E : 0, sub, m) : 1.0;
            const int c = sub < n ? lt.expert[lane] : 0;
            const float y = sub < n ? lt.logit[lane] : -INFINITY;
            const uint64_t mykey = wide_key<BIAS>(y, lt.bias[lane], c, a.sigmoid, m, sum);
            lt.key[lane] = mykey;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            int rank = 0;
#pragma unroll
            for (int i = 0; i < LANES; ++i) rank += lt.key[grp * LANES + i] > mykey;
            if (mykey && rank <= a.k) lt.choice[grp * LANES + rank] = c;
            xj = -INFINITY;
            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
            mine = lt.choice[lane];
            // equal scores meet in one place and leave the next one empty (the one behind the last choice counts): by the index then
            if (BIAS && __any(mine < 0 && sub <= a.k && sub < n)) {
#pragma unroll
              for (int i = 0; i < LANES; ++i) rank += lt.key[grp * LANES + i] == mykey && lt.expert[grp * LANES + i] < c;
              if (mykey && rank < a.k) lt.choice[grp * LANES + rank] = c;
              __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
              mine = lt.choice[lane];
            }
            mine = sub < a.k ? mine : -1;
            int ps, pj;
            place_of<LANES>(max(mine, 0), ps, pj);
            if (mine >= 0) xj = stash[pj * 64 + ps - sub];
          }
        }
      }
    }
    if (wide_keys) {
      mine = select_wide<T, LANES, V, BIAS>(row, a.bias, live ? a.E : 0, a.k, a.sigmoid, lane, m, lkeys[wv]);
      xj = mine >= 0 ? load_logit(row + mine) : -INFINITY;
    }
    const bool has = mine >= 0;
    float w = 0.0f;
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
      const float share = bad ? NAN : (total > 0.0f ? 1.0f / total : 0.0f);
#pragma unroll
      for (int j = 0; j < V; ++j) psum[j] = live ? fmaf(u[j], share, psum[j]) : psum[j];
      if (has) atomicAdd(&lcount[mine], 1);
      tokens += live && sub == 0;
    }
  }
  if constexpr (STATS) {
    if (tokens) atomicAdd(&ltokens, tokens);
    float* sums = reinterpret_cast<float*>(lkeys[0]);  // (of every wave and lane, where its keys were)
#pragma unroll
    for (int j = 0; j < V; ++j) sums[(wv * V * 2 + j) * 64 + lane] = psum[j];
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += W * 64) {
      int s, j;
      place_of<LANES>(e, s, j);
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < W; ++i)
#pragma unroll
        for (int g = 0; g < G; ++g) v += sums[(i * V * 2 + j) * 64 + g * LANES + s];
      a.part_sum[(int64_t)blockIdx.x * a.E + e] = v;
      a.part_count[(int64_t)blockIdx.x * a.E + e] = lcount[e];
    }
    if (threadIdx.x == 0) a.part_tokens[blockIdx.x] = ltokens;
  }
}

// The workgroups' partial sums to counts, mean probabilities and the loss.  A workgroup takes 16 experts and adds its
// share of the loss to the totals as an integer (in any order the same); the last one to arrive makes the loss of
// them.  Only atomics carry what it reads, so no workgroup has to write its caches back.
__global__ __launch_bounds__(256) void router_stats_kernel(const float* part_sum, const int32_t* part_count,
                                                           const int32_t* part_tokens, int parts, int E, int top_k,
                                                           int32_t* counts, float* means, float* balance,
                                                           int32_t* tokens, RouterTotals* totals) {
  const int tid = threadIdx.x, col = tid & 15, row = tid >> 4, e = blockIdx.x * 16 + col;
  __shared__ double dsum[16][17];
  __shared__ int icount[16][17];
  __shared__ int red[4];
  double s = 0.0;
  int n = 0, tok = 0;
  float v[kRouterParts / 16];
  int c[kRouterParts / 16];
#pragma unroll
  for (int i = 0; i < kRouterParts / 16; ++i) {  // (all asked for at once; places that are not there are dropped below)
    const int64_t at = (int64_t)min(row + i * 16, parts - 1) * E + min(e, E - 1);
    v[i] = part_sum[at];
    c[i] = part_count[at];
  }
  tok = part_tokens[min(tid, parts - 1)];
  if (tid >= parts) tok = 0;
#pragma unroll
  for (int i = 0; i < kRouterParts / 16; ++i)
    if (row + i * 16 < parts && e < E) {
      s += (double)v[i];
      n += c[i];
    }
  for (int d = 32; d >= 1; d >>= 1) tok += __shfl_xor(tok, d);
  if ((tid & 63) == 0) red[tid >> 6] = tok;
  dsum[row][col] = s;
  icount[row][col] = n;
  __syncthreads();
  if (row > 0) return;
  tok = red[0] + red[1] + red[2] + red[3];
  s = 0.0;
  n = 0;
  for (int i = 0; i < 16; ++i) {
    s += dsum[i][col];
    n += icount[i][col];
  }
  const double mean = tok ? s / (double)tok : 0.0;
  if (e < E) {
    counts[e] = n;
    means[e] = (float)mean;
  }
  double share = e < E ? (double)n * mean : 0.0;
  for (int d = 8; d >= 1; d >>= 1) {
    share += __shfl_xor(share, d);
    n += __shfl_xor(n, d);
  }
  if (col) return;
  if (blockIdx.x == 0) *tokens = tok;
  const double unit = 0x1p60 / ((double)max(tok, 1) * (double)top_k);
  const bool bad = !(share == share);
  __hip_atomic_fetch_add(&totals->loss, bad ? 0ull : (uint64_t)(share * unit), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  __hip_atomic_fetch_add(&totals->slots, (uint32_t)n, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // (both have been performed before this one is counted)
  const uint32_t before = __hip_atomic_fetch_add(&totals->arrived, bad ? 0x10001u : 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  if ((before & 0xFFFFu) != gridDim.x - 1) return;
  const uint64_t all = __hip_atomic_fetch_add(&totals->loss, 0ull, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  const uint32_t slots = __hip_atomic_fetch_add(&totals->slots, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  *balance = bad || before >> 16 ? NAN : (float)((double)all / unit * (double)E / (double)max(slots, 1u));
}

// dx = the router's gradient + the balance loss's, one write of the row.  With q the probabilities, h the
// chosen shares (w = scale * h) and a_e = (d_means[e] + d_balance * E * n_e / sum n) / tokens:
//   loss      q_e (a_e - sum a q), times 1 - s_e for sigmoid scores
//   weights   renormalised: scale * h_j (dw_j - sum dw h), times 1 - s_j for sigmoid scores
//             softmax: scale * p_e ([e chosen] dw_e - sum dw p);  sigmoid: scale * s_j (1 - s_j) dw_j
// The chosen entries reach the lanes that hold their experts through LDS.  All of a token's loads are asked for before
// the first is waited on.
template <typename T, int LANES, int V>
__global__ __launch_bounds__(256) void router_grad_kernel(RouterGradArgs a, int wide) {
  constexpr int G = 64 / LANES;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, sub = lane & (LANES - 1), grp = lane / LANES;
  __shared__ float chosen[4][V][64];
  __shared__ int red[4];
  const bool loss = a.d_balance || a.d_means;
  const int64_t t = ((int64_t)blockIdx.x * 4 + wv) * G + grp;
  const bool in = t < a.M;
  const int64_t tc = in ? t : 0;
  const int32_t mark = a.live ? a.live[tc] : 0;
  const T* row = reinterpret_cast<const T*>(a.logits) + tc * a.ld;
  float x[V], coef[V];
  load_logits<T, LANES, V>(row, sub, a.E, wide & 1, &chosen[wv][0][0], lane, x);
  int id = -1;
  float dw = 0.0f;
  if (a.dw) {
    const int64_t at = tc * a.k + min(sub, a.k - 1);
    id = a.ids[at];
    dw = a.dw[at];
  }
#pragma unroll
  for (int j = 0; j < V; ++j) coef[j] = 0.0f;
  if (loss) {
    int all = 0;
    for (int e = threadIdx.x; e < a.E; e += 256) all += a.counts[e];
#pragma unroll
    for (int j = 0; j < V; ++j) coef[j] = (float)a.counts[min(expert_of<LANES>(sub, j), a.E - 1)];
    const float tokens = (float)max(*a.tokens, 1);
    for (int d = 32; d >= 1; d >>= 1) all += __shfl_xor(all, d);
    if (lane == 0) red[wv] = all;
    __syncthreads();
    all = red[0] + red[1] + red[2] + red[3];
    const float share = a.d_balance ? *a.d_balance * ((float)a.E / (float)max(all, 1)) : 0.0f;
    const float inv = 1.0f / tokens;
#pragma unroll
    for (int j = 0; j < V; ++j) coef[j] *= share * inv;
    if (a.d_means) {
#pragma unroll
      for (int j = 0; j < V; ++j) coef[j] = fmaf(a.d_means[min(expert_of<LANES>(sub, j), a.E - 1)], inv, coef[j]);
    }
  }
  const bool live = in && mark >= 0;
  if (!live || sub >= a.k || id >= a.E) id = -1;
  const float xj = id >= 0 ? load_logit(row + id) : -INFINITY;
  if (a.E < LANES * V || __any(!live)) mask_logits<LANES, V>(sub, live ? a.E : 0, x);
  bool bad;
  const float m = row_max<LANES, V>(x, a.sigmoid, grp, bad);
  float q[V], total = 0.0f, aq = 0.0f;
  const bool dense = loss || (!a.renorm && !a.sigmoid);
  if (dense) {
    total = row_shares<LANES, V>(x, a.sigmoid, m, q);
    const float inv = total > 0.0f ? 1.0f / total : 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      q[j] *= inv;
      aq = fmaf(coef[j], q[j], aq);
    }
    aq = group_sum<LANES>(aq);
  }
  // the chosen entries: lane j holds the j-th
#pragma unroll
  for (int j = 0; j < V; ++j) chosen[wv][j][lane] = 0.0f;
  float rest = 0.0f;  // scale * sum dw p of a softmax over all experts
  if (a.dw) {
    float h = 0.0f, slope = 1.0f;
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
    if (has) {
      int s, j;
      place_of<LANES>(id, s, j);
      atomicAdd(&chosen[wv][j][grp * LANES + s], d);
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  if (!in) return;
  float out[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float v = chosen[wv][j][lane];
    if (dense) {
      float g = coef[j] - aq;
      if (a.sigmoid) {
        const float z = exp_neg(-fabsf(x[j]));
        g *= (x[j] >= 0.0f ? z : 1.0f) * __builtin_amdgcn_rcpf(1.0f + z);
      }
      v = x[j] > -INFINITY ? fmaf(q[j], g - rest, v) : v;  // (0 of padding and of -inf, also where g is not finite)
    }
    out[j] = bad ? NAN : v;
  }
  T* o = reinterpret_cast<T*>(a.dx) + t * a.ld_d;
  if (wide & 2) {
#pragma unroll
    for (int c = 0; c < V; c += 4) {
      const int e = expert_of<LANES>(sub, c);
      if (e >= a.E) continue;
      if constexpr (std::is_same<T, float>::value)
        *reinterpret_cast<float4*>(o + e) = make_float4(out[c], out[c + 1], out[c + 2], out[c + 3]);
      else
        *reinterpret_cast<uint2*>(o + e) = make_uint2(pack_bf16x2(out[c], out[c + 1]), pack_bf16x2(out[c + 2], out[c + 3]));
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < V; ++j) chosen[wv][j][lane] = out[j];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  const float* from = &chosen[wv][0][0] + turned_place(sub, lane);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int e = j * LANES + sub;
    const float v = from[turned_step<LANES>(j)];
    if (e >= a.E) continue;
    if constexpr (std::is_same<T, float>::value) o[e] = v;
    else o[e] = f32_to_bf16(v);
  }
}

// f(lanes, values a lane) of the layout that holds E experts.
template <typename F>
static void router_layout(int E, F f) {
  using std::integral_constant;
  if (E <= 64) f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
  else if (E <= 128) f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
  else if (E <= 192) f(integral_constant<int, 16>{}, integral_constant<int, 12>{});
  else if (E <= 256) f(integral_constant<int, 16>{}, integral_constant<int, 16>{});
  else if (E <= 512) f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
  else f(integral_constant<int, 64>{}, integral_constant<int, 16>{});
}
static int router_group(int E) { return E <= 256 ? 16 : E <= 512 ? 32 : 64; }
// workgroups of `threads` threads that take every token once, and the workgroups that leave partial sums
static int64_t router_blocks(int64_t M, int E, int threads) {
  const int64_t per = threads / router_group(E);
  return (M + per - 1) / per;
}
static int64_t router_parts(int64_t M, int E) {
  return std::max<int64_t>(1, std::min<int64_t>(router_blocks(M, E, kRouterStatThreads), kRouterParts));
}
static int64_t router_bytes(int64_t M, int E) { return (int64_t)sizeof(RouterTotals) + router_parts(M, E) * (8 * (int64_t)E + 4); }

template <typename T>
static void launch_router(const RouterArgs& a, unsigned grid, bool stats, int wide, hipStream_t st) {
  router_layout(a.E, [&](auto lanes, auto v) {
    constexpr int LN = decltype(lanes)::value, V = decltype(v)::value;
    const dim3 g(grid), b(stats ? kRouterStatThreads : kRouterThreads);
    if (a.bias && stats) hipLaunchKernelGGL((router_kernel<T, LN, V, true, true>), g, b, 0, st, a, wide);
    else if (a.bias) hipLaunchKernelGGL((router_kernel<T, LN, V, true, false>), g, b, 0, st, a, wide);
    else if (stats) hipLaunchKernelGGL((router_kernel<T, LN, V, false, true>), g, b, 0, st, a, wide);
    else hipLaunchKernelGGL((router_kernel<T, LN, V, false, false>), g, b, 0, st, a, wide);
  });
}
template <typename T>
static void launch_router_grad(const RouterGradArgs& a, unsigned grid, int wide, hipStream_t st) {
  router_layout(a.E, [&](auto lanes, auto v) {
    hipLaunchKernelGGL((router_grad_kernel<T, decltype(lanes)::value, decltype(v)::value>), dim3(grid), dim3(256), 0, st, a, wide);
  });
}

// Rows that can be read four logits at a time.
static bool wide_rows(const void* p, int64_t ld, int E, bool f32) {
  return ((uintptr_t)p & (f32 ? 15 : 7)) == 0 && ld % 4 == 0 && E % 4 == 0;
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
  *bytes = router_bytes(M, E);
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
    MOE_REQUIRE(work_bytes >= router_bytes(M, E), MOE_ESIZE, "moe_router: workspace of %lld bytes, need %lld",
                (long long)work_bytes, (long long)router_bytes(M, E));
    MOE_REQUIRE(((uintptr_t)work & 7) == 0 && (((uintptr_t)counts | (uintptr_t)means | (uintptr_t)balance | (uintptr_t)tokens) & 3) == 0,
                MOE_EUNSUPPORTED, "moe_router: the workspace must be 8-byte, the statistics 4-byte aligned");
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
    a.totals = (RouterTotals*)work;
    a.part_tokens = (int32_t*)(a.totals + 1);
    a.part_sum = (float*)(a.part_tokens + parts);
    a.part_count = (int32_t*)(a.part_sum + parts * E);
  }
  const int wide = wide_rows(logits, ld, E, logits_f32) | (wide_rows(bias, E, E, true) << 2);
  const unsigned grid = (unsigned)(stats ? parts : router_blocks(M, E, kRouterThreads));
  if (logits_f32) launch_router<float>(a, grid, stats, wide, stream);
  else launch_router<uint16_t>(a, grid, stats, wide, stream);
  if (stats)
    hipLaunchKernelGGL(router_stats_kernel, dim3((E + 15) / 16), dim3(256), 0, stream, a.part_sum, a.part_count,
                       a.part_tokens, (int)parts, E, top_k, counts, means, balance, tokens, a.totals);
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
  const unsigned grid = (unsigned)router_blocks(M, E, 256);
  if (logits_f32) launch_router_grad<float>(a, grid, wide, stream);
  else launch_router_grad<uint16_t>(a, grid, wide, stream);
  return check_launch("moe_router_grad");
}
