// Routing of tokens to experts, and the order of the routed rows.
//
// moe_route_kernel: p = softmax(z) or 1 / (1 + exp(-z)); an expert's value is p + bias, or its logit without a bias
// (p grows with it); of equal groups of experts those with the largest sums of their one or two largest
// values stay; then the top_k largest values, equal ones lowest expert first; weights p (/ their sum) * scale.
// One warp per token, the logits in registers.  Which experts are chosen must not hang on how p was rounded: two
// values may lie closer than FP32 tells apart.  Where p enters such a comparison it is held as a
// sum of two FP32 numbers (about 2^-45 of 1; RouteFF), whose order as (high, low) is the values' order; where logits are compared
// they are exact as they are.  FP64 has no units to speak of on this GPU.
//
// moe_rows_kernel: the stable counting sort of (token, choice) pairs by expert.  See there.
#pragma once

#include "cluster.cuh"
#include "serving_common.cuh"

namespace bsq {

constexpr int kRouteWarps = 4, kRouteMaxExperts = 1024, kRouteMaxTopK = 16, kRouteMaxGroups = 32;

struct RouteArgs {
  const void* logits;
  int64_t ld;
  int64_t tokens;
  const float* bias;  // may be null
  int experts, top_k, groups, top_groups, group_top;
  int per, span_log;  // experts per group, and lanes that share its values (a power of two)
  uint32_t inv;       // 2^20 / per, rounded up: e * inv >> 20 is the group of expert e, for e up to 1024
  int sigmoid, renorm;
  float scale;
  int32_t* ids;
  float* weights;
  unsigned int* err;
};

// A sum of two FP32 numbers, |l| at most half a unit of h.  Sums and products by the classical error-free
// transformations (Knuth's two-sum, Dekker's fast two-sum, the product's error by a fused multiply-add).
struct RouteFF {
  float h, l;
};
__device__ __forceinline__ RouteFF ff_fast(float a, float b) {  // |a| >= |b|
  const float s = __fadd_rn(a, b);
  return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ RouteFF ff_two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t))};
}
__device__ __forceinline__ RouteFF ff_add(RouteFF a, RouteFF b) {
  const RouteFF s = ff_two_sum(a.h, b.h);
  return ff_fast(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ RouteFF ff_mul(RouteFF a, RouteFF b) {
  const float p = __fmul_rn(a.h, b.h);
  return ff_fast(p, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.h, -p))));
}
// 1 / b for b between 1 and 2^20: an approximate reciprocal r and one Newton step, r (1 + e) with e = 1 - b r (its square is lost).
__device__ __forceinline__ RouteFF ff_inverse(RouteFF b) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(b.h));
  const float e = __fmaf_rn(-b.l, r, __fmaf_rn(-b.h, r, 1.f));
  return ff_fast(r, __fmul_rn(r, e));
}
__device__ __forceinline__ bool ff_greater(RouteFF a, RouteFF b) { return a.h > b.h || (a.h == b.h && a.l > b.l); }

// 2^(j/32), j = 0..31.
__device__ const float kRouteExp2[64] = {
    0x1.000000p+0f, 0x0.0p+0f, 0x1.059b0ep+0f, -0x1.9d4f52p-25f, 0x1.0b5586p+0f, 0x1.9f3122p-25f, 0x1.11301ep+0f, -0x1.fdb496p-25f,
    0x1.172b84p+0f, -0x1.c15742p-27f, 0x1.1d4874p+0f, -0x1.d2e8cap-25f, 0x1.2387a6p+0f, 0x1.ceac48p-25f, 0x1.29e9e0p+0f, -0x1.5c0424p-25f,
    0x1.306fe0p+0f, 0x1.4636e2p-25f, 0x1.371a74p+0f, -0x1.18aac6p-25f, 0x1.3dea64p+0f, 0x1.824684p-25f, 0x1.44e086p+0f, 0x1.8624b4p-30f,
    0x1.4bfdaep+0f, -0x1.593abcp-25f, 0x1.5342b6p+0f, -0x1.2c5610p-25f, 0x1.5ab07ep+0f, -0x1.5bd5ecp-27f, 0x1.6247ecp+0f, -0x1.f8b550p-25f,
    0x1.6a09e6p+0f, 0x1.9fcef4p-26f, 0x1.71f75ep+0f, 0x1.1d8beep-25f, 0x1.7a1148p+0f, -0x1.829fd0p-25f, 0x1.82589ap+0f, -0x1.accc7cp-26f,
    0x1.8ace54p+0f, 0x1.15506ep-27f, 0x1.93737cp+0f, -0x1.e64744p-25f, 0x1.9c4918p+0f, 0x1.51f848p-27f, 0x1.a5503cp+0f, -0x1.b83b54p-25f,
    0x1.ae89fap+0f, -0x1.a94b14p-26f, 0x1.b7f770p+0f, -0x1.a09438p-25f, 0x1.c199bep+0f, -0x1.3d56b2p-27f, 0x1.cb720ep+0f, -0x1.8837ccp-27f,
    0x1.d5818ep+0f, -0x1.822dbcp-27f, 0x1.dfc974p+0f, -0x1.908c94p-25f, 0x1.ea4afap+0f, 0x1.52486cp-27f, 0x1.f50766p+0f, -0x1.246eb0p-26f};

// exp(x) for x <= 0, by Tang's table method: x = k ln2/32 + r, 2^(k/32) from lane k mod 32's `tab`, exp(r) by its series
// to r^5 (|r| <= 0.011), the first two terms in two numbers.  Every lane of the warp calls.
__device__ __forceinline__ RouteFF ff_exp(RouteFF x, RouteFF tab) {
  const float xh = fmaxf(x.h, -110.f), xl = x.h < -110.f ? 0.f : x.l;
  const float k = rintf(__fmul_rn(xh, 46.16624130844683f));
  // ln2/32 in parts of 12, 12 and 24 bits: the first two products are exact, and so is the first difference
  const RouteFF s = ff_two_sum(__fsub_rn(xh, __fmul_rn(k, 0x1.62ep-6f)), -__fmul_rn(k, 0x1.0bep-20f));
  const RouteFF r = ff_fast(s.h, __fmaf_rn(-k, 0x1.be8e7cp-32f, __fadd_rn(s.l, xl)));
  const float q = __fmul_rn(r.h, r.h), qe = __fmaf_rn(r.h, r.h, -q);
  const float tail = __fmul_rn(__fmul_rn(q, r.h), fmaf(r.h, fmaf(r.h, 1.f / 120.f, 1.f / 24.f), 1.f / 6.f));
  const RouteFF t = ff_two_sum(r.h, 0.5f * q);
  RouteFF e = ff_two_sum(1.f, t.h);
  e = ff_fast(e.h, __fadd_rn(e.l, __fadd_rn(t.l, __fadd_rn(tail, __fmaf_rn(r.h, r.l, __fadd_rn(r.l, 0.5f * qe))))));
  const int ki = static_cast<int>(k);
  e = ff_mul(e, RouteFF{__shfl_sync(~0u, tab.h, ki & 31), __shfl_sync(~0u, tab.l, ki & 31)});
  const int n = ki >> 5;  // down to -159: in two steps
  const float f = __uint_as_float(static_cast<uint32_t>(127 + n / 2) << 23), g = __uint_as_float(static_cast<uint32_t>(127 + n - n / 2) << 23);
  return {__fmul_rn(__fmul_rn(e.h, f), g), __fmul_rn(__fmul_rn(e.l, f), g)};
}

// Order-preserving keys: larger numbers have larger keys; -0 counts as 0.
__device__ __forceinline__ uint32_t route_key(float z) {
  const uint32_t u = __float_as_uint(z + 0.0f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float route_unkey(uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k); }

// What the choice of groups does with values: one FP32 number, or two.
template <typename V> struct RouteNum;
template <> struct RouteNum<float> {
  static __device__ __forceinline__ float least() { return -INFINITY; }
  static __device__ __forceinline__ float leading(float a) { return a; }
  static __device__ __forceinline__ bool greater(float a, float b) { return a > b; }
  static __device__ __forceinline__ bool equal(float a, float b) { return a == b; }
  static __device__ __forceinline__ float sum(float a, float b) { return a + b; }
  static __device__ __forceinline__ float shuffle(float a, int lane) { return __shfl_sync(~0u, a, lane); }
  static __device__ __forceinline__ float shuffle_xor(float a, int d) { return __shfl_xor_sync(~0u, a, d); }
};
template <> struct RouteNum<RouteFF> {
  static __device__ __forceinline__ RouteFF least() { return {-INFINITY, 0.f}; }
  static __device__ __forceinline__ float leading(RouteFF a) { return a.h; }
  static __device__ __forceinline__ bool greater(RouteFF a, RouteFF b) { return ff_greater(a, b); }
  static __device__ __forceinline__ bool equal(RouteFF a, RouteFF b) { return a.h == b.h && a.l == b.l; }
  static __device__ __forceinline__ RouteFF sum(RouteFF a, RouteFF b) {
    return a.h > -INFINITY && b.h > -INFINITY ? ff_add(a, b) : least();
  }
  static __device__ __forceinline__ RouteFF shuffle(RouteFF a, int lane) {
    return {__shfl_sync(~0u, a.h, lane), __shfl_sync(~0u, a.l, lane)};
  }
  static __device__ __forceinline__ RouteFF shuffle_xor(RouteFF a, int d) {
    return {__shfl_xor_sync(~0u, a.h, d), __shfl_xor_sync(~0u, a.l, d)};
  }
};

// One logit as FP32; DTYPE is a bsq_dtype.
template <int DTYPE>
__device__ __forceinline__ float route_load(const void* row, int e) {
  if constexpr (DTYPE == 2) return __ldg(static_cast<const float*>(row) + e);
  return elem2_to_f32x2<DTYPE == 1>(__ldg(static_cast<const uint16_t*>(row) + e)).x;
}

// The top_k largest keys, in order, equal ones lowest expert (32 slot + lane) first: lane k gets the k-th's expert, and the keys
// become 0.  `margin`: the least distance of neighbours among them and the next one, of their leading 32 bits' numbers;
// `least`: those of the last one.  Every lane does the same work in every round: a branch for the lane that holds the winner costs more.
template <int NL, typename K>
__device__ __forceinline__ int route_select(K (&key)[NL], int top_k, int lane, float& margin, float& least) {
  int my_id = 0;
  margin = INFINITY;
  least = INFINITY;
#pragma unroll 1
  for (int k = 0; k <= top_k; ++k) {
    K best = key[0], top;
#pragma unroll
    for (int i = 1; i < NL; ++i) best = max(best, key[i]);
    if constexpr (sizeof(K) == 8) {
      const uint32_t hi = __reduce_max_sync(~0u, static_cast<uint32_t>(best >> 32));
      const uint32_t lo = __reduce_max_sync(~0u, static_cast<uint32_t>(best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
      top = static_cast<K>(hi) << 32 | lo;
    } else {
      top = __reduce_max_sync(~0u, best);
    }
    uint32_t leading;
    if constexpr (sizeof(K) == 8) leading = static_cast<uint32_t>(top >> 32); else leading = top;
    const float value = leading != 0u ? route_unkey(leading) : -INFINITY;
    if (value > -INFINITY) margin = fminf(margin, least - value);
    if (k == top_k) break;
    least = value;
    uint32_t at = ~0u;
#pragma unroll
    for (int i = NL - 1; i >= 0; --i)
      if (key[i] == top) at = 32 * i + lane;
    const uint32_t id = __reduce_min_sync(~0u, at);
    if (lane == k) my_id = static_cast<int>(id);
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (32 * i + lane == static_cast<int>(id)) key[i] = 0;
  }
  return my_id;
}

// The groups that stay, group g's bit at g times the power of two span_log: the lanes share the groups out, `v` holds the experts' values in shared memory.  `margin`:
// how far the least score that stays lies above the largest that does not.
template <typename V>
__device__ __forceinline__ uint32_t route_groups(const RouteArgs& a, const V* v, int lane, float& margin) {
  const int span = 1 << a.span_log;  // lanes per group
  const int g = lane >> a.span_log, part = lane & (span - 1), per = a.per;
  V first = RouteNum<V>::least(), second = first;
  if (g < a.groups)
#pragma unroll 4
    for (int j = part; j < per; j += span) {
      const V x = v[g * per + j];
      if (RouteNum<V>::greater(x, first)) {
        second = first;
        first = x;
      } else if (RouteNum<V>::greater(x, second)) {
        second = x;
      }
    }
  for (int d = 1; d < span; d <<= 1) {
    const V f = RouteNum<V>::shuffle_xor(first, d), s = RouteNum<V>::shuffle_xor(second, d);
    if (RouteNum<V>::greater(f, first)) {
      second = RouteNum<V>::greater(first, s) ? first : s;
      first = f;
    } else if (RouteNum<V>::greater(f, second)) {
      second = f;
    }
  }
  V score = first;
  if (a.group_top == 2 && per > 1) score = RouteNum<V>::sum(first, second);
  int before = 0;
#pragma unroll 4
  for (int o = 0; o < a.groups; ++o) {
    const V s = RouteNum<V>::shuffle(score, o * span);
    before += RouteNum<V>::greater(s, score) || (o < g && RouteNum<V>::equal(s, score));
  }
  const bool there = g < a.groups && part == 0, stays = there && before < a.top_groups;
  const uint32_t votes = __ballot_sync(~0u, stays);
  const uint32_t low = __reduce_min_sync(~0u, stays ? route_key(RouteNum<V>::leading(score)) : ~0u);
  const uint32_t high = __reduce_max_sync(~0u, there && !stays ? route_key(RouteNum<V>::leading(score)) : 0u);
  margin = high == 0u || route_unkey(high) == -INFINITY ? INFINITY : route_unkey(low) - route_unkey(high);
  return votes;
}

// Whether expert e's group stays.
__device__ __forceinline__ bool route_kept(const RouteArgs& a, uint32_t kept, uint32_t e) { return kept >> (((e * a.inv) >> 20) << a.span_log) & 1u; }

// A logit or bias that takes part: NaN and +inf count as -inf.
__device__ __forceinline__ float route_clean(float x) { return x < INFINITY ? x : -INFINITY; }

// exp of a logit less `top` (softmax), or 1 / (1 + exp(-z)) (sigmoid: exp(min(z, 0)) / (1 + exp(-|z|))).  Every lane calls.
__device__ __forceinline__ RouteFF route_score(float z, float top, int sigmoid, RouteFF tab) {
  const bool off = !(z > -INFINITY);
  RouteFF v = ff_exp(off ? RouteFF{0.f, 0.f} : sigmoid ? RouteFF{-fabsf(z), 0.f} : ff_two_sum(z, -top), tab);
  if (sigmoid) {
    const RouteFF s = ff_fast(1.f, v.h), r = ff_inverse(ff_fast(s.h, __fadd_rn(s.l, v.l)));
    v = z >= 0.f ? r : ff_mul(v, r);
  }
  return off ? RouteFF{0.f, 0.f} : v;
}
// 1 for the sigmoid, 1 / the sum of all experts' exponentials (at least 1 where a logit is there) for the softmax.
template <int DTYPE>
__device__ __forceinline__ RouteFF route_factor(const RouteArgs& a, const void* row, float top, RouteFF tab, int lane) {
  if (a.sigmoid) return {1.f, 0.f};
  RouteFF sum = {0.f, 0.f};
#pragma unroll 2
  for (int e0 = 0; e0 < a.experts; e0 += 32)
    sum = ff_add(sum, route_score(e0 + lane < a.experts ? route_clean(route_load<DTYPE>(row, e0 + lane)) : -INFINITY, top, 0, tab));
#pragma unroll 1
  for (int d = 16; d > 0; d >>= 1) sum = ff_add(sum, RouteFF{__shfl_xor_sync(~0u, sum.h, d), __shfl_xor_sync(~0u, sum.l, d)});
  return sum.h > 0.f ? ff_inverse(sum) : RouteFF{0.f, 0.f};
}
// The value of an expert: its score times the factor, plus its bias.
__device__ __forceinline__ RouteFF route_value(RouteFF score, RouteFF factor, float z, const float* bias, int e) {
  RouteFF v = ff_mul(score, factor);
  if (bias) {
    const float b = route_clean(__ldg(bias + e));
    const RouteFF s = ff_two_sum(v.h, b);
    v = ff_fast(s.h, __fadd_rn(s.l, v.l));
    if (!(b > -INFINITY) || !(z > -INFINITY)) v = {-INFINITY, 0.f};
  }
  return v;
}

// The choice among the experts that FP32 leaves open (`count` of them, at most 32, lane j's in `mine`): their values in two numbers, and each
// one's place by counting those in front.  `out`: shared memory for the top_k.
template <int DTYPE>
__device__ __noinline__ int route_near(const RouteArgs& a, const void* row, int32_t* out, float top, int lane, int mine, int count) {
  const RouteFF tab = {kRouteExp2[2 * lane], kRouteExp2[2 * lane + 1]};
  const RouteFF factor = route_factor<DTYPE>(a, row, top, tab, lane);
  const bool in = lane < count;
  const float z = in ? route_clean(route_load<DTYPE>(row, mine)) : -INFINITY;
  const RouteFF score = route_score(z, top, a.sigmoid, tab);
  const RouteFF v = in ? route_value(score, factor, z, a.bias, mine) : RouteFF{-INFINITY, 0.f};
  int before = 0;
#pragma unroll 4
  for (int o = 0; o < count; ++o) {
    const RouteFF x = {__shfl_sync(~0u, v.h, o), __shfl_sync(~0u, v.l, o)};
    const int id = __shfl_sync(~0u, mine, o);
    before += ff_greater(x, v) || (x.h == v.h && x.l == v.l && id < mine);
  }
  __syncwarp();
  if (in && before < a.top_k) out[before] = mine;
  __syncwarp();
  return lane < a.top_k ? out[lane] : 0;
}

// The choice with all values in two numbers, where the groups' order or more than 32 experts are open: once in many thousand
// tokens, so small rather than fast.
template <int DTYPE, int NL>
__device__ __noinline__ int route_exact(const RouteArgs& a, const void* row, RouteFF* values, float top, int lane) {
  const RouteFF tab = {kRouteExp2[2 * lane], kRouteExp2[2 * lane + 1]};
  const RouteFF factor = route_factor<DTYPE>(a, row, top, tab, lane);
#pragma unroll 1
  for (int e0 = 0; e0 < a.experts; e0 += 32) {
    const int e = e0 + lane;
    const float z = e < a.experts ? route_clean(route_load<DTYPE>(row, e)) : -INFINITY;
    const RouteFF score = route_score(z, top, a.sigmoid, tab);
    if (e < a.experts) values[e] = route_value(score, factor, z, a.bias, e);
  }
  __syncwarp();
  float margin, least;
  const uint32_t kept = a.groups > 1 ? route_groups(a, values, lane, margin) : 1u;
  uint64_t key[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int e = 32 * i + lane;
    key[i] = 0;
    if (e < a.experts) {
      RouteFF v = a.bias ? values[e] : RouteFF{route_clean(route_load<DTYPE>(row, e)), 0.f};
      if (!route_kept(a, kept, e)) v = {-INFINITY, 0.f};
      key[i] = static_cast<uint64_t>(route_key(v.h)) << 32 | route_key(v.l);
    }
  }
  return route_select<NL>(key, a.top_k, lane, margin, least);
}

// Measured, 8 of 256 experts: 64 tokens by softmax 2.6 us, one token by sigmoid with bias and groups 3.9 us; 4096 tokens of those 9.6 us (10.9 with
// logits from DRAM), of plain softmax 5.3 (6.5); 16384 tokens 28.1.  4096 tokens are bound by a warp's own chain, since all of their warps are on the GPU at
// once: issuing their instructions (about 1350 a token) alone would take 4.4 us, and the counters show fixed latency and 35 % of the SMs' throughput; 16384
// tokens are nearer the issue rate (18 us).  The chain: the nine rounds of the choice (2.7 us of 10.9 before the kept groups' experts were put side by
// side, which takes 10.4 to 9.6), the groups (1.8), tokens that are chosen again (0.9), a launch (2); DRAM's part is 0.7 us.
// All values in two numbers from the start, in place of FP32 first: 18.8 us, one token 7.9.  Slots for 128 and 512 experts: 9.2 -> 7.2 and 26.6 -> 18.1.
//
// NL: logits per lane (expert 32 i + lane in slot i).  PAIR: p enters the comparison (a bias, or sums of two in groups).
//
// p is then computed in FP32 first, off by at most some 2^-20 of the largest score; where no two values whose order
// matters lie closer than that allows, the choice is the exact one, and otherwise (about one token in a hundred, at random) it is made again
// with two numbers per value, among the few experts that are open.
template <int DTYPE, int NL, bool PAIR>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const RouteArgs a) {
  extern __shared__ RouteFF route_smem[];  // [warps][experts], with groups or PAIR
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  RouteFF* const values = route_smem + warp * a.experts;
  float* const plain = reinterpret_cast<float*>(values);
  pdl_wait();
  if (token >= a.tokens) return;
  const void* row = static_cast<const char*>(a.logits) + token * a.ld * (DTYPE == 2 ? 4 : 2);

  float z[NL], v[NL];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int e = 32 * i + lane;
    const float x = e < a.experts ? route_load<DTYPE>(row, e) : -INFINITY;
    z[i] = route_clean(x);
    bad |= !(x < INFINITY);
  }
  if constexpr (PAIR) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int e = 32 * i + lane;
      const float x = a.bias && e < a.experts ? __ldg(a.bias + e) : 0.f;
      v[i] = route_clean(x);
      bad |= !(x < INFINITY);
    }
  }
  if (__any_sync(~0u, bad) && lane == 0) record_error_at(a.err, kErrValue);
  float top = -INFINITY, total = 1.f;  // of the softmax
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < NL; ++i) top = fmaxf(top, z[i]);
    top = route_unkey(__reduce_max_sync(~0u, route_key(top)));
  }
  float tol = 0x1p-19f;  // twice what two values may be off
  if (PAIR || (!a.sigmoid && !a.renorm)) {
    float p[NL], sum = 0.f;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const float e = expf(a.sigmoid ? -z[i] : z[i] - top);
      p[i] = !(z[i] > -INFINITY) ? 0.f : a.sigmoid ? __fdividef(1.f, 1.f + fminf(e, 0x1p100f)) : e;
      sum += p[i];
    }
    float factor = 1.f;
    if (!a.sigmoid) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
      total = sum;
      factor = sum > 0.f ? __fdividef(1.f, sum) : 0.f;
      tol = 0x1p-17f * factor;  // scores are at most this factor
    }
    if constexpr (PAIR) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int e = 32 * i + lane;
        const float s = p[i] * factor;
        v[i] = z[i] > -INFINITY || !a.bias ? s + v[i] : -INFINITY;
        if (a.groups > 1 && e < a.experts) plain[e] = v[i];
        if (!a.bias) v[i] = z[i];
      }
    }
  }
  if constexpr (!PAIR) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      v[i] = z[i];
      if (a.groups > 1 && 32 * i + lane < a.experts) plain[32 * i + lane] = z[i];
    }
  }

  float group_margin = INFINITY, margin, least;
  uint32_t kept = 1u;
  if (a.groups > 1) {
    __syncwarp();
    kept = route_groups(a, plain, lane, group_margin);
  }
  if constexpr (PAIR) {
    float size = 0.f;  // of the values, whose rounding counts too
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (v[i] > -INFINITY && 32 * i + lane < a.experts) size = fmaxf(size, fabsf(v[i]));
    tol += 0x1p-21f * __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(size)));
  }
  int my_id = 0;
  // the choice by the keys of 32 slots a lane; expert_of: a slot's expert
  const auto choose = [&](auto& key, auto expert_of) {
    constexpr int N = sizeof(key) / sizeof(key[0]);
    my_id = expert_of(route_select<N>(key, a.top_k, lane, margin, least));
    if constexpr (PAIR) {
      // without a bias the logits themselves are compared, and only the groups' scores are rounded
      const bool groups_open = !(group_margin > 2.f * tol), open = a.bias && !(margin > tol);
      if (groups_open || open) {
        // the chosen experts, and those that may belong in their place
        int mine = my_id, count = a.top_k;
        const float from = least - tol;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const uint32_t near = __ballot_sync(~0u, key[i] != 0u && route_unkey(key[i]) >= from);
          for (uint32_t rest = near; rest != 0u; rest &= rest - 1u, ++count) {
            const int id = expert_of(32 * i + __ffs(rest) - 1);
            if (lane == count) mine = id;
          }
        }
        my_id = groups_open || count > 32 || !(least > -INFINITY) ? route_exact<DTYPE, NL>(a, row, values, top, lane)
                                                                  : route_near<DTYPE>(a, row, reinterpret_cast<int32_t*>(values), top, lane, mine, count);
      }
    }
  };
  bool chosen = false;
  if constexpr (NL >= 4) {
    // where the groups that stay fill at most half of the slots, their experts alone, side by side (in the same order)
    if (a.groups > 1 && a.top_groups * a.per <= 16 * NL && (!PAIR || a.bias)) {
      int* const list = reinterpret_cast<int*>(plain + a.experts);  // the groups that stay
      if (kept >> lane & 1u) list[__popc(kept & ((1u << lane) - 1u))] = lane >> a.span_log;
      __syncwarp();
      const auto expert_of = [&](uint32_t slot) {
        const uint32_t g = (slot * a.inv) >> 20;
        return g < static_cast<uint32_t>(a.top_groups) ? static_cast<int>(slot + (list[g] - g) * a.per) : -1;
      };
      uint32_t key[NL / 2];
#pragma unroll
      for (int i = 0; i < NL / 2; ++i) {
        const int e = expert_of(32 * i + lane);
        key[i] = e >= 0 ? route_key(plain[e]) : 0u;
      }
      // (with fewer than top_k values the rest goes to the lowest experts of any group)
      choose(key, expert_of);
      chosen = least > -INFINITY;
    }
  }
  if (!chosen) {
    uint32_t key[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const uint32_t e = 32 * i + lane;
      key[i] = e < static_cast<uint32_t>(a.experts) ? route_key(route_kept(a, kept, e) ? v[i] : -INFINITY) : 0u;
    }
    choose(key, [](int slot) { return slot; });
  }
  // weights: from the logits, and relative to the largest chosen one where they are divided by their sum, so that small
  // scores keep their ratios: 1 / (1 + exp(-z)) = exp(min(z, 0)) / (1 + exp(-|z|))
  const float zc = lane < a.top_k ? route_clean(route_load<DTYPE>(row, my_id)) : -INFINITY;
  float from = a.sigmoid ? 0.f : top;
  if (a.renorm) from = fminf(from, route_unkey(__reduce_max_sync(~0u, route_key(zc))));
  float w = 0.f, sum = total;
  if (zc > -INFINITY) w = a.sigmoid ? __fdiv_rn(expf(fminf(zc, 0.f) - from), 1.f + expf(-fabsf(zc))) : expf(zc - from);
  if (a.renorm) {
    sum = w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  }
  if (lane < a.top_k) {
    a.ids[token * a.top_k + lane] = my_id;
    a.weights[token * a.top_k + lane] = w > 0.f ? w / sum * a.scale : 0.f;
  }
}

// ---------------------------------------------------------------------------
// Rows of the routed pairs: sorted by expert, equal experts in the pairs' order (token by token).
//
// One cluster of blocks.  Each warp owns a contiguous run of pairs and a row of counters in shared memory; it counts its
// pairs per expert (equal experts among 32 lanes found by one match), the counters become prefix
// sums over warps, blocks (through distributed shared memory) and experts, and the warp goes over its run again:
// a pair's row is its counter plus the number of lower lanes with its expert.  No atomics, so the order
// is the pairs' own.  Bound by latency: a few dependent passes.  Measured, 8 of 256 experts (graph replay, with the
// routing in front, which then took 11 us for 4096 tokens): 4096 tokens 17.9 us in a cluster of 16 blocks, 20.3 with 8, 25.5 with 4, 70 with one;
// 512 tokens 11.2, with one block 14.7.  Runs of up to 8 rounds keep experts and places in registers: 17.9 against 18.9, 128 tokens 8.3 and 9.0.
// Now 16.0 us with the routing's 9.6 (17.4 from DRAM; 131072 pairs 14 us).  Of 12 thousand cycles reading the ids takes 0.8, two rounds of places 2, the sums over warps 1, the cluster's
// 2.6, the scan 1.2, and the scattered stores 2.6.
constexpr int kRowsThreads = 1024, kRowsWarps = kRowsThreads / 32, kRowsMaxBlocks = 16, kRowsHeld = 8;

struct RowsArgs {
  const int32_t* ids;
  int64_t pairs;
  int top_k, experts;
  int64_t run;  // pairs per warp, a multiple of 32
  uint32_t *row_offsets, *scales_offsets;
  int32_t *row_indices, *positions;
  unsigned int* err;
};

inline int rows_smem_bytes(int experts) { return 4 * (kRowsWarps * experts + 2 * experts); }

// The lanes whose id (0 to 1023; others do not matter) is this lane's, by a vote per bit (32768 pairs 6.7 us; with a match of all lanes 7.0).
__device__ __forceinline__ uint32_t rows_same(int id) {
  uint32_t same = ~0u;
#pragma unroll
  for (int b = 0; b < 10; ++b) {
    const bool one = id >> b & 1;
    const uint32_t votes = __ballot_sync(~0u, one);
    same &= one ? votes : ~votes;
  }
  return same & __ballot_sync(~0u, id >= 0);
}

// HELD: a run has at most 32 kRowsHeld pairs, whose experts and places among their warp's stay in registers.
template <bool HELD>
__global__ void __launch_bounds__(kRowsThreads, 1) moe_rows_kernel(const RowsArgs a) {
  extern __shared__ uint32_t rows_smem[];
  __shared__ uint32_t part[2][kRowsWarps];
  __shared__ uint32_t used;
  uint32_t* count = rows_smem;                             // [warps][experts]
  uint32_t* total = rows_smem + kRowsWarps * a.experts;    // [experts] of this block
  uint32_t* base = total + a.experts;                      // [experts] first row of this block's pairs
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = blockIdx.x, blocks = gridDim.x, experts = a.experts;
  for (int i = tid; i < kRowsWarps * experts; i += kRowsThreads) count[i] = 0u;
  pdl_wait();
  const int64_t begin = (static_cast<int64_t>(rank) * kRowsWarps + warp) * a.run;
  const int64_t end = min(begin + a.run, a.pairs);
  uint32_t* mine = count + warp * experts;
  bool bad = false;
  // one round: the pair's expert (-1: none) and its place among those of its expert that the warp has counted, itself left out
  const auto place = [&](int& id, uint32_t& before) {
    if (id >= experts) {
      bad = true;
      id = -1;
    }
    const uint32_t same = rows_same(id);
    uint32_t first = 0;
    if (id >= 0) first = mine[id];
    __syncwarp();
    if (id >= 0 && lane == __ffs(same) - 1) mine[id] = first + __popc(same);
    __syncwarp();
    before = first + __popc(same & ((1u << lane) - 1u));
  };
  int ids[HELD ? kRowsHeld : 1];
  uint32_t offs[HELD ? kRowsHeld : 1];
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < kRowsHeld; ++i) ids[i] = begin + 32 * i + lane < end ? __ldg(a.ids + begin + 32 * i + lane) : -1;
  }
  __syncthreads();
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < kRowsHeld; ++i)
      if (begin + 32 * i < end) place(ids[i], offs[i]);
  } else {
    for (int64_t at = begin; at < end; at += 32) {
      int id = at + lane < end ? __ldg(a.ids + at + lane) : -1;
      uint32_t before;
      place(id, before);
    }
  }
  if (__any_sync(~0u, bad) && lane == 0) record_error_at(a.err, kErrValue);
  __syncthreads();
  // per expert: prefix over the block's warps
  for (int e = tid; e < experts; e += kRowsThreads) {
    uint32_t run = 0;
#pragma unroll
    for (int w0 = 0; w0 < kRowsWarps; w0 += 16) {
      uint32_t c[16];
#pragma unroll
      for (int w = 0; w < 16; ++w) c[w] = count[(w0 + w) * experts + e];
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        count[(w0 + w) * experts + e] = run;
        run += c[w];
      }
    }
    total[e] = run;
  }
  if (blocks > 1) cluster_sync_all(); else __syncthreads();
  // over blocks and experts (at most 1024: a thread each)
  uint32_t all = 0, before = 0;
  if (tid < experts) {
    if (blocks > 1) {
      uint32_t c[kRowsMaxBlocks];
#pragma unroll
      for (int r = 0; r < kRowsMaxBlocks; ++r) c[r] = r < blocks ? cluster_ld_u32(cluster_map(total + tid, r)) : 0u;
#pragma unroll
      for (int r = 0; r < kRowsMaxBlocks; ++r) {
        before += r < rank ? c[r] : 0u;
        all += c[r];
      }
    } else {
      all = total[tid];
    }
  }
  if (blocks > 1) cluster_arrive();  // this block no longer reads the others' memory
  uint32_t rows = all, padded = (all + 127u) & ~127u;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t r = __shfl_up_sync(~0u, rows, d), q = __shfl_up_sync(~0u, padded, d);
    if (lane >= d) {
      rows += r;
      padded += q;
    }
  }
  if (lane == 31) {
    part[0][warp] = rows;
    part[1][warp] = padded;
  }
  __syncthreads();
  {
    const uint32_t r = __reduce_add_sync(~0u, lane < warp ? part[0][lane] : 0u), q = __reduce_add_sync(~0u, lane < warp ? part[1][lane] : 0u);
    rows += r;
    padded += q;
  }
  if (tid < experts) {
    base[tid] = rows - all + before;
    if (rank == 0) {
      a.row_offsets[tid + 1] = rows;
      a.scales_offsets[tid + 1] = padded;
      if (tid == 0) a.row_offsets[0] = a.scales_offsets[0] = 0u;
    }
    if (tid == experts - 1) used = rows;
  }
  __syncthreads();
  const auto put = [&](int64_t pair, int id, uint32_t before) {  // before: in the block, of this expert
    int32_t row = -1;
    if (id >= 0) {
      row = static_cast<int32_t>(base[id] + before);
      a.row_indices[row] = static_cast<int32_t>(static_cast<uint32_t>(pair) / static_cast<uint32_t>(a.top_k));
    }
    a.positions[pair] = row;
  };
  if constexpr (HELD) {
#pragma unroll
    for (int i = 0; i < kRowsHeld; ++i) {
      const int64_t pair = begin + 32 * i + lane;
      // the counters now hold what the warps in front have
      if (pair < end) put(pair, ids[i], ids[i] >= 0 ? mine[ids[i]] + offs[i] : 0u);
    }
  } else {
    for (int64_t at = begin; at < end; at += 32) {
      int id = at + lane < end ? __ldg(a.ids + at + lane) : -1;
      uint32_t before;
      place(id, before);
      if (at + lane < end) put(at + lane, id, before);
    }
  }
  // rows that no pair took (dropped pairs leave them at the end) point at token 0
  for (int64_t r = used + static_cast<int64_t>(rank) * kRowsThreads + tid; r < a.pairs; r += static_cast<int64_t>(blocks) * kRowsThreads)
    a.row_indices[r] = 0;
  if (blocks > 1) cluster_wait();
}

}  // namespace bsq
