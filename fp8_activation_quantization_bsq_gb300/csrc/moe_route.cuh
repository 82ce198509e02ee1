// Routing of tokens to experts, and the order of the routed rows.
//
// moe_route_kernel: p = softmax(z) or 1 / (1 + exp(-z)); an expert's value is p + bias, or its logit without a bias
// (p grows with it); of equal groups of experts those with the largest sums of their one or two largest
// values stay; then the top_k largest values, equal ones lowest expert first; weights p (/ their sum) * scale.
// One warp per token, the logits in registers.  Which experts are chosen must not hang on how p was rounded: two
// values may lie closer than FP32 tells apart.  Where p enters the comparison it is therefore held as a
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
__device__ __forceinline__ RouteFF ff_div(RouteFF a, RouteFF b) {
  const float q = __fdiv_rn(a.h, b.h);
  // a - q b, its leading part exact
  const float p = __fmul_rn(q, b.h), e = __fmaf_rn(q, b.h, -p);
  const float r = __fadd_rn(__fsub_rn(__fsub_rn(a.h, p), e), __fmaf_rn(-q, b.l, a.l));
  return ff_fast(q, __fdiv_rn(r, b.h));
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

// One logit as FP32; DTYPE is a bsq_dtype.
template <int DTYPE>
__device__ __forceinline__ float route_load(const void* row, int e) {
  if constexpr (DTYPE == 2) return __ldg(static_cast<const float*>(row) + e);
  return elem2_to_f32x2<DTYPE == 1>(__ldg(static_cast<const uint16_t*>(row) + e)).x;
}

// The largest key of the warp and its lowest expert, taken out of the lane's keys.  Returns the expert.
template <int NL, typename K>
__device__ __forceinline__ int route_take(K (&key)[NL], int lane, K& top) {
  K best = 0;
#pragma unroll
  for (int i = 0; i < NL; ++i) best = max(best, key[i]);
  if constexpr (sizeof(K) == 8) {
    const uint32_t hi = __reduce_max_sync(~0u, static_cast<uint32_t>(best >> 32));
    const uint32_t lo = __reduce_max_sync(~0u, static_cast<uint32_t>(best >> 32) == hi ? static_cast<uint32_t>(best) : 0u);
    top = static_cast<K>(hi) << 32 | lo;
  } else {
    top = __reduce_max_sync(~0u, best);
  }
  int at = 0x7FFFFFFF;
#pragma unroll
  for (int i = NL - 1; i >= 0; --i)
    if (key[i] == top) at = 32 * i + lane;
  const int id = static_cast<int>(__reduce_min_sync(~0u, static_cast<uint32_t>(at)));
#pragma unroll
  for (int i = 0; i < NL; ++i)
    if (32 * i + lane == id) key[i] = 0;
  return id;
}

// The groups that stay, a bit per group: the lanes share the groups out, `v` holds the experts' values in shared memory.
__device__ __forceinline__ uint32_t route_groups(const RouteArgs& a, const RouteFF* v, int lane) {
  int span = 32;  // lanes per group
  while (span * a.groups > 32) span >>= 1;
  const int g = lane / span, part = lane % span, per = a.experts / a.groups;
  const RouteFF none = {-INFINITY, 0.f};
  RouteFF first = none, second = none;
  if (g < a.groups)
    for (int j = part; j < per; j += span) {
      const RouteFF x = v[g * per + j];
      if (ff_greater(x, first)) {
        second = first;
        first = x;
      } else if (ff_greater(x, second)) {
        second = x;
      }
    }
  for (int d = 1; d < span; d <<= 1) {
    const RouteFF f = {__shfl_xor_sync(~0u, first.h, d), __shfl_xor_sync(~0u, first.l, d)};
    const RouteFF s = {__shfl_xor_sync(~0u, second.h, d), __shfl_xor_sync(~0u, second.l, d)};
    if (ff_greater(f, first)) {
      second = ff_greater(first, s) ? first : s;
      first = f;
    } else if (ff_greater(f, second)) {
      second = f;
    }
  }
  RouteFF score = first;
  if (a.group_top == 2 && per > 1) score = first.h > -INFINITY && second.h > -INFINITY ? ff_add(first, second) : none;
  int before = 0;
  for (int o = 0; o < a.groups; ++o) {
    const RouteFF s = {__shfl_sync(~0u, score.h, o * span), __shfl_sync(~0u, score.l, o * span)};
    before += ff_greater(s, score) || (o < g && s.h == score.h && s.l == score.l);
  }
  const uint32_t votes = __ballot_sync(~0u, g < a.groups && part == 0 && before < a.top_groups);
  uint32_t kept = 0;
  for (int o = 0; o < a.groups; ++o) kept |= (votes >> (o * span) & 1u) << o;
  return kept;
}

// NL: logits per lane (expert 32 i + lane in slot i).  PAIR: p enters the comparison (a bias, or sums of two in groups).
template <int DTYPE, int NL, bool PAIR>
__global__ void __launch_bounds__(kRouteWarps * 32) moe_route_kernel(const RouteArgs a) {
  extern __shared__ RouteFF route_values[];  // [warps][experts] with groups
  __shared__ float chosen[kRouteWarps][kRouteMaxTopK];
  using Key = std::conditional_t<PAIR, uint64_t, uint32_t>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t token = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  RouteFF tab = {0.f, 0.f};
  if constexpr (PAIR) tab = {kRouteExp2[2 * lane], kRouteExp2[2 * lane + 1]};
  pdl_wait();
  if (token >= a.tokens) return;
  const void* row = static_cast<const char*>(a.logits) + token * a.ld * (DTYPE == 2 ? 4 : 2);

  float z[NL];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int e = 32 * i + lane;
    z[i] = e < a.experts ? route_load<DTYPE>(row, e) : -INFINITY;
    if (!(z[i] < INFINITY)) {  // NaN, +inf
      bad = true;
      z[i] = -INFINITY;
    }
  }
  float bias[PAIR ? NL : 1];
  if constexpr (PAIR) {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const int e = 32 * i + lane;
      bias[i] = a.bias && e < a.experts ? __ldg(a.bias + e) : 0.f;
      if (!(bias[i] < INFINITY)) {
        bad = true;
        bias[i] = -INFINITY;
      }
    }
  }
  if (__any_sync(~0u, bad) && lane == 0) record_error_at(a.err, kErrValue);
  float top = -INFINITY;
  if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < NL; ++i) top = fmaxf(top, z[i]);
    top = route_unkey(__reduce_max_sync(~0u, route_key(top)));
  }

  Key key[NL];
  float total = 0.f;  // of the softmax
  if constexpr (PAIR) {
    RouteFF e[NL], sum = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const bool off = !(z[i] > -INFINITY);
      if (a.sigmoid) {
        const RouteFF u = ff_exp(RouteFF{off ? 0.f : -fabsf(z[i]), 0.f}, tab);
        const RouteFF d = ff_add(RouteFF{1.f, 0.f}, u);
        e[i] = ff_div(z[i] >= 0.f ? RouteFF{1.f, 0.f} : u, d);
      } else {
        e[i] = ff_exp(off ? RouteFF{0.f, 0.f} : ff_two_sum(z[i], -top), tab);
      }
      if (off) e[i] = {0.f, 0.f};
      sum = ff_add(sum, e[i]);
    }
    if (!a.sigmoid) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) sum = ff_add(sum, RouteFF{__shfl_xor_sync(~0u, sum.h, d), __shfl_xor_sync(~0u, sum.l, d)});
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (sum.h > 0.f) e[i] = ff_div(e[i], sum);
      total = sum.h;
    }
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      RouteFF v = e[i];
      if (a.bias) {
        const RouteFF s = ff_two_sum(v.h, bias[i]);
        v = ff_fast(s.h, __fadd_rn(s.l, v.l));
        if (!(z[i] > -INFINITY) || !(bias[i] > -INFINITY)) v = {-INFINITY, 0.f};
      }
      if (a.groups > 1 && 32 * i + lane < a.experts) route_values[warp * a.experts + 32 * i + lane] = v;
      if (!a.bias) v = {z[i], 0.f};
      key[i] = 32 * i + lane < a.experts ? static_cast<uint64_t>(route_key(v.h)) << 32 | route_key(v.l) : 0;
    }
  } else {
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      key[i] = 32 * i + lane < a.experts ? route_key(z[i]) : 0u;
      if (a.groups > 1 && 32 * i + lane < a.experts) route_values[warp * a.experts + 32 * i + lane] = {z[i], 0.f};
    }
  }

  if (a.groups > 1) {
    __syncwarp();
    const uint32_t kept = route_groups(a, route_values + warp * a.experts, lane);
    const int per = a.experts / a.groups;
    const uint32_t inv = ((1u << 20) + per - 1) / per;  // e * inv >> 20 is e / per for e, per <= 1024
    const Key least = PAIR ? static_cast<Key>(static_cast<uint64_t>(route_key(-INFINITY)) << 32 | route_key(0.f))
                           : static_cast<Key>(route_key(-INFINITY));
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const uint32_t e = 32 * i + lane;
      if (e < static_cast<uint32_t>(a.experts) && !(kept >> ((e * inv) >> 20) & 1u)) key[i] = least;
    }
  }

  if (!PAIR && !a.sigmoid && !a.renorm) {
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (z[i] > -INFINITY) total += expf(z[i] - top);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) total += __shfl_xor_sync(~0u, total, d);
  }

  int my_id = 0;
  for (int k = 0; k < a.top_k; ++k) {
    Key best;
    const int id = route_take<NL>(key, lane, best);
    if (lane == k) my_id = id;
    if ((id & 31) == lane) {
#pragma unroll
      for (int i = 0; i < NL; ++i)
        if (32 * i + lane == id) chosen[warp][k] = z[i];
    }
  }
  __syncwarp();
  // weights: from the logits, and relative to the largest chosen one where they are divided by their sum, so that small
  // scores keep their ratios: 1 / (1 + exp(-z)) = exp(min(z, 0)) / (1 + exp(-|z|))
  const float zc = lane < a.top_k ? chosen[warp][lane] : -INFINITY;
  float from = a.sigmoid ? 0.f : top;
  if (a.renorm) from = fminf(from, route_unkey(__reduce_max_sync(~0u, route_key(zc))));
  float w = 0.f, sum = a.sigmoid ? 1.f : total;
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
// is the pairs' own.  Bound by latency: a few dependent passes of one to eight blocks.
constexpr int kRowsThreads = 1024, kRowsWarps = kRowsThreads / 32, kRowsMaxBlocks = 8;

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

__global__ void __launch_bounds__(kRowsThreads, 1) moe_rows_kernel(const RowsArgs a) {
  extern __shared__ uint32_t rows_smem[];
  __shared__ uint32_t part[2][kRowsWarps];
  uint32_t* count = rows_smem;                             // [warps][experts]
  uint32_t* total = rows_smem + kRowsWarps * a.experts;    // [experts] of this block
  uint32_t* base = total + a.experts;                      // [experts] first row of this block's pairs
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, rank = blockIdx.x, blocks = gridDim.x, experts = a.experts;
  for (int i = tid; i < kRowsWarps * experts; i += kRowsThreads) count[i] = 0u;
  pdl_wait();
  __syncthreads();
  const int64_t begin = (static_cast<int64_t>(rank) * kRowsWarps + warp) * a.run;
  const int64_t end = min(begin + a.run, a.pairs);
  uint32_t* mine = count + warp * experts;
  bool bad = false;
  for (int64_t at = begin; at < end; at += 32) {
    int id = at + lane < end ? __ldg(a.ids + at + lane) : -1;
    if (id >= experts) {
      bad = true;
      id = -1;
    }
    const uint32_t same = __match_any_sync(~0u, id);
    if (id >= 0 && lane == __ffs(same) - 1) mine[id] += __popc(same);
    __syncwarp();
  }
  if (__any_sync(~0u, bad) && lane == 0) record_error_at(a.err, kErrValue);
  __syncthreads();
  // per expert: prefix over the block's warps
  for (int e = tid; e < experts; e += kRowsThreads) {
    uint32_t run = 0;
#pragma unroll 8
    for (int w = 0; w < kRowsWarps; ++w) {
      const uint32_t c = count[w * experts + e];
      count[w * experts + e] = run;
      run += c;
    }
    total[e] = run;
  }
  cluster_sync_all();
  // over blocks and experts (at most 1024: a thread each)
  uint32_t all = 0, before = 0;
  if (tid < experts)
    for (int r = 0; r < blocks; ++r) {
      const uint32_t c = cluster_ld_u32(cluster_map(total + tid, r));
      before += r < rank ? c : 0u;
      all += c;
    }
  cluster_sync_all();  // the other blocks' memory is no longer read
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
  for (int w = 0; w < warp; ++w) {
    rows += part[0][w];
    padded += part[1][w];
  }
  if (tid < experts) {
    base[tid] = rows - all + before;
    if (rank == 0) {
      a.row_offsets[tid + 1] = rows;
      a.scales_offsets[tid + 1] = padded;
      if (tid == 0) a.row_offsets[0] = a.scales_offsets[0] = 0u;
    }
  }
  __shared__ uint32_t used;
  if (tid == experts - 1) used = rows;
  __syncthreads();
  for (int64_t at = begin; at < end; at += 32) {
    const int64_t pair = at + lane;
    int id = pair < end ? __ldg(a.ids + pair) : -1;
    if (id >= experts) id = -1;
    const uint32_t same = __match_any_sync(~0u, id);
    uint32_t first = 0;
    if (id >= 0) first = mine[id];
    __syncwarp();
    if (id >= 0 && lane == __ffs(same) - 1) mine[id] = first + __popc(same);
    __syncwarp();
    if (pair < end) {
      int32_t row = -1;
      if (id >= 0) {
        row = static_cast<int32_t>(base[id] + first + __popc(same & ((1u << lane) - 1u)));
        a.row_indices[row] = static_cast<int32_t>(pair / a.top_k);
      }
      a.positions[pair] = row;
    }
  }
  // rows that no pair took (dropped pairs leave them at the end) point at token 0
  for (int64_t r = used + static_cast<int64_t>(rank) * kRowsThreads + tid; r < a.pairs; r += static_cast<int64_t>(blocks) * kRowsThreads)
    a.row_indices[r] = 0;
}

}  // namespace bsq
