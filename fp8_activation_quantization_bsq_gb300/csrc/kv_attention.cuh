// Attention over the 8-bit paged cache.
//
// Per query row of a head, over the allowed keys j of its sequence:
//   s_j = sm_scale q.k_j,  out = sum_j exp(s_j) v_j / sum_j exp(s_j).
// One warp per (query token, head), a key at a time, with the running
// maximum and sum of the softmax.
#pragma once

#include "serving_common.cuh"

namespace bsq {

struct KvAttnArgs {
  const uint16_t* q;              // (total, heads, D)
  int64_t q_tok, q_head;          // strides in elements
  const uint8_t* cache[2];
  int64_t cs_page, cs_head, cs_tok;
  const uint8_t* scales[2];       // (num_pages, kv_heads) E8M0 bytes
  const int32_t* table;
  int64_t table_ld;
  const int32_t* offsets;
  const int32_t* lens;
  uint16_t* out;                  // (total, heads, D) contiguous
  float* lse;                     // (total, heads) or NULL
  int64_t total, num_pages;
  int batch, heads, kv_heads, page, table_width, causal, window;
  float scale_log2;               // sm_scale * log2(e)
  unsigned int* err;
};

template <int D, bool F16>
__global__ void __launch_bounds__(128) kv_attention_kernel(const KvAttnArgs a) {
  pdl_wait();
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (unit >= a.total * a.heads) return;
  const int64_t t = unit / a.heads;
  const int h = static_cast<int>(unit % a.heads), kvh = h / (a.heads / a.kv_heads);
  int lo = 0, hi = a.batch;  // the last b with offsets[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (a.offsets[mid] <= t) lo = mid; else hi = mid;
  }
  const int b = lo;
  if (t < a.offsets[b] || t >= a.offsets[b + 1]) return;
  const int64_t n = a.offsets[b + 1] - a.offsets[b];
  int64_t len = a.lens[b];
  if (len < 0 || len > static_cast<int64_t>(a.table_width) * a.page) {
    if (lane == 0) record_error_at(a.err, kErrValue);
    len = 0;
  }
  const int64_t pos = len - n + (t - a.offsets[b]);
  const int64_t last = a.causal ? min(len, pos + 1) : len;
  const int64_t first = a.window > 0 ? max(int64_t{0}, pos - a.window + 1) : 0;
  float q[N], o[N], m = -INFINITY, l = 0.f;
  for (int i = 0; i < N; i += 2) {
    const float2 x = elem2_to_f32x2<F16>(*reinterpret_cast<const uint32_t*>(a.q + t * a.q_tok + h * a.q_head + lane * N + i));
    q[i] = x.x * a.scale_log2; q[i + 1] = x.y * a.scale_log2; o[i] = o[i + 1] = 0.f;
  }
  for (int64_t j = first; j < last; ++j) {
    const int64_t pid = a.table[b * a.table_ld + j / a.page];
    if (pid < 0 || pid >= a.num_pages) {
      if (lane == 0) record_error_at(a.err, kErrValue);
      continue;
    }
    const int64_t at = pid * a.cs_page + kvh * a.cs_head + (j % a.page) * a.cs_tok + lane * N;
    const float ks = pow2f(a.scales[0][pid * a.kv_heads + kvh] - 127), vs = pow2f(a.scales[1][pid * a.kv_heads + kvh] - 127);
    float s = 0.f;
    for (int i = 0; i < N; i += 2) {
      const float2 k = f16x2_to_f32x2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(a.cache[0] + at + i)));
      s += q[i] * k.x + q[i + 1] * k.y;
    }
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    s *= ks;
    const float m2 = fmaxf(m, s), c = exp2f(m - m2), p = exp2f(s - m2);
    m = m2;
    l = l * c + p;
    for (int i = 0; i < N; i += 2) {
      const float2 v = f16x2_to_f32x2(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(a.cache[1] + at + i)));
      o[i] = o[i] * c + p * vs * v.x;
      o[i + 1] = o[i + 1] * c + p * vs * v.y;
    }
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  for (int i = 0; i < N; i += 2)
    *reinterpret_cast<uint32_t*>(a.out + (t * a.heads + h) * D + lane * N + i) = f32x2_to_elem2<F16>(o[i] * inv, o[i + 1] * inv);
  if (lane == 0 && a.lse) a.lse[t * a.heads + h] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace bsq
