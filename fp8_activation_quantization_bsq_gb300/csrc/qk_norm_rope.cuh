// Norm of query and key heads and their rotation by position, in one pass:
//   u = x / sqrt(mean(x^2) + eps) * w  (per head row; without a weight u = x)
//   (u_a, u_b) -> (u_a cos t - u_b sin t, u_b cos t + u_a sin t),  t = position * inv_freq[i]
// for the first `pairs` pairs of a row, (i, i + pairs) or (2i, 2i + 1); what lies behind passes.
//
// Bound by DRAM: 2 bytes read and 2 written per element.  A row's 8 elements per lane are two
// groups of 4 that hold both sides of a lane's pairs, so that no element crosses lanes and the lane's 4
// angles serve every head of the token that the warp takes; 8, 16 or 32 lanes per row (dim to 64, 128, 256).
//
// Angles: t / 2 pi in fixed point.  inv_freq is a 24-bit integer times a power of two, 1 / (2 pi) a 64-bit
// fraction, and the position multiplies their product modulo 2^64, which drops whole turns exactly: off by
// at most position * inv_freq * 2^-64 turns before the last 32 bits are cut off, at any position.
#pragma once

#include "serving_common.cuh"

namespace bsq {

constexpr int kRopeWarps = 4;

struct RopeArgs {
  const uint16_t* src[2];  // queries, keys
  uint16_t* dst[2];
  int64_t src_tok[2], src_head[2], dst_tok[2], dst_head[2];  // strides in elements
  const void* weight[2];                                     // null: no norm
  const int32_t* positions;
  const float* inv_freq;
  int64_t tokens;
  int heads, rows;  // query heads, query and key heads
  int dim, pairs;
  int weight_f32;
  float eps;
  int chunks, per_chunk;  // tasks per token, rows per task
};

// cos and sin of position * f.
__device__ __forceinline__ float2 rope_turn(float f, int position) {
  const uint32_t bits = __float_as_uint(f);
  const int ex = static_cast<int>((bits >> 23) & 255u);
  const uint64_t m = (bits & 0x7FFFFFu) | (ex != 0 ? 0x800000u : 0u);
  const int e = max(ex, 1) - 150;                            // |f| = m 2^e
  constexpr uint64_t kInvTwoPi = 0x28BE60DB9391054Aull;      // 2^64 / (2 pi)
  const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
  // (hi, lo) 2^e modulo 2^64: the frequency in turns per position
  uint64_t turn;
  if (e >= 0)
    turn = e < 64 ? lo << e : 0;
  else if (e > -64)
    turn = (lo >> -e) | (hi << (64 + e));
  else
    turn = e > -128 ? hi >> (-e - 64) : 0;
  turn *= static_cast<uint64_t>(static_cast<uint32_t>(position));
  if (bits >> 31) turn = 0 - turn;
  float2 r;
  // half turns in [-1, 1); the angle's rounding to 24 bits is the only one before the functions'
  sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &r.y, &r.x);
  if (ex == 255) r.x = r.y = __uint_as_float(0x7FC00000u);
  return r;
}

// Rows whose elements a lane reads: MODE 0 pairs (i, i + pairs) with pairs a multiple of 4, 1 neighbouring pairs,
// 2 pairs (i, i + pairs) of any number, whose other sides come through shared memory.  L lanes per row.
template <bool F16, int L, int MODE>
__global__ void __launch_bounds__(kRopeWarps * 32) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int kPer = 32 / L;   // rows at a time
  constexpr int kUnroll = 4;     // row loads in flight per lane
  __shared__ float other[MODE == 2 ? kRopeWarps * 256 : 1];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L, p = lane % L;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
  const int64_t token = task / a.chunks;
  if (token >= a.tokens) return;
  const int position = __ldg(a.positions + token);
  if (position < 0) return;
  const int first = static_cast<int>(task - token * a.chunks) * a.per_chunk, last = min(first + a.per_chunk, a.rows);
  const bool active = p < a.dim / 8;
  const int quarter = a.pairs / 4;  // groups of 4 elements on one side (MODE 0)
  const bool apart = MODE == 0 && p < quarter;
  const int ea = apart ? 4 * p : 8 * p, eb = apart ? 4 * p + a.pairs : 8 * p + 4;

  constexpr int kAngles = MODE == 2 ? 8 : 4;
  float cs[kAngles], sn[kAngles];
  bool turns[kAngles];
#pragma unroll
  for (int j = 0; j < kAngles; ++j) {
    int i = MODE == 2 ? 8 * p + j : 4 * p + j;
    turns[j] = active && (MODE == 0 ? apart : MODE == 1 ? i < a.pairs : i < 2 * a.pairs);
    const bool second = MODE == 2 && i >= a.pairs;
    if (second) i -= a.pairs;
    cs[j] = 1.f;
    sn[j] = 0.f;
    if (turns[j]) {
      const float2 t = rope_turn(__ldg(a.inv_freq + i), position);
      cs[j] = t.x;
      sn[j] = second ? -t.y : t.y;
    }
  }

  float w[8];
  int kind = -1;
  for (int r0 = first; r0 < last; r0 += kPer * kUnroll) {
    uint2 va[kUnroll], vb[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * kPer + sub;
      va[u] = vb[u] = make_uint2(0, 0);
      if (r < last && active) {
        const int k = r >= a.heads;
        const uint16_t* s = a.src[k] + token * a.src_tok[k] + (r - (k ? a.heads : 0)) * a.src_head[k];
        if (apart) {
          va[u] = *reinterpret_cast<const uint2*>(s + ea);
          vb[u] = *reinterpret_cast<const uint2*>(s + eb);
        } else {
          const uint4 v = *reinterpret_cast<const uint4*>(s + ea);
          va[u] = make_uint2(v.x, v.y);
          vb[u] = make_uint2(v.z, v.w);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (r0 + u * kPer >= last) break;  // the whole warp
      const int r = r0 + u * kPer + sub;
      const int k = r >= a.heads;
      const bool has_norm = a.weight[k] != nullptr;
      if (k != kind) {
        kind = k;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int e = j < 4 ? ea + j : eb + j - 4;
          w[j] = 1.f;
          if (has_norm && active) {
            if (a.weight_f32) {
              w[j] = __ldg(static_cast<const float*>(a.weight[k]) + e);
            } else {
              w[j] = elem2_to_f32x2<F16>(__ldg(static_cast<const uint16_t*>(a.weight[k]) + e)).x;
            }
          }
        }
      }
      float x[8];
      {
        const float2 x0 = elem2_to_f32x2<F16>(va[u].x), x1 = elem2_to_f32x2<F16>(va[u].y);
        const float2 x2 = elem2_to_f32x2<F16>(vb[u].x), x3 = elem2_to_f32x2<F16>(vb[u].y);
        x[0] = x0.x, x[1] = x0.y, x[2] = x1.x, x[3] = x1.y, x[4] = x2.x, x[5] = x2.y, x[6] = x3.x, x[7] = x3.y;
      }
      if (a.weight[0] != nullptr || a.weight[1] != nullptr) {
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
#pragma unroll
        for (int d = L / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
        float eps = a.eps;
        if (!F16 && __any_sync(~0u, sum > 3.0e38f)) {  // squares past FP32 (rows beyond 2^63): once more, 2^-96 smaller
          const bool again = sum > 3.0e38f;
          float small = 0.f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (again && has_norm) x[j] *= 0x1p-96f;
            small = fmaf(x[j], x[j], small);
          }
#pragma unroll
          for (int d = L / 2; d > 0; d >>= 1) small += __shfl_xor_sync(~0u, small, d);
          if (again) {
            sum = small;
            eps = 0.f;  // far below the mean
          }
        }
        if (has_norm) {
          const float f = rsqrtf(sum / static_cast<float>(a.dim) + eps);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] *= f * w[j];
        }
      }
      float y[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = x[j];
      if constexpr (MODE == 0) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (turns[j]) {
            y[j] = x[j] * cs[j] - x[j + 4] * sn[j];
            y[j + 4] = x[j + 4] * cs[j] + x[j] * sn[j];
          }
      } else if constexpr (MODE == 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (turns[j]) {
            y[2 * j] = x[2 * j] * cs[j] - x[2 * j + 1] * sn[j];
            y[2 * j + 1] = x[2 * j + 1] * cs[j] + x[2 * j] * sn[j];
          }
      }
      if constexpr (MODE == 2) {
        float* mine = other + (warp * kPer + sub) * 8 * L;  // the row's other lanes
#pragma unroll
        for (int j = 0; j < 8; ++j) mine[8 * p + j] = x[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (turns[j]) y[j] = x[j] * cs[j] - mine[8 * p + j < a.pairs ? 8 * p + j + a.pairs : 8 * p + j - a.pairs] * sn[j];
        __syncwarp();
      }
      if (r < last && active) {
        uint16_t* d = a.dst[k] + token * a.dst_tok[k] + (r - (k ? a.heads : 0)) * a.dst_head[k];
        const uint2 oa = make_uint2(f32x2_to_elem2<F16>(y[0], y[1]), f32x2_to_elem2<F16>(y[2], y[3]));
        const uint2 ob = make_uint2(f32x2_to_elem2<F16>(y[4], y[5]), f32x2_to_elem2<F16>(y[6], y[7]));
        if (apart) {
          *reinterpret_cast<uint2*>(d + ea) = oa;
          *reinterpret_cast<uint2*>(d + eb) = ob;
        } else {
          *reinterpret_cast<uint4*>(d + ea) = make_uint4(oa.x, oa.y, ob.x, ob.y);
        }
      }
    }
  }
}

}  // namespace bsq
