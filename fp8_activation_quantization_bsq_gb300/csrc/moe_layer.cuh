// A mixture-of-experts layer for a few tokens over packed weights.
//   ids, p = top-k of softmax(logits); xq = Q(x, x_sf[e]); g, u = W13[e] xq;
//   h = bf16(silu(g) u); hq = Q(h, h_sf[e]); y = sum_k p_k W2[e] hq.
// Simple form: one warp per output value.
#pragma once

#include "serving_common.cuh"

namespace bsq {

constexpr int kMoeMaxTokens = 64, kMoeMaxTopK = 16, kMoeMaxExperts = 1024;

struct MoeArgs {
  const uint16_t* x;
  int64_t ld_x;
  const float* logits;
  int64_t ld_logits;
  const uint8_t *w13, *w13_s, *w2, *w2_s;
  int64_t w13_expert, w13_s_expert, w2_expert, w2_s_expert;  // bytes per expert
  const float *x_sf, *w13_sf, *h_sf, *w2_sf;                 // NVFP4
  uint16_t* y;
  int64_t ld_y;
  int tokens, hidden, inter, experts, top_k, renorm;
  int* ids;      // tokens * top_k
  float* probs;
  float* xq;     // rows x hidden values
  float* h;      // rows x inter
  unsigned int* err;
};

__global__ void __launch_bounds__(32) moe_route_kernel(const MoeArgs a) {
  pdl_wait();
  const int t = blockIdx.x, lane = threadIdx.x;
  const float* z = a.logits + t * a.ld_logits;
  float top = -INFINITY;
  for (int e = lane; e < a.experts; e += 32) top = fmaxf(top, z[e]);
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, d));
  float sum = 0.f;
  for (int e = lane; e < a.experts; e += 32) sum += expf(z[e] - top);
  for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  float last = INFINITY, chosen = 0.f;
  int last_id = -1;
  for (int k = 0; k < a.top_k; ++k) {
    float best = -INFINITY;
    int id = 0x7FFFFFFF;
    for (int e = lane; e < a.experts; e += 32)
      if ((z[e] < last || (z[e] == last && e > last_id)) && (z[e] > best || id == 0x7FFFFFFF)) { best = z[e]; id = e; }
    for (int d = 16; d > 0; d >>= 1) {
      const float ob = __shfl_xor_sync(~0u, best, d);
      const int oi = __shfl_xor_sync(~0u, id, d);
      if (ob > best || (ob == best && oi < id)) { best = ob; id = oi; }
    }
    if (id == 0x7FFFFFFF) id = 0;  // nothing left to compare (NaN)
    last = best; last_id = id;
    const float p = expf(best - top);
    chosen += p;
    if (lane == 0) { a.ids[t * a.top_k + k] = id; a.probs[t * a.top_k + k] = p; }
  }
  __syncwarp();
  const float by = 1.f / (a.renorm ? chosen : sum);
  for (int k = lane; k < a.top_k; k += 32) a.probs[t * a.top_k + k] *= by;
}

// Values that a warp's block of 32 (or two of 16) elements stands for once quantized.
template <int FMT>
__device__ __forceinline__ float moe_quant(float v, float tsf) {
  constexpr int SF = Fmt<FMT>::SF;
  float amax = fabsf(v);
  for (int d = SF / 2; d > 0; d >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, d));
  if constexpr (FMT == kNVFP4) {
    const float ds = e4m3_to_f32(f32_to_e4m3(__fmul_rn(__fdiv_rn(amax, 6.f), tsf)));
    const float f = ds == 0.f ? 0.f : __fdiv_rn(tsf, ds);
    uint32_t h;
    const float s = v * f;
    asm("{.reg .b8 q, r;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %2, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, q;}" : "=r"(h) : "f"(s), "f"(0.f));
    return f16x2_to_f32x2(h).x * ds / tsf;
  } else {
    const MxScale sc = mx_scale<FMT == kMXFP4 ? 6 : 448>(amax);
    const int e = static_cast<int>(sc.byte) - 127;
    const float s = v * pow2f(-e > 127 ? 127 : -e);
    uint32_t h;
    if constexpr (FMT == kMXFP4)
      asm("{.reg .b8 q, r;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %2, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, q;}" : "=r"(h) : "f"(s), "f"(0.f));
    else
      h = e4m3x2_to_f16x2(f32x2_to_e4m3x2(s, 0.f));
    return f16x2_to_f32x2(h).x * exp2f(static_cast<float>(e));
  }
}

template <int FMT>
__global__ void __launch_bounds__(32) moe_quant_x_kernel(const MoeArgs a) {
  pdl_wait();
  const int row = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  const int e = a.ids[row];
  const float v = __uint_as_float(static_cast<uint32_t>(a.x[(row / a.top_k) * a.ld_x + c]) << 16);
  a.xq[static_cast<int64_t>(row) * a.hidden + c] = moe_quant<FMT>(v, FMT == kNVFP4 ? a.x_sf[e] : 1.f);
}

// Dot product of a packed weight row with FP32 values, per warp.
template <int FMT>
__device__ __forceinline__ float moe_dot(const uint8_t* w, const uint8_t* s5, int row, int K, const float* x) {
  constexpr int SF = Fmt<FMT>::SF;
  const int lane = threadIdx.x & 31, kt = (K / SF + 3) / 4;
  float acc = 0.f;
  const int64_t row_bytes = FMT == kMXFP8 ? K : K / 2;
  for (int k = 2 * lane; k < K; k += 64) {
    uint32_t h;
    if constexpr (FMT == kMXFP8)
      h = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(w + row * row_bytes + k));
    else {
      const uint32_t byte = w[row * row_bytes + k / 2];
      asm("{.reg .b8 q, a, b, c;\n\tmov.b32 {q, a, b, c}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, q;}" : "=r"(h) : "r"(byte));
    }
    const int sc = k / SF;
    const uint32_t byte = s5[(static_cast<int64_t>(row / 128) * kt + sc / 4) * 512 + (row % 32) * 16 + (row % 128) / 32 * 4 + sc % 4];
    const float f = FMT == kNVFP4 ? e4m3_to_f32(byte) : exp2f(static_cast<float>(byte) - 127.f);
    const float2 v = f16x2_to_f32x2(h);
    acc += (v.x * x[k] + v.y * x[k + 1]) * f;
  }
  for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(~0u, acc, d);
  return acc;
}

template <int FMT>
__global__ void __launch_bounds__(128) moe_up_kernel(const MoeArgs a) {
  pdl_wait();
  const int row = blockIdx.y, i = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int64_t e = a.ids[row];
  const float* x = a.xq + static_cast<int64_t>(row) * a.hidden;
  const float sf = FMT == kNVFP4 ? a.w13_sf[e] : 1.f;
  const float g = moe_dot<FMT>(a.w13 + e * a.w13_expert, a.w13_s + e * a.w13_s_expert, i, a.hidden, x) / sf;
  const float u = moe_dot<FMT>(a.w13 + e * a.w13_expert, a.w13_s + e * a.w13_s_expert, a.inter + i, a.hidden, x) / sf;
  if ((threadIdx.x & 31) == 0) a.h[static_cast<int64_t>(row) * a.inter + i] = __bfloat162float(__float2bfloat16_rn(g / (1.f + expf(-g)) * u));
}

template <int FMT>
__global__ void __launch_bounds__(32) moe_quant_h_kernel(const MoeArgs a) {
  pdl_wait();
  const int row = blockIdx.y, c = blockIdx.x * 32 + threadIdx.x;
  float* p = a.h + static_cast<int64_t>(row) * a.inter + c;
  *p = moe_quant<FMT>(*p, FMT == kNVFP4 ? a.h_sf[a.ids[row]] : 1.f);
}

template <int FMT>
__global__ void __launch_bounds__(128) moe_down_kernel(const MoeArgs a) {
  pdl_wait();
  const int t = blockIdx.y, c = blockIdx.x * 4 + (threadIdx.x >> 5);
  float y = 0.f;
  for (int k = 0; k < a.top_k; ++k) {
    const int64_t e = a.ids[t * a.top_k + k];
    y += a.probs[t * a.top_k + k] / (FMT == kNVFP4 ? a.w2_sf[e] : 1.f) *
         moe_dot<FMT>(a.w2 + e * a.w2_expert, a.w2_s + e * a.w2_s_expert, c, a.inter, a.h + static_cast<int64_t>(t * a.top_k + k) * a.inter);
  }
  if ((threadIdx.x & 31) == 0) a.y[t * a.ld_y + c] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
}

}  // namespace bsq
