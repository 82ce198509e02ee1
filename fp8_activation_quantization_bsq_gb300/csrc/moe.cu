// Host side of the few-token mixture-of-experts layer (bsq_moe_layer).
#include <algorithm>

#include "host_common.h"
#include "moe_layer.cuh"

namespace {

using namespace bsq;

bool moe_sizes_ok(int32_t tokens, int64_t hidden, int64_t inter, int32_t experts, int32_t top_k) {
  return tokens >= 0 && tokens <= kMoeMaxTokens && hidden >= 32 && hidden % 32 == 0 && hidden <= (1 << 20) && inter >= 128 &&
         inter % 128 == 0 && inter <= (1 << 20) && experts >= 1 && experts <= kMoeMaxExperts && top_k >= 1 &&
         top_k <= kMoeMaxTopK && top_k <= experts;
}

template <int FMT>
cudaError_t launch_moe(const MoeArgs& a, cudaStream_t st) {
  const unsigned rows = a.tokens * a.top_k;
  launch_pdl(moe_route_kernel, dim3(a.tokens), dim3(32), 0, st, a);
  launch_pdl(moe_quant_x_kernel<FMT>, dim3(a.hidden / 32, rows), dim3(32), 0, st, a);
  launch_pdl(moe_up_kernel<FMT>, dim3(a.inter / 4, rows), dim3(128), 0, st, a);
  launch_pdl(moe_quant_h_kernel<FMT>, dim3(a.inter / 32, rows), dim3(32), 0, st, a);
  launch_pdl(moe_down_kernel<FMT>, dim3(a.hidden / 4, a.tokens), dim3(128), 0, st, a);
  return cudaGetLastError();
}

}  // namespace

extern "C" {

int64_t bsq_moe_layer_workspace_bytes(int32_t fmt, int32_t tokens, int64_t hidden, int64_t inter, int32_t experts,
                                      int32_t top_k) {
  if (!fmt_ok(fmt) || !moe_sizes_ok(tokens, hidden, inter, experts, top_k)) return 0;
  return 1024 + static_cast<int64_t>(tokens) * top_k * (8 + 4 * (hidden + inter));
}

int32_t bsq_moe_layer(int32_t fmt, const void* x, int64_t ld_x, const float* logits, int64_t ld_logits, const void* w13,
                      const void* w13_s, const void* w2, const void* w2_s, const float* x_sf, const float* w13_sf,
                      const float* h_sf, const float* w2_sf, void* y, int64_t ld_y, int32_t tokens, int64_t hidden,
                      int64_t inter, int32_t experts, int32_t top_k, int32_t renormalize, void* workspace,
                      int64_t workspace_bytes, void* stream) {
  if (!fmt_ok(fmt)) return BSQ_ERR_VALUE;
  if (!moe_sizes_ok(tokens, hidden, inter, experts, top_k)) return BSQ_ERR_SHAPE;
  if (tokens == 0) return BSQ_OK;
  if ((tokens > 1 && (ld_x < hidden || ld_y < hidden || ld_logits < experts))) return BSQ_ERR_SHAPE;
  if (!x || !logits || !w13 || !w13_s || !w2 || !w2_s || !y || !workspace) return BSQ_ERR_NULL;
  if (fmt == BSQ_NVFP4 && (!x_sf || !w13_sf || !h_sf || !w2_sf)) return BSQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(logits, 4) || !aligned(w13, 16) || !aligned(w13_s, 16) || !aligned(w2, 16) ||
      !aligned(w2_s, 16) || !aligned(y, 16) || !aligned(workspace, 256) || ld_x % 8 != 0 || ld_y % 8 != 0 ||
      !aligned(x_sf, 4) || !aligned(w13_sf, 4) || !aligned(h_sf, 4) || !aligned(w2_sf, 4))
    return BSQ_ERR_ALIGN;
  if (workspace_bytes < bsq_moe_layer_workspace_bytes(fmt, tokens, hidden, inter, experts, top_k)) return BSQ_ERR_SHAPE;
  HostDevice d;
  if (bsq_status s = host_device(&d); s != BSQ_OK) return s;
  MoeArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.ld_x = ld_x;
  a.logits = logits;
  a.ld_logits = ld_logits;
  a.w13 = static_cast<const uint8_t*>(w13);
  a.w13_s = static_cast<const uint8_t*>(w13_s);
  a.w2 = static_cast<const uint8_t*>(w2);
  a.w2_s = static_cast<const uint8_t*>(w2_s);
  a.w13_expert = 2 * inter * row_bytes_of(fmt, hidden);
  a.w13_s_expert = bsq_scales5d_bytes(fmt, 2 * inter, hidden);
  a.w2_expert = hidden * row_bytes_of(fmt, inter);
  a.w2_s_expert = bsq_scales5d_bytes(fmt, hidden, inter);
  a.x_sf = x_sf;
  a.w13_sf = w13_sf;
  a.h_sf = h_sf;
  a.w2_sf = w2_sf;
  a.y = static_cast<uint16_t*>(y);
  a.ld_y = ld_y;
  a.tokens = tokens;
  a.hidden = static_cast<int>(hidden);
  a.inter = static_cast<int>(inter);
  a.experts = experts;
  a.top_k = top_k;
  a.renorm = renormalize;
  uint8_t* ws = static_cast<uint8_t*>(workspace) + 1024;
  const int64_t rows = static_cast<int64_t>(tokens) * top_k;
  a.ids = reinterpret_cast<int*>(ws);
  a.probs = reinterpret_cast<float*>(ws + 4 * rows);
  a.xq = reinterpret_cast<float*>(ws + 8 * rows);
  a.h = a.xq + rows * hidden;
  a.err = d.error_word;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  switch (fmt) {
    case BSQ_NVFP4: e = launch_moe<kNVFP4>(a, st); break;
    case BSQ_MXFP4: e = launch_moe<kMXFP4>(a, st); break;
    default: e = launch_moe<kMXFP8>(a, st);
  }
  return e == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA;
}

}  // extern "C"
