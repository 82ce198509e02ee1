// Host side of the few-token mixture-of-experts layer (bsq_moe_layer):
// argument checks, the workspace's layout, tensor maps and the cooperative launch.
#include <algorithm>

#include "host_common.h"
#include "moe_layer.cuh"

namespace {

using namespace bsq;

bool moe_sizes_ok(int32_t tokens, int64_t hidden, int64_t inter, int32_t experts, int32_t top_k) {
  return tokens >= 0 && tokens <= kMoeMaxTokens && hidden >= 32 && hidden % 32 == 0 && hidden <= (1 << 16) && inter >= 128 &&
         inter % 128 == 0 && inter <= (1 << 16) && experts >= 1 && experts <= kMoeMaxExperts && top_k >= 1 &&
         top_k <= kMoeMaxTopK && top_k <= experts && experts * std::max(2 * inter, hidden) < (int64_t(1) << 31);
}

// The workspace: counters (at the same place for all sizes), then the
// tokens' operands and scales of both products, parts of split tiles, and
// each choice's rows of y.
struct MoeWorkspace {
  int64_t xq, xq_s, hq, hq_s, part, yp, bytes;
};
MoeWorkspace moe_workspace(int32_t fmt, int32_t tokens, int64_t hidden, int64_t inter, int32_t experts, int32_t top_k) {
  const int64_t pairs = static_cast<int64_t>(tokens) * top_k, active = std::min<int64_t>(experts, pairs);
  const int64_t max_n = ceil_div(tokens, 16) * 16;
  MoeWorkspace w;
  int64_t at = kMoeCounterBytes;
  auto take = [&at](int64_t bytes) {
    const int64_t p = at;
    at = ceil_div(at + bytes, 256) * 256;
    return p;
  };
  w.xq = take(pairs * row_bytes_of(fmt, hidden));
  w.xq_s = take(active * bsq_scales5d_bytes(fmt, 128, hidden));
  w.hq = take(pairs * row_bytes_of(fmt, inter));
  w.hq_s = take(active * bsq_scales5d_bytes(fmt, 128, inter));
  w.part = take(int64_t(kMoeMaxBlocks) * 2 * 2 * max_n * 128 * 4);
  w.yp = take(pairs * hidden * 4);
  w.bytes = at;
  return w;
}

// Rows of `row_bytes` bytes in boxes of 128 bytes x `box_rows` rows with the
// 128-byte swizzle; what lies past the edges reads as zeros.
bool moe_map(CUtensorMap* map, const void* ptr, int64_t rows, int64_t row_bytes, uint32_t box_rows) {
  auto enc = encode_tiled();
  if (!enc) return false;
  const cuuint64_t dim[2] = {static_cast<cuuint64_t>(row_bytes), static_cast<cuuint64_t>(rows)};
  const cuuint64_t stride[1] = {static_cast<cuuint64_t>(row_bytes)};
  const cuuint32_t box[2] = {128, box_rows}, ones[2] = {1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(ptr), dim, stride, box, ones,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Dynamic shared memory of the layer's block: what the SM allows less the kernel's static tables.
constexpr int kMoeDynamicSmem = 227 * 1024 - 1024;

template <int FMT>
bsq_status launch_moe(MoeArgs& a, const void* w13, const void* w2, const HostDevice& d, cudaStream_t st) {
  if (bsq_status s = allow_smem(reinterpret_cast<const void*>(moe_layer_kernel<FMT>), kMoeDynamicSmem, d.index); s != BSQ_OK)
    return s;
  const int64_t pairs = static_cast<int64_t>(a.tokens) * a.top_k;
  CUtensorMap m13, m2, mx, mh;
  if (!moe_map(&m13, w13, static_cast<int64_t>(a.experts) * 2 * a.inter, row_bytes_of(FMT, a.hidden), 128) ||
      !moe_map(&m2, w2, static_cast<int64_t>(a.experts) * a.hidden, row_bytes_of(FMT, a.inter), 128) ||
      !moe_map(&mx, a.xq, pairs, row_bytes_of(FMT, a.hidden), 8) || !moe_map(&mh, a.hq, pairs, row_bytes_of(FMT, a.inter), 8))
    return BSQ_ERR_CUDA;
  a.max_n = static_cast<int>(ceil_div(a.tokens, 16) * 16);
  a.stage_bytes = static_cast<int>(ceil_div(2 * kMoeHalfBytes + a.max_n * 128 + 3 * MoeFmt<FMT>::kAtoms * 512, 1024) * 1024);
  const int tables = moe_table_bytes(a.experts, static_cast<int>(pairs));
  // all that fits: one token 50.9 us, 50.7 with three stages only; 64 tokens 649 and 656
  a.stages = std::min(8, (kMoeDynamicSmem - 1024 - tables) / a.stage_bytes);
  if (a.stages < 2) return BSQ_ERR_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(std::min(d.sm_count, kMoeMaxBlocks));
  cfg.blockDim = dim3(kMoeThreads);
  cfg.dynamicSmemBytes = 1024 + a.stages * a.stage_bytes + tables;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;  // the blocks wait for one another
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, moe_layer_kernel<FMT>, m13, m2, mx, mh, a) == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA;
}

__device__ uint32_t g_selftest_count;  // stays 0

// The serving kernels' waits, each on something that nothing completes, with limits of about a millisecond; then
// once more where another role has given up, and on what is complete.
__global__ void serving_waits_selftest_kernel(unsigned int* err) {
  __shared__ uint64_t never, done;
  __shared__ volatile uint32_t abort_flag;
  pdl_wait();
  if (threadIdx.x != 0) return;
  constexpr long long kLimit = 2000000;
  mbar_init(&never, 1);
  mbar_init(&done, 1);
  abort_flag = 0u;
  fence_mbar_init();
  mbar_arrive(&done);
  const long long t0 = clock64();
  bool right = !mbar_wait_clocked(&never, 0, &abort_flag, kLimit) && !mbar_wait_clocked(&never, 0, kLimit) &&
               !moe_wait_count(&g_selftest_count, 1u, &abort_flag, kLimit) && clock64() - t0 >= 3 * kLimit;
  right = right && mbar_wait_clocked(&done, 0, &abort_flag) && mbar_wait_clocked(&done, 0) && moe_wait_count(&g_selftest_count, 0u, &abort_flag);
  abort_flag = 1u;
  const long long t1 = clock64();
  right = right && !mbar_wait_clocked(&never, 0, &abort_flag) && !moe_wait_count(&g_selftest_count, 1u, &abort_flag) &&
          clock64() - t1 < kWaitLimitCycles;
  record_error_at(err, right ? kErrTimeout : kErrValue);
}

}  // namespace

extern "C" {

int32_t bsq_selftest_serving_waits(void* stream) {
  HostDevice d;
  if (bsq_status s = host_device(&d); s != BSQ_OK) return s;
  return launch_pdl(serving_waits_selftest_kernel, dim3(1), dim3(32), 0, static_cast<cudaStream_t>(stream), d.error_word) == cudaSuccess
             ? BSQ_OK
             : BSQ_ERR_CUDA;
}

int64_t bsq_moe_layer_workspace_bytes(int32_t fmt, int32_t tokens, int64_t hidden, int64_t inter, int32_t experts,
                                      int32_t top_k) {
  if (!fmt_ok(fmt) || !moe_sizes_ok(tokens, hidden, inter, experts, top_k)) return 0;
  return moe_workspace(fmt, tokens, hidden, inter, experts, top_k).bytes;
}

int64_t bsq_moe_layer_counter_bytes(void) { return kMoeCounterBytes; }

int32_t bsq_moe_layer(int32_t fmt, const void* x, int64_t ld_x, const float* logits, int64_t ld_logits, const void* w13,
                      const void* w13_s, const void* w2, const void* w2_s, const float* x_sf, const float* w13_sf,
                      const float* h_sf, const float* w2_sf, void* y, int64_t ld_y, int32_t tokens, int64_t hidden,
                      int64_t inter, int32_t experts, int32_t top_k, int32_t renormalize, void* workspace,
                      int64_t workspace_bytes, void* stream) {
  if (!fmt_ok(fmt)) return BSQ_ERR_VALUE;
  if (!moe_sizes_ok(tokens, hidden, inter, experts, top_k)) return BSQ_ERR_SHAPE;
  if (tokens == 0) return BSQ_OK;
  if (tokens > 1 && (ld_x < hidden || ld_y < hidden || ld_logits < experts)) return BSQ_ERR_SHAPE;
  if (!x || !logits || !w13 || !w13_s || !w2 || !w2_s || !y || !workspace) return BSQ_ERR_NULL;
  if (fmt == BSQ_NVFP4 && (!x_sf || !w13_sf || !h_sf || !w2_sf)) return BSQ_ERR_NULL;
  if (!aligned(x, 16) || !aligned(logits, 4) || !aligned(w13, 16) || !aligned(w13_s, 16) || !aligned(w2, 16) ||
      !aligned(w2_s, 16) || !aligned(y, 16) || !aligned(workspace, 256) || ld_x % 8 != 0 || ld_y % 8 != 0 ||
      !aligned(x_sf, 4) || !aligned(w13_sf, 4) || !aligned(h_sf, 4) || !aligned(w2_sf, 4))
    return BSQ_ERR_ALIGN;
  const MoeWorkspace w = moe_workspace(fmt, tokens, hidden, inter, experts, top_k);
  if (workspace_bytes < w.bytes) return BSQ_ERR_SHAPE;
  HostDevice d;
  if (bsq_status s = host_device(&d); s != BSQ_OK) return s;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  MoeArgs a{};
  a.x = static_cast<const uint16_t*>(x);
  a.ld_x = ld_x;
  a.logits = logits;
  a.ld_logits = ld_logits;
  a.w13_s = static_cast<const uint8_t*>(w13_s);
  a.w2_s = static_cast<const uint8_t*>(w2_s);
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
  a.counters = reinterpret_cast<uint32_t*>(ws);
  a.xq = ws + w.xq;
  a.xq_s = ws + w.xq_s;
  a.hq = ws + w.hq;
  a.hq_s = ws + w.hq_s;
  a.part = reinterpret_cast<float*>(ws + w.part);
  a.yp = reinterpret_cast<float*>(ws + w.yp);
  a.err = d.error_word;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  switch (fmt) {
    case BSQ_NVFP4: return launch_moe<kNVFP4>(a, w13, w2, d, st);
    case BSQ_MXFP4: return launch_moe<kMXFP4>(a, w13, w2, d, st);
    default: return launch_moe<kMXFP8>(a, w13, w2, d, st);
  }
}

}  // extern "C"
