// Host side of the routing to experts (bsq_moe_route, bsq_moe_rows).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "host_common.h"
#include "host_regions.h"
#include "moe_route.cuh"

namespace {

using namespace bsq;

template <int DTYPE, int NL>
cudaError_t launch_route(const RouteArgs& a, bool pair, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(ceil_div(a.tokens, kRouteWarps))), block(kRouteWarps * 32);
  const size_t smem = a.groups > 1 || pair ? sizeof(RouteFF) * kRouteWarps * a.experts : 0;
  return pair ? launch_pdl(moe_route_kernel<DTYPE, NL, true>, grid, block, smem, st, a)
              : launch_pdl(moe_route_kernel<DTYPE, NL, false>, grid, block, smem, st, a);
}

template <int DTYPE>
cudaError_t launch_route_experts(const RouteArgs& a, bool pair, cudaStream_t st) {
  if (a.experts <= 64) return launch_route<DTYPE, 2>(a, pair, st);
  if (a.experts <= 128) return launch_route<DTYPE, 4>(a, pair, st);
  if (a.experts <= 256) return launch_route<DTYPE, 8>(a, pair, st);
  if (a.experts <= 512) return launch_route<DTYPE, 16>(a, pair, st);
  return launch_route<DTYPE, 32>(a, pair, st);
}

}  // namespace

extern "C" {

int32_t bsq_moe_route(int32_t dtype, const void* logits, int64_t ld_logits, int64_t tokens, int32_t experts, int32_t top_k,
                      int32_t sigmoid, const float* bias, int32_t groups, int32_t top_groups, int32_t group_top, int32_t renormalize,
                      float scale, int32_t* ids, float* weights, void* stream) {
  if (dtype != BSQ_BF16 && dtype != BSQ_F16 && dtype != BSQ_F32) return BSQ_ERR_VALUE;
  if (!std::isfinite(scale)) return BSQ_ERR_VALUE;
  if (tokens < 0 || tokens >= (int64_t(1) << 31) || experts < 1 || experts > kRouteMaxExperts || top_k < 1 || top_k > kRouteMaxTopK ||
      groups < 1 || groups > kRouteMaxGroups || experts % groups != 0 || top_groups < 1 || top_groups > groups ||
      group_top < 1 || group_top > 2 || top_k > experts / groups * top_groups || (tokens > 1 && ld_logits < experts) || ld_logits < 0 ||
      ld_logits >= (int64_t(1) << 31))
    return BSQ_ERR_SHAPE;
  if (tokens == 0) return BSQ_OK;
  if (!logits || !ids || !weights) return BSQ_ERR_NULL;
  if (!aligned(logits, dtype == BSQ_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4)) return BSQ_ERR_ALIGN;
  const int64_t wide = dtype == BSQ_F32 ? 4 : 2, out_bytes = tokens * top_k * 4;
  const HostRegion in = {logits, experts * wide, {tokens, 1}, {ld_logits * wide, 0}}, of_bias = host_region(bias, experts * int64_t(4)),
                   out[2] = {host_region(ids, out_bytes), host_region(weights, out_bytes)};
  if (regions_overlap(out[0], out[1])) return BSQ_ERR_VALUE;
  for (const HostRegion& o : out)
    if (regions_overlap(o, in) || regions_overlap(o, of_bias)) return BSQ_ERR_VALUE;
  HostDevice d;
  if (bsq_status s = host_device(&d); s != BSQ_OK) return s;
  RouteArgs a{};
  a.logits = logits;
  a.ld = ld_logits;
  a.tokens = tokens;
  a.bias = bias;
  a.experts = experts;
  a.top_k = top_k;
  a.groups = groups;
  a.top_groups = top_groups;
  a.group_top = group_top;
  a.per = experts / groups;
  a.inv = ((1u << 20) + a.per - 1) / a.per;
  a.span_log = 5;
  while (groups << a.span_log > 32) --a.span_log;
  a.sigmoid = sigmoid != 0;
  a.renorm = renormalize != 0;
  a.scale = scale;
  a.ids = ids;
  a.weights = weights;
  a.err = d.error_word;
  const bool pair = bias || (groups > 1 && group_top == 2);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == BSQ_F32 ? launch_route_experts<2>(a, pair, st)
                        : dtype == BSQ_F16 ? launch_route_experts<1>(a, pair, st)
                                           : launch_route_experts<0>(a, pair, st);
  return e == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA;
}

int32_t bsq_moe_rows(const int32_t* ids, int64_t tokens, int32_t top_k, int32_t experts, uint32_t* row_offsets,
                     uint32_t* scales_offsets, int32_t* row_indices, int32_t* positions, void* stream) {
  if (tokens < 0 || top_k < 1 || top_k > kRouteMaxExperts || experts < 1 || experts > kRouteMaxExperts ||
      tokens > (int64_t(1) << 30) / top_k)
    return BSQ_ERR_SHAPE;
  const int64_t pairs = tokens * top_k;
  if (!row_offsets || !scales_offsets || (pairs && (!ids || !row_indices || !positions))) return BSQ_ERR_NULL;
  if (!aligned(ids, 4) || !aligned(row_offsets, 4) || !aligned(scales_offsets, 4) || !aligned(row_indices, 4) || !aligned(positions, 4))
    return BSQ_ERR_ALIGN;
  const HostRegion all[5] = {host_region(ids, pairs * 4), host_region(row_offsets, (experts + 1) * int64_t(4)),
                             host_region(scales_offsets, (experts + 1) * int64_t(4)), host_region(row_indices, pairs * 4), host_region(positions, pairs * 4)};
  for (int i = 1; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (regions_overlap(all[i], all[j])) return BSQ_ERR_VALUE;
  HostDevice d;
  if (bsq_status s = host_device(&d); s != BSQ_OK) return s;
  RowsArgs a{};
  a.ids = ids;
  a.pairs = pairs;
  a.top_k = top_k;
  a.experts = experts;
  // one block up to a round of 32 pairs per warp, then as many as give each warp such a round, at most a cluster (figures: moe_route.cuh)
  const int64_t rounds = std::max<int64_t>(1, ceil_div(pairs, 32 * kRowsWarps));
  int blocks = 1;
  while (blocks < kRowsMaxBlocks && blocks < rounds) blocks *= 2;
  a.run = ceil_div(ceil_div(std::max<int64_t>(pairs, 1), int64_t(blocks) * kRowsWarps), 32) * 32;
  a.row_offsets = row_offsets;
  a.scales_offsets = scales_offsets;
  a.row_indices = row_indices;
  a.positions = positions;
  a.err = d.error_word;
  const int smem = rows_smem_bytes(experts);
  const auto kernel = a.run <= 32 * kRowsHeld ? moe_rows_kernel<true> : moe_rows_kernel<false>;
  if (bsq_status s = allow_smem(reinterpret_cast<const void*>(kernel), rows_smem_bytes(kRouteMaxExperts), d.index); s != BSQ_OK) return s;
  if (blocks > 8 && cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) return BSQ_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kRowsThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = blocks;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a) == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA;
}

}  // extern "C"
