// Host side of the norm and rotation of query and key heads (bsq_qk_norm_rope).
#include <algorithm>
#include <cmath>

#include "host_common.h"
#include "host_regions.h"
#include "qk_norm_rope.cuh"

namespace {

using namespace bsq;

template <bool F16, int L>
cudaError_t launch_rope(const RopeArgs& a, int mode, unsigned grid, cudaStream_t st) {
  const dim3 g(grid), b(kRopeWarps * 32);
  if (mode == 0) return launch_pdl(qk_norm_rope_kernel<F16, L, 0>, g, b, 0, st, a);
  if (mode == 1) return launch_pdl(qk_norm_rope_kernel<F16, L, 1>, g, b, 0, st, a);
  return launch_pdl(qk_norm_rope_kernel<F16, L, 2>, g, b, 0, st, a);
}

template <bool F16>
cudaError_t launch_rope_dim(const RopeArgs& a, int mode, unsigned grid, cudaStream_t st) {
  if (a.dim <= 64) return launch_rope<F16, 8>(a, mode, grid, st);
  if (a.dim <= 128) return launch_rope<F16, 16>(a, mode, grid, st);
  return launch_rope<F16, 32>(a, mode, grid, st);
}

// Strides that keep every element's offset within 63 bits.
bool stride_ok(int64_t s) { return s >= 0 && s < (int64_t(1) << 31); }

}  // namespace

extern "C" int32_t bsq_qk_norm_rope(int32_t dtype, const void* q, int64_t q_tok, int64_t q_head, const void* k, int64_t k_tok,
                                    int64_t k_head, int64_t tokens, int32_t heads, int32_t kv_heads, int32_t dim,
                                    const int32_t* positions, const float* inv_freq, int32_t pairs, int32_t interleaved,
                                    const void* q_weight, const void* k_weight, int32_t weight_dtype, float eps, void* q_out,
                                    int64_t qo_tok, int64_t qo_head, void* k_out, int64_t ko_tok, int64_t ko_head, void* stream) {
  if (dtype != BSQ_BF16 && dtype != BSQ_F16) return BSQ_ERR_VALUE;
  if ((q_weight || k_weight) && weight_dtype != dtype && weight_dtype != BSQ_F32) return BSQ_ERR_VALUE;
  if (!(eps >= 0.f) || std::isinf(eps)) return BSQ_ERR_VALUE;
  if (tokens < 0 || tokens >= (int64_t(1) << 31) || heads < 0 || kv_heads < 0 || heads > 4096 || kv_heads > 4096 || dim < 8 || dim > 256 ||
      dim % 8 != 0 || pairs < 0 || 2 * pairs > dim || !stride_ok(q_tok) || !stride_ok(q_head) || !stride_ok(k_tok) || !stride_ok(k_head) ||
      !stride_ok(qo_tok) || !stride_ok(qo_head) || !stride_ok(ko_tok) || !stride_ok(ko_head))
    return BSQ_ERR_SHAPE;
  const int rows = heads + kv_heads;
  if (tokens == 0 || rows == 0) return BSQ_OK;
  if ((heads && (!q || !q_out)) || (kv_heads && (!k || !k_out)) || !positions || (pairs && !inv_freq)) return BSQ_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) || !aligned(positions, 4) || !aligned(inv_freq, 4) ||
      (q_tok | q_head | k_tok | k_head | qo_tok | qo_head | ko_tok | ko_head) % 8 != 0 ||
      !aligned(q_weight, weight_dtype == BSQ_F32 ? 4 : 2) || !aligned(k_weight, weight_dtype == BSQ_F32 ? 4 : 2))
    return BSQ_ERR_ALIGN;
  if ((heads > 1 && qo_head < dim) || (kv_heads > 1 && ko_head < dim) || (tokens > 1 && ((heads && qo_tok < dim) || (kv_heads && ko_tok < dim))))
    return BSQ_ERR_SHAPE;
  // [input, output][queries, keys]
  const auto rows_of = [&](const void* at, int64_t tok, int64_t head, int n) {
    return HostRegion{n ? at : nullptr, dim * int64_t(2), {tokens, n}, {tok * 2, head * 2}};
  };
  const HostRegion io[2][2] = {{rows_of(q, q_tok, q_head, heads), rows_of(k, k_tok, k_head, kv_heads)},
                               {rows_of(q_out, qo_tok, qo_head, heads), rows_of(k_out, ko_tok, ko_head, kv_heads)}};
  const int64_t weight_bytes = dim * int64_t(weight_dtype == BSQ_F32 ? 4 : 2);
  const HostRegion also[4] = {host_region(positions, tokens * 4), host_region(inv_freq, pairs * int64_t(4)), host_region(q_weight, weight_bytes),
                              host_region(k_weight, weight_bytes)};
  for (int i = 0; i < 2; ++i) {
    const HostRegion &in = io[0][i], &out = io[1][i];
    const bool itself = in.at == out.at && (tokens == 1 || in.step[0] == out.step[0]) && (in.n[1] == 1 || in.step[1] == out.step[1]);
    if ((!itself && regions_overlap(out, in)) || regions_overlap(out, io[0][1 - i])) return BSQ_ERR_VALUE;
    for (const HostRegion& r : also)
      if (regions_overlap(out, r)) return BSQ_ERR_VALUE;
  }
  if (regions_overlap(io[1][0], io[1][1])) return BSQ_ERR_VALUE;
  if (region_overlaps_itself(io[1][0]) || region_overlaps_itself(io[1][1])) return BSQ_ERR_SHAPE;
  HostDevice d;
  if (bsq_status s = host_device(&d); s != BSQ_OK) return s;
  RopeArgs a{};
  a.src[0] = static_cast<const uint16_t*>(q);
  a.src[1] = static_cast<const uint16_t*>(k);
  a.dst[0] = static_cast<uint16_t*>(q_out);
  a.dst[1] = static_cast<uint16_t*>(k_out);
  a.src_tok[0] = q_tok;
  a.src_tok[1] = k_tok;
  a.src_head[0] = q_head;
  a.src_head[1] = k_head;
  a.dst_tok[0] = qo_tok;
  a.dst_tok[1] = ko_tok;
  a.dst_head[0] = qo_head;
  a.dst_head[1] = ko_head;
  a.weight[0] = q_weight;
  a.weight[1] = k_weight;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.tokens = tokens;
  a.heads = heads;
  a.rows = rows;
  a.dim = dim;
  a.pairs = pairs;
  a.weight_f32 = weight_dtype == BSQ_F32;
  a.eps = eps;
  a.inv_dim = 1.f / static_cast<float>(dim);
  // a warp takes a token's rows, or, where there are too few tokens for 16 warps per SM, an equal share of them (512 tokens of 72 heads then 6.7 us,
  // with 4 warps per SM 8.1, with 64 9.3; 257 tokens of 32 heads 3.6, with 32 or 64 4.7: each warp works out the token's angles)
  const int at_once = dim <= 64 ? 4 : dim <= 128 ? 2 : 1;
  const int steps = static_cast<int>(ceil_div(rows, at_once));
  const int want = static_cast<int>(std::min<int64_t>(steps, ceil_div(int64_t(d.sm_count) * 16, tokens)));
  const int per = static_cast<int>(ceil_div(steps, want));
  a.chunks = static_cast<int>(ceil_div(steps, per));
  a.per_chunk = per * at_once;
  const int mode = interleaved ? 1 : pairs % 4 == 0 ? 0 : 2;
  const int64_t grid = ceil_div(tokens * a.chunks, kRopeWarps);
  if (grid >= (int64_t(1) << 31)) return BSQ_ERR_SHAPE;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == BSQ_F16 ? launch_rope_dim<true>(a, mode, static_cast<unsigned>(grid), st)
                                         : launch_rope_dim<false>(a, mode, static_cast<unsigned>(grid), st);
  return e == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA;
}
