// Host side of the 8-bit paged key/value cache: argument checks and launch
// geometry of bsq_kv_append and bsq_kv_attention (include/bsq.h).
#include <algorithm>
#include <cfloat>
#include <cmath>

#include "host_common.h"
#include "kv_append.cuh"
#include "kv_attention.cuh"
#include "kv_prompt.cuh"

namespace {

using namespace bsq;

// Positions, and rows of a kv head, that leave 32-bit sums of two of them, a window and a tile's end in range.
constexpr int64_t kKvMaxLen = int64_t(1) << 30;

// What the cache calls check alike; BSQ_OK when the call may go on.
bsq_status check_cache(int32_t dtype, int64_t total, int32_t kv_heads, int32_t dim, int64_t tok_stride, int64_t head_stride,
                       const void* k_cache, const void* v_cache, const void* k_scales, const void* v_scales,
                       int64_t num_pages, int32_t page, int64_t cs_page, int64_t cs_head, int64_t cs_tok,
                       const int32_t* table, int64_t table_ld, int32_t table_width, const int32_t* offsets,
                       const int32_t* lens, int32_t batch) {
  if (dtype != BSQ_BF16 && dtype != BSQ_F16) return BSQ_ERR_VALUE;
  if (total < 0 || total >= (int64_t(1) << 31) || batch < 0 || kv_heads < 1 || kv_heads > 1024 || (dim != 64 && dim != 128) ||
      num_pages < 1 || num_pages >= (int64_t(1) << 31) || (page != 16 && page != 32 && page != 64 && page != 128) ||
      table_width < 0 || static_cast<int64_t>(table_width) * page > kKvMaxLen || (batch > 1 && table_ld < table_width) || cs_tok < dim || cs_page < 0 || cs_head < 0 ||
      total / page + 2 * static_cast<int64_t>(batch) >= (int64_t(1) << 31) ||  // blocks of an append
      cs_tok >= (int64_t(1) << 32) || cs_head >= (int64_t(1) << 38) || cs_page >= (int64_t(1) << 38))
    return BSQ_ERR_SHAPE;
  if (total == 0 || batch == 0) return BSQ_OK;
  if (!table || !offsets || !lens || !k_cache || !v_cache || !k_scales || !v_scales) return BSQ_ERR_NULL;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || cs_page % 16 != 0 || cs_head % 16 != 0 || cs_tok % 16 != 0 ||
      tok_stride % 8 != 0 || head_stride % 8 != 0 || !aligned(table, 4) || !aligned(offsets, 4) || !aligned(lens, 4))
    return BSQ_ERR_ALIGN;
  return BSQ_OK;
}

template <int D, bool F16>
cudaError_t launch_append(const KvAppendArgs& a, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.total / a.page + 2 * static_cast<int64_t>(a.batch)), 2u * a.kv_heads);
  switch (a.page * (D / 8) / kKvAppendThreads) {
    case 1: return launch_pdl(kv_append_kernel<D, 1, F16>, grid, dim3(kKvAppendThreads), 0, st, a);
    case 2: return launch_pdl(kv_append_kernel<D, 2, F16>, grid, dim3(kKvAppendThreads), 0, st, a);
    case 4: return launch_pdl(kv_append_kernel<D, 4, F16>, grid, dim3(kKvAppendThreads), 0, st, a);
    case 8: return launch_pdl(kv_append_kernel<D, 8, F16>, grid, dim3(kKvAppendThreads), 0, st, a);
    default: return launch_pdl(kv_append_kernel<D, 16, F16>, grid, dim3(kKvAppendThreads), 0, st, a);
  }
}

// Rows (query tokens x heads of a kv head) up to which the kernel for few rows runs: its
// largest tile.  64 contexts of 1000 to 8192, 64 heads over 8: 32 rows 248 us there and 305 in the kernel for many,
// 64 rows 480 and 307.  Eight contexts to 2000, 32 rows: 26 and 37.
constexpr int kKvFewRows = 32;

// The cache as a 4D tensor of bytes (dimension, token, head, page), in boxes
// of a head's tokens, at most `tile` of them.
bool cache_map(CUtensorMap* map, const void* ptr, int dim, int page, int heads, int64_t pages, int64_t cs_tok, int64_t cs_head,
               int64_t cs_page, int tile, CUtensorMapSwizzle swizzle) {
  auto enc = encode_tiled();
  if (!enc) return false;
  // the stride of an extent of one is never used, but has to be valid
  if (heads == 1) cs_head = cs_tok * page;
  if (pages == 1) cs_page = cs_tok * page;
  const cuuint64_t size[4] = {static_cast<cuuint64_t>(dim), static_cast<cuuint64_t>(page), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(pages)};
  const cuuint64_t stride[3] = {static_cast<cuuint64_t>(cs_tok), static_cast<cuuint64_t>(cs_head), static_cast<cuuint64_t>(cs_page)};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(dim), static_cast<cuuint32_t>(std::min(page, tile)), 1, 1};
  const cuuint32_t ones[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), size, stride, box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE,
             swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int NT, bool F16>
bsq_status launch_attention(const KvAttnArgs& a, const CUtensorMap& mk, const CUtensorMap& mv, const HostDevice& d,
                            cudaStream_t st) {
  using S = KvShape<D, NT>;
  auto kernel = kv_attention_kernel<D, NT, F16>;
  if (bsq_status s = allow_smem(reinterpret_cast<const void*>(kernel), S::kSmem, d.index); s != BSQ_OK) return s;
  const int grid = std::min(d.sm_count * S::kBlocksPerSm, NT == 4 ? kKvMaxBlocks / 2 : kKvMaxBlocks);
  return launch_pdl(kernel, dim3(grid), dim3(S::kThreads), S::kSmem, st, mk, mv, a) == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA;
}

template <int D, bool F16>
bsq_status launch_attention_rows(const KvAttnArgs& a, int64_t max_rows, const CUtensorMap& mk, const CUtensorMap& mv,
                                 const HostDevice& d, cudaStream_t st) {
  // the narrowest tile that holds all rows (those 64 contexts: 8 rows 101 / 115 / 236 us in tiles of 8 / 16 / 32,
  // 16 rows 118 / 240 in tiles of 16 / 32): unused rows are products, registers and warps per SM lost
  if (max_rows <= 8) return launch_attention<D, 1, F16>(a, mk, mv, d, st);
  if (max_rows <= 16) return launch_attention<D, 2, F16>(a, mk, mv, d, st);
  if (max_rows <= kKvFewRows) return launch_attention<D, 4, F16>(a, mk, mv, d, st);
  auto kernel = kv_prompt_kernel<D, F16>;
  if (bsq_status s = allow_smem(reinterpret_cast<const void*>(kernel), KpShape<D>::kSmem, d.index); s != BSQ_OK) return s;
  return launch_pdl(kernel, dim3(std::min(d.sm_count, kKpMaxBlocks)), dim3(kKpThreads), KpShape<D>::kSmem, st, mk, mv, a) == cudaSuccess
             ? BSQ_OK
             : BSQ_ERR_CUDA;
}

}  // namespace

extern "C" {

int32_t bsq_kv_append(int32_t dtype, const void* k, const void* v, int64_t total, int32_t kv_heads, int32_t dim,
                      int64_t src_tok, int64_t src_head, void* k_cache, void* v_cache, void* k_scales, void* v_scales,
                      int64_t num_pages, int32_t page, int64_t cs_page, int64_t cs_head, int64_t cs_tok,
                      const int32_t* table, int64_t table_ld, int32_t table_width, const int32_t* offsets,
                      const int32_t* lens, int32_t batch, void* stream) {
  return bsq_kv_append_strided(dtype, k, v, total, kv_heads, dim, src_tok, src_head, src_tok, src_head, k_cache, v_cache, k_scales,
                               v_scales, num_pages, page, cs_page, cs_head, cs_tok, table, table_ld, table_width, offsets, lens,
                               batch, stream);
}

int32_t bsq_kv_append_strided(int32_t dtype, const void* k, const void* v, int64_t total, int32_t kv_heads, int32_t dim,
                              int64_t k_tok, int64_t k_head, int64_t v_tok, int64_t v_head, void* k_cache, void* v_cache,
                              void* k_scales, void* v_scales, int64_t num_pages, int32_t page, int64_t cs_page, int64_t cs_head,
                              int64_t cs_tok, const int32_t* table, int64_t table_ld, int32_t table_width,
                              const int32_t* offsets, const int32_t* lens, int32_t batch, void* stream) {
  if (bsq_status s = check_cache(dtype, total, kv_heads, dim, k_tok, k_head, k_cache, v_cache, k_scales, v_scales,
                                 num_pages, page, cs_page, cs_head, cs_tok, table, table_ld, table_width, offsets, lens, batch);
      s != BSQ_OK)
    return s;
  if (total == 0 || batch == 0) return BSQ_OK;
  if (!k || !v) return BSQ_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || v_tok % 8 != 0 || v_head % 8 != 0) return BSQ_ERR_ALIGN;
  HostDevice d;
  if (bsq_status s = host_device(&d); s != BSQ_OK) return s;
  KvAppendArgs a{};
  a.src[0] = static_cast<const uint16_t*>(k);
  a.src[1] = static_cast<const uint16_t*>(v);
  a.src_tok[0] = k_tok;
  a.src_tok[1] = v_tok;
  a.src_head[0] = k_head;
  a.src_head[1] = v_head;
  a.cache[0] = static_cast<uint8_t*>(k_cache);
  a.cache[1] = static_cast<uint8_t*>(v_cache);
  a.cs_page = cs_page;
  a.cs_head = cs_head;
  a.cs_tok = cs_tok;
  a.scales[0] = static_cast<uint8_t*>(k_scales);
  a.scales[1] = static_cast<uint8_t*>(v_scales);
  a.table = table;
  a.table_ld = table_ld;
  a.offsets = offsets;
  a.lens = lens;
  a.total = total;
  a.num_pages = num_pages;
  a.batch = batch;
  a.kv_heads = kv_heads;
  a.page = page;
  a.table_width = table_width;
  a.err = d.error_word;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (dim == 64)
    e = dtype == BSQ_F16 ? launch_append<64, true>(a, st) : launch_append<64, false>(a, st);
  else
    e = dtype == BSQ_F16 ? launch_append<128, true>(a, st) : launch_append<128, false>(a, st);
  return e == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA;
}

int64_t bsq_kv_attention_workspace_bytes(int64_t total, int32_t heads, int32_t kv_heads, int32_t dim, int32_t batch,
                                         int32_t max_q) {
  if (total < 0 || heads < 1 || kv_heads < 1 || heads % kv_heads != 0 || (dim != 64 && dim != 128) || batch < 0 || max_q < 0)
    return 0;
  if (static_cast<int64_t>(max_q) * (heads / kv_heads) > kKvFewRows)
    return kKvCounterBytes + 2 * int64_t(kKpMaxBlocks) * (dim == 64 ? KpShape<64>::kPartFloats : KpShape<128>::kPartFloats) * 4;
  // two parts of 16 rows for each of the blocks, or of 32 for half as many
  return kKvCounterBytes + 2 * int64_t(kKvMaxBlocks) * KvShape<128, 2>::kPartFloats * 4;
}

int64_t bsq_kv_attention_counter_bytes(void) { return kKvCounterBytes; }

int32_t bsq_workspace_zero(void* workspace, int64_t bytes, void* stream) {
  if (bytes < 0) return BSQ_ERR_SHAPE;
  if (bytes == 0) return BSQ_OK;
  if (!workspace) return BSQ_ERR_NULL;
  return cudaMemsetAsync(workspace, 0, static_cast<size_t>(bytes), static_cast<cudaStream_t>(stream)) == cudaSuccess ? BSQ_OK : BSQ_ERR_CUDA;
}

int32_t bsq_kv_attention(int32_t dtype, const void* q, int64_t total, int32_t heads, int32_t kv_heads, int32_t dim,
                         int64_t q_tok, int64_t q_head, const void* k_cache, const void* v_cache, const void* k_scales,
                         const void* v_scales, int64_t num_pages, int32_t page, int64_t cs_page, int64_t cs_head,
                         int64_t cs_tok, const int32_t* table, int64_t table_ld, int32_t table_width,
                         const int32_t* offsets, const int32_t* lens, int32_t batch, int32_t max_q, float sm_scale,
                         int32_t causal, int32_t window, void* out, float* lse, void* workspace, int64_t workspace_bytes,
                         void* stream) {
  if (bsq_status s = check_cache(dtype, total, kv_heads, dim, q_tok, q_head, k_cache, v_cache, k_scales, v_scales, num_pages,
                                 page, cs_page, cs_head, cs_tok, table, table_ld, table_width, offsets, lens, batch);
      s != BSQ_OK)
    return s;
  if (heads < 1 || heads % kv_heads != 0 || heads / kv_heads > 64 || total * (heads / kv_heads) > kKvMaxLen || window < 0 ||
      max_q < 0)
    return BSQ_ERR_SHAPE;
  if (!std::isfinite(sm_scale)) return BSQ_ERR_VALUE;
  if (total == 0 || batch == 0) return BSQ_OK;
  if (max_q < 1) return BSQ_ERR_SHAPE;
  if (!q || !out || !workspace) return BSQ_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(workspace, 16)) return BSQ_ERR_ALIGN;
  if (workspace_bytes < bsq_kv_attention_workspace_bytes(total, heads, kv_heads, dim, batch, max_q)) return BSQ_ERR_SHAPE;
  HostDevice d;
  if (bsq_status s = host_device(&d); s != BSQ_OK) return s;
  KvAttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_tok = q_tok;
  a.q_head = q_head;
  a.scales[0] = static_cast<const uint8_t*>(k_scales);
  a.scales[1] = static_cast<const uint8_t*>(v_scales);
  a.table = table;
  a.table_ld = table_ld;
  a.offsets = offsets;
  a.lens = lens;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.total = total;
  a.num_pages = num_pages;
  a.batch = batch;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.group = heads / kv_heads;
  a.group_inv = a.group > 1 ? ~uint64_t{0} / static_cast<uint64_t>(a.group) + 1 : 0;
  a.page = page;
  a.page_shift = page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : 7;
  a.table_width = table_width;
  a.causal = causal;
  a.window = window < kKvMaxLen ? window : 0;  // no two positions are that far apart
  int exponent;
  const float scale = std::fmin(std::fabs(sm_scale * 1.4426950408889634f), FLT_MAX);
  const float significand = std::frexp(scale, &exponent);  // 0, or in [1/2, 1)
  a.scale_sig = 2.f * significand;
  a.scale_pow = std::copysign(std::ldexp(1.f, exponent - 1), sm_scale);
  a.arrived = static_cast<uint32_t*>(workspace);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kKvCounterBytes);
  a.err = d.error_word;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  CUtensorMap mk, mv;
  const int64_t max_rows = static_cast<int64_t>(max_q) * a.group;
  const bool few = max_rows <= kKvFewRows;
  const int tile = few ? kKvTile : kKpKeys;
  const CUtensorMapSwizzle swizzle = !few ? CU_TENSOR_MAP_SWIZZLE_NONE : dim == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  auto at = replace_address();
  if (!at || !cache_map(&mk, k_cache, dim, page, kv_heads, num_pages, cs_tok, cs_head, cs_page, tile, swizzle)) return BSQ_ERR_CUDA;
  mv = mk;  // the values' map differs in its address alone
  if (at(&mv, const_cast<void*>(v_cache)) != CUDA_SUCCESS)
    return BSQ_ERR_CUDA;
  if (dim == 64)
    return dtype == BSQ_F16 ? launch_attention_rows<64, true>(a, max_rows, mk, mv, d, st)
                            : launch_attention_rows<64, false>(a, max_rows, mk, mv, d, st);
  return dtype == BSQ_F16 ? launch_attention_rows<128, true>(a, max_rows, mk, mv, d, st)
                          : launch_attention_rows<128, false>(a, max_rows, mk, mv, d, st);
}

}  // extern "C"
