// New keys and values into the 8-bit paged cache.
//
// A page of a kv head holds E4M3 codes under one power-of-two scale 2^e,
// with e = ceil(log2(amax / 448)) kept at or above kKvMinExp.  Tokens that
// continue a page can raise e: the page's earlier codes c are then rewritten
// as E4M3(c 2^(e_old - e)), which changes only those that fall into the
// subnormal range (a power of two leaves the significand as it is).  A page
// whose first token is new takes its scale from the new tokens alone.
//
// One block of 128 threads per (page that new tokens reach, kv head, key or
// value): the page's new rows are read once, stay in registers over the
// maximum and are written as codes.  Bound by DRAM for prompts (2 bytes read
// and 1 written per element), by latency for single tokens.  A block holds a whole page's
// rows, so that no maximum crosses blocks and nothing is read twice; ITERS follows from the page's size.
// Measured (8 kv heads of 128, pages of 64): six prompts of up to 4500 tokens 24 us,
// 5.4 TB/s or 80 % of a plain copy; a token for each of 64 sequences 5.9 us, most of it the
// chain offsets, table, row, maximum, earlier codes.
#pragma once

#include "serving_common.cuh"

namespace bsq {

constexpr int kKvMinExp = -32;  // least scale exponent of a page
constexpr int kKvAppendThreads = 128;

struct KvAppendArgs {
  const uint16_t* src[2];        // new keys, values: (total, kv_heads, D)
  int64_t src_tok[2], src_head[2];  // strides in elements
  uint8_t* cache[2];             // codes, page p head h token t at p*cs_page + h*cs_head + t*cs_tok
  int64_t cs_page, cs_head, cs_tok;
  uint8_t* scales[2];            // (num_pages, kv_heads) E8M0 bytes
  const int32_t* table;          // (batch, table_ld)
  int64_t table_ld;
  const int32_t* offsets;        // [batch + 1]
  const int32_t* lens;           // [batch]
  int64_t total, num_pages;
  int batch, kv_heads, page, table_width;
  unsigned int* err;
};

// Blocks are numbered per sequence from first_slot(b) = offsets[b] / page + 2 b:
// n tokens reach at most floor((n - 1) / page) + 2 pages, so no two sequences
// share a number, and the surplus blocks leave at once.
__device__ __forceinline__ int64_t kv_first_slot(const KvAppendArgs& a, int b) {
  return static_cast<int64_t>(a.offsets[b]) / a.page + 2 * static_cast<int64_t>(b);
}

// D: head dimension; ITERS: 16-byte pieces of a page's new rows per thread.
template <int D, int ITERS, bool F16>
__global__ void __launch_bounds__(kKvAppendThreads) kv_append_kernel(const KvAppendArgs a) {
  constexpr int kRowThreads = D / 8;                          // threads per row
  constexpr int kRowsPerIter = kKvAppendThreads / kRowThreads;
  __shared__ float warp_max[kKvAppendThreads / 32];
  pdl_wait();
  const int tid = threadIdx.x;
  const int64_t slot = blockIdx.x;
  int found = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kKvAppendThreads) {
    const bool before = b0 + tid < a.batch && kv_first_slot(a, b0 + tid) <= slot;
    const int n = __syncthreads_count(before);
    found += n;
    if (n < kKvAppendThreads) break;  // first slots increase with b
  }
  const int b = found - 1;
  if (b < 0) return;
  const int kv = blockIdx.y & 1, head = blockIdx.y >> 1;
  const int64_t t0 = a.offsets[b], n = a.offsets[b + 1] - t0, len = a.lens[b], start = len - n;
  if (n <= 0) return;
  const int64_t nth = slot - kv_first_slot(a, b);  // page of the new tokens; negative only under falling offsets
  const int64_t pg = start / a.page + nth;
  if (nth < 0 || t0 < 0 || t0 + n > a.total || start < 0 || len > static_cast<int64_t>(a.table_width) * a.page) {
    if (tid == 0) record_error_at(a.err, kErrValue);
    return;
  }
  if (pg > (len - 1) / a.page) return;
  const int64_t pid = a.table[b * a.table_ld + pg];
  if (pid < 0 || pid >= a.num_pages) {
    if (tid == 0) record_error_at(a.err, kErrValue);
    return;
  }
  const int64_t base = pg * a.page;
  const int lo = static_cast<int>(max(start, base) - base), hi = static_cast<int>(min(len, base + a.page) - base);
  const int row0 = tid / kRowThreads, col = tid % kRowThreads * 8;
  const int64_t src_tok = a.src_tok[kv];
  const uint16_t* src = a.src[kv] + (t0 + base - start) * src_tok + head * a.src_head[kv] + col;

  uint4 v[ITERS];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int r = lo + row0 + i * kRowsPerIter;
    v[i] = r < hi ? ld_global_nc_v4(src + r * src_tok) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < ITERS; ++i)
    m = elem_absmax2<F16>(elem_absmax2<F16>(elem_absmax2<F16>(elem_absmax2<F16>(m, v[i].x), v[i].y), v[i].z), v[i].w);
  // magnitudes order like their bit patterns
  const uint32_t wm = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(elem_absmax_final<F16>(m)));
  if ((tid & 31) == 0) warp_max[tid >> 5] = __uint_as_float(wm);
  __syncthreads();
  const float amax = fmaxf(fmaxf(warp_max[0], warp_max[1]), fmaxf(warp_max[2], warp_max[3]));
  // mx_scale's comparison of significands is exact for FP16's 11 bits too:
  // no quotient of such a value by 448 rounds to a power of two that it is not
  int e = max(static_cast<int>(mx_scale<448>(amax).byte) - 127, kKvMinExp);
  uint8_t* scale = a.scales[kv] + pid * a.kv_heads + head;
  uint8_t* codes = a.cache[kv] + pid * a.cs_page + head * a.cs_head + col;
  if (lo > 0) {
    const int e_old = static_cast<int>(*scale) - 127;
    if (e > e_old) {
      const float f = pow2f(max(e_old - e, -126));  // 2^-126 already takes every code to zero
      for (int r = row0; r < lo; r += kRowsPerIter) {
        uint2* p = reinterpret_cast<uint2*>(codes + r * a.cs_tok);
        uint2 w = *p;
        uint32_t* h = &w.x;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const float2 x = f16x2_to_f32x2(e4m3x2_to_f16x2(h[q] & 0xFFFFu)), y = f16x2_to_f32x2(e4m3x2_to_f16x2(h[q] >> 16));
          h[q] = f32x2_to_e4m3x2(x.x * f, x.y * f) | (f32x2_to_e4m3x2(y.x * f, y.y * f) << 16);
        }
        *p = w;
      }
    }
    e = max(e, e_old);
    __syncthreads();  // every thread has read the old scale
  }
  const float f = pow2f(-e);
#pragma unroll
  for (int i = 0; i < ITERS; ++i) {
    const int r = lo + row0 + i * kRowsPerIter;
    if (r < hi) {
      const float2 x = elem2_to_f32x2<F16>(v[i].x), y = elem2_to_f32x2<F16>(v[i].y);
      const float2 z = elem2_to_f32x2<F16>(v[i].z), w = elem2_to_f32x2<F16>(v[i].w);
      *reinterpret_cast<uint2*>(codes + r * a.cs_tok) =
          make_uint2(f32x2_to_e4m3x2(x.x * f, x.y * f) | (f32x2_to_e4m3x2(y.x * f, y.y * f) << 16),
                     f32x2_to_e4m3x2(z.x * f, z.y * f) | (f32x2_to_e4m3x2(w.x * f, w.y * f) << 16));
    }
  }
  if (tid == 0) *scale = static_cast<uint8_t>(e + 127);
}

}  // namespace bsq
