// A mixture-of-experts layer for a few tokens (at most 64) over packed
// weights, in one kernel:
//   ids, p = top-k of softmax(logits);  xq = Q(x, x_sf[e]);
//   g, u = W13[e] xq;  h = bf16(silu(g) u);  hq = Q(h, h_sf[e]);
//   y = sum over the choices of p W2[e] hq.
//
// What bounds it: every chosen expert's weights are read once, 3 I H values
// per expert for a handful of operations per byte, so the kernel is a stream
// of weights from DRAM, and everything else has to hide behind it.
//
// Form.  The weights' codes and 5D scales are exactly what the block-scaled
// tensor-core product takes, so nothing is decoded: with the weights as the
// 128-row operand and an expert's tokens as the narrow one (N = 16..64), a stage
// of 2 x 128 rows x 128 bytes costs its loads and 8 products.  One persistent block per
// SM; blocks wait for one another, so the launch is cooperative.
//  * Every block routes all tokens itself (a warp per token), which saves a
//    grid-wide wait before the first weight can be requested.
//  * A phase's work is cut into units of one stage, numbered expert by
//    expert, tile by tile along K, and every block takes an equal run of them
//    whatever the tiles are.  A tile (pair of 128-row halves: gate and up rows, or
//    256 rows of W2) that several blocks share is finished by the block that began it, which
//    adds the others' parts in block order (no atomics on values: the result does not
//    depend on timing).
//  * warp 0 streams weights through a ring of shared-memory stages.  They do
//    not depend on the activations, so at the start (while the tokens
//    are quantized) and between the two phases (while h is finished) the ring
//    fills ahead; warp 2 adds the tokens' operand to each stage once it is there.
//  * warp 1 copies the stage's scales to tensor memory and issues the products;
//    warps 4-7 drain finished accumulators: silu, the quantization of h along a
//    warp's 32 rows, or the weighted rows of y.
//  * After a last grid-wide wait every block sums its share of y over the choices, in their order.
// Measured (graphs of calls; hidden 7168, inter 2048, NVFP4, top 8 of 256 experts): 64 tokens that reach 156 experts
// 649 us, 6.0 TB/s or 88 % of a plain copy; one token 51 us (3.9 TB/s: 27 us stream the first product's weights
// and x, the rest is the wait for h, the second product's ramp, the last wait and y).  16 tokens, hidden 4096, MXFP8,
// 34 of 64 experts: 152 us, 5.8 TB/s.  7 tokens, 17 experts of 3 MB each: 30 us, most of it those waits.
// All waits are bounded (about a second): an expired one records
// BSQ_ERR_TIMEOUT, stops the block's roles, waits for the copies and products in
// flight, frees the tensor memory and returns.
#pragma once

#include "tcgen05.cuh"

namespace bsq {

constexpr int kMoeMaxTokens = 64, kMoeMaxTopK = 16, kMoeMaxExperts = 1024;
constexpr int kMoeThreads = 384;          // weights, products, tokens, (idle), 4 epilogue and 4 helper warps
constexpr int kMoeQuantThreads = 256;      // warps 4-11 quantize the tokens and sum y
constexpr int kMoeHalfBytes = 128 * 128;  // a stage's 128 rows x 128 bytes of one tile half
constexpr int kMoeMaxBlocks = 160;  // one per SM
// counters at the start of the workspace, zero between calls
// (kMoeSpoiled: not 0 once a call has given up in a wait; what else the workspace holds is then not to be trusted)
constexpr int kMoeBarQuant = 0, kMoeBarDone = 32, kMoeBarExit = 64, kMoeSpoiled = 80, kMoePartReady = 96,
              kMoeExpertDone = kMoePartReady + 2 * kMoeMaxBlocks;
constexpr int kMoeCounterBytes = 4 * (kMoeExpertDone + 1024);

// Columns of a stage and its scale atoms per 128 rows.
template <int FMT> struct MoeFmt {
  static constexpr int kElems = FMT == kMXFP8 ? 128 : 256;
  static constexpr int kAtoms = kElems / Fmt<FMT>::ATOM_COLS;
};

struct MoeArgs {
  const uint16_t* x;
  int64_t ld_x;
  const float* logits;
  int64_t ld_logits;
  const int32_t* ids;    // a finished routing in place of the logits: (tokens, top_k)
  const float* weights;
  const uint8_t *w13_s, *w2_s;
  const float *x_sf, *w13_sf, *h_sf, *w2_sf;  // NVFP4
  uint16_t* y;
  int64_t ld_y;
  int tokens, hidden, inter, experts, top_k, renorm;
  uint32_t* counters;
  uint8_t *xq, *xq_s, *hq, *hq_s;  // tokens' operands by row (expert by expert), scales by active expert
  float* part;                     // [block][phase][2 halves][max_n][128]
  float* yp;                       // [token * top_k + choice][hidden]
  int max_n;                       // tokens rounded up to 16
  int stages, stage_bytes;
  unsigned int* err;
};

// Shared memory before the stages: routing tables (16-byte aligned parts).
struct MoeTables {
  uint32_t* mask;    // [experts][2] tokens that chose the expert, a bit each
  int* active;       // [active] expert of active index
  int* row0;         // [active + 1] first row
  int* index_of;     // [experts] active index
  int* pair_of;      // [rows] token * top_k + choice
  int* id;           // [pairs] expert
  float* prob;       // [pairs]
};
__host__ __device__ inline int moe_align16(int n) { return (n + 15) & ~15; }
__host__ __device__ inline int moe_table_bytes(int experts, int pairs) {
  const int act = (experts < pairs ? experts : pairs) + 1;
  return moe_align16(8 * experts) + 2 * moe_align16(4 * act) + moe_align16(4 * experts) + 3 * moe_align16(4 * pairs);
}

// A phase's units, cut into `parts` runs of equal length, none empty: block b
// takes run b.  The host's size limits keep units below 2^31.
struct MoePhase {
  int units;
  int tiles;   // per expert
  int chunks;  // stages per tile
  int parts;
  int begin, end;  // this block's run
  __device__ __forceinline__ int start_of(int part) const {
    return static_cast<int>(static_cast<uint64_t>(units) * static_cast<uint32_t>(part) / static_cast<uint32_t>(parts));
  }
  // The block whose run holds unit u.
  __device__ __forceinline__ int owner(int u) const {
    return static_cast<int>((static_cast<uint64_t>(u + 1) * static_cast<uint32_t>(parts) - 1) / static_cast<uint32_t>(units));
  }
};

template <int FMT>
__device__ __forceinline__ MoePhase moe_phase(const MoeArgs& a, int phase, int active) {
  MoePhase p;
  const int cols = phase == 0 ? a.hidden : a.inter, block = blockIdx.x;
  p.tiles = phase == 0 ? a.inter / 128 : (a.hidden + 255) / 256;
  p.chunks = (cols + MoeFmt<FMT>::kElems - 1) / MoeFmt<FMT>::kElems;
  p.units = active * p.tiles * p.chunks;
  p.parts = min(p.units, static_cast<int>(gridDim.x));
  p.begin = block < p.parts ? p.start_of(block) : 0;
  p.end = block < p.parts ? p.start_of(block + 1) : 0;
  return p;
}

// Order-preserving key of a logit: larger logits have larger keys, NaN and -inf the least.
__device__ __forceinline__ uint32_t moe_key(float z) {
  const uint32_t u = __float_as_uint(z == z ? z + 0.0f : -INFINITY);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float moe_unkey(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? k & 0x7FFFFFFFu : ~k);
}

// Route token t with one warp, its logits in registers (expert 32 i + lane
// in key[i]): choices and weights into the tables.
template <int NL>
__device__ __forceinline__ void moe_route(const MoeArgs& a, const MoeTables& tb, int t, int lane) {
  const float* z = a.logits + t * a.ld_logits;
  uint32_t key[NL];
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int e = 32 * i + lane;
    const float v = e < a.experts ? __ldg(z + e) : 0.f;
    nan |= v != v;
    key[i] = e < a.experts ? moe_key(v) : 0u;  // 0: none (every key of a logit is larger)
  }
  uint32_t best = 0;
#pragma unroll
  for (int i = 0; i < NL; ++i) best = max(best, key[i]);
  uint32_t m = __reduce_max_sync(~0u, best);
  const float top = moe_unkey(m);
  if (__any_sync(~0u, nan) && lane == 0 && blockIdx.x == 0) record_error_at(a.err, kErrValue);
  float sum = 0.f;
  if (!a.renorm) {
#pragma unroll
    for (int i = 0; i < NL; ++i)
      if (key[i] != 0u) sum += expf(moe_unkey(key[i]) - top);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  }
  uint32_t mine = 0;  // key and expert of choice `lane`
  int my_id = 0;
  for (int k = 0; k < a.top_k; ++k) {
    int at = 0x7FFFFFFF;
#pragma unroll
    for (int i = NL - 1; i >= 0; --i)
      if (key[i] == m) at = 32 * i + lane;
    const int id = static_cast<int>(__reduce_min_sync(~0u, static_cast<uint32_t>(at)));  // equal ones: the lowest expert
    if (lane == k) {
      mine = m;
      my_id = id;
    }
    best = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      if (32 * i + lane == id) key[i] = 0u;
      best = max(best, key[i]);
    }
    m = __reduce_max_sync(~0u, best);
  }
  const float p = lane < a.top_k && top > -INFINITY ? expf(moe_unkey(mine) - top) : 0.f;
  if (a.renorm) {
    sum = p;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
  }
  if (lane < a.top_k) {
    tb.prob[t * a.top_k + lane] = top > -INFINITY ? p / sum : 0.f;
    tb.id[t * a.top_k + lane] = my_id;
    atomicOr(&tb.mask[2 * my_id + (t >> 5)], 1u << (t & 31));
  }
}

// The choices of token t from a finished routing, with one warp, a lane per choice.  One without an expert gets id -1 and
// has no row; an expert that comes again for a token takes the later weights too.
__device__ __forceinline__ void moe_take_route(const MoeArgs& a, const MoeTables& tb, int t, int lane) {
  const bool in = lane < a.top_k;
  int id = in ? __ldg(a.ids + t * a.top_k + lane) : -1;
  const float w = in ? __ldg(a.weights + t * a.top_k + lane) : 0.f;
  if (__any_sync(~0u, id >= a.experts) && lane == 0 && blockIdx.x == 0) record_error_at(a.err, kErrValue);
  if (id >= a.experts) id = -1;
  const uint32_t same = __match_any_sync(~0u, id >= 0 ? id : -1 - lane);
  float sum = 0.f;
  for (int k = 0; k < a.top_k; ++k) {
    const float wk = __shfl_sync(~0u, w, k);
    if (same >> k & 1u) sum += wk;
  }
  if (__ffs(same) - 1 != lane) id = -1;
  if (in) {
    tb.id[t * a.top_k + lane] = id < 0 ? -1 : id;
    tb.prob[t * a.top_k + lane] = sum;
    if (id >= 0) atomicOr(&tb.mask[2 * id + (t >> 5)], 1u << (t & 31));
  }
}

// Rank of token t among the tokens of an expert, and their number.
__device__ __forceinline__ int moe_rank(const MoeTables& tb, int e, int t) {
  const uint32_t lo = tb.mask[2 * e], hi = tb.mask[2 * e + 1], below = (1u << (t & 31)) - 1u;
  return t < 32 ? __popc(lo & below) : __popc(lo) + __popc(hi & below);
}
__device__ __forceinline__ int moe_count(const MoeTables& tb, int e) { return __popc(tb.mask[2 * e]) + __popc(tb.mask[2 * e + 1]); }

// Quantize 32 consecutive BF16 values (16 words): packed bytes and scale bytes.
template <int FMT>
__device__ __forceinline__ void moe_quant_block(const uint4 (&v)[4], float tsf, uint8_t* dst, uint8_t* scale_word) {
  if constexpr (FMT == kNVFP4) {
    uint32_t sb[2], q[4];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 2 * b; i < 2 * b + 2; ++i) m = absmax2(absmax2(absmax2(absmax2(m, v[i].x), v[i].y), v[i].z), v[i].w);
      sb[b] = f32_to_e4m3(__fmul_rn(__fdiv_rn(absmax_final(m), 6.0f), tsf));
      const float ds = e4m3_to_f32(sb[b]);
      const float f = ds == 0.0f ? 0.0f : __fdiv_rn(tsf, ds);
      q[2 * b] = quant8_e2m1(v[2 * b], f);
      q[2 * b + 1] = quant8_e2m1(v[2 * b + 1], f);
    }
    *reinterpret_cast<uint4*>(dst) = make_uint4(q[0], q[1], q[2], q[3]);
    *reinterpret_cast<uint16_t*>(scale_word) = static_cast<uint16_t>(sb[0] | (sb[1] << 8));
  } else {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = absmax2(absmax2(absmax2(absmax2(m, v[i].x), v[i].y), v[i].z), v[i].w);
    const MxScale s = mx_scale<FMT == kMXFP4 ? 6 : 448>(absmax_final(m));
    if constexpr (FMT == kMXFP4) {
      *reinterpret_cast<uint4*>(dst) = make_uint4(quant8_e2m1_pow2(v[0], s.pow2), quant8_e2m1_pow2(v[1], s.pow2),
                                                  quant8_e2m1_pow2(v[2], s.pow2), quant8_e2m1_pow2(v[3], s.pow2));
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint2 lo = quant8_e4m3_pow2(v[2 * h], s.pow2), hi = quant8_e4m3_pow2(v[2 * h + 1], s.pow2);
        *reinterpret_cast<uint4*>(dst + 16 * h) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
    *scale_word = static_cast<uint8_t>(s.byte);
  }
}

// Block `w` of 32 columns of the (token, choice) pairs' rows of x.
__device__ __forceinline__ void moe_load_x(const MoeArgs& a, int w, int total, int per_row, uint4 (&v)[4]) {
  if (w >= total) return;
  const int pair = w / per_row, c = w - pair * per_row;
  const uint16_t* src = a.x + (pair / a.top_k) * a.ld_x + 32 * c;
#pragma unroll
  for (int q = 0; q < 4; ++q) v[q] = ld_global_nc_v4(src + 8 * q);
}

// This thread's h (row i of a warp's 32, one token) quantized with its
// neighbours': blocks run along the lanes.  Every lane calls.
template <int FMT>
__device__ __forceinline__ void moe_quant_lane(float h, float tsf, int lane, uint8_t* row_bytes, uint8_t* scale_word) {
  const uint32_t mag = __float_as_uint(fabsf(h));
  if constexpr (FMT == kNVFP4) {
    uint32_t m = mag;
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = max(m, __shfl_xor_sync(~0u, m, d));
    const uint32_t sb = f32_to_e4m3(__fmul_rn(__fdiv_rn(__uint_as_float(m), 6.0f), tsf));
    const float ds = e4m3_to_f32(sb);
    const float v = __fmul_rn(h, ds == 0.0f ? 0.0f : __fdiv_rn(tsf, ds));
    const float next = __shfl_down_sync(~0u, v, 1);
    if ((lane & 1) == 0) row_bytes[lane >> 1] = f32x2_to_e2m1x2(v, next);
    if ((lane & 15) == 0) scale_word[lane >> 4] = static_cast<uint8_t>(sb);
  } else {
    const MxScale s = mx_scale<FMT == kMXFP4 ? 6 : 448>(__uint_as_float(__reduce_max_sync(~0u, mag)));
    const float v = __fmul_rn(h, __uint_as_float(static_cast<uint32_t>(s.pow2) << 16));
    if constexpr (FMT == kMXFP4) {
      const float next = __shfl_down_sync(~0u, v, 1);
      if ((lane & 1) == 0) row_bytes[lane >> 1] = f32x2_to_e2m1x2(v, next);
    } else {
      row_bytes[lane] = static_cast<uint8_t>(f32x2_to_e4m3x2(v, 0.f));
    }
    if (lane == 0) *scale_word = static_cast<uint8_t>(s.byte);
  }
}

// Rows g and u of one token and this thread's row of the tile: h, quantized
// with the warp's other rows.  Not inlined: one copy of it per format keeps
// the epilogue small in the instruction cache, which a short call starts cold.
template <int FMT>
__device__ __noinline__ void moe_finish_h(float g, float u, float hsf, int lane, uint8_t* row_bytes, uint8_t* scale_word) {
  // the fast exponential is off by about (2 + 1.2 |g|) 2^-23 of itself (2^-19.5 at g = -8, 2^-17 at -60), h is rounded to 2^-9
  const float h = __bfloat162float(__float2bfloat16_rn(__fdividef(g, 1.f + __expf(-g)) * u));
  moe_quant_lane<FMT>(h, hsf, lane, row_bytes, scale_word);
}

// One stage's products into accumulators d and d + 64 (the tile's halves) where
// the stage is not whole (t5_stage_scaled): `slices` products of 32 bytes of each row, `atoms`
// scale atoms, one half or two.  da, db, ds: descriptors of the stage's weights, tokens and scales.
template <int FMT>
__device__ __forceinline__ void moe_products(uint32_t d, uint64_t da, uint64_t db, uint64_t ds, uint32_t n, uint32_t sf,
                                             uint32_t fresh, int slices, int atoms, bool two, uint32_t lead) {
  constexpr int kAtoms = MoeFmt<FMT>::kAtoms;
#pragma unroll 1
  for (int q = 0; q < atoms; ++q) {
    t5_copy_atom(sf + 4 * q, ds + 32 * q, lead);
    if (two) t5_copy_atom(sf + 16 + 4 * q, ds + 32 * (kAtoms + q), lead);
    t5_copy_atom(sf + 32 + 4 * q, ds + 32 * (2 * kAtoms + q), lead);
  }
#pragma unroll 1
  for (int m = 0; m < slices; ++m) {
    constexpr uint32_t kPer = 4 / kAtoms;  // slices per atom
    const uint32_t atom = m / kPer, id = (m % kPer) * (4 / kPer), sfb = sf + 32 + 4 * atom;
    const uint32_t idesc = t5_idesc_scaled<FMT>(n, id);
    t5_mma_scaled<FMT>(d, da + 2 * m, db + 2 * m, idesc, sf + 4 * atom, sfb, fresh | m, lead);
    if (two) t5_mma_scaled<FMT>(d + 64, da + kMoeHalfBytes / 16 + 2 * m, db + 2 * m, idesc, sf + 16 + 4 * atom, sfb, fresh | m, lead);
  }
}

// Byte of the scale of an expert's token r, scale column s, in the tokens'
// scales: the 5D layout of one row tile.
__device__ __forceinline__ int moe_token_scale(int r, int s) { return (s >> 2) * 512 + (r & 31) * 16 + (r >> 5) * 4 + (s & 3); }

// Wait until a counter in global memory reaches `value`, for about a second.
__device__ __forceinline__ bool moe_wait_count(const uint32_t* p, uint32_t value, const volatile uint32_t* abort_flag,
                                               long long limit = kWaitLimitCycles) {
  if (ld_acquire(p) >= value) return true;
  const long long t0 = clock64();
  while (ld_acquire(p) < value)
    if (*abort_flag != 0u || clock64() - t0 > limit) return false;
  return true;
}

// ROUTED: the routing is given (moe_take_route), and may leave choices without an expert.
template <int FMT, bool ROUTED>
__global__ void __launch_bounds__(kMoeThreads, 1)
    moe_layer_kernel(const __grid_constant__ CUtensorMap map_w13, const __grid_constant__ CUtensorMap map_w2,
                     const __grid_constant__ CUtensorMap map_xq, const __grid_constant__ CUtensorMap map_hq, const MoeArgs a) {
  constexpr int kElems = MoeFmt<FMT>::kElems, kAtoms = MoeFmt<FMT>::kAtoms, kSF = Fmt<FMT>::SF;
  constexpr int kAtomElems = Fmt<FMT>::ATOM_COLS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t full_bar[8], empty_bar[8], acc_full[2], acc_empty[2], drain_bar;
  __shared__ uint32_t tmem_slot, last_flag, spoiled;
  __shared__ volatile uint32_t abort_flag, fills_a, fills_b, consumed;
  __shared__ int active_count;
  __shared__ uint32_t warp_sum[kMoeThreads / 32];

  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const int blocks = gridDim.x, block = blockIdx.x, pairs = a.tokens * a.top_k;
  const int stages = a.stages;

  MoeTables tb;
  {
    const int act = (a.experts < pairs ? a.experts : pairs) + 1;
    uint8_t* p = smem + stages * a.stage_bytes;
    tb.mask = reinterpret_cast<uint32_t*>(p);
    p += moe_align16(8 * a.experts);
    tb.active = reinterpret_cast<int*>(p);
    p += moe_align16(4 * act);
    tb.row0 = reinterpret_cast<int*>(p);
    p += moe_align16(4 * act);
    tb.index_of = reinterpret_cast<int*>(p);
    p += moe_align16(4 * a.experts);
    tb.pair_of = reinterpret_cast<int*>(p);
    p += moe_align16(4 * pairs);
    tb.id = reinterpret_cast<int*>(p);
    p += moe_align16(4 * pairs);
    tb.prob = reinterpret_cast<float*>(p);
  }
  if (tid == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full_bar[s], 2);  // weights, tokens
      mbar_init(&empty_bar[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 1);
    }
    mbar_init(&drain_bar, 1);
    abort_flag = 0u;
    fills_a = fills_b = consumed = 0u;
    fence_mbar_init();
    prefetch_tensormap(&map_w13);
    prefetch_tensormap(&map_w2);
    prefetch_tensormap(&map_xq);
    prefetch_tensormap(&map_hq);
  }
  if (warp == 1) t5_alloc(&tmem_slot, 512);
  for (int e = tid; e < 2 * a.experts; e += kMoeThreads) tb.mask[e] = 0u;
  __syncthreads();
  // the first block of x that this thread will quantize is on its way while the tokens are routed
  const int per_row = a.hidden / 32, quant_total = pairs * per_row, quant_step = blocks * kMoeQuantThreads;
  int quant_at = block + blocks * (tid - 128);
  uint4 xv[4];
  if (warp >= 4) moe_load_x(a, quant_at, quant_total, per_row, xv);
  // as many logits a lane as the experts need, in two sizes (256 experts: 649 / 668 us for 64 tokens and 51 / 52
  // for one with the smaller / larger form)
  const uint32_t spoiled_word = tid == 0 ? __ldcg(a.counters + kMoeSpoiled) : 0u;
  if constexpr (ROUTED) {
    for (int t = warp; t < a.tokens; t += kMoeThreads / 32) moe_take_route(a, tb, t, lane);
  } else if (a.experts <= 256) {
    for (int t = warp; t < a.tokens; t += kMoeThreads / 32) moe_route<8>(a, tb, t, lane);
  } else {
    for (int t = warp; t < a.tokens; t += kMoeThreads / 32) moe_route<32>(a, tb, t, lane);
  }
  if (tid == 0) spoiled = spoiled_word;
  __syncthreads();
  if (spoiled != 0u) {  // the whole block, before anything is in flight
    if (tid == 0) record_error_at(a.err, kErrTimeout);
    if (warp == 1) t5_dealloc(tmem_slot, 512);
    return;
  }
  // active experts in increasing order and their first rows: a thread per expert, (rows << 16 | 1) summed
  {
    uint32_t base = 0;
    for (int e0 = 0; e0 < a.experts; e0 += kMoeThreads) {
      const int e = e0 + tid;
      const int c = e < a.experts ? moe_count(tb, e) : 0;
      const uint32_t v = c > 0 ? static_cast<uint32_t>(c) << 16 | 1u : 0u;
      uint32_t sum = v;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(~0u, sum, d);
        if (lane >= d) sum += o;
      }
      if (lane == 31) warp_sum[warp] = sum;
      __syncthreads();
      uint32_t before = base, all = base;
#pragma unroll
      for (int w = 0; w < kMoeThreads / 32; ++w) {
        if (w < warp) before += warp_sum[w];
        all += warp_sum[w];
      }
      before += sum - v;
      if (c > 0) {
        const int i = before & 0xFFFF;
        tb.active[i] = e;
        tb.row0[i] = before >> 16;
        tb.index_of[e] = i;
      }
      base = all;
      __syncthreads();
    }
    if (tid == 0) {
      active_count = base & 0xFFFF;
      tb.row0[base & 0xFFFF] = base >> 16;
    }
  }
  t5_fence_before();
  __syncthreads();
  t5_fence_after();
  for (int p = tid; p < pairs; p += kMoeThreads) {  // rows of an expert in token order
    const int t = p / a.top_k, e = tb.id[p];
    if (ROUTED && e < 0) continue;
    tb.pair_of[tb.row0[tb.index_of[e]] + moe_rank(tb, e, t)] = p;
  }
  __syncthreads();
  const uint32_t tmem = warp_uniform(static_cast<int>(tmem_slot)), smem_base = smem_addr(smem);
  const int active = warp_uniform(active_count);
  const int part_floats = 2 * a.max_n * 128;

  if (warp == 0) {
    // ---- weights
    if (lane == 0) {
      uint32_t stage = 0, phase_bit = 0, fills = 0;
      for (int phase = 0; phase < 2 && abort_flag == 0u; ++phase) {
        const MoePhase p = moe_phase<FMT>(a, phase, active);
        const int cols = phase == 0 ? a.hidden : a.inter, rows = phase == 0 ? 2 * a.inter : a.hidden;
        const int kt = (cols / kSF + 3) / 4;
        const int64_t scale_bytes = static_cast<int64_t>((rows + 127) / 128) * kt * 512;
        const uint8_t* scales = phase == 0 ? a.w13_s : a.w2_s;
        const CUtensorMap* map = phase == 0 ? &map_w13 : &map_w2;
        for (int u = p.begin; u < p.end && abort_flag == 0u;) {
          const int item = u / p.chunks, stop = min(p.end, (item + 1) * p.chunks);
          const int expert = tb.active[item / p.tiles], tile = item % p.tiles;
          const int r0 = phase == 0 ? 128 * tile : 256 * tile, r1 = phase == 0 ? a.inter + r0 : r0 + 128;
          const bool two = r1 < rows;
          const int y = expert * rows;
          const uint8_t* s0 = scales + expert * scale_bytes + static_cast<int64_t>(r0 / 128) * kt * 512;
          const uint8_t* s1 = scales + expert * scale_bytes + static_cast<int64_t>(r1 / 128) * kt * 512;
          for (int kc = u - item * p.chunks; u < stop; ++u, ++kc) {
            const int atoms = min(kAtoms, kt - kc * kAtoms);
            if (!mbar_wait_clocked(&empty_bar[stage], phase_bit ^ 1u, &abort_flag)) {
              if (abort_flag == 0u) record_error_at(a.err, kErrTimeout);
              abort_flag = 1u;
            }
            if (abort_flag != 0u) break;
            uint8_t* st = smem + stage * a.stage_bytes;
            uint8_t* sc = st + 2 * kMoeHalfBytes + a.max_n * 128;
            uint64_t* bar = &full_bar[stage];
            mbar_arrive_expect_tx(bar, (two ? 2 : 1) * (kMoeHalfBytes + atoms * 512));
            tma_load_2d(st, map, kc * 128, y + r0, bar);
            bulk_load(sc, s0 + kc * kAtoms * 512, atoms * 512, bar);
            if (two) {
              tma_load_2d(st + kMoeHalfBytes, map, kc * 128, y + r1, bar);
              bulk_load(sc + kAtoms * 512, s1 + kc * kAtoms * 512, atoms * 512, bar);
            }
            fills_a = ++fills;
            if (++stage == stages) { stage = 0; phase_bit ^= 1u; }
          }
        }
      }
    }
  } else if (warp == 2) {
    // ---- tokens
    if (lane == 0) {
      uint32_t stage = 0, phase_bit = 0, fills = 0;
      bool ok = true;
      for (int phase = 0; phase < 2 && ok; ++phase) {
        const MoePhase p = moe_phase<FMT>(a, phase, active);
        const int cols = phase == 0 ? a.hidden : a.inter, kt = (cols / kSF + 3) / 4;
        const CUtensorMap* map = phase == 0 ? &map_xq : &map_hq;
        const uint8_t* scales = phase == 0 ? a.xq_s : a.hq_s;
        int ready = -1;
        if (phase == 0 && p.begin < p.end) {
          ok = moe_wait_count(a.counters + kMoeBarQuant, blocks, &abort_flag);
          fence_async();
        }
        for (int u = p.begin; u < p.end && ok;) {
          const int item = u / p.chunks, stop = min(p.end, (item + 1) * p.chunks), i = item / p.tiles;
          if (phase == 1 && ready != i) {  // every tile of this expert's h is there
            ok = moe_wait_count(a.counters + kMoeExpertDone + i, a.inter / 128, &abort_flag);
            fence_async();
            ready = i;
          }
          const int row = tb.row0[i], n8 = (tb.row0[i + 1] - row + 7) >> 3;
          const uint8_t* s0 = scales + static_cast<int64_t>(i) * kt * 512;
          for (int kc = u - item * p.chunks; u < stop && ok; ++u, ++kc) {
            ok = mbar_wait_clocked(&empty_bar[stage], phase_bit ^ 1u, &abort_flag) && abort_flag == 0u;
            if (!ok) break;
            const int atoms = min(kAtoms, kt - kc * kAtoms);
            uint8_t* st = smem + stage * a.stage_bytes + 2 * kMoeHalfBytes;
            uint64_t* bar = &full_bar[stage];
            mbar_arrive_expect_tx(bar, n8 * 1024 + atoms * 512);
            for (int b = 0; b < n8; ++b) tma_load_2d(st + b * 1024, map, kc * 128, row + 8 * b, bar);
            bulk_load(st + a.max_n * 128 + 2 * kAtoms * 512, s0 + kc * kAtoms * 512, atoms * 512, bar);
            fills_b = ++fills;
            if (++stage == stages) { stage = 0; phase_bit ^= 1u; }
          }
        }
      }
      if (!ok) {
        if (abort_flag == 0u) record_error_at(a.err, kErrTimeout);
        abort_flag = 1u;
      }
    }
  } else if (warp == 1) {
    // ---- products: the whole warp in step, one lane issuing
    const uint32_t lead = t5_elect();
    uint32_t stage = 0, phase_bit = 0, done = 0, seg = 0;
    bool ok = true;
    for (int phase = 0; phase < 2 && ok; ++phase) {
      const MoePhase p = moe_phase<FMT>(a, phase, active);
      const int cols = phase == 0 ? a.hidden : a.inter, rows = phase == 0 ? 2 * a.inter : a.hidden;
      for (int u = p.begin; u < p.end && ok; ++seg) {
        const int item = u / p.chunks, stop = min(p.end, (item + 1) * p.chunks);
        const int i = item / p.tiles, tile = item % p.tiles;
        const bool two = phase == 0 || 256 * tile + 128 < rows;
        const uint32_t n = warp_uniform((tb.row0[i + 1] - tb.row0[i] + 15) & ~15);
        const uint32_t buf = seg & 1u, d = tmem + buf * 128u;
        ok = __all_sync(~0u, mbar_wait_clocked(&acc_empty[buf], ((seg >> 1) & 1u) ^ 1u, &abort_flag));
        if (!ok) break;
        t5_fence_after();
        int kc = u - item * p.chunks;
        for (uint32_t fresh = 0; u < stop; ++u, ++kc) {
          ok = __all_sync(~0u, mbar_wait_clocked(&full_bar[stage], phase_bit, &abort_flag));
          if (!ok) break;
          t5_fence_after();
          const uint32_t st = smem_base + stage * a.stage_bytes;
          const uint32_t tok = st + 2 * kMoeHalfBytes, sc = tok + a.max_n * 128;
          const uint32_t sf = tmem + 256u + (done & 1u) * 64u;
          const uint64_t da = t5_desc_sw128(st), db = t5_desc_sw128(tok), ds = t5_desc_atom(sc);
          const int left = cols - kc * kElems;
          if (left >= kElems && two)
            t5_stage_scaled<FMT>(d, da, db, ds, t5_idesc_scaled<FMT>(n, 0), sf, fresh, lead);
          else
            moe_products<FMT>(d, da, db, ds, n, sf, fresh, min(4, (left + kElems / 4 - 1) / (kElems / 4)),
                                     min(kAtoms, (left + kAtomElems - 1) / kAtomElems), two, lead);
          fresh = 1;
          t5_commit(smem_addr(&empty_bar[stage]), lead);
          ++done;
          if (lane == 0) consumed = done;
          if (++stage == stages) { stage = 0; phase_bit ^= 1u; }
        }
        if (ok) t5_commit(smem_addr(&acc_full[buf]), lead);
      }
    }
    if (!ok && lane == 0) {
      if (abort_flag == 0u) record_error_at(a.err, kErrTimeout);
      abort_flag = 1u;
    }
    t5_commit(smem_addr(&drain_bar), lead);
    if (!mbar_wait_clocked(&drain_bar, 0) && lane == 0) record_error_at(a.err, kErrTimeout);
  } else if (warp >= 4) {
    // ---- quantize the tokens' rows, a block of 32 columns per thread at a time
    const int et = tid - 128, quarter = warp & 3;
    {
      const int kt = (a.hidden / kSF + 3) / 4, row_bytes = FMT == kMXFP8 ? a.hidden : a.hidden / 2;
      while (quant_at < quant_total) {
        uint4 next[4];
        moe_load_x(a, quant_at + quant_step, quant_total, per_row, next);
        const int pair = quant_at / per_row, c = quant_at - pair * per_row, t = pair / a.top_k;
        const int e = tb.id[pair];
        if (!ROUTED || e >= 0) {
          const int i = tb.index_of[e], r = moe_rank(tb, e, t);
          const int s0 = 32 * c / kSF;  // first scale column
          uint8_t* sc = a.xq_s + static_cast<int64_t>(i) * kt * 512;
          uint8_t* word = sc + moe_token_scale(r, s0);
          moe_quant_block<FMT>(xv, FMT == kNVFP4 ? __ldg(a.x_sf + e) : 1.f,
                               a.xq + static_cast<int64_t>(tb.row0[i] + r) * row_bytes + (FMT == kMXFP8 ? 32 * c : 16 * c), word);
          if (c == per_row - 1)  // the last atom's columns past the row: zero
            for (int s = s0 + 32 / kSF; s < 4 * kt; ++s) sc[moe_token_scale(r, s)] = 0;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) xv[q] = next[q];
        quant_at += quant_step;
      }
      named_sync(2, kMoeQuantThreads);
      if (et == 0) atomic_add_acq_rel(a.counters + kMoeBarQuant, 1u);
    }
    bool ok = true;
    if (warp < 8) {
    // ---- finished accumulators
    uint32_t seg = 0;
    for (int phase = 0; phase < 2 && ok; ++phase) {
      const MoePhase p = moe_phase<FMT>(a, phase, active);
      for (int u = p.begin; u < p.end; ++seg) {
        const int item = u / p.chunks, first = item * p.chunks, stop = min(p.end, first + p.chunks);
        const int i = item / p.tiles, tile = item % p.tiles, expert = tb.active[i];
        const int row0 = tb.row0[i], n = tb.row0[i + 1] - row0;
        const bool whole = u == first && stop == first + p.chunks;
        const uint32_t buf = seg & 1u;
        float by = 1.f, hsf = 1.f;
        if constexpr (FMT == kNVFP4) {
          hsf = __ldg(a.h_sf + expert);
          by = phase == 0 ? 1.f / (__ldg(a.x_sf + expert) * __ldg(a.w13_sf + expert)) : 1.f / (hsf * __ldg(a.w2_sf + expert));
        }
        // The block that began a tile finishes it: it gets there at the end
        // of its run, when the blocks that began theirs inside the tile have
        // long stored their parts.  Parts are added in block order.
        const int more = u == first && !whole ? p.owner(first + p.chunks - 1) - block : 0;  // blocks after this one in the tile
        if (et == 0) {
          bool go = true;
          for (int o = block + 1; o <= block + more && go; ++o) {
            uint32_t* flag = a.counters + kMoePartReady + 2 * o + phase;
            go = moe_wait_count(flag, 1u, &abort_flag);
            *flag = 0u;
          }
          go = go && mbar_wait_clocked(&acc_full[buf], (seg >> 1) & 1u, &abort_flag) && abort_flag == 0u;
          last_flag = go ? 1u : 0u;
        }
        named_sync(1, 128);
        ok = last_flag != 0u;
        if (!ok) break;  // uniform
        t5_fence_after();
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16) + buf * 128u;
        const int r = 32 * quarter + lane;
        if (u != first) {
          float* mine = a.part + (static_cast<int64_t>(block) * 2 + phase) * part_floats;
          for (int c = 0; c < n; c += 8) {
            float x[8], z[8];
            t5_ld8_pair(lanes + c, lanes + 64 + c, x, z);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (c + j < n) {
                __stcg(mine + (c + j) * 128 + r, x[j]);
                __stcg(mine + (a.max_n + c + j) * 128 + r, z[j]);
              }
          }
          t5_fence_before();
          named_sync(1, 128);
          if (et == 0) {
            mbar_arrive(&acc_empty[buf]);
            st_release(a.counters + kMoePartReady + 2 * block + phase, 1u);
          }
        } else {
          for (int c = 0; c < n; c += 8) {
            float x[8], z[8];
            t5_ld8_pair(lanes + c, lanes + 64 + c, x, z);
            for (int o = block + 1; o <= block + more; ++o) {
              const float* part = a.part + (static_cast<int64_t>(o) * 2 + phase) * part_floats;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (c + j < n) {
                  x[j] += __ldcg(part + (c + j) * 128 + r);
                  z[j] += __ldcg(part + (a.max_n + c + j) * 128 + r);
                }
            }
            if (phase == 0) {
              const int i0 = 128 * tile + 32 * quarter;  // first of this warp's rows
              const int kt = a.inter / kAtomElems, s0 = i0 / kSF;
              const int64_t row_bytes = FMT == kMXFP8 ? a.inter : a.inter / 2;
              uint8_t* sc = a.hq_s + static_cast<int64_t>(i) * kt * 512;
              uint8_t* dst = a.hq + row0 * row_bytes + (FMT == kMXFP8 ? i0 : i0 / 2);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const int tok = c + j;
                if (tok >= n) break;  // uniform
                moe_finish_h<FMT>(x[j] * by, z[j] * by, hsf, lane, dst + tok * row_bytes, sc + moe_token_scale(tok, s0));
              }
            } else {
              const int col = 256 * tile + r;
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                if (c + j >= n) break;
                const int pair = tb.pair_of[row0 + c + j];
                const float p = tb.prob[pair], f = p * by;  // p = 0: excluded, whatever its product is
                float* dst = a.yp + static_cast<int64_t>(pair) * a.hidden + col;
                if (col < a.hidden) __stcg(dst, p == 0.f ? 0.f : x[j] * f);
                if (col + 128 < a.hidden) __stcg(dst + 128, p == 0.f ? 0.f : z[j] * f);
              }
            }
          }
          t5_fence_before();
          named_sync(1, 128);
          if (et == 0) {
            mbar_arrive(&acc_empty[buf]);
            if (phase == 0) atomic_add_acq_rel(a.counters + kMoeExpertDone + i, 1u);
          }
        }
        u = stop;
      }
    }
    }
    // ---- y, once every block is done
    named_sync(2, kMoeQuantThreads);
    if (et == 0) {
      bool all = ok && abort_flag == 0u;
      if (all) {
        atomic_add_acq_rel(a.counters + kMoeBarDone, 1u);
        all = moe_wait_count(a.counters + kMoeBarDone, blocks, &abort_flag);
      }
      if (!all) {
        if (abort_flag == 0u) record_error_at(a.err, kErrTimeout);
        abort_flag = 1u;
      }
      last_flag = all ? 1u : 0u;
    }
    named_sync(2, kMoeQuantThreads);
    if (last_flag != 0u) {
      const int quads = a.hidden / 4;
      for (int w = block * kMoeQuantThreads + et; w < a.tokens * quads; w += blocks * kMoeQuantThreads) {
        const int t = w / quads, c = (w - t * quads) * 4;
        const float* src = a.yp + static_cast<int64_t>(t) * a.top_k * a.hidden + c;
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = 0; k0 < a.top_k; k0 += 8) {  // eight choices' loads in flight, added in their order
          float4 v[8];
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k0 + k < a.top_k) {
              if (ROUTED && tb.id[t * a.top_k + k0 + k] < 0)
                v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
              else
                v[k] = __ldcg(reinterpret_cast<const float4*>(src + static_cast<int64_t>(k0 + k) * a.hidden));
            }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (k0 + k < a.top_k) {
              s.x += v[k].x; s.y += v[k].y; s.z += v[k].z; s.w += v[k].w;
            }
        }
        *reinterpret_cast<uint2*>(a.y + t * a.ld_y + c) = make_uint2(f32x2_to_elem2<false>(s.x, s.y), f32x2_to_elem2<false>(s.z, s.w));
      }
      // every block has passed every other wait: clear the counters
      for (int i = block * kMoeQuantThreads + et; i < active; i += blocks * kMoeQuantThreads) a.counters[kMoeExpertDone + i] = 0u;
      if (et == 0) {
        if (atomic_add_acq_rel(a.counters + kMoeBarExit, 1u) == static_cast<uint32_t>(blocks) - 1u) {
          a.counters[kMoeBarQuant] = 0u;
          a.counters[kMoeBarDone] = 0u;
          a.counters[kMoeBarExit] = 0u;
        }
      }
    }
  }

  __syncthreads();
  // after an expired wait: loads that nothing consumed land before the block ends
  if (tid == 0 && abort_flag != 0u) a.counters[kMoeSpoiled] = 1u;
  if (tid == 0) {
    const uint32_t most = max(fills_a, fills_b);
    for (uint32_t f = consumed; f < most; ++f) {
      uint64_t* bar = &full_bar[f % stages];
      if (f >= fills_a) mbar_arrive(bar);
      if (f >= fills_b) mbar_arrive(bar);
      if (!mbar_wait_clocked(bar, (f / stages) & 1u)) record_error_at(a.err, kErrTimeout);
    }
  }
  t5_fence_before();
  __syncthreads();
  t5_fence_after();
  if (warp == 1) {
    __syncwarp();
    t5_dealloc(tmem, 512);
  }
}

}  // namespace bsq
