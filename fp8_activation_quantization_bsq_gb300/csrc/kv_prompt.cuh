// Attention over the 8-bit paged cache, for many query rows per kv head
// (prompts and chunks of them).  The mathematics, the folding of the page
// scales and the equal runs are those of kv_attention.cuh; here the rows fill
// 128-row products of the tcgen05 tensor cores.
//
// A unit is 128 keys of a tile of 256 rows (query tokens x heads of a kv head), as two halves of
// 128 rows.  Per half and 64 keys: S = Q K^T into tensor memory, the softmax weights P
// (FP16) over S in place, O += P V with P as the tensor-memory operand.  A half's two S tiles take
// turns, so that the next 64 keys' scores are there when its softmax comes to them; with two halves the
// tensor cores have products of the other while either softmax runs.  (512 columns: 4 x 64 of S, 2 x 128 of O.)
// What bounds it: 4 x 256 x 128 x D operations a unit, 2048 cycles of the tensor cores at D = 128; and
// shared memory, 3072 cycles at 128 bytes each: a 128 x 64 x 16 product reads 6 KB in its 32 cycles (1536 a unit), the
// values 512, the conversions below and the codes' arrival 1024.  Measured: a 2048-token chunk over 16384, 32 heads of 128
// over 8: 497 us, 1.04 PFLOP/s or 53 % of a library product's rate, 4600 cycles a unit; P then waits for the issuing warp, which the
// products hold up.  (Scores 128 wide would read a third less, but leave no room for a second S tile: 560 us where this form took 515.
// A second issuing warp: 529 against 511.  Products on a scheduler without a converter, its work spread over the
// other three: 484 us against 485.)
//  * warps 0-3 and 4-7: the halves' softmax, a thread per row, 64 scores in registers.
//    O is rescaled only where a row's maximum grew past 2^kKvLag of its reference.  They also bring the
//    query rows (a power of two per row, so that they are exact in FP16) and write the output.
//  * warps 8-11: E4M3 tiles to FP16 in the 128-byte-swizzled layout that both
//    products read (K as rows of the dimension, V as rows of keys, the same bytes); keys outside the
//    item's range become zeros.
//  * warp 12: TMA of the codes, page by page; warp 13: the products.
#pragma once

#include "kv_attention.cuh"

namespace bsq {

constexpr int kKpKeys = 128, kKpRows = 256, kKpThreads = 448;
constexpr int kKpSub = 64;              // keys of an S tile
constexpr int kKpRaw = 4, kKpWide = 3;  // rings of E4M3 and FP16 tiles: K, V, K, V, ...
constexpr int kKpSlots = 8;             // units whose page scales are kept
constexpr int kKpMaxBlocks = 160;

template <int D>
struct KpShape {
  static constexpr int kRawBytes = kKpKeys * D, kWideBytes = 2 * kRawBytes;
  static constexpr int kHalfBytes = 128 * D * 2;  // query rows of a half
  static constexpr int kSmem = 1024 + 2 * kHalfBytes + kKpWide * kWideBytes + kKpRaw * kRawBytes;
  static constexpr int kPartFloats = kKpRows * D + 4 * kKpRows;  // [d][row], m, sums below, z; the block's own: z of the rows at work
};

// Page scales of a unit (up to 8 pages of 16 tokens).
struct KpSlot {
  KvPageScale sc[8];
  uint32_t special;  // 1: some page is missing, 2: some |ev| is above kKvTameExp
};

// A half's softmax state of one row.
struct KpRow {
  float m, l, fac;
  int pos;
  bool live;
};

// Scores of 16 keys, scaled and masked: x = s f + ev, -inf where the row does not see the key.
template <bool EDGE>
__device__ __forceinline__ float kp_score(const KvAttnArgs& a, const KpRow& row, float s, float f, const KvPageScale& ps, int key,
                                          int lo, int hi) {
  const float x = fmaf(s, f, ps.ev);
  if constexpr (!EDGE) return x;
  const bool see = ps.inv != 0.f && key >= lo && key < hi && (!a.causal || key <= row.pos) && (a.window <= 0 || key > row.pos - a.window);
  return see ? x : -INFINITY;
}

// The row's scores of kKpSub keys into registers, scaled and with the values'
// exponent added; their maximum.
template <bool EDGE>
__device__ __forceinline__ float kp_scores(const KvAttnArgs& a, const KpRow& row, uint32_t taddr, const KpSlot& slot, int shift,
                                           int first, int key0, int lo, int hi, float (&x)[kKpSub]) {
  float(&x0)[32] = reinterpret_cast<float(&)[32]>(x[0]);
  float(&x1)[32] = reinterpret_cast<float(&)[32]>(x[32]);
  t5_ld32_async(taddr, x0);
  t5_ld32_async(taddr + 32, x1);
  t5_ld32_wait(x0);
  t5_ld32_wait(x1);
  float top = -INFINITY;
#pragma unroll
  for (int h = 0; h < kKpSub; h += 16) {
    const KvPageScale ps = slot.sc[(first + h) >> shift];
    const float f = fminf(row.fac * ps.kfac, kKvMaxFloat);
    if constexpr (EDGE) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        x[h + i] = kp_score<true>(a, row, x[h + i], f, ps, key0 + first + h + i, lo, hi);
        top = fmaxf(top, x[h + i]);
      }
    } else {
      float m0 = fmaxf(fmaxf(x[h], x[h + 1]), x[h + 2]), m1 = fmaxf(fmaxf(x[h + 3], x[h + 4]), x[h + 5]);
      m0 = fmaxf(fmaxf(m0, x[h + 6]), x[h + 7]);
      m1 = fmaxf(fmaxf(m1, x[h + 8]), x[h + 9]);
      m0 = fmaxf(fmaxf(m0, x[h + 10]), x[h + 11]);
      m1 = fmaxf(fmaxf(m1, x[h + 12]), x[h + 13]);
      m0 = fmaxf(fmaxf(m0, x[h + 14]), x[h + 15]);
      top = fmaxf(top, fmaf(fmaxf(m0, m1), f, ps.ev));  // f >= 0
    }
  }
  return top;
}

// The scores of kKpSub keys (from their t) into a sum below with a z of its own, which lies in memory.
__device__ __forceinline__ float kp_wild_sum(float l, float* z, const KpSlot& slot, int shift, int first, const float (&x)[kKpSub]) {
  const float before = *z;
  float zn = before;
#pragma unroll
  for (int h = 0; h < kKpSub; h += 16) {
    float top = x[h];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, x[h + i]);
    zn = fmaxf(zn, top - slot.sc[(first + h) >> shift].ev);
  }
  const float z0 = zn == -INFINITY ? 0.f : zn;
  l *= fast_exp2(before - z0);
#pragma unroll
  for (int h = 0; h < kKpSub; h += 16) {
    const float e = slot.sc[(first + h) >> shift].ev + z0;
#pragma unroll
    for (int i = 0; i < 16; ++i) l += fast_exp2(x[h + i] - e);
  }
  *z = zn;
  return l;
}

// Weights over the scores' place; returns their sum (of 2^(t - m) 2^-ev).
template <bool EDGE>
__device__ __forceinline__ float kp_weights(const KpRow& row, uint32_t taddr, const KpSlot& slot, int shift, int first, float m,
                                            const float (&x)[kKpSub]) {
  float sum = 0.f;
#pragma unroll
  for (int c = 0; c < kKpSub; c += 32) {
    uint32_t p[16];
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      const KvPageScale ps = slot.sc[(first + c + h) >> shift];
      const float f = fminf(row.fac * ps.kfac, kKvMaxFloat), e = ps.ev - m;
      float2 part = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const float x0 = x[c + h + i], x1 = x[c + h + i + 1];
        float2 w = EDGE ? make_float2(x0 - m, x1 - m) : fma_f32x2(make_float2(x0, x1), make_float2(f, f), make_float2(e, e));
        w = make_float2(fast_exp2(w.x), fast_exp2(w.y));
        part = add_f32x2(part, w);
        p[(h + i) / 2] = f32x2_to_elem2<true>(w.x, w.y);
      }
      sum = fmaf(part.x + part.y, ps.inv, sum);
    }
    t5_st16(taddr + c / 2, p);
  }
  return sum;
}

template <int D, bool F16>
__global__ void __launch_bounds__(kKpThreads, 1)
    kv_prompt_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v, const KvAttnArgs a) {
  using S = KpShape<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  uint8_t* wide = smem + 2 * S::kHalfBytes;
  uint8_t* raw = wide + kKpWide * S::kWideBytes;
  __shared__ uint64_t raw_full[kKpRaw], raw_empty[kKpRaw], wide_full[kKpWide], wide_empty[kKpWide];
  __shared__ uint64_t q_full[2], s_full[2][2], p_full[2][2], pv_done[2], o_full[2], drain_bar;  // [half][S tile]
  __shared__ KpSlot slots[kKpSlots];
  __shared__ KvStart start;
  __shared__ KvWalk<kKpRows, kKpKeys> walks[4];
  __shared__ volatile uint32_t more[2];
  __shared__ int64_t warp_sum[kKpThreads / 32];
  __shared__ uint32_t tmem_slot, spoiled;
  __shared__ volatile uint32_t abort_flag, fills, used_tiles, go_on, last;

  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kKpRaw; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], 4);
    }
    for (int i = 0; i < kKpWide; ++i) {
      mbar_init(&wide_full[i], 4);
      mbar_init(&wide_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 4);
      for (int t = 0; t < 2; ++t) {
        mbar_init(&s_full[i][t], 1);
        mbar_init(&p_full[i][t], 4);
      }
      mbar_init(&pv_done[i], 1);
      mbar_init(&o_full[i], 1);
    }
    mbar_init(&drain_bar, 1);
    abort_flag = 0u;
    fills = used_tiles = 0u;
    fence_mbar_init();
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  pdl_wait();
  if (!kv_start<kKpRows, kKpKeys, kKpThreads>(a, 1, warp_sum, &spoiled, &start)) return;  // the whole block
  if (warp == 13) t5_alloc(&tmem_slot, 512);
  t5_fence_before();
  __syncthreads();
  t5_fence_after();
  const uint32_t tmem = warp_uniform(static_cast<int>(tmem_slot));
  // one walk for the eight softmax warps, one for the converters, one each for codes and products
  KvWalk<kKpRows, kKpKeys>& walk = walks[warp < 8 ? 0 : warp < 12 ? 1 : warp == 12 ? 2 : 3];
  const KvSegment& g = walk.seg;
  walk.begin(a, start, lane == 0 && (warp == 0 || warp == 8 || warp == 12 || warp == 13));
  const auto fail = [&]() {
    if (abort_flag == 0u) record_error_at(a.err, kErrTimeout);
    abort_flag = 1u;
  };

  if (warp == 12) {
    // ---- codes
    uint32_t n = 0, unit = 0;
    const int box = min(a.page, kKpKeys), boxes = kKpKeys / box;
    bool ok = true;
    while (ok && walk.step(a)) {
      const int32_t* table = a.table + static_cast<int64_t>(g.b) * a.table_ld;
      const int pages = (g.hi + a.page - 1) >> a.page_shift;  // beyond these no entry is read
      int batch0 = -1, pid = -1;
      KvPageScale sc{};
      for (int t = g.tile0; t < g.tile1 && ok; ++t, ++unit) {
        const int pg0 = (t * kKpKeys) >> a.page_shift;
        if (batch0 < 0 || pg0 + boxes > batch0 + 32) {
          batch0 = pg0;
          const int pg = pg0 + lane;
          pid = pg < pages ? table[pg] : -1;
          const bool valid = pid >= 0 && pid < a.num_pages;
          if (pg < pages && !valid && (pg + 1) << a.page_shift > g.lo) record_error_at(a.err, kErrValue);
          const int64_t at = static_cast<int64_t>(pid) * a.kv_heads + g.head;
          sc = kv_page_scale(a, valid ? a.scales[0][at] : -1, valid ? a.scales[1][at] : -1);
          if (!valid) pid = -1;
        }
        const int first = pg0 - batch0;
        const uint32_t got = __ballot_sync(~0u, pid >= 0) >> first & ((1u << boxes) - 1u);
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv) {
          const uint32_t slot = n % kKpRaw;
          ok = __all_sync(~0u, mbar_wait_clocked(&raw_empty[slot], (n / kKpRaw & 1u) ^ 1u, &abort_flag));
          if (!ok) break;
          if (kv == 0) {  // the softmax reads these after the unit's scores, long before 8 units on
            if (lane >= first && lane < first + boxes) slots[unit % kKpSlots].sc[lane - first] = sc;
            const uint32_t wild = __ballot_sync(~0u, fabsf(sc.ev) > kKvTameExp) >> first & ((1u << boxes) - 1u);
            if (lane == 0) slots[unit % kKpSlots].special = (got != (1u << boxes) - 1u ? 1u : 0u) | (wild != 0u ? 2u : 0u);
            __syncwarp();
          }
          if (lane == 0) mbar_arrive_expect_tx(&raw_full[slot], __popc(got) * box * D);
          for (int i = 0; i < boxes; ++i) {
            const int id = __shfl_sync(~0u, pid, first + i);
            if (lane == 0 && id >= 0)
              tma_load_4d(raw + slot * S::kRawBytes + i * box * D, kv == 0 ? &map_k : &map_v, 0, (t * kKpKeys + i * box) & (a.page - 1),
                          g.head, id, &raw_full[slot]);
          }
          ++n;
          if (lane == 0) fills = n;
        }
      }
    }
    if (!ok && lane == 0) fail();
  } else if (warp >= 8 && warp < 12) {
    // ---- E4M3 to FP16
    const int ct = tid - 256;
    constexpr int kRowThreads = D / 16, kRowsPerIter = 128 / kRowThreads;
    uint32_t n = 0, unit = 0;
    bool ok = true;
    while (walk.step_together(a, 2, 128, ct == 0, &more[1], &abort_flag)) {
      for (int t = g.tile0; t < g.tile1 && ok; ++t, ++unit) {
        const bool ends = t * kKpKeys < g.lo || (t + 1) * kKpKeys > g.hi;
#pragma unroll 1
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const uint32_t r = n % kKpRaw, w = n % kKpWide;
          ok = __all_sync(~0u, mbar_wait_clocked(&raw_full[r], n / kKpRaw & 1u, &abort_flag) &&
                                   mbar_wait_clocked(&wide_empty[w], (n / kKpWide & 1u) ^ 1u, &abort_flag));
          if (!ok) break;
          const uint8_t* src = raw + r * S::kRawBytes;
          uint8_t* dst = wide + w * S::kWideBytes;
          const KpSlot& slot = slots[unit % kKpSlots];
          const bool some = ends || (slot.special & 1u) != 0u;
          // 16 dimensions of keys key0, key0 + kRowsPerIter, ...; the second 64 dimensions' lanes
          // store their halves the other way round, so that a row's stores fall into different banks
          const int c = ct % kRowThreads, key0 = ct / kRowThreads, block = c >> 2, ch = 2 * (c & 3), sw = key0 & 7;
          const uint8_t* from = src + key0 * D + 16 * c;
          uint8_t* to = dst + block * (kKpKeys * 128) + key0 * 128;
          const int at0 = ((ch + block) ^ sw) << 4, at1 = ((ch + 1 - block) ^ sw) << 4;
          constexpr int kIters = 128 / kRowsPerIter, kBatch = 8 < kIters ? 8 : kIters;
#pragma unroll 1
          for (int i0 = 0; i0 < kIters; i0 += kBatch) {
            uint4 v[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) v[i] = *reinterpret_cast<const uint4*>(from + (i0 + i) * kRowsPerIter * D);
            if (some) {
#pragma unroll
              for (int i = 0; i < kBatch; ++i) {
                const int key = key0 + (i0 + i) * kRowsPerIter, k = t * kKpKeys + key;
                if (k < g.lo || k >= g.hi || slot.sc[key >> a.page_shift].inv == 0.f) v[i] = make_uint4(0, 0, 0, 0);
              }
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const uint4 x = make_uint4(e4m3x2_to_f16x2(v[i].x & 0xFFFFu), e4m3x2_to_f16x2(v[i].x >> 16),
                                         e4m3x2_to_f16x2(v[i].y & 0xFFFFu), e4m3x2_to_f16x2(v[i].y >> 16));
              const uint4 y = make_uint4(e4m3x2_to_f16x2(v[i].z & 0xFFFFu), e4m3x2_to_f16x2(v[i].z >> 16),
                                         e4m3x2_to_f16x2(v[i].w & 0xFFFFu), e4m3x2_to_f16x2(v[i].w >> 16));
              uint8_t* row = to + (i0 + i) * kRowsPerIter * 128;
              *reinterpret_cast<uint4*>(row + at0) = block ? y : x;
              *reinterpret_cast<uint4*>(row + at1) = block ? x : y;
            }
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&wide_full[w]);
            mbar_arrive(&raw_empty[r]);
          }
          if (ct == 0) used_tiles = n + 1;
        }
      }
      if (!ok && lane == 0) fail();
    }
  } else if (warp == 13) {
    // ---- products
    const uint32_t lead = t5_elect();
    const uint32_t q_addr = smem_addr(smem), wide_addr = smem_addr(wide);
    constexpr uint32_t kIdS = t5_idesc_f16(kKpSub, false), kIdO = t5_idesc_f16(D, true);
    uint32_t n = 0, queries[2] = {0u, 0u}, k[2] = {0u, 0u};
    bool ok = true;
    const auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(~0u, mbar_wait_clocked(bar, parity, &abort_flag)); };
    const auto scores = [&](int h, int sub, uint32_t w) {  // S tile: tensor memory columns 128 h + 64 sub ..
      const uint32_t qa = q_addr + h * S::kHalfBytes, ka = wide_addr + w * S::kWideBytes + sub * (kKpSub * 128);
      t5_mma_f16_ss<D / 64>(tmem + 128 * h + kKpSub * sub, t5_desc_sw128(qa), t5_desc_sw128(ka), kIdS, lead);
      t5_commit(smem_addr(&s_full[h][sub]), lead);
    };
    const auto values = [&](int h, int sub, uint32_t w, uint32_t accumulate) {  // O of half h: columns 256 + 128 h ..
      const uint32_t va = wide_addr + w * S::kWideBytes + sub * (kKpSub * 128);
      t5_mma_f16_ts(tmem + 256 + 128 * h, tmem + 128 * h + kKpSub * sub, t5_desc_sw128_n(va, 16384), kIdO, accumulate, lead);
      t5_commit(smem_addr(&pv_done[h]), lead);
    };
    while (ok && walk.step(a)) {
      const int units = warp_uniform(g.tile1 - g.tile0);
      const int halves = warp_uniform(g.s.n * a.group - g.rt * kKpRows) > 128 ? 2 : 1;
      if (units > 0) {
        for (int h = 0; h < halves && ok; ++h) ok = wait(&q_full[h], queries[h]++ & 1u);
        ok = ok && wait(&wide_full[n % kKpWide], n / kKpWide & 1u);
        if (!ok) break;
        t5_fence_after();
        for (int sub = 0; sub < 2; ++sub)
          for (int h = 0; h < halves; ++h) scores(h, sub, n % kKpWide);
        t5_commit(smem_addr(&wide_empty[n % kKpWide]), lead);
        ++n;
      }
      for (int u = 0; u < units && ok; ++u) {
        const uint32_t v = n % kKpWide, nk = (n + 1) % kKpWide;  // this unit's values, the next one's keys
        const bool next = u + 1 < units;
        ok = wait(&wide_full[v], n / kKpWide & 1u);
#pragma unroll 1
        for (int sub = 0; sub < 2 && ok; ++sub) {
#pragma unroll 1
          for (int h = 0; h < halves && ok; ++h) {
            ok = wait(&p_full[h][sub], k[h] & 1u);
            if (!ok) break;
            t5_fence_after();
            values(h, sub, v, u | sub);
            if (sub == 1) {
              if (!next) t5_commit(smem_addr(&o_full[h]), lead);
              ++k[h];
              if (h == halves - 1) t5_commit(smem_addr(&wide_empty[v]), lead);
            }
            if (next) {
              if (sub == 0 && h == 0) {
                ok = wait(&wide_full[nk], (n + 1) / kKpWide & 1u);
                if (!ok) break;
                t5_fence_after();
              }
              scores(h, sub, nk);
            }
          }
        }
        if (ok && next) t5_commit(smem_addr(&wide_empty[nk]), lead);
        n += next ? 2 : 1;
      }
    }
    if (!ok && lane == 0) fail();
    t5_commit(smem_addr(&drain_bar), lead);
    if (!mbar_wait_clocked(&drain_bar, 0) && lane == 0) record_error_at(a.err, kErrTimeout);
  } else if (warp < 8) {
    // ---- softmax of half `half`, a thread per row
    const int half = warp >> 2, quarter = warp & 3, r_half = 32 * quarter + lane, r_tile = 128 * half + r_half;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const uint32_t ts = lanes + 128 * half, to = lanes + 256 + 128 * half;
    const int shift = min(a.page_shift, 7);
    float* const row_z = a.part + 2 * static_cast<int64_t>(blockIdx.x) * S::kPartFloats + kKpRows * D + 3 * kKpRows + r_tile;
    uint32_t unit = 0, k = 0, finished = 0;
    bool ok = true;
    while (walk.step_together(a, 1, 256, tid == 0, &more[0], &abort_flag)) {
      const int rows = g.s.n * a.group, r = g.rt * kKpRows + r_tile, pos0 = g.s.len - g.s.n;
      const int half_rows = min(128, rows - g.rt * kKpRows - 128 * half);  // <= 0: the half is empty
      const bool busy = half_rows > 0 && g.tile1 > g.tile0;
      const int tok = kv_token(a, r);
      const int64_t out_row = static_cast<int64_t>(g.s.t0 + tok) * a.heads + g.head * a.group + r - tok * a.group;
      KpRow row{-INFINITY, 0.f, 0.f, pos0 + tok, r < rows};
      if (busy) {
        // the query row in FP16, 2^-eq of it
        const uint16_t* src = a.q + static_cast<int64_t>(g.s.t0 + tok) * a.q_tok + (g.head * a.group + r - tok * a.group) * a.q_head;
        uint4 v[D / 8];
        uint32_t mag = 0;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) v[i] = row.live ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          mag = elem_absmax2<F16>(elem_absmax2<F16>(elem_absmax2<F16>(elem_absmax2<F16>(mag, v[i].x), v[i].y), v[i].z), v[i].w);
        const float amax = elem_absmax_final<F16>(mag);
        const int eq = kv_query_exp(amax);
        const float f = copysignf(pow2f(-eq), a.scale_pow);  // scores times a factor >= 0
        row.fac = fabsf(a.scale_pow) * pow2f(eq);
        uint8_t* dst = smem + half * S::kHalfBytes + r_half * 128;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const float2 x = elem2_to_f32x2<F16>(v[i].x), y = elem2_to_f32x2<F16>(v[i].y), z = elem2_to_f32x2<F16>(v[i].z), w = elem2_to_f32x2<F16>(v[i].w);
          *reinterpret_cast<uint4*>(dst + (i >> 3) * 16384 + (((i & 7) ^ (r_half & 7)) << 4)) =
              make_uint4(f32x2_to_elem2<true>(x.x * f, x.y * f), f32x2_to_elem2<true>(y.x * f, y.y * f),
                         f32x2_to_elem2<true>(z.x * f, z.y * f), f32x2_to_elem2<true>(w.x * f, w.y * f));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[half]);
      }
      const int last_row = min(rows, g.rt * kKpRows + 128 * (half + 1)) - 1, first_row = g.rt * kKpRows + 128 * half;
      const int tile0 = g.tile0, tile1 = g.tile1, lo = g.lo, hi = g.hi;
      // positions of the half's first and last row
      const int pos_first = pos0 + kv_token(a, first_row), pos_last = pos0 + kv_token(a, last_row);
      int t = tile0;
      // The units from t on; without kWild up to the first page that wants z to be the scores' own (in *row_z).
      const auto walk_units = [&](auto wild_tag) {
        constexpr bool kWild = decltype(wild_tag)::value;
        bool leave = false;
        for (; t < tile1 && ok; ++t, ++unit) {
          if (!busy) continue;
          const KpSlot& slot = slots[unit % kKpSlots];
          const int key0 = t * kKpKeys;
          bool masked = false;
#pragma unroll 1
          for (int sub = 0; sub < 2; ++sub) {
            ok = __all_sync(~0u, mbar_wait_clocked(&s_full[half][sub], k >> 1 & 1u, &abort_flag));
            if (!ok) break;
            t5_fence_after();
            if (sub == 0)
              masked = kWild || slot.special != 0u || key0 < lo || key0 + kKpKeys > hi || (a.causal && key0 + kKpKeys - 1 > pos_first) ||
                       (a.window > 0 && key0 <= pos_last - a.window);
            if (!kWild && masked && (slot.special & 2u) != 0u) {  // while sub is 0
              leave = true;
              break;
            }
            const uint32_t tile = ts + kKpSub * sub;
            const int first = kKpSub * sub;
            float x[kKpSub];
            const float top = masked ? kp_scores<true>(a, row, tile, slot, shift, first, key0, lo, hi, x)
                                     : kp_scores<false>(a, row, tile, slot, shift, first, key0, lo, hi, x);
            if constexpr (kWild) row.l = kp_wild_sum(row.l, row_z, slot, shift, first, x);
            if (__any_sync(~0u, top > row.m + kKvLag)) {
              const float mn = fmaxf(row.m, top - kKvAbove), f = row.m == -INFINITY ? 0.f : fast_exp2(row.m - mn);
              row.m = mn;
              if constexpr (!kWild) row.l *= f;
              // O holds the keys before: wait for the last product (the one before it is done: these
              // scores came after it)
              if (t > tile0 || sub > 0) {
                ok = __all_sync(~0u, mbar_wait_clocked(&pv_done[half], (k - 1u) & 1u, &abort_flag));
                if (!ok) break;
                t5_fence_after();
#pragma unroll 1
                for (int c = 0; c < D; c += 16) {
                  float y[16];
                  t5_ld16(to + c, y);
#pragma unroll
                  for (int i = 0; i < 16; ++i) y[i] *= f;
                  t5_st16f(to + c, y);
                }
              }
            }
            const float m = row.m == -INFINITY ? 0.f : row.m;
            const float sum = masked ? kp_weights<true>(row, tile, slot, shift, first, m, x) : kp_weights<false>(row, tile, slot, shift, first, m, x);
            if constexpr (!kWild) row.l += sum;
            t5_st_wait();
            t5_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_full[half][sub]);
            ++k;
          }
          if (leave) break;
        }
      };
      walk_units(std::false_type{});
      if (ok && t < tile1) {
        *row_z = row.m;
        walk_units(std::true_type{});
        row.l = -row.l;  // as in memory (KvSum)
      }
      if (ok && busy) {
        // of its own, once an item: pv_done may be two phases behind here, which its parity could not tell
        ok = __all_sync(~0u, mbar_wait_clocked(&o_full[half], finished++ & 1u, &abort_flag));
        t5_fence_after();
      }
      if (!ok && lane == 0) fail();
      // ---- the item's share
      const KvJoin team(start, g.first, g.count);
      named_sync(1, 256);
      if (tid == 0) go_on = abort_flag != 0u ? 0u : team.arrived_but_one(a) ? 2u : 1u;
      named_sync(1, 256);
      ok = go_on != 0u;  // one answer for all warps
      const bool direct = go_on == 2u;
      // 32 dimensions of this thread's row, and its sum, to a part, or where there is none to the output
      const auto put = [&](int c, const float (&x)[32], float am, const KvSum& below, float* part) {
        if (part != nullptr) {
#pragma unroll
          for (int i = 0; i < 32; ++i) __stcg(part + (c + i) * kKpRows + r_tile, x[i]);
          if (c == 0) {
            __stcg(part + kKpRows * D + r_tile, am);
            __stcg(part + kKpRows * D + kKpRows + r_tile, below.stored());
            if (below.wild) __stcg(part + kKpRows * D + 2 * kKpRows + r_tile, below.z);
          }
          return;
        }
        // a wild sum's 2^(m - z) in two steps: the whole may pass FP32 where the output does not
        const float half = below.wild ? fast_exp2(0.5f * (am - below.z)) : 1.f, inv = below.l > 0.f ? half / below.l : 0.f;
#pragma unroll
        for (int i = 0; i < 32; i += 8)
          *reinterpret_cast<uint4*>(a.out + out_row * D + c + i) =
              make_uint4(f32x2_to_elem2<F16>(x[i] * inv * half, x[i + 1] * inv * half),
                         f32x2_to_elem2<F16>(x[i + 2] * inv * half, x[i + 3] * inv * half),
                         f32x2_to_elem2<F16>(x[i + 4] * inv * half, x[i + 5] * inv * half),
                         f32x2_to_elem2<F16>(x[i + 6] * inv * half, x[i + 7] * inv * half));
        if (c == 0 && a.lse != nullptr) a.lse[out_row] = below.lse(am);
      };
      const int head = team.head(), groups = team.groups();
      const bool whole = team.count == 1 || direct;
      // Three steps, as far as they are this block's: its own rows (with the group's other parts, where they are there),
      // the group's parts, the groups' parts.  Each takes n of them, from part i0 on every step-th, to a part or
      // the output; a row's thread reads and writes it alone.  Own rows come from tensor memory and are the
      // first of their group: the same operations on the same numbers as from a part.
#pragma unroll 1
      for (int level = whole ? 0 : -1; ok && level < (groups > 1 ? 2 : 1); ++level) {
        const bool own = level < 0 || (level == 0 && whole), top = level == 1;
        const int i0 = top ? 0 : head, step = top ? team.join : 1, n = level < 0 ? 1 : top ? groups : team.members();
        float* const to_part = level < 0 ? team.part(a, team.me, S::kPartFloats) : !top && groups > 1 ? team.part(a, head, S::kPartFloats) : nullptr;
        if (!own && !kv_arrive(top ? team.item_counter(a) : team.group_counter(a), n, 1, 256, tid == 0, &last)) break;
        if (half_rows <= 0) continue;  // uniform per warp
        const int p0 = own ? 1 : 0, p1 = row.live ? n : 0;
        const auto part_of = [&](int p) { return team.part(a, i0 + p * step, S::kPartFloats) + r_tile; };
        KvSum below;
        float am = -INFINITY;
        if (own) {
          below = KvSum{fabsf(row.l), row.l < 0.f ? *row_z : row.m, row.l < 0.f};
          am = row.m;
        }
        for (int p = p0; p < p1; ++p) {
          const float pm = __ldcg(part_of(p) + kKpRows * D), pl = __ldcg(part_of(p) + kKpRows * D + kKpRows);
          const float mm = fmaxf(am, pm);
          if (below.wild || pl < 0.f) {
            if (!below.wild) below.z = am;
            below.add_wild(pm, pl, __ldcg(part_of(p) + kKpRows * D + 2 * kKpRows));
          } else {
            below.l = below.l * (am == -INFINITY ? 0.f : fast_exp2(am - mm)) + pl * (pm == -INFINITY ? 0.f : fast_exp2(pm - mm));
          }
          am = mm;
        }
        const float f0 = row.m == -INFINITY ? 0.f : fast_exp2(row.m - am);
        __syncwarp();  // tensor-memory loads want the whole warp
#pragma unroll 1
        for (int c = D - 32; c >= 0; c -= 32) {  // the maxima are read in every round and replaced in the last
          float x[32];
          if (own && busy) t5_ld32(to + c, x);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = own && busy ? x[i] * f0 : 0.f;
          for (int p = p0; p < p1; ++p) {
            const float pm = __ldcg(part_of(p) + kKpRows * D), f = pm == -INFINITY ? 0.f : fast_exp2(pm - am);
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = fmaf(f, __ldcg(part_of(p) + (c + i) * kKpRows), x[i]);
          }
          if (row.live) put(c, x, am, below, to_part);
          __syncwarp();
        }
        t5_fence_before();
      }
    }
  }
  __syncthreads();
  // after an expired wait: loads that nothing consumed land before the block ends
  if (tid == 0 && abort_flag != 0u) a.arrived[kKvSpoiled] = 1u;
  if (tid == 0)
    for (uint32_t f = used_tiles; f < fills; ++f)
      if (!mbar_wait_clocked(&raw_full[f % kKpRaw], f / kKpRaw & 1u)) record_error_at(a.err, kErrTimeout);
  t5_fence_before();
  __syncthreads();
  t5_fence_after();
  if (warp == 13) {
    __syncwarp();
    t5_dealloc(tmem, 512);
  }
}

}  // namespace bsq
