// Attention over the 8-bit paged cache, for few query rows per kv head
// (single tokens, guessed tokens).
//
// Per query row of a head, over the allowed keys j of its sequence:
//   s_j = sm_scale log2(e) q.k_j,  out = sum_j 2^s_j v_j / sum_j 2^s_j.
// A page holds codes under power-of-two scales, k = c 2^ek and v = c 2^ev.  The
// value scale goes into the exponent: with t_j = s_j + ev_j, a reference m of those (the running maximum less
// kKvAbove, once that is kKvLag above it) and a reference z of the scores,
//   out = 2^(m - z) sum_j 2^(t_j - m) c_j / sum_j 2^(s_j - z),
// so the weights of the codes stay within FP16 whatever the pages' scales are, and
// nothing is multiplied into the values.  While the pages' |ev| are at most kKvTameExp, z is m and the sum below
// takes 2^(t_j - m) 2^-ev, an exponential per key for both: it stays below 2^(55 + 30), and what 2^(t_j - m) loses
// below 2^-126 is less than 2^-53 of the largest.  From the first page past that on, an item's share
// has a z of its own, the scores' running maximum, and exponentials of its own for the sum.
// The key scale is one factor of a tile's scores.  E4M3 codes and scaled query rows (a power of two per row) are exact in FP16
// (but for elements below 2^-29 of a row's largest in BF16, 2^-26 in FP16: off by 2^-37 of it at most);
// weights are rounded to FP16 (a relative 2^-11 each, against 2^-9 of a BF16
// output; the row's largest is between 2^kKvAbove and 2^kKvLag, so that subnormal ones are off by 2^-32 of
// it at most), and all sums are FP32.
//
// What bounds it: the cache is read once, about 2 x heads-per-kv-head operations
// per byte, so DRAM.  Persistent blocks (one to three per SM) of four consumer warps and a
// producer; the units, tiles of 64 keys of one (sequence, kv head, row tile), are cut
// into equal runs, so that ragged lengths and long contexts spread evenly.  The
// producer streams tiles by TMA through a ring.  Each consumer warp takes 16 of a tile's
// keys for all rows and keeps its own maximum, sums and accumulators, so warps meet
// only at the end of an item.  mma.sync products: with 32 rows at most, a 128-row
// tensor-memory product would be mostly padding.  The products are transposed, keys
// (S^T = K Q^T) and dimensions (O^T = V^T P^T) as the 16-row side, so that 8 query rows (NT = 1) are no
// padding either.  Fragments come straight from the codes with wide shared loads: the order of the
// dimension in q.k and of the output rows is free, so a thread takes 16 consecutive bytes of a
// key, and pairs of keys are interleaved bytewise before conversion.
// Measured (64 contexts of 1000 to 8192 tokens, 64 heads of 128 over 8, a graph of calls): 8 rows
// per kv head 101 us, 6.0 TB/s or 89 % of a plain copy; 16 rows 118 us and 32 rows 248 us, where
// the conversions and mma.sync products bound it.  One context of 777: 10.0 us, a chain of
// latencies (lengths, table, codes, the join: 4 of them); two of 131072, 4 kv heads: 53 us.
// An item cut by the runs is joined from its blocks' parts, in block order, by whichever block stores its part last
// (first in groups where there are many).  So no block waits for another, whether it is on the GPU yet or not, and
// the sums' order does not depend on which one is last.
#pragma once

#include <type_traits>

#include "tcgen05.cuh"

namespace bsq {

constexpr int kKvTile = 64;       // keys per unit
constexpr int kKvMaxBlocks = 512;
constexpr int kKvMinRun = 3;      // units of a run, at least, once every SM has one
// Parts of an item that are joined at once, and the size of the groups
// that are joined first where there are more: about their number's square root.  (104 parts, one
// context of 20000 with one kv head: 14.1 us, 27.9 when one block joins them all; 57 parts of
// contexts of 131072: 52.7 / 59.3, and 51.7 for groups of 5, 54.8 for groups of 20.)
__device__ __forceinline__ int kv_join_group(int parts) { return parts <= 20 ? parts : parts <= 72 ? 8 : 16; }
// Parts stored so far, zero between calls: of a group (by its first block, which can be the first of one item and of
// a later group of the item before), of an item's groups (by the item's first block).
constexpr int kKvGroupCounters = 0, kKvLaterCounters = kKvMaxBlocks, kKvItemCounters = 2 * kKvMaxBlocks;
// Not 0 once a call has given up in a wait: what else the workspace holds is then not to be trusted.
constexpr int kKvSpoiled = 3 * kKvMaxBlocks;
constexpr int kKvCounterBytes = 4 * (3 * kKvMaxBlocks + 4);

struct KvAttnArgs {
  const uint16_t* q;              // (total, heads, D)
  int64_t q_tok, q_head;          // strides in elements
  const uint8_t* scales[2];       // (num_pages, kv_heads) E8M0 bytes
  const int32_t* table;
  int64_t table_ld;
  const int32_t* offsets;
  const int32_t* lens;
  uint16_t* out;                  // (total, heads, D) contiguous
  float* lse;                     // (total, heads) or NULL
  int64_t total, num_pages;
  int batch, heads, kv_heads, group, page, page_shift, table_width, causal, window;
  // sm_scale log2(e) as its power of two, with the sign, and its significand in [1, 2) (or 0): a row's power of two
  // takes the one, a page's the other, so that neither product loses bits below FP32's normal numbers
  float scale_pow, scale_sig;
  uint64_t group_inv;             // ceil(2^64 / group), for kv_token
  uint32_t* arrived;              // counters, and whether they hold
  float* part;                    // [block][first of the item, later][rows * D + 3 * rows]: sums, m, sums below, z
  unsigned int* err;
};

// The token of row r of a sequence, r / group (exact for r < 2^32; a division is some forty instructions).
__device__ __forceinline__ int kv_token(const KvAttnArgs& a, int r) {
  return a.group == 1 ? r : static_cast<int>(__umul64hi(static_cast<uint64_t>(r), a.group_inv));
}

// A sequence's rows and, per row tile, its keys.
struct KvSeq {
  int t0, n, len, row_tiles;
};
template <int RT>
__device__ __forceinline__ KvSeq kv_seq(const KvAttnArgs& a, int b, bool report) {
  KvSeq s;
  const int64_t t0 = a.offsets[b], t1 = a.offsets[b + 1];
  s.len = a.lens[b];
  bool ok = t0 >= 0 && t1 <= a.total;
  if (s.len < 0 || s.len > static_cast<int64_t>(a.table_width) * a.page) {
    ok = false;
    s.len = 0;
  }
  if (!ok && report) record_error_at(a.err, kErrValue);
  s.t0 = static_cast<int>(t0);
  s.n = t0 >= 0 && t1 <= a.total && t1 > t0 ? static_cast<int>(t1 - t0) : 0;
  s.row_tiles = (s.n * a.group + RT - 1) / RT;
  return s;
}
// Keys [lo, hi) that any row of tile rt may see (lo = hi: none).
template <int RT>
__device__ __forceinline__ void kv_keys(const KvAttnArgs& a, const KvSeq& s, int rt, int& lo, int& hi) {
  const int rows = s.n * a.group;
  const int i0 = kv_token(a, rt * RT), i1 = rows <= (rt + 1) * RT ? s.n - 1 : kv_token(a, (rt + 1) * RT - 1);
  hi = a.causal ? min(s.len, s.len - s.n + i1 + 1) : s.len;
  lo = a.window > 0 ? max(0, s.len - s.n + i0 - a.window + 1) : 0;
  if (hi <= lo) lo = hi = 0;
}
// Units of an item: tiles of TILE keys, one for an item without keys (its rows are still written).
template <int TILE>
__device__ __forceinline__ int kv_units(int lo, int hi) { return max(1, (hi + TILE - 1) / TILE - lo / TILE); }

template <int RT, int TILE>
__device__ __forceinline__ int64_t kv_seq_units(const KvAttnArgs& a, const KvSeq& s) {
  int64_t u = 0;
  for (int rt = 0; rt < s.row_tiles; ++rt) {
    int lo, hi;
    kv_keys<RT>(a, s, rt, lo, hi);
    u += kv_units<TILE>(lo, hi);
  }
  return u;  // per kv head
}

// A block's run of units, and the sequence it begins in.
struct KvStart {
  int64_t total;       // units in all
  int64_t before;      // units of the sequences before `seq`
  int seq, parts;      // parts: runs, none of them empty
  int64_t begin, end;  // this block's
  // total * i / parts and the run that holds a unit, in 32 bits where they suffice
  __device__ __forceinline__ int64_t start_of(int i) const {
    if (total < (1 << 21)) return static_cast<uint32_t>(total) * static_cast<uint32_t>(i) / static_cast<uint32_t>(parts);
    return total * i / parts;
  }
  __device__ __forceinline__ int owner(int64_t u) const {
    if (total < (1 << 21))
      return static_cast<int>(((static_cast<uint32_t>(u) + 1u) * static_cast<uint32_t>(parts) - 1u) / static_cast<uint32_t>(total));
    return static_cast<int>(((u + 1) * parts - 1) / total);
  }
};

// One item's share of a block's run.
struct KvSegment {
  KvSeq s;
  int b, head, rt, lo, hi;  // kv head, row tile, keys
  int tile0, tile1;         // of this share, in tiles of the sequence
  int64_t first, count;     // the item's units
};

// Walks the units [u, end) item by item.  Each warp has its own in shared
// memory, which its first lane moves on: kept in registers it would cost the
// loop over the keys some fifty of them.
template <int RT, int TILE>
struct KvWalk {
  int64_t u, end, at;       // the next unit, the run's end, the first unit of item (b, head, rt)
  int count, b, head, rt;   // the item's units
  int lo, hi;
  KvSeq s;
  KvSegment seg;
  // Whole warp; true while there is an item, described by seg.
  __device__ __forceinline__ bool step(const KvAttnArgs& a) {
    __syncwarp();
    bool more = false;
    if ((threadIdx.x & 31) == 0) more = next(a, seg);
    __syncwarp();
    return __shfl_sync(~0u, more ? 1 : 0, 0) != 0;
  }
  // The same for warps that share one: `threads` threads meet at barrier `id`;
  // none goes on once one of them has given up.
  __device__ __forceinline__ bool step_together(const KvAttnArgs& a, int id, int threads, bool first, volatile uint32_t* more,
                                                const volatile uint32_t* abort_flag) {
    named_sync(id, threads);
    if (first) *more = *abort_flag == 0u && next(a, seg) ? 1u : 0u;
    named_sync(id, threads);
    return *more != 0u;
  }
  __device__ __forceinline__ void begin(const KvAttnArgs& a, const KvStart& start, bool mine) {
    if (mine) {
      u = start.begin;
      end = start.end;
      b = start.seq;
      load(a);
      at = start.before;
      head = rt = 0;
      int64_t per_head = kv_seq_units<RT, TILE>(a, s);
      while (u >= at + per_head * a.kv_heads) {  // kv_start names a sequence at or before the first unit's
        at += per_head * a.kv_heads;
        ++b;
        load(a);
        per_head = kv_seq_units<RT, TILE>(a, s);
      }
      head = static_cast<int>((u - at) / per_head);
      at += head * per_head;
      keys(a);
    }
    __syncwarp();
  }
  __device__ __forceinline__ void load(const KvAttnArgs& a) { s = kv_seq<RT>(a, b, false); }
  __device__ __forceinline__ void keys(const KvAttnArgs& a) {
    lo = hi = count = 0;
    if (s.row_tiles == 0) return;  // a sequence without rows
    kv_keys<RT>(a, s, rt, lo, hi);
    count = kv_units<TILE>(lo, hi);
  }
  // The item that holds unit u, from the one before it.
  __device__ __forceinline__ bool next(const KvAttnArgs& a, KvSegment& g) {
    if (u >= end) return false;
    while (u >= at + count) {
      at += count;
      if (++rt >= s.row_tiles) {
        rt = 0;
        if (++head >= a.kv_heads || s.row_tiles == 0) {
          head = 0;
          ++b;
          load(a);
        }
      }
      keys(a);
    }
    g.first = at;
    g.count = count;
    g.lo = lo;
    g.hi = hi;
    g.head = head;
    g.rt = rt;
    g.b = b;
    g.s = s;
    const int64_t stop = min(end, at + count);
    g.tile0 = lo / TILE + static_cast<int>(u - at);
    g.tile1 = hi > lo ? g.tile0 + static_cast<int>(stop - u) : g.tile0;
    u = stop;
    return true;
  }
};

__device__ __forceinline__ void kv_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float fast_exp2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// 4D TMA tile (dimension, token, head, page).
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}

// Sum every sequence's units and find this block's run (by all THREADS of the
// block, a thread taking consecutive sequences); false for a block without one, or in a
// workspace that an earlier call spoiled.
template <int RT, int TILE, int THREADS>
__device__ __forceinline__ bool kv_start(const KvAttnArgs& a, int blocks_per_sm, int64_t* warp_sum, uint32_t* spoiled, KvStart* start) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.batch + THREADS - 1) / THREADS, b0 = min(a.batch, tid * per), b1 = min(a.batch, b0 + per);
  const uint32_t word = tid == 0 ? __ldcg(a.arrived + kKvSpoiled) : 0u;  // under way beside the lengths
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += kv_seq_units<RT, TILE>(a, kv_seq<RT>(a, b, blockIdx.x == 0)) * a.kv_heads;
  int64_t sum = mine;
#pragma unroll 1
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t o = __shfl_up_sync(~0u, sum, d);
    if (lane >= d) sum += o;
  }
  if (lane == 31) warp_sum[warp] = sum;
  if (tid == 0) *spoiled = word;
  __syncthreads();
  if (*spoiled != 0u) {
    if (tid == 0) record_error_at(a.err, kErrTimeout);
    return false;
  }
  KvStart s;
  s.total = 0;
#pragma unroll 1
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w == warp) sum += s.total;
    s.total += warp_sum[w];
  }
  // Joining a part costs about as much as a few units: at most one run per SM
  // until they have kKvMinRun units (contexts of 3000 tokens with 8 kv heads / 20000 with one / 8 of up to 2000:
  // 12.7 / 14.1 / 15.1 us, 12.6 / 15.5 / 15.1 with a run for every unit, 12.7 / 14.1 / 14.7 with at least four)
  s.parts = static_cast<int>(min(static_cast<int64_t>(gridDim.x),
                                 max(s.total / kKvMinRun, min(s.total, static_cast<int64_t>(gridDim.x / blocks_per_sm)))));
  if (static_cast<int>(blockIdx.x) >= s.parts) return false;
  s.begin = s.start_of(blockIdx.x);
  s.end = s.start_of(blockIdx.x + 1);
  if (sum - mine <= s.begin && s.begin < sum) {  // one thread
    s.before = sum - mine;
    s.seq = b0;  // KvWalk goes on to the sequence itself
    *start = s;
  }
  __syncthreads();
  return true;
}

// Per page of a stage: factor of the scores (with the significand of sm_scale log2(e)), exponent of the values, and its
// reciprocal power (0: no such page).
struct KvPageScale {
  float kfac, ev, inv;
};
constexpr float kKvAbove = 7.f, kKvLag = 15.f;  // 2^15 leaves FP16 a factor of 2
constexpr float kKvTameExp = 40.f;
// No such page, or |ev| above kKvTameExp, as one comparison of 2^-ev.
__device__ __forceinline__ bool kv_special(const KvPageScale& ps) {
  constexpr uint32_t kLeast = static_cast<uint32_t>(127 - static_cast<int>(kKvTameExp)) << 23;
  return __float_as_uint(ps.inv) - kLeast > static_cast<uint32_t>(2 * static_cast<int>(kKvTameExp)) << 23;
}
constexpr float kKvMaxFloat = 3.402823466e38f;

// From the scale bytes; -1: no such page.
__device__ __forceinline__ KvPageScale kv_page_scale(const KvAttnArgs& a, int ek, int ev) {
  if (ek < 0) return {0.f, 0.f, 0.f};
  return {a.scale_sig * pow2f(min(max(ek - 127, -126), 127)), static_cast<float>(ev - 127), pow2f(min(127 - ev, 127))};
}

// NT: tiles of 8 query rows.
template <int D, int NT>
struct KvShape {
  static constexpr int kWarps = 4;                         // consumers
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kRows = 8 * NT;
  static constexpr int kPassRows = NT == 1 ? 8 : 16;       // rows merged at a time
  // registers allow 15 warps per SM at 128, 10 at 168, 5 at 255 (five warps spread unevenly over four
  // schedulers); 64 contexts to 8192 with 8 rows: 101 us with three blocks, 104 with two of longer rings; with 16
  // rows 118 with two, 156 with three.  For dimensions of 64 the same numbers, not measured apart
  static constexpr int kBlocksPerSm = NT == 1 ? 3 : NT == 2 ? 2 : 1;
  static constexpr int kTileBytes = kKvTile * D;           // of keys, and of values
  static constexpr int kStages = NT == 1 ? 3 : NT == 2 ? 4 : 6;
  // merge buffer: a row's eighths lie 4 floats further apart and rows 4 modulo
  // 16, so that the rows and eighths of a warp's float4 stores fall into different banks
  static constexpr int kEighth = D / 8 + 4, kRow = 8 * kEighth + 4;
  static constexpr int kMergeBytes = kWarps * kPassRows * kRow * 4;
  // query rows in shared memory, in the merge buffer that an item uses after them, where registers are short: with
  // 16 rows of 128 (64 contexts to 8192 / 16 to 800) 118 / 16.1 us against 126 / 16.4 in registers, with 16 of 64
  // (guessed tokens) 28.8 against 26.5
  static constexpr bool kSharedQuery = NT == 4 || (NT == 2 && D == 128);
  static constexpr int kSmem = 1024 + kStages * 2 * kTileBytes + kMergeBytes;
  static constexpr int kPartFloats = kRows * D + 3 * kRows;
};

// A query row enters its products as 2^-eq of itself, with its largest magnitude in
// [2^12, 2^13).  Rows below 2^-114 stay smaller: there 2^-eq would pass FP32, and their
// elements, multiples of 2^-133 at least, are exact in FP16 at 2^126 as well.
__device__ __forceinline__ int kv_query_exp(float amax) {
  return amax > 0.f ? max(static_cast<int>(__float_as_uint(amax) >> 23) - 127 - 12, -126) : 0;
}

// The factor of a row's scores of a page.  Where the two together pass FP32 it is FP32's largest number, so that
// a score of 0 stays 0.
__device__ __forceinline__ float kv_score_factor(float row, float page) {
  return fminf(fmaxf(row * page, -kKvMaxFloat), kKvMaxFloat);
}

// A row's sum below, relative to 2^m, or to 2^z where some page made it wild.  In memory a wild sum is negative,
// and only then does its z count.
struct KvSum {
  float l = 0.f, z = -INFINITY;
  bool wild = false;
  // Adds another (as in memory, with its m and, if it is wild, z) where one of the two is wild.
  __device__ __forceinline__ void add_wild(float pm, float pl, float pz) {
    if (!(pl < 0.f)) pz = pm;
    const float zz = fmaxf(z, pz);
    l = l * (z == -INFINITY ? 0.f : fast_exp2(z - zz)) + fabsf(pl) * (pz == -INFINITY ? 0.f : fast_exp2(pz - zz));
    z = zz;
    wild = true;
  }
  __device__ __forceinline__ float stored() const { return wild ? -l : l; }
  // 0: no key; NaN stays NaN.
  __device__ __forceinline__ float lse(float m) const { return l == 0.f ? -INFINITY : ((wild ? z : m) + log2f(l)) * 0.6931471805599453f; }
};

// The codes of 4 consecutive dimensions of two keys -> for each dimension
// the pair (key 0, key 1) in FP16.
__device__ __forceinline__ void kv_pairs(uint32_t w0, uint32_t w1, uint32_t (&o)[4]) {
  const uint32_t lo = __byte_perm(w0, w1, 0x5140), hi = __byte_perm(w0, w1, 0x7362);
  o[0] = e4m3x2_to_f16x2(lo & 0xFFFFu);
  o[1] = e4m3x2_to_f16x2(lo >> 16);
  o[2] = e4m3x2_to_f16x2(hi & 0xFFFFu);
  o[3] = e4m3x2_to_f16x2(hi >> 16);
}

// Byte offset of 16-byte chunk `c` of row `r` in a tile that TMA wrote with
// the 128-byte (D = 128) or 64-byte (D = 64) swizzle.
template <int D>
__device__ __forceinline__ uint32_t kv_chunk(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// Where an item's blocks meet: block own0 + i is its i-th of `count`, in groups of `join`.
struct KvJoin {
  int own0, me, count, join;
  __device__ __forceinline__ KvJoin(const KvStart& start, int64_t first, int64_t units) {
    own0 = start.owner(first);
    me = static_cast<int>(blockIdx.x) - own0;
    count = start.owner(first + units - 1) - own0 + 1;
    join = kv_join_group(count);
  }
  __device__ __forceinline__ int head() const { return me / join * join; }
  __device__ __forceinline__ int members() const { return min(join, count - head()); }
  __device__ __forceinline__ int groups() const { return (count - 1) / join + 1; }
  __device__ __forceinline__ float* part(const KvAttnArgs& a, int i, int floats) const {
    return a.part + (2 * static_cast<int64_t>(own0 + i) + (i > 0 ? 1 : 0)) * floats;
  }
  __device__ __forceinline__ uint32_t* group_counter(const KvAttnArgs& a) const {
    return a.arrived + (head() > 0 ? kKvLaterCounters : kKvGroupCounters) + own0 + head();
  }
  // Whether this is the group's first block and the last to arrive, as it is as a rule (a block meets its last item's
  // beginning at the end of its run): it then need not store its own part.  The counter is 0 again.  One thread calls.
  __device__ __forceinline__ bool arrived_but_one(const KvAttnArgs& a) const {
    if (count == 1 || me != head() || ld_acquire(group_counter(a)) != static_cast<uint32_t>(members()) - 1u) return false;
    *group_counter(a) = 0u;
    return true;
  }
  __device__ __forceinline__ uint32_t* item_counter(const KvAttnArgs& a) const { return a.arrived + kKvItemCounters + own0; }
};

// The sums of a part onto others, both taken to the larger m; written out, so that it is the same wherever it is done.
__device__ __forceinline__ float kv_add(float x, float f0, float v, float f1) { return __fmaf_rn(v, f1, __fmul_rn(x, f0)); }

// `threads` threads of a block, whose parts are stored, meet at barrier `id`; true if theirs is the last of n
// (then all n can be read and the counter is 0 again).
__device__ __forceinline__ bool kv_arrive(uint32_t* counter, int n, int id, int threads, bool first, volatile uint32_t* last) {
  named_sync(id, threads);
  if (first) {
    const bool is_last = atomic_add_acq_rel(counter, 1u) == static_cast<uint32_t>(n) - 1u;
    if (is_last) *counter = 0u;
    *last = is_last ? 1u : 0u;
  }
  named_sync(id, threads);
  return *last != 0u;
}

// An 8 x 8 matrix of 16-bit elements over the warp, transposed.
__device__ __forceinline__ uint32_t kv_transpose(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

template <int D, int NT, bool F16>
__global__ void __launch_bounds__(KvShape<D, NT>::kThreads, KvShape<D, NT>::kBlocksPerSm)
    kv_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ KvAttnArgs a) {
  using S = KvShape<D, NT>;
  constexpr int RT = S::kRows, kT = 32 * S::kWarps;
  constexpr int kQuads = D / 64;  // 16-byte loads of a key per thread
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  float* merge = reinterpret_cast<float*>(smem + S::kStages * 2 * S::kTileBytes);
  [[maybe_unused]] uint4* query = reinterpret_cast<uint4*>(merge);
  __shared__ uint64_t full_bar[S::kStages], empty_bar[S::kStages];
  __shared__ KvPageScale page_scale[S::kStages][4];
  __shared__ float warp_m2[2][S::kWarps][RT], warp_z2[2][S::kWarps][RT], warp_l2[2][S::kWarps][RT];  // by parity of the item
  __shared__ KvWalk<RT, kKvTile> walks[S::kWarps + 1];
  __shared__ KvStart start;
  __shared__ int64_t warp_sum[S::kWarps + 1];
  __shared__ uint32_t spoiled;
  __shared__ volatile uint32_t abort_flag, fills, used_tiles, go_on, last;

  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(&full_bar[s], 2);  // codes, scales
      mbar_init(&empty_bar[s], S::kWarps);
    }
    abort_flag = 0u;
    fills = 0u;
    fence_mbar_init();
    prefetch_tensormap(&map_k);
    prefetch_tensormap(&map_v);
  }
  __syncthreads();
  pdl_wait();
  KvWalk<RT, kKvTile>& walk = walks[warp];
  const KvSegment& g = walk.seg;
  if (!kv_start<RT, kKvTile, S::kThreads>(a, S::kBlocksPerSm, warp_sum, &spoiled, &start)) return;  // the whole block
  walk.begin(a, start, lane == 0);

  if (warp == S::kWarps) {
    // ---- producer
    uint32_t stage = 0, phase = 0, n = 0;
    const int box = min(a.page, kKvTile), boxes = kKvTile / box;
    bool ok = true;
    while (ok && walk.step(a)) {
      const int32_t* table = a.table + static_cast<int64_t>(g.b) * a.table_ld;
      const int pages = (g.hi + a.page - 1) >> a.page_shift;  // beyond these no entry is read
      int batch0 = -1, pid = -1;
      int ek = -1, ev = -1;
      for (int t = g.tile0; t < g.tile1; ++t) {
        const int pg0 = (t * kKvTile) >> a.page_shift;
        if (batch0 < 0 || pg0 + boxes > batch0 + 32) {  // the next 32 pages' ids and scales, one per lane
          batch0 = pg0;
          const int pg = pg0 + lane;
          pid = pg < pages ? table[pg] : -1;
          const bool valid = pid >= 0 && pid < a.num_pages;
          // pages before the first allowed key are masked anyway and need no entry
          if (pg < pages && !valid && (pg + 1) << a.page_shift > g.lo) record_error_at(a.err, kErrValue);
          if (!valid) pid = -1;
          ek = ev = -1;
          if (valid) {  // used only after the codes have been requested
            const int64_t at = static_cast<int64_t>(pid) * a.kv_heads + g.head;
            ek = a.scales[0][at];
            ev = a.scales[1][at];
          }
        }
        if (lane == 0) ok = mbar_wait_clocked(&empty_bar[stage], phase ^ 1u, &abort_flag);
        ok = __shfl_sync(~0u, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
        const int first = pg0 - batch0;
        const uint32_t got = __ballot_sync(~0u, pid >= 0) >> first & ((1u << boxes) - 1u);
        uint8_t* kd = smem + stage * 2 * S::kTileBytes;
        if (lane == 0) mbar_arrive_expect_tx(&full_bar[stage], 2u * __popc(got) * box * D);
        for (int i = 0; i < boxes; ++i) {
          const int id = __shfl_sync(~0u, pid, first + i);
          if (lane == 0 && id >= 0) {
            const int y = (t * kKvTile + i * box) & (a.page - 1);
            tma_load_4d(kd + i * box * D, &map_k, 0, y, g.head, id, &full_bar[stage]);
            tma_load_4d(kd + S::kTileBytes + i * box * D, &map_v, 0, y, g.head, id, &full_bar[stage]);
          }
        }
        if (lane >= first && lane < first + boxes) page_scale[stage][lane - first] = kv_page_scale(a, ek, ev);
        __syncwarp();
        if (lane == 0) mbar_arrive(&full_bar[stage]);
        ++n;
        if (lane == 0) fills = n;
        if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
      }
    }
    if (!ok && lane == 0) {
      if (abort_flag == 0u) record_error_at(a.err, kErrTimeout);
      abort_flag = 1u;
    }
  } else {
    // ---- consumers: warp w takes keys 16 w .. + 15 of each tile, for all rows
    const int gq = lane >> 2, c = lane & 3;
    uint32_t stage = 0, phase = 0, used = 0;
    bool ok = true;
    for (int item = 0; ok && walk.step(a); ++item) {
      float(*warp_m)[RT] = warp_m2[item & 1];
      float(*warp_z)[RT] = warp_z2[item & 1];
      float(*warp_l)[RT] = warp_l2[item & 1];
      const int rows = g.s.n * a.group, pos0 = g.s.len - g.s.n;
      const int lo = g.lo, hi = g.hi, tile1 = g.tile1;
      // positions of the tile's first and last row
      const int pos_first = pos0 + kv_token(a, g.rt * RT), pos_last = pos0 + kv_token(a, min(rows, (g.rt + 1) * RT) - 1);
      // Query rows 8 t + gq, dimensions D/4 c .. + D/4 - 1: the second operand
      // of K Q^T.  In shared memory all warps read one copy.
      uint32_t q[S::kSharedQuery ? 1 : NT][D / 8];
      int pos[NT][2];       // positions of rows 8 t + 2 c, + 1: those of this thread's scores
      float rowfac[NT][2];  // 2^eq and the power of two of sm_scale log2(e)
      float m[NT][2], l[NT][2];
      if (S::kSharedQuery) named_sync(1, kT);  // the last item's sums have been read
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int r = g.rt * RT + 8 * t + gq, tok = kv_token(a, r);
        float amax = 0.f;
        uint4 v[D / 32];
        const uint16_t* src = a.q + static_cast<int64_t>(g.s.t0 + tok) * a.q_tok + (g.head * a.group + r - tok * a.group) * a.q_head + c * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          v[i] = r < rows ? *reinterpret_cast<const uint4*>(src + 8 * i) : make_uint4(0, 0, 0, 0);
          uint32_t x = 0;
          x = elem_absmax2<F16>(elem_absmax2<F16>(elem_absmax2<F16>(elem_absmax2<F16>(x, v[i].x), v[i].y), v[i].z), v[i].w);
          amax = fmaxf(amax, elem_absmax_final<F16>(x));
        }
        amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
        const int eq = kv_query_exp(amax);
        const float f = pow2f(-eq), rf = a.scale_pow * pow2f(eq);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
          const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
          uint32_t x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 y = elem2_to_f32x2<F16>(w[j]);
            x[j] = f32x2_to_elem2<true>(y.x * f, y.y * f);
            if constexpr (!S::kSharedQuery) q[t][4 * i + j] = x[j];
          }
          if constexpr (S::kSharedQuery)  // every warp stores the same values' quarter
            if (warp == t) query[(t * (D / 32) + i) * 32 + lane] = make_uint4(x[0], x[1], x[2], x[3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          rowfac[t][h] = __shfl_sync(~0u, rf, 4 * (2 * c + h));
          pos[t][h] = pos0 + kv_token(a, g.rt * RT + 8 * t + 2 * c + h);
          m[t][h] = -INFINITY;
          l[t][h] = 0.f;
        }
      }
      if (S::kSharedQuery) named_sync(1, kT);
      // O^T: dimensions D/8 gq + 2 i (elements 0, 1) and + 1 (2, 3), rows 8 t + 2 c (0, 2) and + 1 (1, 3)
      float o[NT][D / 16][4];
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int i = 0; i < D / 16; ++i) o[t][i][0] = o[t][i][1] = o[t][i][2] = o[t][i][3] = 0.f;

      int tile = g.tile0;
      // The tiles from `tile` on; without kWild up to the first page that wants z to be the scores' own (in warp_z).
      // A loop of its own: in one with them the other tiles took 3 to 14 % longer (64 contexts to 8192, 16 and 32 rows).
      const auto walk_tiles = [&](auto wild_tag) {
        constexpr bool kWild = decltype(wild_tag)::value;
        for (; tile < tile1; ++tile) {
          ok = __all_sync(~0u, mbar_wait_clocked(&full_bar[stage], phase, &abort_flag));
          if (!ok) break;
          const uint8_t* kd = smem + stage * 2 * S::kTileBytes;
          const uint8_t* vd = kd + S::kTileBytes;
          const KvPageScale ps = page_scale[stage][(16 * warp) >> min(a.page_shift, 6)];
          // S^T: keys gq (elements 0, 1) and gq + 8 (2, 3), rows 2 c (0, 2) and + 1 (1, 3); two chains of products
          float s[NT][4], s2[NT][4];
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[t][i] = s2[t][i] = 0.f;
#pragma unroll
          for (int j = 0; j < kQuads; ++j) {
            const uint4 u = *reinterpret_cast<const uint4*>(kd + kv_chunk<D>(16 * warp + gq, kQuads * c + j));
            const uint4 w = *reinterpret_cast<const uint4*>(kd + kv_chunk<D>(16 * warp + 8 + gq, kQuads * c + j));
            const uint32_t x[4] = {u.x, u.y, u.z, u.w}, y[4] = {w.x, w.y, w.z, w.w};
            [[maybe_unused]] uint4 qv[S::kSharedQuery ? NT : 1][2];
            if constexpr (S::kSharedQuery) {
#pragma unroll
              for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int i = 0; i < 2; ++i) qv[t][i] = query[(t * (D / 32) + 2 * j + i) * 32 + lane];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // K slice: dimensions D/4 c + 16 j + 4 i .. + 3
              const uint32_t a0 = e4m3x2_to_f16x2(x[i] & 0xFFFFu), a1 = e4m3x2_to_f16x2(y[i] & 0xFFFFu);
              const uint32_t a2 = e4m3x2_to_f16x2(x[i] >> 16), a3 = e4m3x2_to_f16x2(y[i] >> 16);
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                uint32_t b0, b1;
                if constexpr (S::kSharedQuery) {
                  const uint4 z = qv[t][i >> 1];
                  b0 = i & 1 ? z.z : z.x;
                  b1 = i & 1 ? z.w : z.y;
                } else {
                  b0 = q[t][8 * j + 2 * i];
                  b1 = q[t][8 * j + 2 * i + 1];
                }
                if (i & 1) kv_mma(s2[t], a0, a1, a2, a3, b0, b1);
                else kv_mma(s[t], a0, a1, a2, a3, b0, b1);
              }
            }
          }
          const int key0 = tile * kKvTile + 16 * warp;
          // keys that not all rows see, or none: only tiles at the range's ends
          const bool masked = kv_special(ps) || key0 < lo || key0 + 16 > hi || (a.causal && key0 + 15 > pos_first) ||
                              (a.window > 0 && key0 <= pos_last - a.window);
          // two copies of the rest, so that the tiles in between carry no masks
          const auto rest = [&](auto edge) {
            float top[NT][2];
            bool raise = false;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int h = i & 1;
                float x = (s[t][i] + s2[t][i]) * kv_score_factor(rowfac[t][h], ps.kfac) + ps.ev;
                if constexpr (decltype(edge)::value) {
                  const int key = key0 + gq + 8 * (i >> 1);
                  const bool see = ps.inv != 0.f && key >= lo && key < hi && (!a.causal || key <= pos[t][h]) &&
                                   (a.window <= 0 || key > pos[t][h] - a.window);
                  x = see ? x : -INFINITY;
                }
                s[t][i] = x;
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float x = fmaxf(s[t][h], s[t][2 + h]);
                x = fmaxf(x, __shfl_xor_sync(~0u, x, 4));
                x = fmaxf(x, __shfl_xor_sync(~0u, x, 8));
                x = fmaxf(x, __shfl_xor_sync(~0u, x, 16));
                top[t][h] = x;
                raise |= x > m[t][h] + kKvLag;
              }
            }
            if constexpr (kWild) {
              __syncwarp();
#pragma unroll
              for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float z = warp_z[warp][8 * t + 2 * c + h], zn = fmaxf(z, top[t][h] - ps.ev), z0 = zn == -INFINITY ? 0.f : zn;
                  l[t][h] = l[t][h] * fast_exp2(z - z0) + fast_exp2(s[t][h] - ps.ev - z0) + fast_exp2(s[t][2 + h] - ps.ev - z0);
                  __syncwarp();
                  if (gq == 0) warp_z[warp][8 * t + 2 * c + h] = zn;
                }
              }
            }
            if (__any_sync(~0u, raise)) {
#pragma unroll
              for (int t = 0; t < NT; ++t) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float mn = fmaxf(m[t][h], top[t][h] - kKvAbove);
                  const float f = m[t][h] == -INFINITY ? 0.f : fast_exp2(m[t][h] - mn);
                  m[t][h] = mn;
                  if constexpr (!kWild) l[t][h] *= f;
#pragma unroll
                  for (int i = 0; i < D / 16; ++i) {
                    o[t][i][h] *= f;
                    o[t][i][2 + h] *= f;
                  }
                }
              }
            }
            // P^T as the second operand: pairs of rows to pairs of keys
            uint32_t p[NT][2];
#pragma unroll
            for (int t = 0; t < NT; ++t) {
              const float m0 = m[t][0] == -INFINITY ? 0.f : m[t][0], m1 = m[t][1] == -INFINITY ? 0.f : m[t][1];
              const float x0 = fast_exp2(s[t][0] - m0), x1 = fast_exp2(s[t][1] - m1);
              const float x2 = fast_exp2(s[t][2] - m0), x3 = fast_exp2(s[t][3] - m1);
              if constexpr (!kWild) {
                l[t][0] += (x0 + x2) * ps.inv;
                l[t][1] += (x1 + x3) * ps.inv;
              }
              p[t][0] = kv_transpose(f32x2_to_elem2<true>(x0, x1));
              p[t][1] = kv_transpose(f32x2_to_elem2<true>(x2, x3));
            }
            // values: keys 2c, 2c + 1 and 8 + 2c, 9 + 2c; this thread's dimensions D/8 gq ..
            uint32_t vw[4][D / 32];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int r = 16 * warp + 8 * (k >> 1) + 2 * c + (k & 1);
              if constexpr (D == 128) {
                const uint4 w = *reinterpret_cast<const uint4*>(vd + kv_chunk<D>(r, gq));
                vw[k][0] = w.x; vw[k][1] = w.y; vw[k][2] = w.z; vw[k][3] = w.w;
              } else {
                const uint2 w = *reinterpret_cast<const uint2*>(vd + kv_chunk<D>(r, gq >> 1) + 8 * (gq & 1));
                vw[k][0] = w.x; vw[k][1] = w.y;
              }
              if constexpr (decltype(edge)::value) {  // whatever lies outside the allowed keys (NaN codes too) counts as zero
                const int key = tile * kKvTile + r;
                if (key < lo || key >= hi || ps.inv == 0.f) {
#pragma unroll
                  for (int i = 0; i < D / 32; ++i) vw[k][i] = 0u;
                }
              }
            }
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
              uint32_t lo[4], hi[4];
              kv_pairs(vw[0][i], vw[1][i], lo);
              kv_pairs(vw[2][i], vw[3][i], hi);
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                kv_mma(o[t][2 * i], lo[0], lo[1], hi[0], hi[1], p[t][0], p[t][1]);
                kv_mma(o[t][2 * i + 1], lo[2], lo[3], hi[2], hi[3], p[t][0], p[t][1]);
              }
            }
          };
          if constexpr (kWild) {
            rest(std::true_type{});
          } else {
            if (masked) {
              if (fabsf(ps.ev) > kKvTameExp) break;
              rest(std::true_type{});
            } else {
              rest(std::false_type{});
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty_bar[stage]);
          ++used;
          if (++stage == S::kStages) { stage = 0; phase ^= 1u; }
        }
      };
      walk_tiles(std::false_type{});
      const bool wild = ok && tile < tile1;
      if (wild) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            if (gq == 0) warp_z[warp][8 * t + 2 * c + h] = m[t][h];
        walk_tiles(std::true_type{});
      }
      if (!ok && lane == 0) {
        if (abort_flag == 0u) record_error_at(a.err, kErrTimeout);
        abort_flag = 1u;
      }
      // ---- the item's share: the four warps' keys meet
#pragma unroll
      for (int t = 0; t < NT; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int d = 4; d < 32; d <<= 1) l[t][h] += __shfl_xor_sync(~0u, l[t][h], d);
          if (gq == 0) {
            warp_m[warp][8 * t + 2 * c + h] = m[t][h];
            warp_l[warp][8 * t + 2 * c + h] = wild ? -l[t][h] : l[t][h];
          }
        }
      }
      named_sync(1, kT);
      const int live = min(RT, rows - g.rt * RT);  // rows of the tile
      const KvJoin team(start, g.first, g.count);
      if (tid == 0) go_on = abort_flag != 0u ? 0u : team.arrived_but_one(a) ? 2u : 1u;  // one answer for all warps
      // kTpr threads per row, float4s kTpr i + tid % kTpr of it
      constexpr int kTpr = kT / S::kPassRows, kOwn = D / 4 / kTpr;
      const int rl = tid / kTpr, d4 = tid % kTpr;
      const int head = team.head(), groups = team.groups();
      float* const to_group = groups > 1 ? team.part(a, head, S::kPartFloats) : nullptr;
      // Parts p0 to n - 1, of part i0 and every step-th after it, onto row r's sums.
      const auto add_parts = [&](int r, int i0, int step, int p0, int n, float4 (&acc)[kOwn], float& am, KvSum& below) {
        const float m0 = am;
        const KvSum before = below;
#pragma unroll(8 / kOwn)  // more in flight is more code to fetch: one short context 10.0 us, 11.0 with 16
        for (int p = p0; p < n; ++p) {
          const float* part = team.part(a, i0 + p * step, S::kPartFloats);
          float4 v[kOwn];
#pragma unroll
          for (int i = 0; i < kOwn; ++i) v[i] = __ldcg(reinterpret_cast<const float4*>(part + r * D) + kTpr * i + d4);
          const float pm = __ldcg(part + RT * D + r), pl = __ldcg(part + RT * D + RT + r);
          const float mm = fmaxf(am, pm);
          const float f0 = am == -INFINITY ? 0.f : fast_exp2(am - mm), f1 = pm == -INFINITY ? 0.f : fast_exp2(pm - mm);
#pragma unroll
          for (int i = 0; i < kOwn; ++i)
            acc[i] = make_float4(kv_add(acc[i].x, f0, v[i].x, f1), kv_add(acc[i].y, f0, v[i].y, f1),
                                 kv_add(acc[i].z, f0, v[i].z, f1), kv_add(acc[i].w, f0, v[i].w, f1));
          below.wild |= pl < 0.f;
          below.l = kv_add(below.l, f0, pl, f1);
          am = mm;
        }
        if (below.wild) {  // the sum again, with every z
          below = KvSum{};
          if (p0 > 0) below.add_wild(m0, before.stored(), before.z);
#pragma unroll 1
          for (int p = p0; p < n; ++p) {
            const float* part = team.part(a, i0 + p * step, S::kPartFloats) + RT * D + r;
            below.add_wild(__ldcg(part), __ldcg(part + RT), __ldcg(part + 2 * RT));
          }
        }
      };
      // Row r of the tile to a part, or where there is none to the output.
      const auto put = [&](int r, float4 (&acc)[kOwn], float am, const KvSum& below, float* part) {
        if (part != nullptr) {
#pragma unroll
          for (int i = 0; i < kOwn; ++i) __stcg(reinterpret_cast<float4*>(part + r * D) + kTpr * i + d4, acc[i]);
          if (d4 == 0) {
            __stcg(part + RT * D + r, am);
            __stcg(part + RT * D + RT + r, below.stored());
            if (below.wild) __stcg(part + RT * D + 2 * RT + r, below.z);
          }
          return;
        }
        const int rr = g.rt * RT + r;
        const int tok = kv_token(a, rr);
        const int64_t row = static_cast<int64_t>(g.s.t0 + tok) * a.heads + g.head * a.group + rr - tok * a.group;
        float f = below.l > 0.f ? 1.f / below.l : 0.f;
        if (below.wild) {  // 2^(m - z) in two steps: the whole may pass FP32 where the output does not
          const float half = fast_exp2(0.5f * (am - below.z));
          f *= half;
#pragma unroll
          for (int i = 0; i < kOwn; ++i) acc[i] = make_float4(acc[i].x * half, acc[i].y * half, acc[i].z * half, acc[i].w * half);
        }
#pragma unroll
        for (int i = 0; i < kOwn; ++i)
          *reinterpret_cast<uint2*>(a.out + row * D + 4 * (kTpr * i + d4)) =
              make_uint2(f32x2_to_elem2<F16>(acc[i].x * f, acc[i].y * f), f32x2_to_elem2<F16>(acc[i].z * f, acc[i].w * f));
        if (d4 == 0 && a.lse != nullptr) a.lse[row] = below.lse(am);
      };
#pragma unroll
      for (int pass = 0; pass < RT / S::kPassRows; ++pass) {
        if (pass > 0) named_sync(1, kT);  // the buffer has been read
        float* mw = merge + warp * S::kPassRows * S::kRow;
#pragma unroll
        for (int tt = 0; tt < S::kPassRows / 8; ++tt) {
          const int t = pass * (S::kPassRows / 8) + tt;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = 8 * t + 2 * c + h;
            float mm = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) mm = fmaxf(mm, warp_m[w][row]);
            const float f = m[t][h] == -INFINITY ? 0.f : fast_exp2(m[t][h] - mm);
            float* dst = mw + (8 * tt + 2 * c + h) * S::kRow + gq * S::kEighth;
#pragma unroll
            for (int i = 0; i < D / 16; i += 2)
              *reinterpret_cast<float4*>(dst + 2 * i) =
                  make_float4(o[t][i][h] * f, o[t][i][2 + h] * f, o[t][i + 1][h] * f, o[t][i + 1][2 + h] * f);
          }
        }
        named_sync(1, kT);
        ok = go_on != 0u;
        const bool direct = go_on == 2u;
        const int r = pass * S::kPassRows + rl;
        if (ok && r < live) {
          float4 acc[kOwn];
#pragma unroll
          for (int i = 0; i < kOwn; ++i) {
            const int d = 4 * (kTpr * i + d4);
            const float* src = merge + rl * S::kRow + d / (D / 8) * S::kEighth + d % (D / 8);
            constexpr int kWarpStride = S::kPassRows * S::kRow;
            const float4 x = *reinterpret_cast<const float4*>(src), y = *reinterpret_cast<const float4*>(src + kWarpStride);
            const float4 z = *reinterpret_cast<const float4*>(src + 2 * kWarpStride), w = *reinterpret_cast<const float4*>(src + 3 * kWarpStride);
            acc[i] = make_float4((x.x + y.x) + (z.x + w.x), (x.y + y.y) + (z.y + w.y), (x.z + y.z) + (z.z + w.z), (x.w + y.w) + (z.w + w.w));
          }
          KvSum below;
          float am = -INFINITY;
#pragma unroll
          for (int k = 0; k < 4; ++k) am = fmaxf(am, warp_m[k][r]);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float wm = warp_m[k][r], wl = warp_l[k][r];
            below.wild |= wl < 0.f;
            below.l += wl * (wm == -INFINITY ? 0.f : fast_exp2(wm - am));  // a NaN stays
          }
          if (below.wild) {  // the sum again, with every z
            below = KvSum{};
#pragma unroll 1
            for (int k = 0; k < 4; ++k) below.add_wild(warp_m[k][r], warp_l[k][r], warp_z[k][r]);
          }
          if (direct) add_parts(r, head, 1, 1, team.members(), acc, am, below);
          put(r, acc, am, below, direct ? to_group : team.count > 1 ? team.part(a, team.me, S::kPartFloats) : nullptr);
        }
      }
      if (ok && team.count > 1) {
#pragma unroll 1
        for (int level = go_on == 2u ? 1 : 0; level < (groups > 1 ? 2 : 1); ++level) {  // the group's parts, then the groups'
          const bool top = level == 1;
          const int n = top ? groups : team.members();
          if (!kv_arrive(top ? team.item_counter(a) : team.group_counter(a), n, 1, kT, tid == 0, &last)) break;
#pragma unroll 1
          for (int r = rl; r < RT; r += S::kPassRows) {
            const uint32_t mask = __ballot_sync(~0u, r < live);
            if (r >= live) continue;
            float4 acc[kOwn];
#pragma unroll
            for (int i = 0; i < kOwn; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            KvSum below;
            float am = -INFINITY;
            add_parts(r, top ? 0 : head, top ? team.join : 1, 0, n, acc, am, below);
            __syncwarp(mask);  // the row's threads, all in this warp, have read what put may replace
            put(r, acc, am, below, top ? nullptr : to_group);
          }
        }
      }
      // the merge buffer and the flags are written again only after the first
      // barrier of the next item's end, which all threads reach after this
    }
    if (tid == 0) used_tiles = used;
  }
  __syncthreads();
  // after an expired wait: loads that nothing consumed land before the block ends
  if (tid == 0 && abort_flag != 0u) a.arrived[kKvSpoiled] = 1u;
  if (tid == 0)
    for (uint32_t f = used_tiles; f < fills; ++f)
      if (!mbar_wait_clocked(&full_bar[f % S::kStages], (f / S::kStages) & 1u)) record_error_at(a.err, kErrTimeout);
}

}  // namespace bsq
