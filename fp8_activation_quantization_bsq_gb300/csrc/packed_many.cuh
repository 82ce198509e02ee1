// Products of many tokens with packed weights, on the tcgen05 tensor cores (the formula is packed_linear.cuh's).
//
// What bounds it: with many tokens the products; below about 128 the codes' conversion and the way that weights take into the
// products.  The weights are the 128-row operand and lie in tensor memory: a thread owns a row (a lane of tensor memory), reads its codes
// from shared memory, makes numbers of the tokens' type of them, times their scale, and stores them where the product reads them, so that
// weights cost shared memory half a byte or a byte per value, the tokens alone are read from there by the products, and nothing is
// converted twice within a block.  Values are exact: E2M1 and E4M3 significands, and those of an E2M1 code times an E4M3 scale, fit BF16's 8
// bits; with FP16 tokens so do NVFP4 values, and MX values are held relative to their row's largest scale, exact down to 2^-36 (E2M1) and
// 2^-21 (E4M3) of it, and off by at most 2^-35 (2^-23) of it below.
//
// Form.  A block takes MT (1, 2) tiles of 128 rows and up to 256 / MT tokens, K in steps of 64 columns: warp 0 copies the tokens' columns
// by TMA, a step at a time, warp 2 codes and scales, 128 bytes of each row at a time, warps 4-19 convert (groups of four, a warp per 32 rows,
// that take turns with the steps), warp 1 issues the products, FP32 in tensor memory; the converters then store the tile.  A step has one
// barrier for both its tokens and its weights.  Blocks of a cluster share K: each block adds a share of the tokens, whose sums the
// others write from tensor memory into its shared memory, in the blocks' order.  All waits are bounded (about a second): an expired one
// records BSQ_ERR_TIMEOUT, stops the block's roles, waits for the copies and products in flight, frees the tensor memory and returns.
//
// Measured (graph replay, BF16 tokens, NVFP4): 2048 tokens, 10240 x 7168 168 to 171 us (1.76 to 1.79 PFLOP/s; 1.91 measured of the library's plain
// BF16 product), tensor pipe 81 % active; 64 tokens, 7168 x 8192 21.3 us with inputs rotated through twice L2, and 19.5 through three sets, part of which
// stays there; of the latter, as the figures below, products start after 2.7 us, 26 steps take 10, and the sums 4.  From 129 to about 1000 tokens whole
// tiles in whole waves leave SMs idle: 300 tokens of 10240 x 7168 (240 tiles of 112 tokens on 152 SMs) take 56 us where their operations need 23, 512
// tokens 60 (39), 1000 tokens 93 (77).
// A product of 128 x N x 16 takes 64 cycles up to N = 128 and 133 at 256, for its 128-row operand's sake.  With FP16 tokens the 64 take
// 16.9 us, with codes that are not converted 15.7.  The cluster's sums go at about 10 bytes a clock and SM, read (20.6 us) or written (19.6), one or
// four values at a time (21.5).
#pragma once

#include "cluster.cuh"
#include "packed_linear.cuh"
#include "tcgen05.cuh"

namespace bsq {

constexpr int kPmConverters = 16;  // warps
constexpr int kPmThreads = 32 * (4 + kPmConverters);
constexpr int kPmMaxStages = 8;

struct PmArgs {
  PlArgs p;
  int tokens_tile;        // of a block, a multiple of 16
  int row_tiles, token_tiles;
  int share;              // of a block's part of K, in 128 columns
  int depth, w_stages, x_bytes, w_bytes;  // steps (tokens in shared, weights in tensor memory) and stages of weights in flight
  unsigned int* err;
};

// A stage of weights: 128 bytes of each row of a tile, and their scale atoms.  It is converted and multiplied in steps of 64
// columns.
template <int FMT> struct PmFmt {
  static constexpr int kCols = FMT == kMXFP8 ? 128 : 256, kSteps = kCols / 64;
  static constexpr int kTileBytes = 128 * 128;
  static constexpr int kAtoms = kCols / Fmt<FMT>::ATOM_COLS;
};

// D (128 x N, FP32) (+)= A B^T, K = 64: A from tensor memory (packed pairs, 8 columns per 16), B K-major with the 128-byte swizzle.
#define BSQ_PM_TS(AOFF, BOFF, ACC)                             \
  "add.u32 a, %1, " #AOFF ";\n\tadd.u64 b, %2, " #BOFF ";\n\t" \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, " ACC ";\n\t"
__device__ __forceinline__ void pm_mma64(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t lead) {
  asm volatile("{\n\t.reg .pred p, o, q;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.eq.b32 o, 0, 0;\n\t"
               BSQ_PM_TS(0, 0, "p") BSQ_PM_TS(8, 2, "o") BSQ_PM_TS(16, 4, "o") BSQ_PM_TS(24, 6, "o") "}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead) : "memory");
}
#undef BSQ_PM_TS

// An FP16 pair times f -> a BF16 pair, by way of FP32 (exact for codes times scales).  Conversions and packed products use pipes of
// their own: 38 codes a clock and SM; the same by shifts and masks of the FP16 bits 28, of the codes' bits 32.
__device__ __forceinline__ uint32_t pm_scaled_bf16(uint32_t h, float f) {
  float2 v = f16x2_to_f32x2(h);
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %2};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "+f"(v.x), "+f"(v.y)
      : "f"(f));
  return f32x2_to_elem2<false>(v.x, v.y);
}

// With FP16 tokens and MX, weights are held relative to their row's largest scale, which becomes 2^this: the largest codes then fit FP16.
template <int FMT> constexpr int kPmTop = FMT == kMXFP8 ? 7 : 13;

// The factors of a row's step: NVFP4 four, from `word`'s bytes, MX two, from its bytes at `at` and behind, as FP16 pairs or FP32
// numbers.  `top`: with FP16 tokens and MX, the byte that stands for 2^kPmTop.
template <int FMT, bool F16>
__device__ __forceinline__ void pm_factors(uint32_t word, int at, int top, uint32_t (&f)[4]) {
  if constexpr (FMT == kNVFP4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t pair = e4m3x2_to_f16x2(word >> (16 * i) & 0xFFFFu);
      if constexpr (F16) {
        f[2 * i] = __byte_perm(pair, 0, 0x1010);
        f[2 * i + 1] = __byte_perm(pair, 0, 0x3232);
      } else {
        const float2 s = f16x2_to_f32x2(pair);
        f[2 * i] = __float_as_uint(s.x);
        f[2 * i + 1] = __float_as_uint(s.y);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t byte = word >> (8 * (at + i)) & 255u;
      if constexpr (F16) {
        const int e = static_cast<int>(byte) - top + kPmTop<FMT>;  // at most 13
        const uint32_t one = e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
        f[i] = one | one << 16;
      } else {
        f[i] = max(byte << 23, 0x00400000u);  // byte 0 is 2^-127
      }
    }
  }
}

// The codes of 32 columns of a row of 128 bytes, as FP16: one 16-byte piece of E2M1 (piece c), two of E4M3 (2 c and 2 c + 1).
// The pieces lie where the 128-byte swizzle puts them (swz: row mod 8).
template <int FMT>
__device__ __forceinline__ void pm_codes(const uint8_t* row, int c, int swz, uint32_t (&v)[16]) {
  if constexpr (FMT == kMXFP8) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint4 x = *reinterpret_cast<const uint4*>(row + (((2 * c + p) ^ swz) << 4));
      const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[8 * p + 2 * i] = e4m3x2_to_f16x2(u[i] & 0xFFFFu);
        v[8 * p + 2 * i + 1] = e4m3x2_to_f16x2(u[i] >> 16);
      }
    }
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(row + ((c ^ swz) << 4));
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t p[4];
      e2m1x8_to_f16(u[i], p);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[4 * i + j] = p[j];
    }
  }
}

// One row's values of up to 32 tokens: times f, plus add where there is one, to rows `ld` apart.
template <bool F16, typename T>
__device__ __forceinline__ void pm_store(const float (&y)[32], float f, int n, T* out, int64_t ld, const T* add, int64_t ld_add) {
#pragma unroll
  for (int i0 = 0; i0 < 32; i0 += 8) {
    T x[8];
    if (add != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i0 + i < n) {
          x[i] = *add;
          add += ld_add;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (i0 + i >= n) return;
      float s = y[i0 + i] * f;
      if constexpr (sizeof(T) == 4) {
        if (add != nullptr) s += x[i];
        *out = s;
      } else {
        if (add != nullptr) s += elem2_to_f32x2<F16>(x[i]).x;
        *out = static_cast<uint16_t>(f32x2_to_elem2<F16>(s, 0.f));
      }
      out += ld;
    }
  }
}

// Four neighbouring values of the output's type, as far as `left` of them are there, at once where they are aligned.
template <bool F16>
__device__ __forceinline__ void pm_load4(const void* base, int f32, int64_t at, int64_t left, float4& v) {
  float* x = &v.x;
  if (f32) {
    const float* p = static_cast<const float*>(base) + at;
    if (left >= 4 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
      v = *reinterpret_cast<const float4*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) x[i] = p[i];
    }
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(base) + at;
    if (left >= 4 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
      const uint2 w = *reinterpret_cast<const uint2*>(p);
      const float2 lo = elem2_to_f32x2<F16>(w.x), hi = elem2_to_f32x2<F16>(w.y);
      v = make_float4(lo.x, lo.y, hi.x, hi.y);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) x[i] = elem2_to_f32x2<F16>(p[i]).x;
    }
  }
}
template <bool F16>
__device__ __forceinline__ void pm_store4(void* base, int f32, int64_t at, int64_t left, float4 v) {
  const float* x = &v.x;
  if (f32) {
    float* p = static_cast<float*>(base) + at;
    if (left >= 4 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
      *reinterpret_cast<float4*>(p) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = x[i];
    }
  } else {
    uint16_t* p = static_cast<uint16_t*>(base) + at;
    const uint2 w = make_uint2(f32x2_to_elem2<F16>(v.x, v.y), f32x2_to_elem2<F16>(v.z, v.w));
    if (left >= 4 && (reinterpret_cast<uintptr_t>(p) & 7u) == 0) {
      *reinterpret_cast<uint2*>(p) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < left) p[i] = static_cast<uint16_t>((i < 2 ? w.x : w.y) >> (16 * (i & 1)));
    }
  }
}

// MT: tiles of 128 rows that a block takes.
template <int FMT, bool F16, int MT>
__global__ void __launch_bounds__(kPmThreads, 1)
    packed_many_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const PmArgs a) {
  using F = PmFmt<FMT>;
  // tensor memory: the tiles' sums, then the weights of `depth` steps, 32 columns per tile
  constexpr uint32_t kBufCols = 32 * MT;
  const uint32_t d_col = a.tokens_tile <= 64 ? 64 : 128, a_col = MT == 1 ? 256 : 2 * d_col, depth = a.depth;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  // a step is full when its tokens have landed and its weights are converted: one wait and one commit of the products' warp, whose
  // own instructions would otherwise take longer than the products (two waits and commits a step: 236 us for 2048 tokens)
  __shared__ uint64_t full[kPmMaxStages], empty[kPmMaxStages], w_full[kPmMaxStages], w_empty[kPmMaxStages], d_full, d_empty, drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag, x_fills, w_fills, converted[kPmConverters];  // steps of each warp

  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const int ranks = gridDim.y;  // of the cluster
  uint8_t* const xs = smem;
  uint8_t* const ws = smem + depth * a.x_bytes;
  const int col0 = blockIdx.y * a.share * 128, cols = min(a.share * 128, a.p.cols - col0);  // of the block's part of K
  const int steps = (cols + 63) / 64, stages = (cols + F::kCols - 1) / F::kCols;
  const int n_tok = a.tokens_tile;
  if (tid == 0) {
    for (uint32_t i = 0; i < depth; ++i) {
      mbar_init(&full[i], 4 * MT + 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < a.w_stages; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], kPmConverters);
    }
    mbar_init(&d_full, 1);
    mbar_init(&d_empty, kPmConverters);
    mbar_init(&drain_bar, 1);
    abort_flag = 0u;
    x_fills = w_fills = 0u;
    for (int i = 0; i < kPmConverters; ++i) converted[i] = 0u;
    fence_mbar_init();
    prefetch_tensormap(&map_w);
    prefetch_tensormap(&map_x);
  }
  pdl_wait();
  if (warp == 1) t5_alloc(&tmem_slot, 512);
  t5_fence_before();
  __syncthreads();
  t5_fence_after();
  const uint32_t tmem = warp_uniform(static_cast<int>(tmem_slot));
  const int tiles = a.row_tiles * a.token_tiles;
  float row_factor = 1.f;  // a converter's row, in the end
  const auto fail = [&]() {
    if (abort_flag == 0u) record_error_at(a.err, kErrTimeout);
    abort_flag = 1u;
  };

  if (warp == 2) {
    // ---- copies of weights
    if (lane == 0) {
      uint32_t n = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        const int band0 = tile / a.token_tiles * MT;
        const int bands = min(MT, static_cast<int>((a.p.rows - static_cast<int64_t>(band0) * 128 + 127) / 128));
        for (int k = 0; k < stages; ++k) {
          const uint32_t s = n % a.w_stages;
          ok = mbar_wait_clocked(&w_empty[s], (n / a.w_stages & 1u) ^ 1u, &abort_flag);
          if (!ok) break;
          uint8_t* w = ws + s * a.w_bytes;
          const int atom0 = col0 / Fmt<FMT>::ATOM_COLS + k * F::kAtoms, atoms = min(F::kAtoms, a.p.k_atoms - atom0);
          mbar_arrive_expect_tx(&w_full[s], bands * (F::kTileBytes + atoms * 512));
          for (int m = 0; m < bands; ++m) {
            tma_load_2d(w + m * F::kTileBytes, &map_w, col0 / (F::kCols / 128) + k * 128, (band0 + m) * 128, &w_full[s]);
            bulk_load(w + MT * F::kTileBytes + m * F::kAtoms * 512,
                      a.p.scales + (static_cast<int64_t>(band0 + m) * a.p.k_atoms + atom0) * 512, atoms * 512, &w_full[s]);
          }
          w_fills = ++n;
        }
      }
      if (!ok) fail();
    }
  } else if (warp == 0) {
    // ---- copies of tokens
    if (lane == 0) {
      uint32_t n = 0, b = 0, parity = 1;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        const int y = tile % a.token_tiles * n_tok;
        for (int h = 0; h < steps; ++h) {
          ok = mbar_wait_clocked(&empty[b], parity, &abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(&full[b], a.x_bytes);
          tma_load_2d(xs + b * a.x_bytes, &map_x, col0 + h * 64, y, &full[b]);
          x_fills = ++n;
          if (++b == depth) { b = 0; parity ^= 1u; }
        }
      }
      if (!ok) fail();
    }
  } else if (warp == 1) {
    // ---- products
    const uint32_t lead = t5_elect();
    const uint32_t idesc = t5_idesc_f16(n_tok, false) | (F16 ? 0u : (1u << 7) | (1u << 10));
    const auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(~0u, mbar_wait_clocked(bar, parity, &abort_flag)); };
    const uint64_t x_desc = t5_desc_sw128(smem_addr(xs));
    const uint32_t x_step = a.x_bytes >> 4;
    uint32_t b = 0, parity = 0, done = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, ++done) {
      const bool two = MT == 2 && static_cast<int64_t>(tile / a.token_tiles * MT + 1) * 128 < a.p.rows;
      ok = wait(&d_empty, (done & 1u) ^ 1u);
      for (int h = 0; h < steps; ++h) {
        ok = ok && wait(&full[b], parity);
        if (!ok) break;
        t5_fence_after();
        const uint64_t db = x_desc + b * x_step;
        const uint32_t ta = tmem + a_col + b * kBufCols;
        pm_mma64(tmem, ta, db, idesc, h > 0, lead);
        if (two) pm_mma64(tmem + d_col, ta + 32, db, idesc, h > 0, lead);
        t5_commit(smem_addr(&empty[b]), lead);
        if (++b == depth) { b = 0; parity ^= 1u; }
      }
      if (ok) t5_commit(smem_addr(&d_full), lead);
    }
    if (!ok && lane == 0) fail();
    t5_commit(smem_addr(&drain_bar), lead);
    if (!mbar_wait_clocked(&drain_bar, 0) && lane == 0) record_error_at(a.err, kErrTimeout);
  } else if (warp >= 4) {
    // ---- conversion, then the tile's output; a thread per row
    // the groups of four warps of a tile take turns with its steps
    constexpr int kTurns = kPmConverters / 4 / MT;
    const int group = (warp - 4) >> 2, m = group / kTurns, turn = group % kTurns, quarter = warp & 3, r = 32 * quarter + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const float inv = FMT == kNVFP4 ? __fdiv_rn(1.f, __ldg(a.p.sf)) : 1.f;
    uint32_t wn = 0, done = 0, b = turn, parity = 1, next = turn;  // next: this group's next step, counted over all tiles
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, ++done) {
      const int rt = tile / a.token_tiles, tt = tile % a.token_tiles;
      const int64_t band = static_cast<int64_t>(rt) * MT + m, row = band * 128 + r;
      const bool idle = band * 128 >= a.p.rows;  // the second tile lies behind the last row
      // with FP16 tokens and MX: the row's largest scale byte, and no less than what lets the factor at the end be a number (2^-127); smaller
      // scales are then held below 2^13 (E2M1) or 2^7 (E4M3), exactly
      int top = kPmTop<FMT>;
      if constexpr (F16 && FMT != kNVFP4) {
        if (!idle) {
          const uint8_t* s = a.p.scales + band * a.p.k_atoms * 512 + lane * 16 + quarter * 4;
          for (int c = col0; c < col0 + steps * 64; c += 128) {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(s + static_cast<int64_t>(c / 128) * 512));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (c + 32 * i < a.p.cols) top = max(top, static_cast<int>(w >> (8 * i) & 255u));
          }
        }
      }
      for (int k = 0; k < stages && ok; ++k, ++wn) {
        const uint32_t s = wn % a.w_stages;
        // every group waits for and gives back every stage, converted by it or not: a barrier's parity tells only neighbouring
        // phases apart, so none may pass unseen
        ok = __all_sync(~0u, mbar_wait_clocked(&w_full[s], wn / a.w_stages & 1u, &abort_flag));
        const uint32_t base = done * steps, stop = base + min((k + 1) * F::kSteps, steps);
        while (ok && next < stop) {
          const int j = static_cast<int>(next - base) - k * F::kSteps;  // of the stage
          // unambiguous: `depth` is at least kTurns, so this group's last step knew the phase before
          ok = __all_sync(~0u, mbar_wait_clocked(&empty[b], parity, &abort_flag));
          if (!ok) break;
          t5_fence_after();
          if (!idle) {
            // 64 columns: NVFP4 a scale atom, MX half of one
            const int atom = FMT == kNVFP4 ? j : j / 2;
            const uint32_t word = *reinterpret_cast<const uint32_t*>(ws + s * a.w_bytes + MT * F::kTileBytes + (m * F::kAtoms + atom) * 512 +
                                                                     lane * 16 + quarter * 4);
            const uint8_t* w = ws + s * a.w_bytes + m * F::kTileBytes + r * 128;
            uint32_t f[4];
            pm_factors<FMT, F16>(word, 2 * (j & 1), top, f);
#pragma unroll
            for (int q = 0; q < 2; ++q) {  // 32 columns each
              uint32_t v[16];
              pm_codes<FMT>(w, 2 * j + q, r & 7, v);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const uint32_t g = FMT == kNVFP4 ? f[2 * q + i / 8] : f[q];
                v[i] = F16 ? mul_f16x2(v[i], g) : pm_scaled_bf16(v[i], __uint_as_float(g));
              }
              t5_st16(lanes + a_col + b * kBufCols + 32 * m + 16 * q, v);
            }
            t5_st_wait();
          }
          t5_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&full[b]);
            converted[warp - 4] = next / kTurns + 1u;
          }
          next += kTurns;
          b += kTurns;
          if (b >= depth) { b -= depth; parity ^= 1u; }
        }
        if (ok && lane == 0) mbar_arrive(&w_empty[s]);
      }
      // ---- output
      if (ok) ok = __all_sync(~0u, mbar_wait_clocked(&d_full, done & 1u, &abort_flag));
      if (!ok) break;
      t5_fence_after();
      const int tok0 = tt * n_tok, toks = min(n_tok, a.p.tokens - tok0);
      const float f = F16 && FMT != kNVFP4 ? pow2f(top - 127 - kPmTop<FMT>) : inv;
      row_factor = f;
      if (!idle && ranks == 1) {
        for (int c0 = 32 * turn; c0 < toks; c0 += 32 * kTurns) {
          float y[32];
          t5_ld32(lanes + d_col * m + c0, y);
          const int n_out = min(32, toks - c0);
          if (row < a.p.rows) {
            const int64_t at = (tok0 + c0) * a.p.ld_out + row, add_at = (tok0 + c0) * a.p.ld_add + row;
            if (a.p.out_f32)
              pm_store<F16>(y, f, n_out, static_cast<float*>(a.p.out) + at, a.p.ld_out, a.p.add ? static_cast<const float*>(a.p.add) + add_at : nullptr, a.p.ld_add);
            else
              pm_store<F16>(y, f, n_out, static_cast<uint16_t*>(a.p.out) + at, a.p.ld_out,
                            a.p.add ? static_cast<const uint16_t*>(a.p.add) + add_at : nullptr, a.p.ld_add);
          }
          __syncwarp();
        }
      }
      t5_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_empty);
    }
    if (!ok && lane == 0) fail();
  }
  __syncthreads();
  // after an expired wait: loads that nothing consumed land before the block ends (the last fill of each stage)
  if (tid == 0 && abort_flag != 0u) {
    const uint32_t xf = x_fills, wf = w_fills;
    constexpr uint32_t kTurns = kPmConverters / 4 / MT;
    for (uint32_t i = xf > depth ? xf - depth : 0u; i < xf; ++i) {
      for (uint32_t w = 0; w < kPmConverters; ++w)  // in place of the converters that have not come to this step
        if (w / 4 % kTurns == i % kTurns && converted[w] <= i / kTurns) mbar_arrive(&full[i % depth]);
      if (!mbar_wait_clocked(&full[i % depth], i / depth & 1u)) record_error_at(a.err, kErrTimeout);
    }
    for (uint32_t i = wf > static_cast<uint32_t>(a.w_stages) ? wf - a.w_stages : 0u; i < wf; ++i)
      if (!mbar_wait_clocked(&w_full[i % a.w_stages], i / a.w_stages & 1u)) record_error_at(a.err, kErrTimeout);
  }
  t5_fence_before();
  __syncthreads();
  t5_fence_after();
  if (ranks > 1) {
    // One tile per cluster.  Block q gets tokens q n .. of all blocks' sums, written from tensor memory straight into its shared
    // memory, [block][token][row], once every block is done with its rings; then it adds them in the blocks' order.
    const int rt = blockIdx.x / a.token_tiles, tt = blockIdx.x % a.token_tiles, me = blockIdx.y;
    const int toks = min(n_tok, a.p.tokens - tt * n_tok), per = (toks + ranks - 1) / ranks, mine = max(0, min(per, toks - me * per));
    constexpr int kRows = 128 * MT, kQuads = kRows / 4, kTurns = kPmConverters / 4 / MT;
    cluster_sync_all();
    const int m = (warp - 4) / 4 / kTurns, turn = (warp - 4) / 4 % kTurns, quarter = warp & 3;
    if (warp >= 4 && abort_flag == 0u && (static_cast<int64_t>(rt) * MT + m) * 128 < a.p.rows) {
      for (int c0 = 32 * turn; c0 < toks; c0 += 32 * kTurns) {
        float y[32];
        t5_ld32(tmem + (static_cast<uint32_t>(32 * quarter) << 16) + d_col * m + c0, y);
        int owner = c0 / per, t = c0 - owner * per;
        const float* to = reinterpret_cast<const float*>(smem) + me * per * kRows + 128 * m + 32 * quarter + lane;
        uint32_t base = cluster_map(to, owner);
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          if (c0 + i >= toks) break;
          cluster_st_u32(base + t * (kRows * 4), __float_as_uint(y[i] * row_factor));
          if (++t == per && c0 + i + 1 < toks) {
            t = 0;
            base = cluster_map(to, ++owner);
          }
        }
        __syncwarp();
      }
    }
    // the residuals of the first two items are on their way meanwhile: four rows of a token each
    const int items = kQuads * mine;
    const int64_t tok0 = static_cast<int64_t>(tt) * n_tok + me * per, row0 = static_cast<int64_t>(rt) * kRows;
    const auto residual = [&](int e) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (a.p.add && e < items) pm_load4<F16>(a.p.add, a.p.out_f32, (tok0 + e / kQuads) * a.p.ld_add + row0 + e % kQuads * 4, a.p.rows - row0 - e % kQuads * 4, x);
      return x;
    };
    float4 next[2] = {residual(tid), residual(tid + kPmThreads)};
    cluster_sync_all();
    const float4* sums = reinterpret_cast<const float4*>(smem);
    for (int e = tid; e < items; e += kPmThreads) {
      float4 v = sums[e];
      for (int q = 1; q < ranks; ++q) {
        const float4 x = sums[q * per * kQuads + e];
        v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
      }
      if (a.p.add) v.x += next[0].x, v.y += next[0].y, v.z += next[0].z, v.w += next[0].w;
      pm_store4<F16>(a.p.out, a.p.out_f32, (tok0 + e / kQuads) * a.p.ld_out + row0 + e % kQuads * 4, a.p.rows - row0 - e % kQuads * 4, v);
      next[0] = next[1];
      next[1] = residual(e + 2 * kPmThreads);
    }
    t5_fence_before();
    __syncthreads();
    t5_fence_after();
  }
  if (warp == 1) {
    __syncwarp();
    t5_dealloc(tmem, 512);
  }
}

}  // namespace bsq
