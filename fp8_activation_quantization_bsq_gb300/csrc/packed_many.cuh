// Products of many tokens with packed weights, on the tcgen05 tensor cores (the formula is packed_linear.cuh's).
//
// What bounds it: from about a hundred tokens on the products themselves, before that the stream of weights, or rather
// the codes' conversion, which keeps up with DRAM only just.  The weights are the 128-row operand and lie in tensor memory: a
// thread owns a row (a lane of tensor memory), reads its codes from shared memory, makes numbers of the tokens' type of them, times their scale,
// and stores them where the product reads them, so that weights cost shared memory half a byte or a byte per value, the tokens
// alone are read from there by the products, and nothing is converted twice.  Values are exact: E2M1 and E4M3 significands, and
// those of an E2M1 code times an E4M3 scale, fit BF16's 8 bits; with FP16 tokens so do NVFP4 values, and MX values are held
// relative to their row's largest scale, exact down to 2^-36 (E2M1) and 2^-21 (E4M3) of it, and off by at most 2^-35 (2^-23) of it below.
//
// Form.  A block takes MT (1, 2) tiles of 128 rows and up to 256 / MT tokens, K in steps of 128 columns: warp 0 streams codes and scales
// (one ring) and the tokens' columns (another) by TMA, warps 4-11 convert (with one tile the two groups of four take turns, with
// two each has its own), warp 1 issues the products, FP32 in tensor memory; the converters then store the tile.  One
// tile of 256 tokens asks shared memory for 64 bytes per clock and converts 16 weights per clock; two tiles of 128 would ask for as
// much and convert twice as many; for fewer tokens two tiles halve how often those are read.  Where rows are few, the blocks of a
// cluster share K and add their sums through distributed shared memory, in their order.
// All waits are bounded (about a second): an expired one records BSQ_ERR_TIMEOUT, stops the block's roles,
// waits for the copies and products in flight, frees the tensor memory and returns.
#pragma once

#include "cluster.cuh"
#include "packed_linear.cuh"
#include "tcgen05.cuh"

namespace bsq {

constexpr int kPmThreads = 384, kPmCols = 128;  // columns of a step
constexpr int kPmMaxStages = 12;

struct PmArgs {
  PlArgs p;
  int tokens_tile;        // of a block, a multiple of 16
  int row_tiles, token_tiles;
  int steps;              // of a row, in all
  int x_stages, w_stages, x_bytes, w_bytes;
  unsigned int* err;
};

// Rows of codes and scale atoms of a step and tile.
template <int FMT> struct PmFmt {
  static constexpr int kRowBytes = FMT == kMXFP8 ? 128 : 64;
  static constexpr int kTileBytes = 128 * kRowBytes;
  static constexpr int kAtoms = FMT == kNVFP4 ? 2 : 1;
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

// FP16 pairs that hold E2M1 or E4M3 values -> BF16 pairs of 2^-112 of them: the exponent's and the top mantissa bits move down by
// three (FP16's low mantissa bits are zero), the sign stays.
__device__ __forceinline__ uint32_t pm_f16_to_bf16(uint32_t h) { return (h & 0x80008000u) | ((h >> 3) & 0x0FFF0FFFu); }
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The factors of a row's step: NVFP4 eight, MX four, as pairs of the tokens' type; for BF16 2^112 times the scale (at most 2^127:
// what lies past that is a second factor).  `top`: with FP16 tokens and MX, the byte that stands for 2^13 (E2M1) or 2^7 (E4M3).
template <int FMT, bool F16>
__device__ __forceinline__ void pm_factors(const uint32_t (&word)[2], int top, uint32_t (&f)[8]) {
  if constexpr (FMT == kNVFP4) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t pair = e4m3x2_to_f16x2(word[i / 2] >> (16 * (i & 1)) & 0xFFFFu);
      if constexpr (F16) {
        f[2 * i] = __byte_perm(pair, 0, 0x1010);
        f[2 * i + 1] = __byte_perm(pair, 0, 0x3232);
      } else {
        const float2 s = f16x2_to_f32x2(pair);
        f[2 * i] = f32x2_to_elem2<false>(s.x * 0x1p112f, s.x * 0x1p112f);
        f[2 * i + 1] = f32x2_to_elem2<false>(s.y * 0x1p112f, s.y * 0x1p112f);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int byte = word[0] >> (8 * i) & 255u;
      uint32_t one;
      if constexpr (F16) {
        const int e = byte - top + (FMT == kMXFP8 ? 7 : 13);  // at most 13
        one = e >= -14 ? static_cast<uint32_t>(e + 15) << 10 : e >= -24 ? 1u << (e + 24) : 0u;
      } else {
        one = static_cast<uint32_t>(min(byte + 112, 254)) << 7;
      }
      f[i] = one | one << 16;
    }
  }
}

// MT: tiles of 128 rows that a block takes.
template <int FMT, bool F16, int MT>
__global__ void __launch_bounds__(kPmThreads, 1)
    packed_many_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x, const PmArgs a) {
  using F = PmFmt<FMT>;
  constexpr int kABufs = MT == 1 ? 4 : 2, kACol = 256, kABufCols = 64 * MT, kDCol = 128;  // tensor memory: D, second D, A
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  __shared__ uint64_t x_full[kPmMaxStages], x_empty[kPmMaxStages], w_full[kPmMaxStages], w_empty[kPmMaxStages];
  __shared__ uint64_t a_full[kABufs], a_empty[kABufs], d_full, d_empty, drain_bar;
  __shared__ uint32_t tmem_slot;
  __shared__ volatile uint32_t abort_flag, x_fills, w_fills;

  const int tid = threadIdx.x, warp = warp_index(), lane = tid & 31;
  const int ranks = gridDim.y;  // of the cluster
  uint8_t* const xs = smem;
  uint8_t* const ws = smem + a.x_stages * a.x_bytes;
  const int share = static_cast<int>((a.steps + ranks - 1) / ranks);
  const int k_lo = blockIdx.y * share, k_hi = min(k_lo + share, a.steps);
  const int n_tok = a.tokens_tile;
  if (tid == 0) {
    for (int i = 0; i < a.x_stages; ++i) {
      mbar_init(&x_full[i], 1);
      mbar_init(&x_empty[i], 1);
    }
    for (int i = 0; i < a.w_stages; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_empty[i], 4 * MT);
    }
    for (int i = 0; i < kABufs; ++i) {
      mbar_init(&a_full[i], 4 * MT);
      mbar_init(&a_empty[i], 1);
    }
    mbar_init(&d_full, 1);
    mbar_init(&d_empty, 8);
    mbar_init(&drain_bar, 1);
    abort_flag = 0u;
    x_fills = w_fills = 0u;
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
  const auto fail = [&]() {
    if (abort_flag == 0u) record_error_at(a.err, kErrTimeout);
    abort_flag = 1u;
  };

  if (warp == 0) {
    // ---- copies
    if (lane == 0) {
      uint32_t xn = 0, wn = 0;
      bool ok = true;
      for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x) {
        const int rt = tile % a.row_tiles, tt = tile / a.row_tiles;
        for (int k = k_lo; k < k_hi && ok; ++k) {
          const uint32_t s = wn % a.w_stages;
          ok = mbar_wait_clocked(&w_empty[s], (wn / a.w_stages & 1u) ^ 1u, &abort_flag);
          if (!ok) break;
          uint8_t* w = ws + s * a.w_bytes;
          const int atoms = min(F::kAtoms, a.p.k_atoms - k * F::kAtoms);
          const int bands = min(MT, static_cast<int>((a.p.rows - static_cast<int64_t>(rt) * MT * 128 + 127) / 128));
          mbar_arrive_expect_tx(&w_full[s], bands * (F::kTileBytes + atoms * 512));
          for (int m = 0; m < bands; ++m) {
            tma_load_2d(w + m * F::kTileBytes, &map_w, k * F::kRowBytes, (rt * MT + m) * 128, &w_full[s]);
            bulk_load(w + MT * F::kTileBytes + m * F::kAtoms * 512,
                      a.p.scales + (static_cast<int64_t>(rt * MT + m) * a.p.k_atoms + k * F::kAtoms) * 512, atoms * 512, &w_full[s]);
          }
          w_fills = ++wn;
          for (int h = 0; h < 2 && 2 * k * 64 + h * 64 < a.p.cols; ++h) {
            const uint32_t t = xn % a.x_stages;
            ok = mbar_wait_clocked(&x_empty[t], (xn / a.x_stages & 1u) ^ 1u, &abort_flag);
            if (!ok) break;
            mbar_arrive_expect_tx(&x_full[t], a.x_bytes);
            tma_load_2d(xs + t * a.x_bytes, &map_x, (2 * k + h) * 64, tt * n_tok, &x_full[t]);
            x_fills = ++xn;
          }
        }
      }
      if (!ok) fail();
    }
  } else if (warp == 1) {
    // ---- products
    const uint32_t lead = t5_elect();
    const uint32_t idesc = t5_idesc_f16(n_tok, false) | (F16 ? 0u : (1u << 7) | (1u << 10));
    const auto wait = [&](uint64_t* bar, uint32_t parity) { return __all_sync(~0u, mbar_wait_clocked(bar, parity, &abort_flag)); };
    uint32_t xn = 0, an = 0, done = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, ++done) {
      const int rt = tile % a.row_tiles;
      const bool two = MT == 2 && static_cast<int64_t>(rt * MT + 1) * 128 < a.p.rows;
      ok = wait(&d_empty, (done & 1u) ^ 1u);
      for (int k = k_lo; k < k_hi && ok; ++k, ++an) {
        const uint32_t b = an % kABufs;
        ok = wait(&a_full[b], an / kABufs & 1u);
        for (int h = 0; h < 2 && ok && (2 * k + h) * 64 < a.p.cols; ++h, ++xn) {
          const uint32_t t = xn % a.x_stages;
          ok = wait(&x_full[t], xn / a.x_stages & 1u);
          if (!ok) break;
          t5_fence_after();
          const uint64_t db = t5_desc_sw128(smem_addr(xs + t * a.x_bytes));
          const uint32_t acc = k > k_lo || h > 0;
          pm_mma64(tmem, tmem + kACol + b * kABufCols + 32 * h, db, idesc, acc, lead);
          if (two) pm_mma64(tmem + kDCol, tmem + kACol + b * kABufCols + 64 + 32 * h, db, idesc, acc, lead);
          t5_commit(smem_addr(&x_empty[t]), lead);
        }
        if (ok) t5_commit(smem_addr(&a_empty[b]), lead);
      }
      if (ok) t5_commit(smem_addr(&d_full), lead);
    }
    if (!ok && lane == 0) fail();
    t5_commit(smem_addr(&drain_bar), lead);
    if (!mbar_wait_clocked(&drain_bar, 0) && lane == 0) record_error_at(a.err, kErrTimeout);
  } else if (warp >= 4) {
    // ---- conversion, then the tile's output; a thread per row
    const int group = (warp - 4) >> 2, quarter = warp & 3, r = 32 * quarter + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * quarter) << 16);
    const float sf = FMT == kNVFP4 ? __ldg(a.p.sf) : 1.f;
    uint32_t n = 0, done = 0;
    bool ok = true;
    for (int tile = blockIdx.x; tile < tiles && ok; tile += gridDim.x, ++done) {
      const int rt = tile % a.row_tiles, tt = tile / a.row_tiles;
      const int m = MT == 2 ? group : 0;
      const int64_t band = static_cast<int64_t>(rt) * MT + m, row = band * 128 + r;
      const bool idle = band * 128 >= a.p.rows;  // the second tile lies behind the last row
      int top = 0;  // with FP16 tokens and MX: the row's largest scale byte
      if constexpr (F16 && FMT != kNVFP4) {
        if (!idle) {
          const uint8_t* s = a.p.scales + band * a.p.k_atoms * 512 + lane * 16 + quarter * 4;
          for (int k = k_lo; k < k_hi; ++k) {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(s + static_cast<int64_t>(k) * 512));
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (k * 128 + 32 * i < a.p.cols) top = max(top, static_cast<int>(w >> (8 * i) & 255u));
          }
        }
      }
      for (int k = k_lo; k < k_hi && ok; ++k, ++n) {
        if (MT == 1 && (n & 1u) != static_cast<uint32_t>(group)) continue;
        const uint32_t s = n % a.w_stages, b = n % kABufs;
        ok = __all_sync(~0u, mbar_wait_clocked(&w_full[s], n / a.w_stages & 1u, &abort_flag) &&
                                 mbar_wait_clocked(&a_empty[b], (n / kABufs & 1u) ^ 1u, &abort_flag));
        if (!ok) break;
        t5_fence_after();
        if (!idle) {
          const uint8_t* w = ws + s * a.w_bytes + m * F::kTileBytes + r * F::kRowBytes;
          const uint8_t* sc = ws + s * a.w_bytes + MT * F::kTileBytes + m * F::kAtoms * 512 + lane * 16 + quarter * 4;
          uint32_t word[2] = {*reinterpret_cast<const uint32_t*>(sc), 0u};
          if (FMT == kNVFP4 && k * 128 + 64 < a.p.cols) word[1] = *reinterpret_cast<const uint32_t*>(sc + 512);
          uint32_t f[8];
          pm_factors<FMT, F16>(word, top, f);
          const uint32_t to = lanes + kACol + b * kABufCols + 64 * m;
          // past BF16's range (2^127 more than 2^-112): a second factor
          bool wide = false;
          if constexpr (!F16 && FMT != kNVFP4) {
#pragma unroll
            for (int i = 0; i < 4; ++i) wide |= (word[0] >> (8 * i) & 255u) > 142u;
            wide = __any_sync(~0u, wide);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {  // 32 columns each
            uint32_t v[16];
            if constexpr (FMT == kMXFP8) {
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                const uint4 x = *reinterpret_cast<const uint4*>(w + (((2 * q + c) ^ (r & 7)) << 4));
                const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  v[8 * c + 2 * i] = e4m3x2_to_f16x2(u[i] & 0xFFFFu);
                  v[8 * c + 2 * i + 1] = e4m3x2_to_f16x2(u[i] >> 16);
                }
              }
            } else {
              const uint4 x = *reinterpret_cast<const uint4*>(w + ((q ^ ((r >> 1) & 3)) << 4));
              const uint32_t u[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t p[4];
                e2m1x8_to_f16(u[i], p);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[4 * i + j] = p[j];
              }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t g = FMT == kNVFP4 ? f[2 * q + i / 8] : f[q];
              v[i] = F16 ? mul_f16x2(v[i], g) : mul_bf16x2(pm_f16_to_bf16(v[i]), g);
            }
            if (!F16 && FMT != kNVFP4 && wide) {
              const int byte = word[0] >> (8 * q) & 255u;
              const uint32_t e = static_cast<uint32_t>(127 + max(byte + 112 - 254, 0)) << 7;
#pragma unroll
              for (int i = 0; i < 16; ++i) v[i] = mul_bf16x2(v[i], e | e << 16);
            }
            t5_st16(to + 16 * q, v);
          }
          t5_st_wait();
        }
        t5_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&w_empty[s]);
          mbar_arrive(&a_full[b]);
        }
      }
      // ---- output
      if (ok) ok = __all_sync(~0u, mbar_wait_clocked(&d_full, done & 1u, &abort_flag));
      if (!ok) break;
      t5_fence_after();
      const int tok0 = tt * n_tok, toks = min(n_tok, a.p.tokens - tok0);
      const float f = F16 && FMT != kNVFP4 ? pow2f(max(top, 1) - 127 - (FMT == kMXFP8 ? 7 : 13)) : 1.f;
      if (!idle) {
        for (int c0 = MT == 1 ? 32 * group : 0; c0 < n_tok; c0 += MT == 1 ? 64 : 32) {
          float y[32];
          t5_ld32(lanes + kDCol * m + c0, y);
          if (ranks > 1) {
            float* red = reinterpret_cast<float*>(smem);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (c0 + i < toks) red[(c0 + i) * (128 * MT) + 128 * m + r] = y[i] * f;
          } else if (row < a.p.rows) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (c0 + i >= toks) break;
              const int64_t tok = tok0 + c0 + i;
              float s = y[i] * f;
              if (FMT == kNVFP4) s = __fdiv_rn(s, sf);
              if (a.p.out_f32) {
                if (a.p.add) s += static_cast<const float*>(a.p.add)[tok * a.p.ld_add + row];
                static_cast<float*>(a.p.out)[tok * a.p.ld_out + row] = s;
              } else {
                if (a.p.add) s += elem2_to_f32x2<F16>(static_cast<const uint16_t*>(a.p.add)[tok * a.p.ld_add + row]).x;
                static_cast<uint16_t*>(a.p.out)[tok * a.p.ld_out + row] = static_cast<uint16_t>(f32x2_to_elem2<F16>(s, 0.f));
              }
            }
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
    for (uint32_t i = xf > static_cast<uint32_t>(a.x_stages) ? xf - a.x_stages : 0u; i < xf; ++i)
      if (!mbar_wait_clocked(&x_full[i % a.x_stages], i / a.x_stages & 1u)) record_error_at(a.err, kErrTimeout);
    for (uint32_t i = wf > static_cast<uint32_t>(a.w_stages) ? wf - a.w_stages : 0u; i < wf; ++i)
      if (!mbar_wait_clocked(&w_full[i % a.w_stages], i / a.w_stages & 1u)) record_error_at(a.err, kErrTimeout);
  }
  t5_fence_before();
  __syncthreads();
  t5_fence_after();
  if (warp == 1) {
    __syncwarp();
    t5_dealloc(tmem, 512);
  }
  if (ranks > 1) {  // one tile per cluster: every block's sums are in its shared memory
    cluster_sync_all();
    const int rt = blockIdx.x % a.row_tiles, tt = blockIdx.x / a.row_tiles;
    const int tok0 = tt * n_tok, toks = min(n_tok, a.p.tokens - tok0);
    const float* red = reinterpret_cast<const float*>(smem);
    const float sf = FMT == kNVFP4 ? __ldg(a.p.sf) : 1.f;
    const int me = blockIdx.y;
    for (int e = tid; e < 128 * MT * ((toks - me + ranks - 1) / ranks); e += kPmThreads) {
      const int t = me + e / (128 * MT) * ranks, r = e % (128 * MT);
      const int64_t row = static_cast<int64_t>(rt) * MT * 128 + r, tok = tok0 + t;
      if (row >= a.p.rows) continue;
      float s = 0.f;
      for (int q = 0; q < ranks; ++q) s += __uint_as_float(cluster_ld_u32(cluster_map(red + t * 128 * MT + r, q)));
      if (FMT == kNVFP4) s = __fdiv_rn(s, sf);
      if (a.p.out_f32) {
        if (a.p.add) s += static_cast<const float*>(a.p.add)[tok * a.p.ld_add + row];
        static_cast<float*>(a.p.out)[tok * a.p.ld_out + row] = s;
      } else {
        if (a.p.add) s += elem2_to_f32x2<F16>(static_cast<const uint16_t*>(a.p.add)[tok * a.p.ld_add + row]).x;
        static_cast<uint16_t*>(a.p.out)[tok * a.p.ld_out + row] = static_cast<uint16_t>(f32x2_to_elem2<F16>(s, 0.f));
      }
    }
    cluster_sync_all();  // no block leaves while another reads its sums
  }
}

}  // namespace bsq
