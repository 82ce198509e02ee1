// Products of a few tokens with packed weights: y[t][n] = sum_k x[t][k] c[n][k] s[n][k / b] / sf (+ add[t][n]), the
// weights as bsq_quantize packs them (codes c, 5D scales s), x in 16 bits as it is.
//
// What bounds it: the weights are read once, half a byte or a byte each, for 2 T operations, so for few tokens the kernel is a stream
// of weights from DRAM, and what is left to do per weight has to stay below what an SM can issue in the meantime (about 47
// four-bit weights per clock).  Codes become FP16 by one conversion per two (exact: E2M1 and E4M3 have at most 4 significand
// bits) and meet the tokens in mma.sync products with the weights on the 16-row side, so that 8 tokens are no padding.
// An NVFP4 scale multiplies the codes in FP16 (6 significand bits between 2^-10 and 2688: exact).  The 2^e of an MX format may lie
// outside FP16, so there a block of 32 columns is summed by itself, in FP32, and enters the row's sum times 2^e.
// BF16 tokens are scaled by a power of two, to a largest value just below 2^15, and then are exact in FP16 down to 2^-31 of that
// largest value; what lies below is off by at most 2^-39 of it.
//
// Form.  A warp takes 32 rows, 8 q + g + 32 j of a 128-row band (g < 8, j < 4), whose scales in the 5D layout are 16
// consecutive bytes per g, in pieces of 64 bytes per row; it streams them by asynchronous copies of
// 16 bytes through a ring of its own (no barrier: a warp reads what its own lanes copied), and ldmatrix hands a lane
// the 4 bytes of its row that the product's layout wants.  A block's 8 warps take 1 or 4 neighbouring sets of 32 rows (4 share the tokens'
// columns, which lie in shared memory as FP16) and share out K otherwise.  Blocks of a cluster share K too; the warps' sums
// are added in shared memory, the blocks' through the cluster's, in a fixed order.
//
// Measured (graph replay, inputs rotated through twice L2, of 6787 GB/s measured): one token of BF16, 10240 x 7168 NVFP4 11.9 us (3.5 TB/s), MXFP8
// 17.4 (4.4), 16000 x 8192 NVFP4 16.6 to 17.9 (4.1 to 4.5); 5 tokens, 1000 x 2912 MXFP4 3.9 us (3.3 from L2); 16 tokens, 256 x 7168 MXFP8 6.2.
// About 5 us of a call are its start, the tokens' way into shared memory and the sums.  The rest is not DRAM's rate but how the blocks divide over
// the SMs: each SM gets an equal share of that rate, and those with a block more end later (9728 x 7168, two blocks for each SM, takes 9.4 to 9.6 us,
// 5 % more rows 11.9; without its products that takes 10.95).  Every block copies, scans and converts its tokens' columns for at most 128 rows, so
// tokens cost as much as weights from about 16 on: 2, 4, 8, 12 and 16 tokens, 10240 x 7168, 12.5, 13.3, 15.4, 21.9 and 24.3 us.  A ring of 4 or 5
// pieces takes the room of a third block or of the next call's first ones: 9728 x 7168 12.3 and 12.7 us against 8.8.  A copy into L2 ahead of the
// launch's wait: 14.4 against 13.3.
#pragma once

#include "cluster.cuh"
#include "serving_common.cuh"

namespace bsq {

constexpr int kPlWarps = 8, kPlThreads = kPlWarps * 32, kPlRows = 32;
constexpr int kPlDepth = 3;                              // pieces in a warp's ring
constexpr int kPlSlot = kPlRows * 64 + 256;              // codes, then one or two scale atoms' 8 rows of 16 bytes
constexpr int kPlRing = kPlWarps * kPlDepth * kPlSlot;

struct PlArgs {
  const uint16_t* x;
  int64_t ld_x;
  const uint8_t* w;
  const uint8_t* scales;
  const float* sf;        // NVFP4
  const void* add;        // of the output's type, may be null
  int64_t ld_add;
  void* out;
  int64_t ld_out;
  int64_t rows;
  int tokens, cols;
  int pieces;             // of a row, in all
  int per_rank;           // of a block's share of K, a multiple of the warps that share K
  int segment;            // of the tokens' columns held at a time, the same
  int k_atoms;            // scale atoms per band
  int64_t row_bytes;
  int out_f32;
};

template <int FMT> struct PlFmt {
  static constexpr int kCols = FMT == kMXFP8 ? 64 : 128;  // columns of a piece
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Four E2M1 pairs, a byte each -> FP16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// One half (0 low, 1 high) of an FP16 pair, twice.
__device__ __forceinline__ uint32_t f16_twice(uint32_t pair, int half) {
  uint32_t r;
  if (half == 0)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}" : "=r"(r) : "r"(pair));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}" : "=r"(r) : "r"(pair));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 2^k that takes a largest magnitude (FP32 bits) to below 2^15; k from -113 to 127, or -114 for an infinity.
__device__ __forceinline__ int pl_exponent(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23) - 127;  // of an FP32 number, -127 below the normal ones
  return min(127, 14 - max(e, -127));
}
__device__ __forceinline__ float pl_pow2(int k) { return pow2f(min(k, 127)); }
// The factor 2^(byte - 127) of an MX block's sum; for BF16 tokens 2^-14 of it (still exact, subnormal at the least), so that
// sums are of tokens with a largest value between 1 and 2 and pass FP32 no earlier than those.
template <bool F16>
__device__ __forceinline__ float pl_mx_factor(uint32_t word, int byte) {
  const float f = __uint_as_float(max((word >> (8 * byte) & 255u) << 23, 0x00400000u));
  return F16 ? f : f * 0x1p-14f;
}

// NT: tiles of 8 tokens, RT: sets of 32 rows that a block takes.
template <int FMT, bool F16, int NT, int RT>
__global__ void __launch_bounds__(kPlThreads, NT == 1 ? 3 : 2) packed_linear_kernel(const PlArgs a) {
  constexpr int kCols = PlFmt<FMT>::kCols;
  constexpr int kTile = NT * 8, kSplit = kPlWarps / RT;  // warps along K
  extern __shared__ __align__(1024) uint8_t pl_smem[];
  __shared__ uint32_t amax_of[kTile];
  __shared__ int exp_of[kTile];  // the power of two that the tokens are held times
  __shared__ __align__(16) uint8_t zeros[256];
  uint8_t* xs = pl_smem + kPlRing;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x, ranks = gridDim.x;  // blocks of a cluster, along K
  const int part = warp % kSplit;                  // of K
  const int64_t tile = static_cast<int64_t>(blockIdx.y) * RT + warp / kSplit;  // 32 rows
  const int64_t row0 = (tile >> 2) * 128 + (tile & 3) * 8;
  const int toks = a.tokens;  // at most kTile
  const int p_lo = rank * a.per_rank, p_hi = min(p_lo + a.per_rank, a.pieces);
  const int x_stride = a.segment * kCols * 2 + 64;  // bytes of a token: 64 past a multiple of 128, for the banks

  // this lane's part of the copies: piece cp of row cr of every 8, from offsets to the block's first row; what lies behind
  // the last row or column is zeros
  const uint32_t ring = smem_addr(pl_smem) + warp * (kPlDepth * kPlSlot);
  const int cr = lane >> 2, cp = lane & 3;
  constexpr int kAtoms = FMT == kNVFP4 ? 2 : 1, kAtomPieces = FMT == kMXFP8 ? 2 : 1;  // atoms of a piece, pieces of an atom
  const uint8_t* const w0 = a.w + row0 * a.row_bytes;
  const uint8_t* const s0 = a.scales + ((tile >> 2) * a.k_atoms * 512 + (tile & 3) * 128);
  const uint32_t row_step = 32u * static_cast<uint32_t>(a.row_bytes);
  uint32_t byte = static_cast<uint32_t>(p_lo + part) * 64 + cp * 16, from = cr * static_cast<uint32_t>(a.row_bytes) + byte;
  const int rows_in = static_cast<int>(min(int64_t(128), a.rows - row0)) - cr;  // > 32 j: row j is there
  const int end_byte = min(p_hi * 64, static_cast<int>(a.row_bytes));
  const uint32_t to = (cr * 64) + ((cp ^ ((cr >> 1) & 3)) * 16);
  int atom = (p_lo + part) / kAtomPieces * kAtoms + (lane >> 3);  // lanes below 8 kAtoms copy a row of 16 scale bytes
  uint32_t fill = ring;
  const auto issue = [&]() {  // the warp's next piece
    const bool in = static_cast<int>(byte) < end_byte;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool there = in && rows_in > 32 * j;
      cp_async16(fill + to + 512 * j, w0 + (there ? from + j * row_step : 0u), there);
    }
    if (lane < 8 * kAtoms) {
      const bool there = atom < a.k_atoms;
      cp_async16(fill + kPlRows * 64 + lane * 16, s0 + (there ? static_cast<uint32_t>(atom) * 512u + (lane & 7) * 16 : 0u), there);
    }
    cp_async_commit();
    byte += kSplit * 64;
    from += kSplit * 64;
    atom += kSplit * kAtoms / kAtomPieces;
    fill = fill == ring + (kPlDepth - 1) * kPlSlot ? ring : fill + kPlSlot;
  };

  // a segment's tokens as they are, 8 columns per item (a multiple of 32 items per token, so a warp's are of one token);
  // columns past the last one are zeros.  A thread takes every 256th item.
  const int width = a.segment * kCols, groups = width / 8;
  const int tok_step = kPlThreads / groups, c_step = (kPlThreads - tok_step * groups) * 8;
  const int my_tok = tid / groups, my_c = (tid - my_tok * groups) * 8;
  const auto each_item = [&](auto&& f) {
    for (int tok = my_tok, c = my_c; tok < toks;) {
      f(tok, c);
      tok += tok_step;
      c += c_step;
      if (c >= width) {
        c -= width;
        ++tok;
      }
    }
  };
  const auto copy_tokens = [&](int seg) {
    const int col0 = seg * kCols, live = min(min(seg + a.segment, p_hi) * kCols, a.cols) - col0;
    const uint32_t dst = smem_addr(xs);
    const uint16_t* src = a.x + col0;
    each_item([&](int tok, int c) { cp_async16(dst + tok * x_stride + c * 2, src + (c < live ? tok * a.ld_x + c : 0), c < live); });
    cp_async_commit();
  };

  pdl_wait();
  copy_tokens(p_lo);
#pragma unroll
  for (int i = 0; i < kPlDepth - 1; ++i) issue();
  if (tid < kTile) exp_of[tid] = 127;
  if (tid < 16) *reinterpret_cast<uint4*>(zeros + 16 * tid) = make_uint4(0, 0, 0, 0);

  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][nt][i] = 0.f;

  // ldmatrix: lane's row address, without the piece's swizzled part
  const uint32_t lm_row = (8 * ((lane >> 3) & 1) + (lane & 7)) * 64, lm_x = ((lane & 7) >> 1) & 3, lm_p = lane >> 4;
  const uint32_t lm_0 = lm_row + ((lm_p ^ lm_x) * 16), lm_2 = lm_row + (((2 + lm_p) ^ lm_x) * 16);
  // an NVFP4 scale word's bytes for this lane's codes of two 16-byte columns: 8 codes lie in one block
  const uint32_t sel = (t >> 1) | ((2 + (t >> 1)) << 4);
  constexpr int kLaneBytes = FMT == kMXFP8 ? 8 : 16;  // of a token's values for a 16-byte column

  uint32_t read = ring;  // the slot that is next
  int piece = p_lo + part;
  for (int seg = p_lo; seg < p_hi; seg += a.segment) {
    const int seg_end = min(seg + a.segment, p_hi);
    if (tid < kTile) amax_of[tid] = 0u;
    if (seg == p_lo) {
      cp_async_wait<kPlDepth - 1>();
      __syncthreads();  // exp_of and amax_of are set
    } else {
      __syncthreads();  // the segment before has been read
      copy_tokens(seg);
      cp_async_wait<0>();
    }
    // their largest magnitude; then, BF16, as FP16 times the power of two that follows.  Each thread takes the items it copied
    if constexpr (!F16) {
      uint32_t m = 0;
      int of = my_tok;
      const auto flush = [&]() {
        const uint32_t top = __reduce_max_sync(~0u, __float_as_uint(absmax_final(m)));
        if (lane == 0 && of < toks) atomicMax(&amax_of[of], top);
        m = 0;
      };
      each_item([&](int tok, int c) {
        if (tok != of) {
          flush();
          of = tok;
        }
        const uint4 v = *reinterpret_cast<const uint4*>(xs + tok * x_stride + c * 2);
        m = absmax2(absmax2(absmax2(absmax2(m, v.x), v.y), v.z), v.w);
      });
      flush();
    }
    __syncthreads();
    if constexpr (!F16) {
      // sums so far follow to the new power of two, which never grows
      if (seg != p_lo) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int tok = nt * 8 + 2 * t + i;
            const int was = exp_of[tok], now = min(was, pl_exponent(amax_of[tok]));
            if (now != was) {
              const int d = max(now - was, -250), h = d / 2;
              const float f = pl_pow2(h), q = pl_pow2(d - h);
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                acc[m][nt][i] = acc[m][nt][i] * f * q;
                acc[m][nt][i + 2] = acc[m][nt][i + 2] * f * q;
              }
            }
          }
      }
      each_item([&](int tok, int c) {
        uint4* p = reinterpret_cast<uint4*>(xs + tok * x_stride + c * 2);
        uint4 v = *p;
        const float f = pl_pow2(min(exp_of[tok], pl_exponent(amax_of[tok])));
        v.x = f32x2_to_elem2<true>(bf16_lo(v.x) * f, bf16_hi(v.x) * f);
        v.y = f32x2_to_elem2<true>(bf16_lo(v.y) * f, bf16_hi(v.y) * f);
        v.z = f32x2_to_elem2<true>(bf16_lo(v.z) * f, bf16_hi(v.z) * f);
        v.w = f32x2_to_elem2<true>(bf16_lo(v.w) * f, bf16_hi(v.w) * f);
        *p = v;
      });
      __syncthreads();
      if (tid < kTile) exp_of[tid] = min(exp_of[tid], pl_exponent(amax_of[tid]));
    }

    // a lane's token, or zeros (256 bytes of them) for tokens that are not there
    const uint8_t* xp[NT];
    uint32_t x_step[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool there = nt * 8 + g < toks;
      xp[nt] = there ? xs + (nt * 8 + g) * x_stride + (piece - seg) * (kCols * 2) + t * kLaneBytes : zeros + t * kLaneBytes;
      x_step[nt] = there ? kSplit * kCols * 2 : 0u;
    }
    for (; piece < seg_end; piece += kSplit) {
      cp_async_wait<kPlDepth - 2>();
      __syncwarp();
      issue();  // into the slot that the last step read
      uint4 sc[2];
      sc[0] = ld_shared_v4(read + kPlRows * 64 + g * 16);
      if constexpr (FMT == kNVFP4) sc[1] = ld_shared_v4(read + kPlRows * 64 + 128 + g * 16);
#pragma unroll
      for (int pp = 0; pp < 4; pp += 2) {  // two 16-byte columns of the rows
        uint32_t b[NT][8];                 // the tokens' values for them
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (FMT == kMXFP8) {
            const uint2 lo = *reinterpret_cast<const uint2*>(xp[nt] + pp * 32), hi = *reinterpret_cast<const uint2*>(xp[nt] + pp * 32 + 32);
            b[nt][0] = lo.x, b[nt][1] = lo.y, b[nt][2] = hi.x, b[nt][3] = hi.y;
          } else {
            const uint4 lo = *reinterpret_cast<const uint4*>(xp[nt] + pp * 64), hi = *reinterpret_cast<const uint4*>(xp[nt] + pp * 64 + 64);
            b[nt][0] = lo.x, b[nt][1] = lo.y, b[nt][2] = lo.z, b[nt][3] = lo.w;
            b[nt][4] = hi.x, b[nt][5] = hi.y, b[nt][6] = hi.z, b[nt][7] = hi.w;
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {  // rows g + 64 m and 32 on
          uint32_t w[4];               // (row, column), (row + 32, column), (row, column + 1), ...
          ldmatrix_x4(read + m * 1024 + (pp == 0 ? lm_0 : lm_2), w);
          if constexpr (FMT == kNVFP4) {
            const uint32_t b0 = m ? sc[pp / 2].z : sc[pp / 2].x, b1 = m ? sc[pp / 2].w : sc[pp / 2].y;
            const uint32_t f0 = e4m3x2_to_f16x2(__byte_perm(b0, 0, sel)), f1 = e4m3x2_to_f16x2(__byte_perm(b1, 0, sel));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t d0 = f16_twice(f0, h), d1 = f16_twice(f1, h);
              uint32_t r0[4], r1[4];
              e2m1x8_to_f16(w[2 * h], r0);
              e2m1x8_to_f16(w[2 * h + 1], r1);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                r0[i] = mul_f16x2(r0[i], d0);
                r1[i] = mul_f16x2(r1[i], d1);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_f16(acc[m][nt], r0[0], r1[0], r0[1], r1[1], b[nt][4 * h], b[nt][4 * h + 1]);
                mma_f16(acc[m][nt], r0[2], r1[2], r0[3], r1[3], b[nt][4 * h + 2], b[nt][4 * h + 3]);
              }
            }
          } else if constexpr (FMT == kMXFP4) {
            const uint32_t b0 = m ? sc[0].z : sc[0].x, b1 = m ? sc[0].w : sc[0].y;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int block = pp + h;
              const float f0 = pl_mx_factor<F16>(b0, block);
              const float f1 = pl_mx_factor<F16>(b1, block);
              uint32_t r0[4], r1[4];
              e2m1x8_to_f16(w[2 * h], r0);
              e2m1x8_to_f16(w[2 * h + 1], r1);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(d, r0[0], r1[0], r0[1], r1[1], b[nt][4 * h], b[nt][4 * h + 1]);
                mma_f16(d, r0[2], r1[2], r0[3], r1[3], b[nt][4 * h + 2], b[nt][4 * h + 3]);
                acc[m][nt][0] = fmaf(f0, d[0], acc[m][nt][0]);
                acc[m][nt][1] = fmaf(f0, d[1], acc[m][nt][1]);
                acc[m][nt][2] = fmaf(f1, d[2], acc[m][nt][2]);
                acc[m][nt][3] = fmaf(f1, d[3], acc[m][nt][3]);
              }
            }
          } else {
            // both columns make one block of 32
            const uint32_t b0 = m ? sc[0].z : sc[0].x, b1 = m ? sc[0].w : sc[0].y;
            const int block = (piece & 1) * 2 + pp / 2;
            const float f0 = pl_mx_factor<F16>(b0, block);
            const float f1 = pl_mx_factor<F16>(b1, block);
            uint32_t r[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              r[2 * i] = e4m3x2_to_f16x2(w[i] & 0xFFFFu);
              r[2 * i + 1] = e4m3x2_to_f16x2(w[i] >> 16);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float d[4] = {0.f, 0.f, 0.f, 0.f};
              mma_f16(d, r[0], r[2], r[1], r[3], b[nt][0], b[nt][1]);
              mma_f16(d, r[4], r[6], r[5], r[7], b[nt][2], b[nt][3]);
              acc[m][nt][0] = fmaf(f0, d[0], acc[m][nt][0]);
              acc[m][nt][1] = fmaf(f0, d[1], acc[m][nt][1]);
              acc[m][nt][2] = fmaf(f1, d[2], acc[m][nt][2]);
              acc[m][nt][3] = fmaf(f1, d[3], acc[m][nt][3]);
            }
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) xp[nt] += x_step[nt];
      read = read == ring + (kPlDepth - 1) * kPlSlot ? ring : read + kPlSlot;
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // exp_of read below is the last one; the rings and the tokens are done with

  // warps' sums: [part of K][set of rows][token][32 rows]; the first part's place takes the block's
  constexpr int kPart = RT * kTile * 32;
  float* red = reinterpret_cast<float*>(pl_smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = nt * 8 + 2 * t + (i & 1);
      const float f = F16 ? 1.f : pl_pow2((FMT == kNVFP4 ? 0 : 14) - exp_of[tok]);
#pragma unroll
      for (int m = 0; m < 2; ++m)
        red[part * kPart + ((warp / kSplit) * kTile + tok) * 32 + 8 * (2 * m + (i >> 1)) + g] = acc[m][nt][i] * f;
    }
  __syncthreads();
  if (ranks > 1) {
    for (int e = tid; e < kPart; e += kPlThreads) {
      if ((e >> 5) % kTile >= toks) continue;
      float s = red[e];
#pragma unroll
      for (int w = 1; w < kSplit; ++w) s += red[w * kPart + e];
      red[e] = s;
    }
    cluster_sync_all();
  }
  const float sf = FMT == kNVFP4 ? __ldg(a.sf) : 1.f;
  for (int e = tid + rank * kPlThreads; e < kPart; e += ranks * kPlThreads) {
    const int t_in = (e >> 5) % kTile;
    const int64_t row = (static_cast<int64_t>(blockIdx.y) * RT + (e >> 5) / kTile) / 4 * 128 +
                        ((static_cast<int64_t>(blockIdx.y) * RT + (e >> 5) / kTile) & 3) * 8 + 32 * ((e >> 3) & 3) + (e & 7);
    if (t_in >= toks || row >= a.rows) continue;
    const int64_t at = t_in * a.ld_out + row;
    float extra = 0.f;
    if (a.add) extra = a.out_f32 ? static_cast<const float*>(a.add)[t_in * a.ld_add + row]
                                 : elem2_to_f32x2<F16>(static_cast<const uint16_t*>(a.add)[t_in * a.ld_add + row]).x;
    float s = 0.f;
    if (ranks > 1) {
      float v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < ranks) v[r] = __uint_as_float(cluster_ld_u32(cluster_map(red + e, r)));
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < ranks) s += v[r];
    } else {
      s = red[e];
#pragma unroll
      for (int w = 1; w < kSplit; ++w) s += red[w * kPart + e];
    }
    if (FMT == kNVFP4) s = __fdiv_rn(s, sf);
    if (a.add) s += extra;
    if (a.out_f32)
      static_cast<float*>(a.out)[at] = s;
    else
      static_cast<uint16_t*>(a.out)[at] = static_cast<uint16_t>(f32x2_to_elem2<F16>(s, 0.f));
  }
  if (ranks > 1) cluster_sync_all();  // no block leaves while another reads its sums
}

}  // namespace bsq
