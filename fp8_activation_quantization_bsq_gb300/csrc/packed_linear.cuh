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
// Form.  A block of 8 warps takes 32 rows: 8 q + g + 32 j of a 128-row band (g < 8, j < 4), whose scales in the 5D layout are 16
// consecutive bytes per g.  Its warps share out pieces of 64 bytes per row along K; each streams them by asynchronous copies of
// 16 bytes through a ring of its own (no barrier: a warp reads what its own lanes copied), and ldmatrix hands a lane
// the 4 bytes of its row that the product's layout wants.  The tokens' columns lie in shared memory as FP16.  Where rows are few, the blocks
// of a cluster share K; the warps' sums are added in shared memory, the blocks' through the cluster's, in a fixed order.
#pragma once

#include "cluster.cuh"
#include "serving_common.cuh"

namespace bsq {

constexpr int kPlWarps = 8, kPlThreads = kPlWarps * 32, kPlRows = 32;
constexpr int kPlDepth = 4;                              // pieces in a warp's ring
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
  int per_rank;           // of a block's share of K, a multiple of 8
  int segment;            // of the tokens' columns held at a time, a multiple of 8
  int k_atoms;            // scale atoms per band
  int64_t row_bytes;
  int out_f32;
};

template <int FMT> struct PlFmt {
  static constexpr int kCols = FMT == kMXFP8 ? 64 : 128;  // columns of a piece
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
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

// 2^k that takes a largest magnitude (FP32 bits) to below 2^15; k from -113 to 127.
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

// NT: tiles of 8 tokens that a block takes.
template <int FMT, bool F16, int NT>
__global__ void __launch_bounds__(kPlThreads, 2) packed_linear_kernel(const PlArgs a) {
  constexpr int kCols = PlFmt<FMT>::kCols;
  constexpr int kTile = NT * 8;
  extern __shared__ __align__(1024) uint8_t pl_smem[];
  __shared__ uint32_t amax_of[kTile];
  __shared__ int exp_of[kTile];  // the power of two that the tokens are held times
  uint8_t* xs = pl_smem + kPlRing;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int rank = blockIdx.x, ranks = gridDim.x;  // blocks of a cluster, along K
  const int64_t tile = blockIdx.y;                 // 32 rows
  const int64_t row0 = (tile >> 2) * 128 + (tile & 3) * 8;
  const int tok0 = blockIdx.z * kTile, toks = min(kTile, a.tokens - tok0);
  const int p_lo = rank * a.per_rank, p_hi = min(p_lo + a.per_rank, a.pieces);
  const int x_stride = a.segment * kCols * 2 + 64;  // bytes of a token: 64 past a multiple of 128, for the banks

  // this lane's part of a copy
  const uint32_t ring = smem_addr(pl_smem) + warp * (kPlDepth * kPlSlot);
  const int cr = lane >> 2, cp = lane & 3;
  auto issue = [&](int n) {  // the warp's n-th piece
    const int piece = p_lo + warp + kPlWarps * n;
    const uint32_t slot = ring + (n % kPlDepth) * kPlSlot;
    if (piece < p_hi) {
      const int64_t byte = static_cast<int64_t>(piece) * 64 + cp * 16;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t row = row0 + 32 * j + cr;
        const bool in = row < a.rows && byte < a.row_bytes;
        cp_async16(slot + (8 * j + cr) * 64 + ((cp ^ ((cr >> 1) & 3)) * 16), a.w + (in ? row * a.row_bytes + byte : 0), in);
      }
      constexpr int kAtoms = FMT == kNVFP4 ? 2 : 1;
      if (lane < 8 * kAtoms) {
        const int atom = FMT == kMXFP8 ? piece >> 1 : piece * kAtoms + (lane >> 3);
        const bool in = atom < a.k_atoms;
        cp_async16(slot + kPlRows * 64 + lane * 16,
                   a.scales + (in ? ((tile >> 2) * a.k_atoms + atom) * 512 + ((tile & 3) * 8 + (lane & 7)) * 16 : 0), in);
      }
    }
    cp_async_commit();
  };

  pdl_wait();
#pragma unroll
  for (int n = 0; n < kPlDepth - 1; ++n) issue(n);
  if (tid < kTile) exp_of[tid] = 127;

  float acc[2][NT][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][nt][i] = 0.f;

  // ldmatrix: lane's row address, without the piece's swizzled part
  const uint32_t lm_row = (8 * ((lane >> 3) & 1) + (lane & 7)) * 64, lm_x = ((lane & 7) >> 1) & 3, lm_p = lane >> 4;

  int n = 0;
  for (int seg = p_lo; seg < p_hi; seg += a.segment) {
    const int seg_end = min(seg + a.segment, p_hi);
    // the segment's tokens: 8 columns per item; columns past the last one are zeros
    const int groups = a.segment * kCols / 8, items = toks * groups;  // groups: a multiple of 32
    const int col0 = seg * kCols, live = min(seg_end * kCols, a.cols) - col0;
    __syncthreads();  // the segment before has been read, exp_of is set
    if constexpr (!F16) {
      if (tid < kTile) amax_of[tid] = 0u;
      __syncthreads();
      for (int i = tid; i < items; i += kPlThreads) {
        const int tok = i / groups, c = (i - tok * groups) * 8;
        uint32_t m = 0;
        if (c < live) {
          const uint4 v = ld_global_nc_v4(a.x + (tok0 + tok) * a.ld_x + col0 + c);
          m = absmax2(absmax2(absmax2(absmax2(m, v.x), v.y), v.z), v.w);
        }
        const uint32_t top = __reduce_max_sync(~0u, __float_as_uint(absmax_final(m)));
        if (lane == 0) atomicMax(&amax_of[tok], top);
      }
      __syncthreads();
      // sums so far follow to the new power of two, which never grows
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int tok = nt * 8 + 2 * t + i;
          const int was = exp_of[tok], now = min(was, pl_exponent(amax_of[tok]));
          if (now != was && seg != p_lo) {
            const int d = max(now - was, -250), h = d / 2;
            const float f = pl_pow2(h), q = pl_pow2(d - h);
            acc[0][nt][i] = acc[0][nt][i] * f * q;
            acc[0][nt][i + 2] = acc[0][nt][i + 2] * f * q;
            acc[1][nt][i] = acc[1][nt][i] * f * q;
            acc[1][nt][i + 2] = acc[1][nt][i + 2] * f * q;
          }
        }
      __syncthreads();
      if (tid < kTile) exp_of[tid] = min(exp_of[tid], pl_exponent(amax_of[tid]));
      __syncthreads();
    }
    for (int i = tid; i < items; i += kPlThreads) {
      const int tok = i / groups, c = (i - tok * groups) * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (c < live) {
        v = ld_global_nc_v4(a.x + (tok0 + tok) * a.ld_x + col0 + c);
        if constexpr (!F16) {
          const float f = pl_pow2(exp_of[tok]);
          v.x = f32x2_to_elem2<true>(bf16_lo(v.x) * f, bf16_hi(v.x) * f);
          v.y = f32x2_to_elem2<true>(bf16_lo(v.y) * f, bf16_hi(v.y) * f);
          v.z = f32x2_to_elem2<true>(bf16_lo(v.z) * f, bf16_hi(v.z) * f);
          v.w = f32x2_to_elem2<true>(bf16_lo(v.w) * f, bf16_hi(v.w) * f);
        }
      }
      *reinterpret_cast<uint4*>(xs + static_cast<int64_t>(tok) * x_stride + c * 2) = v;
    }
    __syncthreads();

    for (; p_lo + warp + kPlWarps * n < seg_end; ++n) {
      cp_async_wait<kPlDepth - 2>();
      __syncwarp();
      issue(n + kPlDepth - 1);  // into the slot that the last step read
      const int piece = p_lo + warp + kPlWarps * n;
      const uint32_t slot = ring + (n % kPlDepth) * kPlSlot;
      const uint8_t* xp = xs + (piece - seg) * (kCols * 2);
      uint4 sc[2];
      {
        const uint8_t* sp = pl_smem + (slot - smem_addr(pl_smem)) + kPlRows * 64 + g * 16;
        sc[0] = *reinterpret_cast<const uint4*>(sp);
        if constexpr (FMT == kNVFP4) sc[1] = *reinterpret_cast<const uint4*>(sp + 128);
      }
#pragma unroll
      for (int pp = 0; pp < 4; pp += 2) {  // two 16-byte columns of the rows
        uint32_t b[NT][8];                 // the tokens' values for them
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int tok = nt * 8 + g;
          const uint8_t* src = xp + tok * x_stride;
          if constexpr (FMT == kMXFP8) {
            const uint2 lo = tok < toks ? *reinterpret_cast<const uint2*>(src + pp * 32 + t * 8) : make_uint2(0, 0);
            const uint2 hi = tok < toks ? *reinterpret_cast<const uint2*>(src + (pp + 1) * 32 + t * 8) : make_uint2(0, 0);
            b[nt][0] = lo.x, b[nt][1] = lo.y, b[nt][2] = hi.x, b[nt][3] = hi.y;
          } else {
            const uint4 lo = tok < toks ? *reinterpret_cast<const uint4*>(src + pp * 64 + t * 16) : make_uint4(0, 0, 0, 0);
            const uint4 hi = tok < toks ? *reinterpret_cast<const uint4*>(src + (pp + 1) * 64 + t * 16) : make_uint4(0, 0, 0, 0);
            b[nt][0] = lo.x, b[nt][1] = lo.y, b[nt][2] = lo.z, b[nt][3] = lo.w;
            b[nt][4] = hi.x, b[nt][5] = hi.y, b[nt][6] = hi.z, b[nt][7] = hi.w;
          }
        }
#pragma unroll
        for (int m = 0; m < 2; ++m) {  // rows g + 64 m and 32 on
          uint32_t w[4];               // (row, column), (row + 32, column), (row, column + 1), ...
          ldmatrix_x4(slot + m * 1024 + lm_row + (((pp + lm_p) ^ lm_x) * 16), w);
          if constexpr (FMT == kNVFP4) {
            // byte 2 p + t / 2 of a row's scale word: this lane's 8 codes of column p lie in one block
            const uint32_t s0 = m ? sc[pp / 2].z : sc[pp / 2].x, s1 = m ? sc[pp / 2].w : sc[pp / 2].y;
            const uint32_t sel = (t >> 1) | ((2 + (t >> 1)) << 4);
            const uint32_t f0 = e4m3x2_to_f16x2(__byte_perm(s0, 0, sel)), f1 = e4m3x2_to_f16x2(__byte_perm(s1, 0, sel));
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t d0 = __byte_perm(f0, 0, h ? 0x3232 : 0x1010), d1 = __byte_perm(f1, 0, h ? 0x3232 : 0x1010);
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
            const uint32_t s0 = m ? sc[0].z : sc[0].x, s1 = m ? sc[0].w : sc[0].y;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int block = pp + h;
              const float f0 = pl_mx_factor<F16>(s0, block);
              const float f1 = pl_mx_factor<F16>(s1, block);
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
            const uint32_t s0 = m ? sc[0].z : sc[0].x, s1 = m ? sc[0].w : sc[0].y;
            const int block = (piece & 1) * 2 + pp / 2;
            const float f0 = pl_mx_factor<F16>(s0, block);
            const float f1 = pl_mx_factor<F16>(s1, block);
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
    }
  }
  cp_async_wait<0>();
  __syncthreads();  // exp_of read below is the last one; the rings and the tokens are done with

  // warps' sums, [warp][32 rows][tile tokens], then the block's at the same place
  float* red = reinterpret_cast<float*>(pl_smem);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int tok = nt * 8 + 2 * t + (i & 1);
      const float f = F16 ? 1.f : pl_pow2((FMT == kNVFP4 ? 0 : 14) - exp_of[tok]);
#pragma unroll
      for (int m = 0; m < 2; ++m) red[(warp * kTile + tok) * 32 + 8 * (2 * m + (i >> 1)) + g] = acc[m][nt][i] * f;
    }
  __syncthreads();
  for (int e = tid; e < toks * 32; e += kPlThreads) {
    float s = red[e];
#pragma unroll
    for (int w = 1; w < kPlWarps; ++w) s += red[w * kTile * 32 + e];
    red[e] = s;
  }
  if (ranks > 1) cluster_sync_all(); else __syncthreads();
  const float sf = FMT == kNVFP4 ? __ldg(a.sf) : 1.f;
  for (int e = tid + rank * kPlThreads; e < toks * 32; e += ranks * kPlThreads) {
    float s = 0.f;
    if (ranks > 1) {
      for (int r = 0; r < ranks; ++r) s += __uint_as_float(cluster_ld_u32(cluster_map(red + e, r)));
    } else {
      s = red[e];
    }
    const int tok = tok0 + (e >> 5);
    const int64_t row = row0 + 32 * ((e >> 3) & 3) + (e & 7);
    if (row < a.rows) {
      if (FMT == kNVFP4) s = __fdiv_rn(s, sf);
      const int64_t at = tok * a.ld_out + row;
      if (a.out_f32) {
        if (a.add) s += static_cast<const float*>(a.add)[tok * a.ld_add + row];
        static_cast<float*>(a.out)[at] = s;
      } else {
        if (a.add) s += elem2_to_f32x2<F16>(static_cast<const uint16_t*>(a.add)[tok * a.ld_add + row]).x;
        static_cast<uint16_t*>(a.out)[at] = static_cast<uint16_t>(f32x2_to_elem2<F16>(s, 0.f));
      }
    }
  }
  if (ranks > 1) cluster_sync_all();  // no block leaves while another reads its sums
}

}  // namespace bsq
