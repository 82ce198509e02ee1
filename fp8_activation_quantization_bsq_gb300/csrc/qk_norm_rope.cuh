// Norm of query and key heads and their rotation by position, in one pass:
//   u = x / sqrt(mean(x^2) + eps) * w  (per head row; without a weight u = x)
//   (u_a, u_b) -> (u_a cos t - u_b sin t, u_b cos t + u_a sin t),  t = position * inv_freq[i]
// for the first `pairs` pairs of a row, (i, i + pairs) or (2i, 2i + 1); what lies behind passes.
//
// Bound by DRAM: 2 bytes read and 2 written per element.  Measured: 4096 tokens of 64 + 8 heads of 128 26.5 to 26.8 us (5.6 TB/s; of 6.8 copied), neighbouring
// pairs 26.1 to 28.1, without norm 25.1, 16384 tokens 6.2 TB/s; one token of 32 + 8 heads 2.6 us, a launch.  Pairs (i, i + n) of a number that no 4
// divides (MODE 2) take 50 us: their other sides go through shared memory, whose banks and latency bound it (half of
// the cycles between a warp's instructions are waits for it).  A row's 8 elements per lane are two
// groups of 4 that hold both sides of a lane's pairs, so that no element crosses lanes in registers and the lane's 4
// angles serve every head of the token that the warp takes; 8, 16 or 32 lanes per row (dim to 64, 128, 256).  A warp keeps 4 steps of its rows in
// flight through a ring in shared memory, 16 bytes a lane: with 3, 5, 6 and 8 steps 28.1, 26.8, 27.5 and 28.5 us (heads of 256 51.9, 59.4, 60.4, 61.0, with
// 4 56.3; 16384 tokens of 128 100.6, 95.8, 95.1, 95.7, with 4 97.1); each lane copying its own two groups of 8 bytes 29.4; two steps in registers 48.7.
//
// Angles: t / 2 pi in fixed point.  inv_freq is a 24-bit integer times a power of two, 1 / (2 pi) a 64-bit
// fraction, and the position multiplies their product, cut off at 2^-64 turns, modulo 2^64, which drops whole turns exactly: off by
// at most position (1 + |inv_freq|) 2^-64 turns before the last 32 bits are cut off.
#pragma once

#include "tcgen05.cuh"  // fma_f32x2

namespace bsq {

constexpr int kRopeWarps = 4, kRopeDepth = 4;  // steps of a warp in flight

struct RopeArgs {
  const uint16_t* src[2];  // queries, keys
  uint16_t* dst[2];
  int64_t src_tok[2], src_head[2], dst_tok[2], dst_head[2];  // strides in elements
  const void* weight[2];                                     // null: no norm
  const int32_t* positions;
  const float* inv_freq;
  int64_t tokens;
  int heads, rows;  // query heads, query and key heads
  int dim, pairs;
  int weight_f32;
  float eps, inv_dim;
  int chunks, per_chunk;  // tasks per token, rows per task
};

// cos and sin of position * f.
__device__ __forceinline__ float2 rope_turn(float f, int position) {
  const uint32_t bits = __float_as_uint(f);
  const int ex = static_cast<int>((bits >> 23) & 255u);
  const uint64_t m = (bits & 0x7FFFFFu) | (ex != 0 ? 0x800000u : 0u);
  const int e = max(ex, 1) - 150;                            // |f| = m 2^e
  constexpr uint64_t kInvTwoPi = 0x28BE60DB9391054Aull;      // 2^64 / (2 pi)
  const uint64_t lo = m * kInvTwoPi, hi = __umul64hi(m, kInvTwoPi);
  // (hi, lo) 2^e modulo 2^64: the frequency in turns per position
  uint64_t turn;
  if (e >= 0)
    turn = e < 64 ? lo << e : 0;
  else if (e > -64)
    turn = (lo >> -e) | (hi << (64 + e));
  else
    turn = e > -128 ? hi >> (-e - 64) : 0;
  turn *= static_cast<uint64_t>(static_cast<uint32_t>(position));
  if (bits >> 31) turn = 0 - turn;
  float2 r;
  // half turns in [-1, 1); the angle's rounding to 24 bits is the only one before the functions'
  sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f, &r.y, &r.x);
  if (ex == 255) r.x = r.y = __uint_as_float(0x7FC00000u);
  return r;
}

__device__ __forceinline__ float2 mul_f32x2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Rows whose elements a lane reads: MODE 0 pairs (i, i + pairs) with pairs a multiple of 4, 1 neighbouring pairs,
// 2 pairs (i, i + pairs) of any number, whose other sides come through shared memory.  L lanes per row.  Arithmetic goes two
// elements at a time.
template <bool F16, int L, int MODE>
__global__ void __launch_bounds__(kRopeWarps * 32, MODE == 2 ? 5 : 8) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int kPer = 32 / L;  // rows at a time
  __shared__ float other[MODE == 2 ? kRopeWarps * 256 : 1];
  __shared__ uint4 ring[kRopeWarps][kRopeDepth][32];  // the rows of a step, 16 bytes a lane
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane / L, p = lane % L;
  const int64_t task = static_cast<int64_t>(blockIdx.x) * kRopeWarps + warp;
  const int64_t token = task / a.chunks;
  if (token >= a.tokens) return;
  const int position = __ldg(a.positions + token);
  if (position < 0) return;
  const int first = static_cast<int>(task - token * a.chunks) * a.per_chunk, last = min(first + a.per_chunk, a.rows);
  const bool active = p < a.dim / 8;
  const int quarter = a.pairs / 4;  // groups of 4 elements on one side (MODE 0)
  const bool apart = MODE == 0 && p < quarter;
  const int ea = apart ? 4 * p : 8 * p, eb = apart ? 4 * p + a.pairs : 8 * p + 4;

  constexpr int kAngles = MODE == 2 ? 8 : 4;
  float cs[kAngles], sn[kAngles];
  uint32_t turns = 0;  // a bit per angle
#pragma unroll
  for (int j = 0; j < kAngles; ++j) {
    int i = MODE == 2 ? 8 * p + j : 4 * p + j;
    const bool turn = active && (MODE == 0 ? apart : MODE == 1 ? i < a.pairs : i < 2 * a.pairs);
    const bool second = MODE == 2 && i >= a.pairs;
    if (second) i -= a.pairs;
    cs[j] = 1.f;
    sn[j] = 0.f;
    if (turn) {
      turns |= 1u << j;
      const float2 t = rope_turn(__ldg(a.inv_freq + i), position);
      cs[j] = t.x;
      sn[j] = second ? -t.y : t.y;
    }
  }

#pragma unroll 1
  for (int k = 0; k < 2; ++k) {  // the task's queries, then its keys
    const int r0 = max(first, k ? a.heads : 0), r1 = min(last, k ? a.rows : a.heads);
    if (r0 >= r1) continue;
    const bool norm = a.weight[k] != nullptr;
    float2 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = j < 2 ? ea + 2 * j : eb + 2 * j - 4;
      w[j] = make_float2(1.f, 1.f);
      if (norm && active) {
        if (a.weight_f32) {
          const float* src = static_cast<const float*>(a.weight[k]) + e;
          w[j] = make_float2(__ldg(src), __ldg(src + 1));
        } else {
          const uint16_t* src = static_cast<const uint16_t*>(a.weight[k]) + e;
          w[j] = elem2_to_f32x2<F16>(__ldg(src) | static_cast<uint32_t>(__ldg(src + 1)) << 16);
        }
      }
    }
    const int h = r0 + sub - (k ? a.heads : 0), n = r1 - r0;
    const uint16_t* s = a.src[k] + token * a.src_tok[k] + h * a.src_head[k];
    uint16_t* d = a.dst[k] + token * a.dst_tok[k] + h * a.dst_head[k];
    const int64_t s_step = kPer * a.src_head[k], d_step = kPer * a.dst_head[k];
    uint4* const mine_in = &ring[warp][0][lane];
    const uint8_t* const row_in = reinterpret_cast<const uint8_t*>(&ring[warp][0][sub * L]);
    int left = active ? n - sub : 0;  // rows not yet asked for, this lane's at every kPer-th
    const auto ask = [&](int slot) {
      if (left > 0) cp_async16(smem_addr(mine_in + slot * 32), s + 8 * p);
      cp_async_commit();
      left -= kPer;
      s += s_step;
    };
#pragma unroll
    for (int i = 0; i < kRopeDepth - 1; ++i) ask(i);
    int slot = 0;
#pragma unroll 1
    for (int i = sub; i - sub < n; i += kPer, d += d_step) {
      const bool in = i < n && active;
      cp_async_wait<kRopeDepth - 2>();
      uint2 va = make_uint2(0, 0), vb = va;
      if constexpr (MODE == 0) {
        __syncwarp();  // a lane reads what others copied
        if (in) {
          va = *reinterpret_cast<const uint2*>(row_in + slot * 512 + ea * 2);
          vb = *reinterpret_cast<const uint2*>(row_in + slot * 512 + eb * 2);
        }
      } else if (in) {
        const uint4 v = mine_in[slot * 32];
        va = make_uint2(v.x, v.y);
        vb = make_uint2(v.z, v.w);
      }
      ask(slot == 0 ? kRopeDepth - 1 : slot - 1);
      slot = slot == kRopeDepth - 1 ? 0 : slot + 1;
      float2 x[4] = {elem2_to_f32x2<F16>(va.x), elem2_to_f32x2<F16>(va.y), elem2_to_f32x2<F16>(vb.x), elem2_to_f32x2<F16>(vb.y)};
      if (norm) {
        const auto squares = [&]() {
          float2 q = mul_f32x2(x[0], x[0]);
#pragma unroll
          for (int j = 1; j < 4; ++j) q = fma_f32x2(x[j], x[j], q);
          float sum = q.x + q.y;
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
          return sum;
        };
        float sum = squares(), eps = a.eps;
        // Squares that near FP32's ends (BF16 rows only): once more, of 2^-72 or 2^96 times the row, where sums below 2^-90 (FP32 may have lost some)
        // matter beside an eps as small, above 2^124, and above 2^100 beside an eps that with their mean passes FP32.  That is exact: what 2^-72
        // takes below FP32's subnormal numbers lies below BF16's once it is divided by its row's root.  (Limits from the arguments in place of these
        // constants cost 3 % of a prompt's time.)
        if (!F16 && __any_sync(~0u, sum > 0x1p100f || sum < 0x1p-90f)) {
          const float by = sum > (eps > 0x1p126f ? 0x1p100f : 0x1p124f) ? 0x1p-72f : sum < 0x1p-90f && eps < 0x1p-70f ? 0x1p96f : 1.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = mul_f32x2(x[j], make_float2(by, by));
          sum = squares();
          eps = eps * by * by;
        }
        const float f = rsqrtf(sum * a.inv_dim + eps);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = mul_f32x2(mul_f32x2(x[j], make_float2(f, f)), w[j]);  // f w alone may pass FP32
      }
      float2 y[4] = {x[0], x[1], x[2], x[3]};
      if constexpr (MODE == 0) {
        if (turns != 0u) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float2 c = make_float2(cs[2 * j], cs[2 * j + 1]), t = make_float2(sn[2 * j], sn[2 * j + 1]);
            y[j] = fma_f32x2(x[j], c, mul_f32x2(x[j + 2], make_float2(-t.x, -t.y)));
            y[j + 2] = fma_f32x2(x[j + 2], c, mul_f32x2(x[j], t));
          }
        }
      } else if constexpr (MODE == 1) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (turns >> j & 1u) y[j] = make_float2(x[j].x * cs[j] - x[j].y * sn[j], x[j].y * cs[j] + x[j].x * sn[j]);
      } else {
        float* mine = other + (warp * kPer + sub) * 8 * L;  // the row's other lanes
        float* out = reinterpret_cast<float*>(y);
#pragma unroll
        for (int j = 0; j < 4; ++j) *reinterpret_cast<float2*>(mine + 8 * p + 2 * j) = x[j];
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (turns >> j & 1u) out[j] = out[j] * cs[j] - mine[8 * p + j < a.pairs ? 8 * p + j + a.pairs : 8 * p + j - a.pairs] * sn[j];
        __syncwarp();
      }
      if (in) {
        const uint2 oa = make_uint2(f32x2_to_elem2<F16>(y[0].x, y[0].y), f32x2_to_elem2<F16>(y[1].x, y[1].y));
        const uint2 ob = make_uint2(f32x2_to_elem2<F16>(y[2].x, y[2].y), f32x2_to_elem2<F16>(y[3].x, y[3].y));
        if (apart) {
          *reinterpret_cast<uint2*>(d + ea) = oa;
          *reinterpret_cast<uint2*>(d + eb) = ob;
        } else {
          *reinterpret_cast<uint4*>(d + ea) = make_uint4(oa.x, oa.y, ob.x, ob.y);
        }
      }
    }
    cp_async_wait<0>();
    __syncwarp();  // the keys' first rows go where a lane may still read the queries' last ones
  }
}

}  // namespace bsq
