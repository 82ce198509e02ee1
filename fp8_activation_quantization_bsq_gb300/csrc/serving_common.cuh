// Device helpers shared by the key/value cache and expert-layer kernels:
// conversions between E4M3 codes and FP16 / FP32, BF16 and FP16 element
// pairs, and the error word, which these kernels get as an argument.
#pragma once

#include <cuda_bf16.h>

#include "device_common.cuh"

namespace bsq {

// The first recorded code wins (as record_error, on a given word).
__device__ __forceinline__ void record_error_at(unsigned int* word, unsigned code) { atomicCAS(word, 0u, code); }

// Two E4M3 codes (low byte first) -> two FP16 (exact; NaN codes stay NaN).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}

// Two FP32 -> two E4M3 codes, `lo` in the low byte (nearest even, saturating).
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two FP32 -> a byte of two E2M1 codes, `lo` in the low nibble.
__device__ __forceinline__ uint8_t f32x2_to_e2m1x2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 q;\n\tcvt.rn.satfinite.e2m1x2.f32 q, %2, %1;\n\tmov.b32 %0, {q, q, q, q};\n\t}" : "=r"(r) : "f"(lo), "f"(hi));
  return static_cast<uint8_t>(r);
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t w) {
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// A word of two 16-bit elements (BF16 or FP16) -> FP32.
template <bool F16>
__device__ __forceinline__ float2 elem2_to_f32x2(uint32_t w) {
  if constexpr (F16) return f16x2_to_f32x2(w);
  return make_float2(bf16_lo(w), bf16_hi(w));
}

template <bool F16>
__device__ __forceinline__ uint32_t f32x2_to_elem2(float lo, float hi) {
  uint32_t r;
  if constexpr (F16)
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// max of magnitudes over pairs of 16-bit elements, as absmax2 (whose signs
// are masked off at the end).
template <bool F16>
__device__ __forceinline__ uint32_t elem_absmax2(uint32_t acc, uint32_t w) {
  if constexpr (!F16) return absmax2(acc, w);
  uint32_t r;
  asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(acc), "r"(w));
  return r;
}
template <bool F16>
__device__ __forceinline__ float elem_absmax_final(uint32_t acc) {
  const float2 v = elem2_to_f32x2<F16>(acc & 0x7FFF7FFFu);
  return fmaxf(v.x, v.y);
}

// 2^e for -127 <= e <= 127 (2^-127 is subnormal).
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float(e > -127 ? static_cast<uint32_t>(e + 127) << 23 : 0x00400000u); }

// Asynchronous copies of 16 bytes into shared memory (zeros where not valid, nothing is read then), and their groups.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

}  // namespace bsq
