// tcgen05 (5th-generation tensor core) and TMA wrappers shared by the
// serving kernels, as inline PTX: tensor-memory allocation, shared-memory and
// instruction descriptors, block-scaled and FP16 matrix products, copies of
// scale factors into tensor memory, and bulk copies.
#pragma once

#include "serving_common.cuh"

namespace bsq {

// Waits are bounded by the SM's clock, about a second (the global timer that
// mbar_wait_bounded reads costs about a microsecond when a wait is not over at once).
constexpr long long kWaitLimitCycles = 2000000000ll;

// Wait until the phase with the given parity has completed; false when the
// limit expired or another role of the block has given up.
__device__ __forceinline__ bool mbar_wait_clocked(uint64_t* bar, uint32_t parity, const volatile uint32_t* abort_flag,
                                                  long long limit = kWaitLimitCycles) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (*abort_flag != 0u || clock64() - t0 > limit) return false;
  return true;
}

// The same for copies and products that have to land whatever happened.
__device__ __forceinline__ bool mbar_wait_clocked(uint64_t* bar, uint32_t parity, long long limit = kWaitLimitCycles) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity))
    if (clock64() - t0 > limit) return false;
  return true;
}

// This thread's warp, broadcast: the compiler then knows it to be the same for
// the whole warp, and keeps what a role's code computes in uniform registers.
__device__ __forceinline__ int warp_index() { return __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) >> 5, 0); }
__device__ __forceinline__ int warp_uniform(int x) { return __shfl_sync(0xFFFFFFFFu, x, 0); }

__device__ __forceinline__ void t5_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void t5_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }

// Whole warp.
__device__ __forceinline__ void t5_alloc(uint32_t* slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(slot)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void t5_dealloc(uint32_t taddr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
}

// The products, scale copies and commits below are issued by a whole warp in
// uniform control flow and executed by its one lane with `lead` set: their
// operands live in uniform registers, and inside a branch of one lane every one of them would be
// moved there by itself, one after the other (about 90 cycles per product).

// Whether this lane is the warp's leader.
__device__ __forceinline__ uint32_t t5_elect() {
  uint32_t lead;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(lead));
  return lead;
}

// Arrive on `bar` when every tcgen05 operation the leader has issued is done.
__device__ __forceinline__ void t5_commit(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(lead)
      : "memory");
}

// K-major operand tile with the 128-byte swizzle: rows of 128 bytes, groups of 8
// rows 1024 bytes apart.  Fields: address >> 4, leading offset (unused, 1),
// stride offset >> 4 at 32, 0b001 at 46, swizzle mode 2 at 61.
__device__ __forceinline__ uint64_t t5_desc_sw128(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(1) << 16) | (static_cast<uint64_t>(64) << 32) |
         (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// A 512-byte scale atom (32 rows of 16 bytes, no swizzle): groups of 8 rows 128 bytes apart.
__device__ __forceinline__ uint64_t t5_desc_atom(uint32_t saddr) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(8) << 32) | (static_cast<uint64_t>(1) << 46);
}

// One scale atom into 4 columns of tensor memory: column c, lane i of every
// quarter gets the 4 bytes of the atom's row 32 c + i.
__device__ __forceinline__ void t5_copy_atom(uint32_t taddr, uint64_t desc, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %2, 0;\n\t@q tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
      "l"(desc), "r"(lead)
      : "memory");
}

// A whole stage of the block-scaled products of two 128-row tiles (accumulators d
// and d + 64, operand a and 16 KB on) with the same second operand b: the scale
// atoms ds.. of both tiles and of b (ATOMS each) to tensor memory at sf, sf + 16 and sf + 32, then four
// slices of 32 bytes of each row.  One statement, as for FP16 below.
#define BSQ_T5_CP(TOFF, DOFF)                                      \
  "add.u32 t, %6, " #TOFF ";\n\tadd.u64 e, %5, " #DOFF ";\n\t"     \
  "@q tcgen05.cp.cta_group::1.32x128b.warpx4 [t], e;\n\t"
#define BSQ_T5_BS(KIND, OFF, OFF2, SA, SA2, SB, ID, ACC)                                                            \
  "add.u64 x, %2, " #OFF ";\n\tadd.u64 y, %3, " #OFF ";\n\tadd.u32 t, %6, " #SA ";\n\tadd.u32 u, %6, " #SB ";\n\t"       \
  "add.u32 i, %4, " #ID ";\n\t@q tcgen05.mma.cta_group::1.kind::" KIND " [%0], x, y, i, [t], [u], " ACC ";\n\t"          \
  "add.u64 x, %2, " #OFF2 ";\n\tadd.u32 t, %6, " #SA2 ";\n\t@q tcgen05.mma.cta_group::1.kind::" KIND                  \
  " [%1], x, y, i, [t], [u], " ACC ";\n\t"
#define BSQ_T5_OPEN                                                                                                 \
  "{\n\t.reg .pred p, o, q;\n\t.reg .b32 t, u, i;\n\t.reg .b64 e, x, y;\n\tsetp.ne.b32 p, %7, 0;\n\t"                 \
  "setp.ne.b32 q, %8, 0;\n\tsetp.eq.b32 o, 0, 0;\n\t"
#define BSQ_T5_ARGS                                                                                                 \
  ::"r"(d), "r"(d + 64), "l"(a), "l"(b), "r"(idesc), "l"(ds), "r"(sf), "r"(accumulate), "r"(lead) : "memory"
template <int FMT>
__device__ __forceinline__ void t5_stage_scaled(uint32_t d, uint64_t a, uint64_t b, uint64_t ds, uint32_t idesc, uint32_t sf,
                                                uint32_t accumulate, uint32_t lead) {
  // the scale ids of a slice (bits 4 and 29 of idesc): 2 -> 0x40000020, 1 -> 0x20000010, 3 -> 0x60000030
  if constexpr (FMT == kNVFP4)
    asm volatile(BSQ_T5_OPEN BSQ_T5_CP(0, 0) BSQ_T5_CP(16, 128) BSQ_T5_CP(32, 256) BSQ_T5_CP(4, 32) BSQ_T5_CP(20, 160) BSQ_T5_CP(36, 288)
                 BSQ_T5_CP(8, 64) BSQ_T5_CP(24, 192) BSQ_T5_CP(40, 320) BSQ_T5_CP(12, 96) BSQ_T5_CP(28, 224) BSQ_T5_CP(44, 352)
                 BSQ_T5_BS("mxf4nvf4.block_scale.scale_vec::4X", 0, 1024, 0, 16, 32, 0, "p")
                 BSQ_T5_BS("mxf4nvf4.block_scale.scale_vec::4X", 2, 1026, 4, 20, 36, 0, "o")
                 BSQ_T5_BS("mxf4nvf4.block_scale.scale_vec::4X", 4, 1028, 8, 24, 40, 0, "o")
                 BSQ_T5_BS("mxf4nvf4.block_scale.scale_vec::4X", 6, 1030, 12, 28, 44, 0, "o") "}" BSQ_T5_ARGS);
  else if constexpr (FMT == kMXFP4)
    asm volatile(BSQ_T5_OPEN BSQ_T5_CP(0, 0) BSQ_T5_CP(16, 64) BSQ_T5_CP(32, 128) BSQ_T5_CP(4, 32) BSQ_T5_CP(20, 96) BSQ_T5_CP(36, 160)
                 BSQ_T5_BS("mxf4.block_scale.scale_vec::2X", 0, 1024, 0, 16, 32, 0, "p")
                 BSQ_T5_BS("mxf4.block_scale.scale_vec::2X", 2, 1026, 0, 16, 32, 0x40000020, "o")
                 BSQ_T5_BS("mxf4.block_scale.scale_vec::2X", 4, 1028, 4, 20, 36, 0, "o")
                 BSQ_T5_BS("mxf4.block_scale.scale_vec::2X", 6, 1030, 4, 20, 36, 0x40000020, "o") "}" BSQ_T5_ARGS);
  else
    asm volatile(BSQ_T5_OPEN BSQ_T5_CP(0, 0) BSQ_T5_CP(16, 32) BSQ_T5_CP(32, 64)
                 BSQ_T5_BS("mxf8f6f4.block_scale.scale_vec::1X", 0, 1024, 0, 16, 32, 0, "p")
                 BSQ_T5_BS("mxf8f6f4.block_scale.scale_vec::1X", 2, 1026, 0, 16, 32, 0x20000010, "o")
                 BSQ_T5_BS("mxf8f6f4.block_scale.scale_vec::1X", 4, 1028, 0, 16, 32, 0x40000020, "o")
                 BSQ_T5_BS("mxf8f6f4.block_scale.scale_vec::1X", 6, 1030, 0, 16, 32, 0x60000030, "o") "}" BSQ_T5_ARGS);
}
#undef BSQ_T5_CP
#undef BSQ_T5_BS
#undef BSQ_T5_OPEN
#undef BSQ_T5_ARGS

// D (128 x N, FP32) (+)= A B^T with block scales, K = 32 bytes of each row.
#define BSQ_T5_MMA_SCALED(KIND)                                                                                        \
  asm volatile(                                                                                                        \
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %7, 0;\n\t"                                      \
      "@q tcgen05.mma.cta_group::1.kind::" KIND " [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d), "l"(a), "l"(b),     \
      "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate), "r"(lead)                                                       \
      : "memory")
template <int FMT>
__device__ __forceinline__ void t5_mma_scaled(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                              uint32_t accumulate, uint32_t lead) {
  if constexpr (FMT == kNVFP4)
    BSQ_T5_MMA_SCALED("mxf4nvf4.block_scale.scale_vec::4X");
  else if constexpr (FMT == kMXFP4)
    BSQ_T5_MMA_SCALED("mxf4.block_scale.scale_vec::2X");
  else
    BSQ_T5_MMA_SCALED("mxf8f6f4.block_scale.scale_vec::1X");
}
#undef BSQ_T5_MMA_SCALED

// Instruction descriptor of the block-scaled products, M = 128: scale id of B
// at 4-5, operand formats at 7 and 10 (E2M1 1, E4M3 0), N >> 3 at 17, scale type at 23
// (E4M3 0, E8M0 1), M >> 4 at 24, scale id of A at 29-30.  The id picks the
// byte of a scale word that a K slice uses.
template <int FMT>
__device__ __forceinline__ uint32_t t5_idesc_scaled(uint32_t n, uint32_t sf_id) {
  constexpr uint32_t fmt = FMT == kMXFP8 ? 0u : 1u;
  return (sf_id << 4) | (fmt << 7) | (fmt << 10) | ((n >> 3) << 17) | ((FMT == kNVFP4 ? 0u : 1u) << 23) | (8u << 24) | (sf_id << 29);
}

// 8 consecutive columns of this thread's tensor-memory lane at two addresses,
// waited for in the same statement, so that no register is read early.
__device__ __forceinline__ void t5_ld8_pair(uint32_t ta, uint32_t tb, float (&x)[8], float (&y)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, [%17];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(y[0]), "=f"(y[1]),
        "=f"(y[2]), "=f"(y[3]), "=f"(y[4]), "=f"(y[5]), "=f"(y[6]), "=f"(y[7])
      : "r"(ta), "r"(tb)
      : "memory");
}

// FP16 products in batches: one statement of straight code, so that an operand
// costs one addition on its base.  (A product at a time came to about 60 cycles of a
// single warp's issue, as long as the product itself.)
#define BSQ_T5_F16_SS(OFF, ACC)                              \
  "add.u64 a, %1, " #OFF ";\n\tadd.u64 b, %2, " #OFF ";\n\t" \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, " ACC ";\n\t"
// D (128 x N, FP32) = A B^T, K = 64 KBLOCKS: operand blocks of 64 columns 16384 bytes apart, both in
// shared memory with the 128-byte swizzle.
template <int KBLOCKS>
__device__ __forceinline__ void t5_mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t lead) {
  if constexpr (KBLOCKS == 1)
    asm volatile("{\n\t.reg .pred z, o, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.ne.b32 z, 0, 0;\n\tsetp.eq.b32 o, 0, 0;\n\t"
                 BSQ_T5_F16_SS(0, "z") BSQ_T5_F16_SS(2, "o") BSQ_T5_F16_SS(4, "o") BSQ_T5_F16_SS(6, "o") "}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(lead) : "memory");
  else
    asm volatile("{\n\t.reg .pred z, o, q;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 q, %4, 0;\n\tsetp.ne.b32 z, 0, 0;\n\tsetp.eq.b32 o, 0, 0;\n\t"
                 BSQ_T5_F16_SS(0, "z") BSQ_T5_F16_SS(2, "o") BSQ_T5_F16_SS(4, "o") BSQ_T5_F16_SS(6, "o")
                 BSQ_T5_F16_SS(1024, "o") BSQ_T5_F16_SS(1026, "o") BSQ_T5_F16_SS(1028, "o") BSQ_T5_F16_SS(1030, "o") "}"
                 ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(lead) : "memory");
}
#undef BSQ_T5_F16_SS
#define BSQ_T5_F16_TS(AOFF, BOFF, ACC)                        \
  "add.u32 a, %1, " #AOFF ";\n\tadd.u64 b, %2, " #BOFF ";\n\t" \
  "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, " ACC ";\n\t"
// D (128 x N, FP32) (+)= A B, K = 64: A from tensor memory (packed pairs, 8 columns per 16), B rows of
// K 128 bytes apart.
__device__ __forceinline__ void t5_mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate, uint32_t lead) {
  asm volatile("{\n\t.reg .pred p, o, q;\n\t.reg .b32 a;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\tsetp.eq.b32 o, 0, 0;\n\t"
               BSQ_T5_F16_TS(0, 0, "p") BSQ_T5_F16_TS(8, 128, "o") BSQ_T5_F16_TS(16, 256, "o") BSQ_T5_F16_TS(24, 384, "o") "}"
               ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(lead) : "memory");
}
#undef BSQ_T5_F16_TS
// Its instruction descriptor, M = 128: FP32 sums (4), FP16 operands (0 at 7
// and 10), the second operand N-major (16), N >> 3 at 17, M >> 4 at 24.
__host__ __device__ constexpr uint32_t t5_idesc_f16(uint32_t n, bool b_n_major) {
  return (1u << 4) | ((b_n_major ? 1u : 0u) << 16) | ((n >> 3) << 17) | (8u << 24);
}
// N-major operand tile with the 128-byte swizzle: rows (of K) of 64 elements of
// N, groups of 8 rows 1024 bytes apart (stride offset), the next 64 elements of N
// `lead_bytes` on (leading offset).
__device__ __forceinline__ uint64_t t5_desc_sw128_n(uint32_t saddr, uint32_t lead_bytes) {
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead_bytes >> 4) << 16) |
         (static_cast<uint64_t>(64) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// 32 columns of this thread's tensor-memory lane, waited for.
__device__ __forceinline__ void t5_ld32(uint32_t taddr, float (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]),
        "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15]), "=f"(x[16]), "=f"(x[17]), "=f"(x[18]),
        "=f"(x[19]), "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]), "=f"(x[24]), "=f"(x[25]), "=f"(x[26]), "=f"(x[27]),
        "=f"(x[28]), "=f"(x[29]), "=f"(x[30]), "=f"(x[31])
      : "r"(taddr)
      : "memory");
}
// 16 columns, waited for, and back.
__device__ __forceinline__ void t5_ld16(uint32_t taddr, float (&x)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]),
        "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void t5_st16f(uint32_t taddr, const float (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
          taddr),
      "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]), "f"(x[8]), "f"(x[9]), "f"(x[10]),
      "f"(x[11]), "f"(x[12]), "f"(x[13]), "f"(x[14]), "f"(x[15])
      : "memory");
}
// The same without the wait; t5_ld32_wait on the same registers (once no other
// load matters) comes before their first use.
__device__ __forceinline__ void t5_ld32_async(uint32_t taddr, float (&x)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3]), "=f"(x[4]), "=f"(x[5]), "=f"(x[6]), "=f"(x[7]), "=f"(x[8]), "=f"(x[9]),
        "=f"(x[10]), "=f"(x[11]), "=f"(x[12]), "=f"(x[13]), "=f"(x[14]), "=f"(x[15]), "=f"(x[16]), "=f"(x[17]), "=f"(x[18]),
        "=f"(x[19]), "=f"(x[20]), "=f"(x[21]), "=f"(x[22]), "=f"(x[23]), "=f"(x[24]), "=f"(x[25]), "=f"(x[26]), "=f"(x[27]),
        "=f"(x[28]), "=f"(x[29]), "=f"(x[30]), "=f"(x[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void t5_ld32_wait(float (&x)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(x[0]), "+f"(x[1]), "+f"(x[2]), "+f"(x[3]), "+f"(x[4]), "+f"(x[5]), "+f"(x[6]), "+f"(x[7]), "+f"(x[8]),
                 "+f"(x[9]), "+f"(x[10]), "+f"(x[11]), "+f"(x[12]), "+f"(x[13]), "+f"(x[14]), "+f"(x[15]), "+f"(x[16]),
                 "+f"(x[17]), "+f"(x[18]), "+f"(x[19]), "+f"(x[20]), "+f"(x[21]), "+f"(x[22]), "+f"(x[23]), "+f"(x[24]),
                 "+f"(x[25]), "+f"(x[26]), "+f"(x[27]), "+f"(x[28]), "+f"(x[29])
               :
               : "memory");
  asm volatile("" : "+f"(x[30]), "+f"(x[31]));
}
__device__ __forceinline__ void t5_st16(uint32_t taddr, const uint32_t (&x)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
          taddr),
      "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7]), "r"(x[8]), "r"(x[9]), "r"(x[10]),
      "r"(x[11]), "r"(x[12]), "r"(x[13]), "r"(x[14]), "r"(x[15])
      : "memory");
}
__device__ __forceinline__ void t5_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Contiguous copy of `bytes` (a multiple of 16) into shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)),
               "l"(src), "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

// Two FP32 at a time.
__device__ __forceinline__ float2 fma_f32x2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tadd.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}

// Order generic-proxy accesses before and after it with the async proxy's (TMA).
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }

__device__ __forceinline__ uint32_t ld_acquire(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

__device__ __forceinline__ void st_release(uint32_t* p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}

// Adds and returns the old value; orders this thread's accesses, and those
// it has seen through a barrier, before and after it (GPU scope).
__device__ __forceinline__ uint32_t atomic_add_acq_rel(uint32_t* p, uint32_t v) {
  uint32_t old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
  return old;
}

// Barrier of `threads` threads of the block (id 1..15).
__device__ __forceinline__ void named_sync(int id, int threads) {
  __syncwarp();  // the barrier wants whole warps
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

}  // namespace bsq
