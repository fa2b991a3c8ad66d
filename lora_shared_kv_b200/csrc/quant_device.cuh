// Device helpers of the 8-bit cache kernels: codes to fp16, wide loads, MMA forms.
#pragma once

#include <stdint.h>

#include "common.cuh"

namespace lrkv {

// Four codes (bytes 0 .. 3 of w) as two fp16 pairs, exact.
//   e4m3: lo = bytes 0, 1 and hi = bytes 2, 3; one conversion per pair.
//   int8: lo = bytes 0, 2 and hi = bytes 1, 3: fp16 0x6400 | u is 1024 + u, so with
//         u = code + 128 the subtraction of 1152 leaves the code.  (Three integer
//         operations: one masks and flips bytes 0, 2 in place, two flip and permute
//         bytes 1, 3.  A shift in place of the permutation took the 32 x 8k decode from
//         58.3 to 60.0 us, a multiplication's high word 62.8.)
template <int FMT>
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (FMT == LRKV_Q_E4M3) {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  } else {
    lo = (w & 0x00FF00FFu) ^ 0x64806480u;
    hi = __byte_perm(w ^ 0x80808080u, 0x64646464u, 0x4341);
    asm("sub.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
    asm("sub.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
  }
}
// Which byte of w element `i` (0, 1: of lo; 2, 3: of hi) comes from.
template <int FMT>
__host__ __device__ constexpr int code_byte(int i) {
  return FMT == LRKV_Q_E4M3 ? i : (i & 1) * 2 + (i >> 1);
}

// 16 bytes that are read once.
__device__ __forceinline__ uint4 ld_stream(const void* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void st_shared_zero16(uint32_t addr) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(addr), "r"(0u) : "memory");
}

// Two 16 x 16 blocks of bytes, transposed: lane l gets rows 4 (l % 4) .. + 3 of
// columns l / 4 (r0, r2) and 8 + l / 4 (r1, r3) of the first and second block;
// lane i gives the address of row i % 16 of block i / 16.
__device__ __forceinline__ void ldsm_b8_x2_t(uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

// D += A * B, A 16x16 (row), B 16x8 (col), fp16 in, fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A * B (no accumulator to clear).
__device__ __forceinline__ void mma_f16_16816_first(float* d, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                    uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace lrkv
