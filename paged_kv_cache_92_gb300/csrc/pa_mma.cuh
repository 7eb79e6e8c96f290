// Warp-level building blocks shared by the 4-bit decode and the token-weight
// kernels: the m16n8k16 product with its operands in registers, the 4-bit and
// 8-bit codes converted to f16 pairs, the 8x8 transpose, and the fragments
// that these kernels build from cached rows.
//
// Why operands in registers. A 4-bit cache feeds an SM about 23 bytes a clock
// at full HBM rate, which is 41 elements; as f16 operands in shared memory
// those are 83 bytes written and 83 read back by the matrix unit, more than
// the 128 bytes a clock that shared memory moves. Converted in registers the
// element never returns there, and the products need about a third of the
// warp-level matrix rate.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "pa_device.cuh"

namespace pa {
namespace dev {

// C (16 x 8, fp32) += A (16 x 16) * B (16 x 8). With g = lane / 4 and
// t = lane % 4 a thread holds A rows g and g + 8 at k = 2t, 2t+1 (a0, a1) and
// 2t+8, 2t+9 (a2, a3), B at the same k for column g, and C rows g (c0, c1)
// and g + 8 (c2, c3) at columns 2t, 2t+1.
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16_regs(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 8x8 matrix of 16-bit elements, row g in lanes 4g..4g+3, transposed.
__device__ __forceinline__ uint32_t transpose_8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The four bytes of a word, each two E2M1 codes (low nibble first), as f16 pairs (exact).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two E4M3 codes (low byte first) as an f16 pair (exact).
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t c) {
  uint32_t h;
  asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}"
      : "=r"(h)
      : "r"(c));
  return h;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
// a in the low half
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  uint32_t y;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(y) : "f"(b), "f"(a));
  return y;
}

// Key row of a 16-key tile that a thread with row index g (0..7) reads (its
// other row is 8 further on). With 64-byte rows, rows 2i and 2i+1 differ in
// parity, so the 16-byte reads of K are free of bank conflicts, and rows
// 0, 2, 4, 6 fall two and two on either parity, which halves those of V.
__device__ __forceinline__ int key_row(int g) { return g ^ (g >> 2); }

}  // namespace dev
}  // namespace pa
