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

// Pairs of floats in one instruction, each rounded as by itself.
__device__ __forceinline__ float2 sub_pair(float2 a, const float (&b)[2]) {
  float2 y;
  asm("{\n\t.reg .b64 x, z;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 z, {%4, %5};\n\t"
      "sub.rn.f32x2 x, x, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b[0]), "f"(b[1]));
  return y;
}
// a * b + c
__device__ __forceinline__ float2 fma_pair(float2 a, const float (&b)[2], float c) {
  float2 y;
  asm("{\n\t.reg .b64 x, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 z, {%4, %5};\n\tmov.b64 w, {%6, %6};\n\t"
      "fma.rn.f32x2 x, x, z, w;\n\tmov.b64 {%0, %1}, x;\n\t}"
      : "=f"(y.x), "=f"(y.y)
      : "f"(a.x), "f"(a.y), "f"(b[0]), "f"(b[1]), "f"(c));
  return y;
}

// Key row of a 16-key tile that a thread with row index g (0..7) reads (its
// other row is 8 further on). With 64-byte rows, rows 2i and 2i+1 differ in
// parity, so the 16-byte reads of K are free of bank conflicts, and rows
// 0, 2, 4, 6 fall two and two on either parity, which halves those of V.
__device__ __forceinline__ int key_row(int g) { return g ^ (g >> 2); }

}  // namespace dev
}  // namespace pa

// ---------------------------------------------------------------------------
// Cached key rows times query rows. FMT is the cache's type (PA_KV_BF16,
// PA_KV_FP8_E4M3, PA_KV_FP4_E2M1). The order of elements in the contraction is
// free as long as both operands share it: a lane (t = lane % 4) takes every
// fourth run of KeyRow::E elements of a row, one 16-byte read of the cache (8
// bytes of a 4-bit row of 64), and the queries follow.
// ---------------------------------------------------------------------------
namespace pa {
namespace dev {

template <int FMT, int D>
struct KeyRow {
  static constexpr int E = FMT == 0 ? 8 : (FMT == 1 ? 16 : D / 4);  // elements of a run
  static constexpr int BYTES = FMT == 0 ? 2 * D : (FMT == 1 ? D : D / 2);  // of a row (its codes)
  static constexpr int RUN = BYTES * E / D;           // bytes of a run: 16, or 8
  static constexpr int RUNS = D / (4 * E);            // runs of a lane
  static constexpr int STEPS = D / 16;                // products of 16 elements
  static constexpr int SCALES = FMT == 2 ? D / 16 : 0;  // scale bytes of a row
  // bytes of one (block, KV head) tile, by block size
  __host__ __device__ static constexpr int tile(int bs) { return bs * (BYTES + SCALES); }

  uint32_t w[RUNS * RUN / 4];
  uint32_t sc[D / 64];  // 4-bit: the group scales as f16 pairs

  // The row whose first byte for this lane is `row` (RUN * (lane % 4) into the
  // row), its scales for this lane at `s` (D / 64 * (lane % 4) into its scales).
  __device__ __forceinline__ void load(const unsigned char* row, const unsigned char* s) {
#pragma unroll
    for (int j = 0; j < RUNS; ++j) {
      const unsigned char* at = row + 4 * j * RUN;
      if constexpr (RUN == 16) {
        const uint4 x = *reinterpret_cast<const uint4*>(at);
        w[4 * j] = x.x; w[4 * j + 1] = x.y; w[4 * j + 2] = x.z; w[4 * j + 3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2*>(at);
        w[2 * j] = x.x; w[2 * j + 1] = x.y;
      }
    }
    if constexpr (FMT == 2) {
      if constexpr (D == 128) {
        const uint32_t y = e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(s));
        sc[0] = __byte_perm(y, 0, 0x1010);
        sc[1] = __byte_perm(y, 0, 0x3232);
      } else {
        sc[0] = __byte_perm(e4m3x2_to_f16(*s), 0, 0x1010);
      }
    }
  }
  // elements [8 c, 8 c + 8) of the lane's list as pairs (two products' worth)
  __device__ __forceinline__ void pairs(int c, uint32_t (&x)[4]) const {
    if constexpr (FMT == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = w[4 * c + j];
    } else if constexpr (FMT == 1) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = e4m3x2_to_f16((w[2 * c + j / 2] >> (16 * (j & 1))) & 0xffffu);
    } else {
      e2m1x8_to_f16(w[c], x);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = mul_f16x2(x[j], sc[c / 2]);
    }
  }
};

// s[nt] (16 keys x 8 columns) += keys * queries^T; `lo` holds the lane's rows
// for fragment rows 0..7, `hi` those for 8..15.
template <int FMT, int D, int NT>
__device__ __forceinline__ void key_product(float (&s)[NT][4], const KeyRow<FMT, D>& lo,
                                            const KeyRow<FMT, D>& hi,
                                            const uint32_t (&qf)[NT][D / 16][2]) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t x[4], y[4];
    lo.pairs(c, x);
    hi.pairs(c, y);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t(&b)[2] = qf[nt][2 * c + k];
        if constexpr (FMT == 0)
          mma_bf16_regs(s[nt], x[2 * k], y[2 * k], x[2 * k + 1], y[2 * k + 1], b[0], b[1]);
        else
          mma_f16(s[nt], x[2 * k], y[2 * k], x[2 * k + 1], y[2 * k + 1], b[0], b[1]);
      }
  }
}

// The same for one column tile whose queries lie in shared memory: entry
// [c][lane] of `qs` holds the lane's pairs of products 2c and 2c + 1.
template <int FMT, int D>
__device__ __forceinline__ void key_product_shared(float (&s)[4], const KeyRow<FMT, D>& lo,
                                                   const KeyRow<FMT, D>& hi, const uint4* qs) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint32_t x[4], y[4];
    lo.pairs(c, x);
    hi.pairs(c, y);
    const uint4 b = qs[c * 32];
    mma_f16(s, x[0], y[0], x[1], y[1], b.x, b.y);
    mma_f16(s, x[2], y[2], x[3], y[3], b.z, b.w);
  }
}

// The lane's part of a query row (t = lane % 4), in the order of its key
// elements; `on` false: a row of zeros (`row` is read all the same).
template <int FMT, int D>
__device__ __forceinline__ void query_load(const __nv_bfloat16* row, bool on, int t,
                                           uint4 (&raw)[D / 32]) {
  using R = KeyRow<FMT, D>;
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {  // 8 elements of the lane's list
    const int e = 8 * c;
    const uint4 x =
        *reinterpret_cast<const uint4*>(row + (4 * (e / R::E) + t) * R::E + e % R::E);
    raw[c] = make_uint4(on ? x.x : 0u, on ? x.y : 0u, on ? x.z : 0u, on ? x.w : 0u);
  }
}

// A query row as the products' B operand; all lanes call together. bf16 rows
// stay as they are and the result is 1. The others are scaled to f16 by a power
// of two that brings the row's largest magnitude into [2^12, 2^13), exactly for
// every element within 2^-29 of it (8 significant bits above f16's last, 2^-24),
// and its inverse is returned.
template <int FMT, int D>
__device__ __forceinline__ float query_fragment(const uint4 (&raw)[D / 32],
                                                uint32_t (&qf)[D / 16][2]) {
  if constexpr (FMT == 0) {
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      qf[2 * c][0] = raw[c].x; qf[2 * c][1] = raw[c].y;
      qf[2 * c + 1][0] = raw[c].z; qf[2 * c + 1][1] = raw[c].w;
    }
    return 1.0f;
  } else {
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      float f[8];
      unpack8(raw[c], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) amax = fmaxf(amax, fabsf(f[i]));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // amax < 2^e from its exponent field; zeros, infinities and NaN keep 2^13
    const int field = int(__float_as_uint(amax) >> 23);
    const int e = field == 0 || field == 255 ? (amax > 0.0f && field == 0 ? -100 : 0)
                                             : max(field - 126, -100);
    const float a = __uint_as_float(uint32_t(13 - e + 127) << 23);  // 2^(13 - e): normal
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      float f[8];
      unpack8(raw[c], f);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        qf[2 * c + i / 2][i & 1] = pack_f16(f[2 * i] * a, f[2 * i + 1] * a);
    }
    return __uint_as_float(uint32_t(e - 13 + 127) << 23);
  }
}

}  // namespace dev
}  // namespace pa
