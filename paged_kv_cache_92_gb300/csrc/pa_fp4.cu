// The 4-bit KV cache for sm_103a: the quantising KV write and the read-back.
//
// The pages say only that paging combines with KV quantisation ("PagedAttention"
// glossary page, §What paging costs). The format is this library's:
//  - a (block, KV head) tile is block_size rows of E2M1 codes, head_dim / 2
//    bytes each (element 2i in the low nibble of byte i), followed by
//    block_size rows of E4M3 group scales, one per 16 elements; 9/16 byte an
//    element, and one contiguous copy a tile;
//  - value = code * group scale * scale[h], scale[h] one float per KV head;
//  - write: with a the largest magnitude of a group,
//      group scale = E4M3(fl(a / fl(6 scale[h])))   (nearest even, at most 448)
//      step        = fl(group scale * scale[h])
//      code        = E2M1(fl(x / step))             (nearest even, at most +-6)
//    where fl rounds to float. A group whose scale rounds to zero gets zero
//    codes; one that holds a NaN gets the NaN scale, so the NaN stays visible.
// Six is the largest E2M1 magnitude, so the group's largest element lands on
// the top code; a product of a 2-bit and a 4-bit significand is exact in f16,
// which is what the decode relies on.
//
// Both kernels are bound by memory traffic: one thread per group of 16
// elements reads or writes 32 bytes of bf16 and 9 bytes of cache. The codes of
// a row are written by head_dim / 16 neighbouring threads, 8 bytes each. Neither
// reaches the copy rate: past some 3 us of start and end (7 k tokens of 8 heads,
// d 128, take 10.9 and 9.9 us, 29 k 34.3 and 31.1) they move 4.8 and 5.3 TB/s, with
// two thirds of the issue slots busy -- the index of a thread is divided by the
// groups of a row and by the heads, each of the 32 elements by its step -- and each
// thread's one round of loads before its work. At a decode step's sizes the launch
// is what they cost (64 tokens: 4.6 us for the two of them, against 0.1 us of
// traffic).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_device.cuh"
#include "pa_fp4.h"
#include "pa_mma.cuh"
#include "pa_ordered.cuh"

namespace pa {
namespace {

__device__ unsigned int g_fp4_errors;

// E2M1 codes of 8 values, nearest even, saturating; element i in nibble i.
__device__ __forceinline__ uint32_t to_e2m1x8(const float* y) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return w;
}

// Largest magnitude of 16 bf16 values, NaN if one of them is.
__device__ __forceinline__ float group_max(const uint4& lo, const uint4& hi) {
  const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  uint32_t m = w[0] & 0x7FFF7FFFu;
#pragma unroll
  for (int i = 1; i < 8; ++i)
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7FFF7FFFu));
  const float a = dev::bf16_lo(m), b = dev::bf16_hi(m);
  return a != a ? a : (b != b ? b : fmaxf(a, b));
}

// fl(x / step) where it lies within the grid (below 8), with inv = fl(1 / step):
// one correction by the remainder, which is exact in a fused multiply-add
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990). Beyond, the code saturates whatever the last place, and
// an infinity stays one. The sign is that of x, zeros included.
__device__ __forceinline__ float quotient(float x, float step, float inv) {
  const float q0 = __fmul_rn(x, inv);
  const float q = __fmaf_rn(__fmaf_rn(-q0, step, x), inv, q0);
  return copysignf(fabsf(q0) < 8.0f ? q : q0, x);
}

struct Fp4Rows {
  int64_t num_groups;  // tokens * num_kv_heads * groups of a row
  int64_t num_slots;
  int num_kv_heads, groups, bs_log2;  // groups = head_dim / 16
};

// Where group c of row (token t, KV head h) sits: byte offsets of its codes
// and of its scale.
__device__ __forceinline__ void fp4_place(const Fp4Rows& r, int64_t slot, int h, int c,
                                          int64_t& codes, int64_t& scale) {
  const int BS = 1 << r.bs_log2;
  const int off = int(slot & (BS - 1));
  const int64_t tile = ((slot >> r.bs_log2) * r.num_kv_heads + h) * (int64_t(BS) * r.groups * 9);
  codes = tile + int64_t(off) * r.groups * 8 + c * 8;
  scale = tile + int64_t(BS) * r.groups * 8 + off * r.groups + c;
}

// 16 bf16 values quantised with the head's scale: their codes and group scale.
__device__ __forceinline__ uint2 quantise_group(const uint4& lo, const uint4& hi, float s,
                                                uint8_t& sf) {
  float x[16];
  {
    float a[8], b[8];
    dev::unpack8(lo, a);
    dev::unpack8(hi, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = a[i];
      x[i + 8] = b[i];
    }
  }
  // the largest magnitude, two elements at a time; a NaN stays one
  const float amax = group_max(lo, hi);
  const bool nan = amax != amax;
  sf = nan ? 0x7F : dev::to_e4m3(__fdiv_rn(amax, __fmul_rn(6.0f, s)));
  uint2 codes;
  if (sf == 0 || nan) {
    // no step to divide by: zeros that keep their sign
    codes.x = codes.y = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      codes.x |= (__float_as_uint(x[i]) >> 31) << (4 * i + 3);
      codes.y |= (__float_as_uint(x[i + 8]) >> 31) << (4 * i + 3);
    }
  } else {
    const float step = __fmul_rn(dev::from_e4m3(sf), s);
    const float inv = __frcp_rn(step);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = quotient(x[i], step, inv);
    codes.x = to_e2m1x8(x);
    codes.y = to_e2m1x8(x + 8);
  }
  return codes;
}

// One thread per group, of K and of V: their loads are in flight together
// (four prompts of 1.5 to 2 k tokens, 8 heads, dim 128: 11.8 us; one thread for each
// 13.4 us). No pointer is __restrict__ here: what a kernel reads through its
// read-only path must not change from its start on, and this one may start
// before the preceding kernel has written it.
__global__ void __launch_bounds__(256)
    reshape_and_cache_fp4_kernel(const uint4* k_new, const uint4* v_new, uint8_t* k_cache,
                                 uint8_t* v_cache, const int64_t* slot_mapping,
                                 const float* k_scale, const float* v_scale, Fp4Rows r,
                                 AppendCheck check) {
  dev::griddep_enter();
  const int64_t idx = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= r.num_groups) return;
  const int c = int(idx % r.groups);
  const int64_t row = idx / r.groups;  // t * num_kv_heads + h
  const int h = int(row % r.num_kv_heads);
  const int64_t t = row / r.num_kv_heads;
  const int64_t slot = slot_mapping[t];
  const uint4 k0 = k_new[idx * 2], k1 = k_new[idx * 2 + 1];
  const uint4 v0 = v_new[idx * 2], v1 = v_new[idx * 2 + 1];
  const float ks = k_scale[h], vs = v_scale[h];
  if (slot < 0) return;  // padding token: no write
  const bool report = h == 0 && c == 0;
  if (slot >= r.num_slots) {
    if (report) atomicOr(&g_fp4_errors, PA_DEVERR_SLOT);
    return;
  }
  if (check.block_tables) {
    // decode step: token t is new token i of sequence b, written only at its
    // position's slot (the last q_len tokens of the sequence)
    const int64_t b = t / check.q_len;
    const int i = int(t - b * check.q_len);
    const int L = min(check.context_lens[b], check.cap);
    if (L < check.q_len) return;  // no room for the new tokens: the decode flags the length
    const int pos = L - check.q_len + i;
    const int e = check.block_tables[b * check.max_blocks_per_seq + (pos >> r.bs_log2)];
    if (slot != (int64_t(e) << r.bs_log2) + (pos & ((1 << r.bs_log2) - 1))) {
      if (report) atomicOr(&g_fp4_errors, PA_DEVERR_APPEND_SLOT);
      return;
    }
  }
  int64_t at, at_scale;
  fp4_place(r, slot, h, c, at, at_scale);
  uint8_t sf;
  *reinterpret_cast<uint2*>(k_cache + at) = quantise_group(k0, k1, ks, sf);
  k_cache[at_scale] = sf;
  *reinterpret_cast<uint2*>(v_cache + at) = quantise_group(v0, v1, vs, sf);
  v_cache[at_scale] = sf;
}

// Codes of 16 elements to bf16: fl(code * group scale * scale[h]) rounded to
// bf16. The product of code and group scale is exact.
__device__ __forceinline__ void read_group(const uint2& codes, float sf, float s, uint4* dst) {
  uint32_t out[8];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t p[4];
    dev::e2m1x8_to_f16(half ? codes.y : codes.x, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&p[i]));
      const __nv_bfloat162 b = __floats2bfloat162_rn(__fmul_rn(f.x * sf, s), __fmul_rn(f.y * sf, s));
      out[half * 4 + i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

// One thread per group of a row read back; blockIdx.y = 0 reads K, 1 reads V.
// (A thread for both, as in the write, took 10.3 us on those prompts where this
// takes 9.2: here the stores are what is wide.)
__global__ void __launch_bounds__(256)
    gather_fp4_kernel(const uint8_t* k_cache, const uint8_t* v_cache, uint4* k_out, uint4* v_out,
                      const int64_t* slot_mapping, const float* k_scale, const float* v_scale,
                      Fp4Rows r) {
  dev::griddep_enter();
  const int64_t idx = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
  if (idx >= r.num_groups) return;
  const bool is_v = blockIdx.y != 0;
  const int c = int(idx % r.groups);
  const int64_t row = idx / r.groups;
  const int h = int(row % r.num_kv_heads);
  const int64_t slot = slot_mapping[row / r.num_kv_heads];
  const float s = (is_v ? v_scale : k_scale)[h];
  uint4* dst = (is_v ? v_out : k_out) + idx * 2;
  if (slot < 0 || slot >= r.num_slots) {  // padding, or no such row: zeros
    if (slot >= 0 && h == 0 && c == 0 && !is_v) atomicOr(&g_fp4_errors, PA_DEVERR_SLOT);
    dst[0] = dst[1] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  const uint8_t* cache = is_v ? v_cache : k_cache;
  int64_t at, at_scale;
  fp4_place(r, slot, h, c, at, at_scale);
  const uint2 codes = *reinterpret_cast<const uint2*>(cache + at);
  read_group(codes, dev::from_e4m3(cache[at_scale]), s, dst);
}

Fp4Rows fp4_rows(int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                 int32_t num_blocks) {
  Fp4Rows r;
  r.groups = head_dim / 16;
  r.num_groups = int64_t(num_tokens) * num_kv_heads * r.groups;
  r.num_slots = int64_t(num_blocks) * block_size;
  r.num_kv_heads = num_kv_heads;
  r.bs_log2 = log2_of(block_size);
  return r;
}

}  // namespace

int launch_reshape_and_cache_fp4(const void* k_new, const void* v_new, void* k_cache,
                                 void* v_cache, const int64_t* slot_mapping, const float* k_scale,
                                 const float* v_scale, int32_t num_tokens, int32_t num_kv_heads,
                                 int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                 void* stream, const AppendCheck& check) {
  const Fp4Rows r = fp4_rows(num_tokens, num_kv_heads, head_dim, block_size, num_blocks);
  if (r.num_groups == 0) return int(cudaSuccess);
  const int threads = 256;
  const unsigned grid = unsigned((r.num_groups + threads - 1) / threads);
  return launch_ordered(reshape_and_cache_fp4_kernel, dim3(grid), threads, 0,
                        static_cast<cudaStream_t>(stream), 1, static_cast<const uint4*>(k_new),
                        static_cast<const uint4*>(v_new), static_cast<uint8_t*>(k_cache),
                        static_cast<uint8_t*>(v_cache), slot_mapping, k_scale, v_scale, r, check);
}

int launch_gather_fp4(const void* k_cache, const void* v_cache, void* k_out, void* v_out,
                      const int64_t* slot_mapping, const float* k_scale, const float* v_scale,
                      int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                      int32_t block_size, int32_t num_blocks, void* stream) {
  const Fp4Rows r = fp4_rows(num_tokens, num_kv_heads, head_dim, block_size, num_blocks);
  if (r.num_groups == 0) return int(cudaSuccess);
  const int threads = 256;
  const dim3 grid(unsigned((r.num_groups + threads - 1) / threads), 2);
  return launch_ordered(gather_fp4_kernel, grid, threads, 0, static_cast<cudaStream_t>(stream), 1,
                        static_cast<const uint8_t*>(k_cache),
                        static_cast<const uint8_t*>(v_cache), static_cast<uint4*>(k_out),
                        static_cast<uint4*>(v_out), slot_mapping, k_scale, v_scale, r);
}

int read_and_clear_fp4_errors(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp4_errors, sizeof(v));
  if (e != cudaSuccess) return int(e);
  if (v != 0) e = cudaMemcpyToSymbol(g_fp4_errors, &zero, sizeof(zero));
  *flags = v;
  return int(e);
}

}  // namespace pa
