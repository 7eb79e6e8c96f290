// Which blocks of a long context a step has to read, for sm_103a: bounds of every
// block's keys, an upper bound of the scores that they can reach, and the choice of
// the best under a budget. The attention over them is in pa_decode_selected.cu. The
// pages stop at reading the whole context; the policy is this library's.
//
// For a block whose keys lie between lo and hi, element by element,
//   q . k = sum_d q_d k_d <= sum_d max(q_d lo_d, q_d hi_d) = q+ . hi + q- . lo
// with q+ and q- the positive and the negative part of q: a block that scores low
// holds no key that this query would weigh much.
//
//  * block_bounds_kernel: one warp per (block, KV head). Minimum and maximum of pairs
//    in bf16, or in f16 for the 8-bit and 4-bit codes (times group scales), which are
//    exact in either: no rounding. Bound by the bytes of K.
//  * block_scores_kernel: the two products as one of length 2 d on the matrix units,
//    A the bounds (16 blocks a tile, read from memory straight into fragments: the
//    order of a contraction is free, so a lane takes 16-byte runs), B the query rows
//    of a KV head. fp32 sums of exact products. Bound by the bytes of the bounds.
//  * block_select_kernel: one CTA per (sequence, KV head), or a cluster of four for few long
//    rows, with the row's scores as ordered 32-bit keys in registers; the key of the budget's
//    rank is found by histograms in shared memory, the first over the range that the scores
//    span, in bins of equal widths, the next over the bin that holds it, until that has 32
//    keys or fewer, which are ranked one against the other (mostly after one histogram). Ties
//    go to the lowest index through ranks. Bound by latency: straight code without branches a
//    key, since an instruction runs once a warp.
//
// Measured (GB300, in a graph; the floor is the bytes at the copy rate of 6.68 TB/s):
//  * bounds, 8 KV heads, d 128: the last blocks of 64 sequences 1.8 us; 16 prompts of 8 to
//    32 k tokens, bf16, 102.5 us (floor 106.9: a copy writes as much as it reads), 8-bit 62.3
//    (59.4); 32 contexts of 4 to 16 k, 4-bit, block size 32, 49.5 us (35.8): the ALU is 83 % busy, with
//    a conversion, a minimum and a maximum a pair of codes. Tried: several tiles' loads in
//    flight (103.8 and 52.9), the next tile's ahead of this one's work (115 and 64.7).
//  * scores: 64 contexts of 8 to 32 k, block size 16, 32 / 8 heads 53.9 us (52.1); two of
//    64 to 128 k with four new tokens, 64 / 8 heads 14.5 us (9.2): a warp's chain of length,
//    table, rows twice over, and 1.7 waves of CTAs. Query rows of several tiles loaded from
//    memory for every 16 blocks: 23.2. 32 contexts of 32 to 128 k, 64 / 8 heads: one new token
//    149 us, four 109.5 (96): the form for one tile of query rows is far from memory there.
//  * choice: 512 rows of up to 2,048 blocks, 128 kept 5.4 us (length, scores, the histogram,
//    its scan, the last bin and the lists take 1,100 to 1,700 cycles each), 32 rows of up to
//    16,384, 512 kept 6.5 us. Histograms over the keys' bits only: 8.6 and 9.0; bit by bit:
//    10.9 and 18.8; a warp's equal bins counted at once: 10.7 for the latter (equal scores
//    cost a third more without). The next kernel's CTAs come with this one's end: dispatched
//    at the start they take the room unevenly (7.0 for 5.4). Many long rows are far from their
//    bytes: of 16,000 blocks, 256 kept, 304 rows 16.2 us (3.0), 512 rows 30.8 (5.0), 1,024 rows
//    57.5 (10.0): one CTA of 32 warps an SM, whose steps are latencies that nothing overlaps.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_blocks.h"
#include "pa_device.cuh"
#include "pa_mma.cuh"
#include "pa_ordered.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned int g_blocks_errors;

// ---------------------------------------------------------------- bounds

constexpr int BOUND_WARPS = 4;

struct Bounds {
  const unsigned char* k_cache;
  __nv_bfloat16* bounds;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* old_lens;  // or nullptr: zeros
  int max_blocks_per_seq, num_kv_heads, num_blocks, per_seq;
};

template <int FMT>
__device__ __forceinline__ void lower(uint32_t& a, uint32_t b) {
  if constexpr (FMT == PA_KV_BF16)
    asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  else
    asm("min.NaN.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
}
template <int FMT>
__device__ __forceinline__ void raise(uint32_t& a, uint32_t b) {
  if constexpr (FMT == PA_KV_BF16)
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
  else
    asm("max.NaN.f16x2 %0, %0, %1;" : "+r"(a) : "r"(b));
}
// A pair of f16 as a pair of bf16 (exact for what the codes can hold).
__device__ __forceinline__ uint32_t bf16_of_f16(uint32_t x) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x));
  const __nv_bfloat162 y = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// Lanes take chunks of the rows: LPR lanes a row, 32 / LPR rows at a time. 16 bytes, of
// 4-bit codes 8 (a group of 16 elements): those are bound by the ALU, and the fewer
// elements a lane has of more rows, the fewer have to meet between lanes.
template <int FMT, int D, int BS>
__global__ void __launch_bounds__(BOUND_WARPS * 32) block_bounds_kernel(const Bounds P) {
  constexpr int ROWB = FMT == PA_KV_BF16 ? 2 * D : (FMT == PA_KV_FP8_E4M3 ? D : D / 2);
  constexpr int SCALES = FMT == PA_KV_FP4_E2M1 ? D / 16 : 0;
  constexpr int TILE = BS * (ROWB + SCALES);
  constexpr int CHUNK = FMT == PA_KV_FP4_E2M1 ? 8 : 16, WORDS = CHUNK / 4;
  constexpr int LPR = ROWB / CHUNK, RPL = 32 / LPR;    // lanes of a row, rows of a load
  constexpr int LOADS = (BS + RPL - 1) / RPL;
  constexpr int PAIRS = FMT == PA_KV_BF16 ? 4 : 8;     // of a chunk
  dev::griddep_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  const int L = P.context_lens[b], old = P.old_lens != nullptr ? max(P.old_lens[b], 0) : 0;
  const int cap = P.max_blocks_per_seq * BS;
  const int end = min(L, cap), first = old / BS, last = (end + BS - 1) / BS;  // the blocks to do
  if (blockIdx.x == 0 && threadIdx.x == 0 && (L > cap || last - first > P.per_seq))
    atomicOr(&g_blocks_errors, PA_DEVERR_CONTEXT_LEN);
  // (without a new token none, though `first` may be a block with tokens: another sequence that
  // shares it may have gained some)
  const int n = old < end ? min(last - first, P.per_seq) : 0;
  const uint32_t heads = uint32_t(P.num_kv_heads), units = uint32_t(n) * heads;
  for (uint32_t u = blockIdx.x * BOUND_WARPS + warp; u < units; u += gridDim.x * BOUND_WARPS) {
    const int k = int(u / heads), head = int(u - k * heads);
    const int j = first + k;
    const int e = P.block_tables[int64_t(b) * P.max_blocks_per_seq + j];
    if (e < 0 || e >= P.num_blocks) {
      if (lane == 0 && head == 0) atomicOr(&g_blocks_errors, PA_DEVERR_TABLE_ENTRY);
      continue;
    }
    const int rows = min(BS, L - j * BS);  // that hold tokens
    const int64_t at = int64_t(e) * P.num_kv_heads + head;
    const unsigned char* tile = P.k_cache + at * TILE;
    const int row0 = lane / LPR, chunk = lane % LPR;
    uint32_t raw[LOADS][WORDS];
    uint8_t sf[LOADS];
    auto load = [&](int i, const unsigned char* codes, const unsigned char* scale) {
      if constexpr (CHUNK == 16) {
        const uint4 y = *reinterpret_cast<const uint4*>(codes);
        raw[i][0] = y.x; raw[i][1] = y.y; raw[i][2] = y.z; raw[i][3] = y.w;
      } else {
        const uint2 y = *reinterpret_cast<const uint2*>(codes);
        raw[i][0] = y.x; raw[i][1] = y.y;
        sf[i] = *scale;
      }
    };
    const unsigned char* scales = tile + BS * ROWB + chunk;
    if (BS >= RPL && rows == BS) {  // addresses apart by constants
#pragma unroll
      for (int i = 0; i < LOADS; ++i)
        load(i, tile + row0 * ROWB + chunk * CHUNK + i * RPL * ROWB,
             scales + row0 * SCALES + i * RPL * SCALES);
    } else {
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int r = min(row0 + i * RPL, rows - 1);  // (a row that counts twice changes nothing)
        load(i, tile + r * ROWB + chunk * CHUNK, scales + r * SCALES);
      }
    }
    uint32_t v[2 * PAIRS];  // least, then largest
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const uint32_t(&w)[WORDS] = raw[i];
      uint32_t x[PAIRS];
      if constexpr (FMT == PA_KV_BF16) {
#pragma unroll
        for (int p = 0; p < 4; ++p) x[p] = w[p];
      } else if constexpr (FMT == PA_KV_FP8_E4M3) {
#pragma unroll
        for (int p = 0; p < 8; ++p) x[p] = dev::e4m3x2_to_f16((w[p / 2] >> (16 * (p & 1))) & 0xffffu);
      } else {
        const uint32_t s = __byte_perm(dev::e4m3x2_to_f16(sf[i]), 0, 0x1010);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t y[4];
          dev::e2m1x8_to_f16(w[c], y);
#pragma unroll
          for (int p = 0; p < 4; ++p) x[4 * c + p] = dev::mul_f16x2(y[p], s);
        }
      }
#pragma unroll
      for (int p = 0; p < PAIRS; ++p) {
        if (i == 0) {
          v[p] = v[PAIRS + p] = x[p];
        } else {
          lower<FMT>(v[p], x[p]);
          raise<FMT>(v[PAIRS + p], x[p]);
        }
      }
    }
    // Over the lanes of a chunk (one per row0). The largest become least of the negated,
    // so that both halves reduce alike: at every exchange a lane keeps half of what it
    // has, until it has 4 pairs, the 16-byte piece row0 % PIECES of the chunk's result.
#pragma unroll
    for (int p = 0; p < PAIRS; ++p) v[PAIRS + p] ^= 0x80008000u;
    constexpr int PIECES = 2 * PAIRS / 4;
    static_assert(PIECES <= RPL, "a lane for every piece");
#pragma unroll
    for (int half = PAIRS, o = LPR * PIECES / 2; half >= 4; half /= 2, o /= 2) {
      const bool upper = lane & o;
#pragma unroll
      for (int p = 0; p < half; ++p) {
        const uint32_t mine = upper ? v[half + p] : v[p], other = upper ? v[p] : v[half + p];
        v[p] = mine;
        lower<FMT>(v[p], __shfl_xor_sync(0xffffffffu, other, o));
      }
    }
#pragma unroll
    for (int o = LPR * PIECES; o < 32; o <<= 1)
#pragma unroll
      for (int p = 0; p < 4; ++p) lower<FMT>(v[p], __shfl_xor_sync(0xffffffffu, v[p], o));
    const bool largest = row0 & (PIECES / 2);
    uint4 piece;
    uint32_t* y = reinterpret_cast<uint32_t*>(&piece);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      y[p] = largest ? v[p] ^ 0x80008000u : v[p];
      if constexpr (FMT != PA_KV_BF16) y[p] = bf16_of_f16(y[p]);
    }
    if (row0 < PIECES)
      *reinterpret_cast<uint4*>(reinterpret_cast<unsigned char*>(P.bounds) + at * (4 * D) +
                                (largest ? 2 * D : 0) + chunk * PAIRS * 4 +
                                row0 % (PIECES / 2) * 16) = piece;
  }
}

// ---------------------------------------------------------------- scores

// Warps of a CTA. With one tile of query rows they share nothing, and the more CTAs the
// evener the SMs' ends: 64 long contexts take 61 us with four, 56 with two, 54 with one.
template <bool ONE>
constexpr int score_warps = ONE ? 1 : 4;
constexpr int SCORE_RUN = 4;  // 16-block tiles of a warp

struct Scores {
  const __nv_bfloat16* q;
  const unsigned char* bounds;
  const float* k_scale;  // or nullptr: ones
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* scores;
  float scale;
  int scores_stride, max_blocks_per_seq, num_kv_heads, num_blocks, cap;
  int bs_log2, g_log2, q_len;
  int part_tiles;  // 16-block tiles of a CTA
};

// The part of a bf16 pair whose sign is `neg`.
__device__ __forceinline__ uint32_t part_of(uint32_t x, bool neg) {
  const uint32_t s = (neg ? x : ~x) & 0x80008000u;  // sign of the halves to keep
  return x & ((s >> 15) * 0xffffu);
}

// A lane's runs of a row of bounds. In order, all before the products that use them: left
// to the compiler some are put off, and 64 long contexts take 67 us instead of 58.
template <int D>
__device__ __forceinline__ void load_bounds(dev::KeyRow<PA_KV_BF16, D>& x, const unsigned char* at) {
#pragma unroll
  for (int j = 0; j < D / 32; ++j)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(x.w[4 * j]), "=r"(x.w[4 * j + 1]), "=r"(x.w[4 * j + 2]), "=r"(x.w[4 * j + 3])
                 : "l"(at + j * 64)
                 : "memory");
}

// grid (partition, KV head, sequence). A warp takes 16 blocks at a time, whose bounds are
// read into fragments; the next 16 blocks' table entries are on their way meanwhile. ONE:
// one tile of 8 query rows, in registers; else up to MAX_SHARED tiles of them in shared
// memory (both parts of every row), more tiles in turn, with the bounds read again.
constexpr int MAX_SHARED = 8;
template <int D, bool ONE>
__global__ void __launch_bounds__(score_warps<ONE> * 32, 16 / score_warps<ONE>)
    block_scores_kernel(const Scores P) {
  constexpr int WARPS = score_warps<ONE>;
  using Row = dev::KeyRow<PA_KV_BF16, D>;
  dev::griddep_wait();
  extern __shared__ __align__(16) uint4 sm_q[];  // [tile][part][D / 32][32 lanes]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int head = blockIdx.y, b = blockIdx.z;
  const int BS = 1 << P.bs_log2, G = 1 << P.g_log2;
  // the first tile's entries are on their way while the length is
  const int32_t* table = P.block_tables + int64_t(b) * P.max_blocks_per_seq;
  const int first = blockIdx.x * P.part_tiles + warp;
  auto entry = [&](int tile, int r) {
    const int j = tile * 16 + r * 8 + g;
    return j < P.max_blocks_per_seq ? table[j] : 0;
  };
  int e[2] = {entry(first, 0), entry(first, 1)};
  const float f = P.k_scale != nullptr ? P.scale * P.k_scale[head] : P.scale;
  int L = P.context_lens[b];
  if (L > P.cap || (L > 0 && L < P.q_len)) {
    if (blockIdx.x == 0 && head == 0 && threadIdx.x == 0)
      atomicOr(&g_blocks_errors, PA_DEVERR_CONTEXT_LEN);
    if (L < P.q_len) return;
    L = P.cap;
  }
  if (L < P.q_len || L <= 0) return;
  const int n_blocks = (L + BS - 1) >> P.bs_log2;
  const int tiles = (n_blocks + 15) / 16;
  const int tile1 = min(tiles, (int(blockIdx.x) + 1) * P.part_tiles);
  if (int(blockIdx.x) * P.part_tiles >= tiles) return;
  const int n_cols = P.q_len << P.g_log2, col_tiles = ONE ? 1 : (n_cols + 7) / 8;
  // a negative factor turns the queries instead
  const uint32_t turn = f < 0.0f ? 0x80008000u : 0u;
  const float factor = fabsf(f);
  auto load_queries = [&](int ct, uint32_t (&up)[1][D / 16][2], uint32_t (&down)[1][D / 16][2]) {
    const int n = min(ct * 8 + g, n_cols - 1);
    const int64_t row = (int64_t(b) * P.q_len + (n >> P.g_log2)) * (P.num_kv_heads << P.g_log2) +
                        head * G + (n & (G - 1));
    uint4 raw[D / 32];
    dev::query_load<PA_KV_BF16, D>(P.q + row * D, ct * 8 + g < n_cols, t, raw);
    uint32_t qf[D / 16][2];
    dev::query_fragment<PA_KV_BF16, D>(raw, qf);
#pragma unroll
    for (int s = 0; s < D / 16; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        up[0][s][i] = part_of(qf[s][i] ^ turn, false);
        down[0][s][i] = part_of(qf[s][i] ^ turn, true);
      }
  };
  float* out = P.scores + (int64_t(b) * P.num_kv_heads + head) * P.scores_stride;
  bool bad_entry = false;
  uint32_t up[1][D / 16][2], down[1][D / 16][2];
  if (ONE) load_queries(0, up, down);
  for (int c0 = 0; c0 < col_tiles; c0 += MAX_SHARED) {
    const int n_ct = ONE ? 1 : min(MAX_SHARED, col_tiles - c0);
    if (!ONE) {
      if (c0 > 0) __syncthreads();  // the previous rows have been read
      for (int ct = warp; ct < n_ct; ct += WARPS) {
        load_queries(c0 + ct, up, down);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint4* at = sm_q + (ct * 2 * (D / 32) + c) * 32 + lane;
          at[0] = make_uint4(up[0][2 * c][0], up[0][2 * c][1], up[0][2 * c + 1][0], up[0][2 * c + 1][1]);
          at[D / 32 * 32] =
              make_uint4(down[0][2 * c][0], down[0][2 * c][1], down[0][2 * c + 1][0], down[0][2 * c + 1][1]);
        }
      }
      __syncthreads();
    }
    for (int tile = first; tile < tile1; tile += WARPS) {
      Row lo[2], hi[2];  // of blocks g and g + 8 of the tile
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const bool there = tile * 16 + r * 8 + g < n_blocks;
        const bool bad = there && (e[r] < 0 || e[r] >= P.num_blocks);
        bad_entry |= bad;
        const unsigned char* at =
            P.bounds + (int64_t(!there || bad ? 0 : e[r]) * P.num_kv_heads + head) * (4 * D) + t * 16;
        load_bounds<D>(lo[r], at);
        load_bounds<D>(hi[r], at + 2 * D);
      }
      const int next = tile + WARPS < tile1 ? tile + WARPS : first;
      e[0] = entry(next, 0);
      e[1] = entry(next, 1);
      float best[2] = {-INFINITY, -INFINITY};
      for (int ct = 0; ct < n_ct; ++ct) {
        float s[2][1][4];  // of largest and least, apart: half the chain
#pragma unroll
        for (int i = 0; i < 4; ++i) s[0][0][i] = s[1][0][i] = 0.0f;
        if constexpr (ONE) {
          dev::key_product<PA_KV_BF16, D, 1>(s[0], hi[0], hi[1], up);
          dev::key_product<PA_KV_BF16, D, 1>(s[1], lo[0], lo[1], down);
        } else {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const uint4* at = sm_q + (ct * 2 * (D / 32) + c) * 32 + lane;
            const uint4 x = at[0], y = at[D / 32 * 32];
            uint32_t a[4], z[4];
            hi[0].pairs(c, a);
            hi[1].pairs(c, z);
            dev::mma_bf16_regs(s[0][0], a[0], z[0], a[1], z[1], x.x, x.y);
            dev::mma_bf16_regs(s[0][0], a[2], z[2], a[3], z[3], x.z, x.w);
            lo[0].pairs(c, a);
            lo[1].pairs(c, z);
            dev::mma_bf16_regs(s[1][0], a[0], z[0], a[1], z[1], y.x, y.y);
            dev::mma_bf16_regs(s[1][0], a[2], z[2], a[3], z[3], y.z, y.w);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = (c0 + ct) * 8 + 2 * t + (i & 1), j = tile * 16 + (i >> 1) * 8 + g;
          const bool sees = n < n_cols && (j << P.bs_log2) <= L - P.q_len + (n >> P.g_log2);
          float x = (s[0][0][i] + s[1][0][i]) * factor;
          x = x != x ? INFINITY : x;  // a bound that is no number hides nothing
          if (sees) best[i >> 1] = fmaxf(best[i >> 1], x);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
        best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
        const int j = tile * 16 + r * 8 + g;
        if (t == 0 && j < n_blocks) out[j] = c0 == 0 ? best[r] : fmaxf(out[j], best[r]);
      }
    }
  }
  if (bad_entry) atomicOr(&g_blocks_errors, PA_DEVERR_TABLE_ENTRY);
}

// ---------------------------------------------------------------- choice

struct Choose {
  const float* scores;
  const int32_t* context_lens;
  int32_t* selected;
  int64_t scores_stride;
  int bs_log2, budget, sink, recent;
};

// Order-preserving map of a score to an unsigned key; NaN below everything, both
// zeros alike.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// The score of a key that is no NaN's.
__device__ __forceinline__ float key_score(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// A count in shared memory, without a branch.
__device__ __forceinline__ void count_if(int* at, bool here) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n @p red.shared.add.u32 [%0], 1;\n}\n" ::"r"(
          uint32_t(__cvta_generic_to_shared(at))),
      "r"(uint32_t(here))
      : "memory");
}

constexpr int LOG_BINS = 10, BINS = 1 << LOG_BINS;

// A cluster of C CTAs per (sequence, KV head). Of a span a warp holds `runs` runs of 32
// candidates, no more than the span needs, key e of a lane in the e-th of them. What a warp
// or a CTA finds is written to all CTAs, or read from all; the rest they do alike.
template <int W, int E, int C>
__global__ void __launch_bounds__(W * 32) block_select_kernel(const Choose P) {
  constexpr int THREADS = W * 32, WARPS = W * C, OWN = BINS / THREADS;
  static_assert(WARPS <= 32 && (C == 1 || OWN == 4));
  constexpr bool PAIRS = W * E >= 512;  // two bins a register: there are 64 a thread
  __shared__ __align__(16) int hist[C > 1 ? 2 : 1][BINS];
  __shared__ int counts[2][WARPS];
  __shared__ uint32_t ends[2][WARPS];
  __shared__ int found[3];  // a bin, how many of its keys are kept, how many it has
  __shared__ uint32_t few[32];
  __shared__ int n_few;
  __shared__ int32_t* list;  // (64 registers a thread do not hold it as well)
  dev::griddep_wait();
  const int tid = threadIdx.x, lane = tid & 31;
  const int L = max(P.context_lens[blockIdx.y], 0), BS = 1 << P.bs_log2;
  const int row = int(blockIdx.y * (gridDim.x / C) + blockIdx.x / C);
  const int first = int(blockIdx.x % C) * THREADS + tid, warp = first >> 5;  // in the cluster
  cg::cluster_group cluster = cg::this_cluster();
  auto sync_row = [&]() {
    if constexpr (C > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  // x to *at of every CTA, by the first lanes of a warp
  auto put = [&](auto* at, auto x) {
    if constexpr (C > 1) {
      if (lane < C) *cluster.map_shared_rank(at, unsigned(lane)) = x;
    } else {
      if (lane == 0) *at = x;
    }
  };
#pragma unroll
  for (int k = 0; k < (C > 1 ? 2 : 1) * OWN; ++k) hist[k / OWN][tid + k % OWN * THREADS] = 0;
  const float* scores = P.scores + int64_t(row) * P.scores_stride;
  int64_t blocks = (int64_t(L) + BS - 1) >> P.bs_log2;
  if (blocks > P.scores_stride) {
    if (first == 0) atomicOr(&g_blocks_errors, PA_DEVERR_CONTEXT_LEN);
    blocks = P.scores_stride;
  }
  const int n = int(blocks), n_keep = min(n, P.budget);
  int32_t* out = P.selected + int64_t(row) * P.budget;
  if (tid == 0) {
    n_few = 0;
    list = out;
  }
  for (int j = n_keep + first; j < P.budget; j += WARPS * 32) out[j] = -1;
  if (n <= P.budget) {
    for (int j = first; j < n; j += WARPS * 32) out[j] = j;
    return;
  }
  const int c0 = P.sink, c1 = n - P.recent;         // the candidates
  const int need = P.budget - P.sink - P.recent;    // of them, fewer than there are
  for (int j = first; j < P.sink; j += WARPS * 32) out[j] = j;
  for (int j = first; j < P.recent; j += WARPS * 32) out[P.sink + need + j] = c1 + j;
  if (need == 0) return;
  if constexpr (C > 1) cluster.barrier_arrive();

  const int runs = min(E, (c1 - c0 + WARPS * 32 - 1) / (WARPS * 32)), span = runs * WARPS * 32;
  const int spans = (c1 - c0 + span - 1) / span;
  const int mine0 = c0 + warp * runs * 32 + lane;
  auto index = [&](int s, int e) { return mine0 + s * span + e * 32; };
  uint32_t key[E];
  int there;                // of the keys, the first so many are
  auto load = [&](int s) {  // all on their way together
    there = min(runs, (c1 - index(s, 0) + 31) >> 5);
    float x[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      x[e] = 0.0f;
      if (e < there) x[e] = scores[index(s, e)];
    }
#pragma unroll
    for (int e = 0; e < E; ++e) key[e] = score_key(x[e]);
  };
  // The key of rank `need`: the range of the keys in up to BINS bins, then that of the keys
  // in the bin that holds it, until a bin is kept whole, is one key, or has no more than 32
  // keys, which every warp ranks for itself. The bins are first of equal widths in score,
  // where the ends are finite, then in key, which ends after four. `left`: how many of the
  // range's keys are kept.
  uint32_t threshold = 0, width = 0xffffffffu;
  uint32_t bin = 0;
  int left = need, shift = 0;
  float scale = 0.0f;  // of bins in score, or zero
  bool whole = false;
  constexpr uint32_t NONE = 0xffffu;
  uint32_t slots[PAIRS ? E / 2 : E];  // the keys' bins, NONE of one outside the range
  auto set_slot = [&](int e, uint32_t x) {
    if constexpr (PAIRS)
      slots[e / 2] = e % 2 ? slots[e / 2] | x << 16 : x;
    else
      slots[e] = x;
  };
  auto slot = [&](int e) -> uint32_t {
    if constexpr (PAIRS)
      return e % 2 ? slots[e / 2] >> 16 : slots[e / 2] & 0xffffu;
    else
      return slots[e];
  };
  auto place = [&]() {
    if (scale > 0.0f) {
      const float low = key_score(threshold);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (e % 4 == 0 && e >= runs) break;
        const int k = min(int((key_score(key[e]) - low) * scale), BINS - 1);
        set_slot(e, e < there ? uint32_t(k) : NONE);
      }
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (e % 4 == 0 && e >= runs) break;
        const uint32_t x = key[e] - threshold;
        set_slot(e, e < there && x <= width ? x >> shift : NONE);
      }
    }
  };
  auto members = [&]() {  // which of the keys are in the bin, a bit each
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (e % 4 == 0 && e >= runs) break;
      m |= (slot(e) == bin ? 1u : 0u) << e;
    }
    return m;
  };
  for (int level = 0; level < 6; ++level) {  // (an end even for scores that change meanwhile)
    uint32_t least = 0xffffffffu, most = 0u;
    for (int s = 0; s < spans; ++s) {
      if (level == 0 || spans > 1) load(s);
      if (level > 0 && spans > 1) place();
      const uint32_t m = level == 0 ? ~(~0u << max(there, 0)) : members();
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (e % 4 == 0 && e >= runs) break;
        most = max(most, m >> e & 1u ? key[e] : 0u);
        least = min(least, m >> e & 1u ? key[e] : 0xffffffffu);
      }
    }
    least = __reduce_min_sync(0xffffffffu, least);
    most = __reduce_max_sync(0xffffffffu, most);
    if constexpr (C > 1) {  // (all of the cluster's CTAs run, and have cleared)
      if (level == 0) cluster.barrier_wait();
    }
    put(&ends[0][warp], least);
    put(&ends[1][warp], most);
    sync_row();
    threshold = __reduce_min_sync(0xffffffffu, lane < WARPS ? ends[0][lane] : 0xffffffffu);
    width = __reduce_max_sync(0xffffffffu, lane < WARPS ? ends[1][lane] : 0u) - threshold;
    if (whole || width == 0) break;
    shift = max(0, 32 - __clz(width) - LOG_BINS);
    scale = __fdividef(float(BINS - 1), key_score(threshold + width) - key_score(threshold));
    // (of a NaN or an infinity among the ends it is no number or zero)
    if (level > 0 || !(scale < INFINITY)) scale = 0.0f;
    int* bins = hist[C > 1 ? level & 1 : 0];
    if constexpr (C > 1) {  // (what the other one held has been read)
      if (level > 0)
        reinterpret_cast<int4*>(hist[~level & 1])[tid] = make_int4(0, 0, 0, 0);
    }
    for (int s = 0; s < spans; ++s) {
      if (spans > 1) load(s);
      place();
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (e % 4 == 0 && e >= runs) break;
        count_if(&bins[slot(e) & (BINS - 1)], slot(e) != NONE);
      }
    }
    sync_row();
    // bins from the top, OWN a thread: where the count reaches `left`
    int mine[OWN], sum = 0;
    if constexpr (C > 1) {
      const int4* at = reinterpret_cast<int4*>(bins) + THREADS - 1 - tid;
      int4 x[C];
#pragma unroll
      for (int c = 0; c < C; ++c) x[c] = *cluster.map_shared_rank(at, unsigned(c));
      mine[0] = mine[1] = mine[2] = mine[3] = 0;
#pragma unroll
      for (int c = 0; c < C; ++c)
        mine[0] += x[c].w, mine[1] += x[c].z, mine[2] += x[c].y, mine[3] += x[c].x;
    } else {
#pragma unroll
      for (int k = 0; k < OWN; ++k) {
        int& at = bins[BINS - 1 - (tid * OWN + k)];
        mine[k] = at;
        at = 0;
      }
    }
#pragma unroll
    for (int k = 0; k < OWN; ++k) sum += mine[k];
    int upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    if (lane == 31) counts[0][tid >> 5] = upto;
    __syncthreads();
    upto += __reduce_add_sync(0xffffffffu, lane < tid >> 5 ? counts[0][lane] : 0);
    int above = upto - sum;
    if (above < left && left <= upto) {
#pragma unroll
      for (int k = 0; k < OWN; ++k) {
        if (above < left && left <= above + mine[k]) {
          found[0] = BINS - 1 - (tid * OWN + k);
          found[1] = left - above;
          found[2] = mine[k];
        }
        above += mine[k];
      }
    }
    __syncthreads();
    bin = uint32_t(found[0]);
    left = found[1];
    const int held = found[2];
    whole = left == held;
    if (held > 32) continue;
    for (int s = 0; s < spans; ++s) {
      if (spans > 1) {
        load(s);
        place();
      }
      const uint32_t m = members();
      if (m == 0) continue;
      if constexpr (C > 1) {
        const int at = atomicAdd(cluster.map_shared_rank(&n_few, 0), __popc(m));
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (m >> e & 1u) {
            uint32_t* to = &few[(at + __popc(m & ((1u << e) - 1u))) & 31];
#pragma unroll
            for (int c = 0; c < C; ++c) *cluster.map_shared_rank(to, unsigned(c)) = key[e];
          }
        }
      } else {
        const int at = atomicAdd(&n_few, __popc(m));
#pragma unroll
        for (int e = 0; e < E; ++e)
          if (m >> e & 1u) few[(at + __popc(m & ((1u << e) - 1u))) & 31] = key[e];
      }
    }
    sync_row();
    const uint32_t x = few[min(lane, held - 1)];
    int larger = 0, as_large = 0;
    for (int i = 0; i < held; ++i) {
      larger += few[i] > x;
      as_large += few[i] >= x;
    }
    const int at = __ffs(__ballot_sync(0xffffffffu, larger < left && left <= as_large)) - 1;
    threshold = __shfl_sync(0xffffffffu, x, at);
    whole = left == __shfl_sync(0xffffffffu, as_large, at);
    left -= __shfl_sync(0xffffffffu, larger, at);
    break;
  }
  // kept: keys above the threshold (from it on, where its bin is kept whole), and the first
  // `left` of those that equal it
  int equal_base = 0, keep_base = P.sink, turn = 0;
  const uint32_t below = (1u << lane) - 1u;
  // exclusive prefix over the warps; `all` is the total
  auto prefix = [&](int x, int& all) {
    put(&counts[turn][warp], x);
    sync_row();
    const int y = lane < WARPS ? counts[turn][lane] : 0;
    all = __reduce_add_sync(0xffffffffu, y);
    turn ^= 1;
    return __reduce_add_sync(0xffffffffu, lane < warp ? y : 0);
  };
  for (int s = 0; s < spans; ++s) {
    if (spans > 1) load(s);
    uint32_t kept[E];
    int n_kept = 0, all_equal = 0, all_kept;
    if (whole) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (e % 4 == 0 && e >= runs) break;
        kept[e] = __ballot_sync(0xffffffffu, e < there && key[e] >= threshold);
        n_kept += __popc(kept[e]);
      }
    } else {
      int n_equal = 0;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (e % 4 == 0 && e >= runs) break;
        n_equal += __popc(__ballot_sync(0xffffffffu, e < there && key[e] == threshold));
      }
      int at = equal_base + prefix(n_equal, all_equal);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        if (e % 4 == 0 && e >= runs) break;
        const bool same = e < there && key[e] == threshold;
        const uint32_t equal = __ballot_sync(0xffffffffu, same);
        const bool tie = same && at + __popc(equal & below) < left;
        kept[e] = __ballot_sync(0xffffffffu, tie || (e < there && key[e] > threshold));
        at += __popc(equal);
        n_kept += __popc(kept[e]);
      }
    }
    int at = keep_base + prefix(n_kept, all_kept);
    int32_t* to = list;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (e % 4 == 0 && e >= runs) break;
      if (kept[e] >> lane & 1u) to[at + __popc(kept[e] & below)] = index(s, e);
      at += __popc(kept[e]);
    }
    equal_base += all_equal;
    keep_base += all_kept;
  }
}

template <int FMT, int D, int BS>
int launch_bounds_t(const Bounds& P, int num_seqs, int num_sms, cudaStream_t s) {
  constexpr int TILE = BS * (FMT == PA_KV_BF16 ? 2 * D : (FMT == PA_KV_FP8_E4M3 ? D : D * 9 / 16));
  // Tiles a warp, one after the other: 16 KB of them, of 4-bit codes 8 (the GPU starts about
  // a CTA a nanosecond: with a tile a warp 106.5 for 102.5 us, 58.2 for 49.5 in 4 bits, and
  // blocks of 8 tokens in 4 bits 129 for 72), fewer where that leaves fewer than 32 warps an
  // SM.
  constexpr int BYTES = FMT == PA_KV_FP4_E2M1 ? 8192 : 16384;
  const int64_t units = int64_t(P.per_seq) * P.num_kv_heads;
  int64_t run = units * num_seqs / (int64_t(num_sms > 0 ? num_sms : 152) * 32);
  run = run < 1 ? 1 : (run > BYTES / TILE ? (BYTES + TILE - 1) / TILE : run);
  int64_t x = (units + BOUND_WARPS * run - 1) / (BOUND_WARPS * run);
  if (x > 65535) x = 65535;  // (warps go on by the grid's width)
  const dim3 grid{unsigned(x), unsigned(num_seqs)};
  return launch_ordered(block_bounds_kernel<FMT, D, BS>, grid, BOUND_WARPS * 32, 0, s, 1, P);
}
template <int FMT, int D>
int launch_bounds_bs(const Bounds& P, int block_size, int num_seqs, int num_sms, cudaStream_t s) {
  switch (block_size) {
    case 8: return launch_bounds_t<FMT, D, 8>(P, num_seqs, num_sms, s);
    case 16: return launch_bounds_t<FMT, D, 16>(P, num_seqs, num_sms, s);
    case 32: return launch_bounds_t<FMT, D, 32>(P, num_seqs, num_sms, s);
    default: return int(cudaErrorInvalidValue);
  }
}
template <int FMT>
int launch_bounds_d(const Bounds& P, const pa_block_bounds_params* p, int num_sms, cudaStream_t s) {
  return p->head_dim == 64 ? launch_bounds_bs<FMT, 64>(P, p->block_size, p->num_seqs, num_sms, s)
                           : launch_bounds_bs<FMT, 128>(P, p->block_size, p->num_seqs, num_sms, s);
}

template <int D, bool ONE>
int launch_scores_t(Scores P, int64_t tiles, int num_seqs, int num_sms, cudaStream_t s) {
  constexpr int WARPS = score_warps<ONE>;
  // SCORE_RUN tiles a warp, fewer where that leaves fewer than 16 warps an SM
  const int64_t rows = int64_t(num_seqs) * P.num_kv_heads;
  int64_t run = SCORE_RUN;
  while (run > 1 && (tiles + run - 1) / run * rows < int64_t(num_sms) * 16) run /= 2;
  P.part_tiles = int(run * WARPS);
  const dim3 grid{unsigned((tiles + P.part_tiles - 1) / P.part_tiles), unsigned(P.num_kv_heads),
                  unsigned(num_seqs)};
  const int col_tiles = ((P.q_len << P.g_log2) + 7) / 8;
  const size_t smem = ONE ? 0 : size_t(col_tiles < MAX_SHARED ? col_tiles : MAX_SHARED) * 32 * D;
  return launch_ordered(block_scores_kernel<D, ONE>, grid, WARPS * 32, smem, s, 1, P);
}

}  // namespace

int launch_block_bounds(const pa_block_bounds_params* p, int num_sms, void* stream) {
  Bounds P;
  P.k_cache = static_cast<const unsigned char*>(p->k_cache);
  P.bounds = static_cast<__nv_bfloat16*>(p->bounds);
  P.block_tables = p->block_tables;
  P.context_lens = p->context_lens;
  P.old_lens = p->old_lens;
  P.max_blocks_per_seq = p->max_blocks_per_seq;
  P.num_kv_heads = p->num_kv_heads;
  P.num_blocks = p->num_blocks;
  // blocks that max_new_tokens tokens can touch, wherever they begin
  const int64_t touched = (int64_t(p->max_new_tokens) + 2 * p->block_size - 2) / p->block_size;
  P.per_seq = int(touched < p->max_blocks_per_seq ? touched : p->max_blocks_per_seq);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (p->kv_dtype) {
    case PA_KV_BF16: return launch_bounds_d<PA_KV_BF16>(P, p, num_sms, s);
    case PA_KV_FP8_E4M3: return launch_bounds_d<PA_KV_FP8_E4M3>(P, p, num_sms, s);
    default: return launch_bounds_d<PA_KV_FP4_E2M1>(P, p, num_sms, s);
  }
}

int launch_block_scores(const pa_block_scores_params* p, int num_sms, void* stream) {
  Scores P;
  P.q = static_cast<const __nv_bfloat16*>(p->q);
  P.bounds = static_cast<const unsigned char*>(p->bounds);
  P.k_scale = p->k_scale;
  P.block_tables = p->block_tables;
  P.context_lens = p->context_lens;
  P.scores = p->scores;
  P.scale = p->scale;
  P.scores_stride = p->scores_stride;
  P.max_blocks_per_seq = p->max_blocks_per_seq;
  P.num_kv_heads = p->num_kv_heads;
  P.num_blocks = p->num_blocks;
  const int64_t table = int64_t(p->max_blocks_per_seq) * p->block_size;
  P.cap = int(p->max_context_len < table ? p->max_context_len : table);
  P.bs_log2 = log2_of(p->block_size);
  P.g_log2 = log2_of(p->num_q_heads / p->num_kv_heads);
  P.q_len = p->query_len > 1 ? p->query_len : 1;
  const int64_t tiles = ((P.cap + p->block_size - 1) / p->block_size + 15) / 16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((P.q_len << P.g_log2) <= 8)
    return p->head_dim == 64 ? launch_scores_t<64, true>(P, tiles, p->num_seqs, num_sms, s)
                             : launch_scores_t<128, true>(P, tiles, p->num_seqs, num_sms, s);
  return p->head_dim == 64 ? launch_scores_t<64, false>(P, tiles, p->num_seqs, num_sms, s)
                           : launch_scores_t<128, false>(P, tiles, p->num_seqs, num_sms, s);
}

int launch_block_select(const float* scores, const int32_t* context_lens, int32_t* selected,
                        int32_t num_seqs, int32_t num_kv_heads, int32_t scores_stride,
                        int32_t block_size, int32_t budget, int32_t sink, int32_t recent,
                        int num_sms, void* stream) {
  Choose P;
  P.scores = scores;
  P.context_lens = context_lens;
  P.selected = selected;
  P.scores_stride = scores_stride;
  P.bs_log2 = log2_of(block_size);
  P.budget = budget;
  P.sink = sink;
  P.recent = recent;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto launch = [&](auto kernel, unsigned warps, unsigned ctas) {
    const dim3 grid{unsigned(num_kv_heads) * ctas, unsigned(num_seqs)};
    return launch_ordered(kernel, grid, warps * 32, 0, s, ctas, P);
  };
  // A row in registers where it fits; longer ones are read again for every range. A cluster
  // pays where a CTA a row leaves half of the SMs idle: up to 16,384 blocks 6.8 for 8.9 us at
  // 8 rows, 8.3 for 9.0 at 72, but 10.3 for 9.2 at 80; of two CTAs, up to 8,192 blocks, it does
  // not (6.4 for 5.8). The stride stands for the rows' length, which the host does not know:
  // rows much shorter than it take a wider form than they need (512 rows of 8,000 blocks in a
  // stride of 16,384: 22.6 us).
  if (scores_stride <= 2048) return launch(block_select_kernel<8, 8, 1>, 8, 1);
  if (scores_stride <= 4096) return launch(block_select_kernel<8, 16, 1>, 8, 1);
  if (scores_stride <= 8192) return launch(block_select_kernel<16, 16, 1>, 16, 1);
  if (int64_t(num_seqs) * num_kv_heads * 2 <= (num_sms > 0 ? num_sms : 152))
    return launch(block_select_kernel<8, 16, 4>, 8, 4);
  return launch(block_select_kernel<32, 16, 1>, 32, 1);
}

int read_and_clear_blocks_errors(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_blocks_errors, sizeof(v));
  if (e != cudaSuccess) return int(e);
  if (v != 0) e = cudaMemcpyToSymbol(g_blocks_errors, &zero, sizeof(zero));
  *flags = v;
  return int(e);
}

}  // namespace pa
