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
//  * block_select_kernel: one CTA per (sequence, KV head) with the row's scores as
//    ordered 32-bit keys in registers; the key of the budget's rank is found bit by bit
//    from the first bit in which keys differ, a count over the CTA each, until a count
//    meets the budget. Ties go to the lowest index through ranks. Bound by latency.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_blocks.h"
#include "pa_device.cuh"
#include "pa_mma.cuh"
#include "pa_ordered.cuh"

namespace pa {
namespace {

__device__ unsigned int g_blocks_errors;

// ---------------------------------------------------------------- bounds

// Warps of a CTA (64 sequences' prompts in bf16, 32 in 4 bits, d 128: with 8 106.8 and
// 73.7 us, with 4 108.9 and 58.4, with 2 133.6 and 67.3).
template <int FMT>
constexpr int bound_warps = FMT == PA_KV_BF16 ? 8 : 4;

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
__global__ void __launch_bounds__(bound_warps<FMT> * 32) block_bounds_kernel(const Bounds P) {
  constexpr int WARPS = bound_warps<FMT>;
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
  const int first = old / BS, last = (min(L, cap) + BS - 1) / BS;  // the blocks to do
  if (blockIdx.x == 0 && threadIdx.x == 0 && (L > cap || last - first > P.per_seq))
    atomicOr(&g_blocks_errors, PA_DEVERR_CONTEXT_LEN);
  const int n = min(last - first, P.per_seq);
  const uint32_t heads = uint32_t(P.num_kv_heads), units = uint32_t(max(n, 0)) * heads;
  for (uint32_t u = blockIdx.x * WARPS + warp; u < units; u += gridDim.x * WARPS) {
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

constexpr int SCORE_WARPS = 4;

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

// grid (partition, KV head, sequence)
template <int D>
__global__ void __launch_bounds__(SCORE_WARPS * 32) block_scores_kernel(const Scores P) {
  using Row = dev::KeyRow<PA_KV_BF16, D>;
  dev::griddep_enter();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int head = blockIdx.y, b = blockIdx.z;
  const int BS = 1 << P.bs_log2, G = 1 << P.g_log2;
  int L = P.context_lens[b];
  if (L > P.cap || (L > 0 && L < P.q_len)) {
    if (blockIdx.x == 0 && head == 0 && threadIdx.x == 0)
      atomicOr(&g_blocks_errors, PA_DEVERR_CONTEXT_LEN);
    if (L < P.q_len) return;
    L = P.cap;
  }
  if (L < P.q_len || L <= 0) return;
  const int n_blocks = (L + BS - 1) >> P.bs_log2;
  const int n_cols = P.q_len << P.g_log2;
  const float f = P.k_scale != nullptr ? P.scale * P.k_scale[head] : P.scale;
  // a negative factor turns the queries instead
  const uint32_t turn = f < 0.0f ? 0x80008000u : 0u;
  const float factor = fabsf(f);
  auto load_queries = [&](int c0, uint32_t (&up)[1][D / 16][2], uint32_t (&down)[1][D / 16][2]) {
    const int n = c0 + g;
    const int64_t row = (int64_t(b) * P.q_len + (min(n, n_cols - 1) >> P.g_log2)) *
                            (P.num_kv_heads << P.g_log2) + head * G + (min(n, n_cols - 1) & (G - 1));
    uint4 raw[D / 32];
    dev::query_load<PA_KV_BF16, D>(P.q + row * D, n < n_cols, t, raw);
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
  uint32_t up[1][D / 16][2], down[1][D / 16][2];
  load_queries(0, up, down);
  int loaded = 0;  // the columns at hand
  const int tiles = (n_blocks + 15) / 16;
  const int tile1 = min(tiles, (int(blockIdx.x) + 1) * P.part_tiles);
  const int32_t* table = P.block_tables + int64_t(b) * P.max_blocks_per_seq;
  float* out = P.scores + (int64_t(b) * P.num_kv_heads + head) * P.scores_stride;
  bool bad_entry = false;
  for (int tile = blockIdx.x * P.part_tiles + warp; tile < tile1; tile += SCORE_WARPS) {
    Row lo[2], hi[2];  // of blocks g and g + 8 of the tile
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = min(tile * 16 + r * 8 + g, n_blocks - 1);
      int e = table[j];
      bad_entry |= e < 0 || e >= P.num_blocks;
      e = e < 0 || e >= P.num_blocks ? 0 : e;
      const unsigned char* at = P.bounds + (int64_t(e) * P.num_kv_heads + head) * (4 * D) + t * 16;
      lo[r].load(at, nullptr);
      hi[r].load(at + 2 * D, nullptr);
    }
    float best[2] = {-INFINITY, -INFINITY};
    for (int c0 = 0; c0 < n_cols; c0 += 8) {
      if (c0 != loaded) load_queries(loaded = c0, up, down);
      float s[1][4] = {{0.0f, 0.0f, 0.0f, 0.0f}};
      dev::key_product<PA_KV_BF16, D, 1>(s, hi[0], hi[1], up);
      dev::key_product<PA_KV_BF16, D, 1>(s, lo[0], lo[1], down);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = c0 + 2 * t + (i & 1), j = tile * 16 + (i >> 1) * 8 + g;
        const bool sees = n < n_cols && (j << P.bs_log2) <= L - P.q_len + (n >> P.g_log2);
        float x = s[0][i] * factor;
        x = x != x ? INFINITY : x;  // a bound that is no number hides nothing
        if (sees) best[i >> 1] = fmaxf(best[i >> 1], x);
      }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 1));
      best[r] = fmaxf(best[r], __shfl_xor_sync(0xffffffffu, best[r], 2));
      const int j = tile * 16 + r * 8 + g;
      if (t == 0 && j < n_blocks) out[j] = best[r];
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
  int num_kv_heads, bs_log2, budget, sink, recent;
};

// Order-preserving map of a score to an unsigned key; NaN below everything, both
// zeros alike.
__device__ __forceinline__ uint32_t score_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per (sequence, KV head). Warp w holds candidates [w * 32 E, (w + 1) * 32 E)
// of a span, key e of a lane the e-th run of 32.
template <int WARPS, int E>
__global__ void __launch_bounds__(WARPS * 32) block_select_kernel(const Choose P) {
  constexpr int THREADS = WARPS * 32, SPAN = THREADS * E;
  __shared__ int counts[2][WARPS];
  __shared__ uint32_t ends[2][WARPS];
  dev::griddep_enter();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = blockIdx.x, b = row / P.num_kv_heads;
  const int BS = 1 << P.bs_log2;
  const int L = max(P.context_lens[b], 0);
  int64_t blocks = (int64_t(L) + BS - 1) >> P.bs_log2;
  if (blocks > P.scores_stride) {
    if (tid == 0) atomicOr(&g_blocks_errors, PA_DEVERR_CONTEXT_LEN);
    blocks = P.scores_stride;
  }
  const int n = int(blocks), n_keep = min(n, P.budget);
  int32_t* out = P.selected + int64_t(row) * P.budget;
  for (int j = n_keep + tid; j < P.budget; j += THREADS) out[j] = -1;
  if (n <= P.budget) {
    for (int j = tid; j < n; j += THREADS) out[j] = j;
    return;
  }
  const float* scores = P.scores + int64_t(row) * P.scores_stride;
  const int c0 = P.sink, c1 = n - P.recent;         // the candidates
  const int need = P.budget - P.sink - P.recent;    // of them, fewer than there are
  for (int j = tid; j < P.sink; j += THREADS) out[j] = j;
  for (int j = tid; j < P.recent; j += THREADS) out[P.sink + need + j] = c1 + j;
  if (need == 0) return;

  const int spans = (c1 - c0 + SPAN - 1) / SPAN;
  auto index = [&](int span, int e) { return c0 + span * SPAN + (warp * E + e) * 32 + lane; };
  uint32_t key[E];
  auto load = [&](int span) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int j = index(span, e);
      key[e] = j < c1 ? score_key(scores[j]) : 0u;
    }
  };
  int turn = 0;
  // sum over the CTA; one barrier, two buffers
  auto total = [&](int x) {
    x = __reduce_add_sync(0xffffffffu, x);
    if (lane == 0) counts[turn][warp] = x;
    __syncthreads();
    x = __reduce_add_sync(0xffffffffu, lane < WARPS ? counts[turn][lane] : 0);
    turn ^= 1;
    return x;
  };
  // the least and the largest key: bits above the first that differs are known
  uint32_t least = 0xffffffffu, most = 0u;
  for (int s = 0; s < spans; ++s) {
    load(s);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      most = max(most, key[e]);
      if (index(s, e) < c1) least = min(least, key[e]);
    }
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if (lane == 0) {
    ends[0][warp] = least;
    ends[1][warp] = most;
  }
  __syncthreads();
  least = __reduce_min_sync(0xffffffffu, lane < WARPS ? ends[0][lane] : 0xffffffffu);
  most = __reduce_max_sync(0xffffffffu, lane < WARPS ? ends[1][lane] : 0u);
  // threshold: the largest key that at least `need` candidates reach
  int bit = 31 - __clz(least ^ most);  // -1: all alike
  uint32_t threshold = bit < 0 ? most : most >> bit >> 1 << bit << 1;
  bool exact = false;  // exactly `need` reach it
  for (; bit >= 0 && !exact; --bit) {
    const uint32_t x = threshold | 1u << bit;
    int c = 0;
    for (int s = 0; s < spans; ++s) {
      if (spans > 1) load(s);
#pragma unroll
      for (int e = 0; e < E; ++e) c += key[e] >= x;  // (x > 0: not what lies past the row)
    }
    c = total(c);
    if (c >= need) threshold = x;
    exact = c == need;
  }
  // of the keys that equal the threshold the first `ties` are kept
  int ties = need;
  if (!exact) {
    int c = 0;
    for (int s = 0; s < spans; ++s) {
      if (spans > 1) load(s);
#pragma unroll
      for (int e = 0; e < E; ++e) c += key[e] > threshold;
    }
    ties = need - total(c);
  }
  // ranks in index order
  int equal_base = 0, keep_base = P.sink;
  const uint32_t below = (1u << lane) - 1u;
  // exclusive prefix over the warps; `all` is the total
  auto prefix = [&](int x, int& all) {
    if (lane == 0) counts[turn][warp] = x;
    __syncthreads();
    const int y = lane < WARPS ? counts[turn][lane] : 0;
    all = __reduce_add_sync(0xffffffffu, y);
    turn ^= 1;
    return __reduce_add_sync(0xffffffffu, lane < warp ? y : 0);
  };
  for (int s = 0; s < spans; ++s) {
    if (spans > 1) load(s);
    uint32_t equal[E], kept[E];
    int n_equal = 0, n_kept = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      equal[e] = __ballot_sync(0xffffffffu, index(s, e) < c1 && key[e] == threshold);
      n_equal += __popc(equal[e]);
    }
    int all_equal, all_kept;
    int at = equal_base + prefix(n_equal, all_equal);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = index(s, e) < c1;
      const bool tie = in && key[e] == threshold && at + __popc(equal[e] & below) < ties;
      kept[e] = __ballot_sync(0xffffffffu, tie || (in && key[e] > threshold));
      at += __popc(equal[e]);
      n_kept += __popc(kept[e]);
    }
    at = keep_base + prefix(n_kept, all_kept);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if (kept[e] >> lane & 1u) out[at + __popc(kept[e] & below)] = index(s, e);
      at += __popc(kept[e]);
    }
    equal_base += all_equal;
    keep_base += all_kept;
  }
}

template <int FMT, int D>
int launch_bounds_bs(const Bounds& P, int block_size, int num_seqs, cudaStream_t s) {
  constexpr int WARPS = bound_warps<FMT>, threads = WARPS * 32;
  int64_t x = (int64_t(P.per_seq) * P.num_kv_heads + WARPS - 1) / WARPS;
  if (x > 65535) x = 65535;  // (warps go on by the grid's width)
  const dim3 grid{unsigned(x), unsigned(num_seqs)};
  switch (block_size) {
    case 8: return launch_ordered(block_bounds_kernel<FMT, D, 8>, grid, threads, 0, s, 1, P);
    case 16: return launch_ordered(block_bounds_kernel<FMT, D, 16>, grid, threads, 0, s, 1, P);
    case 32: return launch_ordered(block_bounds_kernel<FMT, D, 32>, grid, threads, 0, s, 1, P);
    default: return int(cudaErrorInvalidValue);
  }
}
template <int FMT>
int launch_bounds_d(const Bounds& P, const pa_block_bounds_params* p, cudaStream_t s) {
  return p->head_dim == 64 ? launch_bounds_bs<FMT, 64>(P, p->block_size, p->num_seqs, s)
                           : launch_bounds_bs<FMT, 128>(P, p->block_size, p->num_seqs, s);
}

}  // namespace

int launch_block_bounds(const pa_block_bounds_params* p, void* stream) {
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
    case PA_KV_BF16: return launch_bounds_d<PA_KV_BF16>(P, p, s);
    case PA_KV_FP8_E4M3: return launch_bounds_d<PA_KV_FP8_E4M3>(P, p, s);
    default: return launch_bounds_d<PA_KV_FP4_E2M1>(P, p, s);
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
  // four tiles a warp, fewer where that leaves SMs idle
  const int64_t tiles = ((P.cap + p->block_size - 1) / p->block_size + 15) / 16;
  const int64_t rows = int64_t(p->num_seqs) * p->num_kv_heads;
  int64_t per = 4 * SCORE_WARPS;
  while (per > SCORE_WARPS && (tiles + per - 1) / per * rows < int64_t(num_sms) * 4) per /= 2;
  P.part_tiles = int(per);
  const dim3 grid(unsigned((tiles + per - 1) / per), unsigned(p->num_kv_heads),
                  unsigned(p->num_seqs));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p->head_dim == 64)
    return launch_ordered(block_scores_kernel<64>, grid, SCORE_WARPS * 32, 0, s, 1, P);
  return launch_ordered(block_scores_kernel<128>, grid, SCORE_WARPS * 32, 0, s, 1, P);
}

int launch_block_select(const float* scores, const int32_t* context_lens, int32_t* selected,
                        int32_t num_seqs, int32_t num_kv_heads, int32_t scores_stride,
                        int32_t block_size, int32_t budget, int32_t sink, int32_t recent,
                        void* stream) {
  Choose P;
  P.scores = scores;
  P.context_lens = context_lens;
  P.selected = selected;
  P.scores_stride = scores_stride;
  P.num_kv_heads = num_kv_heads;
  P.bs_log2 = log2_of(block_size);
  P.budget = budget;
  P.sink = sink;
  P.recent = recent;
  const dim3 grid(unsigned(num_seqs) * unsigned(num_kv_heads));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // a row in registers where it fits; longer ones are read again for every count
  if (scores_stride <= 8 * 32 * 8)
    return launch_ordered(block_select_kernel<8, 8>, grid, 8 * 32, 0, s, 1, P);
  return launch_ordered(block_select_kernel<32, 16>, grid, 32 * 32, 0, s, 1, P);
}

int read_and_clear_blocks_errors(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_blocks_errors, sizeof(v));
  if (e != cudaSuccess) return int(e);
  e = cudaMemcpyToSymbol(g_blocks_errors, &zero, sizeof(zero));
  *flags = v;
  return int(e);
}

}  // namespace pa
