// Eviction of cached tokens for sm_103a: the choice of the tokens to keep
// under a budget, and the move of their rows.
//
// The pages describe the pool's side of memory pressure (blocks reclaimed,
// "How Paged Attention and Continuous Batching Actually Work"); which tokens
// go is left open. Here the most recent ones stay, and of the others those
// with the largest accumulated attention weight (pa_weights.cu).
//
//  * evict_select_kernel: one CTA per sequence. The candidates' weights become
//    ordered 32-bit keys in registers (32 a thread; longer sequences re-read
//    them from L2), and the threshold is found bit by bit: a count of the keys
//    at or above a trial value, 32 rounds at most and fewer when a trial
//    splits the keys exactly. No histogram, so equal weights -- most tokens of
//    a long context have nearly none -- cost nothing extra. Ties go to the
//    lowest index through ranks, and the kept indices come out ascending.
//  * compact_rows_kernel: row j of the destination <- row keep[j] of the
//    source. keep ascends, so keep[j] >= j, and moving rows in order within
//    one CTA is safe in place: a tile's rows are in registers before any of
//    them is overwritten, and later tiles read only rows behind it. A CTA
//    owns one (sequence, KV head) and a slice of the row's bytes, so CTAs never
//    meet. Bound by memory traffic: every kept row is read and written once,
//    and rows that stay where they are not at all.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_device.cuh"
#include "pa_internal.h"

namespace pa {
namespace {

__device__ unsigned int g_evict_errors;

// ---------------------------------------------------------------- selection

constexpr int SEL_THREADS = 1024;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_KEYS = 32;  // keys a thread holds at a time
constexpr int SEL_SPAN = SEL_THREADS * SEL_KEYS;

// Order-preserving map of a weight to an unsigned key; NaN below everything,
// both zeros alike.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);  // -0 + 0 = +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

struct Select {
  const float* weights;
  const int32_t* context_lens;
  int32_t* keep;
  int32_t* new_lens;
  int64_t weights_stride;
  int num_seqs, budget, recent, max_len;
};

// Sum over the CTA, the same in every thread. `buf` alternates between two
// rows of shared memory, so one barrier a call is enough.
__device__ __forceinline__ int block_sum(int x, int (*sm)[SEL_WARPS], int& buf) {
  x = __reduce_add_sync(0xffffffffu, x);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) sm[buf][warp] = x;
  __syncthreads();
  const int total = __reduce_add_sync(0xffffffffu, sm[buf][lane]);
  buf ^= 1;
  return total;
}

// Exclusive prefix over cnt[SEL_KEYS][SEL_WARPS] (in place), + base; returns the total.
__device__ __forceinline__ int scan_counts(int* cnt, int base, int* warp_tot) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __syncthreads();
  const int x = cnt[tid];
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  int tot = warp_tot[lane], run = tot;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += y;
  }
  const int before = __shfl_sync(0xffffffffu, run - tot, warp);
  const int all = __shfl_sync(0xffffffffu, run, 31);
  cnt[tid] = base + before + inc - x;
  __syncthreads();
  return all;
}

// Key e of this thread in a span: token span * SEL_SPAN + e * SEL_THREADS + tid.
__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(const Select P) {
  __shared__ int sums[2][SEL_WARPS];
  __shared__ int cnt_eq[SEL_KEYS * SEL_WARPS], cnt_keep[SEL_KEYS * SEL_WARPS];
  __shared__ int warp_tot[SEL_WARPS];
  const int b = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int L = P.context_lens[b];
  if (L > P.max_len) {
    if (tid == 0) atomicOr(&g_evict_errors, PA_DEVERR_CONTEXT_LEN);
    L = P.max_len;
  }
  L = max(L, 0);
  const int n_keep = min(L, P.budget);
  int32_t* keep = P.keep + int64_t(b) * P.budget;
  if (tid == 0) P.new_lens[b] = n_keep;
  for (int j = n_keep + tid; j < P.budget; j += SEL_THREADS) keep[j] = -1;
  if (L <= P.budget) {
    for (int j = tid; j < L; j += SEL_THREADS) keep[j] = j;
    return;
  }
  const int n_cand = L - P.recent;          // the others always stay
  const int need = P.budget - P.recent;     // of the candidates, fewer than n_cand
  const float* w = P.weights + int64_t(b) * P.weights_stride;
  const int spans = (n_cand + SEL_SPAN - 1) / SEL_SPAN;
  uint32_t key[SEL_KEYS];  // candidates only; 0 elsewhere
  auto load = [&](int span) {
#pragma unroll
    for (int e = 0; e < SEL_KEYS; ++e) {
      const int64_t i = int64_t(span) * SEL_SPAN + e * SEL_THREADS + tid;
      key[e] = i < n_cand ? weight_key(w[i]) : 0u;
    }
  };
  if (spans == 1) load(0);

  // the largest threshold that at least `need` keys reach
  uint32_t T = 0;
  bool exact = false;  // exactly `need` keys reach it
  int buf = 0;
  if (need > 0) {
    for (int bit = 31; bit >= 0 && !exact; --bit) {
      const uint32_t c = T | (1u << bit);
      int n = 0;
      for (int span = 0; span < spans; ++span) {
        if (spans > 1) load(span);
#pragma unroll
        for (int e = 0; e < SEL_KEYS; ++e) n += key[e] >= c;
      }
      n = block_sum(n, sums, buf);
      if (n >= need) T = c;
      exact = n == need;
    }
  }
  int ties = 0;  // keys equal to T that are kept: the first ones
  if (need > 0 && !exact) {
    int n = 0;
    for (int span = 0; span < spans; ++span) {
      if (spans > 1) load(span);
#pragma unroll
      for (int e = 0; e < SEL_KEYS; ++e) n += key[e] > T;
    }
    ties = need - block_sum(n, sums, buf);
  }

  // ranks in token order: of the ties, then of the kept
  int eq_base = 0, keep_base = 0;
  for (int span = 0; span < spans; ++span) {
    if (spans > 1) load(span);
    uint32_t in_key = 0, eq = 0;
#pragma unroll
    for (int e = 0; e < SEL_KEYS; ++e) {
      const int64_t i = int64_t(span) * SEL_SPAN + e * SEL_THREADS + tid;
      const bool cand = i < n_cand && need > 0;
      const bool same = cand && !exact && key[e] == T;
      in_key |= uint32_t(cand && (exact ? key[e] >= T : key[e] > T)) << e;
      eq |= uint32_t(same) << e;
      const uint32_t v = __ballot_sync(0xffffffffu, same);
      if (lane == 0) cnt_eq[e * SEL_WARPS + warp] = __popc(v);
    }
    const int eq_all = scan_counts(cnt_eq, eq_base, warp_tot);
    const uint32_t below = (1u << lane) - 1u;
#pragma unroll
    for (int e = 0; e < SEL_KEYS; ++e) {
      const bool same = (eq >> e) & 1u;
      const uint32_t v = __ballot_sync(0xffffffffu, same);
      if (same && cnt_eq[e * SEL_WARPS + warp] + __popc(v & below) < ties) in_key |= 1u << e;
      const uint32_t k = __ballot_sync(0xffffffffu, (in_key >> e) & 1u);
      if (lane == 0) cnt_keep[e * SEL_WARPS + warp] = __popc(k);
    }
    const int keep_all = scan_counts(cnt_keep, keep_base, warp_tot);
#pragma unroll
    for (int e = 0; e < SEL_KEYS; ++e) {
      const bool on = (in_key >> e) & 1u;
      const uint32_t k = __ballot_sync(0xffffffffu, on);
      if (on)
        keep[cnt_keep[e * SEL_WARPS + warp] + __popc(k & below)] =
            span * SEL_SPAN + e * SEL_THREADS + tid;
    }
    eq_base += eq_all;
    keep_base += keep_all;
    __syncthreads();
  }
  for (int j = tid; j < P.recent; j += SEL_THREADS) keep[need + j] = n_cand + j;
}

// ---------------------------------------------------------------- compaction

constexpr int MOVE_THREADS = 128;
constexpr int MOVE_DEPTH = 8;  // rows a thread has in flight, twice

// One set of rows of the caches: `base` + block * block_bytes + head *
// tile_bytes + first + offset * row_bytes.
struct Plane {
  unsigned char* base;
  int tile_bytes, first, row_bytes;
  int vec;     // bytes a thread moves of a row: 16, 8 or 4; 1 = the 8-bit cache's V^T
  int slices;  // CTAs that share a row's bytes
};
constexpr int MAX_PLANES = 4;

struct Compact {
  Plane plane[MAX_PLANES];
  const int32_t* src_tables;
  const int32_t* dst_tables;
  const int32_t* keep;
  const int32_t* new_lens;
  int src_blocks, dst_blocks;  // entries of a table row
  int keep_stride, num_kv_heads, num_blocks, bs_log2;
};

// Rows j of the destination and keep[j] of the source, as (block, offset)
// pairs packed block * BS + offset; -1 where there is nothing to move.
__device__ __forceinline__ bool move_of(const Compact& P, int b, int j, int n, bool report,
                                        int64_t& src, int64_t& dst) {
  src = dst = 0;
  if (j >= n) return false;
  const int BS = 1 << P.bs_log2;
  const int t = P.keep[int64_t(b) * P.keep_stride + j];
  if (t < j || (t >> P.bs_log2) >= P.src_blocks) {  // not ascending, or no such row
    if (report) atomicOr(&g_evict_errors, PA_DEVERR_KEEP);
    return false;
  }
  const int sb = P.src_tables[int64_t(b) * P.src_blocks + (t >> P.bs_log2)];
  const int db = P.dst_tables[int64_t(b) * P.dst_blocks + (j >> P.bs_log2)];
  if (sb < 0 || sb >= P.num_blocks || db < 0 || db >= P.num_blocks) {
    if (report) atomicOr(&g_evict_errors, PA_DEVERR_TABLE_ENTRY);
    return false;
  }
  src = int64_t(sb) * BS + (t & (BS - 1));
  dst = int64_t(db) * BS + (j & (BS - 1));
  return src != dst;  // a row that stays
}

__device__ __forceinline__ int rows_to_move(const Compact& P, int b, bool report) {
  int n = P.new_lens[b];
  const int cap = min(P.keep_stride, P.dst_blocks << P.bs_log2);
  if (n > cap) {
    if (report) atomicOr(&g_evict_errors, PA_DEVERR_CONTEXT_LEN);
    n = cap;
  }
  return n;
}

template <typename V>
__device__ __forceinline__ void move_rows(const Compact& P, const Plane& pl, int b, int head,
                                          int slice) {
  const int per_row = pl.row_bytes / pl.slices / int(sizeof(V));  // threads of a row
  const int lane = threadIdx.x % per_row, r = threadIdx.x / per_row;
  const int rows = MOVE_THREADS / per_row;                        // rows of a pass
  const int tile = rows * MOVE_DEPTH;
  const bool report = lane == 0 && head == 0 && slice == 0;
  const int n = rows_to_move(P, b, threadIdx.x == 0 && head == 0 && slice == 0);
  const int BS = 1 << P.bs_log2;
  const int64_t col = pl.first + (slice * per_row + lane) * int64_t(sizeof(V));
  auto at = [&](int64_t slot) {
    return pl.base + ((slot >> P.bs_log2) * P.num_kv_heads + head) * pl.tile_bytes +
           (slot & (BS - 1)) * pl.row_bytes + col;
  };
  struct Addr {
    const unsigned char* src[MOVE_DEPTH];
    unsigned char* dst[MOVE_DEPTH];
  };
  auto find = [&](int j0, Addr& a) {
#pragma unroll
    for (int u = 0; u < MOVE_DEPTH; ++u) {
      int64_t s, d;
      const bool go = move_of(P, b, j0 + u * rows + r, n, report, s, d);
      a.src[u] = go ? at(s) : nullptr;
      a.dst[u] = go ? at(d) : nullptr;
    }
  };
  V data[MOVE_DEPTH];
  for (int j0 = 0; j0 < n; j0 += tile) {
    Addr a;
    find(j0, a);
#pragma unroll
    for (int u = 0; u < MOVE_DEPTH; ++u)
      if (a.src[u]) data[u] = *reinterpret_cast<const V*>(a.src[u]);
    __syncthreads();  // the tile's rows are read before any of them is overwritten
#pragma unroll
    for (int u = 0; u < MOVE_DEPTH; ++u)
      if (a.dst[u]) *reinterpret_cast<V*>(a.dst[u]) = data[u];
  }
}

// The 8-bit cache's V^T: a token is a column of its sub-tile, one byte in each
// of head_dim rows of W bytes. A thread takes one row and W tokens at a time.
__device__ __forceinline__ void move_columns(const Compact& P, const Plane& pl, int b, int head) {
  const int BS = 1 << P.bs_log2, W = min(BS, 16), D = pl.row_bytes;
  const int n = rows_to_move(P, b, threadIdx.x == 0 && head == 0);
  const bool on = int(threadIdx.x) < D;
  auto at = [&](int64_t slot) {
    const int off = int(slot & (BS - 1));
    return pl.base + ((slot >> P.bs_log2) * P.num_kv_heads + head) * pl.tile_bytes +
           (off / W) * (W * D) + int64_t(threadIdx.x) * W + off % W;
  };
  for (int j0 = 0; j0 < n; j0 += 16) {
    unsigned char x[16];
    unsigned char* to[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) {
      int64_t s, d;
      const bool go = move_of(P, b, j0 + u, n, threadIdx.x == 0 && head == 0, s, d) && on;
      to[u] = go ? at(d) : nullptr;
      if (go) x[u] = *at(s);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < 16; ++u)
      if (to[u]) *to[u] = x[u];
  }
}

// grid (KV head, sequence, slices of every plane)
__global__ void __launch_bounds__(MOVE_THREADS) compact_rows_kernel(const Compact P) {
  int z = blockIdx.z, p = 0;
  while (z >= P.plane[p].slices) z -= P.plane[p++].slices;
  const Plane& pl = P.plane[p];
  const int head = blockIdx.x, b = blockIdx.y;
  switch (pl.vec) {
    case 16: move_rows<uint4>(P, pl, b, head, z); break;
    case 8: move_rows<uint2>(P, pl, b, head, z); break;
    case 4: move_rows<uint32_t>(P, pl, b, head, z); break;
    default: move_columns(P, pl, b, head); break;
  }
}

// The weights of the kept tokens, moved in place; the rest of the row is zeroed.
__global__ void __launch_bounds__(256)
    compact_weights_kernel(const Compact P, float* weights, int64_t stride) {
  const int b = blockIdx.x;
  float* row = weights + b * stride;
  const int n = int(min(int64_t(rows_to_move(P, b, false)), stride));
  for (int j0 = 0; j0 < n; j0 += 256) {
    const int j = j0 + threadIdx.x;
    float x = 0.0f;
    bool go = false;
    if (j < n) {
      const int t = P.keep[int64_t(b) * P.keep_stride + j];
      go = t >= j && t < stride;
      if (go) x = row[t];
    }
    __syncthreads();
    if (go) row[j] = x;
  }
  __syncthreads();
  for (int64_t j = max(n, 0) + threadIdx.x; j < stride; j += 256) row[j] = 0.0f;
}

}  // namespace

int launch_evict_select(const float* token_weights, const int32_t* context_lens, int32_t* keep,
                        int32_t* new_lens, int32_t num_seqs, int64_t weights_stride,
                        int32_t budget, int32_t recent, void* stream) {
  Select P{token_weights, context_lens, keep, new_lens, weights_stride,
           num_seqs, budget, recent, int(weights_stride)};
  evict_select_kernel<<<unsigned(num_seqs), SEL_THREADS, 0, static_cast<cudaStream_t>(stream)>>>(P);
  return int(cudaGetLastError());
}

int launch_evict_compact(const pa_evict_compact_params* p, void* stream) {
  Compact P{};
  const int D = p->head_dim, BS = p->block_size;
  unsigned char* kv[2] = {static_cast<unsigned char*>(p->k_cache),
                          static_cast<unsigned char*>(p->v_cache)};
  int n = 0;
  for (int i = 0; i < 2; ++i) {
    if (p->kv_dtype == PA_KV_BF16) {
      P.plane[n++] = Plane{kv[i], BS * D * 2, 0, D * 2, 16, 1};
    } else if (p->kv_dtype == PA_KV_FP8_E4M3) {
      P.plane[n++] = Plane{kv[i], BS * D, 0, D, i == 0 ? 16 : 1, 1};
    } else {
      P.plane[n++] = Plane{kv[i], BS * D * 9 / 16, 0, D / 2, 16, 1};
      P.plane[n++] = Plane{kv[i], BS * D * 9 / 16, BS * D / 2, D / 16, D / 16, 1};
    }
  }
  // few sequences: several CTAs share a row, down to 32 bytes (a sector) each
  int64_t ctas = int64_t(p->num_seqs) * p->num_kv_heads * n;
  for (int i = 0; i < n; ++i)
    while (P.plane[i].vec == 16 && P.plane[i].row_bytes / P.plane[i].slices > 32 &&
           ctas * P.plane[i].slices < 152 * 4)
      P.plane[i].slices *= 2;
  int z = 0;
  for (int i = 0; i < n; ++i) z += P.plane[i].slices;
  P.src_tables = p->block_tables;
  P.dst_tables = p->dst_tables;
  P.keep = p->keep;
  P.new_lens = p->new_lens;
  P.src_blocks = p->max_blocks_per_seq;
  P.dst_blocks = p->max_dst_blocks_per_seq;
  P.keep_stride = p->keep_stride;
  P.num_kv_heads = p->num_kv_heads;
  P.num_blocks = p->num_blocks;
  P.bs_log2 = log2_of(BS);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const dim3 grid(unsigned(p->num_kv_heads), unsigned(p->num_seqs), unsigned(z));
  compact_rows_kernel<<<grid, MOVE_THREADS, 0, s>>>(P);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && p->token_weights) {
    compact_weights_kernel<<<unsigned(p->num_seqs), 256, 0, s>>>(P, p->token_weights,
                                                                 p->weights_stride);
    e = cudaGetLastError();
  }
  return int(e);
}

int read_and_clear_evict_errors(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_evict_errors, sizeof(v));
  if (e != cudaSuccess) return int(e);
  e = cudaMemcpyToSymbol(g_evict_errors, &zero, sizeof(zero));
  *flags = v;
  return int(e);
}

}  // namespace pa
