// Eviction of cached tokens for sm_103a: the choice of the tokens to keep
// under a budget, and the move of their rows.
//
// The pages describe the pool's side of memory pressure (blocks reclaimed,
// "How Paged Attention and Continuous Batching Actually Work"); which tokens
// go is left open. Here the most recent ones stay, and of the others those
// with the largest accumulated attention weight (pa_weights.cu).
//
//  * evict_select_kernel: one CTA per sequence, or a cluster of up to eight for
//    long ones, each with its share of the tokens. The candidates' weights become
//    ordered 32-bit keys in registers (up to 8 a thread; longer ranges re-read
//    them from L2), and the threshold is found by three rounds of a
//    shared-memory histogram over 11, 11 and 10 bits of the keys that still
//    tie with it (fewer where a bin is kept whole, as one of a single key is);
//    the CTAs of a cluster read each other's. Four copies of the
//    histogram, by lane, keep equal weights -- most tokens of a long context
//    have nearly none -- from serialising more than eight deep. Ties go to the
//    lowest index through ranks, and the kept indices come out ascending.
//  * compact_rows_kernel: row j of the destination <- row keep[j] of the
//    source. keep ascends, so keep[j] >= j, and moving rows in order within
//    one CTA is safe in place: a tile's rows are in registers before any of
//    them is overwritten, and later tiles read only rows behind it. A CTA
//    owns one (sequence, KV head) and a slice of the row's bytes, so CTAs never
//    meet. Bound by memory traffic: every kept row is read and written once,
//    and rows that stay where they are not at all.
// Measured (GB300, copy rate 6.79 TB/s): 64 sequences of up to 2 k tokens cut to
// 512, bf16, 8 KV heads, d 128: 51.0 us, of which the choice takes 7 and the move
// 44 (its bytes: 37.9 us); 8 of 8 to 32 k cut to 4 k: 67.4 us, 16 and 51 (39.7).
// The choice is a chain of short steps in few CTAs, one on an SM: its warps' stalls
// are the first loads and the cluster's reads (23 %), barriers (14 %), the
// histograms (9 %), and the rest instructions. Its CTAs a sequence follow the row of
// weights, not the lengths, which it does not know on the host: 64 sequences of 2 k
// tokens take 6.9 us in rows of 2,051 weights and 53 in rows of 131,072. The weights'
// rows moved along cost 2 to 8 us more (64 sequences cut to 512 4.6 us and 6.4, one
// head of d 64; 8 of 32 k cut to 4 k 19 and 27), 17 us where 64 rows of 131,072 are
// zeroed.
// The move of few sequences has 512 CTAs for 152 SMs and rows in 64-byte slices;
// slices of 128 or 32 bytes take 10 and 16 us more, tiles of twice or half the
// rows 24 and 6 (64 registers let four CTAs share an SM, so that all 512 are
// resident; larger tiles do not), and clusters that share a tile's rows instead of
// their bytes 1 to 4.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_device.cuh"
#include "pa_fp4.h"
#include "pa_ordered.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned int g_evict_errors;

// ---------------------------------------------------------------- selection

constexpr int SEL_THREADS = 1024;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_KEYS = 8;       // keys a thread holds at a time
constexpr int SEL_BINS = 2048;
constexpr int SEL_COPIES = 4;
constexpr int SEL_CLUSTER = 8;    // CTAs of a sequence, at most

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

// Inclusive prefix of x over the CTA's threads; `all` is the total.
__device__ __forceinline__ int block_scan(int x, int* warp_tot, int& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int inc = x;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();  // the previous scan's totals have been read
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  const int tot = warp_tot[lane];
  int run = tot;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, run, o);
    if (lane >= o) run += y;
  }
  all = __shfl_sync(0xffffffffu, run, 31);
  return inc + __shfl_sync(0xffffffffu, run - tot, warp);
}

struct SelectShared {
  int hist[SEL_COPIES][SEL_BINS];
  int bins[2][SEL_BINS];           // their sum, read by the cluster; alternates
  int cnt[SEL_KEYS * SEL_WARPS];
  int warp_tot[SEL_WARPS];
  int bin, left, done;
  int above, equal;                // keys of the CTAs before this one
};

// The choice for one sequence of more than `budget` tokens, E keys a thread at
// a time. This CTA, rank `rank` of `ctas`, has the candidates [c0, c1); key e of
// span s is token c0 + s * SEL_THREADS * E + e * SEL_THREADS + tid.
template <int E>
__device__ __forceinline__ void select_row(const Select& P, const float* w, int32_t* keep, int L,
                                           SelectShared& sm, cg::cluster_group& cluster) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = int(cluster.block_rank()), ctas = int(cluster.num_blocks());
  const int n_cand = L - P.recent;       // the others always stay
  const int need = P.budget - P.recent;  // of the candidates, fewer than n_cand
  const int share = (n_cand + ctas - 1) / ctas;
  const int c0 = min(n_cand, rank * share), c1 = min(n_cand, c0 + share);
  const int span_len = SEL_THREADS * E;
  const int spans = (c1 - c0 + span_len - 1) / span_len;
  uint32_t key[E];
  auto token = [&](int span, int e) { return c0 + span * span_len + e * SEL_THREADS + tid; };
  auto load = [&](int span) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int i = token(span, e);
      key[e] = i < c1 ? weight_key(w[i]) : 0u;
    }
  };
  if (spans == 1) load(0);

  // the key of rank `need`, digit by digit, as far as it has to be known; `left`:
  // how many of the keys that equal it in these digits are kept (the first ones)
  uint32_t prefix = 0, mask = 0;
  int left = need;
  if (tid == 0) sm.above = sm.equal = 0;
  if (need > 0) {
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : (round == 1 ? 10 : 0);
      const uint32_t digits = round == 2 ? 1023u : 2047u;
      for (int i = tid; i < SEL_COPIES * SEL_BINS; i += SEL_THREADS) (&sm.hist[0][0])[i] = 0;
      __syncthreads();
      for (int span = 0; span < spans; ++span) {
        if (spans > 1) load(span);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const bool in = token(span, e) < c1 && (key[e] & mask) == prefix;
          if (in) atomicAdd(&sm.hist[lane % SEL_COPIES][(key[e] >> shift) & digits], 1);
        }
      }
      __syncthreads();
      // bins from the top, two a thread: where the count reaches `left`
      const int b1 = SEL_BINS - 1 - 2 * tid, b0 = b1 - 1;
      int n1 = 0, n0 = 0;
#pragma unroll
      for (int k = 0; k < SEL_COPIES; ++k) {
        n1 += sm.hist[k][b1];
        n0 += sm.hist[k][b0];
      }
      int before1 = 0, before0 = 0;  // of the CTAs before this one
      if (ctas > 1) {
        int* mine = &sm.bins[round & 1][b0];
        *reinterpret_cast<int2*>(mine) = make_int2(n0, n1);
        cluster.sync();  // (the buffer's last readers passed the previous one)
        n1 = n0 = 0;
        int2 x[SEL_CLUSTER];
#pragma unroll
        for (int k = 0; k < SEL_CLUSTER; ++k)
          if (k < ctas)
            x[k] = *reinterpret_cast<const int2*>(cluster.map_shared_rank(mine, unsigned(k)));
#pragma unroll
        for (int k = 0; k < SEL_CLUSTER; ++k) {
          if (k < ctas) {
            n0 += x[k].x;
            n1 += x[k].y;
          }
          if (k < rank) {
            before0 += x[k].x;
            before1 += x[k].y;
          }
        }
      }
      int all;
      const int upto = block_scan(n1 + n0, sm.warp_tot, all), before = upto - n1 - n0;
      if (before < left && left <= upto) {
        const bool first = left <= before + n1;
        sm.bin = first ? b1 : b0;
        const int rest = left - before - (first ? 0 : n1);
        sm.left = rest;
        sm.done = rest == (first ? n1 : n0);  // the whole bin is kept: no need to look further
      }
      __syncthreads();
      const int bin = sm.bin;
      prefix |= uint32_t(bin) << shift;
      mask |= digits << shift;
      left = sm.left;
      const bool done = sm.done || round == 2;
      if (ctas > 1) {
        const int above = __reduce_add_sync(0xffffffffu, (b1 > bin ? before1 : 0) +
                                                             (b0 > bin ? before0 : 0));
        if (lane == 0 && above) atomicAdd(&sm.above, above);
        if (done && (b1 == bin || b0 == bin)) sm.equal = b1 == bin ? before1 : before0;
      }
      __syncthreads();
      if (done) break;
    }
  }
  // of the CTAs before this one: keys that equal the threshold, keys that are kept
  int eq_base = sm.equal, keep_base = sm.above + min(sm.equal, left);
  // ranks in token order: of the keys equal to the threshold, then of the kept
  const uint32_t below = (1u << lane) - 1u;
  // exclusive prefix of the warps' counts, in token order (entry e * SEL_WARPS + warp)
  auto scan_counts = [&](int base) {
    __syncthreads();
    const int x = tid < E * SEL_WARPS ? sm.cnt[tid] : 0;
    int all;
    const int inc = block_scan(x, sm.warp_tot, all);
    if (tid < E * SEL_WARPS) sm.cnt[tid] = base + inc - x;
    __syncthreads();
    return all;
  };
  for (int span = 0; span < spans; ++span) {
    if (spans > 1) load(span);
    uint32_t kept = 0, eq = 0;  // a bit per key
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool cand = token(span, e) < c1 && need > 0;
      const bool same = cand && (key[e] & mask) == prefix;
      kept |= uint32_t(cand && (key[e] & mask) > prefix) << e;
      eq |= uint32_t(same) << e;
      const uint32_t v = __ballot_sync(0xffffffffu, same);
      if (lane == 0) sm.cnt[e * SEL_WARPS + warp] = __popc(v);
    }
    const int eq_all = scan_counts(eq_base);
    uint32_t in_kept[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool same = (eq >> e) & 1u;
      const uint32_t v = __ballot_sync(0xffffffffu, same);
      const int at = sm.cnt[e * SEL_WARPS + warp] + __popc(v & below);
      const bool on = ((kept >> e) & 1u) || (same && at < left);
      in_kept[e] = __ballot_sync(0xffffffffu, on);
    }
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (lane == 0) sm.cnt[e * SEL_WARPS + warp] = __popc(in_kept[e]);
    const int keep_all = scan_counts(keep_base);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if ((in_kept[e] >> lane) & 1u)
        keep[sm.cnt[e * SEL_WARPS + warp] + __popc(in_kept[e] & below)] = token(span, e);
    eq_base += eq_all;
    keep_base += keep_all;
    __syncthreads();
  }
  for (int j = rank * SEL_THREADS + tid; j < P.recent; j += ctas * SEL_THREADS)
    keep[need + j] = n_cand + j;
  if (ctas > 1 && need > 0) cluster.sync();  // no CTA leaves while another reads its bins
}

// grid (CTAs of a sequence, sequence), in clusters of gridDim.x
__global__ void __launch_bounds__(SEL_THREADS) evict_select_kernel(const Select P) {
  __shared__ SelectShared sm;
  dev::griddep_enter();
  cg::cluster_group cluster = cg::this_cluster();
  const int b = blockIdx.y, tid = threadIdx.x;
  const int first = blockIdx.x * SEL_THREADS + tid, stride = gridDim.x * SEL_THREADS;
  int L = P.context_lens[b];
  if (L > P.max_len) {
    if (first == 0) atomicOr(&g_evict_errors, PA_DEVERR_CONTEXT_LEN);
    L = P.max_len;
  }
  L = max(L, 0);
  const int n_keep = min(L, P.budget);
  int32_t* keep = P.keep + int64_t(b) * P.budget;
  if (first == 0) P.new_lens[b] = n_keep;
  for (int j = n_keep + first; j < P.budget; j += stride) keep[j] = -1;
  if (L <= P.budget) {
    for (int j = first; j < L; j += stride) keep[j] = j;
    return;
  }
  const float* w = P.weights + int64_t(b) * P.weights_stride;
  // no more keys a thread than the sequence needs
  if ((L - P.recent + int(gridDim.x) - 1) / int(gridDim.x) <= 2 * SEL_THREADS)
    select_row<2>(P, w, keep, L, sm, cluster);
  else
    select_row<SEL_KEYS>(P, w, keep, L, sm, cluster);
}

// ---------------------------------------------------------------- compaction

constexpr int MOVE_THREADS = 256;
constexpr int MOVE_DEPTH = 4;    // rows a thread has in flight, twice
constexpr int MOVE_LIST = 512;   // rows whose places are looked up at a time

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

// Row j's source and destination as slots (block * block_size + offset);
// src = -1 where the row cannot be moved.
struct Move {
  int64_t src, dst;
};
__device__ __forceinline__ Move places_of(const Compact& P, int b, int j, int t, bool report) {
  Move m{-1, 0};
  if (t < j || (t >> P.bs_log2) >= P.src_blocks) {  // not ascending, or no such row
    if (report) atomicOr(&g_evict_errors, PA_DEVERR_KEEP);
    return m;
  }
  const int sb = P.src_tables[int64_t(b) * P.src_blocks + (t >> P.bs_log2)];
  const int db = P.dst_tables[int64_t(b) * P.dst_blocks + (j >> P.bs_log2)];
  if (sb < 0 || sb >= P.num_blocks || db < 0 || db >= P.num_blocks) {
    if (report) atomicOr(&g_evict_errors, PA_DEVERR_TABLE_ENTRY);
    return m;
  }
  const int mask = (1 << P.bs_log2) - 1;
  m.src = (int64_t(sb) << P.bs_log2) + (t & mask);
  m.dst = (int64_t(db) << P.bs_log2) + (j & mask);
  return m;
}
// The same, with src = -1 also for a row that stays where it is.
__device__ __forceinline__ Move move_of(const Compact& P, int b, int j, int t, bool report) {
  Move m = places_of(P, b, j, t, report);
  if (m.src == m.dst) m.src = -1;
  return m;
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

// The moves of rows [j0, j0 + MOVE_LIST) in shared memory. `t` holds this
// thread's keep entries of those rows, and on return those of the next ones, so
// that a list costs one dependent load (the tables) and not two.
constexpr int MOVE_EACH = MOVE_LIST / MOVE_THREADS;
__device__ __forceinline__ void load_keep(const Compact& P, int b, int j0, int n,
                                          int (&t)[MOVE_EACH]) {
#pragma unroll
  for (int k = 0; k < MOVE_EACH; ++k) {
    const int j = j0 + k * MOVE_THREADS + threadIdx.x;
    t[k] = j < n ? P.keep[int64_t(b) * P.keep_stride + j] : 0;
  }
}
__device__ __forceinline__ void fill_list(const Compact& P, int b, int j0, int n, bool report,
                                          int (&t)[MOVE_EACH], Move* list) {
  Move m[MOVE_EACH];
#pragma unroll
  for (int k = 0; k < MOVE_EACH; ++k) {
    const int j = j0 + k * MOVE_THREADS + threadIdx.x;
    m[k] = j < n ? move_of(P, b, j, t[k], report) : Move{-1, 0};
  }
  __syncthreads();  // the previous list is done with
#pragma unroll
  for (int k = 0; k < MOVE_EACH; ++k) list[k * MOVE_THREADS + threadIdx.x] = m[k];
  load_keep(P, b, j0 + MOVE_LIST, n, t);
  __syncthreads();
}

// One tile of rows is on its way while the previous one is written: its
// sources lie behind the rows that are overwritten, so their order does not
// matter.
template <typename V>
__device__ __forceinline__ void move_rows(const Compact& P, const Plane& pl, int b, int head,
                                          int slice, Move* list) {
  const int per_row = pl.row_bytes / pl.slices / int(sizeof(V));  // threads of a row
  const int lane = threadIdx.x % per_row, r = threadIdx.x / per_row;
  const int rows = MOVE_THREADS / per_row;                        // rows of a pass
  const bool report = head == 0 && slice == 0;
  const int n = rows_to_move(P, b, report && threadIdx.x == 0);
  const int BS = 1 << P.bs_log2;
  unsigned char* base = pl.base + int64_t(head) * pl.tile_bytes + pl.first +
                        (slice * per_row + lane) * int(sizeof(V));
  const int64_t block_bytes = int64_t(P.num_kv_heads) * pl.tile_bytes;
  auto at = [&](int64_t slot) {
    return base + (slot >> P.bs_log2) * block_bytes + int(slot & (BS - 1)) * pl.row_bytes;
  };
  int t[MOVE_EACH];
  load_keep(P, b, 0, n, t);
  for (int j0 = 0; j0 < n; j0 += MOVE_LIST) {
    fill_list(P, b, j0, n, report, t, list);
    const int m = min(MOVE_LIST, n - j0);
    V data[MOVE_DEPTH], more[MOVE_DEPTH];
    auto load = [&](int i0, V (&d)[MOVE_DEPTH]) {
#pragma unroll
      for (int u = 0; u < MOVE_DEPTH; ++u) {
        const int i = i0 + u * rows + r;
        if (i < m && list[i].src >= 0) d[u] = *reinterpret_cast<const V*>(at(list[i].src));
      }
    };
    load(0, data);
    for (int i0 = 0; i0 < m; i0 += rows * MOVE_DEPTH) {
      load(i0 + rows * MOVE_DEPTH, more);
      __syncthreads();  // the tile's rows are read before any of them is overwritten
#pragma unroll
      for (int u = 0; u < MOVE_DEPTH; ++u) {
        const int i = i0 + u * rows + r;
        if (i < m && list[i].src >= 0) *reinterpret_cast<V*>(at(list[i].dst)) = data[u];
        data[u] = more[u];
      }
    }
  }
}

// The 8-bit cache's V^T: a token is a column of its sub-tile, one byte in each
// of head_dim rows of W bytes. A thread takes one row and 16 tokens at a time.
__device__ __forceinline__ void move_columns(const Compact& P, const Plane& pl, int b, int head,
                                             Move* list) {
  const int BS = 1 << P.bs_log2, W = min(BS, 16), D = pl.row_bytes;
  const int n = rows_to_move(P, b, threadIdx.x == 0 && head == 0);
  const bool on = int(threadIdx.x) < D;
  auto at = [&](int64_t slot) {
    const int off = int(slot & (BS - 1));
    return pl.base + ((slot >> P.bs_log2) * P.num_kv_heads + head) * pl.tile_bytes +
           (off / W) * (W * D) + int64_t(threadIdx.x) * W + off % W;
  };
  int t[MOVE_EACH];
  load_keep(P, b, 0, n, t);
  for (int j0 = 0; j0 < n; j0 += MOVE_LIST) {
    fill_list(P, b, j0, n, head == 0, t, list);
    const int m = min(MOVE_LIST, n - j0);
    for (int i0 = 0; i0 < m; i0 += 16) {
      unsigned char x[16];
#pragma unroll
      for (int u = 0; u < 16; ++u)
        if (on && i0 + u < m && list[i0 + u].src >= 0) x[u] = *at(list[i0 + u].src);
      __syncthreads();
#pragma unroll
      for (int u = 0; u < 16; ++u)
        if (on && i0 + u < m && list[i0 + u].src >= 0) *at(list[i0 + u].dst) = x[u];
    }
  }
}

// grid (KV head, sequence, slices of every plane)
__global__ void __launch_bounds__(MOVE_THREADS) compact_rows_kernel(const Compact P) {
  __shared__ Move list[MOVE_LIST];
  dev::griddep_enter();
  int z = blockIdx.z, p = 0;
  while (z >= P.plane[p].slices) z -= P.plane[p++].slices;
  const Plane& pl = P.plane[p];
  const int head = blockIdx.x, b = blockIdx.y;
  switch (pl.vec) {
    case 16: move_rows<uint4>(P, pl, b, head, z, list); break;
    case 8: move_rows<uint2>(P, pl, b, head, z, list); break;
    case 4: move_rows<uint32_t>(P, pl, b, head, z, list); break;
    default: move_columns(P, pl, b, head, list); break;
  }
}

// The weights of the kept tokens, moved in place; the rest of the row is zeroed.
// A weight goes where its row goes: it stays where that is not moved. That of a
// token past the end of the weights is unknown: zero, and flagged.
__global__ void __launch_bounds__(256)
    compact_weights_kernel(const Compact P, float* weights, int64_t stride) {
  dev::griddep_enter();
  const int b = blockIdx.x;
  float* row = weights + b * stride;
  const int n = int(min(int64_t(rows_to_move(P, b, false)), stride));
  auto keep = [&](int j) { return j < n ? P.keep[int64_t(b) * P.keep_stride + j] : 0; };
  int t = keep(threadIdx.x), next;
  for (int j0 = 0; j0 < n; j0 += 256, t = next) {
    const int j = j0 + threadIdx.x;
    float x = 0.0f;
    bool go = false;
    next = keep(j + 256);  // on its way while this one's weight and tables are looked up
    if (j < n) {
      if (t >= 0 && t < stride) x = row[t];
      go = places_of(P, b, j, t, false).src >= 0;
      if (go && t >= stride) atomicOr(&g_evict_errors, PA_DEVERR_KEEP);
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
  const Select P{token_weights, context_lens, keep, new_lens, weights_stride,
                 num_seqs, budget, recent, int(weights_stride)};
  // As many CTAs as hold a row's candidates in registers, by the longest row there
  // may be (8 sequences of 8 k tokens: 10.9 us with one CTA or four; of 10 k: 17.6
  // with one, 14.1 with four; of 32 k: 32 and 15.2, 18.0 with eight; one of 40 k:
  // 25.6 with four, 17.6 with eight; two are no faster than four).
  const int64_t most = weights_stride - recent, one = SEL_THREADS * SEL_KEYS;
  const unsigned ctas = most > 4 * one ? 8 : (most > one ? 4 : 1);
  return launch_ordered(evict_select_kernel, dim3(ctas, unsigned(num_seqs)), SEL_THREADS, 0,
                        static_cast<cudaStream_t>(stream), ctas, P);
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
  // few sequences: several CTAs share a row, down to 64 bytes (an HBM access) each,
  // for about six CTAs an SM
  const int64_t ctas = int64_t(p->num_seqs) * p->num_kv_heads * n;
  for (int i = 0; i < n; ++i)
    while (P.plane[i].vec == 16 && P.plane[i].row_bytes / P.plane[i].slices > 64 &&
           ctas * P.plane[i].slices < 152 * 6)
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
  int e = launch_ordered(compact_rows_kernel, grid, MOVE_THREADS, 0, s, 1, P);
  if (e == 0 && p->token_weights)
    e = launch_ordered(compact_weights_kernel, dim3(unsigned(p->num_seqs)), 256, 0, s, 1, P,
                       p->token_weights, int64_t(p->weights_stride));
  return e;
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
