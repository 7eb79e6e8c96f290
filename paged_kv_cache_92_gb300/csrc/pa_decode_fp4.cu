// Paged decode attention over the 4-bit cache for sm_103a.
//
// For every sequence, new token and query head: softmax(scale q.K^T) V over
// the cached rows, K and V being code * group scale * head scale (the format
// is in pa_fp4.cu), with the block table, the running softmax and the causal
// rule of the bf16 decode ("Paged Attention as a Memory Manager", §How the
// Kernel Executes Paged Attention; "How Paged Attention and Continuous
// Batching Actually Work", §Continuous batching for several new tokens).
//
// What bounds it: the cache's bytes, 9/16 an element, once. That leaves an SM
// about three instruction lanes an element, so the design is about few
// instructions and no shared-memory round trip:
//  * A warp takes 32 keys a step. Its lanes copy the K and V tiles (each
//    contiguous: codes, then scales) into the warp's own ring with 16-byte
//    asynchronous copies; no CTA-wide barrier until the end. (1-D bulk copies
//    of the 1152-byte tiles cost more instructions, which are what is scarce.)
//  * S^T = K Q^T and O^T += V^T P^T are m16n8k16 products whose A operand is
//    the cache: codes go from shared memory to registers, are converted to
//    f16 pairs and multiplied by their group scale there (exact: a 2-bit and
//    a 4-bit significand), and never return. The query rows of a KV head, G
//    heads of up to 8 / G new tokens, are the products' 8 columns; more new
//    tokens are worked off in groups, whose re-read keys mostly come from L2.
//  * The order of elements inside a product is free as long as both operands
//    share it, so a lane reads its K elements as one run of head_dim / 4 codes.
//    For V the contraction runs over keys: the nibbles of two keys are merged
//    into one word (two logic operations for eight pairs) before conversion,
//    so each conversion yields one element of both keys, as the product needs.
//  * P^T comes out of the first product transposed to what the second one
//    wants; an 8x8 register transpose turns it.
//  * Queries are scaled by a power of two per row into f16's range (exact for
//    every element within 2^-29 of the row's largest) and the factor goes to
//    the softmax scale. P is rounded to f16, eight times finer than bf16 (no
//    cheaper form exists); the running maximum, the sums and the output stay in
//    fp32.
//  * P = exp2(score - reference), with the reference 2^7 below the largest weight
//    that it was taken from, and moved only when a weight exceeds that one by 2^8,
//    so O is rescaled rarely. P stays within 2^15, which f16 holds, and weights
//    down to 2^-21 of the row's largest are rounded by at most 2^-11 of their
//    value; lesser ones by at most 2^-32 of the largest (f16's subnormals, and zero
//    below them). With the reference at the largest weight that would be 2^-25: a
//    flat tail of a long context behind one large weight was lost, or half again as
//    large as it is. The difference is taken of the raw products, before the scale:
//    the scaled maximum, rounded, is off by up to 16 units from 2^28 on, which f16
//    does not hold (outputs were NaN). In pairs it costs what the single multiply-
//    add did: 144.9 us for the batch below, 147.0 one by one.
//  * Work is dealt out as a stream: every (sequence, column group, KV head) is
//    an item of so many 32-key steps plus a start cost, and each of the
//    persistent CTAs takes an equal stretch of the stream's cost, so ragged
//    lengths leave no tail. An item cut by a stretch's end leaves partials,
//    at most two a CTA, which a second launch joins by log-sum-exp. Batches
//    whose contexts are all short take one CTA an item and no second launch.
//
// Measured (GB300, whose copy rate is 6.79 TB/s): 32 sequences of 8 to 32 k
// tokens, 64 / 8 heads, d 128: 144.8 us, 5.83 TB/s of cache, 86 % of the copy
// rate; issuing the same instructions without waiting for memory takes 124 us,
// about what the bytes take, so neither hides the other entirely (52 % of issue
// slots, 50 % of the ALU, 24 % of the matrix unit busy on 8 such sequences).
// 64 sequences of up to 2 k tokens, 32 / 8 heads: 26.4 us, of which the bytes
// are 12.2 and some 10 are fixed: two launches, the plan, the first loads, the
// pieces' starts and the merge. Dropped: 5 or 6 CTAs an SM (spills: 175 us), a
// third ring stage (three CTAs an SM), one CTA per fixed partition (164 us), 1-D
// bulk copies (174 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_fp4.h"
#include "pa_mma.cuh"
#include "pa_ordered.cuh"

namespace pa {
namespace {

__device__ unsigned int g_decode_fp4_errors;

constexpr int NWARPS = 4;
constexpr int NTHREADS = NWARPS * 32;
constexpr int KEYS = 32;  // keys of a warp's step
constexpr int CTAS = 4;   // resident on an SM
constexpr float kLog2e = 1.4426950408889634f;
constexpr float HEADROOM = 7.0f;  // log2 of the weight that the reference gets

template <int D, int BS>
struct Cfg {
  static constexpr int NBK = KEYS / BS;              // blocks of a step
  static constexpr int TILE = BS * D * 9 / 16;       // bytes of one (block, KV head) tile
  static constexpr int STAGE = 2 * NBK * TILE;       // K tiles, then V tiles
  static constexpr int ST = D == 128 ? 2 : 4;        // ring stages per warp
  static constexpr int COLS = 8;
  static constexpr int OROW = D + 4;                 // padded row of the warps' merge
  static constexpr int RING = NWARPS * ST * STAGE;
  // after the rings: the queries, then the warps' (maximum, sum) per column; a
  // warp's rows of the merge lie in the second stage of its ring
  static constexpr int QUERIES = D * 16;
  static constexpr int SMEM = RING + QUERIES + NWARPS * COLS * 2 * 4;
  static_assert(COLS * OROW * 4 <= STAGE, "the merge rows fit a stage");
  static constexpr int WINDOW = 32 / NBK;            // steps whose table entries a warp holds
  static_assert(TILE % 16 == 0, "copies move 16 bytes");
};

struct Fp4Decode {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const unsigned char* k_cache;
  const unsigned char* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_tables;
  const int32_t* context_lens;
  int32_t* plan;    // [virtual sequences + 1]: cost before each, then the total
  float* part_ml;   // [2 * grid][COLS][2]: max, sum
  float* part_acc;  // [2 * grid][COLS][D]
  float scale_log2;
  int max_blocks_per_seq, num_kv_heads, num_blocks, cap;
  int g_log2;  // log2 of the query heads per KV head
  int q_len, q_group, n_groups;  // new tokens; of a column group; column groups
  int num_virtual;               // sequences * n_groups
  int whole;                     // one CTA per item, nothing is cut
};

// A virtual sequence: column group `grp` of sequence b.
struct Virtual {
  int see0;   // keys that the group's first token sees
  int n_tok;  // its tokens; the last one sees see0 + n_tok - 1 keys
  int steps;  // 0: an empty sequence, or one without room for the new tokens
};
__device__ __forceinline__ Virtual virtual_of(const Fp4Decode& P, int v) {
  const int b = v / P.n_groups, first = (v - b * P.n_groups) * P.q_group;
  const int L = min(P.context_lens[b], P.cap);
  Virtual x;
  x.n_tok = min(P.q_group, P.q_len - first);
  x.see0 = L - P.q_len + first + 1;
  x.steps = L < P.q_len || L <= 0 ? 0 : (x.see0 + x.n_tok - 1 + KEYS - 1) / KEYS;
  return x;
}
// The stream: an item (virtual sequence, KV head) costs its steps and a start
// (queries, pipeline fill, merge of the warps: about 990 instructions a warp,
// against 570 for one of its steps, four of which run at a time; 4 to 16 measure
// the same).
constexpr int START_COST = 8;
__device__ __forceinline__ int item_cost(const Virtual& x) {
  return x.steps > 0 ? x.steps + START_COST : 0;
}
// The stream's T positions (T below 2^31, checked on the host) in stretches of
// T / n or one more, at most one stretch per position, so that none is empty.
struct Deal {
  int n, base, longer;  // stretches; positions of one; how many hold one more
  __device__ __forceinline__ Deal(int T, int grid) {
    n = T < grid ? T : grid;
    base = n > 0 ? T / n : 0;
    longer = T - base * n;
  }
  __device__ __forceinline__ int start(int c) const { return c * base + min(c, longer); }
  __device__ __forceinline__ int owner(int x) const {  // the stretch that holds position x
    const int cut = longer * (base + 1);
    return x < cut ? x / (base + 1) : longer + (x - cut) / base;
  }
};

// Where this CTA's stretch begins: the virtual sequence that holds position x0
// and the cost before it. CTA 0 also writes the plan for the merge.
struct Start {
  int x0, x1, before, v;
};
__device__ __forceinline__ void find_start(const Fp4Decode& P, Start* out, int* warp_tot) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = (P.num_virtual + NTHREADS - 1) / NTHREADS;
  const int v0 = tid * per, v1 = min(P.num_virtual, v0 + per);
  if (tid == 0) *out = Start{0, 0, 0, 0};  // an empty stretch
  int sum = 0;
  for (int v = v0; v < v1; ++v) sum += item_cost(virtual_of(P, v)) * P.num_kv_heads;
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  int before = inc - sum, T = 0;
#pragma unroll
  for (int w = 0; w < NWARPS; ++w) {
    if (w < warp) before += warp_tot[w];
    T += warp_tot[w];
  }
  const Deal deal(T, gridDim.x);
  const int c = blockIdx.x;
  const int x0 = c < deal.n ? deal.start(c) : T, x1 = c < deal.n ? deal.start(c + 1) : T;
  const bool mine = x0 < x1 && before <= x0 && x0 < before + sum;
  if (mine || c == 0) {
    int at = before;
    for (int v = v0; v < v1; ++v) {
      const int cost = item_cost(virtual_of(P, v)) * P.num_kv_heads;
      if (c == 0) P.plan[v] = at;
      if (mine && at <= x0 && x0 < at + cost) *out = Start{x0, x1, at, v};
      at += cost;
    }
    if (c == 0 && tid == 0) P.plan[P.num_virtual] = T;
  }
  __syncthreads();
}

// A piece of an item: steps [first, last) of (virtual sequence v, KV head).
struct Piece {
  int v, head, first, last, steps;  // steps: of the whole item
  int see0, n_tok;                  // of the virtual sequence
  int valid;                        // 0: the stretch is done
};
// Walks a stretch piece by piece.
struct Walk {
  int x, x1, before, v;  // position, end, cost before virtual sequence v
  __device__ __forceinline__ Piece next(const Fp4Decode& P) {
    Piece p{};
    while (x < x1) {
      const Virtual q = virtual_of(P, v);
      const int cost = item_cost(q), all = cost * P.num_kv_heads;
      if (x >= before + all) {
        before += all;
        ++v;
        continue;
      }
      p.v = v;
      p.head = (x - before) / cost;
      const int base = before + p.head * cost;
      const int end = min(x1, base + cost);
      p.first = max(0, x - base - START_COST);
      p.last = end - base - START_COST;
      p.steps = q.steps;
      p.see0 = q.see0;
      p.n_tok = q.n_tok;
      x = end;
      p.valid = p.first < p.last;
      if (p.valid) break;
    }
    return p;
  }
};

template <int D, int BS>
__global__ void __launch_bounds__(NTHREADS, CTAS)
    paged_decode_fp4_kernel(const Fp4Decode P) {
  using C = Cfg<D, BS>;
  constexpr int ST = C::ST, NBK = C::NBK, TILE = C::TILE, WINDOW = C::WINDOW;
  constexpr int VW = D / 64;  // code words of a lane's share of a V row (D / 8 elements)
  dev::griddep_enter();  // the merge may be dispatched as CTAs end; it waits for all
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = 1 << P.g_log2;
  const int num_q_heads = P.num_kv_heads << P.g_log2;
  extern __shared__ __align__(128) unsigned char smem[];
  unsigned char* ring = smem + warp * ST * C::STAGE;
  uint4* sm_q = reinterpret_cast<uint4*>(smem + C::RING);    // [D / 32][32 lanes]
  float* sm_m = reinterpret_cast<float*>(smem + C::RING + C::QUERIES);  // [NWARPS][COLS]
  float* sm_l = sm_m + NWARPS * C::COLS;                     // [NWARPS][COLS]
  __shared__ Start start;
  __shared__ int warp_tot[NWARPS];
  __shared__ Walk walk;
  __shared__ Piece pieces[3];  // the one being worked on, the next, and the one after

  // thread 0 walks the stretch, two pieces ahead of the CTA
  if (P.whole) {
    if (tid == 0) {
      Piece p{};
      p.v = blockIdx.x / P.num_kv_heads;
      p.head = blockIdx.x - p.v * P.num_kv_heads;
      const Virtual q = virtual_of(P, p.v);
      p.last = p.steps = q.steps;
      p.see0 = q.see0;
      p.n_tok = q.n_tok;
      p.valid = q.steps > 0;
      pieces[0] = p;
      pieces[1] = Piece{};
      walk.x = walk.x1 = 0;
    }
  } else {
    find_start(P, &start, warp_tot);
    if (tid == 0) {
      walk = Walk{start.x0, start.x1, start.before, start.v};
      pieces[0] = walk.next(P);
      pieces[1] = walk.next(P);
    }
  }
  __syncthreads();

  const int64_t block_bytes = int64_t(P.num_kv_heads) * TILE;
  // Table entries of this warp's steps [w0, w0 + WINDOW) of the piece, one a
  // lane: step w0 + lane / NBK, block lane % NBK of it. Those past the piece
  // are read within the table row, and not used.
  auto load_window = [&](const Piece& p, int w0) {
    const int step = p.first + warp + NWARPS * (w0 + lane / NBK);
    const int j = min(step * NBK + lane % NBK, P.max_blocks_per_seq - 1);
    return P.block_tables[int64_t(p.v / P.n_groups) * P.max_blocks_per_seq + j];
  };
  bool bad_entry = false;  // a table entry outside the pool (block 0 is read in its place)
  // One copy group: step i of the warp (table entries in `window`), empty past the last.
  auto issue = [&](const Piece& p, int i, int n_my, int window, int stage) {
    if (i < n_my) {
      unsigned char* dst = ring + stage * C::STAGE + lane * 16;
      const int blk0 = (p.first + warp + NWARPS * i) * NBK;
      const int nblk = (p.see0 + p.n_tok - 1 + BS - 1) / BS;
      const unsigned char* k = P.k_cache + int64_t(p.head) * TILE + lane * 16;
      const unsigned char* v = P.v_cache + int64_t(p.head) * TILE + lane * 16;
#pragma unroll
      for (int j = 0; j < NBK; ++j) {
        int e = __shfl_sync(0xffffffffu, window, (i % WINDOW) * NBK + j);
        if (blk0 + j < nblk) {
          bad_entry |= e < 0 || e >= P.num_blocks;
          e = e < 0 || e >= P.num_blocks ? 0 : e;
          const int64_t off = e * block_bytes;
#pragma unroll
          for (int c = 0; c < TILE; c += 512) {
            const bool on = c + 512 <= TILE || lane * 16 < TILE - c;
            dev::cp_async16(dst + j * TILE + c, k + off + c, on);
            dev::cp_async16(dst + (NBK + j) * TILE + c, v + off + c, on);
          }
        }
      }
    }
    dev::cp_async_commit();
  };
  auto steps_of = [&](const Piece& p) {
    const int n = p.last - p.first;
    return n > warp ? (n - warp + NWARPS - 1) / NWARPS : 0;
  };

  // row of q / out of column n of a piece: new token n / G of the group, query
  // head head * G + n % G
  auto q_row = [&](const Piece& p, int n) {
    const int b = p.v / P.n_groups;
    return (int64_t(b) * P.q_len + (p.v - b * P.n_groups) * P.q_group + (n >> P.g_log2)) *
               num_q_heads + p.head * G + (n & (G - 1));
  };
  // What a warp has in hand when it turns to a piece; the loads start together,
  // then the first copies, into the ring's first stage.
  int window = 0;            // table entries of its first steps
  int n_my = 0;              // its steps
  float k_scale = 0.0f, v_scale = 0.0f;
  uint32_t qf[D / 16][2];    // the queries as the B operand (column g), in f16's range
  float inv_scaling = 1.0f;  // of this lane's query row
  auto begin = [&](const Piece& p) {
    const int n_cols = p.n_tok << P.g_log2;
    window = load_window(p, 0);
    n_my = steps_of(p);
    k_scale = P.k_scale[p.head];
    v_scale = P.v_scale[p.head];
    uint4 raw[D / 32];
    dev::query_load<PA_KV_FP4_E2M1, D>(P.q + q_row(p, min(g, n_cols - 1)) * D, g < n_cols, t, raw);
    issue(p, 0, n_my, window, 0);
    inv_scaling = dev::query_fragment<PA_KV_FP4_E2M1, D>(raw, qf);
    // a negative scale turns the queries, so that a larger product stays a larger score
    const uint32_t sign = k_scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
      qf[s][0] ^= sign;
      qf[s][1] ^= sign;
    }
    k_scale = fabsf(k_scale);
  };
  auto share_queries = [&]() {  // every warp has them; each writes a part
#pragma unroll
    for (int c = 0; c < D / 32; ++c)
      if (c == warp)
        sm_q[c * 32 + lane] = make_uint4(qf[2 * c][0], qf[2 * c][1], qf[2 * c + 1][0],
                                         qf[2 * c + 1][1]);
  };
  if (pieces[0].valid) {
    begin(pieces[0]);
    share_queries();
  }
  __syncthreads();
  int cur = 0;
  for (; pieces[cur].valid; cur = cur == 2 ? 0 : cur + 1) {
  const Piece& piece = pieces[cur];
  const int next = cur == 2 ? 0 : cur + 1, after = next == 2 ? 0 : next + 1;
  const int see0 = piece.see0, see_last = see0 + piece.n_tok - 1;
  const int n_cols = piece.n_tok << P.g_log2;
#pragma unroll
  for (int i = 1; i < ST; ++i) issue(piece, i, n_my, window, i);

  float factor[2];  // of columns 2t and 2t+1: softmax scale * K scale / the row's scaling
  int see[2];       // keys that columns 2t and 2t+1 see
  const float row_factor = P.scale_log2 * k_scale * inv_scaling;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    factor[c] = __shfl_sync(0xffffffffu, row_factor, 4 * (2 * t + c));
    // A scale of zero makes all scores equal, but 0 * -inf is NaN: below 2^-100 the
    // products (under 2^35) count as zero either way. The comparison keeps a NaN scale.
    factor[c] = factor[c] < 0x1p-100f ? 0x1p-100f : factor[c];
    see[c] = min(see_last, see0 + ((2 * t + c) >> P.g_log2));
  }

  float o[D / 16][4];  // O^T: D / 16 tiles of 16 rows
  // Softmax state of columns 2t and 2t+1. A score is s * factor in the log2 domain,
  // s the raw product; ref is the raw product that the reference was taken from (0
  // before the first key that the column sees), and a key's weight exp2((s - ref) *
  // factor + HEADROOM): the difference comes first, as the last place of a large
  // score is many units. limit: the raw product beyond which ref moves, 8 above it.
  float ref[2] = {0.0f, 0.0f}, limit[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;

  using KRow = dev::KeyRow<PA_KV_FP4_E2M1, D>;
  const int row_g = dev::key_row(g);                            // this lane's K rows
  const int row_a = dev::key_row(2 * t), row_b = dev::key_row(2 * t + 1);  // its V rows
  // where they lie in a tile, apart from what is the same for every lane
  const int lane_k = row_g * (D / 2) + t * KRow::RUN;
  const int lane_ks = BS * (D / 2) + row_g * (D / 16) + t * (D / 64);
  const int lane_va = row_a * (D / 2) + g * (D / 16), lane_vb = row_b * (D / 2) + g * (D / 16);
  const int lane_vsa = BS * (D / 2) + row_a * (D / 16) + (g * VW) / 2;
  const int lane_vsb = BS * (D / 2) + row_b * (D / 16) + (g * VW) / 2;

  int nan_from = INT32_MAX;  // first key of an edge step with a NaN among this lane's elements
  // One step; with EDGE the one that holds keys which some column does not see.
  auto step = [&](int i, int stage, auto edge_t) {
    constexpr bool EDGE = decltype(edge_t)::value;
    const unsigned char* kt = ring + stage * C::STAGE;
    const unsigned char* vt = kt + NBK * TILE;
    const int key0 = KEYS * (piece.first + warp + NWARPS * i);

    // ---- raw scores: two tiles of 16 keys
    float s[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int j = 0; j < 4; ++j) s[h][j] = 0.0f;
      KRow rows[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = h * 16 + r * 8;  // of a lane with row_g 0 (which is below 8)
        const unsigned char* tile = kt + (row / BS) * TILE;
        rows[r].load(tile + (row % BS) * (D / 2) + lane_k, tile + (row % BS) * (D / 16) + lane_ks);
      }
      dev::key_product_shared<PA_KV_FP4_E2M1, D>(s[h], rows[0], rows[1], sm_q + lane);
    }
    // ---- softmax; keys past a column's last are -inf
    bool over = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (EDGE && key0 + h * 16 + (j >> 1) * 8 + row_g >= see[j & 1]) s[h][j] = -INFINITY;
        over |= s[h][j] > limit[j & 1];
      }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = fmaxf(fmaxf(s[0][c], s[0][c + 2]), fmaxf(s[1][c], s[1][c + 2]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        // no branch here: lanes of different columns decide differently, and
        // the warp-wide instructions below need them together
        const bool first = limit[c] == -INFINITY;
        const bool take = x != -INFINITY && (first || x > ref[c]);
        const float y = take ? x : ref[c];
        const float b = dev::fast_exp2((ref[c] - y) * factor[c]);
        const float a = take && first ? 0.0f : b;
        ref[c] = y;
        // rounded down, so that no weight passes 2^15
        limit[c] = take ? __fadd_rd(x, __fdividef(8.0f - 0x1p-16f, factor[c])) : limit[c];
        l[c] *= a;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          o[k][c] *= a;
          o[k][c + 2] *= a;
        }
      }
    }
    __syncwarp();
    uint32_t pf[2][2];  // P^T as the second product's B operand
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float p[4];
#pragma unroll
      for (int r = 0; r < 4; r += 2) {  // a row's two columns
        const float2 e = dev::fma_pair(dev::sub_pair(make_float2(s[h][r], s[h][r + 1]), ref),
                                       factor, HEADROOM);
        p[r] = dev::fast_exp2(e.x);
        p[r + 1] = dev::fast_exp2(e.y);
        l[0] += p[r];
        l[1] += p[r + 1];
      }
      pf[h][0] = dev::transpose_8x8(dev::pack_f16(p[0], p[1]));
      pf[h][1] = dev::transpose_8x8(dev::pack_f16(p[2], p[3]));
    }

    // ---- O^T += V^T P^T
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[4][VW], sb[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = h * 16 + (r >> 1) * 8;  // as above
        const unsigned char* tile = vt + (row / BS) * TILE;
        const unsigned char* codes = tile + (row % BS) * (D / 2) + ((r & 1) ? lane_vb : lane_va);
        if constexpr (D == 128) {
          const uint2 x = *reinterpret_cast<const uint2*>(codes);
          w[r][0] = x.x; w[r][1] = x.y;
        } else {
          w[r][0] = *reinterpret_cast<const uint32_t*>(codes);
        }
        sb[r] = tile[(row % BS) * (D / 16) + ((r & 1) ? lane_vsb : lane_vsa)];
        if constexpr (EDGE) {
          // A key that is not there gets scale zero (its codes are finite). So
          // does one with a NaN scale, which some column may not see and which
          // 0 * NaN would carry there; the columns that see it get their NaN at
          // the end.
          const int key = key0 + row + ((r & 1) ? row_b : row_a);
          const bool nan = (sb[r] & 0x7Fu) == 0x7Fu;
          nan_from = nan ? min(nan_from, key) : nan_from;
          sb[r] = nan || key >= see_last ? 0u : sb[r];
        }
      }
      const uint32_t s01 = dev::e4m3x2_to_f16(sb[0] | sb[1] << 8);
      const uint32_t s23 = dev::e4m3x2_to_f16(sb[2] | sb[3] << 8);
#pragma unroll
      for (int c = 0; c < VW; ++c) {
        uint32_t e0[4], o0[4], e1[4], o1[4];
        dev::e2m1x8_to_f16((w[0][c] & 0x0F0F0F0Fu) | ((w[1][c] << 4) & 0xF0F0F0F0u), e0);
        dev::e2m1x8_to_f16(((w[0][c] >> 4) & 0x0F0F0F0Fu) | (w[1][c] & 0xF0F0F0F0u), o0);
        dev::e2m1x8_to_f16((w[2][c] & 0x0F0F0F0Fu) | ((w[3][c] << 4) & 0xF0F0F0F0u), e1);
        dev::e2m1x8_to_f16(((w[2][c] >> 4) & 0x0F0F0F0Fu) | (w[3][c] & 0xF0F0F0F0u), o1);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          dev::mma_f16(o[c * 4 + j], dev::mul_f16x2(e0[j], s01), dev::mul_f16x2(o0[j], s01),
                       dev::mul_f16x2(e1[j], s23), dev::mul_f16x2(o1[j], s23), pf[h][0], pf[h][1]);
      }
    }
  };

  // steps of the item before the first that is an edge, and this warp's share
  const int n_full = see0 / KEYS - piece.first;
  const int n_inner = n_full > warp ? (n_full - warp + NWARPS - 1) / NWARPS : 0;
  int ahead = window;  // table entries of the steps being issued
  for (int i = 0, stage = 0; i < n_my; ++i) {
    dev::cp_async_wait<ST - 1>();
    __syncwarp();
    if (i < n_inner)
      step(i, stage, std::false_type{});
    else
      step(i, stage, std::true_type{});
    __syncwarp();
    if ((i + ST) % WINDOW == 0) ahead = load_window(piece, i + ST);
    issue(piece, i + ST, n_my, ahead, stage);
    stage = stage + 1 == ST ? 0 : stage + 1;
  }
  dev::cp_async_wait<0>();
  __syncwarp();

  // ---- merge the warps through shared memory
  float* my_o = reinterpret_cast<float*>(ring + C::STAGE);  // [COLS][OROW]
  nan_from = min(nan_from, __shfl_xor_sync(0xffffffffu, nan_from, 1));
  nan_from = min(nan_from, __shfl_xor_sync(0xffffffffu, nan_from, 2));
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], x);
    const int n = warp * C::COLS + 2 * t + c;
    if (g == 0) {
      sm_m[n] = limit[c] == -INFINITY ? -INFINITY : fmaf(ref[c], factor[c], -HEADROOM);
      sm_l[n] = l[c];
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k)  // rows g and g + 8 of tile k: elements g D/8 + 2k, + 1
      *reinterpret_cast<float2*>(my_o + (2 * t + c) * C::OROW + g * (D / 8) + 2 * k) =
          nan_from < see[c] ? make_float2(NAN, NAN) : make_float2(o[k][c], o[k][c + 2]);
  }
  // the next piece's first steps are on their way during the merge
  const float scale_v = v_scale;
  if (pieces[next].valid) begin(pieces[next]);
  __syncthreads();
  if (pieces[next].valid) share_queries();
  if (tid == 0) pieces[after] = walk.next(P);
  {
    const Piece& done = piece;
    constexpr int TPC = NTHREADS / C::COLS;  // threads of a column
    constexpr int E = D / TPC;               // elements of a thread
    // columns past n_cols are computed along and not stored, so that no
    // branch parts the threads of a warp
    const int n = tid / TPC, d = tid % TPC * E;
    const bool on = n < n_cols;
    float wt[NWARPS], M = -INFINITY, den = 0.0f;
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) M = fmaxf(M, sm_m[w * C::COLS + n]);
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) {
      const float x = sm_m[w * C::COLS + n];
      const float y = dev::fast_exp2(x - M);
      wt[w] = x == -INFINITY ? 0.0f : y;
      den = fmaf(wt[w], sm_l[w * C::COLS + n], den);
    }
    const bool direct = done.first == 0 && done.last == done.steps;
    const float norm = direct ? scale_v / den : scale_v;
    const int slot = 2 * blockIdx.x + (done.first == 0);  // the CTA's last piece, or its first
    __nv_bfloat16* out = P.out + q_row(done, min(n, n_cols - 1)) * D + d;
    float* acc = P.part_acc + (int64_t(slot) * C::COLS + n) * D + d;
#pragma unroll
    for (int x = 0; x < E; x += 4) {
      float4 sum = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < NWARPS; ++w) {
        const float4 y =
            *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(
                smem + (w * ST + 1) * C::STAGE) + n * C::OROW + d + x);
        sum.x = fmaf(wt[w], y.x, sum.x);
        sum.y = fmaf(wt[w], y.y, sum.y);
        sum.z = fmaf(wt[w], y.z, sum.z);
        sum.w = fmaf(wt[w], y.w, sum.w);
      }
      __nv_bfloat162 r[2] = {__floats2bfloat162_rn(sum.x * norm, sum.y * norm),
                             __floats2bfloat162_rn(sum.z * norm, sum.w * norm)};
      if (direct && on) *reinterpret_cast<uint2*>(out + x) = *reinterpret_cast<const uint2*>(r);
      if (!direct && on)
        *reinterpret_cast<float4*>(acc + x) =
            make_float4(sum.x * norm, sum.y * norm, sum.z * norm, sum.w * norm);
    }
    if (!direct && on && d == 0)
      // (where every score is NaN there is no maximum, but the NaN has to reach the merge)
      *reinterpret_cast<float2*>(P.part_ml + (int64_t(slot) * C::COLS + n) * 2) =
          make_float2(den != den ? 0.0f : M, den);
  }
  __syncwarp();
  __syncthreads();  // before the next piece's copies
  }
  if (bad_entry && lane == 0) atomicOr(&g_decode_fp4_errors, PA_DEVERR_TABLE_ENTRY);

  // bad lengths are flagged, and rows of sequences without keys zeroed, by the CTAs in turn
  for (int v = blockIdx.x; v < P.num_virtual; v += gridDim.x) {
    const int b = v / P.n_groups, first = (v - b * P.n_groups) * P.q_group;
    const int L = P.context_lens[b];
    if (L > 0 && L >= P.q_len && L <= P.cap) continue;
    if (tid == 0 && first == 0 && L > 0) atomicOr(&g_decode_fp4_errors, PA_DEVERR_CONTEXT_LEN);
    if (L > 0 && min(L, P.cap) >= P.q_len) continue;
    const int n = min(P.q_group, P.q_len - first) * num_q_heads * D;
    __nv_bfloat16* row = P.out + (int64_t(b) * P.q_len + first) * num_q_heads * D;
    for (int i = tid; i < n; i += NTHREADS) row[i] = __float2bfloat16_rn(0.0f);
  }
}

// Joins the pieces of the items that were cut: one warp per (item, column).
template <int D>
__global__ void __launch_bounds__(128) merge_fp4_kernel(const Fp4Decode P, int grid) {
  constexpr int E = D / 32, COLS = Cfg<D, 16>::COLS;  // elements of a lane; columns
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int n = int(row % COLS);
  const int64_t item = row / COLS;
  const int v = int(item / P.num_kv_heads), head = int(item - int64_t(v) * P.num_kv_heads);
  if (v >= P.num_virtual) return;
  const Virtual x = virtual_of(P, v);
  // The plan and the partials. (No early dispatch of what follows: its CTAs would
  // find the SMs unevenly taken; the next decode of a 26 us batch took 29.)
  dev::griddep_wait();
  if (x.steps == 0 || n >= (x.n_tok << P.g_log2)) return;
  const int T = P.plan[P.num_virtual];
  const int base = P.plan[v] + head * item_cost(x) + START_COST;
  const Deal deal(T, grid);
  const int c0 = deal.owner(base), c1 = deal.owner(base + x.steps - 1);
  if (c0 == c1) return;  // one piece: written by the decode
  // four pieces at a time, their loads in flight together
  constexpr int BATCH = 4;
  float M = -INFINITY, den = 0.0f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.0f;
  for (int c = c0; c <= c1; c += BATCH) {
    float2 ml[BATCH], row[BATCH][E / 2];
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int64_t slot = int64_t(2 * min(c + k, c1) + (c + k == c0)) * COLS + n;
      ml[k] = *reinterpret_cast<const float2*>(P.part_ml + slot * 2);
#pragma unroll
      for (int e = 0; e < E / 2; ++e)
        row[k][e] = *reinterpret_cast<const float2*>(P.part_acc + slot * D + lane * E + 2 * e);
      if (c + k > c1) ml[k].x = -INFINITY;
    }
    float top = M;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) top = fmaxf(top, ml[k].x);
    const float a = M == -INFINITY ? 0.0f : dev::fast_exp2(M - top);
    M = top;
    den *= a;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] *= a;
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      if (ml[k].x == -INFINITY) continue;  // no keys of this column in the piece
      const float wt = dev::fast_exp2(ml[k].x - M);
      den = fmaf(wt, ml[k].y, den);
#pragma unroll
      for (int e = 0; e < E / 2; ++e) {
        acc[2 * e] = fmaf(wt, row[k][e].x, acc[2 * e]);
        acc[2 * e + 1] = fmaf(wt, row[k][e].y, acc[2 * e + 1]);
      }
    }
  }
  const float inv = __frcp_rn(den);
  const int b = v / P.n_groups, first = (v - b * P.n_groups) * P.q_group;
  const int group = 1 << P.g_log2;
  const int64_t q = (int64_t(b) * P.q_len + first + (n >> P.g_log2)) *
                        (P.num_kv_heads << P.g_log2) + head * group + (n & (group - 1));
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<__nv_bfloat162*>(P.out + q * D + lane * E + e) =
        __floats2bfloat162_rn(acc[e] * inv, acc[e + 1] * inv);
}

template <int D, int BS>
int launch_t(const Fp4Decode& P, int grid, cudaStream_t stream) {
  using C = Cfg<D, BS>;
  // the opt-in to large shared memory is per device
  static std::atomic<uint64_t> configured{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return int(e);
  const uint64_t bit = uint64_t(1) << (device & 63);
  if (!(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(paged_decode_fp4_kernel<D, BS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return int(e);
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  const int err = launch_ordered(paged_decode_fp4_kernel<D, BS>, dim3(unsigned(grid)), NTHREADS,
                                 C::SMEM, stream, 1, P);
  if (err || P.whole) return err;
  const int64_t rows = int64_t(P.num_virtual) * P.num_kv_heads * C::COLS;
  return launch_ordered(merge_fp4_kernel<D>, dim3(unsigned((rows + 3) / 4)), 128, 0, stream, 1, P,
                        grid);
}

template <int D>
int launch_bs(const Fp4Decode& P, int block_size, int grid, cudaStream_t s) {
  switch (block_size) {
    case 8: return launch_t<D, 8>(P, grid, s);
    case 16: return launch_t<D, 16>(P, grid, s);
    case 32: return launch_t<D, 32>(P, grid, s);
    default: return int(cudaErrorInvalidValue);
  }
}

}  // namespace

Fp4Plan fp4_plan(const pa_decode_params* p, int num_sms) {
  Fp4Plan r{};
  const MmaColumns cols = fp4_columns(p);
  const int64_t table = int64_t(p->max_blocks_per_seq) * p->block_size;
  r.cap = int(p->max_context_len < table ? p->max_context_len : table);
  const int64_t items = int64_t(p->num_seqs) * cols.n_groups * p->num_kv_heads;
  r.cols = 8;
  r.whole = r.cap <= kFp4WholeTokens;
  if (r.whole) {
    r.grid = int(items);
  } else {
    // as many CTAs as are resident at once, but no stretch under two start costs (for 2,
    // 3, 4, 8 CTAs an SM: 29.6, 26.6, 26.2, 30.7 us on 64 sequences of up to 2 k tokens,
    // 161, 147, 145, 147 on 32 of up to 32 k)
    const int64_t most = items * ((r.cap + KEYS - 1) / KEYS + START_COST) / (2 * START_COST);
    const int64_t full = int64_t(num_sms > 0 ? num_sms : 256) * CTAS;
    r.grid = int(most < full ? most : full);
    if (r.grid < 1) r.grid = 1;
  }
  return r;
}

int launch_decode_fp4(const DecodeLaunch& L, const Fp4Plan& plan, void* stream) {
  const pa_decode_params* p = L.p;
  const MmaColumns cols = fp4_columns(p);
  Fp4Decode P;
  P.q = static_cast<const __nv_bfloat16*>(p->q);
  P.out = static_cast<__nv_bfloat16*>(p->out);
  P.k_cache = static_cast<const unsigned char*>(p->k_cache);
  P.v_cache = static_cast<const unsigned char*>(p->v_cache);
  P.k_scale = p->k_scale;
  P.v_scale = p->v_scale;
  P.block_tables = p->block_tables;
  P.context_lens = p->context_lens;
  P.plan = L.plan;
  P.part_ml = L.part_m;
  P.part_acc = L.part_acc;
  P.scale_log2 = p->scale * kLog2e;
  P.max_blocks_per_seq = p->max_blocks_per_seq;
  P.num_kv_heads = p->num_kv_heads;
  P.num_blocks = p->num_blocks;
  P.cap = plan.cap;
  P.g_log2 = log2_of(p->num_q_heads / p->num_kv_heads);
  P.q_len = query_len_of(p);
  P.q_group = cols.q_group;
  P.n_groups = cols.n_groups;
  P.num_virtual = p->num_seqs * cols.n_groups;
  P.whole = plan.whole;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (p->head_dim) {
    case 64: return launch_bs<64>(P, p->block_size, plan.grid, s);
    case 128: return launch_bs<128>(P, p->block_size, plan.grid, s);
    default: return int(cudaErrorInvalidValue);
  }
}

int read_and_clear_decode_fp4_errors(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_decode_fp4_errors, sizeof(v));
  if (e != cudaSuccess) return int(e);
  if (v != 0) e = cudaMemcpyToSymbol(g_decode_fp4_errors, &zero, sizeof(zero));
  *flags = v;
  return int(e);
}

}  // namespace pa
