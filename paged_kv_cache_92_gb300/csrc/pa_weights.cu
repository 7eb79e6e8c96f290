// Attention weights of the cached tokens for sm_103a: what the new tokens of
// each sequence look at, summed over query heads and new tokens,
//   w[b][t] (+)= sum_i sum_h exp(scale q[b,i,h].k[b,t] - lse[b,i,h]),
// t in the keys that new token i sees. Accumulated over steps this ranks the
// cached tokens for eviction (pa_evict.cu). The pages leave the policy open.
//
// What bounds it: K read once. A weight needs its row's log-sum-exp, which
// needs every score first, so the work is two launches:
//  * token_scores_kernel reads K (bf16, 8-bit or 4-bit rows, in registers as
//    in the 4-bit decode), writes each score once (fp32, log2 domain, 4 G
//    bytes a K row of 256, 128 or 72) and each partition's (max, sum);
//  * sum_weights_kernel joins the partitions' sums and adds up exp2(score -
//    max) / sum over the rows of a token, in a fixed order: no atomics, the
//    same bits on every run.
// Reading K twice instead would cost 256 (128, 72) bytes a row against the
// scores' 8 G (of one new token), so the scores win for every type up to G = 8.
// The keys of a (sequence, KV head) are split into partitions, a CTA each, for
// about 8 CTAs an SM when every sequence is as long as the longest. Measured
// (GB300, copy rate 6.79 TB/s): 64 sequences of up to 2 k tokens, bf16, 32 / 8
// heads: 31.0 us for 20.0 us of traffic (4.3 TB/s), of which the scores take about
// 26 (three CTAs of four warps on an SM, for the rings' shared memory; DRAM 61 %;
// a third of the stalls are the lengths, tables and queries that a CTA starts with)
// and the sums 5; 8 of 8 to 32 k, 4-bit, 64 / 8 heads: 38.8 us for 15.6, of which
// the scores take about 28 (issue slots half busy, DRAM 39 %: starts and the uneven
// ends of one wave of CTAs) and the sums 10. Dropped: 10 to 16 CTAs an SM (41 to 42
// us; for the bf16 batch 30.8 to 31.2), a persistent stream as in the 4-bit decode
// (49), the partition as the slowest grid index (+5 us), two or three ring stages,
// with as many more CTAs on an SM or without (+4 to +20).
// Scores, sums and weights are fp32; 8-bit and 4-bit rows enter the products
// exactly (f16 holds them), and so do the queries beside them (scaled to f16 by a
// power of two: exact within 2^-29 of a row's largest element).
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

__device__ unsigned int g_weights_errors;

constexpr int NWARPS = 4;
constexpr int NTHREADS = NWARPS * 32;
constexpr int KEYS = 32;  // keys of a warp's step
constexpr float kLog2e = 1.4426950408889634f;

struct Weights {
  const __nv_bfloat16* q;
  const unsigned char* k_cache;
  const float* k_scale;
  const int32_t* block_tables;
  const int32_t* context_lens;
  float* token_weights;
  float* scores;   // [sequence][new token][query head][score_stride]
  float2* part;    // [sequence][new token][query head][partitions]: max, sum
  int64_t score_stride;
  float scale_log2;
  int weights_stride, max_blocks_per_seq, num_seqs, num_kv_heads, num_blocks, cap;
  int bs_log2, g_log2;
  int q_len, q_group, n_groups;
  int partition_tokens, num_partitions;
  int accumulate;
};

// Length of sequence b (0 where it cannot hold the new tokens), flagged once.
__device__ __forceinline__ int checked_len(const Weights& P, int b, bool report) {
  int L = P.context_lens[b];
  if (L > P.cap) {
    if (report) atomicOr(&g_weights_errors, PA_DEVERR_CONTEXT_LEN);
    L = P.cap;
  }
  if (L > 0 && L < P.q_len) {
    if (report) atomicOr(&g_weights_errors, PA_DEVERR_CONTEXT_LEN);
    L = 0;
  }
  return max(L, 0);
}

template <int FMT, int D>
struct Ring {
  static constexpr int STAGE = KEYS * (dev::KeyRow<FMT, D>::BYTES + dev::KeyRow<FMT, D>::SCALES);
  // stages: about 10 KB a warp, two at least (six CTAs of the 4-bit kernel on an SM)
  static constexpr int ST = STAGE >= 8192 ? 2 : (STAGE >= 4096 ? 3 : 4);
};

// grid (partition, KV head, sequence * n_groups + column group)
template <int FMT, int D, int NT>
__global__ void __launch_bounds__(NTHREADS)
    token_scores_kernel(const Weights P) {
  using Row = dev::KeyRow<FMT, D>;
  constexpr int ST = Ring<FMT, D>::ST, STAGE = Ring<FMT, D>::STAGE;
  constexpr int COLS = 8 * NT;
  dev::griddep_enter();  // the sums' blocks wait for all of this kernel
  const int part = blockIdx.x, head = blockIdx.y;
  const int b = blockIdx.z / P.n_groups, grp = blockIdx.z - b * P.n_groups;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int BS = 1 << P.bs_log2, G = 1 << P.g_log2;
  const int tile_bytes = Row::tile(BS);
  const int num_q_heads = P.num_kv_heads << P.g_log2;
  const int tok_i0 = grp * P.q_group;
  const int n_tok = min(P.q_group, P.q_len - tok_i0);
  const int n_cols = n_tok << P.g_log2;
  auto q_row = [&](int n) {
    return (int64_t(b) * P.q_len + tok_i0 + (n >> P.g_log2)) * num_q_heads + head * G +
           (n & (G - 1));
  };
  const int tok0 = part * P.partition_tokens;
  // the partition's table entries, on their way while the length is
  constexpr int ENTRIES = kMaxPartitionTokens / 8 / NTHREADS;
  int32_t entry[ENTRIES];
#pragma unroll
  for (int k = 0; k < ENTRIES; ++k) {
    const int i = tid + k * NTHREADS, j = (tok0 >> P.bs_log2) + i;
    const bool on = i < P.partition_tokens >> P.bs_log2 && j < P.max_blocks_per_seq;
    entry[k] = on ? P.block_tables[int64_t(b) * P.max_blocks_per_seq + j] : 0;
  }
  const int L = checked_len(P, b, tid == 0 && part == 0 && head == 0 && grp == 0);
  if (L == 0) return;
  const int see0 = L - P.q_len + tok_i0 + 1;  // keys of the group's first token
  const int see_last = see0 + n_tok - 1;
  if (tok0 >= see_last) return;
  const int tok1 = min(see_last, tok0 + P.partition_tokens);
  const int nblk = (tok1 - tok0 + BS - 1) >> P.bs_log2;

  extern __shared__ __align__(128) unsigned char smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + NWARPS * ST * STAGE);
  float2* sm_ml = reinterpret_cast<float2*>(bars + NWARPS * ST);  // [NWARPS][COLS]
  int32_t* table = reinterpret_cast<int32_t*>(sm_ml + NWARPS * COLS);
#pragma unroll
  for (int k = 0; k < ENTRIES; ++k) {
    const int i = tid + k * NTHREADS;
    if (i < nblk) {
      const bool bad = entry[k] < 0 || entry[k] >= P.num_blocks;
      if (bad) atomicOr(&g_weights_errors, PA_DEVERR_TABLE_ENTRY);
      table[i] = bad ? 0 : entry[k];
    }
  }
  uint64_t* my_bars = bars + warp * ST;
  unsigned char* ring = smem + warp * ST * STAGE;
  if (lane == 0) {
    for (int s = 0; s < ST; ++s) dev::mbar_init(&my_bars[s], 1);
    dev::fence_barrier_init();
  }
  __syncthreads();

  const int nbk = KEYS >> P.bs_log2;  // blocks of a step
  const int n_steps = (nblk + nbk - 1) / nbk;
  const int n_my = n_steps > warp ? (n_steps - warp + NWARPS - 1) / NWARPS : 0;
  const uint64_t policy = dev::l2_evict_first_policy();
  auto issue = [&](int i) {
    const int blk0 = nbk * (warp + NWARPS * i);
    const int n = min(nbk, nblk - blk0);
    uint64_t* bar = &my_bars[i % ST];
    unsigned char* dst = ring + (i % ST) * STAGE;
    dev::mbar_arrive_expect_tx(bar, n * tile_bytes);
    for (int j = 0; j < n; ++j)
      dev::bulk_load(dst + j * tile_bytes,
                     P.k_cache + (int64_t(table[blk0 + j]) * P.num_kv_heads + head) * tile_bytes,
                     tile_bytes, bar, policy);
  };
  if (lane == 0)
    for (int i = 0; i < ST && i < n_my; ++i) issue(i);

  uint32_t qf[NT][D / 16][2];
  float factor[NT][2];
  int see[NT][2];
  float* out[NT][2];  // score rows of columns 2t and 2t+1
  const float kfac = FMT == PA_KV_BF16 ? P.scale_log2 : P.scale_log2 * P.k_scale[head];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = nt * 8 + g;
    uint4 raw[D / 32];
    dev::query_load<FMT, D>(P.q + q_row(min(n, n_cols - 1)) * D, n < n_cols, t, raw);
    const float f = kfac * dev::query_fragment<FMT, D>(raw, qf[nt]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int m = nt * 8 + 2 * t + c;
      factor[nt][c] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + c));
      see[nt][c] = m < n_cols ? min(tok1, see0 + (m >> P.g_log2)) : 0;
      out[nt][c] = P.scores + q_row(min(m, n_cols - 1)) * P.score_stride;
    }
  }
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      m[nt][c] = -INFINITY;
      l[nt][c] = 0.0f;
    }
  const int row_g = dev::key_row(g);
  const int lane_k = row_g * Row::BYTES + t * Row::RUN;
  const int lane_ks = row_g * Row::SCALES + t * (D / 64);
  int off_k[2][2], off_s[2][2];  // of a step's 8-row quarters: this lane's row and its scales
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = h * 16 + r * 8;  // of a lane with row_g 0 (which is below 8)
      const int tile = (row >> P.bs_log2) * tile_bytes;
      off_k[h][r] = tile + (row & (BS - 1)) * Row::BYTES + lane_k;
      off_s[h][r] = tile + BS * Row::BYTES + (row & (BS - 1)) * Row::SCALES + lane_ks;
    }
  int stalled_at = -1;

  // One step; with EDGE one that holds keys which some column does not see.
  auto step = [&](int i, auto edge_t) {
    constexpr bool EDGE = decltype(edge_t)::value;
    const unsigned char* kt = ring + (i % ST) * STAGE;
    const int key0 = tok0 + KEYS * (warp + NWARPS * i);
    float s[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[h][nt][j] = 0.0f;
      Row rows[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) rows[r].load(kt + off_k[h][r], kt + off_s[h][r]);
      dev::key_product<FMT, D, NT>(s[h], rows[0], rows[1], qf);
    }
    __syncwarp();
    if (lane == 0 && i + ST < n_my) issue(i + ST);

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int key = key0 + h * 16 + r * 8 + row_g;
            float& v = s[h][nt][2 * r + c];
            v *= factor[nt][c];
            if (EDGE && key >= see[nt][c]) {
              v = -INFINITY;
            } else {
              if (EDGE || see[nt][c] > 0) out[nt][c][key] = v;
              top = fmaxf(top, v);
            }
          }
        // each lane keeps the running maximum of its own keys
        const float x = fmaxf(m[nt][c], top);
        const float ref = x == -INFINITY ? 0.0f : x;
        float sum = l[nt][c] * dev::fast_exp2(m[nt][c] - ref);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r) sum += dev::fast_exp2(s[h][nt][2 * r + c] - ref);
        m[nt][c] = x;
        l[nt][c] = sum;
      }
  };
  // steps before the first that is an edge, and this warp's share (columns that no
  // query row has see nothing, and store nothing)
  const int n_full = (min(tok1, see0) - tok0) / KEYS;
  const int n_inner = n_full > warp ? (n_full - warp + NWARPS - 1) / NWARPS : 0;
  // With both forms of the step the one-tile kernel of bf16 rows of 128 spills (72
  // registers; 64 sequences of up to 2 k tokens 31.4 us, against 31.0 with the general
  // form alone); the others gain by them (8 of 8 to 32 k, 4-bit: 40.5 and 38.5).
  constexpr bool APART = FMT != PA_KV_BF16 || D != 128 || NT != 1;
  for (int i = 0; i < n_my; ++i) {
    if (!__all_sync(0xffffffffu, dev::mbar_wait(&my_bars[i % ST], (i / ST) & 1))) {
      stalled_at = i;
      break;
    }
    if (APART && i < n_inner)
      step(i, std::false_type{});
    else
      step(i, std::true_type{});
  }
  if (stalled_at >= 0) {
    if (lane == 0) atomicOr(&g_weights_errors, PA_DEVERR_TIMEOUT);
    for (int j = stalled_at; j < n_my && j < stalled_at + ST; ++j)
      (void)dev::mbar_wait(&my_bars[j % ST], (j / ST) & 1);
  }
  // (max, sum) over the lanes of a column, then over the warps
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, m[nt][c], x);
        const float ol = __shfl_xor_sync(0xffffffffu, l[nt][c], x);
        const float top = fmaxf(m[nt][c], om);
        const float ref = top == -INFINITY ? 0.0f : top;
        l[nt][c] = l[nt][c] * dev::fast_exp2(m[nt][c] - ref) + ol * dev::fast_exp2(om - ref);
        m[nt][c] = top;
      }
      if (g == 0) sm_ml[warp * COLS + nt * 8 + 2 * t + c] = make_float2(m[nt][c], l[nt][c]);
    }
  __syncthreads();
  if (tid < n_cols && tok0 < see0 + (tid >> P.g_log2)) {
    float M = -INFINITY, S = 0.0f;
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) M = fmaxf(M, sm_ml[w * COLS + tid].x);
    const float ref = M == -INFINITY ? 0.0f : M;
#pragma unroll
    for (int w = 0; w < NWARPS; ++w)
      S += sm_ml[w * COLS + tid].y * dev::fast_exp2(sm_ml[w * COLS + tid].x - ref);
    P.part[q_row(tid) * P.num_partitions + part] = make_float2(M, S);
  }
}

constexpr int SUM_THREADS = 256;
constexpr int SUM_GROUPS = 4;   // threads that share a token's rows
constexpr int SUM_TOKENS = SUM_THREADS / SUM_GROUPS * 4;  // of a CTA, four a thread
constexpr int SUM_ROWS = 256;   // rows whose (max, 1/sum) are joined at a time
constexpr int SUM_LANES = 4;    // lanes that join one row's partitions
static_assert(SUM_TOKENS == SUM_THREADS, "the last step takes one token a thread");

// grid (tokens / SUM_TOKENS, sequence). Every block joins the partitions of the
// sequence's rows for itself (8 bytes a row and partition, against 4 a row and
// token that it reads). A thread adds up every fourth row of four tokens, with
// four 16-byte loads in flight; the four sums are added in a fixed order.
__global__ void __launch_bounds__(SUM_THREADS) sum_weights_kernel(const Weights P) {
  const int b = blockIdx.y, tid = threadIdx.x;
  const int L = checked_len(P, b, false);
  dev::griddep_wait();  // the scores (no early dispatch of what follows, which costs it 1 us)
  const int key0 = blockIdx.x * SUM_TOKENS;
  if (key0 >= L) return;
  const int quad = tid % (SUM_THREADS / SUM_GROUPS), group = tid / (SUM_THREADS / SUM_GROUPS);
  const int key = key0 + quad * 4;
  const int num_q_heads = P.num_kv_heads << P.g_log2;
  const int rows = P.q_len * num_q_heads;
  const int64_t row0 = int64_t(b) * rows;
  // keys that the first new token sees: below it nothing is masked
  const int all_see = L - P.q_len + 1;
  __shared__ float2 norm[SUM_ROWS];
  __shared__ float4 part_sum[SUM_GROUPS][SUM_THREADS / SUM_GROUPS];
  float4 w = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int r0 = 0; r0 < rows; r0 += SUM_ROWS) {
    const int n = min(SUM_ROWS, rows - r0);
    __syncthreads();
    const int sub = tid % SUM_LANES;
    for (int r1 = 0; r1 < n; r1 += SUM_THREADS / SUM_LANES) {
      const int r = min(r1 + tid / SUM_LANES, n - 1);
      const int see = all_see + (r0 + r) / num_q_heads;
      const int np = (see + P.partition_tokens - 1) / P.partition_tokens;
      const float2* part = P.part + (row0 + r0 + r) * P.num_partitions;
      float M = -INFINITY, S = 0.0f;
#pragma unroll 4
      for (int p = sub; p < np; p += SUM_LANES) {
        const float2 x = part[p];
        const float top = fmaxf(M, x.x), ref = top == -INFINITY ? 0.0f : top;
        S = S * dev::fast_exp2(M - ref) + x.y * dev::fast_exp2(x.x - ref);
        M = top;
      }
#pragma unroll
      for (int o = 1; o < SUM_LANES; o <<= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, M, o), os = __shfl_xor_sync(0xffffffffu, S, o);
        const float top = fmaxf(M, om), ref = top == -INFINITY ? 0.0f : top;
        S = S * dev::fast_exp2(M - ref) + os * dev::fast_exp2(om - ref);
        M = top;
      }
      if (sub == 0) norm[r] = make_float2(M, 1.0f / S);
    }
    __syncthreads();
    if (key < L) {
      const float* src = P.scores + (row0 + r0) * P.score_stride + key;
      if (key + 3 < all_see) {
#pragma unroll 4
        for (int r = group; r < n; r += SUM_GROUPS) {
          const float4 s = *reinterpret_cast<const float4*>(src + r * P.score_stride);
          const float2 z = norm[r];
          w.x = fmaf(dev::fast_exp2(s.x - z.x), z.y, w.x);
          w.y = fmaf(dev::fast_exp2(s.y - z.x), z.y, w.y);
          w.z = fmaf(dev::fast_exp2(s.z - z.x), z.y, w.z);
          w.w = fmaf(dev::fast_exp2(s.w - z.x), z.y, w.w);
        }
      } else {
        // scores past a row's last key were never written
        for (int r = group; r < n; r += SUM_GROUPS) {
          const int see = all_see + (r0 + r) / num_q_heads;
          const float2 z = norm[r];
          const float* s = src + r * P.score_stride;
          if (key < see) w.x = fmaf(dev::fast_exp2(s[0] - z.x), z.y, w.x);
          if (key + 1 < see) w.y = fmaf(dev::fast_exp2(s[1] - z.x), z.y, w.y);
          if (key + 2 < see) w.z = fmaf(dev::fast_exp2(s[2] - z.x), z.y, w.z);
          if (key + 3 < see) w.w = fmaf(dev::fast_exp2(s[3] - z.x), z.y, w.w);
        }
      }
    }
  }
  part_sum[group][quad] = w;
  __syncthreads();
  // one thread a token now
  const int at = key0 + tid;
  if (at < L) {
    const float* p = reinterpret_cast<const float*>(part_sum) + tid;
    float x = 0.0f;
#pragma unroll
    for (int g = 0; g < SUM_GROUPS; ++g) x += p[g * SUM_TOKENS];
    float* dst = P.token_weights + int64_t(b) * P.weights_stride + at;
    *dst = P.accumulate ? *dst + x : x;
  }
}

template <int FMT, int D, int NT>
int launch_scores(const Weights& P, cudaStream_t stream) {
  auto kernel = token_scores_kernel<FMT, D, NT>;
  constexpr int ST = Ring<FMT, D>::ST;
  const size_t fixed = NWARPS * ST * (Ring<FMT, D>::STAGE + sizeof(uint64_t)) +
                       NWARPS * 8 * NT * sizeof(float2);
  const size_t smem = fixed + size_t((P.partition_tokens >> P.bs_log2) + 1) * sizeof(int32_t);
  static std::atomic<uint64_t> configured{0};  // the opt-in is per device
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return int(e);
  const uint64_t bit = uint64_t(1) << (device & 63);
  if (!(configured.load(std::memory_order_relaxed) & bit)) {
    const size_t most = fixed + size_t(kMaxPartitionTokens / 8 + 1) * sizeof(int32_t);
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(most));
    if (e != cudaSuccess) return int(e);
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  const dim3 grid(unsigned(P.num_partitions), unsigned(P.num_kv_heads),
                  unsigned(P.num_seqs * P.n_groups));
  return launch_ordered(kernel, grid, NTHREADS, smem, stream, 1, P);
}

template <int FMT>
int launch_fmt(const Weights& P, int head_dim, int n_tiles, cudaStream_t s) {
  switch (head_dim * 4 + n_tiles) {
    case 64 * 4 + 1: return launch_scores<FMT, 64, 1>(P, s);
    case 64 * 4 + 2: return launch_scores<FMT, 64, 2>(P, s);
    case 128 * 4 + 1: return launch_scores<FMT, 128, 1>(P, s);
    case 128 * 4 + 2: return launch_scores<FMT, 128, 2>(P, s);
    default: return int(cudaErrorInvalidValue);
  }
}

}  // namespace

int launch_token_weights(const pa_token_weights_params* p, const TokenWeightsSpace& sp,
                         unsigned char* ws, void* stream) {
  const int g = p->num_q_heads / p->num_kv_heads;
  const int q = p->query_len > 1 ? p->query_len : 1;
  const MmaColumns cols = mma_columns(g, q, 2);
  Weights P;
  P.q = static_cast<const __nv_bfloat16*>(p->q);
  P.k_cache = static_cast<const unsigned char*>(p->k_cache);
  P.k_scale = p->k_scale;
  P.block_tables = p->block_tables;
  P.context_lens = p->context_lens;
  P.token_weights = p->token_weights;
  P.part = reinterpret_cast<float2*>(ws + sp.part);
  P.scores = reinterpret_cast<float*>(ws + sp.scores);
  P.score_stride = sp.score_stride;
  P.scale_log2 = p->scale * kLog2e;
  P.weights_stride = p->weights_stride;
  P.max_blocks_per_seq = p->max_blocks_per_seq;
  P.num_seqs = p->num_seqs;
  P.num_kv_heads = p->num_kv_heads;
  P.num_blocks = p->num_blocks;
  P.cap = sp.cap;
  P.bs_log2 = log2_of(p->block_size);
  P.g_log2 = log2_of(g);
  P.q_len = q;
  P.q_group = cols.q_group;
  P.n_groups = cols.n_groups;
  P.partition_tokens = sp.partition_tokens;
  P.num_partitions = sp.num_partitions;
  P.accumulate = p->accumulate != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int e;
  switch (p->kv_dtype) {
    case PA_KV_BF16: e = launch_fmt<PA_KV_BF16>(P, p->head_dim, cols.n_tiles, s); break;
    case PA_KV_FP8_E4M3: e = launch_fmt<PA_KV_FP8_E4M3>(P, p->head_dim, cols.n_tiles, s); break;
    case PA_KV_FP4_E2M1: e = launch_fmt<PA_KV_FP4_E2M1>(P, p->head_dim, cols.n_tiles, s); break;
    default: return int(cudaErrorInvalidValue);
  }
  if (e) return e;
  const dim3 grid(unsigned((sp.cap + SUM_TOKENS - 1) / SUM_TOKENS), unsigned(p->num_seqs));
  return launch_ordered(sum_weights_kernel, grid, SUM_THREADS, 0, s, 1, P);
}

int read_and_clear_weights_errors(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_weights_errors, sizeof(v));
  if (e != cudaSuccess) return int(e);
  e = cudaMemcpyToSymbol(g_weights_errors, &zero, sizeof(zero));
  *flags = v;
  return int(e);
}

}  // namespace pa
