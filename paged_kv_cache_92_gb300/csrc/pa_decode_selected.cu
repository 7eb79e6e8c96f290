// Paged decode attention over selected blocks for sm_103a: for every sequence, new
// token and query head, softmax(scale q.K^T) V over the tokens of the blocks that are
// listed for its (sequence, KV head) alone, with the block table, the running softmax
// and the causal rule of the whole decode ("Paged Attention as a Memory Manager", §How
// the Kernel Executes Paged Attention). Which blocks, pa_blocks.cu says. All three
// caches.
//
// What bounds it: the selected tiles' bytes, once. KV heads have lists of their own, so
// a tile is one (block, KV head), 4 KB of a bf16 cache at block size 16 and head_dim
// 128, anywhere in the pool.
//  * The query rows of a KV head (G heads of up to 8 / G new tokens) are the 8 columns
//    of m16n8k16 products: S^T = K Q^T, O^T += V^T P^T, a warp taking 16 keys a step.
//    Its lanes copy the keys' K and V rows into the warp's own ring with 16-byte
//    asynchronous copies, which may go to any place of a stage, so 16-byte chunks are
//    permuted where the fragments' reads would meet in a bank. No CTA-wide barrier
//    until the end.
//  * bf16: fragments by ldmatrix, V's transposed. P is split into two bf16 terms (2^-17
//    of it is lost); with up to four query rows the second terms are columns 4 to 7 of
//    the same product (their queries are those of columns 0 to 3), so they cost none.
//  * 8-bit and 4-bit codes become f16 pairs in registers (exact), as in the 4-bit
//    decode, with its scaling of queries and its reference for P in f16.
//  * `split` CTAs, a cluster, share the list of one (sequence, column group, KV head)
//    and join their results through distributed shared memory: no workspace, no second
//    launch.
//  * Keys that a column must not see (behind the sequence, or behind one of several new
//    tokens) have weight 0; where V holds no number there, 0 times it would still be
//    none, so such steps zero those rows of V, for every new token by itself.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "pa_blocks.h"
#include "pa_device.cuh"
#include "pa_mma.cuh"
#include "pa_ordered.cuh"

namespace pa {
namespace {

namespace cg = cooperative_groups;

__device__ unsigned int g_selected_errors;

constexpr int NWARPS = 4;
constexpr int NTHREADS = NWARPS * 32;
constexpr int KEYS = 16;  // keys of a warp's step
constexpr int COLS = 8;
constexpr int MAX_SPLIT = 8;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float HEADROOM = 7.0f;  // log2 of the weight that the reference gets
constexpr int NOWHERE = 1 << 30;  // a position that no column sees

struct Sel {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  const unsigned char* k_cache;
  const unsigned char* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_tables;
  const int32_t* context_lens;
  const int32_t* selected;
  float scale_log2;
  int num_selected, max_blocks_per_seq, num_kv_heads, num_blocks, cap;
  int g_log2, q_len, q_group, n_groups;
};

template <int FMT, int D, int BS>
struct Cfg {
  static constexpr int ROWB = FMT == PA_KV_BF16 ? 2 * D : (FMT == PA_KV_FP8_E4M3 ? D : D / 2);
  static constexpr int SCALES = FMT == PA_KV_FP4_E2M1 ? D / 16 : 0;
  static constexpr int TILE = BS * (ROWB + SCALES);         // of one (block, KV head)
  static constexpr int HALF = KEYS * (ROWB + SCALES);       // K (or V) of a step
  static constexpr int STAGE = 2 * HALF;
  static constexpr int ST = FMT == PA_KV_BF16 ? 3 : 4;      // stages of a warp's ring
  static constexpr int NBK = BS < KEYS ? KEYS / BS : 1;     // blocks of a step
  static constexpr int SPB = BS > KEYS ? BS / KEYS : 1;     // steps of a block
  static constexpr int WINDOW = 32 / NBK;                   // steps whose entries a warp holds
  static constexpr int RING = NWARPS * ST * STAGE;
  static constexpr int OROW = D + 4;                        // padded row of the merge
  static constexpr int MERGE = NWARPS * COLS * OROW * 4;    // takes the rings' place at the end
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
  // key row of a step that is row r (0..15) of the products
  __device__ static __forceinline__ int key_of(int r) {
    if constexpr (FMT == PA_KV_FP8_E4M3 && BS >= KEYS)
      // so that a lane's four keys are 4t to 4t + 3: one read of V^T
      return 4 * ((r & 7) >> 1) + (r & 1) + (r >> 3) * 2;
    else if constexpr (FMT == PA_KV_FP4_E2M1)
      return dev::key_row(r & 7) + (r & 8);
    else
      return r;
  }
};

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(dev::smem_addr(p))
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(dev::smem_addr(p))
               : "memory");
}
// a in the low half
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 y = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&y);
}

// DUP (bf16): columns 4 to 7 repeat columns 0 to 3 and take the second terms of P.
template <int FMT, int D, int BS, bool DUP>
__global__ void __launch_bounds__(NTHREADS) decode_selected_kernel(const Sel P) {
  using C = Cfg<FMT, D, BS>;
  constexpr int ST = C::ST;
  dev::griddep_enter();
  cg::cluster_group cluster = cg::this_cluster();
  const int split = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = 1 << P.g_log2;
  const int num_q_heads = P.num_kv_heads << P.g_log2;
  const int unit = blockIdx.x / split;
  const int v = unit / P.num_kv_heads, head = unit - v * P.num_kv_heads;
  const int b = v / P.n_groups, first_tok = (v - b * P.n_groups) * P.q_group;
  const int n_tok = min(P.q_group, P.q_len - first_tok);
  const int n_cols = n_tok << P.g_log2;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sm_m[NWARPS][COLS], sm_l[NWARPS][COLS];
  __shared__ float2 sm_ml[COLS];          // of the CTA, read by the cluster
  __shared__ int sm_pos[NWARPS][ST][2];   // position of the first key of a step's blocks
  unsigned char* ring = smem + warp * ST * C::STAGE;

  int L = P.context_lens[b];
  if (L > P.cap || (L > 0 && L < P.q_len)) {
    if (tid == 0 && rank == 0 && head == 0 && first_tok == 0)
      atomicOr(&g_selected_errors, PA_DEVERR_CONTEXT_LEN);
    L = L < P.q_len ? 0 : P.cap;
  }
  L = max(L, 0);
  const int see0 = L == 0 ? 0 : L - P.q_len + first_tok + 1;  // keys that the first token sees
  const int n_blocks = (L + BS - 1) / BS;
  // this CTA's entries of the list
  const int n_all = min(P.num_selected, n_blocks);
  const int e0 = int(int64_t(n_all) * rank / split), e1 = int(int64_t(n_all) * (rank + 1) / split);
  const int n_steps = C::NBK > 1 ? (e1 - e0 + C::NBK - 1) / C::NBK : (e1 - e0) * C::SPB;
  const int n_my = n_steps > warp ? (n_steps - warp + NWARPS - 1) / NWARPS : 0;
  const int32_t* list = P.selected + (int64_t(b) * P.num_kv_heads + head) * P.num_selected;
  const int32_t* table = P.block_tables + int64_t(b) * P.max_blocks_per_seq;

  // The entries of this warp's steps [w0, w0 + WINDOW), NBK a step, one a lane: the
  // block's first position (NOWHERE: nothing is read) and its place in the pool.
  unsigned errors = 0;
  struct Entry {
    int pos, block;
  };
  auto load_window = [&](int w0) {
    const int step = warp + NWARPS * (w0 + lane / C::NBK);
    const int e = e0 + (C::NBK > 1 ? step * C::NBK + lane % C::NBK : step / C::SPB);
    Entry x{NOWHERE, 0};
    if (e < e1) {
      const int j = list[e];
      if (j >= n_blocks) errors |= PA_DEVERR_KEEP;
      if (j >= 0 && j < n_blocks) {
        const int k = table[j];
        if (k < 0 || k >= P.num_blocks)
          errors |= PA_DEVERR_TABLE_ENTRY;
        else
          x = Entry{j * BS + (C::SPB > 1 ? step % C::SPB * KEYS : 0), k};
      }
    }
    return x;
  };
  Entry window = load_window(0);
  // One copy group: step i of the warp, empty past the last.
  auto issue = [&](int i, int stage) {
    unsigned char* st = ring + stage * C::STAGE;
#pragma unroll
    for (int n = 0; n < C::NBK; ++n) {
      const int src = i % C::WINDOW * C::NBK + n;
      const int pos = __shfl_sync(0xffffffffu, window.pos, src);
      const int block = __shfl_sync(0xffffffffu, window.block, src);
      if (i < n_my) {
        if (lane == 0) sm_pos[warp][stage][n] = pos;
        const int64_t at = (int64_t(block) * P.num_kv_heads + head) * C::TILE;
        const int row0 = C::SPB > 1 ? pos % BS : 0;  // of the step in its block
        const bool on = pos != NOWHERE;
        constexpr int ROWS = BS < KEYS ? BS : KEYS;   // of the block in a step
        // rows (of a code's V in 8 bits: columns) in 16-byte chunks
        constexpr int CHUNKS = ROWS * C::ROWB / 16;
#pragma unroll
        for (int c = 0; c < CHUNKS; c += 32) {
          const int x = c + lane;
          const bool in = on && (c + 32 <= CHUNKS || x < CHUNKS);
          constexpr int CPR = C::ROWB / 16;  // chunks of a row
          const int r = n * ROWS + x / CPR, k = x % CPR;
          int kd = r * C::ROWB, vd = n * ROWS * C::ROWB + x * 16;
          if constexpr (FMT == PA_KV_BF16) {
            kd += (k ^ (r & 7)) * 16;
            vd = kd;
          } else if constexpr (FMT == PA_KV_FP8_E4M3 && D == 128) {
            kd += (k ^ ((r & 1) << 2)) * 16;
          } else {
            kd += k * 16;
          }
          dev::cp_async16(st + kd, P.k_cache + at + row0 * C::ROWB + x * 16, in);
          dev::cp_async16(st + C::HALF + vd, P.v_cache + at + row0 * C::ROWB + x * 16, in);
        }
        if constexpr (C::SCALES > 0) {
          constexpr int N = ROWS * C::SCALES / 16;  // chunks of scales, of K then of V
          const bool of_v = lane >= N;
          const int x = of_v ? lane - N : lane;
          const unsigned char* from = (of_v ? P.v_cache : P.k_cache) + at + BS * C::ROWB +
                                      row0 * C::SCALES + x * 16;
          dev::cp_async16(st + (of_v ? C::HALF : 0) + KEYS * C::ROWB + n * ROWS * C::SCALES + x * 16,
                          from, on && lane < 2 * N);
        }
      }
    }
    dev::cp_async_commit();
  };

  // row of q / out of column n: new token n / G of the group, query head head * G + n % G
  auto q_row = [&](int n) {
    return (int64_t(b) * P.q_len + first_tok + (n >> P.g_log2)) * num_q_heads + head * G +
           (n & (G - 1));
  };
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) issue(i, i);

  uint32_t qf[D / 16][2];  // the queries as the B operand (column g)
  float inv_scaling = 1.0f, k_scale = 1.0f;
  {
    const int col = DUP ? g & 3 : g;
    const __nv_bfloat16* row = P.q + q_row(min(col, n_cols - 1)) * D;
    if constexpr (FMT == PA_KV_BF16) {
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t x = *reinterpret_cast<const uint32_t*>(row + s * 16 + i * 8 + t * 2);
          qf[s][i] = col < n_cols ? x : 0u;
        }
    } else {
      uint4 raw[D / 32];
      dev::query_load<FMT, D>(row, col < n_cols, t, raw);
      inv_scaling = dev::query_fragment<FMT, D>(raw, qf);
      k_scale = P.k_scale[head];
      // a negative scale turns the queries, so that a larger product stays a larger score
      const uint32_t sign = k_scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        qf[s][0] ^= sign;
        qf[s][1] ^= sign;
      }
      k_scale = fabsf(k_scale);
    }
  }
  float factor[2];  // of columns 2t and 2t+1: softmax scale * K scale / the row's scaling
  int see[2];       // keys that they see
  int tok[2];       // their new token, in the group
  const float row_factor = P.scale_log2 * k_scale * inv_scaling;
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    factor[c] = __shfl_sync(0xffffffffu, row_factor, 4 * (2 * t + c));
    // A scale of zero makes all scores equal, but 0 * -inf is NaN: below 2^-100 the
    // products (under 2^35) count as zero either way. The comparison keeps a NaN scale.
    if (FMT != PA_KV_BF16) factor[c] = factor[c] < 0x1p-100f ? 0x1p-100f : factor[c];
    const int col = DUP ? (2 * t + c) & 3 : 2 * t + c;
    tok[c] = min(col >> P.g_log2, n_tok - 1);
    see[c] = see0 + tok[c];
  }

  // Softmax state of columns 2t and 2t+1: a key's weight is exp2((s - ref) * factor +
  // HEADROOM), s the raw product and ref the one that the reference was taken from (0
  // before the first key that the column sees): the difference comes first, as the last
  // place of a large score is many units. limit: the raw product beyond which ref moves,
  // 8 above it, so that no weight passes 2^15.
  float o[D / 16][4];  // O^T: D / 16 tiles of 16 rows
  float ref[2] = {0.0f, 0.0f}, limit[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;

  // A fragments of V^T: rows d (16 i .. 16 i + 15 in some order), keys of the products' rows.
  auto v_fragment = [&](const unsigned char* vt, int i, uint32_t (&a)[4]) {
    if constexpr (FMT == PA_KV_BF16) {
      // lanes 8 m .. 8 m + 7 name the rows of matrix m: keys (m / 2) * 8 .., chunk 2 i + m % 2
      const int m = lane >> 3, r = (m >> 1) * 8 + (lane & 7);
      ldmatrix_x4_trans(a, vt + r * C::ROWB + (((2 * i + (m & 1)) ^ (r & 7)) * 16));
    } else if constexpr (FMT == PA_KV_FP8_E4M3) {
      if constexpr (BS >= KEYS) {
        const uint32_t x = *reinterpret_cast<const uint32_t*>(vt + (16 * i + g) * 16 + 4 * t);
        const uint32_t y = *reinterpret_cast<const uint32_t*>(vt + (16 * i + g + 8) * 16 + 4 * t);
        a[0] = dev::e4m3x2_to_f16(x & 0xffffu);
        a[1] = dev::e4m3x2_to_f16(y & 0xffffu);
        a[2] = dev::e4m3x2_to_f16(x >> 16);
        a[3] = dev::e4m3x2_to_f16(y >> 16);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)  // block k / 2, row g or g + 8
          a[k] = dev::e4m3x2_to_f16(*reinterpret_cast<const uint16_t*>(
              vt + (k >> 1) * BS * D + (16 * i + g + (k & 1) * 8) * BS + 2 * t));
      }
    }
  };

  // One step; with EDGE one that holds keys which some column does not see.
  auto step = [&](int stage, int pos0, int pos1, auto edge_t) {
    constexpr bool EDGE = decltype(edge_t)::value;
    const unsigned char* kt = ring + stage * C::STAGE;
    const unsigned char* vt = kt + C::HALF;
    auto position = [&](int r) {  // of row r of the products
      const int k = C::key_of(r);
      return C::NBK > 1 ? (k < BS ? pos0 + k : pos1 + k - BS) : pos0 + k;
    };
    float s[4];
    if constexpr (FMT == PA_KV_BF16) {
      float s2[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[h][j] = 0.0f;
      // matrix m: keys (m % 2) * 8 .., chunk 2 i + m / 2
      const int m = lane >> 3, r = (m & 1) * 8 + (lane & 7);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t a[4];
        ldmatrix_x4(a, kt + r * C::ROWB + (((2 * i + (m >> 1)) ^ (r & 7)) * 16));
        dev::mma_bf16_regs(s2[i & 1], a[0], a[1], a[2], a[3], qf[i][0], qf[i][1]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = s2[0][j] + s2[1][j];
    } else {
      using Row = dev::KeyRow<FMT, D>;
      Row rows[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = C::key_of(g + 8 * h);
        if constexpr (FMT == PA_KV_FP8_E4M3 && D == 128) {
          // (runs t and t + 4 of the row, permuted as they were copied)
          const uint4 x = *reinterpret_cast<const uint4*>(kt + r * D + ((t ^ ((r & 1) << 2)) * 16));
          const uint4 y =
              *reinterpret_cast<const uint4*>(kt + r * D + (((t + 4) ^ ((r & 1) << 2)) * 16));
          rows[h].w[0] = x.x; rows[h].w[1] = x.y; rows[h].w[2] = x.z; rows[h].w[3] = x.w;
          rows[h].w[4] = y.x; rows[h].w[5] = y.y; rows[h].w[6] = y.z; rows[h].w[7] = y.w;
        } else {
          rows[h].load(kt + r * C::ROWB + t * Row::RUN,
                       kt + KEYS * C::ROWB + r * C::SCALES + t * (D / 64));
        }
      }
      float s1[1][4] = {{0.0f, 0.0f, 0.0f, 0.0f}};
      uint32_t q1[1][D / 16][2];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        q1[0][i][0] = qf[i][0];
        q1[0][i][1] = qf[i][1];
      }
      dev::key_product<FMT, D, 1>(s1, rows[0], rows[1], q1);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] = s1[0][j];
    }
    // ---- softmax; keys that a column does not see are -inf
    bool over = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (EDGE && position(g + (j >> 1) * 8) >= see[j & 1]) s[j] = -INFINITY;
      over |= s[j] > limit[j & 1];
    }
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = fmaxf(s[c], s[c + 2]);
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        // no branch: the lanes of a warp stay together
        const bool first = limit[c] == -INFINITY;
        const bool take = x != -INFINITY && (first || x > ref[c]);
        const float y = take ? x : ref[c];
        const float old = dev::fast_exp2((ref[c] - y) * factor[c]);
        const float a = take && first ? 0.0f : old;
        ref[c] = y;
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
    uint32_t pf[2];                   // P^T as the second product's B operand
    [[maybe_unused]] uint32_t pl[2];  // its second terms
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 e = dev::fma_pair(dev::sub_pair(make_float2(s[2 * h], s[2 * h + 1]), ref),
                                     factor, HEADROOM);
      const float p0 = dev::fast_exp2(e.x), p1 = dev::fast_exp2(e.y);
      l[0] += p0;
      l[1] += p1;
      if constexpr (FMT == PA_KV_BF16) {
        const uint32_t hi = pack_bf16(p0, p1);
        const uint32_t lo = pack_bf16(p0 - dev::bf16_lo(hi), p1 - dev::bf16_hi(hi));
        pf[h] = dev::transpose_8x8(DUP && t >= 2 ? lo : hi);
        if (!DUP) pl[h] = dev::transpose_8x8(lo);
      } else {
        pf[h] = dev::transpose_8x8(dev::pack_f16(p0, p1));
      }
    }
    // ---- O^T += V^T P^T
    auto product = [&](float (&acc)[4], const uint32_t (&a)[4], uint32_t m0, uint32_t m1) {
      if constexpr (FMT == PA_KV_BF16) {
        dev::mma_bf16_regs(acc, a[0] & m0, a[1] & m0, a[2] & m1, a[3] & m1, pf[0], pf[1]);
        if constexpr (!DUP)
          dev::mma_bf16_regs(acc, a[0] & m0, a[1] & m0, a[2] & m1, a[3] & m1, pl[0], pl[1]);
      } else {
        dev::mma_f16(acc, a[0] & m0, a[1] & m0, a[2] & m1, a[3] & m1, pf[0], pf[1]);
      }
    };
    auto tile_product = [&](int i, const uint32_t (&a)[4]) {
      if constexpr (!EDGE) {
        product(o[i], a, 0xffffffffu, 0xffffffffu);
      } else {
        for (int n = 0; n < n_tok; ++n) {  // for the columns of token n, rows that it sees
          const int sees = see0 + n;
          auto mask = [&](int r) {
            return (position(r) < sees ? 0xffffu : 0u) | (position(r + 1) < sees ? 0xffff0000u : 0u);
          };
          float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          product(acc, a, mask(2 * t), mask(2 * t + 8));
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][j] += tok[j & 1] == n ? acc[j] : 0.0f;
        }
      }
    };
    if constexpr (FMT != PA_KV_FP4_E2M1) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t a[4];
        v_fragment(vt, i, a);
        tile_product(i, a);
      }
    } else {
      constexpr int VW = D / 64;  // code words of a lane's share of a V row (D / 8 elements)
      uint32_t w[4][VW], sb[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {  // keys of rows 2t, 2t + 1, 2t + 8, 2t + 9
        const int k = C::key_of(2 * t + (r & 1) + (r >> 1) * 8);
        const unsigned char* codes = vt + k * C::ROWB + g * (D / 16);
        if constexpr (D == 128) {
          const uint2 x = *reinterpret_cast<const uint2*>(codes);
          w[r][0] = x.x;
          w[r][1] = x.y;
        } else {
          w[r][0] = *reinterpret_cast<const uint32_t*>(codes);
        }
        sb[r] = vt[KEYS * C::ROWB + k * C::SCALES + (g * VW) / 2];
      }
      const uint32_t s01 = dev::e4m3x2_to_f16(sb[0] | sb[1] << 8);
      const uint32_t s23 = dev::e4m3x2_to_f16(sb[2] | sb[3] << 8);
#pragma unroll
      for (int c = 0; c < VW; ++c) {
        // the nibbles of two keys in one word, so that a conversion yields one element of both
        uint32_t x0[4], y0[4], x1[4], y1[4];
        dev::e2m1x8_to_f16((w[0][c] & 0x0F0F0F0Fu) | ((w[1][c] << 4) & 0xF0F0F0F0u), x0);
        dev::e2m1x8_to_f16(((w[0][c] >> 4) & 0x0F0F0F0Fu) | (w[1][c] & 0xF0F0F0F0u), y0);
        dev::e2m1x8_to_f16((w[2][c] & 0x0F0F0F0Fu) | ((w[3][c] << 4) & 0xF0F0F0F0u), x1);
        dev::e2m1x8_to_f16(((w[2][c] >> 4) & 0x0F0F0F0Fu) | (w[3][c] & 0xF0F0F0F0u), y1);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a[4] = {dev::mul_f16x2(x0[j], s01), dev::mul_f16x2(y0[j], s01),
                                 dev::mul_f16x2(x1[j], s23), dev::mul_f16x2(y1[j], s23)};
          tile_product(c * 4 + j, a);
        }
      }
    }
  };

  for (int i = 0, stage = 0; i < n_my; ++i) {
    dev::cp_async_wait<ST - 2>();
    __syncwarp();  // the step's copies by all lanes, and its positions
    const int ahead = i + ST - 1;
    if (ahead % C::WINDOW == 0) window = load_window(ahead);
    issue(ahead, stage == 0 ? ST - 1 : stage - 1);
    const int pos0 = sm_pos[warp][stage][0], pos1 = C::NBK > 1 ? sm_pos[warp][stage][1] : 0;
    const bool inner = pos0 + (C::NBK > 1 ? BS : KEYS) <= see0 && (C::NBK == 1 || pos1 + BS <= see0);
    if (inner)
      step(stage, pos0, pos1, std::false_type{});
    else
      step(stage, pos0, pos1, std::true_type{});
    __syncwarp();  // the stage has been read
    stage = stage + 1 == ST ? 0 : stage + 1;
  }
  dev::cp_async_wait<0>();
  if (errors) atomicOr(&g_selected_errors, errors);
  __syncthreads();  // the rings give way to the merge

  // ---- the warps' results, then the CTA's, then the cluster's
  float* rows = reinterpret_cast<float*>(smem);  // [NWARPS][COLS][OROW]
#pragma unroll
  for (int c = 0; c < 2; ++c) {
#pragma unroll
    for (int x = 4; x < 32; x <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], x);
    if (g == 0) {
      // (a sum of NaN without a maximum has to reach the result: +inf carries it)
      sm_m[warp][2 * t + c] = l[c] != l[c] ? INFINITY
                              : (limit[c] == -INFINITY ? -INFINITY
                                                       : fmaf(ref[c], factor[c], -HEADROOM));
      sm_l[warp][2 * t + c] = l[c];
    }
  }
#pragma unroll
  for (int k = 0; k < D / 16; ++k) {
    if constexpr (DUP) {  // first and second terms
#pragma unroll
      for (int j = 0; j < 4; ++j) o[k][j] += __shfl_xor_sync(0xffffffffu, o[k][j], 2);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // rows g and g + 8 of tile k; of a 4-bit V elements g D/8 + 2k, + 1
      const int d = FMT == PA_KV_FP4_E2M1 ? g * (D / 8) + 2 * k + (j >> 1) : 16 * k + g + (j >> 1) * 8;
      rows[(warp * COLS + 2 * t + (j & 1)) * C::OROW + d] = o[k][j];
    }
  }
  __syncthreads();
  constexpr int TPC = NTHREADS / COLS, E = D / TPC;  // threads of a column, their elements
  {
    const int n = tid / TPC, d = tid % TPC * E;
    float M = -INFINITY, den = 0.0f, wt[NWARPS];
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) M = fmaxf(M, sm_m[w][n]);
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) {
      wt[w] = sm_m[w][n] == -INFINITY ? 0.0f : dev::fast_exp2(sm_m[w][n] - M);
      den = fmaf(wt[w], sm_l[w][n], den);
    }
    float sum[E];
#pragma unroll
    for (int x = 0; x < E; ++x) sum[x] = 0.0f;
#pragma unroll
    for (int w = 0; w < NWARPS; ++w)
#pragma unroll
      for (int x = 0; x < E; ++x)
        sum[x] = fmaf(wt[w], rows[(w * COLS + n) * C::OROW + d + x], sum[x]);
    __syncthreads();
#pragma unroll
    for (int x = 0; x < E; ++x) rows[n * C::OROW + d + x] = sum[x];
    if (d == 0) sm_ml[n] = make_float2(M, den);
  }
  cluster.sync();
  {
    // a CTA writes every split-th element pair of the rows
    const float scale_v = FMT == PA_KV_BF16 ? 1.0f : P.v_scale[head];
    for (int i = rank * NTHREADS + tid; i < n_cols * (D / 2); i += split * NTHREADS) {
      const int n = i / (D / 2), d = i % (D / 2) * 2;
      float2 ml[MAX_SPLIT], x[MAX_SPLIT];
      float M = -INFINITY;
#pragma unroll
      for (int k = 0; k < MAX_SPLIT; ++k)
        if (k < split) {
          ml[k] = *cluster.map_shared_rank(&sm_ml[n], unsigned(k));
          x[k] = *reinterpret_cast<const float2*>(
              cluster.map_shared_rank(rows + n * C::OROW + d, unsigned(k)));
          M = fmaxf(M, ml[k].x);
        }
      float den = 0.0f;
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < MAX_SPLIT; ++k)
        if (k < split && ml[k].x != -INFINITY) {
          const float w = dev::fast_exp2(ml[k].x - M);
          den = fmaf(w, ml[k].y, den);
          sum.x = fmaf(w, x[k].x, sum.x);
          sum.y = fmaf(w, x[k].y, sum.y);
        }
      const float norm = den == 0.0f ? 0.0f : scale_v / den;  // no key: a row of zeros
      *reinterpret_cast<__nv_bfloat162*>(P.out + q_row(n) * D + d) =
          __floats2bfloat162_rn(sum.x * norm, sum.y * norm);
    }
  }
  if (split > 1) cluster.sync();  // no CTA leaves while another reads its rows
}

template <int FMT, int D, int BS, bool DUP>
int launch_t(const Sel& P, int split, int64_t units, cudaStream_t stream) {
  using C = Cfg<FMT, D, BS>;
  // the opt-in to large shared memory is per device
  static std::atomic<uint64_t> configured{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return int(e);
  const uint64_t bit = uint64_t(1) << (device & 63);
  if (!(configured.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(decode_selected_kernel<FMT, D, BS, DUP>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (e != cudaSuccess) return int(e);
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  return launch_ordered(decode_selected_kernel<FMT, D, BS, DUP>, dim3(unsigned(units * split)),
                        NTHREADS, C::SMEM, stream, unsigned(split), P);
}

template <int FMT, int D, int BS>
int launch_dup(const Sel& P, int split, int64_t units, cudaStream_t s) {
  if constexpr (FMT == PA_KV_BF16)
    if ((P.q_group << P.g_log2) <= 4) return launch_t<FMT, D, BS, true>(P, split, units, s);
  return launch_t<FMT, D, BS, false>(P, split, units, s);
}
template <int FMT, int D>
int launch_bs(const Sel& P, int block_size, int split, int64_t units, cudaStream_t s) {
  switch (block_size) {
    case 8: return launch_dup<FMT, D, 8>(P, split, units, s);
    case 16: return launch_dup<FMT, D, 16>(P, split, units, s);
    case 32: return launch_dup<FMT, D, 32>(P, split, units, s);
    default: return int(cudaErrorInvalidValue);
  }
}
template <int FMT>
int launch_d(const Sel& P, int head_dim, int block_size, int split, int64_t units, cudaStream_t s) {
  return head_dim == 64 ? launch_bs<FMT, 64>(P, block_size, split, units, s)
                        : launch_bs<FMT, 128>(P, block_size, split, units, s);
}

}  // namespace

SelectedPlan selected_plan(const pa_decode_params* p, int num_selected, int num_sms) {
  SelectedPlan r{};
  r.cols = fp4_columns(p);
  const int64_t table = int64_t(p->max_blocks_per_seq) * p->block_size;
  r.cap = int(p->max_context_len < table ? p->max_context_len : table);
  // CTAs for two an SM several times over, each with two steps a warp at least
  const int64_t units = int64_t(p->num_seqs) * r.cols.n_groups * p->num_kv_heads;
  const int64_t blocks = (int64_t(r.cap) + p->block_size - 1) / p->block_size;
  const int64_t keys = (blocks < num_selected ? blocks : num_selected) * p->block_size;
  r.split = 1;
  while (r.split < MAX_SPLIT && units * r.split < int64_t(num_sms) * 8 &&
         keys / (2 * r.split) >= 2 * NWARPS * KEYS)
    r.split *= 2;
  return r;
}

int launch_decode_selected(const pa_decode_params* p, const int32_t* selected, int num_selected,
                           const SelectedPlan& plan, void* stream) {
  Sel P;
  P.q = static_cast<const __nv_bfloat16*>(p->q);
  P.out = static_cast<__nv_bfloat16*>(p->out);
  P.k_cache = static_cast<const unsigned char*>(p->k_cache);
  P.v_cache = static_cast<const unsigned char*>(p->v_cache);
  P.k_scale = p->k_scale;
  P.v_scale = p->v_scale;
  P.block_tables = p->block_tables;
  P.context_lens = p->context_lens;
  P.selected = selected;
  P.scale_log2 = p->scale * kLog2e;
  P.num_selected = num_selected;
  P.max_blocks_per_seq = p->max_blocks_per_seq;
  P.num_kv_heads = p->num_kv_heads;
  P.num_blocks = p->num_blocks;
  P.cap = plan.cap;
  P.g_log2 = log2_of(p->num_q_heads / p->num_kv_heads);
  P.q_len = query_len_of(p);
  P.q_group = plan.cols.q_group;
  P.n_groups = plan.cols.n_groups;
  const int64_t units = int64_t(p->num_seqs) * plan.cols.n_groups * p->num_kv_heads;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (p->kv_dtype) {
    case PA_KV_BF16:
      return launch_d<PA_KV_BF16>(P, p->head_dim, p->block_size, plan.split, units, s);
    case PA_KV_FP8_E4M3:
      return launch_d<PA_KV_FP8_E4M3>(P, p->head_dim, p->block_size, plan.split, units, s);
    default:
      return launch_d<PA_KV_FP4_E2M1>(P, p->head_dim, p->block_size, plan.split, units, s);
  }
}

int read_and_clear_selected_errors(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_selected_errors, sizeof(v));
  if (e != cudaSuccess) return int(e);
  e = cudaMemcpyToSymbol(g_selected_errors, &zero, sizeof(zero));
  *flags = v;
  return int(e);
}

}  // namespace pa
