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
//    heads of up to 8 NT / G new tokens, are the 8 NT columns.
//  * The order of elements inside a product is free as long as both operands
//    share it, so a lane reads its K elements as one run of head_dim / 4 codes.
//    For V the contraction runs over keys: the nibbles of two keys are merged
//    into one word (two logic operations for eight pairs) before conversion,
//    so each conversion yields one element of both keys, as the product needs.
//  * P^T comes out of the first product transposed to what the second one
//    wants; an 8x8 register transpose turns it.
//  * Queries are scaled by a power of two per row into f16's range (exact for
//    every element within 2^-30 of the row's largest) and the factor goes to
//    the softmax scale. P is rounded to f16 (2^-12 of its value, eight times
//    finer than bf16, and no cheaper form exists); the running maximum, the
//    sums and the output stay in fp32.
//  * The reference maximum moves only when a score exceeds it by 2^8, so O is
//    rescaled rarely; f16 holds the weights up to 2^8 that this allows.
// A sequence longer than a partition is split over CTAs; the partials are
// merged by log-sum-exp.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "pa_device.cuh"
#include "pa_internal.h"
#include "pa_mma.cuh"

namespace pa {
namespace {

__device__ unsigned int g_decode_fp4_errors;

constexpr int NWARPS = 4;
constexpr int NTHREADS = NWARPS * 32;
constexpr int KEYS = 32;  // keys of a warp's step
constexpr float kLog2e = 1.4426950408889634f;

template <int D, int NT, int BS>
struct Cfg {
  static constexpr int NBK = KEYS / BS;              // blocks of a step
  static constexpr int TILE = BS * D * 9 / 16;       // bytes of one (block, KV head) tile
  static constexpr int STAGE = 2 * NBK * TILE;       // K tiles, then V tiles
  static constexpr int ST = D == 128 ? 3 : 4;        // ring stages per warp
  static constexpr int COLS = 8 * NT;
  static constexpr int OROW = D + 4;                 // padded row of the warps' merge
  static constexpr int MERGE = NWARPS * COLS * (OROW + 2) * 4;
  static constexpr int RING = NWARPS * ST * STAGE;
  static constexpr int TILES = RING > MERGE ? RING : MERGE;
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
  float* part_m;
  float* part_l;
  float* part_acc;
  float scale_log2;
  int max_blocks_per_seq, num_kv_heads, num_blocks, max_context_len;
  int g_log2;  // log2 of the query heads per KV head
  int q_len, q_group, n_groups;  // new tokens; of a column group; column groups
  int partition_tokens, num_partitions;
};

// grid (partition, KV head, sequence * n_groups + column group)
template <int D, int NT, int BS>
__global__ void __launch_bounds__(NTHREADS, NT == 1 ? 4 : 3)
    paged_decode_fp4_kernel(const Fp4Decode P) {
  using C = Cfg<D, NT, BS>;
  constexpr int ST = C::ST, NBK = C::NBK, TILE = C::TILE;
  constexpr int VW = D / 64;  // code words of a lane's share of a V row (D / 8 elements)
  const int part = blockIdx.x, head = blockIdx.y;
  const int b = blockIdx.z / P.n_groups, grp = blockIdx.z - b * P.n_groups;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int G = 1 << P.g_log2;
  const int num_q_heads = P.num_kv_heads << P.g_log2;
  const int tok_i0 = grp * P.q_group;                       // first new token of the group
  const int n_tok = min(P.q_group, P.q_len - tok_i0);       // its tokens
  const int n_cols = n_tok << P.g_log2;                     // its columns
  // row of q / out of column n: token tok_i0 + n / G, query head head * G + n % G
  auto q_row = [&](int n) {
    return (int64_t(b) * P.q_len + tok_i0 + (n >> P.g_log2)) * num_q_heads + head * G +
           (n & (G - 1));
  };

  int L = P.context_lens[b];
  const int cap = min(P.max_blocks_per_seq * BS, P.max_context_len);
  const bool report = tid == 0 && part == 0 && head == 0 && grp == 0;
  if (L > cap) {
    if (report) atomicOr(&g_decode_fp4_errors, PA_DEVERR_CONTEXT_LEN);
    L = cap;
  }
  if (L > 0 && L < P.q_len) {  // no room for the new tokens: an empty sequence
    if (report) atomicOr(&g_decode_fp4_errors, PA_DEVERR_CONTEXT_LEN);
    L = 0;
  }
  if (L <= 0) {
    if (part == 0)
      for (int i = tid; i < n_cols * D; i += NTHREADS)
        P.out[q_row(i / D) * D + i % D] = __float2bfloat16_rn(0.0f);
    return;
  }
  // token i of the sequence's new ones sees L - q_len + i + 1 keys
  const int see0 = L - P.q_len + tok_i0 + 1;
  const int see_last = see0 + n_tok - 1;
  const int tok0 = part * P.partition_tokens;
  if (tok0 >= see_last) return;
  const int tok1 = min(see_last, tok0 + P.partition_tokens);
  const int nblk = (tok1 - tok0 + BS - 1) / BS;

  extern __shared__ __align__(128) unsigned char smem[];
  int32_t* table = reinterpret_cast<int32_t*>(smem + C::TILES);
  const int32_t* trow = P.block_tables + int64_t(b) * P.max_blocks_per_seq + tok0 / BS;
  for (int i = tid; i < nblk; i += NTHREADS) {
    int32_t e = trow[i];
    if (e < 0 || e >= P.num_blocks) {
      atomicOr(&g_decode_fp4_errors, PA_DEVERR_TABLE_ENTRY);
      e = 0;
    }
    table[i] = e;
  }
  __syncthreads();

  // step i of this warp: the partition's blocks [NBK * (warp + NWARPS * i), + NBK)
  const int n_steps = (nblk + NBK - 1) / NBK;
  const int n_my = n_steps > warp ? (n_steps - warp + NWARPS - 1) / NWARPS : 0;
  unsigned char* ring = smem + warp * ST * C::STAGE;
  const uint64_t policy = dev::l2_evict_first_policy();
  const unsigned char* k_head = P.k_cache + int64_t(head) * TILE + lane * 16;
  const unsigned char* v_head = P.v_cache + int64_t(head) * TILE + lane * 16;
  const int64_t block_bytes = int64_t(P.num_kv_heads) * TILE;
  auto issue = [&](int i, int stage) {  // one group, empty past the last step
    unsigned char* dst = ring + stage * C::STAGE + lane * 16;
    const int blk0 = NBK * (warp + NWARPS * i);
#pragma unroll
    for (int j = 0; j < NBK; ++j)
      if (blk0 + j < nblk) {
        const int64_t off = table[blk0 + j] * block_bytes;
#pragma unroll
        for (int c = 0; c < TILE; c += 512)
          if (c + 512 <= TILE || lane * 16 < TILE - c) {
            dev::cp_async16(dst + j * TILE + c, k_head + off + c, policy);
            dev::cp_async16(dst + (NBK + j) * TILE + c, v_head + off + c, policy);
          }
      }
    dev::cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < ST; ++i) issue(i, i);

  // Queries as the B operand (columns nt * 8 + g), scaled into f16's range.
  uint32_t qf[NT][D / 16][2];
  float factor[NT][2];  // of columns 2t and 2t+1: softmax scale * K scale / the row's scaling
  int see[NT][2];       // keys that columns 2t and 2t+1 see
  const float kfac = P.scale_log2 * P.k_scale[head];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int n = nt * 8 + g;
    const float f = kfac * dev::query_fragment<PA_KV_FP4_E2M1, D>(
                               n < n_cols ? P.q + q_row(n) * D : nullptr, t, qf[nt]);
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      factor[nt][c] = __shfl_sync(0xffffffffu, f, 4 * (2 * t + c));
      see[nt][c] = min(tok1, see0 + ((nt * 8 + 2 * t + c) >> P.g_log2));
    }
  }
  const int see_first = min(tok1, see0);  // no column sees fewer keys

  float o[D / 16][NT][4];  // O^T: D / 16 tiles of 16 rows
  // Softmax state of columns 2t and 2t+1, in the log2 domain: a score is
  // s * factor (s the raw product), ref the reference maximum (0 before the
  // first key that the column sees), limit the raw product beyond which ref moves.
  float ref[NT][2], limit[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      ref[nt][c] = l[nt][c] = 0.0f;
      limit[nt][c] = -INFINITY;
    }
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][nt][j] = 0.0f;

  using KRow = dev::KeyRow<PA_KV_FP4_E2M1, D>;
  const int row_g = dev::key_row(g);                            // this lane's K rows
  const int row_a = dev::key_row(2 * t), row_b = dev::key_row(2 * t + 1);  // its V rows
  // where they lie in a tile, apart from what is the same for every lane
  const int lane_k = row_g * (D / 2) + t * KRow::RUN;
  const int lane_ks = BS * (D / 2) + row_g * (D / 16) + t * (D / 64);
  const int lane_va = row_a * (D / 2) + g * (D / 16), lane_vb = row_b * (D / 2) + g * (D / 16);
  const int lane_vsa = BS * (D / 2) + row_a * (D / 16) + (g * VW) / 2;
  const int lane_vsb = BS * (D / 2) + row_b * (D / 16) + (g * VW) / 2;

  // One step; with EDGE the one that holds keys which some column does not see.
  auto step = [&](int i, int stage, auto edge_t) {
    constexpr bool EDGE = decltype(edge_t)::value;
    const unsigned char* kt = ring + stage * C::STAGE;
    const unsigned char* vt = kt + NBK * TILE;
    const int key0 = tok0 + KEYS * (warp + NWARPS * i);

    // ---- raw scores: two tiles of 16 keys
    float s[2][NT][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[h][nt][j] = 0.0f;
      KRow rows[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = h * 16 + r * 8;  // of a lane with row_g 0 (which is below 8)
        const unsigned char* tile = kt + (row / BS) * TILE;
        rows[r].load(tile + (row % BS) * (D / 2) + lane_k, tile + (row % BS) * (D / 16) + lane_ks);
      }
      dev::key_product<PA_KV_FP4_E2M1, D, NT>(s[h], rows[0], rows[1], qf);
    }
    // ---- softmax; keys past a column's last are -inf
    if constexpr (EDGE) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (key0 + h * 16 + (j >> 1) * 8 + row_g >= see[nt][j & 1]) s[h][nt][j] = -INFINITY;
    }
    bool over = false;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) over |= s[h][nt][j] > limit[nt][j & 1];
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float x = fmaxf(fmaxf(s[0][nt][c], s[0][nt][c + 2]), fmaxf(s[1][nt][c], s[1][nt][c + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16)) * factor[nt][c];
          const bool first = limit[nt][c] == -INFINITY;
          if (x != -INFINITY && (first || x > ref[nt][c])) {
            const float a = first ? 0.0f : dev::fast_exp2(ref[nt][c] - x);
            ref[nt][c] = x;
            limit[nt][c] = (x + 8.0f) / factor[nt][c];
            l[nt][c] *= a;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              o[k][nt][c] *= a;
              o[k][nt][c + 2] *= a;
            }
          }
        }
    }
    uint32_t pf[2][NT][2];  // P^T as the second product's B operand
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float p[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p[j] = dev::fast_exp2(fmaf(s[h][nt][j], factor[nt][j & 1], -ref[nt][j & 1]));
          l[nt][j & 1] += p[j];
        }
        pf[h][nt][0] = dev::transpose_8x8(dev::pack_f16(p[0], p[1]));
        pf[h][nt][1] = dev::transpose_8x8(dev::pack_f16(p[2], p[3]));
      }

    // ---- O^T += V^T P^T over the keys [.., end) of the step; with `only` >= 0
    // for the columns of that token alone
    auto value_product = [&](int h, int end, int only, auto single) {
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
        // a key that is not there: finite codes times zero
        if (EDGE && key0 + row + ((r & 1) ? row_b : row_a) >= end) sb[r] = 0;
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
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = dev::mul_f16x2(e0[j], s01), a1 = dev::mul_f16x2(o0[j], s01);
          const uint32_t a2 = dev::mul_f16x2(e1[j], s23), a3 = dev::mul_f16x2(o1[j], s23);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (!decltype(single)::value) {
              dev::mma_f16(o[c * 4 + j][nt], a0, a1, a2, a3, pf[h][nt][0], pf[h][nt][1]);
            } else {
              float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
              dev::mma_f16(x, a0, a1, a2, a3, pf[h][nt][0], pf[h][nt][1]);
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (((nt * 8 + 2 * t + (k & 1)) >> P.g_log2) == only) o[c * 4 + j][nt][k] += x[k];
            }
          }
        }
      }
    };
    if constexpr (EDGE) {
      // a NaN in a key that only later new tokens see must not reach the
      // earlier ones as 0 * NaN: such steps run token by token
      uint32_t bad = 0;
#pragma unroll
      for (int x = 0; x < KEYS / 4; ++x) {
        const int row = x * 4 + t;
        const unsigned char* scl =
            vt + (row / BS) * TILE + BS * (D / 2) + (row % BS) * (D / 16) + (g * VW) / 2;
        bad |= uint32_t(key0 + row < tok1 && (*scl & 0x7F) == 0x7F);
      }
      if (P.q_len > 1 && __any_sync(0xffffffffu, bad != 0)) {
        for (int x = 0; x < n_tok; ++x)
#pragma unroll
          for (int h = 0; h < 2; ++h) value_product(h, min(tok1, see0 + x), x, std::true_type{});
        return;
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) value_product(h, tok1, -1, std::false_type{});
  };

  // the steps before the first that is an edge; key0 + KEYS > see_first there
  const int n_full = see_first <= tok0 ? 0 : (see_first - tok0) / KEYS;  // whole steps of the CTA
  const int n_inner = n_full > warp ? (n_full - warp + NWARPS - 1) / NWARPS : 0;
  for (int i = 0, stage = 0; i < n_my; ++i) {
    dev::cp_async_wait<ST - 1>();
    __syncwarp();
    if (i < n_inner)
      step(i, stage, std::false_type{});
    else
      step(i, stage, std::true_type{});
    __syncwarp();
    issue(i + ST, stage);
    stage = stage + 1 == ST ? 0 : stage + 1;
  }

  // ---- merge the warps through shared memory (reusing the rings)
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[nt][c] += __shfl_xor_sync(0xffffffffu, l[nt][c], x);
  __syncthreads();
  float* sm_o = reinterpret_cast<float*>(smem);              // [NWARPS][COLS][OROW]
  float* sm_m = sm_o + NWARPS * C::COLS * C::OROW;           // [NWARPS][COLS]
  float* sm_l = sm_m + NWARPS * C::COLS;                     // [NWARPS][COLS]
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int n = warp * C::COLS + nt * 8 + 2 * t + c;
      if (g == 0) {
        sm_m[n] = limit[nt][c] == -INFINITY ? -INFINITY : ref[nt][c];
        sm_l[n] = l[nt][c];
      }
#pragma unroll
      for (int k = 0; k < D / 16; ++k)  // rows g and g + 8 of tile k: elements g D/8 + 2k, + 1
        *reinterpret_cast<float2*>(sm_o + n * C::OROW + g * (D / 8) + 2 * k) =
            make_float2(o[k][nt][c], o[k][nt][c + 2]);
    }
  __syncthreads();
  const float vs = P.v_scale[head];
  for (int idx = tid; idx < n_cols * (D / 2); idx += NTHREADS) {
    const int n = idx / (D / 2), d = idx % (D / 2) * 2;
    const int last = see0 + (n >> P.g_log2);  // keys this row sees
    if (tok0 >= last) continue;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) M = fmaxf(M, sm_m[w * C::COLS + n]);
    float x = 0.0f, y = 0.0f, den = 0.0f;
#pragma unroll
    for (int w = 0; w < NWARPS; ++w) {
      const int r = w * C::COLS + n;
      const float wt = sm_m[r] == -INFINITY ? 0.0f : dev::fast_exp2(sm_m[r] - M);
      const float2 v = *reinterpret_cast<const float2*>(sm_o + r * C::OROW + d);
      x = fmaf(wt, v.x, x);
      y = fmaf(wt, v.y, y);
      den = fmaf(wt, sm_l[r], den);
    }
    x *= vs;
    y *= vs;
    const int64_t row = q_row(n);
    if (last <= P.partition_tokens) {
      const float inv = __frcp_rn(den);
      *reinterpret_cast<__nv_bfloat162*>(P.out + row * D + d) =
          __floats2bfloat162_rn(x * inv, y * inv);
    } else {
      const int64_t prow = row * P.num_partitions + part;
      *reinterpret_cast<float2*>(P.part_acc + prow * D + d) = make_float2(x, y);
      if (d == 0) {
        P.part_m[prow] = M;
        P.part_l[prow] = den;
      }
    }
  }
}

template <int D, int NT, int BS>
int launch_t(const Fp4Decode& P, const pa_decode_params* p, cudaStream_t stream) {
  using C = Cfg<D, NT, BS>;
  const size_t smem = C::TILES + size_t(P.partition_tokens / BS + 1) * sizeof(int32_t);
  // the opt-in to large shared memory is per device: asked for the most that
  // a partition may need, once each
  static std::atomic<uint64_t> configured{0};
  int device = 0;
  cudaError_t e = cudaGetDevice(&device);
  if (e != cudaSuccess) return int(e);
  const uint64_t bit = uint64_t(1) << (device & 63);
  if (!(configured.load(std::memory_order_relaxed) & bit)) {
    const size_t most = C::TILES + size_t(kMaxPartitionTokens / BS + 1) * sizeof(int32_t);
    e = cudaFuncSetAttribute(paged_decode_fp4_kernel<D, NT, BS>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, int(most));
    if (e != cudaSuccess) return int(e);
    configured.fetch_or(bit, std::memory_order_relaxed);
  }
  const dim3 grid(unsigned(P.num_partitions), unsigned(P.num_kv_heads),
                  unsigned(p->num_seqs * P.n_groups));
  paged_decode_fp4_kernel<D, NT, BS><<<grid, NTHREADS, smem, stream>>>(P);
  return int(cudaGetLastError());
}

template <int D, int NT>
int launch_bs(const Fp4Decode& P, const pa_decode_params* p, cudaStream_t s) {
  switch (p->block_size) {
    case 8: return launch_t<D, NT, 8>(P, p, s);
    case 16: return launch_t<D, NT, 16>(P, p, s);
    case 32: return launch_t<D, NT, 32>(P, p, s);
    default: return int(cudaErrorInvalidValue);
  }
}

}  // namespace

int launch_decode_fp4(const DecodeLaunch& L, void* stream) {
  const pa_decode_params* p = L.p;
  const MmaColumns cols = mma_columns(p->num_q_heads / p->num_kv_heads, query_len_of(p));
  Fp4Decode P;
  P.q = static_cast<const __nv_bfloat16*>(p->q);
  P.out = static_cast<__nv_bfloat16*>(p->out);
  P.k_cache = static_cast<const unsigned char*>(p->k_cache);
  P.v_cache = static_cast<const unsigned char*>(p->v_cache);
  P.k_scale = p->k_scale;
  P.v_scale = p->v_scale;
  P.block_tables = p->block_tables;
  P.context_lens = p->context_lens;
  P.part_m = L.part_m;
  P.part_l = L.part_l;
  P.part_acc = L.part_acc;
  P.scale_log2 = p->scale * kLog2e;
  P.max_blocks_per_seq = p->max_blocks_per_seq;
  P.num_kv_heads = p->num_kv_heads;
  P.num_blocks = p->num_blocks;
  P.max_context_len = p->max_context_len;
  P.g_log2 = log2_of(p->num_q_heads / p->num_kv_heads);
  P.q_len = query_len_of(p);
  P.q_group = cols.q_group;
  P.n_groups = cols.n_groups;
  P.partition_tokens = L.partition_tokens;
  P.num_partitions = L.num_partitions;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (p->head_dim * 4 + cols.n_tiles) {
    case 64 * 4 + 1: return launch_bs<64, 1>(P, p, s);
    case 64 * 4 + 2: return launch_bs<64, 2>(P, p, s);
    case 128 * 4 + 1: return launch_bs<128, 1>(P, p, s);
    case 128 * 4 + 2: return launch_bs<128, 2>(P, p, s);
    default: return int(cudaErrorInvalidValue);
  }
}

int read_and_clear_decode_fp4_errors(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_decode_fp4_errors, sizeof(v));
  if (e != cudaSuccess) return int(e);
  e = cudaMemcpyToSymbol(g_decode_fp4_errors, &zero, sizeof(zero));
  *flags = v;
  return int(e);
}

}  // namespace pa
