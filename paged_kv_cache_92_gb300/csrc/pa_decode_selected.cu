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
//    of m16n8k16 products: S^T = K Q^T, O^T += V^T P^T, a warp taking 16 keys a step (of
//    codes 32). Its lanes copy the keys' K and V rows into the warp's own ring with 16-byte
//    asynchronous copies, which may go to any place of a stage, so 16-byte chunks are
//    permuted where the fragments' reads would meet in a bank. No CTA-wide barrier
//    until the end. (Warp-level products: with 8 columns they take 10 to 25 % of the matrix
//    unit, and their operands come converted from registers; products from tensor memory
//    would want 128 rows of keys a tile, more than a list's short end has.)
//  * bf16: fragments by ldmatrix, V's transposed. P is split into two bf16 terms (2^-17
//    of it is lost); with up to four query rows the second terms are columns 4 to 7 of
//    the same product (their queries are those of columns 0 to 3), so they cost none.
//  * 8-bit and 4-bit codes become f16 pairs in registers (exact), as in the 4-bit
//    decode, with its scaling of queries and its reference for P in f16.
//  * A CTA takes the list of one (sequence, column group, KV head); of few lists a
//    cluster of up to eight, which join their results through distributed shared memory: no
//    workspace, no second launch. The GPU deals out the CTAs as others end, which evens out
//    ragged contexts.
//  * Keys that a column must not see (behind the sequence, or behind one of several new
//    tokens) have weight 0; where V holds no number there, 0 times it would still be
//    none: in the steps that hold such keys, such elements of V are taken out first.
//
// Measured (GB300, in a graph; the floor is the bytes at the copy rate of 6.68 TB/s): 64
// contexts of 8 to 32 k, 128 blocks of 16 each, bf16, 32 / 8 heads 81.9 us (floor 80.6; the
// whole decode 769; the tensor-core decode over a table per KV head, its making left out,
// 95.0); 32 of 32 to 128 k, 256 blocks, 8-bit, 64 / 8 heads 46.6 us (40.4: a start of some 3
// us, and the ends of 256 lists on 152 SMs); one sequence, two new tokens, 64 blocks, 4-bit,
// d 64 4.7 us (a chain of list, table, copies, products and the cluster's two barriers).
// The next kernel is not dispatched ahead of the end: scores, choice and attention layer
// after layer take 145 us, the sum of the three, for 161 with CTAs of the next scores waiting
// beside the attention's last (alone, a kernel is as fast either way).
// 456 lists of 256 blocks in 4 bits 50.5 us (40.5): 600 instructions a step of 32 keys.
// More new tokens than 8 / G are groups of columns, each of which reads and converts the list
// again (from L2): 32 sequences, four new tokens, 256 blocks, 64 / 8 heads (four groups): bf16
// 149 us (81), 8-bit 131 (41), 4-bit 116 (23); 128 blocks, 32 / 8 heads (two groups), bf16 51.9
// (40.5).
// Tried: the lists of all sequences as a stream over persistent warps with a merge of what
// was cut (89.0, 53.8 us for the first two); 2 and 8 warps a CTA (84.2, 89.0); twice the
// ring or two thirds of it (no faster, or slower: codes with two stages and a third more
// CTAs 52.8 for 47.1); steps of 16 keys for the codes (4-bit: a third more time a key); a
// form of the step of its own for steps without unseen keys (twice the code: 1.5 us more
// for 8-bit, from instruction fetches).
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
constexpr int TILE_KEYS = 16;  // keys of a product
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
  int num_virtual;  // sequences * column groups
};

template <int FMT, int D, int BS>
struct Cfg {
  static constexpr int ROWB = FMT == PA_KV_BF16 ? 2 * D : (FMT == PA_KV_FP8_E4M3 ? D : D / 2);
  static constexpr int SCALES = FMT == PA_KV_FP4_E2M1 ? D / 16 : 0;
  static constexpr int TILE = BS * (ROWB + SCALES);         // of one (block, KV head)
  // keys of a warp's step: about 8 KB at head_dim 128 (of the codes half as much: what a
  // step costs beside its keys is a tenth of its instructions)
  static constexpr int KEYS = FMT == PA_KV_BF16 ? 16 : 32;
  static constexpr int HALVES = KEYS / TILE_KEYS;           // products of a step
  static constexpr int HALF = KEYS * (ROWB + SCALES);       // K (or V) of a step
  static constexpr int STAGE = 2 * HALF;
  static constexpr int ST = 3;                              // stages of a warp's ring
  static constexpr int NBK = BS < KEYS ? KEYS / BS : 1;     // blocks of a step
  static constexpr int SPB = BS > KEYS ? BS / KEYS : 1;     // steps of a block
  static constexpr int WINDOW = 32 / NBK;                   // steps whose entries a warp holds
  static constexpr int RING = NWARPS * ST * STAGE;
  // CTAs on an SM: by the rings, then by 65,536 registers
  static constexpr int CTAS = D == 64 ? 4 : (FMT == PA_KV_FP4_E2M1 ? 3 : 2);
  static constexpr int OROW = D + 4;                        // padded row of the merge
  static constexpr int MERGE = NWARPS * COLS * OROW * 4;    // takes the rings' place at the end
  static constexpr int SMEM = RING > MERGE ? RING : MERGE;
  // key row of 16 that is row r of their product
  __device__ static __forceinline__ int key_of(int r) {
    if constexpr (FMT == PA_KV_FP8_E4M3 && BS >= TILE_KEYS)
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

// A virtual sequence: column group `grp` of sequence b.
struct Virtual {
  int b, first_tok, n_tok;  // the group's first new token, its tokens
  int see0;                 // keys that the first one sees
  int blocks;               // of the sequence; 0: empty, or without room for the new tokens
  int entries;              // of a list
};
__device__ __forceinline__ Virtual virtual_of(const Sel& P, int v, int bs) {
  Virtual x;
  x.b = v / P.n_groups;
  x.first_tok = (v - x.b * P.n_groups) * P.q_group;
  x.n_tok = min(P.q_group, P.q_len - x.first_tok);
  int L = min(P.context_lens[x.b], P.cap);
  L = L < P.q_len ? 0 : L;
  x.see0 = L - P.q_len + x.first_tok + 1;
  x.blocks = (L + bs - 1) / bs;
  x.entries = min(P.num_selected, x.blocks);
  return x;
}

// row of q / out of column n: new token n / G of the group, query head head * G + n % G
__device__ __forceinline__ int64_t q_row(const Sel& P, const Virtual& v, int head, int n) {
  return (int64_t(v.b) * P.q_len + v.first_tok + (n >> P.g_log2)) *
             (int64_t(P.num_kv_heads) << P.g_log2) +
         (head << P.g_log2) + (n & ((1 << P.g_log2) - 1));
}

// The queries and scales of a list, on their way: loaded some time before they are used.
// DUP (bf16): columns 4 to 7 repeat columns 0 to 3 and take the second terms of P.
template <int FMT, int D, bool DUP>
struct Raw {
  uint4 q[D / 32];  // column lane / 4; bf16: pairs 2t, 2t + 1 of 8 elements each
  float k_scale, v_scale;
  int n_tok, see0;

  __device__ __forceinline__ void fetch(const Sel& P, const Virtual& v, int head) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const int n_cols = v.n_tok << P.g_log2, col = DUP ? g & 3 : g;
    n_tok = v.n_tok;
    see0 = v.see0;
    const __nv_bfloat16* row = P.q + q_row(P, v, head, min(col, n_cols - 1)) * D;
    // (nothing that needs the values: the warp would wait for them)
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      if constexpr (FMT == PA_KV_BF16) {
        const uint32_t* x = reinterpret_cast<const uint32_t*>(row + 32 * i + 2 * t);
        q[i] = make_uint4(x[0], x[4], x[8], x[12]);
      } else {  // the order of the codes' fragments
        constexpr int E = dev::KeyRow<FMT, D>::E;
        q[i] = *reinterpret_cast<const uint4*>(row + (4 * (8 * i / E) + t) * E + 8 * i % E);
      }
    }
    k_scale = v_scale = 1.0f;
    if constexpr (FMT != PA_KV_BF16) {
      k_scale = P.k_scale[head];
      v_scale = P.v_scale[head];
    }
  }
};

// What a warp needs of a list at hand.
template <int FMT, int D, bool DUP>
struct Columns {
  uint32_t qf[D / 16][2];  // the queries as the B operand (column lane / 4)
  float factor[2];  // of columns 2t and 2t+1: softmax scale * K scale / the row's scaling
  int see[2];       // keys that they see
  int see0, n_tok;
  float v_scale;

  __device__ __forceinline__ void take(const Sel& P, Raw<FMT, D, DUP>& raw) {
    const int t = threadIdx.x & 3, g = (threadIdx.x & 31) >> 2;
    if ((DUP ? g & 3 : g) >= raw.n_tok << P.g_log2)  // no query: zeros
#pragma unroll
      for (int i = 0; i < D / 32; ++i) raw.q[i] = uint4{};
    see0 = raw.see0;
    n_tok = raw.n_tok;
    v_scale = raw.v_scale;
    const float inv_scaling = dev::query_fragment<FMT, D>(raw.q, qf);
    float k_scale = raw.k_scale;
    if constexpr (FMT != PA_KV_BF16) {
      // a negative scale turns the queries, so that a larger product stays a larger score
      const uint32_t sign = k_scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        qf[s][0] ^= sign;
        qf[s][1] ^= sign;
      }
      k_scale = fabsf(k_scale);
    }
    const float row_factor = P.scale_log2 * k_scale * inv_scaling;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      factor[c] = __shfl_sync(0xffffffffu, row_factor, 4 * (2 * t + c));
      // A scale of zero makes all scores equal, but 0 * -inf is NaN: below 2^-100 the
      // products (under 2^35) count as zero either way. The comparison keeps a NaN scale.
      if (FMT != PA_KV_BF16) factor[c] = factor[c] < 0x1p-100f ? 0x1p-100f : factor[c];
      const int n = DUP ? (2 * t + c) & 3 : 2 * t + c;
      see[c] = see0 + min(n >> P.g_log2, n_tok - 1);
    }
  }
};

// Softmax state of columns 2t and 2t+1: a key's weight is exp2((s - ref) * factor +
// HEADROOM), s the raw product and ref the one that the reference was taken from (0
// before the first key that the column sees): the difference comes first, as the last
// place of a large score is many units. limit: the raw product beyond which ref moves,
// 8 above it, so that no weight passes 2^15.
template <int FMT, int D, int BS, bool DUP>
struct State {
  using C = Cfg<FMT, D, BS>;
  float o[D / 16][4];  // O^T: D / 16 tiles of 16 rows
  float ref[2], limit[2], l[2];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      ref[c] = l[c] = 0.0f;
      limit[c] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
  }

  // A fragments of V^T: rows d = 16 i .. 16 i + 15, keys of the products' rows.
  __device__ static __forceinline__ void v_fragment(const unsigned char* vt, int i,
                                                    uint32_t (&a)[4]) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if constexpr (FMT == PA_KV_BF16) {
      // lanes 8 m .. 8 m + 7 name the rows of matrix m: keys (m / 2) * 8 .., chunk 2 i + m % 2
      const int m = lane >> 3, r = (m >> 1) * 8 + (lane & 7);
      ldmatrix_x4_trans(a, vt + r * C::ROWB + (((2 * i + (m & 1)) ^ (r & 7)) * 16));
    } else if constexpr (BS >= TILE_KEYS) {
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

  // position of row r of product h of a step whose blocks begin at `pos`
  __device__ static __forceinline__ int position(const int (&pos)[C::NBK], int h, int r) {
    const int k = C::key_of(r);
    if constexpr (BS < TILE_KEYS)
      return k < BS ? pos[2 * h] + k : pos[2 * h + 1] + k - BS;
    else
      return pos[h * TILE_KEYS / BS] + h * TILE_KEYS % BS + k;
  }
  // The same of key k of the step.
  __device__ static __forceinline__ int key_position(const int* pos, int k) {
    return pos[k / BS] + k % BS;
  }

  // Element d of V's key k in a stage: where it lies (of a 4-bit V its group scale, the
  // codes being finite), and its value where that is no finite number, else 0.
  __device__ static __forceinline__ unsigned char* v_place(unsigned char* stage, int k, int d) {
    unsigned char* vt = stage + C::HALF;
    if constexpr (FMT == PA_KV_BF16) return vt + k * C::ROWB + ((d / 8) ^ (k & 7)) * 16 + d % 8 * 2;
    constexpr int W = BS < TILE_KEYS ? BS : TILE_KEYS;  // keys of a sub-tile of V^T
    if constexpr (FMT == PA_KV_FP8_E4M3) return vt + k / W * W * D + d * W + k % W;
    return vt + C::KEYS * C::ROWB + k * C::SCALES + d / 16;
  }
  __device__ static __forceinline__ float not_finite(const unsigned char* at) {
    if constexpr (FMT == PA_KV_BF16) {
      const float x = __uint_as_float(uint32_t(*reinterpret_cast<const uint16_t*>(at)) << 16);
      return isfinite(x) ? 0.0f : x;
    } else {
      return (*at & 0x7F) == 0x7F ? NAN : 0.0f;
    }
  }

  // For a step that holds keys which some column does not see: their weight is 0 there,
  // but 0 times what is no number is none. Rows of V that no column sees become zero. In
  // those that some see, so do the infinities and NaN, and are added to these columns
  // here (a weight is positive).
  __device__ __forceinline__ void clear_unseen(unsigned char* stage, const int* pos,
                                               const Columns<FMT, D, DUP>& q) {
    const int lane = threadIdx.x & 31;
    const int see_last = q.see0 + q.n_tok - 1;
    unsigned char* vt = stage + C::HALF;
    if constexpr (FMT == PA_KV_BF16) {
#pragma unroll
      for (int x = lane; x < C::KEYS * C::ROWB / 16; x += 32)
        if (key_position(pos, x / (C::ROWB / 16)) >= see_last)
          reinterpret_cast<uint4*>(vt)[x] = uint4{};
    } else if constexpr (FMT == PA_KV_FP8_E4M3) {
      constexpr int W = BS < TILE_KEYS ? BS : TILE_KEYS;  // keys of a sub-tile of V^T
#pragma unroll 1
      for (int u = 0; u < C::KEYS / W; ++u) {
        const int seen = see_last - key_position(pos, u * W);  // of its keys, from the first
        if (seen >= W) continue;
        uint32_t keep[W / 4];
#pragma unroll
        for (int i = 0; i < W / 4; ++i) {
          const int n = min(max(seen - 4 * i, 0), 4);
          keep[i] = n == 4 ? 0xffffffffu : (1u << (8 * n)) - 1u;
        }
#pragma unroll
        for (int d = lane; d < D; d += 32) {
          uint32_t* x = reinterpret_cast<uint32_t*>(vt + (u * D + d) * W);
#pragma unroll
          for (int i = 0; i < W / 4; ++i) x[i] &= keep[i];
        }
      }
    } else {
      static_assert(C::KEYS <= 32, "a lane for every key");
      if (lane < C::KEYS && key_position(pos, lane) >= see_last)
#pragma unroll
        for (int i = 0; i < C::SCALES; i += 4)
          *reinterpret_cast<uint32_t*>(vt + C::KEYS * C::ROWB + lane * C::SCALES + i) = 0;
    }
    __syncwarp();
#pragma unroll 1
    for (int at = q.see0; at < see_last; ++at)  // keys that some see, block by block
#pragma unroll 1
      for (int n = 0; n < C::NBK; ++n) {
        const int in = at - pos[n];
        if (in < 0 || in >= (BS < C::KEYS ? BS : C::KEYS)) continue;
        const int k = n * BS + in;
        float bad[D / 16][2];
        bool any = false;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            bad[i][j] = not_finite(v_place(stage, k, element(i, 2 * j)));
            any |= bad[i][j] != 0.0f;  // (true of a NaN)
          }
        if (__any_sync(0xffffffffu, any)) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (bad[i][j] != 0.0f) {
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  // (of two equal columns the first takes it)
                  if (at < q.see[c] && !(DUP && (threadIdx.x & 3) >= 2)) o[i][2 * j + c] += bad[i][j];
                unsigned char* x = v_place(stage, k, element(i, 2 * j));
                if constexpr (FMT == PA_KV_BF16)
                  *reinterpret_cast<uint16_t*>(x) = 0;
                else
                  *x = 0;
              }
        }
        __syncwarp();
      }
  }

  // One step, its blocks' first positions `blocks`.
  __device__ __forceinline__ void step(unsigned char* stage, const int* blocks,
                                       const Columns<FMT, D, DUP>& q) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    int pos[C::NBK];
    bool edge = false;  // keys that some column does not see
#pragma unroll
    for (int n = 0; n < C::NBK; ++n) {
      pos[n] = blocks[n];
      edge |= pos[n] + (BS < C::KEYS ? BS : C::KEYS) > q.see0;
    }
    float s[C::HALVES][4];
#pragma unroll
    for (int h = 0; h < C::HALVES; ++h) {
      const unsigned char* kt = stage + h * TILE_KEYS * C::ROWB;
      float s2[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s2[i][j] = 0.0f;
      if constexpr (FMT == PA_KV_BF16) {
        // matrix m: keys (m % 2) * 8 .., chunk 2 i + m / 2
        const int m = lane >> 3, r = (m & 1) * 8 + (lane & 7);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t a[4];
          ldmatrix_x4(a, kt + r * C::ROWB + (((2 * i + (m >> 1)) ^ (r & 7)) * 16));
          dev::mma_bf16_regs(s2[i & 1], a[0], a[1], a[2], a[3], q.qf[i][0], q.qf[i][1]);
        }
      } else {
        using Row = dev::KeyRow<FMT, D>;
        Row rows[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = C::key_of(g + 8 * i);
          if constexpr (FMT == PA_KV_FP8_E4M3 && D == 128) {
            // (runs t and t + 4 of the row, permuted as they were copied)
            const uint4 x =
                *reinterpret_cast<const uint4*>(kt + r * D + ((t ^ ((r & 1) << 2)) * 16));
            const uint4 y =
                *reinterpret_cast<const uint4*>(kt + r * D + (((t + 4) ^ ((r & 1) << 2)) * 16));
            rows[i].w[0] = x.x; rows[i].w[1] = x.y; rows[i].w[2] = x.z; rows[i].w[3] = x.w;
            rows[i].w[4] = y.x; rows[i].w[5] = y.y; rows[i].w[6] = y.z; rows[i].w[7] = y.w;
          } else {
            rows[i].load(kt + r * C::ROWB + t * Row::RUN,
                         stage + C::KEYS * C::ROWB + (h * TILE_KEYS + r) * C::SCALES + t * (D / 64));
          }
        }
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t x[4], y[4];
          rows[0].pairs(c, x);
          rows[1].pairs(c, y);
#pragma unroll
          for (int k = 0; k < 2; ++k)
            dev::mma_f16(s2[k], x[2 * k], y[2 * k], x[2 * k + 1], y[2 * k + 1],
                         q.qf[2 * c + k][0], q.qf[2 * c + k][1]);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) s[h][j] = s2[0][j] + s2[1][j];
    }
    // ---- softmax; keys that a column does not see are -inf
    if (edge)
#pragma unroll
      for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (position(pos, h, g + (j >> 1) * 8) >= q.see[j & 1]) s[h][j] = -INFINITY;
    bool over = false;
#pragma unroll
    for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
      for (int j = 0; j < 4; ++j) over |= s[h][j] > limit[j & 1];
    if (__any_sync(0xffffffffu, over)) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float x = -INFINITY;
#pragma unroll
        for (int h = 0; h < C::HALVES; ++h) x = fmaxf(x, fmaxf(s[h][c], s[h][c + 2]));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        // no branch: the lanes of a warp stay together
        const bool first = limit[c] == -INFINITY;
        const bool take = x != -INFINITY && (first || x > ref[c]);
        const float y = take ? x : ref[c];
        const float old = dev::fast_exp2((ref[c] - y) * q.factor[c]);
        const float a = take && first ? 0.0f : old;
        ref[c] = y;
        limit[c] = take ? __fadd_rd(x, __fdividef(8.0f - 0x1p-16f, q.factor[c])) : limit[c];
        l[c] *= a;
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          o[k][c] *= a;
          o[k][c + 2] *= a;
        }
      }
    }
    __syncwarp();
    uint32_t pf[C::HALVES][2];                   // P^T as the second product's B operand
    [[maybe_unused]] uint32_t pl[C::HALVES][2];  // its second terms
#pragma unroll
    for (int h = 0; h < C::HALVES; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 e = dev::fma_pair(dev::sub_pair(make_float2(s[h][2 * i], s[h][2 * i + 1]), ref),
                                       q.factor, HEADROOM);
        const float p0 = dev::fast_exp2(e.x), p1 = dev::fast_exp2(e.y);
        l[0] += p0;
        l[1] += p1;
        if constexpr (FMT == PA_KV_BF16) {
          const uint32_t hi = pack_bf16(p0, p1);
          const uint32_t lo = pack_bf16(p0 - dev::bf16_lo(hi), p1 - dev::bf16_hi(hi));
          pf[h][i] = dev::transpose_8x8(DUP && t >= 2 ? lo : hi);
          if (!DUP) pl[h][i] = dev::transpose_8x8(lo);
        } else {
          pf[h][i] = dev::transpose_8x8(dev::pack_f16(p0, p1));
        }
      }
    if (edge) clear_unseen(stage, blocks, q);
    // ---- O^T += V^T P^T
#pragma unroll
    for (int h = 0; h < C::HALVES; ++h) {
      const unsigned char* vt = stage + C::HALF + h * TILE_KEYS * C::ROWB;
      auto tile_product = [&](int i, const uint32_t (&a)[4]) {
        if constexpr (FMT == PA_KV_BF16) {
          dev::mma_bf16_regs(o[i], a[0], a[1], a[2], a[3], pf[h][0], pf[h][1]);
          if constexpr (!DUP)
            dev::mma_bf16_regs(o[i], a[0], a[1], a[2], a[3], pl[h][0], pl[h][1]);
        } else {
          dev::mma_f16(o[i], a[0], a[1], a[2], a[3], pf[h][0], pf[h][1]);
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
        const unsigned char* scales =
            stage + C::HALF + C::KEYS * C::ROWB + h * TILE_KEYS * C::SCALES;
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
          sb[r] = scales[k * C::SCALES + (g * VW) / 2];
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
    }
  }
  // The warp's result: sums over the lanes of a column, second terms to the first ones.
  // maximum[c]: in the log2 domain; +inf where the sum is NaN, so that it reaches the end.
  __device__ __forceinline__ void finish(const Columns<FMT, D, DUP>& q, float (&maximum)[2]) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l[c] += __shfl_xor_sync(0xffffffffu, l[c], x);
      maximum[c] = l[c] != l[c] ? INFINITY
                                : (limit[c] == -INFINITY ? -INFINITY
                                                         : fmaf(ref[c], q.factor[c], -HEADROOM));
    }
    if constexpr (DUP)
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[k][j] += __shfl_xor_sync(0xffffffffu, o[k][j], 2);
  }
  // element of O that o[k][j] is, of column 2t + j % 2
  __device__ static __forceinline__ int element(int k, int j) {
    const int g = (threadIdx.x & 31) >> 2;
    // rows g and g + 8 of tile k; of a 4-bit V elements g D/8 + 2k, + 1
    return FMT == PA_KV_FP4_E2M1 ? g * (D / 8) + 2 * k + (j >> 1) : 16 * k + g + (j >> 1) * 8;
  }
};

// A block of a step: its first position there (NOWHERE: nothing is read) and its tile
// (block * num_kv_heads + head).
struct Entry {
  int pos, tile;
};
// Entry e of the list of (sequence b, head): a logical block.
__device__ __forceinline__ int listed(const Sel& P, int b, int head, int e) {
  return P.selected[(int64_t(b) * P.num_kv_heads + head) * P.num_selected + e];
}
// Logical block j of v, from its row `row0` on.
template <int BS>
__device__ __forceinline__ Entry entry_of(const Sel& P, const Virtual& v, int head, int j, int row0,
                                          unsigned& errors) {
  Entry x{NOWHERE, 0};
  if (j >= v.blocks) errors |= PA_DEVERR_KEEP;
  if (j >= 0 && j < v.blocks) {
    const int k = P.block_tables[int64_t(v.b) * P.max_blocks_per_seq + j];
    if (k < 0 || k >= P.num_blocks)
      errors |= PA_DEVERR_TABLE_ENTRY;
    else
      x = Entry{j * BS + row0, k * P.num_kv_heads + head};
  }
  return x;
}
// Copies block n of a step (K and V) into its stage.
template <int FMT, int D, int BS>
__device__ __forceinline__ void copy_block(const Sel& P, unsigned char* st, int n, Entry e) {
  using C = Cfg<FMT, D, BS>;
  const int lane = threadIdx.x & 31;
  const bool on = e.pos != NOWHERE;
  const int row0 = C::SPB > 1 ? e.pos % BS : 0;  // of the step in the block
  const int64_t at = int64_t(e.tile) * C::TILE + row0 * C::ROWB + lane * 16;
  constexpr int ROWS = BS < C::KEYS ? BS : C::KEYS;  // of the block in a step
  constexpr int CHUNKS = ROWS * C::ROWB / 16;   // 16-byte chunks
  constexpr int CPR = C::ROWB / 16;             // of a row (of V in 8 bits: just so many bytes)
#pragma unroll
  for (int c = 0; c < CHUNKS; c += 32) {
    const int x = c + lane;
    const bool in = on && (c + 32 <= CHUNKS || x < CHUNKS);
    const int r = n * ROWS + x / CPR, k = x % CPR;
    int kd = r * C::ROWB + k * 16, vd = n * ROWS * C::ROWB + x * 16;
    if constexpr (FMT == PA_KV_BF16) {
      kd = r * C::ROWB + (k ^ (r & 7)) * 16;
      vd = kd;
    } else if constexpr (FMT == PA_KV_FP8_E4M3 && D == 128) {
      kd = r * C::ROWB + (k ^ ((r & 1) << 2)) * 16;
    }
    dev::cp_async16(st + kd, P.k_cache + at + c * 16, in);
    dev::cp_async16(st + C::HALF + vd, P.v_cache + at + c * 16, in);
  }
  if constexpr (C::SCALES > 0) {
    constexpr int N = ROWS * C::SCALES / 16;  // chunks of scales, of K then of V
    const bool of_v = lane >= N;
    const int x = of_v ? lane - N : lane;
    const unsigned char* from = (of_v ? P.v_cache : P.k_cache) + int64_t(e.tile) * C::TILE +
                                BS * C::ROWB + row0 * C::SCALES + x * 16;
    dev::cp_async16(st + (of_v ? C::HALF : 0) + C::KEYS * C::ROWB + n * ROWS * C::SCALES + x * 16,
                    from, on && lane < 2 * N);
  }
}

// A length that is too long or too short, flagged once: by the first CTA of the sequence's
// first list. (No index of its own: CTAs times threads passes 32 bits with 2^24 lists.)
__device__ __forceinline__ void report_length(const Sel& P, const Virtual& v, int head, int rank) {
  if (threadIdx.x != 0 || rank != 0 || head != 0 || v.first_tok != 0) return;
  const int L = P.context_lens[v.b];
  if (L > P.cap || (L > 0 && L < P.q_len)) atomicOr(&g_selected_errors, PA_DEVERR_CONTEXT_LEN);
}

// One list per cluster: its CTAs take equal stretches and join their results.
template <int FMT, int D, int BS, bool DUP>
__global__ void __launch_bounds__(NTHREADS, Cfg<FMT, D, BS>::CTAS)
    decode_selected_kernel(const Sel P) {
  using C = Cfg<FMT, D, BS>;
  constexpr int ST = C::ST;
  dev::griddep_wait();  // (the next kernel's CTAs come as these end: see above)
  cg::cluster_group cluster = cg::this_cluster();
  const int split = int(cluster.num_blocks()), rank = int(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int unit = blockIdx.x / split;
  const int head = unit % P.num_kv_heads, vseq = unit / P.num_kv_heads;
  // The list's entry for this lane's place in the warp's first steps (place_of below) if
  // the sequence fills the list: on its way while the length is.
  auto place_of = [&](int w0, int e0) {
    const int step = warp + NWARPS * (w0 + lane / C::NBK);
    return e0 + (C::NBK > 1 ? step * C::NBK + lane % C::NBK : step / C::SPB);
  };
  const int guess = place_of(0, int(int64_t(P.num_selected) * rank / split));
  const int early = guess < P.num_selected ? listed(P, vseq / P.n_groups, head, guess) : -1;
  const Virtual v = virtual_of(P, vseq, BS);
  const int n_cols = v.n_tok << P.g_log2;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ float sm_m[NWARPS][COLS], sm_l[NWARPS][COLS];
  __shared__ float2 sm_ml[COLS];          // of the CTA, read by the cluster
  __shared__ int sm_pos[NWARPS][ST][C::NBK];  // position of the first key of a step's blocks
  unsigned char* ring = smem + warp * ST * C::STAGE;

  // this CTA's entries of the list
  const int e0 = int(int64_t(v.entries) * rank / split);
  const int e1 = int(int64_t(v.entries) * (rank + 1) / split);
  const int n_steps = C::NBK > 1 ? (e1 - e0 + C::NBK - 1) / C::NBK : (e1 - e0) * C::SPB;
  const int n_my = n_steps > warp ? (n_steps - warp + NWARPS - 1) / NWARPS : 0;
  // The entries of this warp's steps [w0, w0 + WINDOW), NBK a step, one a lane.
  unsigned errors = 0;
  auto load_window = [&](int w0) {
    const int e = place_of(w0, e0);
    if (e >= e1) return Entry{NOWHERE, 0};
    const int j = w0 == 0 && v.entries == P.num_selected ? early : listed(P, v.b, head, e);
    const int step = warp + NWARPS * (w0 + lane / C::NBK);
    return entry_of<BS>(P, v, head, j, step % C::SPB * C::KEYS, errors);
  };
  Entry window = load_window(0);
  Raw<FMT, D, DUP> raw;
  raw.fetch(P, v, head);
  // One copy group: step i of the warp, empty past the last.
  auto issue = [&](int i, int stage) {
#pragma unroll
    for (int n = 0; n < C::NBK; ++n) {
      const int src = i % C::WINDOW * C::NBK + n;
      const Entry e{__shfl_sync(0xffffffffu, window.pos, src),
                    __shfl_sync(0xffffffffu, window.tile, src)};
      if (i < n_my) {
        if (lane == 0) sm_pos[warp][stage][n] = e.pos;
        copy_block<FMT, D, BS>(P, ring + stage * C::STAGE, n, e);
      }
    }
    dev::cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < ST - 1; ++i) issue(i, i);

  Columns<FMT, D, DUP> cols;
  State<FMT, D, BS, DUP> st;
  cols.take(P, raw);
  st.clear();
  for (int i = 0, stage = 0; i < n_my; ++i) {
    dev::cp_async_wait<ST - 2>();
    __syncwarp();  // the step's copies by all lanes, and its positions
    const int ahead = i + ST - 1;
    if (ahead % C::WINDOW == 0) window = load_window(ahead);
    issue(ahead, stage == 0 ? ST - 1 : stage - 1);
    st.step(ring + stage * C::STAGE, sm_pos[warp][stage], cols);
    __syncwarp();  // the stage has been read
    stage = stage + 1 == ST ? 0 : stage + 1;
  }
  dev::cp_async_wait<0>();
  if (errors) atomicOr(&g_selected_errors, errors);
  report_length(P, v, head, rank);
  __syncthreads();  // the rings give way to the merge

  // ---- the warps' results, then the CTA's, then the cluster's
  float* rows = reinterpret_cast<float*>(smem);  // [NWARPS][COLS][OROW]
  float maximum[2];
  st.finish(cols, maximum);
#pragma unroll
  for (int c = 0; c < 2; ++c)
    if (g == 0) {
      sm_m[warp][2 * t + c] = maximum[c];
      sm_l[warp][2 * t + c] = st.l[c];
    }
#pragma unroll
  for (int k = 0; k < D / 16; ++k)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      rows[(warp * COLS + 2 * t + (j & 1)) * C::OROW + st.element(k, j)] = st.o[k][j];
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
    // a CTA writes every split-th stretch of element pairs
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
      const float norm = den == 0.0f ? 0.0f : cols.v_scale / den;  // no key: a row of zeros
      *reinterpret_cast<__nv_bfloat162*>(P.out + q_row(P, v, head, n) * D + d) =
          __floats2bfloat162_rn(sum.x * norm, sum.y * norm);
    }
  }
  if (split > 1) cluster.sync();  // no CTA leaves while another reads its rows
}

template <int FMT, int D, int BS, bool DUP>
int launch_t(const Sel& P, const SelectedPlan& plan, cudaStream_t stream) {
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
  const int64_t lists = int64_t(P.num_virtual) * P.num_kv_heads;
  return launch_ordered(decode_selected_kernel<FMT, D, BS, DUP>,
                        dim3(unsigned(lists * plan.split)), NTHREADS, C::SMEM, stream,
                        unsigned(plan.split), P);
}

template <int FMT, int D, int BS>
int launch_dup(const Sel& P, const SelectedPlan& plan, cudaStream_t s) {
  if constexpr (FMT == PA_KV_BF16)
    if ((P.q_group << P.g_log2) <= 4) return launch_t<FMT, D, BS, true>(P, plan, s);
  return launch_t<FMT, D, BS, false>(P, plan, s);
}
template <int FMT, int D>
int launch_bs(const Sel& P, int block_size, const SelectedPlan& plan, cudaStream_t s) {
  switch (block_size) {
    case 8: return launch_dup<FMT, D, 8>(P, plan, s);
    case 16: return launch_dup<FMT, D, 16>(P, plan, s);
    case 32: return launch_dup<FMT, D, 32>(P, plan, s);
    default: return int(cudaErrorInvalidValue);
  }
}
template <int FMT>
int launch_d(const Sel& P, int head_dim, int block_size, const SelectedPlan& plan, cudaStream_t s) {
  return head_dim == 64 ? launch_bs<FMT, 64>(P, block_size, plan, s)
                        : launch_bs<FMT, 128>(P, block_size, plan, s);
}

int resident_ctas(int kv_dtype, int d) {
  switch (kv_dtype) {
    case PA_KV_BF16: return d == 64 ? Cfg<PA_KV_BF16, 64, 16>::CTAS : Cfg<PA_KV_BF16, 128, 16>::CTAS;
    case PA_KV_FP8_E4M3:
      return d == 64 ? Cfg<PA_KV_FP8_E4M3, 64, 16>::CTAS : Cfg<PA_KV_FP8_E4M3, 128, 16>::CTAS;
    default: return d == 64 ? Cfg<PA_KV_FP4_E2M1, 64, 16>::CTAS : Cfg<PA_KV_FP4_E2M1, 128, 16>::CTAS;
  }
}

}  // namespace

SelectedPlan selected_plan(const pa_decode_params* p, int num_selected, int num_sms) {
  SelectedPlan r{};
  r.cols = fp4_columns(p);
  const int64_t table = int64_t(p->max_blocks_per_seq) * p->block_size;
  r.cap = int(p->max_context_len < table ? p->max_context_len : table);
  const int64_t lists = int64_t(p->num_seqs) * r.cols.n_groups * p->num_kv_heads;
  const int64_t steps = selected_steps(p, num_selected);  // of a list, at most
  // CTAs a list: as many as are resident at once if it is few lists, with two steps a warp
  // at least; lists beyond that are worked off as CTAs end, whole (512 lists of 128 blocks in
  // bf16, 304 CTAs resident: 82.9 us whole, 90.4 in halves).
  const int64_t slots =
      int64_t(num_sms > 0 ? num_sms : 152) * resident_ctas(p->kv_dtype, p->head_dim);
  r.split = 1;
  while (r.split < MAX_SPLIT && lists * r.split * 2 <= slots && steps >= 4 * NWARPS * r.split)
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
  P.num_virtual = p->num_seqs * plan.cols.n_groups;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (p->kv_dtype) {
    case PA_KV_BF16: return launch_d<PA_KV_BF16>(P, p->head_dim, p->block_size, plan, s);
    case PA_KV_FP8_E4M3: return launch_d<PA_KV_FP8_E4M3>(P, p->head_dim, p->block_size, plan, s);
    default: return launch_d<PA_KV_FP4_E2M1>(P, p->head_dim, p->block_size, plan, s);
  }
}

int read_and_clear_selected_errors(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_selected_errors, sizeof(v));
  if (e != cudaSuccess) return int(e);
  if (v != 0) e = cudaMemcpyToSymbol(g_selected_errors, &zero, sizeof(zero));
  *flags = v;
  return int(e);
}

}  // namespace pa
