// Declarations of the 4-bit cache, the token weights and the eviction, shared by
// their translation units and the API.
#pragma once

#include "pa_internal.h"

namespace pa {

// Column layout of the 4-bit decode and of the token weights: the query rows
// of a KV head are the columns of its products, token by token, in `n_tiles`
// tiles of 8; a sequence with more new tokens than those hold is worked off as
// several groups, each reading the keys.
struct MmaColumns {
  int n_tiles, q_group, n_groups;
};
inline MmaColumns mma_columns(int g, int q, int max_tiles) {
  MmaColumns c;
  c.n_tiles = g * q <= 8 ? 1 : max_tiles;
  c.q_group = q < 8 * c.n_tiles / g ? q : 8 * c.n_tiles / g;
  c.n_groups = (q + c.q_group - 1) / c.q_group;
  return c;
}
inline MmaColumns fp4_columns(const pa_decode_params* p) {
  return mma_columns(p->num_q_heads / p->num_kv_heads, query_len_of(p), 1);
}

// 4-bit cache (pa_fp4.cu, pa_decode_fp4.cu)
int launch_reshape_and_cache_fp4(const void* k_new, const void* v_new, void* k_cache,
                                 void* v_cache, const int64_t* slot_mapping, const float* k_scale,
                                 const float* v_scale, int32_t num_tokens, int32_t num_kv_heads,
                                 int32_t head_dim, int32_t block_size, int32_t num_blocks,
                                 void* stream, const AppendCheck& check = AppendCheck());
int launch_gather_fp4(const void* k_cache, const void* v_cache, void* k_out, void* v_out,
                      const int64_t* slot_mapping, const float* k_scale, const float* v_scale,
                      int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                      int32_t block_size, int32_t num_blocks, void* stream);
// How the 4-bit decode deals out its work: contexts up to kFp4WholeTokens take
// one CTA per (sequence, column group, KV head); longer ones a stream over
// `grid` persistent CTAs, with two partials a CTA for the pieces it cuts. (32 / 8
// heads, d 128, whole against stream: one sequence of 512 tokens 6.2 and 9.2 us, of
// 1,024 8.8 and 9.4, of 2,048 14.6 and 10.0; 64 of up to 1,024 16.8 and 17.9, of up
// to 2,048 28.9 and 24.5.)
constexpr int kFp4WholeTokens = 1024;
struct Fp4Plan {
  int grid, cols, cap;  // CTAs; columns of a partial; keys a sequence may have
  bool whole;
};
Fp4Plan fp4_plan(const pa_decode_params* p, int num_sms);
// Stream positions (steps and starts of every item) fit 32 bits, and so do the
// keys of a sequence rounded up to whole steps.
inline bool fp4_stream_ok(const pa_decode_params* p) {
  const int64_t table = int64_t(p->max_blocks_per_seq) * p->block_size;
  const int64_t cap = p->max_context_len < table ? p->max_context_len : table;
  return cap <= (int64_t(1) << 31) - 64 &&
         double(p->num_seqs) * fp4_columns(p).n_groups * p->num_kv_heads *
             double(cap / 32 + 9) < 2147483648.0;
}
int launch_decode_fp4(const DecodeLaunch& L, const Fp4Plan& plan, void* stream);
int read_and_clear_fp4_errors(uint32_t* flags);
int read_and_clear_decode_fp4_errors(uint32_t* flags);

// Token weights (pa_weights.cu): the workspace and how the keys are split.
struct TokenWeightsSpace {
  size_t part, scores, total;  // byte offsets; the partitions' (max, sum), the scores
  int64_t score_stride;        // floats of a score row
  int cap;                     // keys a sequence may have
  int partition_tokens, num_partitions;
};
int launch_token_weights(const pa_token_weights_params* p, const TokenWeightsSpace& sp,
                         unsigned char* ws, void* stream);
int read_and_clear_weights_errors(uint32_t* flags);
// Eviction (pa_evict.cu)
int launch_evict_select(const float* token_weights, const int32_t* context_lens, int32_t* keep,
                        int32_t* new_lens, int32_t num_seqs, int64_t weights_stride,
                        int32_t budget, int32_t recent, void* stream);
int launch_evict_compact(const pa_evict_compact_params* p, void* stream);
int read_and_clear_evict_errors(uint32_t* flags);

}  // namespace pa
