// Declarations of the device-side tables and of the attention over selected
// blocks, shared by their translation units and the API.
#pragma once

#include "pa_fp4.h"
#include "pa_internal.h"

namespace pa {

// Tables, slots and positions from lengths (pa_tables.cu); `num_sms`: of the device.
int launch_update_tables(const pa_update_tables_params* p, int num_sms, void* stream);
int read_and_clear_tables_errors(uint32_t* flags);

// Bounds, scores and choice of blocks (pa_blocks.cu)
int launch_block_bounds(const pa_block_bounds_params* p, int num_sms, void* stream);
int launch_block_scores(const pa_block_scores_params* p, int num_sms, void* stream);
int launch_block_select(const float* scores, const int32_t* context_lens, int32_t* selected,
                        int32_t num_seqs, int32_t num_kv_heads, int32_t scores_stride,
                        int32_t block_size, int32_t budget, int32_t sink, int32_t recent,
                        int num_sms, void* stream);
int read_and_clear_blocks_errors(uint32_t* flags);

// Attention over selected blocks (pa_decode_selected.cu): the query rows of a KV head
// are the 8 columns of its products, as in the 4-bit decode; `split` CTAs, a cluster, take
// the list of one (sequence, column group, KV head).
struct SelectedPlan {
  MmaColumns cols;
  int cap;    // keys a sequence may have
  int split;  // CTAs of a cluster: 1, 2, 4 or 8
};
// 16-key steps of a list, at most.
inline int64_t selected_steps(const pa_decode_params* p, int num_selected) {
  const int64_t table = int64_t(p->max_blocks_per_seq) * p->block_size;
  const int64_t cap = p->max_context_len < table ? p->max_context_len : table;
  const int64_t blocks = (cap + p->block_size - 1) / p->block_size;
  const int64_t n = blocks < num_selected ? blocks : num_selected;
  return (n * p->block_size + 15) / 16;
}
SelectedPlan selected_plan(const pa_decode_params* p, int num_selected, int num_sms);
int launch_decode_selected(const pa_decode_params* p, const int32_t* selected, int num_selected,
                           const SelectedPlan& plan, void* stream);
int read_and_clear_selected_errors(uint32_t* flags);

}  // namespace pa
