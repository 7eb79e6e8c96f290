// A step's metadata made on the device for sm_103a: block tables resized to new
// lengths, slots and positions of the new tokens.
//
// The host pool (pa_pool.cpp) keeps tables where the scheduler is ("How Paged
// Attention and Continuous Batching Actually Work", §One step, end to end:
// allocate_slots). Where the lengths are on the device -- after an eviction, or in
// a captured loop -- this does the same there: sequence b, which holds blocks for
// old_lens[b] tokens, shall hold them for new_lens[b].
//
// Free blocks are a ring {head, count}: fresh ones come from its head and released
// ones go to its tail, so what is taken does not depend on what is given back in the
// same call, and no thread reads what another one writes: fresh blocks lie in ring
// entries [head, head + count), released ones go behind them; a token's block is read
// from the ring where it is fresh and from the table's old part where it is not. The
// state's new value goes to memory of its own. So the CTAs need no order among them,
// and every one finds its items by itself: it adds up the blocks and tokens of all
// sequences (three prefix sums, a few instructions a sequence) and looks the items
// that it deals with up in the sums by binary search in shared memory. The sums are
// kept per thread: with more than 512 sequences a thread has several in a row, and a
// search ends in a walk over those (up to 128, two dependent loads a step).
//
// All or nothing: whether the step is possible is known to every CTA from the same
// sums before it writes.
//
// What bounds it: latency. A step of 64 sequences moves under 2 KB; the kernel is a
// chain of the lengths' load, a scan, a search and the dependent loads of a table or
// ring entry. One launch; a second one to hold the sums would cost as much again. With
// thousands of sequences it is the walk, and the lengths, which every CTA reads whole.
// Measured (GB300, in a graph): a decode step of 64 sequences 3.4 us; 256 sequences, of
// which a quarter end and a quarter begin with prompts of up to 4 k tokens (116 k slots
// and positions, 1.5 MB), 4.4 us; a decode step of 4,096 sequences 6.7 us, of 65,535 151 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "pa_device.cuh"
#include "pa_ordered.cuh"
#include "pa_blocks.h"

namespace pa {
namespace {

__device__ unsigned int g_tables_errors;

constexpr int NTHREADS = 512;
constexpr int NWARPS = NTHREADS / 32;
constexpr uint32_t kMany = 1u << 30;  // the sums stop here; no legal one reaches it

struct Tables {
  int32_t* block_tables;
  const int32_t* old_lens;
  const int32_t* new_lens;
  int32_t* ring;
  const int32_t* state;
  int32_t* new_state;
  int64_t* slots;
  int32_t* positions;
  int32_t* starts;
  int max_blocks_per_seq, num_seqs, bs_log2, num_blocks, ring_size, max_new_tokens;
};

struct Count {  // blocks taken, blocks given back, tokens
  uint32_t pop, push, tok;
};
__device__ __forceinline__ Count operator+(Count a, Count b) {
  return Count{min(a.pop + b.pop, kMany), min(a.push + b.push, kMany), min(a.tok + b.tok, kMany)};
}

struct Seq {
  int have, want, old_len, new_len;
};
__device__ __forceinline__ Seq seq_of(const Tables& P, int b) {
  Seq s;
  s.old_len = P.old_lens[b];
  s.new_len = P.new_lens[b];
  const unsigned up = (1u << P.bs_log2) - 1u;
  s.have = int((unsigned(s.old_len) + up) >> P.bs_log2);
  s.want = int((unsigned(s.new_len) + up) >> P.bs_log2);
  return s;
}
__device__ __forceinline__ Count count_of(const Seq& s) {
  return Count{uint32_t(max(s.want - s.have, 0)), uint32_t(max(s.have - s.want, 0)),
               uint32_t(max(s.new_len - s.old_len, 0))};
}

struct Shared {
  uint32_t pop[NTHREADS], push[NTHREADS], tok[NTHREADS];  // before a thread's sequences
  Count warp_tot[NWARPS];
};

// The last entry of the ascending `a` that is at most x; a[0] = 0.
__device__ __forceinline__ int find(const uint32_t* a, uint32_t x) {
  int lo = 0;
#pragma unroll
  for (int step = NTHREADS / 2; step > 0; step >>= 1)
    if (a[lo + step] <= x) lo += step;
  return lo;
}

__global__ void __launch_bounds__(NTHREADS) update_tables_kernel(const Tables P) {
  __shared__ Shared sm;
  dev::griddep_enter();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int BS = 1 << P.bs_log2;
  const int per = (P.num_seqs + NTHREADS - 1) / NTHREADS;  // sequences of a thread
  const int b0 = min(P.num_seqs, tid * per), b1 = min(P.num_seqs, b0 + per);
  const int head = P.state[0], free_blocks = P.state[1];

  Count mine{0, 0, 0};
  bool bad = false;
  for (int b = b0; b < b1; ++b) {
    const Seq s = seq_of(P, b);
    bad |= s.old_len < 0 || s.new_len < 0 || s.have > P.max_blocks_per_seq ||
           s.want > P.max_blocks_per_seq;
    mine = mine + count_of(s);
  }
  Count inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Count y{__shfl_up_sync(0xffffffffu, inc.pop, o), __shfl_up_sync(0xffffffffu, inc.push, o),
                  __shfl_up_sync(0xffffffffu, inc.tok, o)};
    if (lane >= o) inc = inc + y;
  }
  if (lane == 31) sm.warp_tot[warp] = inc;
  bad = __syncthreads_or(bad);
  Count before{0, 0, 0}, all{0, 0, 0};
#pragma unroll
  for (int w = 0; w < NWARPS; ++w) {
    if (w == warp) before = all;
    all = all + sm.warp_tot[w];
  }
  // (sums that stopped at kMany leave a step that is refused below)
  sm.pop[tid] = before.pop + inc.pop - mine.pop;
  sm.push[tid] = before.push + inc.push - mine.push;
  sm.tok[tid] = before.tok + inc.tok - mine.tok;

  const bool state_ok = head >= 0 && head < P.ring_size && free_blocks >= 0 &&
                        free_blocks <= P.ring_size;
  const bool tokens_ok = all.tok < kMany && ((P.slots == nullptr && P.positions == nullptr) ||
                                             all.tok <= uint32_t(P.max_new_tokens));
  const bool enough = state_ok && all.pop <= uint32_t(free_blocks);
  const bool room = state_ok && uint32_t(free_blocks) + all.push <= uint32_t(P.ring_size);
  const bool lens_ok = !bad && tokens_ok;
  const bool ok = lens_ok && enough && room;
  const int first = blockIdx.x * NTHREADS + tid, stride = gridDim.x * NTHREADS;
  if (first == 0) {
    int h = head, n = free_blocks, lack = 0;
    if (ok) {
      h = int((uint32_t(head) + all.pop) % uint32_t(P.ring_size));
      n = free_blocks - int(all.pop) + int(all.push);
    } else {
      lack = lens_ok && state_ok && !enough ? int(all.pop) - free_blocks : -1;
      atomicOr(&g_tables_errors, lens_ok ? PA_DEVERR_POOL : PA_DEVERR_CONTEXT_LEN);
    }
    P.new_state[0] = h;
    P.new_state[1] = n;
    P.new_state[2] = lack;
    P.new_state[3] = 0;
  }
  __syncthreads();
  if (P.starts != nullptr) {
    // (a CTA writes the starts of its share of the threads' sequences)
    uint32_t at = sm.tok[tid];
    for (int b = b0; b < b1; ++b) {
      if (b % gridDim.x == blockIdx.x) P.starts[b] = ok ? int(at) : 0;
      at += count_of(seq_of(P, b)).tok;
    }
    if (first == 0) P.starts[P.num_seqs] = ok ? int(all.tok) : 0;
  }
  if (!ok) {
    for (int64_t i = first; i < P.max_new_tokens; i += stride) {
      if (P.slots != nullptr) P.slots[i] = -1;
      if (P.positions != nullptr) P.positions[i] = -1;
    }
    return;
  }

  bool bad_entry = false;
  auto checked = [&](int e) {
    const bool in = e >= 0 && e < P.num_blocks;
    bad_entry |= !in;
    return in ? e : -1;
  };
  auto ring_at = [&](uint32_t k) {  // k entries behind the head; k < 2 * ring_size
    uint32_t at = uint32_t(head) + k;  // (both below 2^30)
    return at >= uint32_t(P.ring_size) ? at - uint32_t(P.ring_size) : at;
  };
  // Sequence of item x in the sums `which` of the threads, and the counts before it.
  auto seek = [&](const uint32_t* sums, uint32_t Count::* which, uint32_t x, Count& c, Seq& s) {
    const int owner = find(sums, x);
    int b = owner * per;
    c = Count{sm.pop[owner], sm.push[owner], sm.tok[owner]};
    s = seq_of(P, b);
    for (Count n = count_of(s); x - c.*which >= n.*which; n = count_of(s)) {
      c = c + n;
      s = seq_of(P, ++b);
    }
    return b;
  };
  // fresh entries
  for (uint32_t x = first; x < all.pop; x += stride) {
    Count c;
    Seq s;
    const int b = seek(sm.pop, &Count::pop, x, c, s);
    P.block_tables[int64_t(b) * P.max_blocks_per_seq + s.have + (x - c.pop)] =
        checked(P.ring[ring_at(x)]);
  }
  // released ones
  for (uint32_t x = first; x < all.push; x += stride) {
    Count c;
    Seq s;
    const int b = seek(sm.push, &Count::push, x, c, s);
    P.ring[ring_at(uint32_t(free_blocks) + x)] =
        checked(P.block_tables[int64_t(b) * P.max_blocks_per_seq + s.want + (x - c.push)]);
  }
  // tokens, then the padding behind them
  if (P.slots != nullptr || P.positions != nullptr) {
    for (int64_t i = first; i < P.max_new_tokens; i += stride) {
      int64_t slot = -1;
      int pos = -1;
      if (i < int64_t(all.tok)) {
        Count c;
        Seq s;
        const int b = seek(sm.tok, &Count::tok, uint32_t(i), c, s);
        pos = s.old_len + int(uint32_t(i) - c.tok);
        if (P.slots != nullptr) {
          const int j = pos >> P.bs_log2;
          const int e = checked(j >= s.have
                                    ? P.ring[ring_at(c.pop + uint32_t(j - s.have))]
                                    : P.block_tables[int64_t(b) * P.max_blocks_per_seq + j]);
          slot = e < 0 ? -1 : (int64_t(e) << P.bs_log2) + (pos & (BS - 1));
        }
      }
      if (P.slots != nullptr) P.slots[i] = slot;
      if (P.positions != nullptr) P.positions[i] = pos;
    }
  }
  if (bad_entry) atomicOr(&g_tables_errors, PA_DEVERR_TABLE_ENTRY);
}

}  // namespace

int launch_update_tables(const pa_update_tables_params* p, int num_sms, void* stream) {
  Tables P;
  P.block_tables = p->block_tables;
  P.old_lens = p->old_lens;
  P.new_lens = p->new_lens;
  P.ring = p->free_ring;
  P.state = p->ring_state;
  P.new_state = p->new_ring_state;
  P.slots = p->slot_mapping;
  P.positions = p->positions;
  P.starts = p->token_starts;
  P.max_blocks_per_seq = p->max_blocks_per_seq;
  P.num_seqs = p->num_seqs;
  P.bs_log2 = log2_of(p->block_size);
  P.num_blocks = p->num_blocks;
  P.ring_size = p->ring_size;
  P.max_new_tokens = p->max_new_tokens;
  // One CTA for what one can write in two rounds; at most one an SM (every CTA adds up
  // all sequences).
  const int64_t items = int64_t(p->max_new_tokens) + p->num_seqs;
  int64_t grid = (items + 2 * NTHREADS - 1) / (2 * NTHREADS);
  if (grid > num_sms) grid = num_sms;
  if (grid < 1) grid = 1;
  return launch_ordered(update_tables_kernel, dim3(unsigned(grid)), NTHREADS, 0,
                        static_cast<cudaStream_t>(stream), 1, P);
}

int read_and_clear_tables_errors(uint32_t* flags) {
  unsigned int v = 0, zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_tables_errors, sizeof(v));
  if (e != cudaSuccess) return int(e);
  if (v != 0) e = cudaMemcpyToSymbol(g_tables_errors, &zero, sizeof(zero));
  *flags = v;
  return int(e);
}

}  // namespace pa
