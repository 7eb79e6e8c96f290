/*
 * pagedkv.h -- C ABI of libpagedkv.so: paged KV-cache decode attention for
 * GB300 (sm_103a), its companion cache kernels, and a host-side block pool.
 *
 * Sources for what each call computes:
 *  [P1] "How Paged Attention and Continuous Batching Actually Work"
 *       (netraruntime.com): §Paged attention: virtual memory for the KV cache
 *       (16-token blocks, free list, block table, the indexing rule: divide
 *       for the logical block, look up the physical block, multiply out, add
 *       the offset); §One step, end to end (write KV through the slot
 *       mapping, allocate_slots).
 *  [P2] "Paged Attention as a Memory Manager" (praveentn.live): §How the
 *       Kernel Executes Paged Attention (score_i = q.k_i / sqrt(d_k), the
 *       per-block loop: read the table entry, load the block, dot products,
 *       mask padding, running max and sum, weighted sum of V); §Prefix
 *       Caching and Copy-on-Write (refcounts; allocate, copy, decrement,
 *       update the table).
 *  [P3] PagedAttention architecture walk-through (aicassindra.com):
 *       §The architecture: every piece explained (entry i of the block table
 *       backs tokens [16i, 16i+15]; every 16th token takes a fresh block;
 *       a write to a shared block triggers copy-on-write).
 *  [P4] "PagedAttention and continuous batching" (ai-knowledge-tree):
 *       §Block table example; §Attention kernel modification (K/V loaded
 *       block by block through the table, running softmax across blocks).
 *
 * Data layout (the pages fix none; this library's choice):
 *   k_cache, v_cache  bf16 [num_blocks][num_kv_heads][block_size][head_dim]
 *                     (one (block, KV head) tile is block_size*head_dim*2
 *                     contiguous bytes: 4 KiB at block 16, head dim 128)
 *   q, out            bf16 [num_seqs][num_q_heads][head_dim]
 *   block_tables      int32 [num_seqs][max_blocks_per_seq]; entry j of row b
 *                     is the physical block of logical tokens
 *                     [j*block_size, (j+1)*block_size); entries past
 *                     ceil(len/block_size) are never read
 *   context_lens      int32 [num_seqs], the number of cached tokens of each
 *                     sequence including the one written this step
 *   slot_mapping      int64 [num_tokens]; slot = block*block_size + offset
 *   GQA               query head h reads KV head h / (num_q_heads/num_kv_heads)
 *
 * Conventions for every device call:
 *  - All array pointers are caller-owned DEVICE memory, 16-byte aligned,
 *    dense (no strides). The library never allocates device memory and never
 *    synchronises the stream (except pa_device_errors).
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and runs asynchronously.
 *  - Arguments are validated on the host before anything is launched; a
 *    failing check returns PA_ERR_INVALID_ARG or PA_ERR_UNSUPPORTED and
 *    launches nothing. A launch failure returns PA_ERR_CUDA.
 *  - Values that live only on the device (table entries, lengths, slots) are
 *    checked inside the kernels: an out-of-range value is never dereferenced
 *    (the access is clamped or skipped), a sticky device error bit is set,
 *    and the affected output is unspecified. pa_device_errors() reads the
 *    bits. No kernel faults or hangs on bad device-side values.
 *  - pa_last_error() returns a thread-local message for the last failing
 *    call on that thread.
 *
 * Supported shapes: block_size 8, 16 or 32 ("Paged Attention as a Memory
 * Manager", §PagedAttention: a compile-time constant, typically 8, 16 or 32);
 * head_dim 64 or 128; num_q_heads / num_kv_heads in {1, 2, 4, 8}. Both decode
 * kernels take every block size (the tensor-core kernel's 8-bit cache: head_dim
 * 128 and block size 16 or 32; the 8-bit cache at block size 8 decodes on the
 * CUDA-core kernel). Anything else returns PA_ERR_UNSUPPORTED.
 */
#ifndef PAGEDKV_H
#define PAGEDKV_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* pa_stream_t; /* same type as cudaStream_t */

typedef enum {
  PA_OK = 0,
  PA_ERR_INVALID_ARG = 1,  /* a host-checkable argument is wrong */
  PA_ERR_UNSUPPORTED = 2,  /* valid, but a shape this build does not implement */
  PA_ERR_OOM = 3,          /* block pool exhausted; pool state unchanged */
  PA_ERR_REFCOUNT = 4,     /* refcount underflow / block not allocated */
  PA_ERR_BOUNDS = 5,       /* an id or index out of range */
  PA_ERR_CUDA = 6          /* a CUDA runtime call or launch failed */
} pa_status;

/* Device error bits reported by pa_device_errors(). */
#define PA_DEVERR_TABLE_ENTRY 0x1u   /* block table entry outside [0, num_blocks) */
#define PA_DEVERR_CONTEXT_LEN 0x2u   /* context_len > max_context_len or > table capacity */
#define PA_DEVERR_SLOT 0x4u          /* slot_mapping entry >= num_blocks*block_size */
#define PA_DEVERR_COPY_PAIR 0x8u     /* copy_blocks pair outside [0, num_blocks) */
#define PA_DEVERR_TIMEOUT 0x10u      /* an mbarrier wait hit its iteration limit */
#define PA_DEVERR_APPEND_SLOT 0x20u  /* pa_append_decode: a slot_mapping entry is not the slot
                                        of its token (context_lens[b]-1 for one new token per
                                        sequence); that token is not written */
#define PA_DEVERR_KEEP 0x40u         /* pa_evict_compact: a keep entry that does not ascend or is
                                        past the source table (that row is not moved), or past the
                                        token weights (that weight becomes 0);
                                        pa_decode_selected: a selected entry past the sequence's
                                        blocks (it is skipped) */
#define PA_DEVERR_POOL 0x80u         /* pa_update_tables: too few free blocks, or no room in the
                                        ring for the released ones; nothing is done */

const char* pa_status_string(pa_status s);
const char* pa_last_error(void);
int32_t pa_version(void);

/* Sticky device error bits accumulated by every kernel of this library on the
 * current device since the last call. Synchronises `stream`, returns the bits
 * in *flags and clears them. */
pa_status pa_device_errors(pa_stream_t stream, uint32_t* flags);

/* ------------------------------------------------------------------------
 * pa_decode -- paged decode attention [P2 §How the Kernel Executes Paged
 * Attention; P4 §Attention kernel modification].
 *
 * For every sequence b and query head h (KV head g = h / G):
 *   K_b, V_b = rows t = 0..L_b-1 of the cache, row t read from physical block
 *              block_tables[b][t / block_size] at offset t % block_size [P1]
 *   s_t      = scale * (q[b][h] . K_b[t])
 *   out[b][h]= sum_t softmax(s)_t * V_b[t]                (bf16, round to nearest even)
 * computed with fp32 accumulation and a running (online) softmax. Sequences
 * longer than `partition_tokens` are split into partitions of that many
 * tokens; each partition yields (max, sum, weighted sum) and a second kernel
 * merges them by log-sum-exp (flash-decoding split; not on the pages).
 * Rows with L_b <= 0 are written as zeros.
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* q;               /* bf16 [num_seqs][num_q_heads][head_dim] */
  void* out;                   /* bf16 [num_seqs][num_q_heads][head_dim] */
  const void* k_cache;         /* bf16 [num_blocks][num_kv_heads][block_size][head_dim] */
  const void* v_cache;         /* same layout as k_cache */
  const int32_t* block_tables; /* int32 [num_seqs][max_blocks_per_seq] */
  const int32_t* context_lens; /* int32 [num_seqs] */
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t block_size;
  int32_t num_blocks;
  int32_t max_context_len;     /* host-known upper bound of every context_lens[b] (>= 1) */
  float scale;                 /* softmax scale, normally 1/sqrt(head_dim) */
  int32_t partition_tokens;    /* split-K partition length; 0 = 512; else a multiple of 16 in
                                  [16, 4096], and on the CUDA-core kernel of block_size too (the
                                  4-bit cache: checked like that, not used) */
  int32_t variant;             /* PA_DECODE_TENSOR_CORE (default) or PA_DECODE_CUDA_CORE */
  int32_t overlap_prologue;    /* nonzero: context_lens and block_tables were final before the
                                  previous kernel on `stream` began (e.g. uploaded once per step),
                                  so the tensor-core kernel may read them -- and plan its work --
                                  while that kernel still runs (programmatic dependent launch).
                                  q, the caches and every output are read or written only after
                                  the previous kernel has completed; before that the kernel only
                                  prefetches its first cache blocks into L2, which cannot change
                                  any result even if that kernel writes them. 0 = plain stream
                                  order. */
  int32_t kv_dtype;            /* PA_KV_BF16 (0, default), PA_KV_FP8_E4M3 (1) or PA_KV_FP4_E2M1
                                  (2) */
  const float* k_scale;        /* the 8-bit and 4-bit caches only: device float [num_kv_heads], the
                                  dequantisation scale of each KV head's K (8-bit: value = code *
                                  scale) */
  const float* v_scale;        /* the same for V */
  int32_t query_len;           /* new tokens per sequence: 0 or 1 = one (the layouts above).
                                  Q > 1 ("How Paged Attention and Continuous Batching Actually
                                  Work", §Continuous batching: several scheduled tokens of one
                                  request, as in a chunked prefill): q and out are
                                  [num_seqs][Q][num_q_heads][head_dim], the new tokens are the
                                  last Q of each sequence's context_lens[b] (already in the cache),
                                  and query token i attends to the first context_lens[b] - Q + i + 1
                                  of them (causal among the new tokens). On the tensor-core
                                  variant with the bf16 cache, head_dim 128, block size 16 or 32
                                  and G in {1, 2, 4, 8}, a query-major kernel takes the new tokens
                                  when they are more than one column group holds (below), or
                                  when Q * G >= 16 and num_seqs * num_kv_heads * ceil(Q * G /
                                  128) >= 128: the query rows of one or two KV heads share each
                                  load of their keys; batches with fewer than 256 such units
                                  split each unit's keys over CTAs and merge the partials
                                  (workspace: pa_decode_workspace_size). Otherwise the
                                  tensor-core kernel's MMAs take the query tokens in column
                                  groups: G * Qp <= 16 columns per KV head (8 at block size 8,
                                  Qp = the group's tokens rounded up to a power of two) and
                                  num_kv_heads * G * Qp <= 128 (64 for the 8-bit cache); a
                                  sequence with more new tokens is decoded as several groups,
                                  each streaming the keys its last token sees, with num_seqs *
                                  groups <= 16384. Shapes beyond that (or with num_kv_heads
                                  other than 1, 2, 4 and 8), and the CUDA-core variant, need
                                  num_seqs * Q <= 65535 (else PA_ERR_UNSUPPORTED), also where
                                  the query-major kernel takes them; off that kernel they decode
                                  each (sequence, token) on its own. A sequence
                                  with 0 < context_lens[b] < Q gets zero rows and
                                  PA_DEVERR_CONTEXT_LEN. */
  int32_t wait_timeout_us;     /* tensor-core kernel: the longest one of its barrier waits may
                                  take, in microseconds; 0 = 2 s. A wait that runs out sets
                                  PA_DEVERR_TIMEOUT, and every CTA that saw it stops, lets the
                                  copies it has in flight land, frees its tensor memory and
                                  exits: the outputs are then unspecified, the context stays
                                  usable. A budget far below a launch's normal waits makes a
                                  well-formed launch run out (what the tests do to exercise that
                                  exit). Must be >= 0. */
} pa_decode_params;

/* Decode kernel variants; both compute the same function. The tensor-core
 * kernel handles num_kv_heads in {1, 2, 4, 8}, num_q_heads <= 64 and up to
 * 16384 sequences per call; other shapes run on the CUDA-core kernel
 * whatever `variant` says. */
/* Cache element types. PA_KV_FP8_E4M3 -- the 8-bit KV cache ("PagedAttention"
 * glossary page, §What paging costs: 8-bit KV quantisation halves the bytes per
 * block; the format is this library's reading): OCP E4M3 codes (uint8) with one
 * dequantisation scale per KV head for K and for V.
 *   k_cache  uint8 [num_blocks][num_kv_heads][block_size][head_dim]
 *   v_cache  uint8 [num_blocks][num_kv_heads][block_size/W][head_dim][W],
 *            W = min(block_size, 16) (V^T of each (block, head) tile in
 *            sub-tiles of W keys)
 * Written by pa_reshape_and_cache_fp8, copied by pa_copy_blocks_fp8. The decode
 * computes on the tensor cores (variant PA_DECODE_TENSOR_CORE, head_dim 128 and
 * the rest of the tensor-core shape rules) with the queries and the softmax
 * weights each split into two E4M3 terms, or on CUDA cores (variant
 * PA_DECODE_CUDA_CORE and shapes the tensor-core kernel does not take: head_dim
 * 64, block size 8) with the codes dequantised in fp32; either result is
 * within the bf16 tolerance of the exact decode over the dequantised cache.
 * Other shapes return PA_ERR_UNSUPPORTED. */
#define PA_KV_BF16 0
#define PA_KV_FP8_E4M3 1
/* PA_KV_FP4_E2M1 -- the 4-bit KV cache (same page and section; the format is
 * this library's): E2M1 codes with an E4M3 scale for every 16 elements of a row
 * and one float scale per KV head, 9/16 byte an element:
 *   value = code * group scale * scale[h]
 *   k_cache, v_cache  uint8 [num_blocks][num_kv_heads][tile], tile =
 *            block_size * head_dim * 9 / 16 bytes: the codes of the block's
 *            rows [block_size][head_dim / 2] (element 2i in the low nibble of
 *            byte i), then their scales [block_size][head_dim / 16]
 * Written by pa_reshape_and_cache_fp4, read back by pa_gather_fp4, copied by
 * pa_copy_blocks_fp4. One kernel decodes it whatever `variant` says: head_dim
 * 64 or 128, every block size, G in {1, 2, 4, 8}, any number of KV heads,
 * num_seqs * query_len <= 65535 and num_seqs * ceil(query_len / (8 / G)) *
 * num_kv_heads * (max_context_len / 32 + 9) < 2^31, max_context_len <= 2^31 - 64
 * (else PA_ERR_UNSUPPORTED; max_context_len here no more than the table holds).
 * The codes are multiplied exactly; the softmax weights are rounded to f16, by at
 * most 2^-11 of their value or 2^-32 of the row's largest. With several new
 * tokens, up to 8 / G of them share each load of the keys. overlap_prologue and
 * wait_timeout_us are accepted and not used (the kernel waits on no barrier of
 * its own). */
#define PA_KV_FP4_E2M1 2

#define PA_DECODE_TENSOR_CORE 0 /* tcgen05 MMAs, TMEM accumulators, tensor-map TMA ring */
#define PA_DECODE_CUDA_CORE 1   /* fp32 FMAs on CUDA cores, 1-D bulk-copy rings */

/* Bytes of device workspace pa_decode needs for these parameters on the
 * current device: a 256-byte header, then what the kernel these parameters
 * select needs -- the tensor-core kernel's work plan and per-(sequence + SM)
 * partials of every query column (variant PA_DECODE_TENSOR_CORE on a shape it
 * handles), else the CUDA-core kernel's per-partition partials (none when no
 * sequence can split). Returns 0 for invalid params. */
size_t pa_decode_workspace_size(const pa_decode_params* p);

/* Enqueue the decode. `workspace` is caller-owned device memory of at least
 * pa_decode_workspace_size(p) bytes, 256-byte aligned. Every call writes what
 * it later reads there, so its contents on entry do not matter; two calls in
 * flight at once must not share it. */
pa_status pa_decode(const pa_decode_params* p, void* workspace, size_t workspace_bytes,
                    pa_stream_t stream);

/* ------------------------------------------------------------------------
 * pa_decode_noalloc -- the same decode as pa_decode, for callers that cannot
 * allocate device memory at decode time. The pages have no counterpart: it
 * exists because an engine that hands all free HBM to its KV block pool at
 * start-up has nothing left for a workspace, and a serving loop cannot take
 * cudaMalloc's implicit device synchronisation.
 *
 * The split-K partials go to a fixed device array inside the library
 * (PA_NOALLOC_SCRATCH_BYTES, held on every GPU that loads the library until
 * the process exits). Nothing is allocated or freed by the call.
 *  - Shapes whose workspace (pa_decode_workspace_size, which sizes the
 *    kernel the parameters select) exceeds that are rejected with
 *    PA_ERR_INVALID_ARG.
 *  - The first call in each CUDA context looks up the array's device address
 *    with that context's device current; make that first call before any
 *    stream capture. A device reset (cudaDeviceReset) or another context on
 *    the same device is a new context, and its first call looks the address
 *    up again.
 *  - Every call on a device shares the one array and leaves its partials in
 *    it. Calls whose kernels overlap on the GPU (different streams, no
 *    ordering between them) race on it and give unspecified results.
 * ---------------------------------------------------------------------- */
#define PA_NOALLOC_SCRATCH_BYTES (16u << 20) /* 16 MiB */
pa_status pa_decode_noalloc(const pa_decode_params* p, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * pa_reshape_and_cache -- write each new token's K/V row into its slot
 * [P1 §One step, end to end: "gather and write KV through the slot-mapping
 * formula"; P3 §The architecture: the forward pass appends the new token's
 * K/V into the right physical block].
 *   for t in [0, num_tokens): slot = slot_mapping[t]; if slot < 0: skip
 *     k_cache[slot / block_size][h][slot % block_size][:] = k_new[t][h][:]  (every KV head h)
 *     v_cache[...]                                         = v_new[t][h][:]
 * Bit-exact copies. k_new/v_new: bf16 [num_tokens][num_kv_heads][head_dim].
 * Two tokens with the same slot race (unspecified which one lands).
 * ---------------------------------------------------------------------- */
pa_status pa_reshape_and_cache(const void* k_new, const void* v_new, void* k_cache,
                               void* v_cache, const int64_t* slot_mapping, int32_t num_tokens,
                               int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                               int32_t num_blocks, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * pa_append_decode -- one decode step's KV write and attention in one
 * launch: the effect of
 *   pa_reshape_and_cache(a->k_new, a->v_new, k_cache, v_cache,
 *                        a->slot_mapping, num_seqs, ...)
 *   pa_decode(p, ...)
 * [P1 §One step, end to end: the forward pass writes the new token's KV
 * through the slot mapping, then attention reads the paged cache].
 * Token b is sequence b's new token: k_new/v_new are bf16
 * [num_seqs][num_kv_heads][head_dim], slot_mapping is int64 [num_seqs], and
 * p->context_lens already counts the new token. The write of sequence b is
 * done by the part of the decode that reads b's last block, just before that
 * block is loaded, so
 *  - slot_mapping[b] must be the slot of token context_lens[b]-1 of b, i.e.
 *    block_tables[b][(L-1)/16]*16 + (L-1)%16. Any other non-negative value
 *    sets PA_DEVERR_APPEND_SLOT and is not written; a negative value writes
 *    nothing (padding); sequences of length 0 write nothing.
 *  - the written block must not be read by another sequence of the batch,
 *    which copy-on-write guarantees (a shared block is copied before a write).
 *  - with query_len Q > 1 every sequence brings Q new tokens (rows b*Q + i of
 *    k_new/v_new/slot_mapping, token L-Q+i); each is written by the part of
 *    the decode that reads its block, with the same slot rule.
 * a->k_cache / a->v_cache must equal p->k_cache / p->v_cache (the caches are
 * written through these). With the 8-bit cache (p->kv_dtype PA_KV_FP8_E4M3)
 * the write is that of pa_reshape_and_cache_fp8 with p->k_scale / p->v_scale
 * (bit-identical codes), with the 4-bit cache that of pa_reshape_and_cache_fp4,
 * in a launch of its own. Same workspace as pa_decode. The CUDA-core variant
 * and shapes the tensor-core kernel does not cover run the KV-write kernel
 * and then the decode, with the same result.
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* k_new;            /* bf16 [num_seqs * Q][num_kv_heads][head_dim], 16-byte aligned
                                   (Q = the decode's query_len, at least 1); row b * Q + i is
                                   token context_lens[b] - Q + i of sequence b */
  const void* v_new;            /* same */
  const int64_t* slot_mapping;  /* int64 [num_seqs * Q], the slots of those tokens */
  void* k_cache;                /* == p->k_cache, written */
  void* v_cache;                /* == p->v_cache, written */
} pa_append_params;
pa_status pa_append_decode(const pa_decode_params* p, const pa_append_params* a, void* workspace,
                           size_t workspace_bytes, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * pa_step_host -- one whole decode step driven from host memory, for a host
 * that builds each step's batch (the scheduler of [P1 §One step, end to
 * end]) and reads the result back: copy-on-write copies, the KV write of
 * one new token per sequence and paged decode attention, with the inputs
 * taken from one packed host buffer and the output returned to host memory.
 *
 * The call enqueues on `stream`
 *   1. the staging of the packed inputs into the workspace,
 *   2. pa_copy_blocks (pa_copy_blocks_fp8 for the 8-bit cache; if
 *      num_cow_pairs > 0), then pa_append_decode on the staged inputs and the
 *      device-resident caches (bf16, or 8-bit with kv_dtype and the scales),
 *   3. the return of the output to host_out,
 * and synchronises the stream before it returns (the output is in host_out).
 * Pinned host memory (page-locked through CUDA, hence mapped under unified
 * addressing) that is 16-byte aligned is read and written by the kernels
 * themselves over the host link (NVLink-C2C on a Grace-Blackwell part): a
 * staging kernel copies host_in into the workspace, the tensor-core decode
 * reads the lengths and tables in host_in to plan its work while that kernel
 * runs, and the decode writes its output rows straight into host_out. Any
 * other host memory goes through one DMA copy each way (cudaMemcpyAsync).
 * The bytes moved are the same. host_in must not change until the call
 * returns.
 *
 * Packed input (host memory; pinned memory lets the copy run at full speed):
 * sections at the byte offsets pa_step_host_layout reports, each 256-byte
 * aligned, in this order:
 *   q             bf16  [num_seqs][num_q_heads][head_dim]     (x Q: see query_len)
 *   k_new, v_new  bf16  [num_seqs][num_kv_heads][head_dim]    (x Q)
 *   slot_mapping  int64 [num_seqs]          (x Q; rules of pa_append_decode)
 *   block_tables  int32 [num_seqs][max_blocks_per_seq]
 *   context_lens  int32 [num_seqs]          (counting the new token)
 *   cow_pairs     int32 [num_cow_pairs][2]  (rules of pa_copy_blocks)
 * host_out: bf16 [num_seqs][num_q_heads][head_dim], host memory.
 * The workspace (device memory, 256-byte aligned, at least
 * pa_step_host_workspace_size bytes) holds the staged inputs, the staged
 * output and the decode workspace; nothing in it needs initialising.
 * Errors: host-checkable arguments as pa_decode (no copy is issued);
 * PA_ERR_CUDA when a copy, a launch or the synchronisation fails.
 * ---------------------------------------------------------------------- */
typedef struct {
  uint64_t q, k_new, v_new, slot_mapping, block_tables, context_lens, cow_pairs;
  uint64_t total;  /* bytes of the whole packed input */
} pa_step_layout;

typedef struct {
  const void* host_in;        /* packed inputs (see above) */
  void* host_out;             /* bf16 [num_seqs][num_q_heads][head_dim] */
  void* k_cache;              /* device caches, layout of pa_decode; written */
  void* v_cache;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t block_size;
  int32_t num_blocks;
  int32_t max_blocks_per_seq;
  int32_t max_context_len;    /* host-known upper bound of every context length */
  int32_t num_cow_pairs;
  float scale;
  int32_t variant;            /* PA_DECODE_TENSOR_CORE or PA_DECODE_CUDA_CORE */
  int32_t kv_dtype;           /* PA_KV_BF16 (0), PA_KV_FP8_E4M3 or PA_KV_FP4_E2M1: the caches as
                                 in pa_decode; the 8-bit cache takes the tensor-core variant, the
                                 quantising KV write and pa_copy_blocks_fp8, the 4-bit cache its
                                 own decode, write and pa_copy_blocks_fp4 */
  const float* k_scale;       /* the 8-bit and 4-bit caches only: device float [num_kv_heads], as
                                 in pa_decode_params */
  const float* v_scale;
  int32_t query_len;          /* new tokens per sequence, Q (0 or 1 = one): q and host_out hold
                                 [num_seqs][Q][num_q_heads][head_dim], k_new / v_new
                                 [num_seqs * Q][num_kv_heads][head_dim], slot_mapping
                                 [num_seqs * Q]; row b * Q + i is token context_lens[b] - Q + i
                                 (as in pa_append_decode) */
} pa_step_host_params;

pa_status pa_step_host_layout(const pa_step_host_params* p, pa_step_layout* out);
size_t pa_step_host_workspace_size(const pa_step_host_params* p); /* 0 if p is invalid */
pa_status pa_step_host(const pa_step_host_params* p, void* workspace, size_t workspace_bytes,
                       pa_stream_t stream);

/* ------------------------------------------------------------------------
 * pa_reshape_and_cache_fp8 -- the KV write into an 8-bit (PA_KV_FP8_E4M3)
 * cache: for token t and KV head h,
 *   code = E4M3(float32(x) / scale[h])   (round to nearest even; finite values
 *                                         beyond +-448 saturate)
 * K codes go to row (slot / block_size, h, slot % block_size); the V code of
 * offset o = slot % block_size, element d, to byte d*16 + o%16 of sub-tile
 * o/16 of the (block, h) tile. k_scale, v_scale: device float
 * [num_kv_heads]. Otherwise as pa_reshape_and_cache (negative slots skipped,
 * out-of-range slots set PA_DEVERR_SLOT). head_dim a multiple of 8; block_size
 * 16 or 32.
 * ---------------------------------------------------------------------- */
pa_status pa_reshape_and_cache_fp8(const void* k_new, const void* v_new, void* k_cache,
                                   void* v_cache, const int64_t* slot_mapping,
                                   const float* k_scale, const float* v_scale,
                                   int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                                   int32_t block_size, int32_t num_blocks, pa_stream_t stream);

/* pa_copy_blocks for an 8-bit cache: the same whole-block copy of both caches
 * (block_size * head_dim bytes per KV head); block_size 16 or 32. */
pa_status pa_copy_blocks_fp8(void* k_cache, void* v_cache, const int32_t* pairs,
                             int32_t num_pairs, int32_t num_kv_heads, int32_t head_dim,
                             int32_t block_size, int32_t num_blocks, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * pa_reshape_and_cache_fp4 -- the KV write into a 4-bit (PA_KV_FP4_E2M1)
 * cache. For token t, KV head h and every group of 16 elements of its row,
 * with a the group's largest magnitude and fl() rounding to float:
 *   group scale = E4M3(fl(a / fl(6 * scale[h])))   nearest even, at most 448
 *   step        = fl(group scale * scale[h])
 *   code        = E2M1(fl(x / step))               nearest even, at most +-6
 * A group whose scale rounds to zero is stored as (signed) zeros; an infinity
 * saturates; a group that holds a NaN gets the E4M3 NaN as its scale, so all
 * 16 elements read back as NaN. k_scale, v_scale: device float [num_kv_heads],
 * each in [2^-60, 2^60] (others: unspecified codes). head_dim 64 or 128;
 * block_size 8, 16 or 32. Otherwise as pa_reshape_and_cache (negative slots
 * skipped, out-of-range slots set PA_DEVERR_SLOT; two tokens with the same slot
 * race, and may leave codes of one with scales of the other).
 * ---------------------------------------------------------------------- */
pa_status pa_reshape_and_cache_fp4(const void* k_new, const void* v_new, void* k_cache,
                                   void* v_cache, const int64_t* slot_mapping,
                                   const float* k_scale, const float* v_scale,
                                   int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                                   int32_t block_size, int32_t num_blocks, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * pa_gather_fp4 -- rows of a 4-bit cache read back, for a caller that moves a
 * sequence to a bf16 cache or feeds cached rows to another kernel: row t of
 * k_out / v_out (bf16 [num_tokens][num_kv_heads][head_dim]) is the row at
 * slot_mapping[t], each element fl(code * group scale * scale[h]) rounded to
 * bf16. A negative slot gives a row of zeros; an out-of-range slot does too,
 * and sets PA_DEVERR_SLOT. A slot may occur any number of times.
 * ---------------------------------------------------------------------- */
pa_status pa_gather_fp4(const void* k_cache, const void* v_cache, void* k_out, void* v_out,
                        const int64_t* slot_mapping, const float* k_scale, const float* v_scale,
                        int32_t num_tokens, int32_t num_kv_heads, int32_t head_dim,
                        int32_t block_size, int32_t num_blocks, pa_stream_t stream);

/* pa_copy_blocks for a 4-bit cache: the same whole-block copy of both caches
 * (block_size * head_dim * 9 / 16 bytes per KV head); head_dim 64 or 128,
 * block_size 8, 16 or 32. */
pa_status pa_copy_blocks_fp4(void* k_cache, void* v_cache, const int32_t* pairs,
                             int32_t num_pairs, int32_t num_kv_heads, int32_t head_dim,
                             int32_t block_size, int32_t num_blocks, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * pa_copy_blocks -- the data half of copy-on-write [P2 §Prefix Caching and
 * Copy-on-Write: "allocates a fresh physical block, copies the existing
 * content"]. For each pair i: block pairs[i][1] of both caches becomes a
 * bit-exact copy of block pairs[i][0] (all KV heads, all slots).
 * pairs: int32 [num_pairs][2] (src, dst), device memory. Destinations must
 * be pairwise distinct and disjoint from the sources (what the pool's
 * copy-on-write produces); overlapping pairs give unspecified contents.
 * ---------------------------------------------------------------------- */
pa_status pa_copy_blocks(void* k_cache, void* v_cache, const int32_t* pairs, int32_t num_pairs,
                         int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                         int32_t num_blocks, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * Eviction: fewer cached tokens instead of smaller ones. The pages leave open
 * which tokens a cache under pressure gives up; here the most recent ones
 * stay, and of the others those that attention has looked at most. A step is
 *   pa_token_weights   what this step's queries look at, accumulated
 *   pa_evict_select    the tokens to keep under a budget
 *   pa_pool_compact    (host pool) the blocks that hold them
 *   pa_evict_compact   their rows moved there
 * after which the sequence is an ordinary one of new_lens[b] tokens: its next
 * token is appended behind them (keys keep the position encoding that they
 * were written with).
 *
 * pa_token_weights -- for every sequence b and cached token t
 *   token_weights[b][t] (+)= sum over new tokens i and query heads h of
 *                            softmax(scale * q[b][i][h] . K_b)_t
 * over the keys that new token i sees (the causal rule of pa_decode). fp32;
 * summed in a fixed order. Entries t >= context_lens[b] are left as they were,
 * and so is the whole row of a sequence of length 0 or with fewer keys than
 * new tokens (the latter sets PA_DEVERR_CONTEXT_LEN). Reads K only, of any of
 * the three caches, at every block size. num_seqs * ceil(query_len / (16 / G))
 * <= 65535 (else PA_ERR_UNSUPPORTED); table rows hold up to 2^30 tokens, here
 * and below.
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* q;               /* bf16 [num_seqs][query_len][num_q_heads][head_dim] */
  const void* k_cache;         /* as in pa_decode_params, of type kv_dtype */
  const int32_t* block_tables; /* int32 [num_seqs][max_blocks_per_seq] */
  const int32_t* context_lens; /* int32 [num_seqs], the new tokens included */
  float* token_weights;        /* float [num_seqs][weights_stride], written */
  int32_t weights_stride;      /* >= min(max_context_len, max_blocks_per_seq * block_size) */
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t block_size;
  int32_t num_blocks;
  int32_t max_context_len;     /* host-known upper bound of every context_lens[b] (>= 1) */
  float scale;
  int32_t kv_dtype;            /* PA_KV_BF16, PA_KV_FP8_E4M3 or PA_KV_FP4_E2M1 */
  const float* k_scale;        /* the 8-bit and 4-bit caches only: float [num_kv_heads] */
  int32_t query_len;           /* new tokens per sequence (0 or 1 = one), up to 1024 */
  int32_t accumulate;          /* nonzero: add to token_weights; 0: overwrite entries
                                  [0, context_lens[b]) */
} pa_token_weights_params;

/* The scores of every (new token, query head) pass through the workspace:
 * 4 * num_seqs * query_len * num_q_heads * max_context_len bytes and a little
 * more. Caller-owned, 256-byte aligned, contents on entry do not matter; two
 * calls in flight at once must not share it. 0 if the params are invalid. */
size_t pa_token_weights_workspace_size(const pa_token_weights_params* p);
pa_status pa_token_weights(const pa_token_weights_params* p, void* workspace,
                           size_t workspace_bytes, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * pa_evict_select -- the tokens each sequence keeps: all of them if it has at
 * most `budget`, else its last `recent` ones and, of the others, the budget -
 * recent with the largest token_weights (ties: the lower index; +0 and -0 are
 * equal, a NaN ranks below every number).
 *   keep      int32 [num_seqs][budget]: their indices, ascending; -1 behind
 *   new_lens  int32 [num_seqs]: min(context_lens[b], budget); not context_lens
 *             itself nor overlapping it (PA_ERR_INVALID_ARG)
 * token_weights: float [num_seqs][weights_stride]; a length beyond
 * weights_stride is cut to it and sets PA_DEVERR_CONTEXT_LEN. num_seqs up to
 * 65535, weights_stride and budget in [1, 2^30], recent in [0, budget]. No
 * workspace.
 * ---------------------------------------------------------------------- */
pa_status pa_evict_select(const float* token_weights, const int32_t* context_lens, int32_t* keep,
                          int32_t* new_lens, int32_t num_seqs, int32_t weights_stride,
                          int32_t budget, int32_t recent, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * pa_evict_compact -- the move: for every sequence b and j < new_lens[b], the
 * K and V rows of token keep[b][j] (through block_tables) become those of
 * token j (through dst_tables), bit for bit, for every KV head.
 *  - dst_tables may be block_tables itself (in place), or name other blocks
 *    at some indices: entry j must be a block that none of the call's source
 *    tables holds, or the source's own entry j, held by no other sequence of
 *    the call unless every row of the block stays where it is; no two
 *    sequences may write the same block. pa_pool_compact produces such tables.
 *    Rows that already are where they belong are not touched.
 *  - keep must ascend strictly (what pa_evict_select produces); an entry below
 *    its own index or past the source table is not moved and sets
 *    PA_DEVERR_KEEP.
 *  - new_lens beyond keep_stride or the destination table is cut and sets
 *    PA_DEVERR_CONTEXT_LEN; a table entry outside [0, num_blocks) moves nothing
 *    and sets PA_DEVERR_TABLE_ENTRY.
 *  - token_weights, if not NULL, is compacted the same way in place (a weight
 *    stays where its row is not moved; one of a token at or beyond weights_stride
 *    becomes 0 and sets PA_DEVERR_KEEP), and its rows are zeroed from new_lens[b]
 *    on. Other rows behind the kept tokens are left as they were.
 * ---------------------------------------------------------------------- */
typedef struct {
  void* k_cache;               /* of type kv_dtype, as in pa_decode_params; written */
  void* v_cache;
  const int32_t* block_tables; /* int32 [num_seqs][max_blocks_per_seq] */
  const int32_t* dst_tables;   /* int32 [num_seqs][max_dst_blocks_per_seq] */
  const int32_t* keep;         /* int32 [num_seqs][keep_stride] */
  const int32_t* new_lens;     /* int32 [num_seqs] */
  float* token_weights;        /* float [num_seqs][weights_stride] or NULL */
  int32_t weights_stride;
  int32_t max_blocks_per_seq;
  int32_t max_dst_blocks_per_seq;
  int32_t keep_stride;         /* the budget given to pa_evict_select */
  int32_t num_seqs;
  int32_t num_kv_heads;
  int32_t head_dim;            /* 64 or 128 */
  int32_t block_size;          /* 8, 16 or 32 */
  int32_t num_blocks;
  int32_t kv_dtype;
} pa_evict_compact_params;
pa_status pa_evict_compact(const pa_evict_compact_params* p, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * Tables on the device: what pa_seq_append_tokens and pa_seq_free do for a batch on
 * the host ([P1 §One step, end to end: allocate_slots]), where the lengths are on the
 * device -- after pa_evict_select, or in a captured loop.
 *
 * Free blocks are a ring in device memory: of free_ring [ring_size] the `count` entries
 * from `head` on (wrapping around) are free block ids; ring_state is {head, count, 0, 0}.
 * Row b of block_tables holds blocks for old_lens[b] tokens and gets them for
 * new_lens[b], with have = ceil(old_lens[b] / block_size), want = ceil(new_lens[b] /
 * block_size), sequence after sequence:
 *  - want > have: entries [have, want) become the next blocks from the ring's head;
 *  - want < have: the blocks of entries [want, have) go to the ring's tail, in order
 *    (they can be handed out from the next call on). The entries themselves are left as
 *    they were: entries past a sequence's length are never read.
 * The rows of tokens old_lens[b] <= t < new_lens[b], packed sequence after sequence:
 *  - slot_mapping: block * block_size + offset, what pa_reshape_and_cache takes;
 *  - positions: t;
 *  - token_starts[b]: the first row of sequence b; token_starts[num_seqs] the number of
 *    rows. Rows from there to max_new_tokens get slot and position -1 (padding, which
 *    the KV writes skip).
 * Blocks of a row must be its own: the ring knows no reference counts, so a released
 * block that another row shares would be handed out while that row reads it. A ring may
 * be filled with blocks that a pa_pool has handed out (pa_pool_alloc).
 * All or nothing: if the blocks do not suffice (PA_DEVERR_POOL), if a length is negative
 * or past the table row, or if there are more than max_new_tokens tokens
 * (PA_DEVERR_CONTEXT_LEN), tables and ring stay as they are, slots and positions are -1
 * and token_starts 0. new_ring_state is {head, count, short, 0}: short is 0 when the step
 * was done, the number of missing blocks when they did not suffice, else -1.
 * A ring entry or a released entry outside [0, num_blocks) sets PA_DEVERR_TABLE_ENTRY
 * and is passed on as -1; so is an old entry that a new token's slot needs (that slot
 * is -1).
 * Lengths and state are read while outputs are written: no output may overlap them
 * (PA_ERR_INVALID_ARG). A call may be repeated with the same arguments as long as the
 * tables' old entries are unchanged: it gives the same result. num_seqs up to 65535;
 * ring_size, max_new_tokens and the tokens of a table row below 2^30.
 * ---------------------------------------------------------------------- */
typedef struct {
  int32_t* block_tables;       /* int32 [num_seqs][max_blocks_per_seq], updated */
  const int32_t* old_lens;     /* int32 [num_seqs], tokens that the rows hold blocks for */
  const int32_t* new_lens;     /* int32 [num_seqs], tokens that they shall hold blocks for */
  int32_t* free_ring;          /* int32 [ring_size], updated */
  const int32_t* ring_state;   /* int32 [4]: head, count; the others are not read */
  int32_t* new_ring_state;     /* int32 [4], written */
  int64_t* slot_mapping;       /* int64 [max_new_tokens] or NULL */
  int32_t* positions;          /* int32 [max_new_tokens] or NULL */
  int32_t* token_starts;       /* int32 [num_seqs + 1] or NULL */
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t block_size;          /* 8, 16 or 32 */
  int32_t num_blocks;          /* of the cache */
  int32_t ring_size;           /* at least the blocks that the ring ever holds */
  int32_t max_new_tokens;      /* rows of slot_mapping and positions; 0 if both are NULL (then
                                  any number of new tokens is taken) */
} pa_update_tables_params;
pa_status pa_update_tables(const pa_update_tables_params* p, pa_stream_t stream);

/* ------------------------------------------------------------------------
 * Attention over selected blocks. The pages read the whole context for every token; a
 * long one mostly holds blocks that a query gives no weight to. A step is
 *   pa_block_bounds    the bounds of the keys of the blocks that it wrote
 *   pa_block_scores    how high a key of each block can score
 *   pa_block_select    the blocks to read under a budget
 *   pa_decode_selected the attention over them
 * with a list of blocks per sequence and KV head. Every cache type, block size, head_dim
 * 64 or 128, G in {1, 2, 4, 8}; table rows of up to 2^30 tokens.
 *
 * pa_block_bounds -- for every block that holds a token t with old_lens[b] <= t <
 * context_lens[b] (old_lens NULL: all blocks of the sequences), every KV head and element:
 * the least and the largest value among the keys of its tokens t < context_lens[b]
 * (rows behind them do not count).
 *   bounds  bf16 [num_blocks][num_kv_heads][2][head_dim]: least, largest; for the 8-bit
 *           and 4-bit caches of code (* group scale), the head's scale left out. Exact
 *           for every cache type. A NaN among the keys makes both NaN.
 * Bounds of other blocks are left as they were, those of a sequence that gains no token
 * (old_lens[b] >= context_lens[b]) among them (max_blocks_per_seq * num_kv_heads below
 * 2^31). Two sequences that share a block and both gain tokens in it write the same bounds
 * if both hold all of its tokens. max_new_tokens is a host-known upper
 * bound of context_lens[b] - old_lens[b]; blocks beyond those that so many tokens can
 * touch are not done, and set PA_DEVERR_CONTEXT_LEN, as a length past the table row does.
 * After pa_evict_compact or pa_copy_blocks the bounds of the written blocks are stale.
 * ---------------------------------------------------------------------- */
typedef struct {
  const void* k_cache;         /* of type kv_dtype, as in pa_decode_params */
  void* bounds;                /* bf16 [num_blocks][num_kv_heads][2][head_dim], written */
  const int32_t* block_tables; /* int32 [num_seqs][max_blocks_per_seq] */
  const int32_t* context_lens; /* int32 [num_seqs] */
  const int32_t* old_lens;     /* int32 [num_seqs] or NULL (zeros) */
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t block_size;
  int32_t num_blocks;
  int32_t max_new_tokens;      /* >= 1 */
  int32_t kv_dtype;
} pa_block_bounds_params;
pa_status pa_block_bounds(const pa_block_bounds_params* p, pa_stream_t stream);

/* pa_block_scores -- for every sequence b, KV head g and block j < ceil(context_lens[b] /
 * block_size), over the query heads h of g and the new tokens i that see the block's
 * first token (the causal rule of pa_decode):
 *   scores[b][g][j] = max over i, h of  sum over d of max(f q_d least_d, f q_d largest_d),
 *   f = scale * k_scale[g], q = q[b][i][h]
 * In exact arithmetic no logit of a key in the block exceeds it; it is held in fp32, within
 * 2^-17 times the sum of its terms' magnitudes. The sum is taken as f+ times (q's
 * positive part . largest + q's negative part . least); where that is no number (an
 * infinite or NaN bound), the score is +infinity. Entries from there on are left as they
 * were, and so are the rows of a sequence of length 0 or with fewer keys than new tokens
 * (the latter sets PA_DEVERR_CONTEXT_LEN). */
typedef struct {
  const void* q;               /* bf16 [num_seqs][query_len][num_q_heads][head_dim] */
  const void* bounds;          /* of pa_block_bounds */
  const float* k_scale;        /* float [num_kv_heads], or NULL (ones: the bf16 cache) */
  const int32_t* block_tables; /* int32 [num_seqs][max_blocks_per_seq] */
  const int32_t* context_lens; /* int32 [num_seqs], the new tokens included */
  float* scores;               /* float [num_seqs][num_kv_heads][scores_stride], written */
  int32_t scores_stride;       /* >= the blocks of min(max_context_len, a table row) tokens */
  int32_t max_blocks_per_seq;
  int32_t num_seqs;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t head_dim;
  int32_t block_size;
  int32_t num_blocks;
  int32_t max_context_len;     /* host-known upper bound of every context_lens[b] (>= 1) */
  float scale;                 /* the softmax scale: positive, finite */
  int32_t query_len;           /* new tokens per sequence (0 or 1 = one), up to 1024 */
} pa_block_scores_params;
pa_status pa_block_scores(const pa_block_scores_params* p, pa_stream_t stream);

/* pa_block_select -- the blocks that every (sequence, KV head) reads: all n =
 * ceil(context_lens[b] / block_size) of them if they are at most `budget`, else the first
 * `sink`, the last `recent` and, of the others, the budget - sink - recent with the
 * largest scores (ties: the lower index; +0 and -0 are equal, a NaN ranks below every
 * number).
 *   selected  int32 [num_seqs][num_kv_heads][budget]: their indices, ascending; -1 behind
 * scores: float [num_seqs][num_kv_heads][scores_stride]; blocks beyond scores_stride do
 * not take part and set PA_DEVERR_CONTEXT_LEN. scores_stride and budget in [1, 2^30],
 * sink and recent >= 0 with sink + recent <= budget. No workspace. */
pa_status pa_block_select(const float* scores, const int32_t* context_lens, int32_t* selected,
                          int32_t num_seqs, int32_t num_kv_heads, int32_t scores_stride,
                          int32_t block_size, int32_t budget, int32_t sink, int32_t recent,
                          pa_stream_t stream);

/* pa_decode_selected -- pa_decode over the tokens of the selected blocks alone: of
 * selected [num_seqs][num_kv_heads][num_selected] row (b, g) names the logical blocks (of
 * sequence b) that the query heads of KV head g attend to. Of a row the first
 * min(num_selected, ceil(context_lens[b] / block_size)) entries count; negative ones among
 * them are skipped, one past the sequence's blocks is too and sets PA_DEVERR_KEEP. Any
 * order; a block that is listed twice counts twice. A query token that sees none of the
 * listed tokens (or whose every score is -infinity) gets a row of zeros.
 * p is as in pa_decode: all caches, several new tokens (causal among them); the columns
 * of a KV head's products are G heads of 8 / G new tokens, more of those read the blocks
 * again. num_seqs * ceil(query_len / (8 / G)) * num_kv_heads below 2^27 (else
 * PA_ERR_UNSUPPORTED), num_blocks * num_kv_heads below 2^31, table rows of up to 2^30
 * tokens. One kernel whatever `variant` says;
 * partition_tokens, overlap_prologue and wait_timeout_us are checked like those of
 * pa_decode and not used.
 * Softmax weights: two bf16 terms (2^-17 of a weight is lost) with the bf16 cache; f16
 * with the others, as in the 4-bit decode.
 * The kernel needs no workspace: pa_decode_selected_workspace_size is 0, and `workspace`,
 * there as in pa_decode, may be NULL and is not looked at. */
size_t pa_decode_selected_workspace_size(const pa_decode_params* p, int32_t num_selected);
pa_status pa_decode_selected(const pa_decode_params* p, const int32_t* selected,
                             int32_t num_selected, void* workspace, size_t workspace_bytes,
                             pa_stream_t stream);

/* ------------------------------------------------------------------------
 * Host block pool [P1 §Paged attention; P2 §Prefix Caching and Copy-on-Write;
 * P3 §The architecture]. All memory here is host memory owned by the pool.
 * Not thread-safe: one pool per thread, or external locking.
 *
 * Free list: a stack. free_order[0] (or block 0 when free_order is NULL) is
 * handed out first; a block whose refcount drops to zero is pushed on top
 * and handed out next (blocks of the prefix cache, below, excepted). Every
 * failing call leaves the pool unchanged. free_blocks in the stats counts
 * every block that can be handed out, evictable cached blocks included.
 * ---------------------------------------------------------------------- */
typedef struct pa_pool pa_pool;

typedef struct {
  int32_t num_blocks;
  int32_t block_size;
  int32_t free_blocks;
  int32_t used_blocks;   /* refcount >= 1 */
  int32_t shared_blocks; /* refcount >= 2 */
  int32_t max_refcount;
  int32_t live_seqs;
} pa_pool_stats_t;

/* free_order: host int32 [num_blocks], a permutation of 0..num_blocks-1, or NULL. */
pa_status pa_pool_create(int32_t num_blocks, int32_t block_size, const int32_t* free_order,
                         pa_pool** out);
void pa_pool_destroy(pa_pool* pool);
/* Pop one block (refcount 1). PA_ERR_OOM when empty. */
pa_status pa_pool_alloc(pa_pool* pool, int32_t* block);
pa_status pa_pool_incref(pa_pool* pool, int32_t block);
/* Refcount - 1; pushed back on the free list at 0. PA_ERR_REFCOUNT if not allocated. */
pa_status pa_pool_decref(pa_pool* pool, int32_t block);
/* Refcount of `block` (0 = free), or -1 for an out-of-range id. */
int32_t pa_pool_refcount(const pa_pool* pool, int32_t block);
pa_status pa_pool_stats(const pa_pool* pool, pa_pool_stats_t* stats);

/* Sequences: each owns a block table and a length. */
pa_status pa_seq_create(pa_pool* pool, int32_t* seq);
/* Release every block of the sequence (in logical order) and retire the id. */
pa_status pa_seq_free(pa_pool* pool, int32_t seq);
/* New sequence sharing the parent's first ceil(num_tokens/block_size) blocks
 * (each refcount + 1), length num_tokens <= parent length. */
pa_status pa_seq_fork(pa_pool* pool, int32_t parent, int32_t num_tokens, int32_t* child);
/* Reserve the slot of the sequence's next token (allocate_slots for one
 * token). If the length is a multiple of block_size a fresh block is
 * appended to the table. Otherwise, if the target block is shared
 * (refcount > 1), copy-on-write: a fresh block replaces it in this table, the
 * old block's refcount drops by one, and (src, dst) is returned in cow_pair
 * with *has_cow = 1 -- the caller must run pa_copy_blocks on that pair before
 * writing the token. *slot = table[len / bs] * bs + len % bs. */
pa_status pa_seq_append_slot(pa_pool* pool, int32_t seq, int64_t* slot, int32_t cow_pair[2],
                             int32_t* has_cow);
/* Append n tokens; slots (nullable, [n]) and cow_pairs (nullable, [n][2])
 * receive the results, *num_cow (nullable) the number of pairs. All or
 * nothing: on PA_ERR_OOM the pool is unchanged. */
pa_status pa_seq_append_tokens(pa_pool* pool, int32_t seq, int32_t n, int64_t* slots,
                               int32_t* cow_pairs, int32_t* num_cow);
/* Shorten the sequences seqs[0..n) (distinct) to new_lens[0..n) tokens, each at
 * most the sequence's length, in blocks that they may write: the pool's half of
 * pa_evict_compact for a batch. A sequence that keeps its length keeps its
 * table. Of the others the first ceil(new_len/block_size) entries stay, except
 * that one whose block is shared (refcount > 1 before the call) or in the prefix
 * cache is replaced by a fresh block; the replaced and the remaining blocks are
 * released, after every fresh one has been taken. Read the tables before
 * (block_tables) and after (dst_tables). The rows still lie in the old blocks,
 * released ones among them, until the move has run: enqueue it before any work
 * that writes a block handed out after this call. All or nothing: PA_ERR_OOM
 * leaves the pool unchanged. */
pa_status pa_pool_compact(pa_pool* pool, const int32_t* seqs, const int32_t* new_lens, int32_t n);
pa_status pa_seq_length(const pa_pool* pool, int32_t seq, int32_t* length);
/* Copy the sequence's table into out[0..cap); *n_blocks = its block count. */
pa_status pa_seq_table(const pa_pool* pool, int32_t seq, int32_t* out, int32_t cap,
                       int32_t* n_blocks);
/* Pack the tables and lengths of seqs[0..n) into host arrays
 * tables[n][max_blocks] (unused entries -1) and lens[n], ready to upload. */
pa_status pa_pool_export(const pa_pool* pool, const int32_t* seqs, int32_t n, int32_t max_blocks,
                         int32_t* tables, int32_t* lens);

/* ------------------------------------------------------------------------
 * Prefix cache [P1 FAQ "Where does prefix caching fit?": blocks are
 * content-hashed and a new request whose prompt hashes to resident blocks
 * points at them; P3 §The architecture: the prefix cache hashes each full
 * block's token ids chained with its prefix hash, a match maps the existing
 * physical block with a bumped refcount and skips its prefill; §End-to-end
 * flow: on completion the shared blocks' refcounts tick down and the
 * preamble stays warm in the cache for the next request].
 *
 * pa_seq_create_prompt creates a sequence holding a prompt of num_tokens
 * token ids (host int32). Its full blocks are looked up in order by the chain
 * key (previous block's key, this block's block_size token ids); the leading
 * run of matches is mapped (refcount + 1) and the rest of the prompt gets
 * fresh blocks, whose full ones are entered in the cache. Matching stops at
 * the first miss. A key match is confirmed on the stored token ids, so a
 * hash collision never maps the wrong block.
 *  *cached_tokens = block_size * (matched blocks): their K/V is already in
 *   the cache; the caller writes only tokens [*cached_tokens, num_tokens).
 *  slots (nullable, [num_tokens]): every token's slot.
 * A block whose refcount drops to zero while it is in the cache stays in it
 * (evictable): pa_pool_alloc and appends hand out never-cached free blocks
 * first and then the least recently freed cached block, which leaves the
 * cache at that moment. A cached block is never written in place: an append
 * into it copies it first (copy-on-write), whatever its refcount. All or
 * nothing: on PA_ERR_OOM the pool is unchanged. Without this call the pool
 * behaves exactly as described above.
 * ---------------------------------------------------------------------- */
pa_status pa_seq_create_prompt(pa_pool* pool, const int32_t* tokens, int32_t num_tokens,
                               int32_t* seq, int32_t* cached_tokens, int64_t* slots);

typedef struct {
  int32_t cached_blocks;     /* blocks in the cache (in use or evictable) */
  int32_t evictable_blocks;  /* cached blocks with refcount 0 (counted as free) */
  int64_t lookups;           /* full prompt blocks looked up */
  int64_t hits;              /* of which mapped from the cache */
} pa_prefix_stats_t;
pa_status pa_pool_prefix_stats(const pa_pool* pool, pa_prefix_stats_t* stats);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDKV_H */
