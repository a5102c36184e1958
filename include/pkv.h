/*
 * pkv.h -- C ABI of the paged KV-cache library for one NVIDIA GB300 (sm_103a).
 *
 * Two operations, as the course page "P09 · Paged KV 写入 + decode attention
 * （参考实现）" (kuanzhou.online, nano-vllm-omni drills) defines them in its
 * section 题面速览 and its two shape-trace tables (框架视角 · shape trace):
 *
 *   pkv_write             write_kv: cache[slot // bs, slot % bs] = k[i] (and v),
 *                         in place; a negative slot is a padding token and is
 *                         not written.
 *   pkv_decode_attention  paged decode attention: each sequence's single query
 *                         attends to the first context_lens[b] tokens of its
 *                         paged context, gathered through block_tables[b, :nb]
 *                         with nb = ceil(n / bs); query head h reads KV head
 *                         h // (H / KVH); softmax(q . K^T * scale) . V with the
 *                         softmax in fp32, output in q's dtype.
 * Long contexts are split into partitions whose partial results are merged
 * with a log-sum-exp rescale, the partitioned variant the interview note
 * "PagedAttention kernel: paged KV cache 与 block table"
 * (inference-learning-path.pages.dev), section 深入原理 ("v1 vs v2"),
 * describes; the result equals the unsplit one up to rounding.
 *
 * Common rules
 *   - Every pointer argument except the host-side ones named below is a
 *     DEVICE pointer on the current CUDA device.  The caller owns all memory;
 *     the library allocates nothing on the call path and keeps no pointer
 *     after a call returns.
 *   - All work is enqueued on `stream` (NULL = the legacy default stream);
 *     calls return once the work is enqueued, before it runs.
 *   - Argument errors that need no device data are caught on the host before
 *     anything is enqueued and returned as a status.
 *   - Errors that depend on device data (a slot past the pool, a table entry
 *     outside [0, num_blocks), an over-long context) cannot be seen on the
 *     host: the kernels skip the offending access and OR a PKV_FLAG_* bit into
 *     *err_flags (a device int, may be NULL).  The caller reads it after the
 *     stream has synchronised.  Nothing in the library traps or asserts on
 *     the device.
 *   - Cache layout: K and V are separate tensors
 *     [num_blocks, block_size, num_kv_heads, head_dim], contiguous, one
 *     token's row of num_kv_heads * head_dim elements contiguous.
 */
#ifndef PKV_H
#define PKV_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define PKV_API __attribute__((visibility("default")))
#else
#define PKV_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

/* The same handle type as cudaStream_t (a CUstream). */
typedef struct CUstream_st *pkv_stream_t;

typedef enum pkv_status {
  PKV_OK = 0,
  PKV_ERR_INVALID_ARG = 1,   /* a size, pointer, alignment or count is not valid */
  PKV_ERR_UNSUPPORTED = 2,   /* valid, but a shape/dtype this build does not handle */
  PKV_ERR_CUDA = 3,          /* a CUDA runtime call or a kernel launch failed */
  PKV_ERR_WORKSPACE = 4,     /* the workspace is missing or smaller than needed */
  PKV_ERR_OUT_OF_BLOCKS = 5  /* block manager (pkv_block_manager.h): not enough free blocks */
} pkv_status;

typedef enum pkv_dtype {
  PKV_F32 = 0,   /* float32 */
  PKV_BF16 = 1,  /* bfloat16 */
  PKV_F16 = 2    /* float16 */
} pkv_dtype;

/* Bits the kernels OR into *err_flags. */
#define PKV_FLAG_SLOT_OUT_OF_RANGE 0x1   /* pkv_write: slot >= num_blocks * block_size; token skipped */
#define PKV_FLAG_BLOCK_OUT_OF_RANGE 0x2  /* decode: an entry of block_tables[b, :nb] outside
                                            [0, num_blocks); block 0 is read in its place and
                                            that sequence's output is unspecified */
#define PKV_FLAG_CONTEXT_TOO_LONG 0x4    /* decode: context_lens[b] > max_blocks * block_size;
                                            clamped, output of that sequence unspecified */
#define PKV_FLAG_CONTEXT_NEGATIVE 0x8    /* decode: context_lens[b] < 0; treated as 0 */
#define PKV_FLAG_CONTEXT_OVER_HINT 0x10  /* decode: context_lens[b] > max_context_len (the host
                                            hint sized the grid too small); output of that
                                            sequence unspecified */
#define PKV_FLAG_TIMEOUT 0x20            /* a bounded wait for an asynchronous copy ran out
                                            (should never happen); outputs unspecified, and a
                                            decode workspace used by that call must be
                                            zero-filled again before its next use */
#define PKV_FLAG_QUERY_LEN 0x80          /* prefill: a sequence with qlen < 0, qlen > context_lens[b]
                                            or a context longer than the table; skipped, its
                                            output rows unspecified */
#define PKV_FLAG_QUERY_OVER_HINT 0x100   /* prefill: a sequence has more queries than max_q_len;
                                            rows past max_q_len are not computed */
#define PKV_FLAG_STEP_INVALID 0x200      /* pkv_build_step: a length, block count or total the step
                                            cannot have; the step is empty, nothing changed */
#define PKV_FLAG_OUT_OF_BLOCKS 0x400     /* pkv_build_step: more blocks needed than are free; the
                                            step is empty, nothing changed */
#define PKV_FLAG_TOKENS_OVER 0x1000      /* pkv_build_step: more than max_tokens new tokens; the
                                            lists hold the first max_tokens, all else is done */
#define PKV_FLAG_POSITION 0x800          /* pkv_rope_write: a kept token's position is outside
                                            [0, max_position); the token is skipped */
#define PKV_FLAG_BEAM 0x2000             /* pkv_beam_reorder: a parent or a length that a beam cannot
                                            have; the child is unused */
#define PKV_FLAG_LOGITS 0x4000           /* pkv_beam_select: a beam with a NaN or +inf among its logits
                                            or as its score; it proposes nothing */
#define PKV_FLAG_APPEND_MISMATCH 0x40    /* pkv_write_decode_attention: a kept slot is not the
                                            slot of position context_lens[b] - 1 through
                                            block_tables (or context_lens[b] == 0); the token
                                            is still written, that sequence's output is
                                            unspecified */

/*
 * pkv_write -- write_kv / reshape_and_cache.
 * Definition: course page "P09 · Paged KV 写入 + decode attention（参考实现）",
 * section 题面速览 ("写: cache[slot // bs, slot % bs] = k[i]") and the
 * write_kv shape trace (keep = slot >= 0; blk = s // bs; off = s % bs;
 * k_cache[blk, off] = k[keep]; same for v; in place, returns nothing).
 *
 *   k_cache, v_cache  [num_blocks, block_size, num_kv_heads, head_dim], dtype dt,
 *                     written in place (only rows named by a kept slot change)
 *   k, v              [num_tokens, num_kv_heads, head_dim]; token i starts at
 *                     element i * k_token_stride (resp. v_token_stride);
 *                     each token's num_kv_heads * head_dim elements contiguous
 *   slot_mapping      [num_tokens] int64: flat slot block * block_size + offset;
 *                     any negative value = padding, skipped silently
 *   err_flags         device int or NULL: PKV_FLAG_SLOT_OUT_OF_RANGE
 * The copy is bit-exact.  Two kept tokens with the same slot in one call
 * race (which one lands is unspecified).  num_tokens == 0 enqueues nothing.
 * Errors: PKV_ERR_INVALID_ARG for a NULL pointer with num_tokens > 0, a
 * non-positive size, or a token stride smaller than one row;
 * PKV_ERR_CUDA if the launch fails.
 */
PKV_API pkv_status pkv_write(void *k_cache, void *v_cache, const void *k, const void *v,
                             const int64_t *slot_mapping, int64_t num_tokens,
                             int64_t k_token_stride, int64_t v_token_stride,
                             int64_t num_blocks, int block_size, int num_kv_heads,
                             int head_dim, pkv_dtype dt, int *err_flags, pkv_stream_t stream);

/*
 * pkv_decode_workspace_size -- bytes of device workspace pkv_decode_attention
 * needs for these sizes (host only, no CUDA call).  partition_size as in
 * pkv_decode_attention (0 = automatic: the size covers every partition size
 * the automatic choice can make).  max_context_len: the longest context the
 * calls will see (0 = max_blocks * block_size).  Returns 0 for invalid sizes.
 *
 * The workspace holds per-partition partial results and one counter per
 * (sequence, head group).  Before its FIRST use it must be zero-filled
 * (e.g. cudaMemset); every call that completes without PKV_FLAG_TIMEOUT
 * leaves the counters at zero again, so the same workspace can be reused by
 * later calls on the same stream without clearing.  A call that raised
 * PKV_FLAG_TIMEOUT may have left a partition uncounted: zero-fill the
 * workspace again before reusing it.  Calls that run concurrently need
 * separate workspaces.
 */
PKV_API size_t pkv_decode_workspace_size(int B, int H, int num_kv_heads, int head_dim,
                                         int block_size, int max_blocks, int max_context_len,
                                         int partition_size);

/*
 * pkv_decode_attention -- paged decode attention (one query per sequence).
 * Definition: course page "P09 · Paged KV 写入 + decode attention（参考实现）",
 * section 题面速览 ("decode 读") and the paged_decode_attention shape trace:
 * n = context_lens[b]; nb = ceil(n / bs); table = block_tables[b, :nb];
 * gather k_cache[table] in table order; keep the first n rows; head h uses
 * KV head h // (H / KVH); fp32 scores times scale, softmax over the n
 * tokens in fp32, weighted sum of V, cast to q's dtype.
 *
 *   out           [B, H, head_dim], dtype dt (written; rows of sequences with
 *                 context_lens[b] == 0 are set to zero).  Device memory, or
 *                 host memory the GPU addresses directly (pinned memory under
 *                 unified addressing; any host memory where the system
 *                 translates host addresses for the GPU): the kernels only
 *                 store to out -- no reads, atomics or TMA -- so the result
 *                 crosses to the host inside the launch and needs no copy
 *                 after it.  Its rows are complete for the host once the
 *                 stream is synchronised.
 *   q             [B, H, head_dim], dtype dt
 *   k_cache, v_cache  [num_blocks, block_size, num_kv_heads, head_dim], dtype dt
 *   block_tables  [B, max_blocks] int32; only the first ceil(n/bs) entries of
 *                 row b are read -- the rest may hold anything (e.g. 99999)
 *   context_lens  [B] int32
 *   scale         multiplies q.K before the softmax (e.g. 1/sqrt(head_dim))
 *   max_context_len  host-side upper bound on context_lens (sizes the grid;
 *                 0 = max_blocks * block_size).  A longer context sets
 *                 PKV_FLAG_CONTEXT_OVER_HINT.
 *   partition_size   tokens per partition of the split-KV path: 0 = choose
 *                 from the sizes and the SM count, else a positive multiple
 *                 of 16 (any other value is PKV_ERR_INVALID_ARG), whatever
 *                 the block size (a partition may end inside a block).  A
 *                 context longer than one partition is processed by several
 *                 CTAs whose (max, sum, weighted-V) partials are merged in the
 *                 workspace with a log-sum-exp rescale.
 *   workspace, workspace_bytes  device scratch of at least
 *                 pkv_decode_workspace_size(...) bytes, 256-byte aligned,
 *                 zero-filled before first use; always required (it holds the
 *                 merge counters even when nothing is split)
 *   err_flags     device int or NULL (PKV_FLAG_BLOCK_OUT_OF_RANGE,
 *                 PKV_FLAG_CONTEXT_*, PKV_FLAG_TIMEOUT)
 * Supported: H % num_kv_heads == 0; head_dim a multiple of 8 in [8, 512] (fp32:
 * a multiple of 4); block_size >= 1; q, out, caches 16-byte aligned.  bf16 /
 * fp16 with head_dim in {64, 128, 192, 256} and block_size a multiple of 16
 * run a tensor-core kernel: groups of exactly 16 query heads per KV head at
 * head_dim 128 or 256 (MQA-like) the wide-group kernel (persistent, one CTA
 * per SM claiming (sequence, KV head, partition) items from a device
 * counter; 5th-generation tensor cores with the KV tile's tokens as the
 * product's M; with partition_size 0 its items may be larger than the
 * plan's partition -- about 1.2 CTA shares of the batch's 128-token tiles,
 * worked out on the device from context_lens -- never smaller, so the
 * workspace the plan sizes always holds them), the others the TMA +
 * mma.sync kernel; every other supported shape runs the CUDA-core kernel.
 * An explicit partition_size is used as given.  The output does not depend
 * on the partitioning beyond fp32 rounding order.
 * Inside a stream capture the tensor-core kernels launch as programmatic
 * dependents of the kernel before them (their start-up overlaps that
 * kernel's end in the graph): they read q, block_tables, context_lens and
 * (fused step) the new rows and slots before waiting for that kernel, and
 * the caches, the workspace and out only after.  So a kernel captured just
 * before them that releases its dependents early (griddepcontrol.
 * launch_dependents) must not write those inputs; this library's kernels
 * never do, and any other kernel is waited for in full.
 * Errors: PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE,
 * PKV_ERR_CUDA.  B == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_decode_attention(void *out, const void *q, const void *k_cache,
                                        const void *v_cache, const int32_t *block_tables,
                                        const int32_t *context_lens, int B, int H,
                                        int num_kv_heads, int head_dim, int block_size,
                                        int max_blocks, int64_t num_blocks, float scale,
                                        pkv_dtype dt, int max_context_len, int partition_size,
                                        void *workspace, size_t workspace_bytes, int *err_flags,
                                        pkv_stream_t stream);

/*
 * pkv_decode_attention_static -- pkv_decode_attention without a workspace
 * argument, for callers that may not allocate device memory: for example an
 * engine plugin whose execute step is forbidden to call cudaMalloc, code that
 * enqueues work while some other component owns the device allocator, or a
 * deployment whose device memory is fixed when the process starts.  The
 * pages have no counterpart: this is a convenience of this library.
 *
 * Arguments, results and errors are those of pkv_decode_attention, minus
 * workspace / workspace_bytes.  The split-KV scratch comes instead from a
 * fixed array of PKV_STATIC_SCRATCH_BYTES bytes inside the library, which
 * every GPU the library runs on keeps until the process exits.
 *   - Sizes whose split-KV scratch would exceed PKV_STATIC_SCRATCH_BYTES are
 *     rejected with PKV_ERR_WORKSPACE before anything is enqueued (pass a
 *     larger partition_size, or use pkv_decode_attention with a workspace).
 *   - Every argument check of pkv_decode_attention, and the size check, is
 *     made before anything is enqueued: a rejected call enqueues nothing.
 *   - No cudaMalloc, cudaFree or other allocating call is made.  The first
 *     call on each device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current, and keeps it for that
 *     device's context (after cudaDeviceReset it is looked up again); make
 *     that first call before any stream capture.
 *   - Each call clears the array's merge counters on `stream` before the
 *     kernel runs.  All calls share the one array: calls whose work overlaps
 *     on the GPU (different streams, or concurrent host threads) race and
 *     give wrong results; serialise them.
 */
#define PKV_STATIC_SCRATCH_BYTES (16u * 1024u * 1024u)
PKV_API pkv_status pkv_decode_attention_static(void *out, const void *q, const void *k_cache,
                                               const void *v_cache, const int32_t *block_tables,
                                               const int32_t *context_lens, int B, int H,
                                               int num_kv_heads, int head_dim, int block_size,
                                               int max_blocks, int64_t num_blocks, float scale,
                                               pkv_dtype dt, int max_context_len,
                                               int partition_size, int *err_flags,
                                               pkv_stream_t stream);

/*
 * pkv_decode_attention_with_kernel -- pkv_decode_attention with the kernel
 * named by the caller instead of chosen by the plan, for tests and tuning
 * (the pages have no counterpart: it exists to measure one kernel against
 * another on the same batch).  kernel: -1 = the plan's choice (exactly
 * pkv_decode_attention), 0 = the CUDA-core kernel (any supported shape),
 * 1 = the TMA + mma.sync tensor-core kernel, 2 = the wide-group tcgen05
 * kernel.  A kernel that cannot run the given shape returns
 * PKV_ERR_UNSUPPORTED before anything is enqueued; any other kernel value is
 * PKV_ERR_INVALID_ARG.  Arguments, workspace (sized by
 * pkv_decode_workspace_size, which covers every kernel), results and errors
 * otherwise as in pkv_decode_attention.
 */
PKV_API pkv_status pkv_decode_attention_with_kernel(
    void *out, const void *q, const void *k_cache, const void *v_cache,
    const int32_t *block_tables, const int32_t *context_lens, int B, int H, int num_kv_heads,
    int head_dim, int block_size, int max_blocks, int64_t num_blocks, float scale, pkv_dtype dt,
    int max_context_len, int partition_size, void *workspace, size_t workspace_bytes,
    int *err_flags, int kernel, pkv_stream_t stream);

/*
 * pkv_write_decode_attention -- one decode step in one launch: pkv_write of
 * each sequence's new token followed by pkv_decode_attention over contexts
 * that already count it.
 * Definition: course page "P09 · Paged KV 写入 + decode attention（参考实现）",
 * section 在系统中的位置 -- each model-runner step first writes the new
 * tokens' K/V into the cache by slot_mapping, then attention reads the
 * history through block_tables; the result is that of the two calls above
 * made one after the other.
 *
 *   k, v          [B, num_kv_heads, head_dim]: the new token of sequence b
 *                 starts at element b * k_token_stride (resp. v_token_stride)
 *   slot_mapping  [B] int64: slot of sequence b's new token; negative = no
 *                 new token (padding), nothing written for b
 *   everything else as in pkv_decode_attention (k_cache, v_cache are
 *   written in place at the kept slots).
 * Precondition (the decode append): a kept slot_mapping[b] is the slot of
 * logical position context_lens[b] - 1 of sequence b,
 *   block_tables[b, (n-1) / bs] * bs + (n-1) % bs,   n = context_lens[b],
 * and no other sequence's context reads that slot.  The kernel checks the
 * first part and raises PKV_FLAG_APPEND_MISMATCH when it does not hold.
 * The launch that reads position n-1 takes the new token's K/V from k/v
 * directly, so it does not wait for its own cache write; one CTA per
 * (sequence, KV head) writes the cache row.  (On the wide-group kernel --
 * see pkv_decode_attention -- the row read at position n-1 is replaced in
 * shared memory by the new token's once the tile has landed; still one
 * launch.)  The
 * cache ends bit-identical to pkv_write's; the output is bit-identical to
 * pkv_write + pkv_decode_attention with the same partition size.
 * Additional requirements: k, v, k_cache, v_cache 16-byte aligned;
 * head_dim * element size a multiple of 16 bytes; k_token_stride and
 * v_token_stride >= num_kv_heads * head_dim and multiples of 16 bytes.
 * Errors: those of pkv_decode_attention; PKV_ERR_INVALID_ARG for a NULL
 * k, v or slot_mapping or a misaligned row.
 */
PKV_API pkv_status pkv_write_decode_attention(
    void *out, const void *q, const void *k, const void *v, int64_t k_token_stride,
    int64_t v_token_stride, const int64_t *slot_mapping, void *k_cache, void *v_cache,
    const int32_t *block_tables, const int32_t *context_lens, int B, int H, int num_kv_heads,
    int head_dim, int block_size, int max_blocks, int64_t num_blocks, float scale, pkv_dtype dt,
    int max_context_len, int partition_size, void *workspace, size_t workspace_bytes,
    int *err_flags, pkv_stream_t stream);

/*
 * pkv_prefill_attention -- paged causal prefill attention: several new query
 * tokens per sequence (varlen), each attending to the context up to itself.
 * Definition: the course page "P09 · Paged KV 写入 + decode attention（参考
 * 实现）" asks how the varlen prefill version is written (section 面试官追问)
 * without giving it; this library's reading is the multi-query form of its
 * decode (section 细节: the decode query is the newest token, already
 * written, and sees the whole context including itself):
 *   qlen = cu_seqlens_q[b+1] - cu_seqlens_q[b] queries of sequence b are the
 *   LAST qlen of its n = context_lens[b] tokens, all already written to the
 *   cache (pkv_write); query i (row cu_seqlens_q[b] + i) sits at position
 *   p = n - qlen + i and attends to tokens 0 .. p; head h uses KV head
 *   h // (H / KVH); fp32 scores times scale, fp32 softmax, output in q's
 *   dtype.  With qlen = 1 it is pkv_decode_attention.
 *
 *   out, q        [total_q, H, head_dim], total_q = cu_seqlens_q[B]
 *   cu_seqlens_q  [B + 1] int32, cu_seqlens_q[0] = 0, non-decreasing
 *   k_cache, v_cache, block_tables, context_lens: as in pkv_decode_attention
 *   max_q_len     host-side upper bound on qlen (sizes the grid; 0 = total_q);
 *                 a longer sequence raises PKV_FLAG_QUERY_OVER_HINT
 *   err_flags     device int or NULL (PKV_FLAG_QUERY_LEN,
 *                 PKV_FLAG_QUERY_OVER_HINT, PKV_FLAG_BLOCK_OUT_OF_RANGE,
 *                 PKV_FLAG_TIMEOUT)
 * Supported: bf16 / fp16, head_dim 64 or 128, block_size a multiple of 16,
 * q, out, caches 16-byte aligned (tensor-core kernel, tcgen05).  No
 * workspace.  Errors: PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA.
 * B == 0 or total_q == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_prefill_attention(void *out, const void *q, const void *k_cache,
                                         const void *v_cache, const int32_t *block_tables,
                                         const int32_t *cu_seqlens_q, const int32_t *context_lens,
                                         int B, int64_t total_q, int H, int num_kv_heads,
                                         int head_dim, int block_size, int max_blocks,
                                         int64_t num_blocks, float scale, pkv_dtype dt,
                                         int max_q_len, int *err_flags, pkv_stream_t stream);

/*
 * pkv_build_step -- one serving step's block tables, slots, positions and
 * query offsets, built on the GPU from the requests' lengths, with the blocks
 * taken from and returned to a free list in device memory: what the host
 * block manager (pkv_block_manager.h) hands out, without the host in the
 * loop, so that a captured graph can replay whole steps whose lengths change
 * on the device (drafted tokens accepted or turned down, requests that end).
 *
 *   block_tables  [B, max_blocks] int32, updated in place: request b's first
 *                 held[b] entries are its blocks
 *   held, held_out  [B] int32: blocks request b holds before / after
 *   free_blocks   [free_capacity] int32, updated in place: a stack whose first
 *                 *free_count entries are the free blocks
 *   free_count, free_count_out  one int32: free blocks before / after
 *   cached_lens   [B] int32: tokens of request b that are in the cache already
 *   new_lens      [B] int32: tokens it adds in this step (0 = none)
 *   context_lens  [B] int32 out: cached_lens[b] + new_lens[b]
 *   cu_seqlens_q  [B + 1] int32 out: exclusive sums of new_lens
 *   slot_mapping  [max_tokens] int64 out: slots of the new tokens, requests in
 *                 order, -1 behind the last one
 *   positions     [max_tokens] int32 out: their positions, 0 behind the last
 *   num_blocks    blocks in the pool (every table and free entry read is
 *                 checked against it)
 * Request b ends with want = ceil((cached_lens[b] + new_lens[b]) / block_size)
 * blocks.  Requests that hold more give theirs back first -- entries
 * [want, held) of their rows are pushed on the stack, requests and entries in
 * ascending order (the entries stay in the table row as they were) -- then
 * requests that hold fewer take theirs from its top, requests and entries in
 * ascending order.  A request that ended has both lengths 0; one whose drafted
 * tokens were turned down comes with the smaller cached length.
 * held_out may be held, free_count_out may be free_count, and context_lens
 * may be cached_lens; no other two arguments may overlap.
 * All or nothing: with a negative length, a held outside [0, max_blocks], a
 * request that holds fewer than ceil(cached_lens[b] / block_size) blocks or
 * needs more than max_blocks, 2^30 new tokens or more in all, or a free list
 * that is (or would become) larger than free_capacity, the call raises
 * PKV_FLAG_STEP_INVALID; with too few free blocks PKV_FLAG_OUT_OF_BLOCKS.  In
 * both cases tables, free list and counts stay as they were (held_out and
 * free_count_out get the old values) and the step is empty: context_lens 0,
 * cu_seqlens_q 0, every slot -1.  More than max_tokens new tokens raise
 * PKV_FLAG_TOKENS_OVER: slot_mapping and positions hold the first max_tokens,
 * everything else is as without the bound (what attends over max_tokens query
 * rows skips and flags the requests past it).  An entry outside [0, num_blocks)
 * raises PKV_FLAG_BLOCK_OUT_OF_RANGE where a token or a request would get it;
 * that token's slot is -1.
 * Supported: B <= 16384, max_tokens < 2^30, free_capacity < 2^30.  Errors:
 * PKV_ERR_INVALID_ARG (NULL or misaligned pointers, sizes),
 * PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA.
 * B == 0 with max_tokens == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_build_step(int32_t *block_tables, const int32_t *held, int32_t *held_out,
                                  int32_t *free_blocks, const int32_t *free_count,
                                  int32_t *free_count_out, const int32_t *cached_lens,
                                  const int32_t *new_lens, int32_t *context_lens,
                                  int32_t *cu_seqlens_q, int64_t *slot_mapping, int32_t *positions,
                                  int B, int max_blocks, int64_t num_blocks, int block_size,
                                  int64_t free_capacity, int64_t max_tokens, int *err_flags,
                                  pkv_stream_t stream);

/*
 * pkv_rope_write -- rotary positions and pkv_write in one pass: every kept
 * token's query heads are rotated into q_out, its key heads are rotated into
 * the cache and its value heads copied there.
 *
 *   q             [num_tokens, H, head_dim], token i at element i * q_token_stride
 *   k, v          [num_tokens, num_kv_heads, head_dim], strides as in pkv_write
 *   q_out         [num_tokens, H, head_dim] contiguous; may be q itself (with
 *                 q_token_stride = H * head_dim), else overlaps no other
 *                 argument
 *   k_cache, v_cache, slot_mapping  as in pkv_write; the caches do not overlap
 *   cos_sin       [max_position, rot_dim] float32: row p holds the cosines of
 *                 the rot_dim / 2 pairs' angles at position p, then the sines
 *   positions     [num_axes, num_tokens] int32, axis a at element
 *                 a * positions_stride: a token's position on each axis (for
 *                 images and video: time, height, width); stride 0 gives every
 *                 axis the same positions (text)
 *   pair_axis     HOST array of rot_dim / 2 bytes: the axis in [0, num_axes)
 *                 whose position turns pair j (sections, or any interleaving
 *                 of the axes); NULL = axis 0 for all; read during the call
 *   rot_dim       even, 0 .. head_dim: the leading elements of a head that
 *                 turn; the rest is copied
 *   interleaved   0: pair j is elements (j, j + rot_dim / 2); else (2j, 2j + 1)
 * With (x, y) a pair and c, s its table entries: (x c - y s, y c + x s), in
 * fp32, rounded once to dtype.  A negative slot is a padding token: nothing
 * is written for it (its q_out row stays as it was).  A kept token
 * with a used axis' position outside [0, max_position) raises
 * PKV_FLAG_POSITION and is skipped the same way; a slot past the pool raises
 * PKV_FLAG_SLOT_OUT_OF_RANGE, its q_out row is written and the cache is not.
 * Two kept tokens with the same slot race, as in pkv_write.
 * Supported: head_dim <= 512, num_axes 1 .. 4, any alignment of elements
 * (16-byte aligned rows are fastest).  Errors: PKV_ERR_INVALID_ARG,
 * PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA.  num_tokens == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_rope_write(void *q_out, void *k_cache, void *v_cache, const void *q,
                                  const void *k, const void *v, const float *cos_sin,
                                  const int32_t *positions, const uint8_t *pair_axis,
                                  const int64_t *slot_mapping, int64_t num_tokens,
                                  int64_t q_token_stride, int64_t k_token_stride,
                                  int64_t v_token_stride, int64_t positions_stride, int num_axes,
                                  int H, int num_kv_heads, int head_dim, int rot_dim,
                                  int interleaved, int64_t max_position, int64_t num_blocks,
                                  int block_size, pkv_dtype dt, int *err_flags,
                                  pkv_stream_t stream);

/*
 * pkv_chunk_attention -- attention of each sequence's newest tokens over its
 * paged context, with the score forms models use beside plain causal
 * attention.  As in pkv_prefill_attention the qlen = cu_seqlens_q[b+1] -
 * cu_seqlens_q[b] queries of sequence b are the last qlen of its
 * n = context_lens[b] tokens, query i at position p = n - qlen + i; qlen = 1
 * is decode.  For key j and query head h:
 *   x = scale * q . k_j
 *   x = softcap * tanh(x / softcap)           if softcap > 0
 *   x = x - slopes[h] * |p - j|               if slopes
 *   visible:  (j <= p  or  j < prefix_lens[b])
 *             and (window == 0 or p - j < window)  and  j >= kv_starts[row]
 * then an fp32 softmax over the visible keys and the weighted sum of V.  A
 * query that sees no key gives a row of zeros.  Scores, softmax statistics and
 * sums are fp32; on the tensor-core kernels the weights 2^(x - max) are rounded
 * to the tensors' 16-bit type for the product with V (off by half a step each,
 * as the output is by its own rounding).
 *
 *   out, q, cu_seqlens_q, k_cache, v_cache, block_tables, context_lens
 *                 as in pkv_prefill_attention (neither out nor the workspace
 *                 overlaps another argument); out rows behind cu_seqlens_q[B] are left as they
 *                 were
 *   softcap       0 = none, else > 0; up to 256 is fastest on the tensor-core
 *                 kernels (larger ones take a form whose error does not grow
 *                 with the cap)
 *   window        0 = none, else a query sees at most the last `window` keys
 *                 up to itself (and the prefix positions above p)
 *   slopes        [H] float32 or NULL: linear distance bias per query head
 *   prefix_lens   [B] int32 or NULL: keys below it are visible to every query
 *                 of the sequence, also to earlier positions (prefix mask);
 *                 values past n act as n, negative ones as 0
 *   kv_starts     [total_q] int32 or NULL: the first key a query may see, for
 *                 example its document's first position in a packed sequence
 *   max_q_len     host bound on qlen (0 = total_q); a longer sequence raises
 *                 PKV_FLAG_QUERY_OVER_HINT, its output rows are unspecified.
 *                 The bounds choose the kernel and the split, and with them the
 *                 speed: 64 single tokens of 4 heads a KV head take 104 us with
 *                 max_q_len 1 and 127 us without it (planned as 64 queries of
 *                 one sequence)
 *   max_context_len  host bound on context_lens (0 = max_blocks *
 *                 block_size); a longer one raises PKV_FLAG_CONTEXT_OVER_HINT,
 *                 its output rows are unspecified
 *   partition_size  0 = automatic, else a positive multiple of 128: keys per
 *                 part of the split over the context (raised where it would
 *                 give more than 256 parts, at most 2^20 on the tcgen05 kernel
 *                 where that gives no more; with more than 65520 units of 16
 *                 rows nothing is split)
 *   workspace     pkv_chunk_workspace_size(...) bytes, 256-byte aligned,
 *                 zero-filled before its first use; every call that completes
 *                 without PKV_FLAG_TIMEOUT leaves it ready for the next on the
 *                 same stream.  Calls that may overlap need workspaces of
 *                 their own (two captured graphs that share one must not
 *                 replay at the same time).
 * A sequence with qlen < 0, qlen > n or a context longer than its table
 * raises PKV_FLAG_QUERY_LEN and is skipped, its rows unspecified.  Cache rows
 * that no query of a sequence sees (behind its context, before its window)
 * may hold anything, NaN included, and an invisible key or value never
 * changes a row, whatever it holds.  Table entries of blocks that no query
 * sees are not read.
 * Supported: fp32, bf16, fp16; head_dim <= 512; any block size; element-
 * aligned pointers; max_q_len * H / num_kv_heads < 2^31 - 64.  bf16 / fp16 with 16-byte aligned tensors, block_size a
 * multiple of 16 and head_dim 64, 128, 192 or 256 run tensor-core kernels:
 * an mma.sync kernel where max_q_len * H / num_kv_heads is 32 at most or the
 * whole call is small, else a tcgen05 kernel (three launches: plan, attention
 * and, when split, join).  Everything else runs on the CUDA cores.
 * Errors: PKV_ERR_INVALID_ARG (also a scale that is not finite, a softcap
 * that is negative, not finite or too small for scale / softcap, a negative
 * window), PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE, PKV_ERR_CUDA.  B == 0 or
 * total_q == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_chunk_attention(
    void *out, const void *q, const void *k_cache, const void *v_cache,
    const int32_t *block_tables, const int32_t *cu_seqlens_q, const int32_t *context_lens,
    const float *slopes, const int32_t *prefix_lens, const int32_t *kv_starts, int B,
    int64_t total_q, int H, int num_kv_heads, int head_dim, int block_size, int max_blocks,
    int64_t num_blocks, float scale, float softcap, int window, pkv_dtype dt, int max_q_len,
    int max_context_len, int partition_size, void *workspace, size_t workspace_bytes,
    int *err_flags, pkv_stream_t stream);

/*
 * pkv_chunk_workspace_size -- bytes of workspace pkv_chunk_attention needs for
 * these sizes, for every dtype, window and score form (host only).  Returns 0
 * for invalid sizes.
 */
PKV_API size_t pkv_chunk_workspace_size(int B, int64_t total_q, int H, int num_kv_heads,
                                        int head_dim, int block_size, int max_blocks,
                                        int max_q_len, int max_context_len, int partition_size);

/*
 * pkv_chunk_plan -- the kernel (2 tcgen05, 1 mma.sync, 0 CUDA cores) and the
 * split that pkv_chunk_attention would use for these arguments with 16-byte
 * aligned tensors (host only; for tests and tuning).  has_prefix: prefix_lens
 * is given.  Returns the keys per part, or 0 for invalid sizes.
 */
PKV_API int pkv_chunk_plan(int B, int64_t total_q, int H, int num_kv_heads, int head_dim,
                           int block_size, int max_blocks, int max_q_len, int max_context_len,
                           int window, int has_prefix, int partition_size, pkv_dtype dt,
                           int *max_parts, int *kernel);

/*
 * A cache held in 8 or 4 bits.  Each row (one token's head_dim values of one
 * KV head) is quantised by itself:
 *   PKV_QUANT_INT8  code = rint(x * inv),                       value = scale * code
 *   PKV_QUANT_E4M3  code = e4m3(fl(x * inv)),                   value = scale * code
 *   PKV_QUANT_INT4  code = clamp(rint(x * inv) + zero, 0, 15),  value = scale * (code - zero)
 * with scale = fl(A * fl(1 / top)) and inv = fl(fl(1 / A) * top), top = 127,
 * 448 or 15; fl() a rounding to float32, rint the nearest whole number (halves
 * to even) of the exact product.  A is the row's largest magnitude; for INT4
 * lo = min(x, 0), hi = max(x, 0), A = fl(hi - lo), zero = rint(-lo * inv).
 * A row with A below 2^-100 is held as zeros (scale 0); one that is not
 * finite, or whose A is not, has scale NaN and codes 0, so that everything
 * read from it is NaN.
 *   codes   [num_blocks, block_size, num_kv_heads, head_dim] bytes; INT4
 *           head_dim / 2 bytes a row, the even element in the low half
 *   params  float32 [num_blocks, num_kv_heads, block_size]: scale; INT4
 *           [num_blocks, num_kv_heads, block_size, 2]: scale, zero.  A head's
 *           numbers of one block lie together, as the decode reads them.
 * Scales must not be negative; zero points are whole numbers from 0 to 15.
 */
typedef enum pkv_quant_format {
  PKV_QUANT_INT8 = 0,
  PKV_QUANT_E4M3 = 1,
  PKV_QUANT_INT4 = 2
} pkv_quant_format;

/*
 * pkv_quant_write -- pkv_write into a quantised cache: k and v (fp32, bf16 or
 * fp16; arguments as in pkv_write) are quantised row by row as they are
 * written.  A negative slot is a padding token and is skipped; one past the
 * pool raises PKV_FLAG_SLOT_OUT_OF_RANGE and is skipped.  Two kept tokens with
 * the same slot race.
 * Supported: head_dim <= 512, for INT4 even; any alignment of elements (codes:
 * of bytes); 16-byte aligned rows are fastest.  The four written arrays
 * overlap no other argument.  Errors: PKV_ERR_INVALID_ARG,
 * PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA.  num_tokens == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_quant_write(void *k_codes, void *v_codes, float *k_params, float *v_params,
                                   const void *k, const void *v, const int64_t *slot_mapping,
                                   int64_t num_tokens, int64_t k_token_stride,
                                   int64_t v_token_stride, int64_t num_blocks, int block_size,
                                   int num_kv_heads, int head_dim, pkv_quant_format fmt,
                                   pkv_dtype dt, int *err_flags, pkv_stream_t stream);

/*
 * pkv_quant_read -- the values of cached rows: token i of k_out and v_out
 * [num_tokens, num_kv_heads, head_dim] (dtype dt, token strides in elements)
 * gets the row at slot_mapping[i], computed in fp32 and rounded once.  For
 * work that the decode below does not do: a prompt's chunk attends a context
 * read back into 16-bit blocks, a sequence moves to another cache.  A
 * negative slot leaves its rows as they were, one past the pool does too and
 * raises PKV_FLAG_SLOT_OUT_OF_RANGE.  The same slot may come more than once.
 * Sizes, alignment and errors as in pkv_quant_write; k_out and v_out overlap
 * no other argument (rows side by side in one buffer, of one stride, do not).
 */
PKV_API pkv_status pkv_quant_read(void *k_out, void *v_out, const void *k_codes,
                                  const void *v_codes, const float *k_params,
                                  const float *v_params, const int64_t *slot_mapping,
                                  int64_t num_tokens, int64_t k_out_stride, int64_t v_out_stride,
                                  int64_t num_blocks, int block_size, int num_kv_heads,
                                  int head_dim, pkv_quant_format fmt, pkv_dtype dt, int *err_flags,
                                  pkv_stream_t stream);

/*
 * pkv_quant_decode_attention -- pkv_decode_attention over a quantised cache:
 * one new token per sequence, q and out [B, H, head_dim] in dtype dt,
 *   x_j = scale * q . K_j,  x_j = softcap * tanh(x_j / softcap) if softcap > 0,
 *   out = softmax(x) . V over the visible keys j < n = context_lens[b] and, if
 *   window > 0, j >= n - window,
 * with K and V the values that the codes stand for.  Scores, statistics and
 * sums are fp32; queries and weights enter the products as two fp16 numbers
 * each (good to 2^-22; what a key adds is held to 2^-30 of the largest value
 * scale among the visible keys).  The division comes after the sums, whose
 * weights are at most 2^8: values above 2^120 / n may leave fp32 on the way.
 * An empty context gives zeros.
 *   block_tables, context_lens, max_context_len as in pkv_decode_attention
 *   (the same flags; a context over the table is clamped)
 *   partition_size  0 = automatic, else a positive multiple of 128: keys per
 *                 part of the split over the context (raised where it would
 *                 give more than 256 parts); on the tensor cores the fewest
 *                 keys that a warp takes of its stretch
 *   workspace     pkv_quant_decode_workspace_size(...) bytes, 256-byte
 *                 aligned, zero-filled before its first use; every call that
 *                 completes without PKV_FLAG_TIMEOUT leaves it ready for the
 *                 next on the same stream.  Calls that may overlap need
 *                 workspaces of their own (two captured graphs that share one
 *                 must not replay at the same time).
 * Rows no query sees may hold anything, NaN included; table entries of blocks
 * that hold only such rows are not read.  A table entry outside
 * [0, num_blocks) raises PKV_FLAG_BLOCK_OUT_OF_RANGE, that sequence's output is
 * unspecified.  A visible row whose scale is NaN makes its KV head's outputs
 * NaN.  out and the workspace overlap no other argument.
 * Supported: head_dim <= 512, for INT4 even; any block size and alignment of
 * elements.  16-byte aligned codes (INT4: parameters 8-byte aligned) with
 * head_dim 64, 80, 96, 128, 192 or 256 (INT4: not 80) run a tensor-core
 * kernel, everything else the CUDA cores.  Errors: PKV_ERR_INVALID_ARG (also a
 * scale that is not finite, a softcap that is negative, not finite or too
 * small for scale / softcap), PKV_ERR_UNSUPPORTED, PKV_ERR_WORKSPACE,
 * PKV_ERR_CUDA.  B == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_quant_decode_attention(
    void *out, const void *q, const void *k_codes, const void *v_codes, const float *k_params,
    const float *v_params, const int32_t *block_tables, const int32_t *context_lens, int B, int H,
    int num_kv_heads, int head_dim, int block_size, int max_blocks, int64_t num_blocks, float scale,
    float softcap, int window, pkv_quant_format fmt, pkv_dtype dt, int max_context_len,
    int partition_size, void *workspace, size_t workspace_bytes, int *err_flags,
    pkv_stream_t stream);

/*
 * pkv_quant_decode_workspace_size -- bytes of workspace
 * pkv_quant_decode_attention needs for these sizes and for a smaller batch or
 * context length, for every format, dtype and window (host only).  Returns 0
 * for invalid sizes.
 */
PKV_API size_t pkv_quant_decode_workspace_size(int B, int H, int num_kv_heads, int head_dim,
                                               int block_size, int max_blocks, int max_context_len,
                                               int partition_size);

/*
 * pkv_beam_select -- one step of beam search: the K best continuations of each
 * request over its W beams and the vocabulary.  Beam w of request b has the
 * score c = scores[b, w] (its log-probability so far; -inf: the beam is not in
 * use) and proposes
 *   every token v with the score c + x_v - log sum_u exp(x_u), x its row of
 *   logits (a logit of -inf is no proposal), or,
 *   where finished[b, w] is not 0, itself: end_token with the score c.
 * Taken are the K best by score; of equal ones the lowest beam, then the lowest
 * token.  The order is that of the scores in 64 bits (a beam's own proposals
 * go by their logits), the sum behind the logarithm is accurate to some 1e-7
 * for finite logits of any size: they enter as differences from the row's
 * largest.
 *   scores_out    [B, K] float32; -inf where fewer than K were proposed
 *   parents       [B, K] int32: the beam that each one continues, -1 there
 *   tokens        [B, K] int32: the token it adds, -1 there
 *   finished_out  [B, K] uint8: 1 where the parent was finished or the token
 *                 is end_token; 0 there
 *   logits        [B, W, V] of dtype dt; beam row r = b * W + w at element
 *                 r * row_stride; rows of finished and unused beams are not read
 *   finished      [B, W] uint8 or NULL (none is)
 *   end_token     the token that ends a sequence, or -1
 * A beam whose logits hold a NaN or +inf, or whose score is NaN or +inf,
 * raises PKV_FLAG_LOGITS and proposes nothing.
 *   workspace     pkv_beam_select_workspace_size(...) bytes, 256-byte aligned,
 *                 zero-filled before its first use; every call leaves it ready
 *                 for the next of any sizes on the same stream.  Calls that may
 *                 overlap need workspaces of their own.
 * scores_out may be scores and finished_out finished where K == W; no other
 * written array overlaps another argument.  Supported: W, K <= 32, B <= 16384,
 * V <= 2^21, any alignment of elements (rows that are 16-byte aligned are
 * fastest).  Errors: PKV_ERR_INVALID_ARG, PKV_ERR_UNSUPPORTED,
 * PKV_ERR_WORKSPACE, PKV_ERR_CUDA.  B == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_beam_select(float *scores_out, int32_t *parents, int32_t *tokens,
                                   uint8_t *finished_out, const void *logits, const float *scores,
                                   const uint8_t *finished, int B, int W, int K, int64_t V,
                                   int64_t row_stride, int end_token, pkv_dtype dt,
                                   void *workspace, size_t workspace_bytes, int *err_flags,
                                   pkv_stream_t stream);

/* Bytes of workspace pkv_beam_select needs for these sizes and for smaller B,
 * W, K and V, for every dtype (host only); 0 for invalid sizes. */
PKV_API size_t pkv_beam_select_workspace_size(int B, int W, int K, int64_t V);

/*
 * pkv_beam_reorder -- the paged cache follows the beams that were chosen:
 * child k of request b continues beam parents[b, k] (-1: none).  Full blocks
 * are shared by naming them in both tables; a last block that is not full goes
 * to the first child that has it, and every other one gets a block of the
 * request's own and a copy of its rows, so that no two beams ever write the
 * same block.
 *   tables        [B, W, max_blocks] int32: the beams' block tables
 *   lens          [B, W] int32: their tokens in the cache
 *   parents       [B, K] int32, as from pkv_beam_select
 *   owned         [B, K, max_blocks] int32: for every column behind the
 *                 prompt's full blocks K blocks that are this request's alone,
 *                 reserved when it was admitted (the prompt's last block, if
 *                 not full, may be one of them)
 *   finished      [B, K] uint8 or NULL: children that get no further token
 *   tables_out    [B, K, max_blocks] int32
 *   lens_out      [B, K] int32: lens with the next token counted
 *   slots         [B, K] int64: the next token's slot, for the write; -1 for
 *                 finished and unused children, whose length stays
 * With n a child's length and c = n / block_size: columns before c are its
 * parent's; column c is its parent's block if n is not a multiple of
 * block_size and no child before it continues in that block and no other child
 * holds it whole; else, children in order, owned[b, k, c] or, where that is in
 * use in this column, the first of owned[b, :, c] that is not, with the
 * n % block_size rows copied; columns behind c are owned[b, k].
 *   num_pools     caches to copy in, 0 .. 256: K and V of every layer, quantised
 *                 ones with their parameters
 *   pools         HOST array of device pointers, each to num_blocks blocks
 *   block_bytes   HOST array: bytes of a block of each
 *   row_bytes     HOST array: bytes of one token where a block is its tokens'
 *                 rows one after the other, or 0: the block is copied whole
 *                 (quantisation parameters)
 * A parent outside [-1, W) or a length outside [0, max_blocks * block_size]
 * raises PKV_FLAG_BEAM, the child is then unused; a child without room for a
 * token raises PKV_FLAG_CONTEXT_TOO_LONG (slot -1, length unchanged); a
 * block outside [0, num_blocks) where one is written or copied raises
 * PKV_FLAG_BLOCK_OUT_OF_RANGE, and no block left PKV_FLAG_OUT_OF_BLOCKS: in
 * both cases the child's slot is -1, its length stays and nothing is copied
 * for it.
 * No written array overlaps another argument, nor pools one another.
 * Supported: W, K <= 32, B <= 16384.  Errors: PKV_ERR_INVALID_ARG,
 * PKV_ERR_UNSUPPORTED, PKV_ERR_CUDA.  B == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_beam_reorder(int32_t *tables_out, int32_t *lens_out, int64_t *slots,
                                    const int32_t *tables, const int32_t *lens,
                                    const int32_t *parents, const int32_t *owned,
                                    const uint8_t *finished, int B, int W, int K, int max_blocks,
                                    int64_t num_blocks, int block_size, int num_pools,
                                    void *const *pools, const int64_t *block_bytes,
                                    const int64_t *row_bytes, int *err_flags, pkv_stream_t stream);

/*
 * The layout experiment: vLLM's packed cache layout, which the interview
 * note "PagedAttention kernel: paged KV cache 与 block table" describes in
 * section 深入原理 (K cache [num_blocks, num_kv_heads, head_size / x,
 * block_size, x] with x = 16 / element size so that loads are aligned
 * 16-byte vectors; V cache [num_blocks, num_kv_heads, head_size,
 * block_size]).  For 16-bit types x = 8:
 *   k_cache_x[blk][kvh][d / 8][off][d % 8],   v_cache_x[blk][kvh][d][off]
 * holding the same values as the token-major caches of pkv_write /
 * pkv_decode_attention.  Only block_size 16, bf16 / fp16.  The library's
 * main path keeps the token-major layout; these two calls exist to measure
 * the difference (one contiguous copy per (block, KV head) instead of
 * head_dim / 64 tiled boxes).
 *
 * pkv_write_xpacked -- pkv_write into the packed layout (same arguments and
 * errors; block_size must be 16, head_dim a multiple of 8, k and the
 * caches 16-byte aligned, token strides multiples of 8 elements).
 * pkv_decode_attention_xpacked -- pkv_decode_attention over packed caches
 * (same arguments, workspace and errors, out in device memory; head_dim 64,
 * 128 or 256; returns PKV_ERR_UNSUPPORTED for other shapes and for fp32).
 */
PKV_API pkv_status pkv_write_xpacked(void *k_cache_x, void *v_cache_x, const void *k, const void *v,
                                     const int64_t *slot_mapping, int64_t num_tokens,
                                     int64_t k_token_stride, int64_t v_token_stride,
                                     int64_t num_blocks, int block_size, int num_kv_heads,
                                     int head_dim, pkv_dtype dt, int *err_flags,
                                     pkv_stream_t stream);
PKV_API pkv_status pkv_decode_attention_xpacked(
    void *out, const void *q, const void *k_cache_x, const void *v_cache_x,
    const int32_t *block_tables, const int32_t *context_lens, int B, int H, int num_kv_heads,
    int head_dim, int block_size, int max_blocks, int64_t num_blocks, float scale, pkv_dtype dt,
    int max_context_len, int partition_size, void *workspace, size_t workspace_bytes,
    int *err_flags, pkv_stream_t stream);

/*
 * pkv_decode_plan -- the partition size and the partitions per sequence that
 * pkv_decode_attention would use for these arguments on a GPU with
 * num_sms SMs (host only, no CUDA call; for tests and tuning; on the
 * wide-group kernel with partition_size 0, the floor of its item size and
 * the most partitions a sequence can have).  Returns the
 * partition size in tokens (>= 16), or 0 for invalid sizes; *kernel is set to
 * 2 for the wide-group tensor-core kernel, 1 for the TMA + mma.sync
 * tensor-core kernel, 0 for the CUDA-core kernel.
 */
PKV_API int pkv_decode_plan(int B, int H, int num_kv_heads, int head_dim, int block_size,
                            int max_blocks, int max_context_len, int partition_size,
                            pkv_dtype dt, int num_sms, int *max_partitions, int *kernel);

/*
 * pkv_hbm_copy -- a plain streaming copy of `bytes` bytes from src to dst
 * (device pointers, 16-byte aligned, bytes a multiple of 16, the ranges
 * not overlapping), enqueued on `stream`.  It is the yardstick the other
 * kernels are measured against: the HBM bandwidth a copy reaches on this
 * GPU (2 * bytes of traffic per call), taken in the same run.  The pages
 * have no counterpart.  Errors: PKV_ERR_INVALID_ARG (alignment, size,
 * overlap, NULL), PKV_ERR_CUDA.  bytes == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_hbm_copy(void *dst, const void *src, size_t bytes, pkv_stream_t stream);

/*
 * pkv_hbm_gather_read -- reads nchunks chunks of chunk_bytes bytes, chunk i
 * starting at base + chunk_index[i] * chunk_stride_bytes (device pointers;
 * base 16-byte aligned, chunk_bytes and chunk_stride_bytes multiples of 16;
 * every chunk inside the caller's buffer -- the indices are not checked),
 * and XORs the 16-byte words read into *sink (a device uint64; the XOR of
 * the two 64-bit halves of every word, folded in, so no read is dead).  The
 * yardstick for the decode kernels' access pattern: the bandwidth reads of
 * randomly placed whole cache blocks reach on this GPU (bytes read =
 * nchunks * chunk_bytes), taken in the same run.  The pages have no
 * counterpart.  Errors: PKV_ERR_INVALID_ARG, PKV_ERR_CUDA.  nchunks == 0 or
 * chunk_bytes == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_hbm_gather_read(const void *base, const int32_t *chunk_index,
                                       int64_t nchunks, int64_t chunk_stride_bytes,
                                       int64_t chunk_bytes, unsigned long long *sink,
                                       pkv_stream_t stream);

/*
 * pkv_hbm_gather_read_pair -- the same reads over two buffers in one launch:
 * every listed chunk of base_a, then every listed chunk of base_b (both
 * 16-byte aligned, both holding every listed chunk), all folded into
 * *sink.  Bytes read = 2 * nchunks * chunk_bytes.  The decode reads a
 * batch's K and V blocks in one launch; so does this yardstick (two
 * launches of half the size each pay their own ramp and tail).  Errors:
 * PKV_ERR_INVALID_ARG (as pkv_hbm_gather_read, or base_b NULL), PKV_ERR_CUDA.
 */
PKV_API pkv_status pkv_hbm_gather_read_pair(const void *base_a, const void *base_b,
                                            const int32_t *chunk_index, int64_t nchunks,
                                            int64_t chunk_stride_bytes, int64_t chunk_bytes,
                                            unsigned long long *sink, pkv_stream_t stream);

/*
 * pkv_fp32_fma_peak -- the CUDA-core yardstick: `blocks` blocks of 256
 * threads, each thread running eight independent fp32 multiply-add chains
 * x <- x * a + b from x = 0 for `iters` steps (fmaf, or with paired != 0 the
 * two-lane fma.rn.f32x2 on four pairs): 2 * 8 * iters flops per thread.
 * Thread 0 of block i stores the sum of its chains in out[i] (device
 * float[blocks]); any other thread stores it only if it equals `never`, so
 * no chain is dead code (pass a value no sum reaches).  With a = b = 1 every
 * chain ends at exactly iters (iters < 2^24), which makes the result
 * checkable.  The fp32 rate the CUDA cores reach in the same run, against
 * which a decode's arithmetic (2 * G * D flops per key and per value row of
 * D elements) is set when choosing tensor cores for a group of G query
 * heads.  The pages have no counterpart.  Errors: PKV_ERR_INVALID_ARG
 * (out NULL or not 4-byte aligned, blocks < 1 or > 2^20, iters < 0),
 * PKV_ERR_CUDA.
 */
PKV_API pkv_status pkv_fp32_fma_peak(float *out, int blocks, int iters, float a, float b,
                                     float never, int paired, pkv_stream_t stream);

/*
 * pkv_copy_async -- enqueues one copy of `bytes` bytes from src to dst on
 * `stream`, between any two memories the GPU addresses (device memory,
 * pinned or pageable host memory; the runtime tells which from the
 * pointers).  It is how a serving loop built on this library moves a step's
 * staged inputs in and its output out around a prepared step call, one
 * call per copy, without a framework's tensor copy in between.  The ranges
 * must not overlap.  Pinned host memory gives an asynchronous copy;
 * pageable host memory is staged by the runtime and may return only once
 * the copy is done.  Errors: PKV_ERR_INVALID_ARG (dst or src NULL with
 * bytes > 0, overlapping ranges), PKV_ERR_CUDA (the runtime refused the
 * copy).  bytes == 0 enqueues nothing.
 */
PKV_API pkv_status pkv_copy_async(void *dst, const void *src, size_t bytes, pkv_stream_t stream);

/* A static, human-readable name for a status code. */
PKV_API const char *pkv_status_string(pkv_status status);

/* Version string of the library build. */
PKV_API const char *pkv_version(void);

#ifdef __cplusplus
}
#endif

#endif /* PKV_H */
