/*
 * attn.h -- C ABI of libattn.so: exact tiled attention with an online softmax
 * on NVIDIA GB300 (sm_103a).
 *
 * The operations (definitions from the pages this library implements):
 *
 *   attention of a query row over the keys it may see --
 *     "Why your local LLM feels dumber than it is" (Part 3.14), section
 *     "What attention is trying to calculate": score_t = scale * dot(q, k_t),
 *     weights exp(score_t) normalised over the visible tokens, output the
 *     weighted sum of the values.
 *
 *   tiled prefill with a running max and running sum --
 *     "Streaming process -- How the SM works inside a transformer", Steps 3-8
 *     and its code snippet.
 *
 *   split-KV decode over a paged cache and the merge of per-group partials --
 *     "GPU Datapath: Where Every Byte Moves in One LLM Inference Step",
 *     section D "Paged decode attention -- the zero-reuse stream", and
 *     "Why your local LLM feels dumber than it is", sections "Why the
 *     calculation is split into groups" and "Backend names expand into four
 *     decode algorithms".
 *
 * Conventions for every entry point:
 *   - Tensor pointers are DEVICE pointers (CUDA global memory of the current
 *     device), 16-byte aligned, densely packed in the layout stated, except
 *     the host pointers of attn_prefill_host.  bf16 is
 *     IEEE bfloat16 (2 bytes); LSE values are float32 natural logarithms of
 *     the sum of exp(scaled scores).
 *   - `stream` is a cudaStream_t passed as an opaque pointer (NULL = legacy
 *     default stream).  Kernels are enqueued on it and run asynchronously;
 *     outputs are valid once the stream reaches that point.
 *   - The caller owns all memory.  The library allocates nothing on the
 *     device and keeps no per-call state (attn_prefill_host keeps two copy
 *     streams per device; attn_decode_paged_noalloc uses a fixed array inside
 *     the library).  Argument errors are detected on the host before
 *     anything is enqueued and leave the outputs untouched.
 *   - Grouped-query attention: Hq must be a multiple of Hkv; query head h uses
 *     KV head h / (Hq / Hkv).
 *   - Return value: ATTN_OK, or one of the error codes below.  No exception
 *     crosses the ABI.  Errors detected by a kernel while it runs (a wait that
 *     timed out, a block-table entry out of range) are recorded in a device
 *     status word that attn_device_status() reads.
 */
#ifndef ATTN_H_
#define ATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  ATTN_OK = 0,
  ATTN_ERR_INVALID_ARG = 1, /* null pointer, bad shape, misalignment, Hq % Hkv != 0 */
  ATTN_ERR_UNSUPPORTED = 2, /* a head dim or option this build has no kernel for */
  ATTN_ERR_WORKSPACE = 3,   /* decode workspace missing or too small */
  ATTN_ERR_CUDA = 4,        /* a CUDA runtime/driver call or kernel launch failed */
  ATTN_ERR_DEVICE = 5       /* a kernel recorded an error (see attn_device_status) */
} attn_status_t;

/* Human-readable name of a status code (static string, never NULL). */
const char* attn_status_string(attn_status_t status);

/*
 * Prefill forward.
 *   q   [B, S, Hq,  d] bf16      k, v [B, S, Hkv, d] bf16
 *   o   [B, S, Hq,  d] bf16 (output)
 *   lse [B, Hq, S]     f32 (output, may be NULL)
 *   d in {64, 128, 256}; B, S >= 1; Hq, Hkv >= 1 with Hq % Hkv == 0.  d = 256
 *   uses 64-key tiles (the rest 128-key tiles).
 *   scale: multiplier of q.k (for example 1/sqrt(d)); finite and > 0, else
 *   ATTN_ERR_INVALID_ARG (the kernels keep the row maximum in unscaled units
 *   and mask keys with -inf before scaling).  The same holds for every entry
 *   point below that takes a scale.
 *   causal != 0: row i sees keys 0..i (itself included); causal == 0: all S keys.
 * Row i of o is sum_j softmax_j(scale * q_i.k_j) v_j over the visible keys;
 * lse[b, h, i] = ln sum_j exp(scale * q_i.k_j).
 * Arithmetic: bf16 inputs, f32 scores and accumulators, the probabilities
 * rounded to bf16 for P.V while the normaliser sums the unrounded f32 values,
 * output rounded to bf16 (nearest even).
 */
attn_status_t attn_prefill(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq,
                           int Hkv, int S, int d, float scale, int causal, void* stream);

/*
 * Prefill forward over packed sequences of different lengths: the varlen
 * attention call that "GPU Datapath: Where Every Byte Moves in One LLM
 * Inference Step", section "Measuring the Real Kernels, One at a Time", says
 * its attention cells dispatch (cumulative sequence offsets, one packed token
 * dimension).
 *   q, o       [total_tokens, Hq,  d] bf16 (o is output)
 *   k, v       [total_tokens, Hkv, d] bf16
 *   cu_seqlens [num_seqs + 1] int32, DEVICE memory: sequence n holds tokens
 *              cu_seqlens[n] .. cu_seqlens[n+1]-1; cu_seqlens[0] = 0,
 *              non-decreasing, cu_seqlens[num_seqs] <= total_tokens.
 *   max_seqlen upper bound of every sequence length (host value; sizes the
 *              work list).
 *   lse        [Hq, total_tokens] f32 (output, may be NULL).
 * Each sequence is attended on its own, exactly as attn_prefill does for one
 * batch element (causal positions counted from the sequence's first token).
 * Rows of o that belong to no sequence are not written.  A zero-length
 * sequence has no rows.  A cu_seqlens entry that breaks the rules above is
 * recorded as device status 5 and that sequence is skipped.
 * d, Hq, Hkv, scale, causal and the arithmetic are as for attn_prefill.
 */
attn_status_t attn_prefill_varlen(const void* q, const void* k, const void* v, void* o, float* lse,
                                  const int32_t* cu_seqlens, int num_seqs, int max_seqlen, int total_tokens, int Hq,
                                  int Hkv, int d, float scale, int causal, void* stream);

/*
 * Chunked prefill against the paged KV cache: the new tokens of each
 * sequence attend to all of its cached tokens (their own K/V already
 * appended to the cache) -- the prefill form of the varlen call with a block
 * table that "GPU Datapath: Where Every Byte Moves in One LLM Inference
 * Step", section "Measuring the Real Kernels, One at a Time", dispatches.
 *   q, o         [total_q, Hq, d] bf16: the new tokens of every sequence,
 *                back to back (o is output)
 *   k_cache,
 *   v_cache      [num_blocks, page_size, Hkv, d] bf16, as for
 *                attn_decode_paged
 *   block_table  [num_seqs, max_blocks_per_seq] int32, DEVICE memory
 *   cu_seqlens_q [num_seqs + 1] int32, DEVICE memory: sequence n's new
 *                tokens are q rows cu_seqlens_q[n] .. cu_seqlens_q[n+1]-1
 *   seq_lens     [num_seqs] int32, DEVICE memory: cached tokens of sequence
 *                n, its new tokens included (they are the last ones)
 *   lse          [Hq, total_q] f32 (output, may be NULL)
 *   max_seqlen_q upper bound of the new tokens per sequence (host value)
 *   d in {64, 128, 256}; page_size == 16.
 * New token i of sequence n sits at position seq_lens[n] - q_len + i; with
 * causal != 0 it sees the keys at positions 0 .. that position, otherwise all
 * seq_lens[n] keys.  Tokens of the last page past seq_len are never used,
 * even if they hold NaN.  A sequence whose offsets break the rules of
 * attn_prefill_varlen or whose seq_len is below its new tokens or beyond its
 * block-table row is recorded as device status 5 and skipped; a block-table
 * entry outside [0, num_blocks) as status 2 (page 0 is read instead).
 * Arithmetic as for attn_prefill.
 */
attn_status_t attn_prefill_paged(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                 const int32_t* cu_seqlens_q, const int32_t* seq_lens, void* o, float* lse,
                                 int num_seqs, int max_seqlen_q, int total_q, int Hq, int Hkv, int d, int page_size,
                                 int max_blocks_per_seq, int num_blocks, float scale, int causal, void* stream);

/*
 * Causal (or full) prefill of one sequence whose inputs and outputs are in
 * HOST memory, with the transfers inside the call.  The attention is that of
 * attn_prefill with B = 1 ("Why your local LLM feels dumber than it is" (Part
 * 3.14), section "What attention is trying to calculate"); the queries are
 * cut into `chunks` runs of ceil(S / chunks) rows.  Row i only sees keys
 * 0 .. i, so a chunk needs only the keys up to its own last row: each chunk
 * runs as one chunked prefill (attn_prefill_paged, the keys and values seen
 * as a paged cache with an identity block table) as soon as its rows are
 * on the device, while the next chunk is copied in and the previous one
 * copied out.  With causal == 0 every row sees all S keys: all of k and v
 * are copied in before the first chunk, and only the queries and outputs
 * are pipelined.
 *   q_host        [S, Hq, d] bf16, host memory
 *   k_host,
 *   v_host        [S, Hkv, d] bf16, host memory
 *   o_host        [S, Hq, d] bf16, host memory (output)
 *   lse_host      [Hq, S] f32, host memory (output, may be NULL)
 *   chunks        1 .. 64
 *   workspace     DEVICE memory, 256-byte aligned, of at least
 *                 attn_prefill_host_workspace_bytes(S, Hq, Hkv, d, chunks)
 *                 bytes: the device copies of q, k, v, o and LSE, the
 *                 block table and the chunks' offsets.  It must not be in use
 *                 by other work until the call's work on `stream` is done.
 * Host buffers should be page-locked (cudaHostAlloc or cudaHostRegister): the
 * copies then run asynchronously and overlap.  Pageable memory gives the
 * same results, but its copies stop the calling thread and do not overlap.
 * The chunks' prefills run on `stream`; the copies run on two streams the
 * library creates once per device (with four events) and keeps for the life
 * of the process: the only state the library keeps between calls.  The copies
 * start after the work enqueued on `stream` before the call, and work
 * enqueued on `stream` after the call starts after the last copy out, so the
 * host outputs are complete once `stream` reaches that point (for example
 * after cudaStreamSynchronize(stream)).  Enqueueing is serialised across host
 * threads.
 * Errors: argument errors (d, Hq, Hkv, S, chunks, scale, NULL pointers, an
 * unaligned or too small workspace) return before anything is enqueued; a
 * CUDA error while enqueueing returns ATTN_ERR_CUDA with part of the work
 * enqueued and the outputs undefined.
 * Arithmetic as for attn_prefill; every output equals that of attn_prefill on
 * the same sequence.
 */
attn_status_t attn_prefill_host(const void* q_host, const void* k_host, const void* v_host, void* o_host,
                                float* lse_host, int S, int Hq, int Hkv, int d, float scale, int causal, int chunks,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Workspace bytes attn_prefill_host needs; 0 for invalid arguments. */
size_t attn_prefill_host_workspace_bytes(int S, int Hq, int Hkv, int d, int chunks);

/*
 * Number of partial slots per (sequence, query head) that attn_decode_paged
 * uses for the given split settings (1 means the split kernel writes the
 * output directly and needs no workspace).
 *   split_tokens > 0: groups of split_tokens tokens (must be a multiple of
 *     page_size); slots = ceil(max_blocks_per_seq * page_size / split_tokens).
 *   split_tokens == 0: num_splits (>= 1) groups per sequence.
 * Returns 0 for invalid arguments.
 */
int attn_decode_num_slots(int max_blocks_per_seq, int page_size, int num_splits, int split_tokens);

/*
 * Split-count rule of "Why your local LLM feels dumber than it is" (Part
 * 3.14), section "Why FlashAttention 2 selects 54, 62, or 87 groups": among
 * c = 1 .. min(max_splits, capacity, blocks), a count is a candidate when it
 * changes ceil(blocks / c) compared with c - 1 (c = 1 always is); its
 * estimated efficiency is w / ceil(w) with w = units * c / capacity; the
 * smallest candidate whose efficiency is at least 85% of the best one wins.
 *   units      independent work items per split (sequences x KV heads)
 *   capacity   work items the device runs at once
 *   blocks     key/value blocks of the longest sequence
 * Pure host arithmetic (no CUDA call).  With units = 4, capacity = 2 x SMs and
 * blocks = 431 it gives the page's 54 / 62 / 87 for 132 / 148 / 188 SMs.
 * Returns 0 for invalid arguments.
 */
int attn_split_heuristic(int units, int capacity, int blocks, int max_splits);

/*
 * The same rule restated for this library's split kernel on the current
 * device: units = num_seqs * Hkv, capacity = SMs x resident split-kernel CTAs
 * per SM, blocks = max_blocks_per_seq (16-token pages), at most 128 splits.
 * Pass the result as num_splits to attn_decode_paged (and to
 * attn_decode_num_slots for the workspace size).  Returns 0 for invalid
 * arguments or when no CUDA device can be queried.
 */
int attn_decode_auto_splits(int num_seqs, int Hkv, int d, int max_blocks_per_seq);

/*
 * Length-aware group size for attn_decode_paged (pass the result as
 * split_tokens).  The rule of "Why your local LLM feels dumber than it is"
 * (Part 3.14), section "Why FlashAttention 2 selects 54, 62, or 87 groups",
 * sizes every sequence's groups from the longest one; with mixed lengths that
 * leaves long groups on the long sequences and short ones on the rest.  This
 * rule instead gives every group the same number of pages s, so a sequence's
 * group count is proportional to its length (ceil(pages_n / s)):
 *   items(s) = Hkv * sum_n ceil(pages_n / s) groups, capacity = CTAs the
 *   device runs at once;
 *   one wave: s1 is the smallest page count with items(s1) <= capacity, but
 *   at least 32 pages (512 tokens) or the longest sequence's page count if
 *   that is smaller; it is taken when such a count exists and its groups are
 *   near-equal, i.e. 4 * s1 * capacity <= 5 * (total pages * Hkv), or s1 is
 *   that lower bound;
 *   otherwise (several waves): s is the largest power of two that is at most
 *   max(32, total pages * Hkv / (3 * capacity)), capped by the longest
 *   sequence (about three waves of equal groups).
 *   seq_lens   host array [num_seqs] of the lengths the decode will see
 *              (entries are clamped to [0, max_blocks_per_seq * 16]).
 * Returns s * 16 (a multiple of page_size = 16), or 0 for invalid arguments.
 * attn_split_tokens_rule is the pure host arithmetic with an explicit
 * capacity; attn_decode_auto_split_tokens applies it on the current device
 * (capacity = SMs x resident split-kernel CTAs per SM) and also returns 0 when
 * no CUDA device can be queried.
 */
int attn_split_tokens_rule(const int32_t* seq_lens, int num_seqs, int Hkv, int capacity, int max_blocks_per_seq);
int attn_decode_auto_split_tokens(const int32_t* seq_lens, int num_seqs, int Hkv, int d, int max_blocks_per_seq);

/*
 * Bytes of workspace attn_decode_paged needs: num_seqs * Hq * slots * (d + 2)
 * floats when slots > 1, else 0.
 */
size_t attn_decode_workspace_bytes(int num_seqs, int Hq, int d, int slots);

/*
 * Bytes of workspace attn_decode_paged needs in balanced mode (num_splits == 0
 * and split_tokens == 0) on the current device:
 * (worker warps + Hkv * num_seqs) * (Hq / Hkv) * (d + 2) floats, where the
 * number of worker warps follows the device's SM count.  Returns 0 for
 * invalid arguments or when no CUDA device can be queried.
 */
size_t attn_decode_balanced_workspace_bytes(int num_seqs, int Hq, int Hkv, int d);

/*
 * Single-token decode over a paged KV cache, split over the context.
 *   q            [num_seqs, Hq, d] bf16
 *   k_cache,
 *   v_cache      [num_blocks, page_size, Hkv, d] bf16: physical pages of
 *                page_size consecutive token rows
 *   block_table  [num_seqs, max_blocks_per_seq] int32: physical page of each
 *                logical page (entries past a sequence's last page are ignored)
 *   seq_lens     [num_seqs] int32, 0 <= len <= max_blocks_per_seq * page_size
 *   o            [num_seqs, Hq, d] bf16 (output)
 *   lse          [num_seqs, Hq] f32 (output, may be NULL)
 *   d in {128, 256}; page_size == 16.
 *   Splits: contiguous, page-aligned groups of tokens -- split_tokens per
 *   group if split_tokens > 0, else ceil(pages / num_splits) pages per group.
 *   Each group gives a partial (normalised f32 output, max, sum); when there
 *   is more than one slot the partials go to `workspace` and a second kernel
 *   merges them (same arithmetic as attn_combine).
 *   workspace: device buffer of at least attn_decode_workspace_bytes(...)
 *   bytes (may be NULL when that is 0).
 *   Balanced mode (num_splits == 0 and split_tokens == 0): the pages of all
 *   sequences and KV heads form one list, and every worker warp of a grid
 *   sized to the device takes an equal contiguous share of it, whatever the
 *   mix of lengths; each share yields one partial per (sequence, KV head) it
 *   touches and a second kernel merges them.  Needs
 *   attn_decode_balanced_workspace_bytes(...) bytes of workspace.
 * The query sees all seq_len tokens.  A sequence with seq_len == 0 gets o = 0
 * and lse = -inf.  Tokens of the last page past seq_len are never used, even
 * if they hold NaN.  A block-table entry outside [0, num_blocks) is recorded
 * as ATTN_ERR_DEVICE (page 0 is read instead).
 */
attn_status_t attn_decode_paged(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_table,
                                const int32_t* seq_lens, void* o, float* lse, int num_seqs, int Hq, int Hkv, int d,
                                int page_size, int max_blocks_per_seq, int num_blocks, int num_splits,
                                int split_tokens, float scale, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * Paged decode that allocates nothing.  The pages have no counterpart to
 * this entry point: it exists for callers that cannot provide a workspace,
 * such as a plugin inside a host framework that owns all device memory and
 * hands out no scratch buffers, or a serving loop that forbids device
 * allocations once it has started.
 *   Arguments, layouts, results and errors are those of attn_decode_paged
 *   (balanced mode included), without workspace / workspace_bytes: the
 *   partials live in a fixed array of ATTN_DECODE_NOALLOC_SCRATCH_BYTES
 *   inside the library's own device memory, present on every device that
 *   loads the library until the process exits.  No cudaMalloc, cudaFree or
 *   other allocating call is made.  The array is passed to attn_decode_paged
 *   as a workspace of that many bytes, so argument errors are reported first,
 *   and a call whose partials need more (attn_decode_workspace_bytes, or
 *   attn_decode_balanced_workspace_bytes in balanced mode) returns
 *   ATTN_ERR_WORKSPACE and enqueues nothing.
 *   The first call on a device looks up the array's device address (once per
 *   device, with that device current) and keeps it; make that first call
 *   before any stream capture.  The kept address belongs to the device's
 *   primary context: do not reset the device (cudaDeviceReset) while the
 *   library is in use, nor call it from another context on the same device.
 *   All calls share the array: calls whose work overlaps on the GPU (other
 *   streams, other host threads) race on it.  Every partial a call reads was
 *   written earlier in the same call, so leftovers of earlier calls are
 *   harmless.
 */
#define ATTN_DECODE_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
attn_status_t attn_decode_paged_noalloc(const void* q, const void* k_cache, const void* v_cache,
                                        const int32_t* block_table, const int32_t* seq_lens, void* o, float* lse,
                                        int num_seqs, int Hq, int Hkv, int d, int page_size, int max_blocks_per_seq,
                                        int num_blocks, int num_splits, int split_tokens, float scale, void* stream);

/*
 * Merge per-group partials ("Why your local LLM feels dumber than it is",
 * section "Backend names expand into four decode algorithms": normalised
 * group outputs merged by their log-sum statistics).
 *   part_o [rows, num_splits, d] f32: normalised output of each group
 *   part_m [rows, num_splits]    f32: max scaled score of the group (-inf if empty)
 *   part_l [rows, num_splits]    f32: sum of exp(score - part_m) (0 if empty)
 *   rows = num_seqs * Hq.
 *   o   [rows, d] bf16 = sum_i w_i part_o_i / sum_i w_i, w_i = part_l_i exp(part_m_i - M),
 *       M = max over non-empty groups; groups with part_l <= 0 carry no weight.
 *   lse [rows] f32 (may be NULL) = M + ln sum_i w_i.  A row with no
 *       non-empty group gets o = 0 and lse = -inf.
 *   d in {64, 128, 256}.
 */
attn_status_t attn_combine(const float* part_o, const float* part_m, const float* part_l, int rows,
                           int num_splits, int d, void* o, float* lse, void* stream);

/*
 * Decode numerics of other backends ("Why your local LLM feels dumber than it
 * is" (Part 3.14), section "Backend names expand into four decode
 * algorithms").  Each backend splits the context into groups in its own way,
 * stores its own per-group value and merges the groups in its own float32
 * order:
 *   ATTN_NUMERICS_TRITON  `partitions` contiguous groups of whole 16-token
 *       tiles (ceil(pages / partitions) pages each; the page's Triton uses
 *       16); stores the float32 weighted-value sum; merge: c_i = exp(m_i - M),
 *       M = max m_i, L = sum l_i c_i, N = sum n_i c_i, out = N / L.
 *   ATTN_NUMERICS_FA2     `partitions` contiguous groups of whole 64-token
 *       blocks (ceil(blocks / partitions) blocks each); stores the float32
 *       normalised output; merge: lse_i = m_i + log l_i, w_i =
 *       exp(lse_i - max lse), out = sum o_i w_i / sum w_i.
 *   ATTN_NUMERICS_XQA     256-token tiles dealt round-robin over
 *       `partitions` groups (group p takes tiles p, p + partitions, ...); the
 *       sum of weights adds the bf16-rounded weights; stores the normalised
 *       output rounded to bf16; merge: w_i = l_i exp(m_i - M),
 *       out = sum o_i w_i / sum w_i.
 *   ATTN_NUMERICS_TRT     one group per 128-token tile (`partitions` is not
 *       used); stores the weighted-value sum rounded to bf16; merge: the
 *       groups one after another, with a running max M' = max(M, m_i),
 *       L = L exp(M - M') + l_i exp(m_i - M'), and likewise for N;
 *       out = N / L.
 * Inside a group the weights are exp(score - group max), and the
 * weighted-value sum multiplies the values by the bf16-rounded weights.  The
 * merges run in group order, with each float32 add, multiply and divide
 * rounded on its own (no fused multiply-add).  exp and log are evaluated in
 * double precision and rounded once to float32.  The group arithmetic itself
 * runs on tensor cores, whose sums have their own order: the emulation holds
 * the geometry, the stored types and the merge order, not the bits of every
 * partial.
 */
typedef enum {
  ATTN_NUMERICS_TRITON = 1,
  ATTN_NUMERICS_FA2 = 2,
  ATTN_NUMERICS_XQA = 3,
  ATTN_NUMERICS_TRT = 4
} attn_numerics_t;

/*
 * Group count that the backend would pick for a batch of num_seqs sequences
 * with Hkv KV heads, the longest max_tokens long, on a GPU of sm_count SMs
 * (pure host arithmetic):
 *   TRITON  16;
 *   FA2     attn_split_heuristic(num_seqs * Hkv, 2 * sm_count,
 *           ceil(max_tokens / 64), 128), which gives the page's 54 / 62 / 87
 *           for 132 / 148 / 188 SMs at 27,525 tokens and 4 KV heads;
 *   XQA     min(max(1, sm_count / (num_seqs * Hkv)), ceil(max_tokens / 256)):
 *           the page's 33 on H200 (132 SMs) and 47 on SM120 (188 SMs);
 *   TRT     ceil(max_tokens / 128), the number of its 128-token groups.
 * Returns 0 for invalid arguments.
 */
int attn_emulated_partitions(int numerics, int num_seqs, int Hkv, int max_tokens, int sm_count);

/*
 * Partial slots per (sequence, query head): `partitions` (1 .. 65535) for
 * TRITON, FA2 and XQA; ceil(max_blocks_per_seq * page_size / 128) for TRT.
 * Returns 0 for invalid arguments (page_size must be 16).
 */
int attn_emulated_num_slots(int numerics, int max_blocks_per_seq, int page_size, int partitions);

/* Workspace bytes of attn_decode_paged_emulated: num_seqs * Hq * slots * (d + 2) floats. */
size_t attn_emulated_workspace_bytes(int num_seqs, int Hq, int d, int slots);

/*
 * Paged decode with the numerics of another backend.  Arguments, layouts and
 * errors are those of attn_decode_paged, with `numerics` and `partitions` (as
 * above) in place of num_splits / split_tokens.  It always writes partials and
 * merges them, even with one group.  The workspace (at least
 * attn_emulated_workspace_bytes(num_seqs, Hq, d, slots) bytes, 16-byte
 * aligned) holds, after the call:
 *   part_o [num_seqs * Hq, slots, d] f32  the stored value of each group
 *   part_m [num_seqs * Hq, slots]    f32  group max of the scaled scores
 *   part_l [num_seqs * Hq, slots]    f32  group sum of weights
 * in that order.  An empty group has m = -inf, l = 0 and part_o = 0.
 * o [num_seqs, Hq, d] bf16 is the merged output rounded to bf16.  lse (may be
 * NULL) is the merge's largest max (FA2: log-sum) plus log of its merged sum.
 */
attn_status_t attn_decode_paged_emulated(const void* q, const void* k_cache, const void* v_cache,
                                         const int32_t* block_table, const int32_t* seq_lens, void* o, float* lse,
                                         int num_seqs, int Hq, int Hkv, int d, int page_size, int max_blocks_per_seq,
                                         int num_blocks, int numerics, int partitions, float scale, void* workspace,
                                         size_t workspace_bytes, void* stream);

/*
 * The backend's merge alone, on caller-supplied partials in the layout above:
 *   part_o [rows, num_splits, d] f32, part_m / part_l [rows, num_splits] f32
 *   (a slot with part_l <= 0 is empty and skipped);
 *   o_f32 [rows, d] f32 (may be NULL): the float32 result before the final rounding;
 *   o     [rows, d] bf16 (may be NULL, not both): that result rounded to bf16;
 *   lse   [rows] f32 (may be NULL).
 * A row with no non-empty slot gets 0 and lse = -inf.  1 <= d <= 1024.
 */
attn_status_t attn_merge_emulated(int numerics, const float* part_o, const float* part_m, const float* part_l,
                                  int rows, int num_splits, int d, float* o_f32, void* o, float* lse, void* stream);

/*
 * ---- The serving step around the attention calls.
 *
 * A step of a serving program: attn_step_tables turns request lengths into
 * block tables, positions and slots; attn_qk_norm_rope prepares queries and
 * keys and writes K and V to the paged bf16 cache (or attn_cache_append_q4 to
 * a 4-bit one); then attn_decode_paged / attn_prefill_paged run on the bf16
 * cache, attn_decode_paged_q4 / attn_prefill_paged_q4 on the 4-bit one.  A
 * slot is page * 16 + row: the place of one token in a paged cache.  A step may
 * have no tokens for attn_step_tables; the others take at least one (the
 * Python functions check their arguments and return without a launch for none).
 */

/*
 * Tables of one serving step.
 *   cached_lens [num_seqs] int32: tokens of each request already in the cache
 *   new_lens    [num_seqs] int32: tokens the request adds in this step (>= 0);
 *               the step's tokens are packed, request after request
 *   free_pages  [num_free] int32: unused physical pages, taken from the front
 *   block_table [num_seqs, max_blocks_per_seq] int32, in and out: holds the
 *               pages of the cached tokens; the pages this step takes are
 *               entered behind them, nothing else is written
 *   seq_lens    [num_seqs] (output) = cached + new
 *   cu_seqlens  [num_seqs + 1] (output): exclusive prefix sum of new_lens
 *   positions   [num_tokens] (output): position of each new token in its sequence
 *   slots       [num_tokens] (output): block_table[n][position / 16] * 16 + position % 16
 *   pages_used  [1] (output): pages taken from the front of free_pages
 * No output, block_table among them, may overlap another tensor of the call: a
 * step's seq_lens are not its own cached_lens (a program that keeps its lengths
 * in one place copies them over after the call).
 * num_tokens >= sum of new_lens; the tokens behind the last request (padding,
 * for example of a captured graph) get position 0 and slot -1.  num_tokens may
 * be 0.  Pages go to the requests in order, a request's in the order of its
 * tokens; a step that is repeated on the same inputs gives the same tables.
 * A request whose lengths are negative or exceed the block table, for which
 * the free pages do not suffice, or whose tokens do not fit num_tokens, is
 * recorded as device status 6: it takes no page, its seq_len stays
 * cached_len, its tokens get position 0 and slot -1.  Once a request has found
 * too few free pages, so has every later one that needs any, though it may be
 * fewer than are left; those that need none are served.  A page id
 * outside [0, num_blocks) is recorded as 2, the slots on it are -1 and the
 * table is not written.
 */
attn_status_t attn_step_tables(const int32_t* cached_lens, const int32_t* new_lens, const int32_t* free_pages,
                               int32_t* block_table, int32_t* seq_lens, int32_t* cu_seqlens, int32_t* positions,
                               int32_t* slots, int32_t* pages_used, int num_seqs, int num_tokens, int num_free,
                               int page_size, int max_blocks_per_seq, int num_blocks, void* stream);

/*
 * Rotation table: table [max_positions, rot] f32; row p holds cos(p w_i) for
 * i = 0 .. rot / 2 - 1, then sin(p w_i), with w_i = theta^(-2 i / rot), the
 * angle computed in double.  rot is a multiple of 16, at most 256.
 */
attn_status_t attn_rope_table(float* table, int max_positions, int rot, double theta, void* stream);

/*
 * RMS norm of each query and key head and rotation by position, in one pass;
 * keys and values can be written to the paged cache in the same pass.
 *   q [num_tokens, Hq, d], k and v [num_tokens, Hkv, d] bf16: the heads of a
 *     token are dense, tokens are q_stride / k_stride / v_stride elements
 *     apart (views of one projection's output); strides are multiples of 8.
 *     d in {64, 128, 256}; Hq need not be a multiple of Hkv here.
 *   q_weight, k_weight [d] bf16 or NULL: y = x * rsqrt(mean(x^2) + eps) * w;
 *     NULL: no norm
 *   the first rot channels (a multiple of 16, 0 .. d; 0: no rotation) are
 *     turned: (a, b) -> (a cos - b sin, b cos + a sin) with pair i = channels
 *     (i, i + rot / 2), or (2 i, 2 i + 1) if interleaved != 0, and cos, sin
 *     from row positions[token] of table (attn_rope_table's layout)
 *   q_out [num_tokens, Hq, d], k_out [num_tokens, Hkv, d] (or NULL) bf16, with
 *     token strides of their own; either may be its input (same pointer and
 *     stride), and overlaps no other tensor of the call
 *   k_cache, v_cache [num_blocks, 16, Hkv, d] bf16 or both NULL: the result
 *     for k and v itself go to slots[token]; a token with a negative slot is
 *     not written.  The non-negative slots of a call are distinct.
 *   v and slots are read only with a cache; k_out may be NULL only with one.
 * Arithmetic: float32, one rounding to bf16 (nearest even).  A position
 * outside [0, max_positions) is recorded as device status 7 (the nearest row
 * is used), a slot past the last page as 8 (the token is not written).
 */
attn_status_t attn_qk_norm_rope(const void* q, long long q_stride, const void* k, long long k_stride, const void* v,
                                long long v_stride, const void* q_weight, const void* k_weight, float eps,
                                const int32_t* positions, const float* table, int max_positions, int rot,
                                int interleaved, void* q_out, long long q_out_stride, void* k_out,
                                long long k_out_stride, void* k_cache, void* v_cache, const int32_t* slots,
                                int num_tokens, int Hq, int Hkv, int d, int page_size, int num_blocks, void* stream);

/*
 * The 4-bit paged cache: [num_blocks, Hkv, 17 d] bytes, one record for each
 * page and KV head (attn_cache_q4_record_bytes(d) = 17 d for d in {64, 128,
 * 256}, else 0): 17 / 32 of a byte a value, against 2 in bf16.
 * Format: a group is 64 consecutive channels of one token's key (or value)
 * head.  With hi = max(x, 0) and lo = min(x, 0) over the group,
 *   s = (hi - lo) / 15 rounded up to 4 significant bits (to a multiple of
 *       2^-129 below 2^-126),
 *   z = rint(-lo / s), code = clamp(rint(x / s) + z, 0, 15)
 * and the code stands for s * (code - z): within half a step s of x, and a
 * bf16 number exactly, so that reading a cache back loses nothing more (a
 * product past the type's largest number is an infinity).  A group that holds
 * an infinity or NaN, or whose hi - lo overflows float32, reads back as NaN.
 * A record holds 16 tokens:
 *   bytes [0, 8 d): K codes, d / 2 bytes a token; the 32-bit word that holds
 *     channels 64 e + 16 t + 8 h + (0 .. 7) of a token, channel j in nibble
 *     j, then rotated left by 3 bits, is word
 *     (e / P) * 8 P + t * 2 P + (e % P) * 2 + h of its row, P = min(2, d / 64);
 *   bytes [8 d, 16 d): V codes; channels 2 j (low nibble) and 2 j + 1 of
 *     token k are byte (32 (j / 32) + 4 (j % 8) + (k % 8) / 2) * 16 +
 *     4 (j / 8 % 4) + k / 8 + 2 (k % 2);
 *   bytes [16 d, 16.5 d): K parameters, [16][d / 64] 16-bit words: s as bf16,
 *     whose lower 4 bits are zero, plus z;
 *   bytes [16.5 d, 17 d): V parameters, likewise.
 */
size_t attn_cache_q4_record_bytes(int d);

/*
 * Writes new tokens into the 4-bit cache.
 *   k, v  [num_tokens, Hkv, d] bf16, tokens k_stride / v_stride elements apart
 *         (multiples of 8), the heads of a token dense
 *   slots [num_tokens] int32; a token with a negative slot is not written
 *   cache [num_blocks, Hkv, 17 d] (in and out): only the given tokens' bytes change
 * The non-negative slots of a call are distinct.  A slot past the last page is
 * recorded as device status 8 and skipped.
 */
attn_status_t attn_cache_append_q4(const void* k, long long k_stride, const void* v, long long v_stride,
                                   const int32_t* slots, void* cache, int num_tokens, int Hkv, int d, int page_size,
                                   int num_blocks, void* stream);

/*
 * Reads sequences of the 4-bit cache back.
 *   block_table [num_seqs, max_blocks_per_seq], seq_lens [num_seqs] as for
 *   attn_decode_paged
 *   k_out, v_out [num_seqs, max_blocks_per_seq * 16, Hkv, d] bf16 (output);
 *   rows behind a sequence's end are not written
 * A block-table entry outside [0, num_blocks) is recorded as device status 2
 * (page 0 is read instead), a seq_len the table cannot cover as 5 (clamped).
 */
attn_status_t attn_cache_gather_q4(const void* cache, const int32_t* block_table, const int32_t* seq_lens,
                                   void* k_out, void* v_out, int num_seqs, int Hkv, int d, int page_size,
                                   int max_blocks_per_seq, int num_blocks, void* stream);

/*
 * Bytes of workspace attn_decode_paged_q4 needs on the current device, whatever
 * the batch: two partials of 8 query heads for each CTA of a grid that fills
 * the device.  0 for a head dim other than 64, 128, 256 or when no CUDA device
 * can be queried.
 */
size_t attn_decode_q4_workspace_bytes(int d);

/*
 * attn_decode_paged over the 4-bit cache: q, block_table, seq_lens, o, lse,
 * scale and the conventions for empty sequences, last pages and block-table
 * entries out of range are as there.  d in {64, 128, 256}; any number of
 * query heads per KV head.  The split over the context is chosen on the
 * device, from the lengths: equal shares of all pages, one a CTA.
 * Arithmetic: products of the bf16 queries and the codes, which are exact;
 * float32 scores, sums and accumulators; each probability times its value's
 * scale enters the product with V as one fp16 number: 11 bits down to 2^-20 of
 * the largest scale that a sequence's values have in that group of channels,
 * 2^-31 of that scale in absolute terms below it (2^-151 where the largest
 * scale is below 2^-120).
 * workspace: device buffer, 16-byte aligned, of at least
 * attn_decode_q4_workspace_bytes(d) bytes.  What a call reads from it the same
 * call has written; calls that overlap on the GPU (two streams, two graphs)
 * need one each.
 */
attn_status_t attn_decode_paged_q4(const void* q, const void* cache, const int32_t* block_table,
                                   const int32_t* seq_lens, void* o, float* lse, int num_seqs, int Hq, int Hkv, int d,
                                   int page_size, int max_blocks_per_seq, int num_blocks, float scale,
                                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * Bytes of workspace attn_prefill_paged_q4 needs: keys and values of num_seqs *
 * max_blocks_per_seq pages in bf16 and their block table, each rounded up to
 * 256.  0 for invalid arguments (also more than 2^30 token rows).  A block
 * table cut to the columns that the longest sequence fills takes less.
 */
size_t attn_prefill_q4_workspace_bytes(int num_seqs, int Hkv, int d, int max_blocks_per_seq);

/*
 * attn_prefill_paged over the 4-bit cache: the sequences are read back into
 * the workspace (256-byte aligned), which loses nothing, and attended there.
 * Arguments, results and arithmetic are otherwise those of
 * attn_prefill_paged.  Calls that overlap on the GPU need a workspace each.
 */
attn_status_t attn_prefill_paged_q4(const void* q, const void* cache, const int32_t* block_table,
                                    const int32_t* cu_seqlens_q, const int32_t* seq_lens, void* o, float* lse,
                                    int num_seqs, int max_seqlen_q, int total_q, int Hq, int Hkv, int d,
                                    int page_size, int max_blocks_per_seq, int num_blocks, float scale, int causal,
                                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Device-side status: waits for all work on the current device, then stores
 * the first error code any kernel of this library recorded since the last
 * clear (0 = none; 1 = a pipeline wait timed out; 2 = block-table entry out of
 * range; 3 = a seq_len the block table cannot cover; 4 = shared memory not
 * 1 KB-aligned; 5 = cu_seqlens decreasing, past total_tokens or longer than
 * max_seqlen, or a seq_len that does not fit its chunk or block table; 6 = a
 * step's lengths do not fit its block table or token count, or its free pages
 * are used up; 7 = a position outside the rotation table; 8 = a cache slot
 * past the last page) and, if `clear` != 0, resets it.
 */
attn_status_t attn_device_status(uint32_t* code, int clear);

/* Library version as major * 10000 + minor * 100 + patch. */
int attn_version(void);

#ifdef __cplusplus
}
#endif

#endif /* ATTN_H_ */
