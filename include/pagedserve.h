/*
 * pagedserve.h -- C ABI of the GB300 (sm_103a) paged KV attention library.
 *
 * One attention step over a paged KV cache for a packed ragged batch:
 *   1. ps_slot_mapping       -- the pool slot of every packed token;
 *   2. ps_reshape_and_cache  -- scatter each token's K/V row into the pool at its slot;
 *   3. ps_paged_attention    -- causal grouped-query attention of every packed query row
 *                               over its sequence's context, read through block tables.
 *
 * Sources (three web pages on paged KV serving):
 *   - PageServe, section 01 "Scheduler loop": one packed [1, T] forward per step with
 *     explicit position ids and a slot mapping per token; the forward writes K/V into the
 *     pool and reads context via block tables; a token's slot is
 *     block_table[pos // 16] * 16 + pos % 16; every step computes the tokens that do not
 *     yet have K/V ("num_computed_tokens").
 *   - PageServe, section 03 "Paged KV cache" and development-history phases 6-8: fixed
 *     16-token blocks in one pre-allocated pool [layers, blocks, 16, H, D]; per-sequence
 *     block tables; a custom attention backend that scatters new K/V and attends through
 *     the table.
 *   - tinyserve, "How it works": K/V slabs [layers, blocks x 16, H_kv, D] (the same memory
 *     order); shared prefix blocks referenced from several tables; one fused pass over a
 *     flattened ragged batch mixing prefill chunks and decodes; k+1 speculative-verify
 *     tokens scored at once under a stepped causal mask; grouped-query attention
 *     ("Highlights" table, forward-pass row).
 *
 * Conventions shared by every entry point:
 *   - Every pointer is a DEVICE pointer owned by the caller, unless the argument says
 *     otherwise. The library allocates no device memory and keeps no pointer after return.
 *   - Every call is asynchronous on `stream` (a cudaStream_t; NULL = the legacy default
 *     stream) and returns PS_OK once its kernels are enqueued, or a negative ps_status.
 *     Host-side argument errors are detected before anything is enqueued.
 *   - Tensors are dense and row-major with the shapes given. 16-bit values are IEEE fp16
 *     or bfloat16 as `dtype` says. Tensor pointers must be 16-byte aligned.
 *   - Block size is 16 tokens. head_dim D is 64 or 128. H_q is a multiple of H_kv; query
 *     head h reads KV head h / (H_q / H_kv).
 *   - Device-side index errors (a block id outside the pool, a slot past the pool, a
 *     sequence with more query tokens than context) never trap: the kernel records the
 *     first such error in the library's device error word (ps_get_device_error) and
 *     skips the access; the affected outputs are left unwritten.
 */
#ifndef PAGEDSERVE_H
#define PAGEDSERVE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PS_BLOCK_SIZE 16

typedef enum { PS_F16 = 0, PS_BF16 = 1, PS_F32 = 2 } ps_dtype; /* F32: ps_beam_select's logits */

typedef enum {
  PS_OK = 0,
  PS_ERR_ARG = -1,          /* a size, count or required pointer is invalid            */
  PS_ERR_UNSUPPORTED = -2,  /* dtype, head_dim or head counts not supported            */
  PS_ERR_ALIGN = -3,        /* a tensor pointer is not 16-byte aligned                 */
  PS_ERR_WORKSPACE = -4,    /* workspace missing, misaligned or too small              */
  PS_ERR_CUDA = -5          /* a CUDA call or kernel launch failed                     */
} ps_status;

/* Device error codes reported by ps_get_device_error. */
typedef enum {
  PS_DEV_OK = 0,
  PS_DEV_BAD_BLOCK_ID = 1,   /* a block-table entry outside [0, num_blocks)            */
  PS_DEV_BAD_SLOT = 2,       /* a slot_mapping entry >= num_blocks * 16                */
  PS_DEV_BAD_SEQUENCE = 3,   /* query count > context, context beyond the table, or a
                                parent outside its group (ps_fork_sequences)           */
  PS_DEV_WAIT_TIMEOUT = 4,   /* a kernel's bounded wait ran out (the kernel returned)  */
  PS_DEV_PLAN_OVERFLOW = 5,  /* the work plan did not fit the workspace                */
  PS_DEV_BAD_TOKEN = 6       /* a draft token id outside [0, V)                          */
} ps_device_error;

/*
 * ps_slot_mapping -- slot of every packed query token (PageServe section 01).
 *
 *   block_tables     int32 [B, max_blocks_per_seq]: physical block ids of each sequence;
 *                    entries past a sequence's context are never read.
 *   seq_lens         int32 [B]: context length of each sequence AFTER this step's tokens.
 *   query_start_loc  int32 [B + 1]: packed offsets, [0] = 0, [B] = T, non-decreasing.
 *                    Sequence b owns packed tokens [query_start_loc[b], query_start_loc[b+1]).
 *   slot_mapping     int32 [T], written: for token i of the n_b tokens of sequence b,
 *                    pos = seq_lens[b] - n_b + i and
 *                    slot = block_tables[b][pos / 16] * 16 + pos % 16;
 *                    -1 (and a device error) where the entry would be invalid.
 *   num_blocks       pool size in blocks, for the bounds check.
 * B = 0 requires T = 0. Returns PS_ERR_ARG for negative sizes or null pointers with T > 0.
 */
int ps_slot_mapping(const int32_t* block_tables, int max_blocks_per_seq,
                    const int32_t* seq_lens, const int32_t* query_start_loc, int B, int T,
                    int num_blocks, int32_t* slot_mapping, void* stream);

/*
 * ps_reshape_and_cache -- KV scatter (PageServe section 01 "Execute"; section 03).
 *
 *   k, v          [T, H_kv, D] of dtype: the new tokens' keys and values.
 *   slot_mapping  int32 [T]: destination slot of each token; a negative slot skips the
 *                 token; a slot >= num_blocks * 16 is skipped and recorded as
 *                 PS_DEV_BAD_SLOT.
 *   k_pool, v_pool [num_blocks, 16, H_kv, D] of dtype, updated in place:
 *                 pool[slot / 16, slot % 16, :, :] = k[t] (bit-exact copy).
 * Two tokens mapped to one slot leave one of the two rows (which one is unspecified).
 */
int ps_reshape_and_cache(const void* k, const void* v, const int32_t* slot_mapping,
                         void* k_pool, void* v_pool, int T, int H_kv, int D, int num_blocks,
                         int dtype, void* stream);

/*
 * ps_copy_blocks -- copy whole KV blocks between pools, bit-exact.
 *
 * Copy-on-write of a block that several block tables share, before one of them writes
 * into it (tinyserve "How it works"; "Highlights" table, paged KV-cache row), and the
 * swap of a preempted sequence's blocks to a pinned host pool and back (PageServe
 * section 04 "Phase 9 · Preemption"; tinyserve "How it works": swapped KV is lossless).
 *
 *   src_k, src_v   [src_num_blocks, 16, H_kv, D] of dtype: the source pools.
 *   dst_k, dst_v   [dst_num_blocks, 16, H_kv, D] of dtype: the destination pools, updated
 *                  in place. Source and destination may be the same pools (copy-on-write)
 *                  or different ones. Each pool may be DEVICE memory or PINNED HOST memory
 *                  (page-locked and mapped, e.g. cudaHostAlloc): the kernel reads and
 *                  writes it through unified addressing, so a swap out or in is one call.
 *   src_ids, dst_ids  int32 [n], device-accessible (device or pinned host memory): for
 *                  every i, block dst_ids[i] of both destination pools becomes a copy of
 *                  block src_ids[i] of the source pools (all 16 x H_kv x D values).
 * The pairs are copied concurrently: destination ids must be distinct and no block may be
 * both a source and a destination of one call (otherwise the result is unspecified). An
 * id outside its pool records PS_DEV_BAD_BLOCK_ID and that pair is skipped. n = 0 is a
 * no-op.
 */
int ps_copy_blocks(const void* src_k, const void* src_v, int src_num_blocks, void* dst_k,
                   void* dst_v, int dst_num_blocks, const int32_t* src_ids,
                   const int32_t* dst_ids, int n, int H_kv, int D, int dtype, void* stream);

/*
 * ps_rope_reshape_and_cache -- rotary position embedding fused with the KV scatter.
 *
 * Every new token's query and key are rotated by its position before the key is cached
 * (tinyserve "Highlights" table, forward-pass row: rotary embeddings in the Qwen2
 * decoder; PageServe section 01: explicit position ids per packed token). Rotate-half
 * form, for each head and frequency i < D/2, with a = positions[t] * rope_theta^(-2i/D):
 *     x'[i]       = x[i] cos(a) - x[i + D/2] sin(a)
 *     x'[i + D/2] = x[i + D/2] cos(a) + x[i] sin(a)
 * The angle is formed and reduced in fp64, its cosine and sine taken in fp32, and each
 * output rounded once to dtype: within one unit in the last place of the exact value
 * plus 2^-20 (|x[i]| + |x[i + D/2]|), the fp32 cosine's share.
 *
 *   q             [T, H_q, D] of dtype, rotated IN PLACE.
 *   k, v          [T, H_kv, D] of dtype (k is not modified).
 *   positions     int32 [T]: position of each token.
 *   slot_mapping  int32 [T]: as for ps_reshape_and_cache; the rotated key row and the V
 *                 row go to the slot (a negative slot skips the token's K/V, a slot past
 *                 the pool records PS_DEV_BAD_SLOT; q is rotated either way).
 *   k_pool, v_pool [num_blocks, 16, H_kv, D] of dtype, updated in place.
 *   rope_theta    the rotary base (> 1), e.g. 1e6 for Qwen2.5 models.
 */
int ps_rope_reshape_and_cache(void* q, const void* k, const void* v, const int32_t* positions,
                              const int32_t* slot_mapping, void* k_pool, void* v_pool, int T,
                              int H_q, int H_kv, int D, int num_blocks, float rope_theta,
                              int dtype, void* stream);

/*
 * ps_rotary_reshape_and_cache -- rotary positions in their other forms, fused with the KV
 * scatter: pairs of neighbours or of halves, over a part of the head, with a table of
 * frequencies.
 *
 * For token t and frequency i < R / 2 (R = rotary_dim), with a = positions[t] * inv_freq[i],
 * c = magnitude * cos(a), s = magnitude * sin(a), the pair (x, y) of every query and key head
 * becomes (x c - y s, y c + x s), where
 *     interleaved != 0:  x = head[2 i],  y = head[2 i + 1]
 *     interleaved == 0:  x = head[i],    y = head[i + R / 2]
 * and elements R .. D - 1 pass through. Any scaling of the positions for contexts longer
 * than the model was trained on (a factor on all frequencies, another base, a factor by
 * wavelength) is in the table, its gain in `magnitude`. The angle is reduced exactly but for
 * the table entry's rounding (2^-53 relative); cosine, sine, products and sums are fp32 and
 * each output is rounded once.
 *
 *   q, k, v       [T, heads, D] of dtype, tokens q_stride, k_stride, v_stride ELEMENTS apart
 *                 (multiples of 8, at least heads * D): views of one projection's output
 *                 serve as they are. k and v are not modified.
 *   q_out         [T, H_q, D], tokens q_out_stride apart: the rotated queries. q_out == q
 *                 (equal strides) rotates in place; otherwise the two must not overlap.
 *   positions     int32 [T]; negative positions turn backwards.
 *   slot_mapping, k_pool, v_pool   as for ps_rope_reshape_and_cache.
 *   inv_freq      double [R / 2], radians per position (finite).
 *   rotary_dim    R: a positive multiple of 16 (other values: PS_ERR_UNSUPPORTED), at most D.
 */
int ps_rotary_reshape_and_cache(const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                const void* v, int64_t v_stride, const int32_t* positions,
                                const int32_t* slot_mapping, void* k_pool, void* v_pool,
                                const double* inv_freq, int rotary_dim, int interleaved,
                                float magnitude, void* q_out, int64_t q_out_stride, int T,
                                int H_q, int H_kv, int D, int num_blocks, int dtype,
                                void* stream);

/*
 * ps_beam_select -- beam search's selection over beams and vocabulary.
 *
 * For each prompt b, beam w and token v the continuation's score is
 *     score(w, v) = scores[b, w] + (logits[b, w, v] - lse_w),
 *     lse_w = log sum_v exp(logits[b, w, v]),
 * and the n_select best of the W * V are returned in falling order, ties to the lowest beam,
 * then the lowest token. A finished beam has one continuation: pad_token, at its score as it
 * is. A logit of -inf or NaN is no continuation (and adds nothing to lse_w); nor has a beam
 * whose score is not finite, or one with a logit of +inf, any. Finite logits are served whatever
 * their size: tokens masked by a large negative number, the type's least value included, are
 * continuations with the scores that follow from it. Where fewer than n_select
 * remain, the rest are parent -1, token -1, score -inf.
 * lse is summed in fp32 within a chunk of the row and in fp64 across chunks, and is off by
 * 2^-16 at most for vocabularies to 2^17 (the exponentials, 64 adds and 16 rescalings of a
 * thread, 15 joins, the logarithm; usually by 2^-20): continuations of two beams whose scores
 * lie closer than twice that may change places. Given lse, scores are compared as pairs of
 * floats (48 bits of the largest of x - max x, scores[b, w] and lse_w - max x; what is below
 * that counts as equal) and rounded once to fp32, below its range to -inf. So the order within
 * a beam is its logits' as long as scores[b, w] leaves room for their differences.
 *
 *   logits        [B, W, V] of logits_dtype (PS_F16, PS_BF16 or PS_F32), rows row_stride
 *                 ELEMENTS apart (at least V: a padded vocabulary is left out by it),
 *                 aligned to an element. Read once; nothing outside the rows is read.
 *   scores        float [B, W]: the beams' sums of log probabilities.
 *   finished      uint8 [B, W], nonzero for a finished beam, or NULL.
 *   pad_token     in [0, V) when finished is given.
 *   parents, tokens  int32 [B, n_select], out_scores float [B, n_select], written.
 *   workspace     device scratch of ps_beam_select_workspace_size() bytes, 256-byte aligned;
 *                 calls that share one must not overlap on the device.
 * W and n_select up to 32, W * V below 2^31 - 2^17; PS_ERR_UNSUPPORTED beyond. B = 0 is a
 * no-op.
 */
size_t ps_beam_select_workspace_size(int B, int W, int V, int n_select);
int ps_beam_select(const void* logits, int64_t row_stride, const float* scores,
                   const uint8_t* finished, int pad_token, int B, int W, int V, int n_select,
                   int logits_dtype, int32_t* parents, int32_t* tokens, float* out_scores,
                   void* workspace, size_t workspace_bytes, void* stream);

/*
 * ps_fork_sequences -- the cache after a selection: n_out children of each group's n_in
 * sequences, each continuing one parent (the beams of a prompt; a prompt forked into its
 * first beams with n_in = 1).
 *
 * Child c = (g, i) continues sequence r = g * n_in + parents[g, i], of length L =
 * seq_lens[r]. Its table takes the parent's L / 16 full blocks as they are (shared from now
 * on); the L % 16 rows of the parent's last, partly filled block are copied, K and V in
 * every layer, into the child's own tail_blocks[g, i], which becomes the child's last block.
 * With L % 16 = 0 nothing is copied and the tail block is not used. The caller keeps count
 * of who holds which block; the blocks of the parents' tails are free again once every
 * child has one of its own.
 *
 *   block_tables  int32 [groups * n_in, max_blocks_per_seq], seq_lens int32 [groups * n_in].
 *   parents       int32 [groups, n_out], each in [0, n_in), the same one any number of
 *                 times; negative for a child that is none (length 0, table left as it was);
 *                 another value records PS_DEV_BAD_SEQUENCE and counts as none.
 *   tail_blocks   int32 [groups, n_out]: distinct, and in no parent's table.
 *   k_pool, v_pool [layers, num_blocks, 16, H_kv, D] of dtype, updated in place.
 *   out_block_tables int32 [groups * n_out, max_blocks_per_seq], out_seq_lens int32
 *                 [groups * n_out], written; other arrays than the parents'. Entries past a
 *                 child's last block are left as they were.
 * A length beyond the table records PS_DEV_BAD_SEQUENCE (length 0); a block outside the pool
 * records PS_DEV_BAD_BLOCK_ID and its rows are not copied. groups = 0 is a no-op.
 */
int ps_fork_sequences(const int32_t* block_tables, int max_blocks_per_seq,
                      const int32_t* seq_lens, const int32_t* parents,
                      const int32_t* tail_blocks, int groups, int n_in, int n_out, void* k_pool,
                      void* v_pool, int layers, int num_blocks, int H_kv, int D, int dtype,
                      int32_t* out_block_tables, int32_t* out_seq_lens, void* stream);

/*
 * ps_spec_accept -- speculative-decoding acceptance after the verify pass.
 *
 * tinyserve "How it works" (speculative decoding): draft d_i is accepted with probability
 * min(1, p_i(d_i) / q_i(d_i)); at the first rejection the replacement is drawn from
 * normalize(max(p_i - q_i, 0)); if all k drafts survive, a bonus token is drawn from the
 * last target distribution. The greedy rule (temperature 0) accepts a draft while it
 * equals argmax p_i and emits argmax p_i at the first mismatch, or argmax p_k when all
 * match. Randomness is an input, and every decision is fixed to a precision, so the tokens
 * are reproducible:
 *   - acceptance of draft i: (double)R_i * (double)q_i(d_i) < (double)p_i(d_i) * 2^32,
 *     each product rounded once in fp64 (q = 1 when draft_probs is null);
 *   - residual weights w = max(p - q, 0) in fp32 (q the one-hot of the draft token when
 *     draft_probs is null; w = p for the bonus row), as integers W = trunc(w * 2^40);
 *   - the sample is the first token v whose running sum W_0 + ... + W_v exceeds
 *     floor(R_k * Z / 2^32), Z the sum of all W (if Z = 0, the same draw from p itself);
 *   - argmax ties go to the lowest token.
 *
 *   target_probs  float [B, k + 1, V]: p_0 .. p_k of each sequence (the verify rows).
 *   draft_probs   float [B, k, V]: q_0 .. q_{k-1}, or NULL for a deterministic proposer
 *                 (n-gram drafts: q is the one-hot of the draft token).
 *   draft_tokens  int32 [B, k]; an id outside [0, V) records PS_DEV_BAD_TOKEN and counts
 *                 as rejected, its replacement drawn from p alone.
 *   random_bits   uint32 [B, k + 1]: R_0 .. R_{k-1} for the acceptance tests, R_k for the
 *                 final draw; may be NULL when greedy != 0.
 *   out_tokens    int32 [B, k + 1], written: the accepted drafts, then the replacement or
 *                 bonus token, then -1.
 *   num_accepted  int32 [B], written: accepted drafts (0 .. k); num_accepted + 1 tokens
 *                 are emitted.
 *   workspace     device scratch of ps_spec_accept_workspace_size(B, k, V) bytes,
 *                 256-byte aligned.
 * Probabilities are expected in [0, 1]; other values give unspecified tokens, never a
 * fault. B = 0 is a no-op; k = 0 draws one token from p_0; k > 31 or V > 2^30 returns
 * PS_ERR_UNSUPPORTED. Rows are read as 16-byte words when V is a multiple of 4 and both
 * probability arrays are 16-byte aligned, and as 4-byte words otherwise.
 */
size_t ps_spec_accept_workspace_size(int B, int k, int V);
int ps_spec_accept(const float* target_probs, const float* draft_probs,
                   const int32_t* draft_tokens, const uint32_t* random_bits, int B, int k, int V,
                   int greedy, int32_t* out_tokens, int32_t* num_accepted, void* workspace,
                   size_t workspace_bytes, void* stream);

/*
 * ps_paged_attention_workspace_size -- bytes of device workspace ps_paged_attention wants
 * for a batch of at most T packed tokens, B sequences and contexts of at most
 * max_seq_len tokens. A smaller workspace (at least the size returned for
 * max_seq_len = 0) still works; the attention then splits long contexts into fewer parts.
 * Returns 0 for invalid sizes or head counts, and for a batch whose plan could not be
 * indexed with 32-bit integers (such a batch is rejected by ps_paged_attention too).
 */
size_t ps_paged_attention_workspace_size(int T, int B, int H_q, int H_kv, int D,
                                         int max_seq_len);

/*
 * ps_paged_attention -- causal paged attention over a packed ragged batch.
 *
 * For packed row r = query_start_loc[b] + i of sequence b (n_b rows, context
 * L_b = seq_lens[b], position p = L_b - n_b + i) and query head h, with G = H_q / H_kv:
 *     out[r, h, :] = sum_{j <= p} softmax_j(scale * q[r, h, :] . K_b[j]) V_b[j]
 * where K_b[j] = k_pool[block_tables[b][j / 16], j % 16, h / G, :] (V likewise).
 * One-token decodes, k+1-token speculative-verify rows and prefill chunks mix freely
 * (PageServe section 01; tinyserve "How it works").
 *
 *   q              [T, H_q, D] of dtype.
 *   k_pool, v_pool [num_blocks, 16, H_kv, D] of dtype (already holding this step's K/V).
 *   block_tables, seq_lens, query_start_loc  as for ps_slot_mapping; 0 <= n_b <= L_b.
 *   scale          softmax scale (normally 1 / sqrt(D)).
 *   out            [T, H_q, D] of dtype, written for every packed row.
 *   workspace      device scratch of workspace_bytes bytes, 256-byte aligned, owned by the
 *                  caller; contents on entry are ignored and on return are undefined.
 *                  Calls that share a workspace must not overlap on the device.
 * Accumulation is fp32; the output is rounded to dtype.
 */
int ps_paged_attention(const void* q, const void* k_pool, const void* v_pool,
                       const int32_t* block_tables, int max_blocks_per_seq,
                       const int32_t* seq_lens, const int32_t* query_start_loc, int B, int T,
                       int H_q, int H_kv, int D, int num_blocks, float scale, void* out,
                       void* workspace, size_t workspace_bytes, int dtype, void* stream);

/*
 * ps_paged_attention_masked -- ps_paged_attention with capped scores, a bias by distance,
 * and masks that are an interval of keys per row.
 *
 * For packed row r at position p of sequence b (context L) and query head h:
 *     x_j = softcap * tanh(scale * q . K_j / softcap)    (softcap > 0; else scale * q . K_j)
 *           - distance_slopes[h] * |p - j|                (with distance_slopes)
 *     out[r, h, :] = sum_j softmax_j(x_j) V_j over the keys j that the row sees:
 *     lo <= j < hi,  hi = max(p + 1, min(prefix_lens[b], L)),
 *                    lo = max(0, p - window + 1 if window > 0, key_starts[r])
 * A row that sees no key (lo >= hi) gives zeros. With all of it absent the result is
 * ps_paged_attention's up to rounding.
 *
 *   scale         > 0 and finite.     softcap  >= 0, 0: none. A capped score is off by 2^-20 of
 *                 itself at most (or 2^-15 in log2 units, up to caps of 88, if that is more),
 *                 so that a large cap tends to none; from 2^100 times the scale it is none.
 *   distance_slopes float [H_q] (finite) or NULL: the linear distance bias.
 *   window        keys a row sees, its own included (a sliding window); 0: none. Block-table
 *                 entries of pages that lie before the first page any row of the sequence
 *                 sees are not read: those blocks may have been given back.
 *   prefix_lens   int32 [B] or NULL: keys j < prefix_lens[b] are seen by every row of the
 *                 sequence, those after it in the prefix included (they must be in the
 *                 cache: values beyond L count as L, negative ones as 0).
 *   key_starts    int32 [T] or NULL: first key of the row's document in a sequence packed of
 *                 several; must not fall from one row of a sequence to the next (else keys
 *                 that a row should see may be left out). Negative counts as 0.
 * Other arguments, workspace and errors as for ps_paged_attention, but that
 * query_start_loc[B] may be below T (a batch padded to a fixed size): rows from there on
 * belong to no sequence and are left as they were. A sequence whose tokens lie outside
 * [0, T) records PS_DEV_BAD_SEQUENCE and its rows are left unwritten; with offsets that fall
 * all rows may be.
 * K and V at keys that no row of the sequence sees (rows of a block never written, blocks
 * given back) may hold anything, NaN included. V at a key that one row of the step sees must
 * be finite for the others' sake: a NaN or infinity there may reach rows of the same
 * sequence and step that do not see it. In bf16 the fp32 sums hold values of V up to 2^40 in
 * magnitude whatever the scores; beyond, they may overflow.
 */
int ps_paged_attention_masked(const void* q, const void* k_pool, const void* v_pool,
                              const int32_t* block_tables, int max_blocks_per_seq,
                              const int32_t* seq_lens, const int32_t* query_start_loc, int B,
                              int T, int H_q, int H_kv, int D, int num_blocks, float scale,
                              float softcap, const float* distance_slopes, int window,
                              const int32_t* prefix_lens, const int32_t* key_starts, void* out,
                              void* workspace, size_t workspace_bytes, int dtype, void* stream);

/*
 * ps_paged_attention_noalloc -- ps_paged_attention for callers that cannot allocate.
 *
 * The pages describe no such call; it exists for users of this library. Some callers
 * are handed only their input and output buffers and may not create device memory:
 * a plug-in inside a host framework whose allocator owns all device memory, or a
 * latency-critical loop that must not call cudaMalloc/cudaFree (they can synchronise
 * the device). This variant takes no workspace: its scratch is a fixed device array of
 * PS_NOALLOC_SCRATCH_BYTES compiled into the library, held by every GPU that loads the
 * library until the process exits. Arguments and results are those of
 * ps_paged_attention without workspace/workspace_bytes.
 *
 *   - Returns PS_ERR_WORKSPACE, before doing anything, when the batch needs more scratch
 *     than the fixed maximum (a work list of about H_kv * (T * H_q / H_kv / 16 + B)
 *     64-byte entries plus 8 bytes per token must fit; long contexts are split into
 *     fewer parts when the partials would not fit).
 *   - The first call on each device (with that device current) looks up the array's
 *     device address with cudaGetSymbolAddress; make that first call before any stream
 *     capture.
 *   - Every call reuses the same array and leaves its contents behind; each call
 *     rewrites what it reads. Calls whose kernels overlap on the device (from two
 *     streams or two host threads) race on the array: the caller must serialise them.
 *   - Allocates nothing: no cudaMalloc, cudaFree or allocating library routine.
 */
#define PS_NOALLOC_SCRATCH_BYTES (32u << 20)
int ps_paged_attention_noalloc(const void* q, const void* k_pool, const void* v_pool,
                               const int32_t* block_tables, int max_blocks_per_seq,
                               const int32_t* seq_lens, const int32_t* query_start_loc, int B,
                               int T, int H_q, int H_kv, int D, int num_blocks, float scale,
                               void* out, int dtype, void* stream);

/*
 * ps_attention_step -- the whole step in one call, with the results of ps_slot_mapping,
 * ps_reshape_and_cache and then ps_paged_attention, on one stream (the slot mapping is
 * computed by the attention planner and the kernels are chained with programmatic
 * dependent launch). k, v are the step's new tokens [T, H_kv, D]; slot_mapping is
 * caller-provided device memory of T int32 (written with the slots). Other arguments as
 * above.
 */
int ps_attention_step(const void* q, const void* k, const void* v, void* k_pool, void* v_pool,
                      const int32_t* block_tables, int max_blocks_per_seq,
                      const int32_t* seq_lens, const int32_t* query_start_loc, int B, int T,
                      int H_q, int H_kv, int D, int num_blocks, float scale, void* out,
                      int32_t* slot_mapping, void* workspace, size_t workspace_bytes,
                      int dtype, void* stream);

/*
 * ps_attention_step_host -- one step from HOST buffers: copies the step's inputs to the
 * device, runs ps_attention_step, and copies the output back, all on `stream`.
 *
 *   q, k, v, block_tables, seq_lens, query_start_loc   HOST pointers (pinned memory lets
 *                  the copies run asynchronously), shapes as for ps_attention_step.
 *   out            HOST pointer [T, H_q, D] of dtype; valid once `stream` has completed.
 *   k_pool, v_pool DEVICE pointers: the resident KV cache, updated in place.
 *   staging        DEVICE scratch of at least ps_attention_step_host_staging_size() bytes,
 *                  256-byte aligned, owned by the caller (inputs, slot mapping, output and
 *                  the attention workspace are placed in it).
 * Host memory must stay valid and unmodified until the stream completes. Page-locked host
 * arrays that the device can address (pinned and mapped, 4-byte aligned) are read by one
 * kernel that gathers all such inputs across the host link; such k and v (16-byte aligned)
 * are instead read by the step's KV scatter directly. Such an `out` (16-byte aligned)
 * is written by the step's kernels themselves when it is at most 4 MB, and otherwise by a
 * kernel after the step's last one; any other array is copied with one cudaMemcpyAsync.
 */
size_t ps_attention_step_host_staging_size(int T, int B, int max_blocks_per_seq, int H_q,
                                           int H_kv, int D, int max_seq_len);

/*
 * ps_attention_step_host_graph_create -- ps_attention_step_host recorded once into a CUDA
 * graph, so that a serving loop pays one graph launch per step instead of the copies' and
 * kernels' launch costs (PageServe, "Next steps": CUDA graphs for decode, against Python
 * and launch overhead at small batch sizes).
 *
 *   Arguments as ps_attention_step_host, without the stream; `graph` receives an opaque
 *   handle. Nothing runs at creation: the pools are not touched.
 *   Each ps_graph_launch(graph, stream) copies the CURRENT contents of the host buffers q,
 *   k, v, block_tables, seq_lens, query_start_loc to the device, runs the step and copies
 *   the output to `out`, as one call of ps_attention_step_host with the same arguments
 *   would. Shapes (T, B, max_blocks_per_seq, heads, D, num_blocks) are fixed at creation;
 *   the contents (lengths, block tables, tokens) may change between launches, with lengths
 *   within the max_seq_len `staging` was sized for (longer ones get fewer splits, and
 *   PS_DEV_PLAN_OVERFLOW if even those do not fit).
 *   The host buffers must be page-locked (cudaHostAlloc, cudaHostRegister); a host pointer
 *   that is not is rejected with PS_ERR_ARG before anything is recorded.
 *   Ownership: the caller keeps every buffer alive, in place and page-locked while the
 *   graph exists; ps_graph_destroy releases the graph.
 * Errors: PS_ERR_ARG for a null `graph` or a host buffer that is not page-locked; those of
 * ps_attention_step_host's argument checks; PS_ERR_CUDA if the capture or instantiation
 * fails. The handle is set only on success.
 */
int ps_attention_step_host_graph_create(const void* q, const void* k, const void* v,
                                        const int32_t* block_tables, const int32_t* seq_lens,
                                        const int32_t* query_start_loc, void* out,
                                        void* k_pool, void* v_pool, int max_blocks_per_seq,
                                        int B, int T, int H_q, int H_kv, int D, int num_blocks,
                                        float scale, void* staging, size_t staging_bytes,
                                        int dtype, void** graph);
/* Launch a graph from ps_attention_step_host_graph_create on `stream` (asynchronous; the
 * output is valid once the stream has completed). PS_ERR_ARG for a null handle. */
int ps_graph_launch(void* graph, void* stream);
/* Release a graph (after its last launch has completed). PS_ERR_ARG for a null handle. */
int ps_graph_destroy(void* graph);
int ps_attention_step_host(const void* q, const void* k, const void* v,
                           const int32_t* block_tables, const int32_t* seq_lens,
                           const int32_t* query_start_loc, void* out, void* k_pool,
                           void* v_pool, int max_blocks_per_seq, int B, int T, int H_q,
                           int H_kv, int D, int num_blocks, float scale, void* staging,
                           size_t staging_bytes, int dtype, void* stream);

/*
 * ps_get_device_error -- read (and clear) the device error word of the current device.
 * Synchronises with the device. *code receives a ps_device_error value. Returns PS_OK or
 * PS_ERR_CUDA / PS_ERR_ARG.
 */
int ps_get_device_error(int* code);

/*
 * ps_last_error_message -- after a call returned PS_ERR_CUDA, the step that failed and
 * CUDA's message, for the calling host thread ("" if none). The string stays valid until
 * the next failing call on the same thread.
 */
const char* ps_last_error_message(void);

/* Human-readable name of a ps_status value. The string is static. */
const char* ps_status_string(int status);

/*
 * Kernel timing hook for benchmarks. ps_profile_begin(n) starts recording CUDA events
 * around the next n launches of each kernel kind (host memory only; events are created
 * here, not in the timed calls). ps_profile_end() waits for the recorded events and
 * stops recording. ps_profile_read(kind, &ms, &launches) then gives the summed device
 * time and the launch count of one kind: 0 slot mapping, 1 KV scatter as its own launch
 * (ps_reshape_and_cache, or the step's scatter ahead of the tile kernel's direct mode),
 * 2 planner (carrying the step's KV scatter when there is one), 3 split attention (decode
 * and verify rows), 4 split combine, 5 tile attention (prefill rows, tcgen05), 6 block
 * copy (and sequence forks), 7 speculative acceptance (and beam selection), 8 rotary KV
 * scatter (either form). The masked attention's kernels count under 2 to 5.
 */
int ps_profile_begin(int max_launches_per_kind);
int ps_profile_end(void);
int ps_profile_read(int kind, float* total_ms, int* launches);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDSERVE_H */
