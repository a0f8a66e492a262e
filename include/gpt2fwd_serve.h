/*
 * gpt2fwd_serve.h -- C ABI of libgpt2fwd.so, second part: operators for
 * serving and scoring many continuations of one prompt beside the calls of
 * gpt2fwd.h (whose conventions on pointers, streams, alignment, errors and
 * the device error word hold here too).
 *
 *   paged_build_tables        block tables and slot maps of a paged KV cache,
 *                             built on the GPU from request lengths
 *   gpt2_prefill_slots        a prefill that stores its keys and values by
 *                             such a slot map
 *   attention_shared_prefix   decode attention of a batch whose sequences
 *                             share their first positions, read once for all
 *   gpt2_decode_step_shared   the decode step over that attention
 *   logprobs_forward          log probabilities of given tokens, with the
 *                             entropy and the top alternatives of each row
 *   logprobs_backward         the gradient of the log probabilities and
 *                             entropies with respect to the logits
 *
 * No call allocates, synchronises or copies between host and device: all of
 * them can be captured into a CUDA graph.  Results do not depend on timing.
 * Calls that run at the same time need outputs and workspaces of their own.
 * Pointers are of the device that is current at the call.
 */
#ifndef GPT2FWD_SERVE_H
#define GPT2FWD_SERVE_H

#include "gpt2fwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------ tables of a paged cache */

/* Gives B requests the blocks for their next positions and writes where each
 * new position lives [NTU "KV Caching"; the block-table layout of
 * GPT2PagedKVCache].  Request b has cached_len[b] positions cached, in blocks
 * that its row of block_table names already, and gets new_len[b] more.  With
 * bs = block_size:
 *   have[b] = ceil(cached_len[b] / bs),
 *   need[b] = ceil((cached_len[b] + new_len[b]) / bs),
 *   end[b]  = sum over b' <= b of (need[b'] - have[b']).
 * A request that needs no block, or whose end[b] <= num_free - taken_in[0],
 * is granted: entries [have, need) of its row become the free blocks
 *   free_blocks[taken_in[0] + end[b] - (need - have) + i],  i = 0, 1, ...;
 * slots[b][t] = block * bs + offset of position cached_len[b] + t for t <
 * new_len[b] (-1 for t >= new_len[b]); next_len[b] = cached_len[b] +
 * new_len[b].  A request that does not get its blocks keeps its row (but for
 * the shared prefix's entries, below) and its length (next_len[b] =
 * cached_len[b]) and its slots are -1: the caller sees by next_len who has to
 * wait, and gives that request no position to decode at (-1 in
 * gpt2_decode_step_shared), since its entry there names no block of its own.
 * taken_out[0] = taken_in[0] + the blocks given, always a prefix of the free
 * blocks that were left.
 *   block_table  int32 [B][max_blocks_per_seq], updated in place
 *   slots        int32 [B][T] or NULL; next_len int32 [B] or NULL;
 *   taken_out    int32 [1] or NULL; none of the outputs may overlap an input
 *                (taken_out is another buffer than taken_in: a loop swaps
 *                the two, as it does cached_len and next_len)
 *   cached_len   int32 [B]; new_len int32 [B], each in [0, T], or NULL: every
 *                request gets min(T, 1) (a decode step)
 *   free_blocks  int32 [num_free] (NULL when num_free is 0); taken_in int32
 *                [1]: the free blocks given away by earlier calls, or NULL: 0
 *   prefix_blocks, prefix_len: prefix_len > 0 (a multiple of block_size):
 *                every request's first prefix_len positions are the shared
 *                ones in these prefix_len / block_size blocks (int32, DEVICE),
 *                which are written to every row, granted or not
 *                (attention_shared_prefix reads them through row 0);
 *                cached_len counts them.  NULL and 0 otherwise.
 * On the device: a negative length, new_len[b] > T, a sequence past
 * max_blocks_per_seq * block_size positions, or cached_len[b] < prefix_len
 * sets GPT2_DEVERR_POSITION_BIT and refuses the request, which then needs no
 * block; a block id outside [0, num_blocks) that a slot needs sets
 * GPT2_DEVERR_BLOCK_BIT and leaves that slot -1.
 * B <= 65536, T <= 2^30, max_blocks_per_seq <= 1024, num_blocks * block_size
 * < 2^31, block_size a power of two.  Pointers 4-byte aligned. */
GPT2_API int paged_build_tables(int* block_table, int* slots, int* next_len, int* taken_out, const int* cached_len,
                                const int* new_len, const int* free_blocks, int num_free, const int* taken_in,
                                const int* prefix_blocks, int prefix_len, int B, int T, int num_blocks, int block_size,
                                int max_blocks_per_seq, void* stream);

/* gpt2_prefill_paged with a slot map in place of the block table: the keys
 * and values of token (b, t) go to slot slots[b][t] (block * block_size +
 * offset) of the pool, and a token whose slot is -1 (the padding of a batch of
 * prompts of different lengths) is not stored, so that padding needs no
 * blocks.  slots: DEVICE int32 [B][T], distinct where not negative.  A slot >=
 * num_blocks * block_size sets GPT2_DEVERR_BLOCK_BIT and is not stored.
 * kv->block_table and kv->max_blocks_per_seq are not read.  The outputs are
 * gpt2_forward's. */
GPT2_API int gpt2_prefill_slots(const GPT2Config* cfg, const float* params, const void* packed, const int* tok, int B,
                                int T, float* logits, float* probs, const GPT2PagedKVCache* kv, const int* slots,
                                void* workspace, size_t ws_bytes, int precision, void* stream);

/* ------------------------------------- attention over a shared prefix */

/* Scratch bytes attention_shared_prefix needs: 0 for invalid arguments and for
 * a prefix too short to need any.  Enough for this and every smaller batch and
 * shorter prefix of the same heads and precision. */
GPT2_API size_t attention_shared_prefix_workspace_size(int B, int C, int NH, int prefix_len, int precision);

/* The decode attention of one layer [NTU "KV Caching"; FlashAttention
 * Algorithm 0 defines the result, Algorithm 1's online softmax computes it]
 * for B sequences whose first prefix_len positions are the same (several
 * continuations of one prompt).  Sequence b has pos[b] >= prefix_len positions
 * cached; its new token's query, key and value are row b of qkv:
 *   out[b, head h] = sum_j softmax_j(q_b . k_j / sqrt(hs)) v_j,  j <= pos[b],
 * where positions j < prefix_len are read through row 0 of the block table
 * for every sequence (each key and value once, for all B queries), positions
 * [prefix_len, pos[b]) through row b, and position pos[b] from qkv; the new
 * key and value are appended to the cache at pos[b].  The result is that of
 * the unshared attention when the blocks of rows b hold the same prefix.
 * prefix_len need not be a multiple of the block size.
 *   kv: one layer's slab [2][num_blocks][NH][block_size][hs], and the table
 *   [B][max_blocks_per_seq]; a sequence holds at most max_blocks_per_seq *
 *   block_size positions, and 2^30.  qkv [B,3C], out [B,C] and the slab have one
 *   element type: fp32 in GPT2_FP32 and GPT2_TF32 (both fp32 arithmetic), the
 *   16-bit type in GPT2_BF16 and GPT2_FP16 (the products over the prefix on
 *   tensor cores with fp32 accumulation, its probabilities as sums of two
 *   values of the 16-bit type: off by 2^-15 relative in bf16, by 2^-22 or an
 *   absolute 2^-25 in fp16).
 * Head size 16, 32 or 64.  pos: DEVICE int32 [B]; -1 is a sequence without a
 * token in this step (one that waits for a block, or has ended): a zero row,
 * nothing appended.  Any other pos[b] outside [prefix_len, capacity) sets
 * GPT2_DEVERR_POSITION_BIT too.  A reached table entry outside [0,
 * num_blocks) sets GPT2_DEVERR_BLOCK_BIT: block 0 is read in its place, and at
 * pos[b] nothing is appended.  Sequences'
 * positions pos[b] lie in blocks of their own.  out must not alias qkv.
 * Workspace: 16-byte aligned, attention_shared_prefix_workspace_size bytes. */
GPT2_API int attention_shared_prefix(void* out, const void* qkv, const GPT2PagedKVCache* kv, const int* pos, int B,
                                     int C, int NH, int prefix_len, int precision, void* workspace, size_t ws_bytes,
                                     void* stream);

/* Workspace bytes of gpt2_decode_step_shared, for up to B sequences and a
 * prefix of up to prefix_len positions (0 for invalid arguments). */
GPT2_API size_t gpt2_shared_workspace_size(const GPT2Config* cfg, int B, int prefix_len, int precision);

/* gpt2_decode_step_paged for sequences that share their first prefix_len
 * positions (attention_shared_prefix in every layer): the same cache, table and
 * positions, and the same results but for another order of fp32 sums, the
 * prefix's keys and values read once a layer instead of once a sequence.  A
 * sequence at pos[b] = -1 has no token in this step: nothing is appended for it
 * and its logits and probs mean nothing, the others' are as they were without
 * it.  A loop over paged_build_tables passes cached_len[b] where next_len[b] >
 * cached_len[b] and -1 where the request got no block: its table entry at that
 * position names no block of its own. 0 <= prefix_len < the capacity of a
 * sequence (0: nothing is shared).  Workspace of gpt2_shared_workspace_size
 * bytes. */
GPT2_API int gpt2_decode_step_shared(const GPT2Config* cfg, const float* params, const void* packed,
                                     const GPT2PagedKVCache* kv, const int* tok, const int* pos, int B, int prefix_len,
                                     float* logits, float* probs, void* workspace, size_t ws_bytes, int precision,
                                     void* stream);

/* ------------------------------------------------- log probabilities */

/* Most alternatives a row can list. */
#define GPT2_LOGPROBS_MAX_TOP 32

/* Log probabilities of given tokens, entropy and top alternatives of each row
 * of logits [llm.c classifier: the softmax over the vocabulary].  Over the V
 * real tokens of row n,
 *   lse[n]      = log sum_v exp(l[n,v]),
 *   logprob[n]  = l[n, targets[n]] - lse[n],
 *   entropy[n]  = -sum_v p_v log p_v,  p_v = exp(l[n,v] - lse[n]) (natural
 *                 logarithms; a token of probability 0 adds nothing),
 *   top_ids[n,:], top_logprobs[n,:] = the K tokens of largest logit, largest
 *                 first, equal ones by the lowest id.
 * logits [N,Vp] of logits_type (a GPT2ProbsType: fp32, fp16 or bf16), each row
 * a whole number of 16 bytes (Vp % 4 == 0 for fp32, Vp % 8 == 0 for the
 * 16-bit types), Vp <= 2^30, and 16-byte aligned; all outputs fp32 (arithmetic in fp32)
 * but top_ids (int32), 4-byte aligned.
 * targets int32 [N], or NULL (then logprob is NULL too); a target of -1 (a
 * padding position) gives logprob 0; one outside [-1, V) sets
 * GPT2_DEVERR_TOKEN_BIT and is treated as -1.  Any output may be NULL;
 * 0 <= K <= GPT2_LOGPROBS_MAX_TOP, and K 0 needs no top outputs.
 * A logit of -inf is a token ruled out: no alternative (its place holds id -1
 * and -inf when fewer than K tokens are left).  A row with every token ruled
 * out: lse and logprob -inf, entropy 0.  A row that holds a NaN or +inf has no
 * distribution: its results are NaN (logprob of target -1 stays 0), its ids
 * -1. */
GPT2_API int logprobs_forward(float* logprob, float* entropy, float* lse, int* top_ids, float* top_logprobs,
                              const void* logits, int logits_type, const int* targets, int N, int V, int Vp, int K,
                              void* stream);

/* The gradient of the loss through logprob and entropy:
 *   dlogits[n,v] = dlogprob[n] ([v = targets[n]] - p_v)
 *                  - dentropy[n] p_v (log p_v + entropy[n])   for v < V,
 *   dlogits[n,v] = 0 for V <= v < Vp; every element is written.
 * lse and entropy [N] are logprobs_forward's; dlogprob [N] or NULL (then
 * targets may be NULL), dentropy [N] or NULL (then entropy may be NULL): a
 * NULL gradient is zero.  A row with target -1 (or one outside [-1, V), which
 * sets GPT2_DEVERR_TOKEN_BIT) gets no gradient through its logprob; a token
 * of probability 0 gets none but the target's own dlogprob; a row with every
 * token ruled out gets zeros.  p is taken from lse, whose fp32 rounding is a
 * relative error of |lse| 2^-24 in it; from |lse| = 1024 on the row's maximum
 * and sum are taken anew instead (about twice the time).  dlogits has the type and layout of logits and
 * may be logits itself. */
GPT2_API int logprobs_backward(void* dlogits, const void* logits, int logits_type, const int* targets,
                               const float* lse, const float* entropy, const float* dlogprob, const float* dentropy,
                               int N, int V, int Vp, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GPT2FWD_SERVE_H */
