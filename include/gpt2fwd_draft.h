/*
 * gpt2fwd_draft.h -- C ABI of libgpt2fwd.so, third part: operators for
 * verifying drafted tokens, several new positions of a sequence in one step
 * over a paged KV cache, beside the calls of gpt2fwd.h and gpt2fwd_serve.h
 * (whose conventions on pointers, streams, alignment, errors and the device
 * error word hold here too).
 *
 *   attention_tree         attention of each sequence's tree of drafted tokens
 *                          over its cached positions and the tree itself
 *   gpt2_decode_step_tree  the decode step over that attention
 *   logits_adjust          penalties for repeated tokens, biases and grammar
 *                          masks on logits, one row a node (or a sequence)
 *   gpt2_accept_tree       the path of the tree that the model agrees with,
 *                          and its rows of the cache moved together
 *
 * A step of a loop: paged_build_tables for the nodes' positions,
 * gpt2_decode_step_tree, logits_adjust, gpt2_argmax over the B * N rows (or any
 * sampler), gpt2_accept_tree, whose next_tok and next_pos are the next tree's
 * first node and place.  A row of the block table keeps the blocks behind the
 * accepted positions for the next tree: the lengths that paged_build_tables gets
 * and returns are those of the positions that have blocks, its new_len is what
 * pos + N has more, and a sequence whose length stays below pos + N waits (-1
 * for its pos).  No call allocates, synchronises or copies between host
 * and device: all of them can be captured into a CUDA graph.  Results do not
 * depend on timing.  Calls that run at the same time need outputs and
 * workspaces of their own.  Pointers are of the device that is current at the
 * call.
 *
 * A tree.  parent: DEVICE int32 [B][N], N <= GPT2_TREE_MAX_NODES: node i of
 * sequence b comes behind node parent[b][i] < i; -1: behind the cached
 * positions (as node 0, in general the last token known, whose key and value
 * are not cached yet); -2: no node (a tree of fewer than N).  parent NULL: a
 * chain, node i behind node i - 1.  A node's path is the node and all nodes it
 * comes behind.  A parent outside [-2, i) sets GPT2_DEVERR_TREE_BIT and is
 * read as -2; a node behind a missing one is missing too (so one behind -2 is
 * no mistake).
 */
#ifndef GPT2FWD_DRAFT_H
#define GPT2FWD_DRAFT_H

#include "gpt2fwd_serve.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Most nodes of a tree. */
#define GPT2_TREE_MAX_NODES 64

/* Further bit of the device error word (gpt2_get_error). */
#define GPT2_DEVERR_TREE_BIT 16 /* a node's parent, or a row's mask, outside its range */

/* ------------------------------------------------------------ attention */

/* Scratch bytes attention_tree needs (0 for invalid arguments).  Enough for
 * this and every smaller tree and every number of sequences, of the same heads
 * and precision. */
GPT2_API size_t attention_tree_workspace_size(int B, int N, int C, int NH, int precision);

/* The attention of one layer [NTU "KV Caching"; FlashAttention Algorithm 0
 * defines the result, Algorithm 1's online softmax computes it] for B sequences
 * with a tree of N new tokens each.  Sequence b has pos[b] positions cached;
 * row b * N + i of qkv is node i's query, key and value:
 *   out[b * N + i, head h] = sum_j softmax_j(q . k_j / sqrt(hs)) v_j
 * over the cached positions j < pos[b], read through row b of the block table,
 * and the nodes j of node i's path, from qkv; nothing else, whatever its
 * values, reaches a row (an infinity or a NaN among the values that a row does
 * see makes that dimension of it infinite or NaN).  Node i's key and value are stored at position pos[b]
 * + i of the cache (by its number, not its depth: gpt2_accept_tree moves the
 * accepted ones).  A missing node has a zero row and is not stored.
 *   kv: one layer's slab [2][num_blocks][NH][block_size][hs], and the table
 *   [B][max_blocks_per_seq]; a sequence holds at most max_blocks_per_seq *
 *   block_size positions, and 2^30.  qkv [B*N,3C], out [B*N,C] and the slab have
 *   one element type: fp32 in GPT2_FP32 and GPT2_TF32 (both fp32 arithmetic),
 *   the 16-bit type in GPT2_BF16 and GPT2_FP16 (products on tensor cores with
 *   fp32 accumulation, probabilities as sums of two values of the 16-bit type:
 *   off by 2^-15 relative in bf16, by 2^-22 or an absolute 2^-25 in fp16).
 * Head size 16, 32 or 64.  pos: DEVICE int32 [B]; -1 is a sequence without a
 * tree in this step (one that waits for a block, or has ended): zero rows,
 * nothing stored.  Any other pos[b] outside [0, capacity) sets
 * GPT2_DEVERR_POSITION_BIT too, and so does a node whose position pos[b] + i is
 * outside it, which is then missing.  A reached table entry outside [0,
 * num_blocks) sets GPT2_DEVERR_BLOCK_BIT: block 0 is read in its place, and no
 * node is stored through it.  Positions from pos[b] on lie in blocks that no
 * other sequence, and no other position of this one, has.  out must not overlap
 * qkv.
 * The lengths stand on the device, so the kernel is chosen by what a row of the table
 * can hold: a program whose sequences are short does well to give a table hardly wider
 * than the longest (384 pairs of sequence and head, 16 nodes, 60 positions, bf16: 5.0
 * us in a table of 1024 positions, 9.5 in one of 4096; 500: 10.8 and 14.4).
 * Workspace: 16-byte aligned, attention_tree_workspace_size bytes. */
GPT2_API int attention_tree(void* out, const void* qkv, const GPT2PagedKVCache* kv, const int* pos, const int* parent,
                            int B, int N, int C, int NH, int precision, void* workspace, size_t ws_bytes,
                            void* stream);

/* Workspace bytes of gpt2_decode_step_tree for up to B sequences with trees of
 * up to N nodes (0 for invalid arguments). */
GPT2_API size_t gpt2_tree_workspace_size(const GPT2Config* cfg, int B, int N, int precision);

/* One step of the model over the paged cache for a tree of N tokens a sequence
 * (attention_tree in every layer): sequence b has pos[b] positions cached, its
 * nodes' tokens are tok [B][N].  Node i stands at the model's position pos[b] +
 * d, d the number of nodes it comes behind.  logits [B*N,Vp] (and probs
 * [B*N,Vp] when non-null): row b * N + i is what gpt2_decode_step_paged would
 * give for node i's token after the tokens of its path, but for another order
 * of fp32 sums.  Rows of missing nodes, and of sequences with pos[b] = -1, mean
 * nothing; their tokens are not read.  A sequence holds min(maxT,
 * max_blocks_per_seq * block_size) positions.  Workspace of
 * gpt2_tree_workspace_size bytes, 256-byte aligned.  Launch behaviour as
 * gpt2_decode_step. */
GPT2_API int gpt2_decode_step_tree(const GPT2Config* cfg, const float* params, const void* packed,
                                   const GPT2PagedKVCache* kv, const int* tok, const int* parent, const int* pos, int B,
                                   int N, float* logits, float* probs, void* workspace, size_t ws_bytes, int precision,
                                   void* stream);

/* --------------------------------------------------------------- logits */

/* Most biases of a sequence. */
#define GPT2_LOGIT_MAX_BIASES 1023
/* Most tokens of a history. */
#define GPT2_LOGIT_MAX_HISTORY (1 << 20)

/* What logits_adjust applies.  Each part may be left out (NULL, and 0 for its
 * number); all pointers are DEVICE pointers, 4-byte aligned, the struct itself
 * is read on the host during the call. */
typedef struct {
  const int* history;      /* [B][history_stride] tokens so far, -1: none in this place */
  const int* history_len;  /* [B], 0 .. history_stride; NULL: history_stride each */
  const int* prompt_len;   /* [B]: the first of them, that the user gave; NULL: 0 */
  const float* repetition; /* [B] > 0, 1 for none */
  const float* presence;   /* [B] */
  const float* frequency;  /* [B] */
  const int* bias_ids;     /* [B][num_bias] tokens, -1: none in this place */
  const float* bias_values; /* [B][num_bias] */
  const unsigned* masks;   /* [num_masks][ceil(V / 32)]: token v may be drawn where bit v % 32 of word v / 32 is 1 */
  const int* mask_rows;    /* [B*N]: the mask of each row, -1 for none */
  int history_stride;      /* 0 .. GPT2_LOGIT_MAX_HISTORY */
  int num_bias;            /* 0 .. GPT2_LOGIT_MAX_BIASES */
  int num_masks;
} GPT2LogitRules;

/* Penalties, biases and masks on B * N rows of logits [llm.c classifier: what
 * stands between its logits and the next token].  Row b * N + i belongs to node
 * i of sequence b; with N = 1 and tok NULL it is one row a sequence.  With
 * out_v the number of times token v stands in history[prompt_len ..
 * history_len) and on node i's path (tok [B][N]; NULL: no drafted tokens), and
 * seen_v whether it stands there or in the prompt, for every v < V in fp32:
 *   x = l_v;
 *   seen_v:     x = x > 0 ? x / repetition : x * repetition;
 *   out_v > 0:  x = x - frequency * out_v - presence;
 *   a bias:     x = x + bias (of a token that the list names twice the later);
 *   masked:     x = -inf (whatever x was),
 * rounded once to the logits' type; columns from V on are set to -inf.  A token
 * that nothing names keeps its logit bit for bit.  Rows of missing nodes are
 * left as they are.
 * logits, out [B*N,Vp] of logits_type (a GPT2ProbsType), each row a whole number
 * of 16 bytes, 16-byte aligned, Vp <= 2^30.  out may be logits itself (then of a
 * row without a mask only the tokens that the rules name are read and written, and the
 * columns from V on written; a row under a mask is read and written whole.  That is
 * faster than another buffer without masks for few nodes and short histories, 128
 * sequences of 8 nodes, 50257 bf16, 300 tokens 23.5 us against 31.9, and slower
 * otherwise, 32 of 16, fp32, 1000 tokens 39.2 against 34.8, under masks 67.5 against
 * 38.1); otherwise they must not overlap.
 * parent: the trees, NULL for chains.  A token of the history, the path or the
 * biases outside [-1, V) sets GPT2_DEVERR_TOKEN_BIT and is left out; one of the
 * missing nodes is not read.  A history_len outside [0, history_stride], or a
 * prompt_len outside [0, history_len], sets GPT2_DEVERR_POSITION_BIT and is
 * moved to the nearer end.  A mask row outside [-1, num_masks) sets
 * GPT2_DEVERR_TREE_BIT and rules everything out. */
GPT2_API int logits_adjust(void* out, const void* logits, int logits_type, const GPT2LogitRules* rules, const int* tok,
                           const int* parent, int B, int N, int V, int Vp, void* stream);

/* ----------------------------------------------------------- acceptance */

/* The part of each tree that the model agrees with.  next[b][i] (DEVICE int32
 * [B][N]) is the token chosen behind node i: gpt2_argmax of its logits, or a
 * draw from them (drawn with random numbers of each node's own, the accepted
 * tokens are distributed as if they had been drawn one after the other).  The
 * path begins with node 0 and goes on with the child whose token is the one
 * chosen (the lowest of several), as long as there is one:
 *   path[b][k]     the path's nodes, -1 behind them;
 *   count[b]       their number n;
 *   emitted[b][k]  the new tokens: those of path[b][1 .. n-1], then
 *                  next[b][path[b][n-1]], n in all; -1 behind them;
 *   next_tok[b]    the last of them; next_pos[b] = pos[b] + n;
 * and in every layer of the cache the keys and values of position pos[b] +
 * path[b][k] are moved to pos[b] + k, so that positions [0, next_pos[b]) are
 * those of the sequence.  Positions from next_pos[b] on hold what is left of the
 * tree; blocks that only they reach can be given back.
 *   cfg, precision: of the model whose cache kv is (its pool with all layers).
 *   kv NULL: nothing is moved (cfg is not read then).
 *   path, emitted int32 [B][N], count, next_tok, next_pos int32 [B], each may be
 *   NULL, none may overlap another or an input (a loop swaps two buffers).
 * A sequence with pos[b] = -1, or whose node 0 is missing: count 0, path,
 * emitted and next_tok -1, next_pos = pos[b], nothing moved.  Any other pos[b]
 * outside [0, capacity) sets GPT2_DEVERR_POSITION_BIT too; a node whose
 * position pos[b] + i is outside it sets that bit and is missing, as in
 * attention_tree (without a cache the capacity is 2^30).  A table entry
 * outside [0, num_blocks) that a moved row needs sets GPT2_DEVERR_BLOCK_BIT:
 * the row is not moved. */
GPT2_API int gpt2_accept_tree(int* path, int* count, int* emitted, int* next_tok, int* next_pos, const GPT2Config* cfg,
                              const GPT2PagedKVCache* kv, const int* tok, const int* parent, const int* next,
                              const int* pos, int B, int N, int precision, void* stream);

/* ---------------------------------------------------------- diagnostics */

/* The launch that ends an attention_tree whose work is cut into shares (long
 * tables), by itself, so that it can be tested: it joins what the workspace says
 * is to be joined, from the parts of `shares` CTAs.  An attention whose waits gave
 * up (GPT2_DEVERR_TIMEOUT_BIT) leaves entries unwritten; whatever they hold, the
 * launch reads and writes nothing outside the workspace and the B * N rows of out.
 * GPT2_ERR_SHAPE for shares outside 1 .. the most that N nodes have.  Arguments as
 * in attention_tree. */
GPT2_API int gpt2_diag_tree_join(void* out, int B, int N, int C, int NH, int shares, int precision, void* workspace,
                                 size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GPT2FWD_DRAFT_H */
