/*
 * dflash.h - C ABI of the block-diffusion speculative drafting library
 * (DFlash drafter + DDTree draft trees) for one NVIDIA GB300 (sm_103a).
 *
 * One drafter cycle is four calls, in the order the pages describe a round:
 *
 *   dflash_inject_kv    project the target's fused hidden features into every
 *                       drafter layer's KV cache
 *                       ("DFlash: Block Diffusion for Flash Speculative Decoding",
 *                       section 3.4.3, feature fusion and KV injection);
 *   dflash_draft_block  one parallel pass of the drafter over
 *                       [anchor, mask x (L-1)], LM head, log-softmax and top-K
 *                       (same page, section 3.4.4; "Accelerating Speculative
 *                       Decoding with Block Diffusion Draft Trees", section 3.4.2);
 *   ddtree_build        Algorithm 1: the best-first heap over rank tuples, with
 *                       the flattened tree, depth position ids and the ancestor
 *                       attention mask (DDTree page, sections 3.4.4-3.4.5);
 *   ddtree_accept       the verifier walk against the target's token choices
 *   dflash_tree_attention / dflash_tree_rope
 *                       the verification pass's attention over the flattened
 *                       tree (ancestor mask, depth position ids)
 *                       (DDTree page, section 3.4.5);
 *   dflash_commit_accepted
 *                       the accepted path becomes the next cycle's injected
 *                       context (sizes stay on the device, so a whole cycle
 *                       replays as one CUDA graph).
 * dflash_draft_cycle runs the first two calls as one.  With a dflash_sampling
 * the drafter draws tokens at temperature T (vanilla DFlash), and
 * dflash_chain_tree lays the drafted block out as a chain in ddtree_build's
 * layout.  dflash_logits_topk / dflash_logits_sample run step a6 alone.
 * The target's own side of a cycle over a paged cache is dflash_qk_norm_rope,
 * dflash_paged_append, dflash_paged_attention and, after its LM head,
 * dflash_logits_adjust and dflash_logits_sample_filtered (the walk's
 * target_tok).  dflash_paged_append_e4m3 and dflash_paged_attention_e4m3 serve a
 * cache held in 8 bits.
 *
 * Conventions shared by every call
 * --------------------------------
 * - Memory: every tensor argument is a DEVICE pointer unless marked "host".
 *   The caller owns all memory.  The library never allocates device memory;
 *   scratch space comes from a caller-provided workspace (see
 *   dflash_workspace_bytes).  The only host allocation is the model handle.
 * - Layout: row-major, innermost index last, densely packed unless a leading
 *   dimension is given.  "T" below is the model dtype: fp32 (DFLASH_F32) or
 *   bf16 (DFLASH_BF16, IEEE-754 binary32 truncated to its top 16 bits, round to
 *   nearest even when produced here).
 * - Streams: `stream` is a cudaStream_t (NULL = legacy default stream).  Every
 *   call only enqueues work on it and returns; nothing synchronises.  Calls are
 *   capturable into a CUDA graph (no allocation, no host synchronisation).
 * - Errors: arguments are validated on the host before anything is enqueued; a
 *   rejected call returns non-zero, enqueues nothing and leaves outputs
 *   untouched.  DFLASH_ERR_CUDA means a launch failed (the CUDA error string is
 *   in dflash_last_error()).  Problems found on the device (a bounded wait that
 *   ran out) are recorded in the workspace status word, read with
 *   dflash_read_status.  dflash_last_error() returns a thread-local message for
 *   the last non-OK status of the calling thread.
 * - Concurrency: calls that share a workspace must be ordered on one stream.
 */
#ifndef DFLASH_H
#define DFLASH_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define DFLASH_ABI_VERSION 2
#define DFLASH_MAX_LAYERS 16

typedef enum {
  DFLASH_OK = 0,
  DFLASH_ERR_INVALID_ARG = 1,   /* null pointer, bad size, unsupported shape    */
  DFLASH_ERR_UNSUPPORTED = 2,   /* valid request the library does not implement */
  DFLASH_ERR_WORKSPACE = 3,     /* workspace missing or smaller than required   */
  DFLASH_ERR_CUDA = 4,          /* a CUDA runtime/driver call failed            */
  DFLASH_ERR_TIMEOUT = 5        /* device-side bounded wait expired (status word)*/
} dflash_status;

typedef enum { DFLASH_F32 = 0, DFLASH_BF16 = 1 } dflash_dtype;

/* Temperature of the drafted tokens (DFlash page, 3.4.4: argmax at temperature
 * 0, a sample from softmax(logits) at temperature 1).  A top-K pass given a
 * dflash_sampling with temperature T > 0 ranks, instead of the logits l_v, the
 * Gumbel scores s_v = l_v * f32(1/T) + G_v (an fp32 multiply then an fp32
 * add), G_v = -log(-log U_v) in fp32, and keeps the K best (score desc, token
 * id asc): entry 0 is a sample from softmax(l / T), the K entries a draw
 * without replacement.  U_v: the SplitMix64 generator (Steele, Lea, Flood,
 * 2014) seeded with `seed`; element v of counter row c takes output number
 * (c << 32 | v) + 1 and U = (its top 23 bits + 1/2) / 2^23.  Output row r of a
 * call uses counter row row_offset + r.  The log-probabilities written are
 * log q(token) = logit - logsumexp(row), the logit recovered from the score as
 * (s - G) * T (exact to the fp32 rounding of s).  A NULL pointer or T == 0
 * selects the plain top-K (ranked by logit).  Requires T == 0 or
 * 1e-6 <= T <= 1e6. */
typedef struct dflash_sampling {
  float temperature;
  uint64_t seed;
  int64_t row_offset;
} dflash_sampling;

/* Drafter shape and the readings the pages leave open.
 * - Pre-norm RMSNorm: x / sqrt(mean(x^2) + rms_eps) * gain, before attention,
 *   before the MLP and before the LM head; SwiGLU MLP; no biases.
 * - Rotary embedding (rotate-half, base rope_theta) on queries and keys at
 *   absolute positions: cache slot t has position t, block row j of a request
 *   whose context holds ctx_len entries has position ctx_len + j.
 * - anchor_sees_block = 1: every block row attends to the whole context and the
 *   whole block (bidirectional block).  0: the anchor row attends only to the
 *   context and itself, as the DFlash page's attention bullet list states.
 * Supported: 1 <= n_layers <= 16; head_dim in {64, 128}; n_q % n_kv == 0;
 * bf16 models need d, d_feat*n_feat, n_q*head_dim and d_ff multiples of 128
 * (every GEMM reduction dimension a multiple of 64). */
typedef struct {
  int n_layers;
  int d;            /* hidden size; also the fused feature size            */
  int n_q;          /* query heads                                         */
  int n_kv;         /* key/value heads                                     */
  int head_dim;
  int d_ff;         /* SwiGLU inner size                                   */
  int vocab;
  int n_feat;       /* target layers whose hidden states are concatenated  */
  int d_feat;       /* target hidden size                                  */
  int dtype;        /* dflash_dtype                                        */
  float rope_theta;
  float rms_eps;
  int mask_id;      /* token id of the mask token, 0 <= mask_id < vocab    */
  int anchor_sees_block;
} dflash_dims;

/* Device pointers to the drafter weights (type T unless noted), in the packed
 * layouts the kernels stream.  [out][in] matrices are the usual y = W x form.
 *   w_proj      [d][n_feat*d_feat]        fusion projection W_proj
 *   embed       [vocab][d]                token embedding (shared with target)
 *   lm_head     [vocab][d]                LM head (shared with target)
 *   final_norm  [d]                       gain of the norm before the LM head
 *   u_kv        [n_layers][2][n_kv*head_dim][d]
 *                                         injection projections: per layer
 *                                         U_K rows, then U_V rows
 *   per layer l < n_layers:
 *   attn_norm   [d]
 *   w_qkv       [(n_q + 2*n_kv)*head_dim][d]   rows of W_q, then W_k, then W_v
 *   wo          [d][n_q*head_dim]
 *   mlp_norm    [d]
 *   w_gate_up   [2*d_ff][d]               interleaved: row 2j = gate row j,
 *                                         row 2j+1 = up row j
 *   w_down      [d][d_ff]
 * All pointers 16-byte aligned.  The weights must stay valid and unchanged for
 * the lifetime of a dflash_model built from them. */
typedef struct {
  const void* w_proj;
  const void* embed;
  const void* lm_head;
  const void* final_norm;
  const void* u_kv;
  const void* attn_norm[DFLASH_MAX_LAYERS];
  const void* w_qkv[DFLASH_MAX_LAYERS];
  const void* wo[DFLASH_MAX_LAYERS];
  const void* mlp_norm[DFLASH_MAX_LAYERS];
  const void* w_gate_up[DFLASH_MAX_LAYERS];
  const void* w_down[DFLASH_MAX_LAYERS];
} dflash_weights;

/* The drafter's injected-context KV cache (DFlash page, 3.4.3: the projected
 * features are stored in the drafter's KV cache and reused across cycles).
 * Per layer l: k[l], v[l] are T [n_req][n_kv][cap][head_dim]; slot t of a
 * request holds the entry injected for position t (keys already rotated at t).
 * Written by dflash_inject_kv, read by dflash_draft_block. */
typedef struct {
  void* k[DFLASH_MAX_LAYERS];
  void* v[DFLASH_MAX_LAYERS];
  int n_req;
  int cap;
} dflash_cache;

/* Opaque model handle: the dims, the weight pointers and the TMA descriptors
 * built for them once.  Host memory only. */
typedef struct dflash_model dflash_model;

/* Build a model handle.  Validates dims and weight pointers (non-null, 16-byte
 * aligned).  Returns DFLASH_ERR_INVALID_ARG / DFLASH_ERR_UNSUPPORTED on a bad
 * or unsupported shape, DFLASH_ERR_CUDA if the TMA descriptors cannot be
 * encoded.  *out is set only on success; free it with dflash_model_destroy. */
dflash_status dflash_model_create(const dflash_dims* dims, const dflash_weights* weights,
                                  dflash_model** out);
void dflash_model_destroy(dflash_model* model);

/* Workspace bytes for calls on this model with at most n_req requests,
 * max_inject_rows feature rows per dflash_inject_kv call, block length L <= 16
 * and top-K K <= 1024.  The same workspace also serves dflash_logits_topk for up
 * to n_req*(L-1) rows of this model's vocabulary.  0 on invalid arguments. */
size_t dflash_workspace_bytes(const dflash_model* model, int n_req, int max_inject_rows,
                              int L, int K);

/* Zero a workspace (its status word and arrival counters).  Required once before
 * first use, and again after a call reported a device-side error. */
dflash_status dflash_workspace_init(void* ws, size_t ws_bytes, void* stream);

/* Read (synchronously) and clear the device status word of a workspace:
 * *device_status receives DFLASH_OK or the first device-side error recorded. */
dflash_status dflash_read_status(void* ws, int* device_status, void* stream);

/* Set the time limit of every bounded device-side wait of the tensor-core GEMM
 * launches that use this workspace (ring slots, the phase counters of a GEMM
 * chain, split-tile partial sums, the fused top-K's arrivals) and of the paged
 * attention's tensor-core launches (its kernel for at most 16 query rows of a
 * request and KV head waits for nothing but its own copies).  The pages have
 * no counterpart: this is the failure-detection hook.  limit_ns = 0 restores
 * the default of 2 s; values above 60 s also mean the default.  A wait that
 * runs out records DFLASH_ERR_TIMEOUT in the status word; the CTA then waits
 * (up to 2 s) for its own copies and MMAs in flight, frees its tensor memory
 * and returns, so the context stays usable.  The outputs of that call are
 * undefined and the workspace must go through dflash_workspace_init (which
 * also restores the default limit) before its next use.  The limit is stored
 * in the workspace header (bytes 8..15) by an asynchronous copy on `stream`.
 * Errors: DFLASH_ERR_INVALID_ARG for a null or too small workspace,
 * DFLASH_ERR_CUDA if the copy cannot be queued. */
dflash_status dflash_workspace_set_wait_limit(void* ws, size_t ws_bytes, uint64_t limit_ns,
                                              void* stream);

/* Step a1 + a2: KV injection (DFlash page, 3.4.3).
 * For each request r and each of its feature rows i (global row
 * row_off[r] + i, i < row_off[r+1] - row_off[r]):
 *   f       = W_proj * feats[row]                       (fusion, no norm)
 *   K_l,pos = RoPE(U_K,l f, pos),  V_l,pos = U_V,l f    for every layer l
 * stored at cache slot pos = pos0[r] + i of request r.
 *   row_off  int32 [n_req+1] (device) prefix offsets, row_off[0] = 0,
 *            row_off[n_req] <= n_rows; rows at or past row_off[n_req] are
 *            computed but stored nowhere (a fixed n_rows can then serve a
 *            device-side row count, as dflash_commit_accepted writes it)
 *   pos0     int32 [n_req]   (device) first cache slot written per request;
 *            pos0[r] + rows of r must not exceed cache->cap (not checked on
 *            the device: the caller guarantees it)
 *   feats    T [n_rows][n_feat*d_feat] (device)
 * n_rows may be 0 (nothing is enqueued).  Overwrites only the addressed slots. */
dflash_status dflash_inject_kv(const dflash_model* model, const dflash_cache* cache,
                               int n_req, int n_rows, const int32_t* row_off,
                               const int32_t* pos0, const void* feats,
                               void* ws, size_t ws_bytes, void* stream);

/* Steps a3 - a6: one drafter pass over the block [anchor, mask x (L-1)] of each
 * request, then per-position log-softmax and top-K (DFlash page, 3.4.4; DDTree
 * page, 3.4.2: q_i = softmax(l_i)), or, with `sampling` at T > 0, the Gumbel
 * draw of dflash_sampling (output row r = request * (L-1) + position - 1).
 *   anchor    int32 [n_req] (device) the bonus token of each request
 *   ctx_len   int32 [n_req] (device) context entries of each request in the
 *             cache, 0 <= ctx_len[r] <= max_ctx <= cache->cap
 *   max_ctx   host bound on ctx_len used to size the attention grid
 *   L         block length, 2 <= L <= 16; D = L-1 draft positions
 *   K         1 <= K <= 1024 (and K <= vocab; with sampling K <= 32).  At
 *             batch 1 (n_req * L <= 16) and K <= 8 on bf16 models the top-K
 *             rides in the LM head's epilogue; otherwise the logits are
 *             stored in the workspace and a top-K pass follows
 *   topk_ids  int32 [n_req][L-1][K] (device) out: token ids by (logit desc,
 *             id asc)
 *   topk_logp fp32  [n_req][L-1][K] (device) out: logit - logsumexp(row)
 *   logits    fp32  [n_req][L-1][vocab] (device) out, optional (NULL skips)
 */
dflash_status dflash_draft_block(const dflash_model* model, const dflash_cache* cache,
                                 int n_req, const int32_t* anchor, const int32_t* ctx_len,
                                 int max_ctx, int L, int K, const dflash_sampling* sampling,
                                 int32_t* topk_ids, float* topk_logp, float* logits,
                                 void* ws, size_t ws_bytes, void* stream);

/* Steps a1 - a6 in one call: dflash_inject_kv(n_rows, row_off, pos0, feats)
 * followed by dflash_draft_block(anchor, ctx_len, max_ctx, L, K, ...), with the
 * same arguments, meanings and results as the two calls in sequence (the new
 * context entries are visible to the block pass).  When the injected row count
 * equals n_req * L (bf16 models), the injection's two GEMMs and the first
 * layer's QKV projection run in one GEMM launch.  The workspace must be sized
 * by dflash_workspace_bytes(model, n_req, >= n_rows, L, >= K).  n_rows may be
 * 0 (the block pass alone). */
dflash_status dflash_draft_cycle(const dflash_model* model, const dflash_cache* cache,
                                 int n_req, int n_rows, const int32_t* row_off,
                                 const int32_t* pos0, const void* feats,
                                 const int32_t* anchor, const int32_t* ctx_len, int max_ctx,
                                 int L, int K, const dflash_sampling* sampling,
                                 int32_t* topk_ids, float* topk_logp, float* logits, void* ws,
                                 size_t ws_bytes, void* stream);

/* Step a6 on its own: log-softmax + top-K over given logits rows (DDTree page,
 * 3.4.2 and Lemma 1 in 3.4.4: only the top-K tokens per depth are needed).
 *   logits  [rows][ld] of dtype (DFLASH_F32 or DFLASH_BF16), vocab <= ld
 *   ids     int32 [rows][K], logp fp32 [rows][K] (device) out; order is
 *           (logit desc, token id asc); logp = logit - logsumexp over the row
 * Requires 1 <= K <= 1024, K <= vocab, rows >= 0 (K > 8: a two-pass radix
 * select whose merge holds a row's per-chunk lists in shared memory, so K
 * times the number of 16384-logit chunks is bounded; DFLASH_ERR_UNSUPPORTED
 * beyond); ws of at least
 * dflash_topk_workspace_bytes(rows, vocab, K) bytes (zero-initialised once). */
size_t dflash_topk_workspace_bytes(int rows, int vocab, int K);
dflash_status dflash_logits_topk(int rows, int vocab, int ld, int dtype, const void* logits,
                                 int K, int32_t* ids, float* logp,
                                 void* ws, size_t ws_bytes, void* stream);

/* Step a6 with temperature sampling (DFlash page, 3.4.4; see dflash_sampling):
 * the same pass as dflash_logits_topk ranking Gumbel scores, so ids[r][0] is a
 * sample from softmax(logits[r] / T) and ids[r][0..K) a draw without
 * replacement; logq[r][k] = log q(ids[r][k]).  Same arguments, limits and
 * workspace as dflash_logits_topk; sampling NULL or T == 0 is
 * dflash_logits_topk. */
dflash_status dflash_logits_sample(int rows, int vocab, int ld, int dtype, const void* logits,
                                   const dflash_sampling* sampling, int K, int32_t* ids,
                                   float* logq, void* ws, size_t ws_bytes, void* stream);

/* Step a6 for callers that cannot provide a workspace.  The pages have no
 * counterpart: this variant exists for callers that cannot allocate device
 * memory when they run this step (a serving loop whose device memory is carved
 * up once at start-up and that must not call cudaMalloc afterwards, since that
 * can synchronise the device; a plugin host that passes inputs and outputs but
 * offers no scratch).  Same arguments and results as dflash_logits_topk,
 * without ws, for K <= 32 (always the single-pass kernel, which dflash_logits_topk
 * uses for K <= 8 only): the scratch lives in a fixed array inside the library
 * image (about 286 KB on every device that loads the library, held until the
 * process exits).  Limits: rows <= 4096 and K <= 32, larger requests return
 * DFLASH_ERR_UNSUPPORTED (rows) or DFLASH_ERR_INVALID_ARG (K).  The first call on each device looks up the array's
 * device address (cudaGetSymbolAddress) and caches it; make that first call
 * before any stream capture.  Every call on a device shares the array and
 * clears its counters first, so calls that overlap on the GPU race: order them
 * on one stream.  Allocates nothing. */
dflash_status dflash_logits_topk_noalloc(int rows, int vocab, int ld, int dtype,
                                         const void* logits, int K, int32_t* ids, float* logp,
                                         void* stream);

/* Step a7: DDTree tree construction, Algorithm 1 (DDTree page, 3.4.4), plus the
 * flattened tree and its ancestor-only mask (3.4.5).  Per request r:
 *   topk_logp fp32 [n_req][D][K] log q of the rank-k token at depth d+1,
 *             descending along k; topk_ids int32 [n_req][D][K] its token id
 *   root_tok  int32 [n_req] the bonus token (tree root)
 * Outputs (device), width W1 = B+1 nodes per request, node 0 = root, nodes
 * 1..n in pop order:
 *   n_nodes   int32 [n_req]        n = min(B, number of prefixes available)
 *   tok       int32 [n_req][B+1]   token of the node (root: root_tok)
 *   parent    int32 [n_req][B+1]   parent node index (root: -1)
 *   depth     int32 [n_req][B+1]   depth = position id (root: 0)
 *   rank      int32 [n_req][B+1]   1-based rank of the node's token (root: 0)
 *   mask      uint32 [n_req][B+1][ceil((B+1)/32)] bit j of row i set iff node
 *             j is node i or an ancestor of it
 * Entries past node n are -1 (mask rows 0).  Scores: the candidate score is the
 * parent's score plus logp, one fp32 add; the heap pops the highest score and,
 * on equal scores, the candidate created first (each pop creates its next
 * sibling before its first child).  Requires 0 <= B <= 1024, 1 <= K <= 1024,
 * 1 <= D <= 16.  Needs no workspace. */
dflash_status ddtree_build(int n_req, int D, int K, int B, const float* topk_logp,
                           const int32_t* topk_ids, const int32_t* root_tok,
                           int32_t* n_nodes, int32_t* tok, int32_t* parent,
                           int32_t* depth, int32_t* rank, uint32_t* mask, void* stream);

/* The vanilla DFlash draft as a tree (DFlash page, 3.4.1 and 3.4.4): the chain
 * root -> drafted token of position 1 -> ... -> position D, in ddtree_build's
 * output layout so that tree attention and ddtree_accept serve both drafters.
 * Node d (1 <= d <= n = min(D, B)) holds topk_ids[r][d-1][0] (the argmax, or
 * the sample of a dflash_sampling call), parent d-1, depth d, rank 1; mask row
 * i has bits 0..i.  The walk over a chain accepts the longest prefix the
 * target agrees with.  topk_ids int32 [n_req][D][K]; outputs as ddtree_build
 * (entries past node n are -1, mask rows 0).  Requires 1 <= D <= 16,
 * 1 <= K <= 1024, 0 <= B <= 1024.  Needs no workspace. */
dflash_status dflash_chain_tree(int n_req, int D, int K, int B, const int32_t* topk_ids,
                                const int32_t* root_tok, int32_t* n_nodes, int32_t* tok,
                                int32_t* parent, int32_t* depth, int32_t* rank, uint32_t* mask,
                                void* stream);

/* Steady state between two cycles (DFlash page, 3.4.3: verified tokens are
 * injected as context and the cache is reused across cycles; DDTree page,
 * 3.4.5: only the accepted path stays).  Per request r with a = accept_len[r]
 * (ddtree_accept's outputs for this cycle's tree of budget B and depth D):
 *   the accepted path is node 0 (this cycle's anchor) then accepted[r][0..a),
 *   at positions ctx_len[r] .. ctx_len[r] + a;
 *   feats row row_off[r] + i = tree_feats[r][node i of the path], i <= a
 *   (the target's hidden features of the tree nodes, rows of feat_dim
 *   elements, tree_ld elements apart, [n_req][B+1]);
 *   row_off = prefix sums of a + 1 ([n_req+1]); pos0[r] = ctx_len[r];
 *   then ctx_len[r] += a + 1 and anchor[r] = bonus[r].
 * So a following dflash_draft_cycle with n_rows = n_req * (D+1) and these
 * row_off / pos0 / feats appends exactly the accepted path to the cache and
 * drafts from the bonus token; every size is on the device, so the cycle can
 * be captured in a CUDA graph and replayed.  The drafter's block keys and
 * values never enter the cache, so rejected positions need no rollback.
 * Requires 1 <= D <= 16, 0 <= B <= 1024, feature rows and tree_ld multiples
 * of 16 bytes, 16-byte aligned buffers; dtype DFLASH_BF16 or DFLASH_F32.  The
 * caller guarantees ctx_len[r] + D + 1 <= the cache capacity (not checked on
 * the device).  Needs no workspace. */
dflash_status dflash_commit_accepted(int n_req, int D, int B, int feat_dim, int dtype,
                                     const void* tree_feats, long long tree_ld,
                                     const int32_t* accept_len, const int32_t* accepted,
                                     const int32_t* bonus, int32_t* ctx_len, int32_t* anchor,
                                     int32_t* row_off, int32_t* pos0, void* feats, void* stream);

/* Step a8: greedy verifier walk (DDTree page, 3.4.5).  From the root, while the
 * current node has a child whose token equals target_tok[current], move to it.
 *   target_tok int32 [n_req][B+1]  the target's choice at every node
 *   accept_len int32 [n_req]       accepted draft tokens (tau = accept_len + 1)
 *   accepted   int32 [n_req][D]    accepted node indices, -1 padded
 *   bonus      int32 [n_req]       target_tok at the node where the walk stops
 * Tree arrays as produced by ddtree_build with the same B. */
dflash_status ddtree_accept(int n_req, int D, int B, const int32_t* n_nodes,
                            const int32_t* tok, const int32_t* parent,
                            const int32_t* target_tok, int32_t* accept_len,
                            int32_t* accepted, int32_t* bonus, void* stream);

/* Verification-side tree attention (DDTree page, 3.4.5): one target-model
 * attention layer over the flattened draft tree.  Per request r, tree node i
 * (0 <= i <= n_nodes[r]; node 0 is the root) attends, head h reading KV head
 * h / (n_q / n_kv), to
 *   - the request's context: cache slots t < ctx_len[r] of cache_k / cache_v
 *     ([n_req][n_kv][cap][head_dim] bf16, as the drafter's cache), and
 *   - the tree nodes j whose bit j is set in mask row i (its ancestors and
 *     itself; the mask ddtree_build writes, [n_req][B+1][ceil((B+1)/32)]),
 * with softmax(q . key / sqrt(head_dim)) weights.
 *   q    bf16 [n_req][B+1][q_ld]: query heads at columns h * head_dim,
 *        already rotated at position ctx_len + depth (dflash_tree_rope)
 *   k, v bf16 [n_req][B+1][kv_ld]: the nodes' own keys (rotated) and values,
 *        KV head g at column g * head_dim
 *   out  bf16 [n_req][B+1][out_ld]: rows of nodes past n_nodes[r] are zero
 * Requires head_dim == 128, n_q a multiple of n_kv with at most 4 query heads
 * per KV head, 0 <= B <= 1024, 0 <= ctx_len[r] <= max_ctx <= cap, strides that
 * are multiples of 8 elements and 16-byte aligned cache, q, k and v.  Device
 * pointers; ws of dflash_tree_attention_workspace_bytes(...) bytes, zeroed once
 * (dflash_workspace_init) before the first call: it holds arrival counters that
 * every call leaves at zero.  Calls sharing a workspace must not overlap. */
size_t dflash_tree_attention_workspace_bytes(int n_req, int n_q, int n_kv, int head_dim, int B,
                                             int max_ctx);
dflash_status dflash_tree_attention(int n_req, int n_q, int n_kv, int head_dim, int B,
                                    const int32_t* ctx_len, int max_ctx, int cap,
                                    const void* cache_k, const void* cache_v, const void* q,
                                    long long q_ld, const void* k, const void* v, long long kv_ld,
                                    const uint32_t* mask, const int32_t* n_nodes, void* out,
                                    long long out_ld, void* ws, size_t ws_bytes, void* stream);

/* Depth position ids of the flattened tree (DDTree page, 3.4.5): rotates heads
 * 0 .. n_heads-1 of x[r][i] (rows of ld elements, dtype DFLASH_BF16 or
 * DFLASH_F32, in place) at position ctx_len[r] + depth[r][i] with the
 * rotate-half RoPE of base theta; rows with depth < 0 (past the last node) are
 * left alone.  depth is ddtree_build's [n_req][B+1] output. */
dflash_status dflash_tree_rope(int n_req, int B, int n_heads, int head_dim, float theta,
                               const int32_t* ctx_len, const int32_t* depth, void* x,
                               long long ld, int dtype, void* stream);

/* A paged KV cache of one target layer, for the verification pass over
 * requests whose contexts grow (the pages serve DFlash and DDTree from engines
 * that keep the target's cache in pages; DFlash page, section 4).  Slot t of
 * request r (its t-th token) lies in page table[r][t / page_size] at place
 * t % page_size.  Pages belong to the caller, may lie in any order, and a table
 * entry outside [0, n_pages) (say -1) is a page that is not there.
 *   k, v   T [n_pages][n_kv][page_size][head_dim] (device), 16-byte aligned
 *   table  int32 [n_req][table_ld] (device)
 * Requires page_size a power of two in [16, 1024], head_dim 64 or 128,
 * table_ld >= 1, table_ld * page_size <= 2^30, n_pages >= 1,
 * n_pages * n_kv * page_size < 2^31; dtype DFLASH_BF16 or DFLASH_F32. */
typedef struct dflash_pages {
  void* k;
  void* v;
  const int32_t* table;
  int table_ld;
  int n_pages;
  int page_size;
  int n_kv;
  int head_dim;
  int dtype;
} dflash_pages;

/* Per-head RMSNorm of queries and keys and their position rotation, in one pass
 * (the target of the pages' experiments normalises both per head before the
 * rotate-half RoPE).  For every row i and every head x of its n_q query and
 * n_kv key heads:
 *   y   = x / sqrt(mean(x^2) + eps) * gain      (gain NULL: no norm, y = x)
 *   out = RoPE(y, pos[i], theta)                (theta == 0: no rotation)
 * in fp32, rounded once.  A row whose pos is negative is left as it is (the
 * rows past a tree's last node); pos may be NULL when theta == 0.
 *   q, k          T [n_rows] rows q_ld / k_ld elements apart, head h at column
 *                 h * head_dim; q_out, k_out likewise.  q_out may be q and k_out
 *                 may be k (in place, with the same row stride); other overlap
 *                 is not allowed
 *   q_gain/k_gain T [head_dim]
 *   pos           int32 [n_rows] (device)
 * n_q or n_kv may be 0 (its pointers are then not read), and 16384 at most.
 * head_dim 64 or 128; T = dtype.  Any stride of at least heads * head_dim elements; rows and
 * buffers on 16-byte boundaries take the vector path.  Needs no workspace. */
dflash_status dflash_qk_norm_rope(int n_rows, int n_q, int n_kv, int head_dim, int dtype,
                                  const void* q_gain, const void* k_gain, float eps, float theta,
                                  const int32_t* pos, const void* q, long long q_ld,
                                  const void* k, long long k_ld, void* q_out,
                                  long long q_out_ld, void* k_out, long long k_out_ld,
                                  void* stream);

/* New keys and values into a paged cache, the keys rotated on the way.  Global
 * row row_off[r] + i of request r (i < row_off[r+1] - row_off[r]) goes to slot
 * pos0[r] + i, its key rotated at pos[row], or at its slot where pos is NULL
 * (theta == 0: stored as it comes, for keys dflash_qk_norm_rope has rotated).
 *   row_off  int32 [n_req+1] (device), row_off[0] = 0, non-decreasing; rows at
 *            or past row_off[n_req] are stored nowhere
 *   pos0     int32 [n_req] (device)   pos  int32 [n_rows] (device) or NULL
 *   k, v     T [n_rows] rows kv_ld elements apart, head g at column g*head_dim
 * Not stored: a row with a negative pos, and a row whose slot has no page (past
 * the table, or an entry outside [0, n_pages)).  No other slot is written.  Two
 * rows of one call must not share a slot (requests that share a page may share
 * only slots that neither writes).  n_rows may be 0, n_kv 8192 at most.  Needs
 * no workspace. */
dflash_status dflash_paged_append(const dflash_pages* pages, int n_req, int n_rows,
                                  const int32_t* row_off, const int32_t* pos0,
                                  const int32_t* pos, const void* k, const void* v,
                                  long long kv_ld, float theta, void* stream);

/* Attention of new tokens over a paged cache (DDTree page, 3.4.5, over pages):
 * the rows of request r, global rows row_off[r] .. row_off[r+1] - 1, are its
 * tokens at slots pos0[r] .., whose keys and values the cache already holds
 * (dflash_paged_append).  Row i of the request, head h reading KV head
 * h / (n_q / n_kv), takes softmax(q . key / sqrt(head_dim)) over
 *   mask NULL  slots t <= pos0[r] + i (causal: decoding, chains, prompt chunks)
 *   mask       slots t < pos0[r], and slots pos0[r] + j with bit j of its mask
 *              row set, j < row_off[r+1] - row_off[r]: a draft tree with the
 *              mask ddtree_build writes, or any other pattern.  A row with no
 *              bit set attends to the context alone.
 * A row that sees no slot gets zeros.  Keys and values no row may see are not
 * read into any result, whatever they hold.
 *   q     bf16 [n_rows] rows q_ld elements apart, head h at column h*head_dim
 *   mask  uint32 [n_rows][mask_ld] (device), bit j in word j / 32; mask_ld * 32
 *         >= the most rows of a request (bits past it count as not set)
 *   out   bf16 [n_rows] rows out_ld apart; rows at or past row_off[n_req] are
 *         left as they are
 * max_rows is a host bound on the rows of one request, used to choose the
 * kernel; it need not be tight, nor hold (results differ by the order of fp32
 * sums).  Sizes stay on the device, so a captured call serves contexts that
 * grow.  The work (requests x KV heads x query tiles x key tiles) is split
 * evenly over the SMs; a tile split between CTAs is joined in key order, so
 * results do not depend on timing.
 * DFLASH_ERR_INVALID_ARG in the workspace status word: some row sees a slot
 * whose page is not there (it reads as zeros), or a slot past the table,
 * pos0[r] + j >= table_ld * page_size (it is left out of the softmax), or a
 * request with rows has a pos0 that is negative (taken as 0) or past the table
 * (taken as its end).  Slots that no row sees, as behind a tree's last node,
 * need neither a page nor a place in the table.
 * Requires DFLASH_BF16 pages, n_q a multiple of n_kv, n_rows * n_q < 2^30,
 * strides that are multiples of 8 elements and 16-byte aligned q and out.  ws of
 * dflash_paged_attention_workspace_bytes bytes, zeroed once
 * (dflash_workspace_init) before the first call; every call leaves its counters
 * at zero, unless the status word reads DFLASH_ERR_TIMEOUT: then the workspace
 * has to be zeroed again.  Calls sharing a workspace must not overlap; it may
 * serve calls of any heads, of dflash_paged_attention_e4m3 too, if it has the
 * bytes that each asks for. */
size_t dflash_paged_attention_workspace_bytes(int n_q, int n_kv, int head_dim);
dflash_status dflash_paged_attention(const dflash_pages* pages, int n_req, int n_rows, int n_q,
                                     const int32_t* row_off, const int32_t* pos0, int max_rows,
                                     const void* q, long long q_ld, const uint32_t* mask,
                                     int mask_ld, void* out, long long out_ld, void* ws,
                                     size_t ws_bytes, void* stream);

/* A paged KV cache held in 8 bits: slots, pages and table as in dflash_pages,
 * elements as e4m3 codes (one sign, four exponent, three fraction bits; largest
 * 448, 0x7F and 0xFF NaN, no infinities), and one scale for every 16 slots (a
 * block) of a KV head, keys and values apart.  A scale is a power of two kept as
 * its biased exponent: byte b stands for 2^(b - 127) (255, which no append
 * writes, is read as 254), and an element for its code's value times its block's
 * scale.
 *   k, v              uint8 [n_pages][n_kv][page_size][head_dim] (device),
 *                     16-byte aligned
 *   k_scale, v_scale  uint8 [n_pages][n_kv][page_size / 16] (device)
 *   table             int32 [n_req][table_ld] (device)
 * Limits as for dflash_pages. */
typedef struct dflash_pages_e4m3 {
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  const int32_t* table;
  int table_ld;
  int n_pages;
  int page_size;
  int n_kv;
  int head_dim;
} dflash_pages_e4m3;

/* dflash_paged_append into a cache held in 8 bits; k and v are rows of T = dtype.
 * For every block that takes rows of a request, and each KV head of keys (rotated,
 * in fp32) and of values:
 *   e     the smallest exponent >= -127 with max |y| <= 448 * 2^e over the
 *         elements y that are stored; if slots of the block lie before pos0[r]
 *         (earlier tokens of the request), at least the block's present exponent,
 *         and where it grew their codes c become round(c * 2^(old - e))
 *   code  round(y * 2^-e), to the nearest, ties to even; NaN for a y that is
 *         infinite or NaN, which counts for no maximum
 * So a block that begins at or after pos0[r] forgets what it held, and slots at or
 * past pos0[r] (of a drafted token that was refused, say) are void.  A code keeps
 * its value exactly at a larger scale unless that value falls below 2^-6 of the
 * scale (the codes' subnormals): token by token or at once makes a difference
 * there alone.
 * Rows, row_off, pos0, pos, theta and rows that are not stored: as there.
 * Requests that share a page may share only blocks that neither writes.  Needs no
 * workspace. */
dflash_status dflash_paged_append_e4m3(const dflash_pages_e4m3* pages, int n_req, int n_rows,
                                       const int32_t* row_off, const int32_t* pos0,
                                       const int32_t* pos, int dtype, const void* k,
                                       const void* v, long long kv_ld, float theta, void* stream);

/* dflash_paged_attention over a cache held in 8 bits: the same rows, masks, bounds,
 * workspace rules (of dflash_paged_attention_e4m3_workspace_bytes bytes) and
 * errors; q and out bf16.  Codes enter the products as they are, exactly; scales
 * are applied to fp32 scores and weights.  A NaN code reaches the rows that see
 * its slot; what no row sees, scales included, may hold anything.  Sums are held
 * in fp32 and divided at the end: outputs are finite while the largest value times
 * the slots that a row sees stays below 2^113.  Queries enter as fp16 (rounded by
 * 2^-39 of a row's largest element at most) or, in requests of many rows, as two
 * e4m3 codes (2^-17), so max_rows moves results by that besides the order of sums. */
size_t dflash_paged_attention_e4m3_workspace_bytes(int n_q, int n_kv, int head_dim);
dflash_status dflash_paged_attention_e4m3(const dflash_pages_e4m3* pages, int n_req, int n_rows,
                                          int n_q, const int32_t* row_off, const int32_t* pos0,
                                          int max_rows, const void* q, long long q_ld,
                                          const uint32_t* mask, int mask_ld, void* out,
                                          long long out_ld, void* ws, size_t ws_bytes,
                                          void* stream);

/* Logits before sampling: bias, penalties for repeated tokens, and the tokens a
 * grammar allows, for the rows of every request, rows row_off[r] ..
 * row_off[r+1] - 1 (one decoded token, a drafted chain, the nodes of a tree).  In
 * this order, in fp32, rounded once:
 *   bias        y = l + bias_val[r][j] for v = bias_tok[r][j] (listed twice: the
 *               later entry counts)
 *   repetition  y = y > 0 ? y / repetition[r] : y * repetition[r] for a token that
 *               the row's past holds
 *   frequency,  y = y - frequency[r] * c - presence[r] for a token that it holds
 *   presence    c > 0 times outside the prompt
 *   allowed     y = -inf where bit v % 32 of word v / 32 of the row is not set
 * A row's past: history[r][0 .. history_len[r]), of which the first prompt_len[r]
 * are the prompt's (the request's tokens before its rows), then the tokens
 * tok[row_off[r] + j] of the rows j of its request that it sees, by bit j of its
 * mask row (a tree: its ancestors and itself; the mask ddtree_build writes), or
 * j <= its own place where mask is NULL.  So drafted rows are penalised as they
 * would be if their path had been generated.  Tokens outside [0, vocab) count for
 * nothing (-1 fills a list).
 *   logits   T [rows] rows ld elements apart, T = dtype; out T likewise, out_ld
 *            apart.  out may be logits (with one row stride); other overlap is
 *            not allowed.  Columns from vocab on, and rows at or past
 *            row_off[n_req], are left as they are
 *   history  int32 [n_req][history_ld]; history_len, prompt_len int32 [n_req]
 *            (lengths below 0 count as 0, past history_ld as history_ld;
 *            prompt_len NULL: 0).  history may be NULL: none
 *   repetition, presence, frequency  fp32 [n_req], NULL: off
 *   tok      int32 [rows], NULL: rows' own tokens count for nothing
 *   mask     uint32 [rows][mask_ld], NULL: a chain.  Bits past mask_ld words are
 *            not set
 *   bias_tok int32, bias_val fp32 [n_req][n_bias], n_bias 0: none
 *   allowed  uint32 [rows] rows allowed_ld words apart, NULL: all
 * All device pointers; lengths and offsets stay on the device, so a captured call
 * serves histories that grow.  Results do not depend on timing.  rows may be 0.
 * Requires 1 <= vocab <= 2^22, history_ld <= 2^30, allowed_ld * 32 >= vocab,
 * n_bias <= 2^20, rows + n_req < 2^30.  Needs no workspace. */
dflash_status dflash_logits_adjust(int n_req, int rows, int vocab, int dtype, const void* logits,
                                   long long ld, void* out, long long out_ld,
                                   const int32_t* row_off, const int32_t* history, int history_ld,
                                   const int32_t* history_len, const int32_t* prompt_len,
                                   const float* repetition, const float* presence,
                                   const float* frequency, const int32_t* tok,
                                   const uint32_t* mask, int mask_ld, const int32_t* bias_tok,
                                   const float* bias_val, int n_bias, const uint32_t* allowed,
                                   long long allowed_ld, void* stream);

/* The target's token of every row, from given random numbers (DFlash page,
 * 3.4.4: verification at temperature 1; DDTree page, 3.4.5: the walk's target
 * choices).  Per row, over logits l and in this order:
 *   temperature  w_v = exp((l_v - max l) / T); T <= 0 (or NaN): the best token
 *   top_k        k > 0 keeps the k best tokens (logit desc, id asc)
 *   top_p        p < 1 keeps, of those in that order, a token if the mass before
 *                it is below p times theirs (the best always)
 *   min_p        m > 0 keeps tokens with l_v - max l >= T ln m, and from m = 1 on
 *                those alone that equal the best, at any T
 *   draw         the first kept token, by id, whose cumulated mass exceeds u
 *                times the kept mass, u in [0, 1) (clamped)
 *   tok  int32 [rows], logp fp32 [rows] (device) out: the token, and the log of
 *        its share of the kept mass (0 for T <= 0)
 *   temperature, top_p, min_p, u  fp32 [rows], top_k int32 [rows] (device); a
 *        NULL parameter is off (temperature: 1), u is required
 * A NaN logit counts as -inf; tokens at -inf are never drawn; where some are
 * +inf they share the mass.  A row of -inf alone gives tok -1, logp -inf.
 *   logits  [rows] of dtype, ld elements apart, vocab <= ld
 * A token's mass is its fp32 exponential in steps of 2^-40 of the best's, and
 * masses are added as 64-bit whole numbers, so results depend neither on timing
 * nor on the other rows, their number included.  rows may be 0.
 * Requires 1 <= vocab <= 2^22.  Needs no workspace. */
dflash_status dflash_logits_sample_filtered(int rows, int vocab, long long ld, int dtype,
                                            const void* logits, const float* temperature,
                                            const int32_t* top_k, const float* top_p,
                                            const float* min_p, const float* u, int32_t* tok,
                                            float* logp, void* stream);

/* The dense contraction every step above is built on, exposed on its own:
 * Y[M][N] = X[M][K] . W[N][K]^T with bf16 X and W and fp32 Y, on the tcgen05
 * tensor cores (the same kernel, work split and reduction the drafter's GEMMs
 * use, with a plain fp32 store as epilogue).  Requires K % 64 == 0, N % 128 ==
 * 0, X, W 16-byte aligned; M >= 0.  ws of dflash_linear_workspace_bytes(M, N,
 * K) bytes, zero-initialised once. */
size_t dflash_linear_workspace_bytes(int M, int N, int K);
dflash_status dflash_linear_bf16(int M, int N, int K, const void* X, const void* W, float* Y,
                                 void* ws, size_t ws_bytes, void* stream);

/* Launch tracing.  When a hook is set, the library calls it on the host right
 * before (phase 0) and right after (phase 1) it enqueues each kernel, with the
 * kernel's name and the stream, so a caller can record CUDA events around
 * every kernel (also while a stream is being captured into a graph).  One hook
 * per process; NULL removes it.  The hook must not call back into the library. */
typedef void (*dflash_trace_fn)(void* user, const char* kernel, int phase, void* stream);
void dflash_set_trace_hook(dflash_trace_fn fn, void* user);

/* Thread-local message for the calling thread's last non-OK status. */
const char* dflash_last_error(void);
int dflash_abi_version(void);

#ifdef __cplusplus
}
#endif
#endif /* DFLASH_H */
