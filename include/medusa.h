/*
 * medusa.h - C ABI of the Medusa decode-verify step on NVIDIA B200 (sm_100a).
 *
 * One decode-verify step of Medusa speculative decoding, in five stage calls:
 *
 *   medusa_heads_topk      K Medusa heads on the last hidden state, then a
 *                          top-k over the vocabulary per head;
 *   medusa_tree_build      candidate tree from those top-k lists: candidate
 *                          ids, position ids, ancestor mask, retrieve paths;
 *   medusa_tree_attention  attention of every tree node over the cached
 *                          prefix and its own ancestors;
 *   medusa_verify_accept   the longest branch the base model agrees with
 *                          (greedy match or typical acceptance);
 *   medusa_kv_compact      the kept branch's K/V moved into contiguous slots.
 *
 * Around them: medusa_lmhead_verify (the verification from the nodes' hidden
 * states, lm_head fused), medusa_next_step (inputs of the next step),
 * medusa_sample_bonus (a drawn bonus token), medusa_heads_topk_tree and
 * medusa_verify_accept_compact (the first two and the last two calls, each
 * pair in one), medusa_tree_from_accuracies
 * (the sparse tree of the most accurate combinations, host only), the
 * vocabulary-sharding calls (medusa_topk_merge, medusa_verify_records,
 * medusa_verify_from_records), medusa_verify_accept_noalloc and
 * medusa_wait_flag (a check of the bounded device waits).  Before them, the
 * prompt side: medusa_rope, medusa_rope_append, medusa_chunk_attention and
 * medusa_sample_tokens (with medusa_rope_freqs on the host).
 *
 * Sources (page title, then section):
 *   "Medusa Heads" glossary - "Comment les têtes prédisent les tokens
 *     suivants" (the head) and "Attention arborescente et acceptation" (tree,
 *     tree mask, greedy and typical acceptance, longest kept branch);
 *   "Medusa Decoding Heads" overview - "Diepe duik" (one-pass verification of
 *     the whole tree, losslessness);
 *   "Medusa no contexto de LLMs" - "o que significa medusa na prática de
 *     deploy" (accepted tokens enter the sequence without another pass; the
 *     conventionally generated token on rejection);
 *   "Medusa: Simple LLM Inference Acceleration Framework with Multiple
 *     Decoding Heads" - abstract (tree-based attention over candidate
 *     continuations, one decoding step).
 *
 * Conventions for every call
 *   - Pointers named as device pointers must point to memory of the current
 *     CUDA device; host pointers are read before the call returns.  The
 *     caller owns every buffer.  The library never allocates device memory
 *     and never synchronises: all work is enqueued on `stream`
 *     (a cudaStream_t passed as void*; NULL = legacy default stream).
 *   - All arrays are dense, row-major, with the layouts given per call.
 *     bf16 arrays are IEEE bfloat16 bit patterns (uint16).
 *   - Errors the host can see (null pointer, unsupported size, misaligned
 *     pointer, workspace too small) are returned before anything is launched.
 *     MEDUSA_ERR_CUDA reports a failed launch; medusa_last_error() then holds
 *     the CUDA error text.
 *   - Errors only the device can see (an index out of range in a tree or an
 *     accepted path, a NaN logit, a bounded wait that ran out) are written
 *     into *dev_status (device int32, 0 = OK) with an atomic compare-and-swap,
 *     so the first error sticks.  The caller zeroes it once and reads it after
 *     its own synchronisation.  No kernel traps; outputs of a call that set a
 *     device error are unspecified but every write stays inside its buffer.
 *   - The library is re-entrant.  Calls on the same stream run in order; the
 *     caller orders calls on different streams.
 */
#ifndef MEDUSA_B200_H
#define MEDUSA_B200_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define MEDUSA_API __attribute__((visibility("default")))
#else
#define MEDUSA_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  MEDUSA_OK = 0,
  MEDUSA_ERR_INVALID_ARG = 1,  /* null pointer, bad enum, negative size      */
  MEDUSA_ERR_SHAPE = 2,        /* sizes outside the supported limits          */
  MEDUSA_ERR_UNSUPPORTED = 3,  /* valid request this build does not handle    */
  MEDUSA_ERR_CUDA = 4,         /* a CUDA runtime/driver call failed           */
  MEDUSA_ERR_TIMEOUT = 5,      /* device: a bounded wait ran out              */
  MEDUSA_ERR_DEVICE_CHECK = 6, /* device: index out of range, NaN input       */
  MEDUSA_ERR_WORKSPACE = 7,    /* workspace pointer null or too small         */
  MEDUSA_ERR_ALIGNMENT = 8     /* pointer not aligned as the call requires    */
} medusa_status_t;

typedef enum { MEDUSA_BF16 = 0, MEDUSA_F32 = 1 } medusa_dtype_t;
typedef enum { MEDUSA_ACCEPT_GREEDY = 0, MEDUSA_ACCEPT_TYPICAL = 1 } medusa_accept_t;

/* Limits of this build. */
#define MEDUSA_MAX_NODES 256   /* tree nodes, root included                  */
#define MEDUSA_MAX_KMAX 32     /* top-k width per head                       */
#define MEDUSA_MAX_HEADS 16    /* Medusa heads = deepest possible tree level */
#define MEDUSA_MAX_BATCH 128   /* sequences per call (bf16 heads)            */

/*
 * A candidate tree.  Nodes are in breadth-first order (parents before
 * children); node 0 is the root.  The struct lives in host memory; the three
 * arrays are DEVICE arrays of n_nodes int32 each:
 *   parent[i]  parent node (parent[0] = -1, 0 <= parent[i] < i otherwise);
 *   depth[i]   depth (depth[0] = 0, depth[i] = depth[parent[i]] + 1);
 *   rank[i]    for i > 0, which entry of head depth[i]'s top-k list the node
 *              carries (0 <= rank[i] < kmax).
 * max_depth is the largest depth[i]; n_leaves the number of nodes without a
 * child.  Kernels check these relations and report violations through
 * dev_status.
 */
typedef struct medusa_tree {
  int32_t n_nodes;
  int32_t max_depth;
  int32_t n_leaves;
  const int32_t* parent;
  const int32_t* depth;
  const int32_t* rank;
} medusa_tree_t;

/* Text for a status code (static storage). */
MEDUSA_API const char* medusa_status_string(medusa_status_t status);
/* Text of the last failing call on this host thread ("" if none). */
MEDUSA_API const char* medusa_last_error(void);
/* ABI version: major*10000 + minor*100 + patch. */
MEDUSA_API int medusa_version(void);

/* ------------------------------------------------------------------------
 * medusa_heads_topk
 *
 * "Medusa Heads" glossary, "Comment les têtes prédisent les tokens
 * suivants": head k is one feed-forward layer with a SiLU activation and a
 * residual connection, followed by a projection to the vocabulary; every
 * head reads the same last hidden state.  "Attention arborescente et
 * acceptation": the heads' top choices (top-2, top-3, ...) feed the tree.
 *
 *   y_k   = h + SiLU(W1_k h + b1_k)
 *   z_k   = W2_k y_k                      (no bias)
 *   top-kmax of z_k per (sequence, head): values descending, equal values by
 *   ascending token id.
 *
 * Inputs (device, dtype dt for h/W1/b1/W2):
 *   h  [B, d]        last hidden state per sequence
 *   W1 [K, d, d]     W1[k][j][:] = weights of output feature j (Linear layout)
 *   b1 [K, d]
 *   W2 [K, V, d]     W2[k][v][:] = weights of token v
 * Outputs (device):
 *   topk_ids  [B, K, kmax] int32
 *   topk_vals [B, K, kmax] float32
 *   logits    [B, K, V] float32, or NULL to skip (parity checks).
 * Workspace: ws of at least medusa_heads_topk_workspace_size(...) bytes,
 *   256-byte aligned; contents on entry are ignored.
 * Precision: bf16 inputs, fp32 accumulation; y is fed to the vocabulary
 *   projection as the sum of two bf16 terms (hi + lo) so its rounding stays
 *   far below the fp32 accumulation error.  dt = MEDUSA_F32 runs an fp32
 *   CUDA-core path (small shapes).
 * Limits: 1 <= B <= MEDUSA_MAX_BATCH, 1 <= K <= MEDUSA_MAX_HEADS,
 *   1 <= kmax <= min(MEDUSA_MAX_KMAX, V); bf16: d % 64 == 0, all pointers
 *   16-byte aligned.
 * ---------------------------------------------------------------------- */
MEDUSA_API size_t medusa_heads_topk_workspace_size(int B, int d, int V, int K, int kmax,
                                        medusa_dtype_t dt);
MEDUSA_API medusa_status_t medusa_heads_topk(const void* h, const void* W1, const void* b1,
                                  const void* W2, medusa_dtype_t dt, int B, int d,
                                  int V, int K, int kmax, int32_t* topk_ids,
                                  float* topk_vals, float* logits, void* ws,
                                  size_t ws_bytes, int32_t* dev_status,
                                  void* stream);

/* ------------------------------------------------------------------------
 * medusa_tree_build
 *
 * "Medusa Heads" glossary, "Attention arborescente et acceptation": the
 * heads' top choices combine into candidate continuations forming a tree
 * (a Cartesian product, or a sparse selection of it); head 2 proposes the
 * same tokens under every head-1 branch; a mask lets each token see only its
 * ancestors in the tree.
 *
 *   cand_ids[b][0] = root_tok[b] (the base model's own next token);
 *   cand_ids[b][i] = topk_ids[b][depth[i]-1][rank[i]] for i > 0;
 *   pos_ids[b][i]  = prefix_len[b] + depth[i];
 *   anc_mask[i][w] bit t set iff node 32*w+t is i or an ancestor of i;
 *   retrieve[p][t] = node at depth t on the path root -> p-th leaf (leaves in
 *                    node order), -1 past the leaf.
 *
 * Inputs (device): root_tok [B] int32, topk_ids [B, K, kmax] int32,
 *   prefix_len [B] int32; tree as above (depth[i] <= K required).
 * Outputs (device): cand_ids [B, N], pos_ids [B, N] int32;
 *   anc_mask [N, ceil(N/32)] uint32; retrieve [n_leaves, max_depth+1] int32.
 * Limits: N <= MEDUSA_MAX_NODES, max_depth <= K <= MEDUSA_MAX_HEADS,
 *   kmax <= MEDUSA_MAX_KMAX.
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_tree_build(const medusa_tree_t* tree, const int32_t* root_tok,
                                  const int32_t* topk_ids, int K, int kmax,
                                  const int32_t* prefix_len, int B, int32_t* cand_ids,
                                  int32_t* pos_ids, uint32_t* anc_mask,
                                  int32_t* retrieve, int32_t* dev_status,
                                  void* stream);

/* ------------------------------------------------------------------------
 * medusa_heads_topk_tree
 *
 * medusa_heads_topk followed by medusa_tree_build of its top-k lists, in the
 * launches of medusa_heads_topk alone: the thread block that finishes the
 * last of a sequence's K lists builds that sequence's candidates (the
 * sections cited at the two calls).  Every output equals that of the two
 * calls made one after the other on the same stream, with the tree build's
 * K and kmax the heads'.
 *
 * Arguments: those of medusa_heads_topk, then those of medusa_tree_build
 *   (tree, root_tok [B], prefix_len [B]; cand_ids, pos_ids [B, N]; anc_mask
 *   [N, ceil(N/32)]; retrieve [n_leaves, max_depth+1]).  Workspace as
 *   medusa_heads_topk.
 * Host checks: medusa_heads_topk's arguments, then the tree's (as
 *   medusa_tree_build), then the workspace; nothing is launched on an error.
 * Device checks: medusa_tree_build's.
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_heads_topk_tree(
    const void* h, const void* W1, const void* b1, const void* W2, medusa_dtype_t dt, int B, int d,
    int V, int K, int kmax, int32_t* topk_ids, float* topk_vals, float* logits, void* ws,
    size_t ws_bytes, const medusa_tree_t* tree, const int32_t* root_tok, const int32_t* prefix_len,
    int32_t* cand_ids, int32_t* pos_ids, uint32_t* anc_mask, int32_t* retrieve, int32_t* dev_status,
    void* stream);

/* ------------------------------------------------------------------------
 * medusa_tree_attention
 *
 * "Medusa Heads" glossary, "Attention arborescente et acceptation": every
 * candidate token is appended to the input at once and attends only to its
 * ancestors, so one forward pass scores every branch; abstract of the Medusa
 * paper: tree-based attention verifies all candidates in one step.
 *
 * The N tree tokens' K/V are written to cache slots prefix_len[b] + i.  Query
 * (node i, head hq) then attends with weights softmax(scale * q.k) to slots
 * [0, prefix_len[b]) and to slots prefix_len[b] + j for every j set in
 * anc_mask row i.  Query head hq reads kv head hq / (Hq / Hkv).  No
 * positional rotation is applied: q and k are taken as already positioned.
 *
 * Inputs (device, dtype dt): q [B, N, Hq, dh]; k_new, v_new [B, N, Hkv, dh];
 *   caches Kc, Vc [B, Hkv, cap, dh] (read, and written at the tree slots);
 *   prefix_len [B] int32 with prefix_len[b] <= max_prefix and
 *   prefix_len[b] + N <= cap; anc_mask from medusa_tree_build.
 * Output (device): out [B, N, Hq, dh] of dtype out_dt (bf16 or f32).
 * max_prefix: host-side upper bound on every prefix_len[b]; sizes the launch.
 * Workspace: medusa_tree_attention_workspace_size(...) bytes (partial
 *   results of key ranges, merged at the end), 256-byte aligned.
 * Precision: bf16 q/k/v, fp32 scores, fp32 softmax statistics; the softmax
 *   weights (at most 2^8 relative to the running maximum) enter the value
 *   product as fp16, with V converted to fp16 in shared memory.  A V tile
 *   that fp16 cannot carry (some |v| >= 65536, or every |v| < 2^-6, where fp16
 *   would lose mantissa bits) puts its kv head's query rows on a list that an
 *   exact pass recomputes afterwards on CUDA cores in fp32, so any finite bf16
 *   V is supported; with no such tile the pass only reads an empty list.  Inf
 *   or NaN in V is reported as MEDUSA_ERR_DEVICE_CHECK.
 *   dt = MEDUSA_F32 runs an fp32 CUDA-core path.
 * Limits: Hq % Hkv == 0; bf16: dh in {64, 128}, B <= 256, pointers 16-byte
 *   aligned; f32: dh <= 256 and dh % 32 == 0; N <= MEDUSA_MAX_NODES.
 * ---------------------------------------------------------------------- */
MEDUSA_API size_t medusa_tree_attention_workspace_size(int B, int N, int Hq, int Hkv, int dh,
                                            int max_prefix, medusa_dtype_t dt);
MEDUSA_API medusa_status_t medusa_tree_attention(const void* q, const void* k_new, const void* v_new,
                                      void* Kc, void* Vc, const int32_t* prefix_len,
                                      const uint32_t* anc_mask, medusa_dtype_t dt, int B,
                                      int N, int Hq, int Hkv, int dh, int cap,
                                      int max_prefix, float scale, void* out,
                                      medusa_dtype_t out_dt, void* ws, size_t ws_bytes,
                                      int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * medusa_verify_accept
 *
 * "Medusa Heads" glossary, "Attention arborescente et acceptation": the
 * longest branch the model agrees with is kept.  Greedy: a candidate is
 * accepted when it equals the model's first choice.  Typical: a candidate is
 * kept when its probability under the base model exceeds a threshold tied to
 * the entropy of the distribution; here thr = min(eps, delta * exp(-H(p))),
 * p = softmax(logits / temperature), H in nats, strict ">".  "Medusa no
 * contexto de LLMs": on rejection the conventionally generated token is
 * used (the bonus token).
 *
 *   g[i]   = argmax_v logits[b][i][v] (lowest v among equal maxima);
 *   node c > 0 passes iff g[parent[c]] == cand_ids[b][c] (greedy) or
 *          p_parent[c](cand_ids[b][c]) > thr_parent[c] (typical);
 *   the root is accepted; c is accepted iff it passes and parent[c] is;
 *   kept node = deepest accepted node, lowest index among equally deep;
 *   accept_len[b] = its depth; accepted_nodes[b] = root..kept node, then -1;
 *   accepted_tokens[b] = kept candidates' tokens (root excluded), then the
 *   bonus token, then -1; bonus[b] = g[kept node].
 *
 * Inputs (device): logits [B, N, V] of dtype dt; cand_ids [B, N] int32; tree.
 * Outputs (device): accept_len [B], accepted_nodes [B, max_depth+1],
 *   accepted_tokens [B, max_depth+1], bonus [B], all int32.
 * Workspace: medusa_verify_accept_workspace_size(...) bytes, 256-byte aligned.
 * Limits: N <= MEDUSA_MAX_NODES; temperature > 0 (typical); eps, delta >= 0.
 * Device checks: a NaN logit, a candidate id outside [0, V).
 * ---------------------------------------------------------------------- */
MEDUSA_API size_t medusa_verify_accept_workspace_size(int B, int N, int V);
MEDUSA_API medusa_status_t medusa_verify_accept(const void* logits, medusa_dtype_t dt,
                                     const int32_t* cand_ids, const medusa_tree_t* tree,
                                     int B, int V, medusa_accept_t mode, float temperature,
                                     float eps, float delta, int32_t* accept_len,
                                     int32_t* accepted_nodes, int32_t* accepted_tokens,
                                     int32_t* bonus, void* ws, size_t ws_bytes,
                                     int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * medusa_kv_compact
 *
 * "Medusa no contexto de LLMs": an accepted candidate enters the sequence
 * without another full pass; "Medusa Heads" glossary: only the longest
 * accepted branch is kept.  The cache therefore keeps the kept branch's K/V
 * in contiguous slots after the prefix and drops the rest of the tree.
 *
 *   for j = 0..L (L = accept_len[b], P = prefix_len[b]):
 *       slot P + j of Kc and Vc (every kv head) <- slot P + accepted_nodes[b][j]
 *   (as if done for ascending j; the kernel stages the sources first, so the
 *   result is the same whichever slots overlap);
 *   compact_src[b][j] = P + accepted_nodes[b][j] for j <= L, else -1;
 *   prefix_len[b] = P + L + 1.
 *
 * In/out (device): Kc, Vc [B, Hkv, cap, dh] of dtype dt; prefix_len [B] int32.
 * Inputs (device): accepted_nodes [B, max_depth+1], accept_len [B] int32.
 * Output (device): compact_src [B, max_depth+1] int32.
 * Limits: max_depth < MEDUSA_MAX_HEADS; bf16 pointers 16-byte aligned.
 * Device checks: accept_len outside [0, max_depth], a source slot outside
 *   [P, cap).
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_kv_compact(void* Kc, void* Vc, medusa_dtype_t dt, int32_t* prefix_len,
                                  const int32_t* accepted_nodes, const int32_t* accept_len,
                                  int B, int Hkv, int dh, int cap, int max_depth,
                                  int32_t* compact_src, int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * medusa_verify_accept_compact
 *
 * medusa_verify_accept followed by medusa_kv_compact of its result, in the
 * same launches as medusa_verify_accept alone: the block that picks a
 * sequence's kept branch then moves that branch's K/V (the sections cited at
 * the two calls).  Results, in every output of both calls, equal those of
 * the two calls made one after the other on the same stream.
 *
 * Arguments: those of medusa_verify_accept, then the caches Kc, Vc
 *   [B, Hkv, cap, dh] of dtype kv_dt, prefix_len [B] (in/out) and
 *   compact_src [B, max_depth+1] (out) as in medusa_kv_compact; its B and
 *   max_depth are the verification's.  Workspace as medusa_verify_accept.
 * Host checks: medusa_verify_accept's, then medusa_kv_compact's, then the
 *   workspace; nothing is launched on an error.
 * Device checks: medusa_verify_accept's; a kept slot P + node outside
 *   [0, cap).  A sequence whose tree fails the device check, or whose kept
 *   slots fail it, is not compacted and its prefix_len is unchanged.
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_verify_accept_compact(
    const void* logits, medusa_dtype_t dt, const int32_t* cand_ids, const medusa_tree_t* tree,
    int B, int V, medusa_accept_t mode, float temperature, float eps, float delta,
    int32_t* accept_len, int32_t* accepted_nodes, int32_t* accepted_tokens, int32_t* bonus,
    void* Kc, void* Vc, medusa_dtype_t kv_dt, int32_t* prefix_len, int Hkv, int dh, int cap,
    int32_t* compact_src, void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * medusa_verify_accept_noalloc
 *
 * No counterpart on the Medusa pages: a service of this library for callers
 * that cannot provide device memory per call - a host framework that reserves
 * all device memory up front and forbids allocating more at run time, or hot
 * paths that must avoid cudaMalloc/cudaFree because those calls can
 * synchronise the device.
 *
 * Same arguments, results, checks and errors as medusa_verify_accept, without
 * ws/ws_bytes: the row statistics go to a 4 MiB array compiled into the
 * library (every GPU that loads the library holds it until the process
 * exits).  Requests needing more, i.e. B * n_nodes * ceil(V / 4096) * 16 bytes
 * > 4 MiB, are rejected with MEDUSA_ERR_WORKSPACE before any launch, after
 * the argument checks medusa_verify_accept makes (so a bad tree or shape gets
 * the same error as there).  Nothing is allocated.  Every call looks up the
 * array's device address (cudaGetSymbolAddress, a host-side query) with the
 * caller's device and context current, so the address stays right after a
 * device reset or in another context; the first call on a device may load
 * the library's device code there, so make it before any stream capture.
 * All calls share the one array and it keeps the last call's contents:
 * calls whose kernels overlap on the GPU (e.g. on two streams at once) race
 * and give wrong results.
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_verify_accept_noalloc(
    const void* logits, medusa_dtype_t dt, const int32_t* cand_ids, const medusa_tree_t* tree,
    int B, int V, medusa_accept_t mode, float temperature, float eps, float delta,
    int32_t* accept_len, int32_t* accepted_nodes, int32_t* accepted_tokens, int32_t* bonus,
    int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * medusa_lmhead_verify
 *
 * "Medusa Heads" glossary, "Attention arborescente et acceptation": one
 * forward pass scores every tree node, and the longest branch the base model
 * agrees with is kept; "Comment les têtes prédisent les tokens suivants": the
 * base model's next-token scores at a node are its lm_head applied to the
 * node's last hidden state.
 *
 * The verification of medusa_verify_accept, with the verify logits never
 * materialised: logits[b][i][v] = sum_j lm_head[v][j] * hidden[b][i][j]
 * (bf16 inputs, fp32 accumulation on the tensor cores), reduced tile by tile
 * to each node's argmax (greedy) or to its log-sum-exp and entropy
 * (typical); then exactly the acceptance rules of medusa_verify_accept.  In
 * typical mode the candidate's logit at its parent is recomputed as one dot
 * product (fp32), so near the threshold its decision may differ from one
 * taken on the GEMM's own value by the rounding of the two sums.
 *
 * Inputs (device): hidden [B, N, d] bf16 (node rows in tree order); lm_head
 *   [V, d] bf16 (torch Linear layout, no bias); cand_ids [B, N] int32; tree.
 * Outputs (device): accept_len [B], accepted_nodes [B, max_depth+1],
 *   accepted_tokens [B, max_depth+1], bonus [B] (int32, as
 *   medusa_verify_accept).  logits: optional [B, N, V] fp32 copy of the
 *   logits for checking (NULL in normal use; it adds B*N*V*4 bytes of writes).
 * dt must be MEDUSA_BF16 (MEDUSA_ERR_UNSUPPORTED otherwise).
 * Workspace: medusa_lmhead_verify_workspace_size(...) bytes, 256-byte
 *   aligned; the size depends on the current device's multiprocessor count.
 * Limits: d a positive multiple of 64; N <= MEDUSA_MAX_NODES; B * N <= 65535;
 *   hidden and lm_head 16-byte aligned; temperature > 0 (typical).
 * Device checks: a NaN logit, a candidate id outside [0, V).
 * ---------------------------------------------------------------------- */
MEDUSA_API size_t medusa_lmhead_verify_workspace_size(int B, int N, int d, int V);
MEDUSA_API medusa_status_t medusa_lmhead_verify(
    const void* hidden, const void* lm_head, medusa_dtype_t dt, const int32_t* cand_ids,
    const medusa_tree_t* tree, int B, int d, int V, medusa_accept_t mode, float temperature,
    float eps, float delta, int32_t* accept_len, int32_t* accepted_nodes,
    int32_t* accepted_tokens, int32_t* bonus, float* logits, void* ws, size_t ws_bytes,
    int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * medusa_next_step
 *
 * "Medusa Heads" glossary, "Attention arborescente et acceptation": the
 * accepted candidates join the sequence, and the heads of the next round
 * read the base model's last hidden state - that of the kept node; "Medusa
 * no contexto de LLMs": the base model's own token at the kept node (the
 * bonus token) is the next generated token, the next tree's root.
 *
 *   kept = accepted_nodes[b][accept_len[b]];
 *   h_next[b][:] = node_hidden[b][kept][:];   root_next[b] = bonus[b].
 *
 * Inputs (device): node_hidden [B, N, d] of dtype dt (the base model's last
 *   hidden states of the tree nodes); accept_len [B], accepted_nodes
 *   [B, max_depth+1], bonus [B] (int32, as written by the verification).
 * Outputs (device): h_next [B, d] of dtype dt; root_next [B] int32.
 * Limits: d * element size a multiple of 16; N <= MEDUSA_MAX_NODES;
 *   node_hidden and h_next 16-byte aligned.
 * Device checks: accept_len outside [0, max_depth] or a kept node outside
 *   [0, N) (that sequence's outputs are left unwritten).
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_next_step(const void* node_hidden, medusa_dtype_t dt,
                                            const int32_t* accept_len,
                                            const int32_t* accepted_nodes, const int32_t* bonus,
                                            int B, int N, int d, int max_depth, void* h_next,
                                            int32_t* root_next, int32_t* dev_status,
                                            void* stream);

/* ------------------------------------------------------------------------
 * Vocabulary sharding (several GPUs, each holding a slice of the vocabulary)
 *
 * No counterpart on the pages; these calls split medusa_heads_topk and
 * medusa_verify_accept at their only reduction over the vocabulary, so that
 * a caller can keep W2 rows and verify logits for tokens [v_offset,
 * v_offset + V_shard) on each GPU and exchange a few KB between them (for
 * example one all-gather and one max all-reduce).  The arithmetic of every
 * shard and of the merge runs here; the exchange is the caller's.
 *
 * A row record summarises one row of logits over a set of tokens: its
 * largest logit, the lowest token id holding it, and for typical acceptance
 * s = sum exp(z/T - maxz/T) and t = sum exp(z/T - maxz/T) * z/T.
 * ---------------------------------------------------------------------- */
typedef struct medusa_row_record {
  float maxz;
  int32_t idx;
  float s;
  float t;
} medusa_row_record_t;

/* medusa_topk_merge: the best kmax of n_lists lists of list_len candidates
 * per row (values descending, equal values by ascending id).  Candidate j of
 * list g of row r is vals/ids[r * row_stride + g * list_stride + j] (device);
 * its id gains id_offsets[g] (device int32 [n_lists], or NULL).  With the
 * per-shard outputs of medusa_heads_topk all-gathered as [G][B*K][kmax]:
 * rows = B*K, n_lists = G, list_len = kmax, row_stride = kmax, list_stride =
 * B*K*kmax, id_offsets = each shard's first token.  Outputs (device):
 * topk_ids, topk_vals [rows, kmax].  Limits: kmax <= MEDUSA_MAX_KMAX and
 * <= n_lists * list_len; rows <= 65535. */
MEDUSA_API medusa_status_t medusa_topk_merge(const float* vals, const int32_t* ids, int rows,
                                             int n_lists, int list_len, long long row_stride,
                                             long long list_stride, const int32_t* id_offsets,
                                             int kmax, int32_t* topk_ids, float* topk_vals,
                                             void* stream);

/* medusa_verify_records: this shard's row records and candidate logits.
 * Inputs (device): logits [B, N, V_shard] of dtype dt (tokens v_offset ..
 * v_offset + V_shard - 1), cand_ids [B, N] (global token ids), tree.
 * Outputs (device): records [B*N] (token ids global); cand_logit [B*N]
 * float: node c's candidate token's logit at its parent when that token is in
 * this shard, else -inf (root: -inf).  Workspace:
 * medusa_verify_records_workspace_size(B, N, V_shard) bytes, 256-aligned. */
MEDUSA_API size_t medusa_verify_records_workspace_size(int B, int N, int V_shard);
MEDUSA_API medusa_status_t medusa_verify_records(const void* logits, medusa_dtype_t dt,
                                                 const int32_t* cand_ids,
                                                 const medusa_tree_t* tree, int B, int V_shard,
                                                 int v_offset, medusa_accept_t mode,
                                                 float temperature,
                                                 medusa_row_record_t* records, float* cand_logit,
                                                 void* ws, size_t ws_bytes, int32_t* dev_status,
                                                 void* stream);

/* medusa_verify_from_records: the verification of medusa_verify_accept from
 * the G shards' records, shard-major [G][B*N] (device), and the candidate
 * logits [B*N] maximised over the shards (device; typical mode only, may be
 * NULL for greedy).  V is the full vocabulary size.  Outputs as
 * medusa_verify_accept. */
MEDUSA_API medusa_status_t medusa_verify_from_records(
    const medusa_row_record_t* records, int G, const float* cand_logit, const int32_t* cand_ids,
    const medusa_tree_t* tree, int B, int V, medusa_accept_t mode, float temperature, float eps,
    float delta, int32_t* accept_len, int32_t* accepted_nodes, int32_t* accepted_tokens,
    int32_t* bonus, int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * medusa_sample_bonus
 *
 * "Medusa no contexto de LLMs", "o que significa medusa na prática de
 * deploy": the token the base model generates itself at the kept node enters
 * the sequence after the kept candidates.  medusa_verify_accept writes its
 * first choice; this call replaces it with a draw from the base model's
 * distribution there, p = softmax(logits[b][kept] / temperature):
 *
 *   x = first word of Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel
 *       Random Numbers: As Easy as 1, 2, 3", SC 2011) with key
 *       (seed low 32 bits, seed high 32 bits) and counter (offset low,
 *       offset high, b, 0);  u = (x >> 8) * 2^-24 in [0, 1);
 *   token = the first v whose cumulative probability exceeds u.
 *
 * Call it after medusa_verify_accept on the same logits; it overwrites
 * bonus[b] and accepted_tokens[b][accept_len[b]].  Advance offset between
 * steps for fresh draws.  The cumulative sums are fp32 (chunked scan), so a u
 * within about 1e-6 of a boundary may select the neighbouring token of an
 * fp64 inverse CDF.
 * Inputs (device): logits [B, N, V] of dtype dt; accept_len [B] and
 *   accepted_nodes [B, max_depth+1] int32 from the verification.
 * Outputs (device): bonus [B], accepted_tokens [B, max_depth+1] (one entry).
 * Limits: temperature > 0.  Device checks: a kept node outside [0, N), a
 *   row with no probability mass (NaN logits).
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_sample_bonus(const void* logits, medusa_dtype_t dt,
                                               const int32_t* accept_len,
                                               const int32_t* accepted_nodes, int B, int N,
                                               int V, int max_depth, float temperature,
                                               uint64_t seed, uint64_t offset, int32_t* bonus,
                                               int32_t* accepted_tokens, int32_t* dev_status,
                                               void* stream);

/* ------------------------------------------------------------------------
 * medusa_tree_from_accuracies   (host only: no device memory, no launch)
 *
 * "Medusa Heads" glossary, "Attention arborescente et acceptation": a sparse
 * tree built from the most accurate combinations of the heads' top choices
 * beats a dense one.
 *
 * acc [n_heads * kmax] (host, row-major): acc[t-1][r] = probability that head
 * t's rank-r token is the base model's choice, in [0, 1].  A node with rank
 * path (r1..rt) is accepted with probability prod acc[i-1][r_i] (one rank at
 * most is right, heads independent); the tree holds the root and the
 * n_nodes - 1 paths of depth <= min(n_heads, max_depth) with the largest
 * products (equal products: lexicographically smaller path first), which
 * maximises the expected accept length (the sum of the products, returned in
 * *expected_accept_len when that pointer is not NULL).  Nodes are numbered by
 * depth, then lexicographic path: parent[0] = -1, parent[i] < i.
 * Outputs (host): parent, depth, rank [n_nodes] int32 - the arrays of a
 *   medusa_tree_t once copied to the device.
 * Errors: MEDUSA_ERR_SHAPE when fewer than n_nodes - 1 paths exist or a size
 *   is out of range; MEDUSA_ERR_INVALID_ARG for an accuracy outside [0, 1].
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_tree_from_accuracies(const float* acc, int n_heads, int kmax,
                                                       int n_nodes, int max_depth,
                                                       int32_t* parent, int32_t* depth,
                                                       int32_t* rank,
                                                       double* expected_accept_len);

/* ------------------------------------------------------------------------
 * Prompt side of the step: rotary positions, a paged key/value cache, the
 * attention of a chunk of new tokens over it, and tokens sampled from
 * filtered logits.
 *
 * No counterpart on the pages.  The decode step takes q and k "as already
 * positioned", a cache that holds the prompt, and a root token; these calls
 * produce them: a chunk of the prompt is rotated and written into the cache
 * (medusa_rope_append), attends to everything before it
 * (medusa_chunk_attention), and the logits of its last token give the first
 * root (medusa_sample_tokens).  medusa_rope positions the tree's q and k_new
 * at the pos_ids of medusa_tree_build.
 *
 * Row strides ("*_stride") count elements between consecutive tokens; the
 * heads and elements of one token are dense.  They let q, k and v be slices
 * of one packed projection.
 * ---------------------------------------------------------------------- */

typedef enum {
  MEDUSA_ROPE_NONE = 0,   /* f_i = theta^(-2i / rot)                              */
  MEDUSA_ROPE_LINEAR = 1, /* f_i / factor (positions divided by factor)           */
  MEDUSA_ROPE_LLAMA3 = 2, /* f_i divided by factor below low_turns turns over the */
                          /* original length, kept above high_turns, a linear     */
                          /* blend in the number of turns between                 */
  MEDUSA_ROPE_YARN = 3    /* the same two ends, blended linearly in the index i   */
                          /* between the indices of high_turns and low_turns      */
                          /* (rounded outwards); rotated elements gain the factor */
                          /* 0.1 ln(factor) + 1                                   */
} medusa_rope_scaling_t;

/*
 * A rotation.  The first rot elements of each head are rotated in rot / 2
 * pairs, the rest pass through: pair i is (i, i + rot/2), or (2i, 2i + 1)
 * when interleaved.  turns[i] (DEVICE array of rot/2) is the pair's frequency
 * in full turns per position, as a fraction of 2^64; the angle of position p
 * is the wrapping 64-bit product p * turns[i], so it keeps its precision at
 * any position (also negative ones).  Rotated elements are multiplied by
 * scale.
 */
typedef struct medusa_rope {
  int32_t rot;
  int32_t interleaved;
  float scale;
  const uint64_t* turns;
} medusa_rope_t;

/*
 * A paged cache.  Slot s of sequence b is row s % page_size of page
 * table[b * max_pages + s / page_size] (DEVICE array, int32); K and V are
 * pools [n_pages, Hkv, page_size, dh].  The dense cache [B, Hkv, cap, dh] of
 * the other calls is the pool with n_pages = B, page_size = cap, max_pages = 1
 * and table[b] = b.  Table entries past a sequence's last page are not read.
 */
typedef struct medusa_pages {
  void* K;
  void* V;
  const int32_t* table;
  int32_t n_pages;
  int32_t page_size;
  int32_t max_pages;
} medusa_pages_t;

/* medusa_rope_freqs (host only): the turns array (host, [rot/2]) and scale of
 * a medusa_rope_t.  f_i = theta^(-2i / rot) for i = 0..rot/2-1 in extended
 * precision, then the scaling; turns[i] = round(f_i / (2 pi) * 2^64).
 * low_turns, high_turns and original_max_position are read by LLAMA3 and YARN
 * only, factor by all but NONE.
 * Errors: MEDUSA_ERR_SHAPE for rot odd or outside [2, 512];
 *   MEDUSA_ERR_INVALID_ARG unless theta > 1, factor >= 1,
 *   0 < low_turns < high_turns and original_max_position > 0 (where read). */
MEDUSA_API medusa_status_t medusa_rope_freqs(int rot, double theta,
                                             medusa_rope_scaling_t scaling, double factor,
                                             double low_turns, double high_turns,
                                             double original_max_position, uint64_t* turns,
                                             float* scale);

/* ------------------------------------------------------------------------
 * medusa_rope
 *
 *   y0 = scale * (x0 cos a - x1 sin a),  y1 = scale * (x0 sin a + x1 cos a)
 *   for every pair (x0, x1) of the first rot elements of a head, with
 *   a = 2 pi * positions[t] * turns[i] / 2^64 (inverse = 0) or its negative
 *   (inverse = 1: the transpose, i.e. the gradient of the forward call).
 *
 * Inputs (device, dtype dt): q [T, Hq, dh] and k [T, Hkv, dh], tokens
 *   q_stride / k_stride elements apart (k NULL: q alone, Hkv ignored);
 *   positions [T] int32, any value.
 * Outputs (device, dtype dt): q_out, k_out, tokens q_out_stride /
 *   k_out_stride apart.  An output may be its input (in place, same stride);
 *   otherwise outputs overlap no input.
 * Precision: angles to 2^-28 turns, products in fp32, one rounding.
 * Limits: T >= 0 (nothing is launched for 0); rot <= dh <= 1024;
 *   Hq, Hkv >= 1; strides >= heads * dh.  No alignment beyond the type's own.
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_rope(const medusa_rope_t* rope, const void* q,
                                       long long q_stride, const void* k, long long k_stride,
                                       medusa_dtype_t dt, const int32_t* positions, int T, int Hq,
                                       int Hkv, int dh, int inverse, void* q_out,
                                       long long q_out_stride, void* k_out,
                                       long long k_out_stride, void* stream);

/* ------------------------------------------------------------------------
 * medusa_rope_append
 *
 * The new tokens of B sequences, rotated and written into the cache in one
 * launch.  Sequence b's rows are cu_q[b] .. cu_q[b+1]-1; its i-th row goes to
 * slot kv_len[b] - (cu_q[b+1] - cu_q[b]) + i, so kv_len counts the new tokens
 * already.  k is rotated by its position, v copied, q rotated into q_out.
 *
 * Inputs (device): q, k, v (dtype dt) as in medusa_rope; positions [T] int32,
 *   or NULL for the slots; cu_q [B + 1] int32, non-decreasing from 0;
 *   kv_len [B] int32.  rope NULL: no rotation, and q and q_out must be NULL.
 *   q may be NULL (then q_out too): only k and v.
 * In/out: the pools of pages (dtype dt).
 * T is the number of rows the caller holds; rows from cu_q[B] on (a padded
 *   batch) are left as they are, in q_out too.  A row whose slot is negative
 *   (kv_len shorter than the chunk) is rotated but not written.
 * Device checks: a slot past max_pages pages, a page outside [0, n_pages)
 *   (that row is not written); a row in front of cu_q[0] (left, in q_out too);
 *   cu_q decreasing, negative or above T (no row is written).
 * Limits: B >= 1, T >= 0, page_size, n_pages, max_pages >= 1; the rest as
 *   medusa_rope.
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_rope_append(
    const medusa_rope_t* rope, const void* q, long long q_stride, const void* k,
    long long k_stride, const void* v, long long v_stride, medusa_dtype_t dt,
    const int32_t* positions, const int32_t* cu_q, const int32_t* kv_len, int B, int T, int Hq,
    int Hkv, int dh, void* q_out, long long q_out_stride, const medusa_pages_t* pages,
    int32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------
 * medusa_chunk_attention
 *
 * The new tokens of B sequences attend to the cache, their own keys (already
 * written, e.g. by medusa_rope_append) included.  Row i of sequence b sits at
 * slot p = kv_len[b] - (cu_q[b+1] - cu_q[b]) + i and attends with weights
 * softmax(scale * q.k) to slots 0..p; with p < 0 it sees nothing and its
 * output is zero.  Query head hq reads kv head hq / (Hq / Hkv).  Chunks of
 * one token (decoding), of whole prompts and of anything between can be
 * mixed in a call; sequences may have no new token.
 *
 * Inputs (device): q [T, Hq, dh] of dtype dt, tokens q_stride elements apart;
 *   pages (dtype dt); cu_q [B + 1], kv_len [B] int32 as above.
 * Output (device): out [T, Hq, dh] of dtype dt, dense, apart from q; rows from
 *   cu_q[B] on are left as they are.
 * Workspace: medusa_chunk_attention_workspace_size(...) bytes, 256-byte
 *   aligned; the size depends on the current device's multiprocessor count
 *   and on none of the lengths.
 * Precision: bf16: scores and softmax statistics fp32, the softmax weights
 *   rounded to bf16 for the value product, which accumulates in fp32.
 *   MEDUSA_F32: fp32 throughout (CUDA cores).
 * Cache slots from kv_len[b] on are never used, whatever they hold; below it
 *   K and V must be finite.
 * Device checks: a page outside [0, n_pages), kv_len[b] outside
 *   [0, max_pages * page_size], cu_q decreasing, negative or above T, a
 *   non-finite output; bf16 also a call beyond its schedule: a sequence of
 *   more than 2^28 key tiles, or more than about 2^27 tiles a multiprocessor,
 *   counting a tile once for each group of up to 256 query rows and each kv
 *   head (a prompt of some six million tokens of 32 + 8 heads).  Where kv_len,
 *   cu_q or the schedule fails, no row is written.
 * Limits: B in [1, 1024], T >= 0, Hq % Hkv == 0, Hq / Hkv <= 128, Hkv <= 1024,
 *   scale > 0; pools 16-byte aligned; bf16: dh in {64, 128}, q_stride % 8 == 0,
 *   q and out 16-byte aligned; f32: dh % 32 == 0, dh <= 256.  Any page_size;
 *   in bf16, sizes of 128 or more and multiples of 8 fill the 128-key tiles
 *   best (any other size below 128 takes a tile a page).
 * ---------------------------------------------------------------------- */
MEDUSA_API size_t medusa_chunk_attention_workspace_size(int Hq, int Hkv, int dh,
                                                        medusa_dtype_t dt);
MEDUSA_API medusa_status_t medusa_chunk_attention(const void* q, long long q_stride,
                                                  const medusa_pages_t* pages, medusa_dtype_t dt,
                                                  const int32_t* cu_q, const int32_t* kv_len,
                                                  int B, int T, int Hq, int Hkv, int dh,
                                                  float scale, void* out, void* ws,
                                                  size_t ws_bytes, int32_t* dev_status,
                                                  void* stream);

/* ------------------------------------------------------------------------
 * medusa_sample_tokens
 *
 * One token per row of logits, drawn with the caller's random numbers after
 * the row's filters.  With the row's tokens in the order of descending logit
 * (equal logits: ascending id) and w_v = exp((z_v - max z) / temperature):
 *
 *   top_k  > 0: the first top_k tokens of the order stay (0 or less: all);
 *   top_p  < 1: of these, a token stays when the mass before it in the order
 *               is below top_p times their mass (the first always stays);
 *   min_p  > 0: a token stays when w_v >= min_p;
 *   token = the lowest id among the tokens that stay whose cumulative mass in
 *           id order exceeds u times their mass.
 *   temperature = 0: the first token of the order (kept = 1).
 *
 * Inputs (device): logits [n_rows, V] of dtype dt, rows row_stride elements
 *   apart; row_idx [R] int32, the logits row of each drawn token (NULL: row
 *   r), e.g. b * N + the kept node for a bonus token; u [R] fp32 in [0, 1);
 *   temperature, top_p, min_p [R] fp32 and top_k [R] int32, each NULL for 1,
 *   1, 0 and 0.
 * Outputs (device): tokens [R] int32; kept [R] int32, the number of tokens
 *   that stay (NULL to skip).
 * Logits of -inf are never drawn and stay out of kept.
 * Precision: weights are 64-bit fixed point in units of 2^-42 of the largest
 *   one, from fp64 exponents; sums are exact, so results do not depend on
 *   the order of summation.  A weight below 2^-43 of the largest counts as
 *   zero (it still counts in kept, and can be drawn when u = 0).
 * Limits: 1 <= V <= 327680 (fp32) or 655360 (bf16); R >= 0, R, n_rows <= 65535;
 *   row_stride >= V.
 * Device checks: a NaN or +inf logit, a row without a finite logit, u outside
 *   [0, 1), a NaN or negative parameter, temperature above 1e30, min_p above
 *   1, row_idx outside [0, n_rows); that row's token is -1 and kept 0.
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_sample_tokens(const void* logits, medusa_dtype_t dt,
                                                long long row_stride, int n_rows,
                                                const int32_t* row_idx, int R, int V,
                                                const float* u, const float* temperature,
                                                const int32_t* top_k, const float* top_p,
                                                const float* min_p, int32_t* tokens,
                                                int32_t* kept, int32_t* dev_status,
                                                void* stream);

/* ------------------------------------------------------------------------
 * medusa_wait_flag
 *
 * No counterpart on the pages: a check of this library's failure handling.
 * Every wait inside the library's kernels (on a shared-memory barrier, or on
 * a flag another block raises) is bounded: when it runs out it writes
 * MEDUSA_ERR_TIMEOUT into *dev_status and the kernel returns, instead of
 * holding the GPU.  This call runs that same bounded flag wait (the one the
 * heads' first GEMM uses for its stream-K partials) in one thread on a
 * caller's flag: it waits until *flag == value (acquire, device scope) or
 * until budget_cycles SM clock cycles have passed, and in the second case
 * writes MEDUSA_ERR_TIMEOUT into *dev_status.  The budget is checked every
 * 64 polls of about 64 ns, so the wait lasts at least a few microseconds.
 * budget_cycles <= 0 takes the library's own bound (2e9 cycles, one to two
 * seconds).  A flag that nothing sets thus shows, on a given device and
 * driver, that a stalled wait ends with a status the host can read and
 * leaves the context usable.
 * Inputs (device): flag, 4-byte aligned.  Output (device): dev_status.
 * Errors: MEDUSA_ERR_SHAPE for budget_cycles above the library's bound.
 * ---------------------------------------------------------------------- */
MEDUSA_API medusa_status_t medusa_wait_flag(const int32_t* flag, int32_t value,
                                            long long budget_cycles, int32_t* dev_status,
                                            void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MEDUSA_B200_H */
