/*
 * spec_verify.h -- C ABI of libspecverify.so, the verify-and-sample step of
 * speculative decoding on NVIDIA GB300 (sm_103a).
 *
 * The operation ("Beschleunigung von Sonar durch Spekulation", Perplexity,
 * section "Spekulatives Decoding", phases "Akzeptanz" and "Zielgenerierung";
 * section "Ziel-Entwurf"): after the target model has scored a draft of K
 * tokens, find the longest prefix of the draft the target accepts, and draw
 * one extra token from the target at the first mismatch or after the last
 * draft token, so that at most K + 1 tokens leave one step.  Acceptance
 * compares the full draft and target distributions; the rule used is that of
 * the method the page cites ("Fast Inference from Transformers via
 * Speculative Decoding"):
 *
 *   p_i = softmax(target_i / T), q_i = softmax(draft_i / T)      (over V)
 *   accept draft token x_i  iff  u_i < min(1, p_i(x_i) / q_i(x_i)), in order i = 0..K-1
 *   j = first rejected position, or K if none
 *   extra token ~ max(0, p_j - q_j) / W  if j < K,   ~ p_K  if j == K
 *   (inverse CDF: first v with cumulative weight C_v > u_b * W)
 *
 * With T == 0 (greedy): accept iff x_i == argmax target_i (lowest index on
 * ties) and the extra token is argmax target_j.  The tree variant ("Speculative-
 * Decoding / Medusa" blog, section 三 Attention Tree) follows, from the root,
 * the child whose token equals the target's argmax at the current node.
 *
 * Conventions shared by every entry point
 *   - Every pointer except `stream` is DEVICE memory owned by the caller; the
 *     library allocates nothing and keeps no pointer after the call returns
 *     (spec_cache and the strides of the calls on a cache are host memory, read
 *     during the call).
 *   - Logits are row-major with the vocabulary contiguous (row stride V
 *     elements), fp32 or bf16, aligned to their element size.
 *   - Calls are stream-ordered and asynchronous: they enqueue kernels on
 *     `stream` (a cudaStream_t; NULL means the legacy default stream) and
 *     return without synchronising.  Outputs are valid once the stream has
 *     reached that point.
 *   - Argument errors are found on the host before anything is enqueued and
 *     return a status (nothing is written).  A failed launch returns
 *     SPEC_ERR_CUDA.  Errors that depend on device data are OR-ed as
 *     SPEC_DEV_* bits into *dev_status (which the caller zeroes); kernels never
 *     trap and never abort.
 *   - All arithmetic on the device is fp32 (bf16 inputs are widened exactly);
 *     cumulative sums for the inverse CDF are exact int64 sums of the fp32
 *     weights of 16-byte groups of logits, in units of 2^-52.
 *   - Workspace: spec_verify_linear, spec_sample_bonus, spec_sample_rows,
 *     spec_verify_tree and spec_verify_tree_sample need a caller-owned device
 *     workspace of spec_workspace_bytes_*() bytes (the others need none), 16-byte aligned and zero-filled before
 *     its first use.  Every call leaves it zero-filled again -- also a call
 *     that reports SPEC_DEV_TIMEOUT: its last CTA then clears every byte the
 *     call used -- so one zeroing suffices for any number of calls, but one
 *     workspace must not be shared by calls that may run at the same time.
 *     spec_tree_attention's workspace need not be cleared; it too must not be
 *     shared by calls that may run at the same time, two captured graphs among them.
 *   - Residency: the verify kernel's warps wait (bounded) on values that
 *     warps of other CTAs publish, so it is launched cooperatively: all its
 *     CTAs (at most one per SM) are resident at once, or the launch fails and
 *     the call returns SPEC_ERR_CUDA.  A launch can fail that way when other
 *     work holds SMs (an MPS client limited to part of the GPU, a green
 *     context); it never deadlocks waiting for a CTA that cannot start.
 *   - Apart from a per-thread copy of the last error message, the library keeps
 *     only caches filled once per device and guarded by locks (a kernel's
 *     occupancy, in blocks or clusters, and shared-memory limit, the static workspace's address, the
 *     address of the driver's encoder of tensor maps); the functions may be called from several host threads.
 */
#ifndef SPEC_VERIFY_H
#define SPEC_VERIFY_H

#include <stddef.h>
#include <stdint.h>

/* Exported symbols: the library is built with hidden visibility, and only the
 * functions declared here are exported from it. */
#if defined(__GNUC__)
#define SPEC_API __attribute__((visibility("default")))
#else
#define SPEC_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum spec_status {
    SPEC_OK = 0,
    SPEC_ERR_INVALID_ARG = 1, /* a null, misaligned or out-of-range argument */
    SPEC_ERR_UNSUPPORTED = 2, /* valid, but beyond what this library handles (e.g. V too large) */
    SPEC_ERR_CUDA = 3,        /* the CUDA runtime reported an error; see spec_last_error() */
    SPEC_ERR_WORKSPACE = 4    /* workspace missing, too small or misaligned */
} spec_status;

typedef enum spec_dtype {
    SPEC_F32 = 0,  /* IEEE binary32 logits */
    SPEC_BF16 = 1, /* bfloat16 logits (upper half of an IEEE binary32) */
    SPEC_F16 = 2,  /* IEEE binary16: queries, keys and values alone */
    SPEC_E4M3 = 3  /* 8-bit floats (4 bits of exponent, 3 of mantissa), a cache's alone, with a power of two a row */
} spec_dtype;

/* Bits OR-ed into *dev_status by the kernels. */
#define SPEC_DEV_BAD_TOKEN     1u  /* a draft token outside [0, V): treated as rejected;
                                      spec_distill: a teacher's token outside [-1, V): left out;
                                      spec_adjust_logits: any token outside [-1, V): left out */
#define SPEC_DEV_NONFINITE     2u  /* a row whose max or exp-sum is not finite; outputs unspecified */
#define SPEC_DEV_TIMEOUT       4u  /* a bounded wait (a copy, or a value another warp publishes) gave up; outputs unspecified, workspace cleared */
#define SPEC_DEV_ZERO_RESIDUAL 8u  /* residual weight W == 0 at a rejection: drew from p_j instead */
#define SPEC_DEV_BAD_TREE     16u  /* parents[] not topological (0 <= parents[c] < c): edge ignored */
#define SPEC_DEV_BAD_LENGTH   32u  /* spec_sample_bonus: accept_len[b] outside [0, K] (token -1);
                                      spec_mtp_plug: num_emitted[b] outside [0, K+1];
                                      the cache's calls: a position behind the page table's end, or a length that
                                      its call excludes; spec_adjust_logits: a length outside the history */
#define SPEC_DEV_BAD_PARAM    64u  /* spec_sample_filtered: a row's parameter out of range (token -1);
                                      spec_adjust_logits: a penalty out of range (taken as none) */
#define SPEC_DEV_BAD_PAGE    128u  /* the cache's calls: a page table entry outside [0, pages) that a call needs */

/* Limits of the operators on rows of logits (spec_sample_filtered,
 * spec_top_logits, spec_distill, which keeps a row in a cluster's shared memory). */
#define SPEC_MAX_ROW_BYTES (1 << 20) /* V * element size: 262144 fp32 or 524288 bf16 logits */
#define SPEC_MAX_TOP       1024      /* K of spec_top_logits and spec_distill */

/* Bytes of workspace spec_verify_linear needs for B sequences of K draft
 * tokens over a vocabulary of V logits of `dtype` (0 for invalid sizes). */
SPEC_API size_t spec_workspace_bytes_linear(int B, int K, int V, spec_dtype dtype);

/* Bytes of workspace spec_sample_bonus needs for B sequences. */
SPEC_API size_t spec_workspace_bytes_bonus(int B, int V, spec_dtype dtype);

/* Bytes of workspace spec_sample_rows needs for B rows of V logits. */
SPEC_API size_t spec_workspace_bytes_rows(int B, int V, spec_dtype dtype);

/* Bytes of workspace spec_verify_tree needs for B sequences of N tree nodes. */
SPEC_API size_t spec_workspace_bytes_tree(int B, int N, int V, spec_dtype dtype);

/* Bytes of workspace spec_verify_tree_sample needs (one draw per node: grows
 * with B * N * V). */
SPEC_API size_t spec_workspace_bytes_tree_sample(int B, int N, int V, spec_dtype dtype);

/*
 * Linear verify and (optionally) the extra token, in one launch.
 *
 *   target_logits [B, K+1, V]  row i scores draft token i; row K is the tail.
 *   draft_logits  [B, K, V]    the draft's logits for the same positions; may be
 *                              NULL when temperature == 0 (greedy) or K == 0.
 *   dtype, B >= 0, K >= 0, V >= 1.
 *   draft_tokens  [B, K] int32 the drafted tokens x_i (may be NULL when K == 0).
 *   u_accept      [B, K] fp32  uniforms in [0, 1) for the acceptance tests;
 *                              ignored (may be NULL) when greedy or K == 0.
 *   u_bonus       [B]    fp32  uniform in [0, 1) for the extra token, or NULL to
 *                              emit no extra token (spec_sample_bonus can draw it
 *                              later); ignored when greedy except as the switch.
 *   temperature   T >= 0, finite; T == 0 selects greedy mode.
 * Outputs (device, caller-owned):
 *   accept_len    [B]      j = number of accepted draft tokens, 0 <= j <= K.
 *   out_tokens    [B, K+1] x_0..x_{j-1}, then the extra token (if u_bonus), then -1.
 *                          Required when u_bonus != NULL, else may be NULL.
 *   num_emitted   [B]      j + 1 with an extra token, j without.
 *   probs_out     [B, K, 3] or NULL: p_i(x_i), q_i(x_i), min(1, p_i/q_i) for every
 *                          position (computed for all K, not only up to j); sampling only.
 *   dev_status    [1]      SPEC_DEV_* bits OR-ed in.
 *   workspace, workspace_bytes: see the conventions above.
 */
SPEC_API spec_status spec_verify_linear(const void *target_logits, const void *draft_logits,
                               spec_dtype dtype, int B, int K, int V,
                               const int32_t *draft_tokens, const float *u_accept,
                               const float *u_bonus, float temperature,
                               int32_t *accept_len, int32_t *out_tokens, int32_t *num_emitted,
                               float *probs_out, uint32_t *dev_status,
                               void *workspace, size_t workspace_bytes, void *stream);

/*
 * The extra token alone, for callers that already hold accept_len: draws from
 * max(0, p_j - q_j) / W at j = accept_len[b] < K, or from p_K when j == K
 * (argmax of target row j when temperature == 0).  Same layouts as above.
 *   accept_len  [B] int32 (device, input); u_bonus [B] (ignored when greedy).
 *   bonus_token [B] int32 (device, output); -1 where accept_len[b] is out of
 *               range (and SPEC_DEV_BAD_LENGTH is set).
 *   workspace, workspace_bytes: spec_workspace_bytes_bonus(B, V, dtype) bytes.
 */
SPEC_API spec_status spec_sample_bonus(const void *target_logits, const void *draft_logits,
                              spec_dtype dtype, int B, int K, int V,
                              const int32_t *accept_len, const float *u_bonus, float temperature,
                              int32_t *bonus_token, uint32_t *dev_status,
                              void *workspace, size_t workspace_bytes, void *stream);

/*
 * One token per row: the draft side's choice of its next draft token (the
 * draft proposes tokens drawn from its own distribution q in the cited
 * speculative-sampling method), or any row a caller wants sampled.
 *   logits [B, V] (device, row-major, fp32 or bf16), u [B] fp32 in [0, 1)
 *   (ignored, may be NULL, when temperature == 0), temperature T >= 0.
 *   tokens [B] int32 (device, output): the first v whose cumulative weight of
 *   softmax(l / T) exceeds u[b] * W (exact int64 sums, as in the extra token),
 *   or the lowest-index argmax when T == 0.
 *   workspace, workspace_bytes: spec_workspace_bytes_rows(B, V, dtype) bytes.
 * It runs the extra-token path with no draft (K = 0).
 */
SPEC_API spec_status spec_sample_rows(const void *logits, spec_dtype dtype, int B, int V, const float *u, float temperature,
                             int32_t *tokens, uint32_t *dev_status, void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * Greedy verify of a candidate tree ("Speculative-Decoding / Medusa" blog,
 * section 三): at the current node take argmax of its target row; move to the
 * lowest-index child whose token equals it; stop when none does or max_depth
 * nodes were accepted; the extra token is argmax at the last accepted node.
 *
 *   target_logits [B, N, V]  row n holds the target logits after node n;
 *                            node 0 is the root (the last accepted token).
 *   parents       [N] int32  parents[0] ignored; 0 <= parents[c] < c for c >= 1.
 *   node_tokens   [B, N]     candidate token of each node (column 0 ignored).
 *   max_depth >= 0, N >= 1, V >= 1.
 * Outputs (max_depth + 1 columns, -1 padded):
 *   path_nodes [B, max_depth+1]  0, n_1, n_2, ... (node ids of the accepted path)
 *   path_len   [B]               number of accepted non-root nodes
 *   out_tokens [B, max_depth+1]  tokens of n_1..n_len, then the extra token
 */
SPEC_API spec_status spec_verify_tree(const void *target_logits, spec_dtype dtype, int B, int N, int V,
                             const int32_t *parents, const int32_t *node_tokens, int max_depth,
                             int32_t *path_nodes, int32_t *path_len, int32_t *out_tokens,
                             uint32_t *dev_status, void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * Tree verify in sampling mode ("Speculative-Decoding / Medusa" blog, section
 * 三: the target's choice at a node may be greedy or sampled).  At every node n
 * the target's choice is a draw from softmax(target_n / T) by inverse CDF with
 * the caller's uniform u_nodes[b, n] (the first v whose cumulative weight
 * exceeds u * W, over exact int64 sums as in the linear draw).  The walk is that
 * of spec_verify_tree with the draw in place of the argmax: from the root, move
 * to the lowest-index child whose token equals the draw at the current node;
 * stop when none does or max_depth nodes were accepted.  The extra token is
 * the draw at the last accepted node.  Every node is drawn, visited or not
 * (a data-parallel pass: two reads of every row, the second mostly from L2).
 *
 *   target_logits [B, N, V], parents [N], node_tokens [B, N]: as spec_verify_tree.
 *   u_nodes       [B, N] fp32 in [0, 1): one uniform per node (device).
 *   temperature   T > 0, finite.
 *   max_depth, path_nodes, path_len, out_tokens, dev_status: as spec_verify_tree.
 *   workspace, workspace_bytes: spec_workspace_bytes_tree_sample(B, N, V, dtype).
 */
SPEC_API spec_status spec_verify_tree_sample(const void *target_logits, spec_dtype dtype, int B, int N, int V,
                                    const int32_t *parents, const int32_t *node_tokens, const float *u_nodes,
                                    float temperature, int max_depth, int32_t *path_nodes, int32_t *path_len,
                                    int32_t *out_tokens, uint32_t *dev_status, void *workspace,
                                    size_t workspace_bytes, void *stream);

/*
 * The tree attention mask of a candidate tree ("Speculative-Decoding / Medusa"
 * blog, section 三: the tree is flattened into one sequence and a mask modelled
 * on the causal mask keeps tokens of different paths apart).  Row i holds node
 * i and every ancestor of node i; depth[i] is the number of edges from the
 * root (the token's position offset).
 *   parents    [N] int32 (device): parents[0] ignored, 0 <= parents[c] < c.
 *   mask_words [N, ceil(N/32)] uint32 (device, output): bit (j % 32) of word
 *              j / 32 of row i is set iff node j is node i or its ancestor.
 *   depth      [N] int32 (device, output).
 *   dev_status [1]: SPEC_DEV_BAD_TREE when a parent breaks the rule; that
 *              node's row and depth then hold the path up to the bad edge.
 * 1 <= N <= 16384.  No workspace; one small launch.
 */
SPEC_API spec_status spec_tree_mask(const int32_t *parents, int N, uint32_t *mask_words, int32_t *depth, uint32_t *dev_status,
                           void *stream);

/*
 * Sparse candidate tree ("Speculative-Decoding / Medusa" blog, section 四,
 * optimized tree construction).  With a_k^(i) the accuracy of head k's i-th
 * ranked token (taken as independent), the node reached by the rank path
 * [i_1 .. i_m] is accepted with probability prod_j a_j^(i_j), and E[L] is the
 * sum of that product over the tree's non-root nodes.  The tree grows from
 * the root one node at a time by the candidate (a child of a node already in
 * the tree) of largest product, until it holds n_nodes nodes or no candidate
 * is left.  Equal products go to the smaller depth, then to the
 * lexicographically smaller rank path.  Nodes are numbered by (depth, rank
 * path), so 0 <= parents[c] < c and the result feeds spec_tree_mask and
 * spec_verify_tree / spec_verify_tree_sample as it is.
 *
 * Unlike every other entry point this one runs on the HOST (all pointers are
 * host memory, no stream): the tree has a few dozen nodes and is built once
 * per accuracy table, not per decode step.
 *   accuracy     [K * S] double: accuracy[(k-1) * S + (i-1)] = a_k^(i), in [0, 1].
 *   K            heads (the tree's depth limit), 1 <= K <= 64.
 *   S            ranked tokens per head, 1 <= S <= 4096.
 *   n_nodes      nodes wanted, the root included, 1 <= n_nodes <= 16384.
 * Outputs (n_nodes entries each; the first *n_built are written):
 *   parents      parents[0] = -1, else the parent's number.
 *   depth        the node's depth (0 for the root).
 *   rank         the rank i of the node's token among its head's candidates
 *                (1-based; 0 for the root).
 *   n_built      min(n_nodes, the full tree's size).
 *   expected_len E[L] of the tree, or NULL.
 * Errors: SPEC_ERR_INVALID_ARG for sizes out of range, a null pointer, or an
 * accuracy that is not a finite value in [0, 1].
 */
SPEC_API spec_status spec_build_sparse_tree(const double *accuracy, int K, int S, int n_nodes, int32_t *parents,
                                            int32_t *depth, int32_t *rank, int *n_built, double *expected_len);

/*
 * MTP token plug-in ("Beschleunigung von Sonar durch Spekulation", sections
 * "MTP" and "MTP-Zeitplan für ein einzelnes Token"): the draft layer at
 * position i reads the target's hidden state H_i with the token that follows
 * position i, so its input is the target's input shifted left by one; after
 * verification the target's next tokens go into their places on the device,
 * and the sequence lengths advance, with no host round trip.
 *
 *   in_tokens   [B, K+1] int32  the target's input tokens of the step: row b is
 *                               (the token the step started from, x_0 .. x_{K-1});
 *                               for single-token MTP (K = 1) these are the 2 * B
 *                               tokens the target scored.
 *   out_tokens  [B, K+1] int32  spec_verify_linear's out_tokens (accepted draft
 *                               tokens, then the extra token).
 *   num_emitted [B] int32       spec_verify_linear's num_emitted.
 *   pad                         the token written at position K when nothing is
 *                               shifted into it (only when fewer than K + 1 tokens
 *                               were emitted).
 * Outputs (device, caller-owned):
 *   next_tokens [B, K+1] int32  next[b, i] = out_tokens[b, i] for i < n_b, else
 *                               in_tokens[b, i + 1] for i < K, else pad; it may be
 *                               in_tokens itself (in place), but not out_tokens.
 *   seq_lens    [B] int32       incremented by num_emitted[b] in place; NULL to skip.
 *   dev_status  [1]             SPEC_DEV_BAD_LENGTH when num_emitted[b] is outside
 *                               [0, K+1] (that row is only shifted, its length unchanged).
 * B >= 0, K >= 0, every pointer 4-byte aligned.  No workspace; one small launch
 * (one warp per sequence), ordered after the verify on the same stream.
 */
SPEC_API spec_status spec_mtp_plug(const int32_t *in_tokens, int B, int K, const int32_t *out_tokens,
                                   const int32_t *num_emitted, int32_t pad, int32_t *next_tokens,
                                   int32_t *seq_lens, uint32_t *dev_status, void *stream);

/*
 * One token per row under the usual serving filters, each row with parameters
 * of its own (a batch mixes requests): spec_sample_rows with temperature,
 * top-k, top-p and min-p.  With w_v = exp((l_v - max l) / T) and the tokens in
 * the order of falling logits (the lower index first among equal ones), the
 * kept tokens are, one filter after the other:
 *   top-k   the first k;
 *   top-p   of those, the shortest prefix whose weight is at least p times
 *           theirs (at least one token);
 *   min-p   of those, the ones with w_v >= min_p.
 * Each leaves a prefix of the order.  The token is the first v, in index order,
 * whose running sum of kept weights exceeds u * (their sum).
 * Not for draft tokens that spec_verify_linear is to test, where a filter limits
 * or rows differ in T: it takes q for the whole draft row's softmax at one T, and
 * what it emits follows the target only if the draft was drawn from that
 * (spec_sample_rows, or this call without filters at that T).
 *
 *   logits      [B, V]  fp32 or bf16; -inf masks a token (it is never kept).
 *   temperature [B] fp32: 0 (the lowest-index argmax; the row's other
 *               parameters are not used) or in [1e-6, 1e6].
 *   top_k       [B] int32 or NULL; <= 0 or >= V: no limit.
 *   top_p       [B] fp32 or NULL, in [0, 1]; 1: no limit.
 *   min_p       [B] fp32 or NULL, in [0, 1]; 0: no limit.
 *   u           [B] fp32 in [0, 1).
 *   tokens      [B] int32 (output).
 *   dev_status  SPEC_DEV_BAD_PARAM: a row's parameter is out of range or NaN;
 *               SPEC_DEV_NONFINITE: a row holds NaN or +inf, or every token of
 *               it is masked.  Such a row's token is -1; the others are drawn.
 * Weights are whole numbers in units of 2^-U, U = min(48, 62 - ceil(log2 V))
 * (43 for the longest rows, 47 for 32000 logits), each right to 2^-37 of itself
 * and 0.8 units; their sums are exact.  So with W the sum over the N tokens that
 * a filter or the draw looks at, the token is the definition's unless u W, or
 * top-p's share, lies within 2^-37 W + 0.8 N 2^-U of a border; a tail of many
 * tokens below half a unit weighs nothing.  Which tokens min-p keeps is right to 2^-36 of
 * min-p, whatever its size.  At u = 0 a weight counts that is not 0 in 64 bits
 * (2^-1075 and above), units or not.  A call gives the same token every time.
 * Rows of at most SPEC_MAX_ROW_BYTES bytes (SPEC_ERR_UNSUPPORTED above).
 * No workspace; one launch.
 */
SPEC_API spec_status spec_sample_filtered(const void *logits, spec_dtype dtype, int B, int V, const float *temperature,
                                          const int32_t *top_k, const float *top_p, const float *min_p,
                                          const float *u, int32_t *tokens, uint32_t *dev_status, void *stream);

/*
 * The K largest logits of each row, in falling order (the lower index first
 * among equal ones), and optionally the row's log-normaliser: the candidate
 * tokens of a draft head (spec_build_sparse_tree's rank i is entry i - 1), or
 * the target's distribution as spec_distill takes it.
 *   logits [B, V] fp32 or bf16; -inf masks a token.
 *   1 <= K <= SPEC_MAX_TOP; K may exceed V.
 *   temperature in [1e-6, 1e6]: the log-normaliser's, not the values'.
 *   values [B, K] fp32, ids [B, K] int32: entries past the row's last unmasked
 *          token are (-inf, -1).
 *   lse    [B] fp32 or NULL: log sum_v exp(l_v / T); -inf for a masked row.
 *   dev_status  SPEC_DEV_NONFINITE: a row holds NaN or +inf; its values and lse
 *          are NaN and its ids -1.
 * Rows of at most SPEC_MAX_ROW_BYTES bytes.  No workspace; one launch.
 */
SPEC_API spec_status spec_top_logits(const void *logits, spec_dtype dtype, int B, int V, int K, float temperature,
                                     float *values, int32_t *ids, float *lse, uint32_t *dev_status, void *stream);

/*
 * Distillation from a teacher's largest logits: how far the student's (the
 * draft's) distribution is from the teacher's (the target's), whose agreement
 * decides how many draft tokens a verify accepts.  Row by row, with
 * q = softmax(s / T) and the teacher's K entries (t_k, id_k) as
 * spec_top_logits gives them:
 *   p_k  = exp(t_k / T - lse)           with top_lse (taken at the same T), or
 *          softmax of t / T over the entries without it;  P = sum_k p_k
 *   loss = w * sum_k p_k (log p_k - log q[id_k])
 *   d loss / d s_v = (w / T) * (P q_v - sum of p_k over the entries with id_k = v)
 * The teacher is a constant: it gets no gradient.
 * The mass that top_lse leaves outside the K entries, 1 - P, enters neither loss
 * nor gradient: with it the gradient is P times the one without it (the least
 * loss is at q = p / P on the entries, 0 elsewhere, either way), so it weighs
 * each row by how much of the teacher its entries hold.  The loss is then a
 * divergence only at P = 1; below it may be negative.
 *
 *   student_logits [N, V] fp32 or bf16; -inf masks a token (a masked token that
 *                  the teacher gives weight makes the loss +inf).
 *   top_ids    [N, K] int32, 1 <= K <= SPEC_MAX_TOP, in any order: -1 is an empty
 *              slot (its logit is not used); a token named twice counts twice.
 *   top_logits [N, K] fp32; -inf has no weight.
 *   top_lse    [N] fp32 or NULL.
 *   temperature T in [1e-6, 1e6].
 *   row_weight [N] fp32 or NULL (1): a row of weight 0 is ignored: its logits and
 *              its teacher are not read, its loss, statistics and gradient are 0.
 * Outputs:
 *   loss  [N] fp32;  stats [N, 2] fp32 (8-byte aligned): the row's largest logit and
 *         sum_v exp((s_v - largest) / T), for spec_distill_backward.
 *   grad  [N, V] of the logits' type, or NULL: the gradient of the sum of the
 *         losses, overwritten; it may be student_logits itself (in place), and
 *         must not overlap it otherwise (SPEC_ERR_INVALID_ARG).
 *         With it the logits are read once for both.
 *   dev_status  SPEC_DEV_BAD_TOKEN; SPEC_DEV_NONFINITE: a row of weight other
 *         than 0 with NaN or +inf among its logits or its teacher's, or nothing
 *         but -inf: its loss, statistics and gradient are NaN.
 * A row without a teacher's token (P = 0) has loss and gradient 0.
 * Rows of at most SPEC_MAX_ROW_BYTES bytes.  No workspace; one launch; the same
 * result every time.
 */
SPEC_API spec_status spec_distill(const void *student_logits, spec_dtype dtype, int N, int V, const int32_t *top_ids,
                                  const float *top_logits, int K, const float *top_lse, float temperature,
                                  const float *row_weight, float *loss, float *stats, void *grad, uint32_t *dev_status,
                                  void *stream);

/*
 * The gradient alone, for losses whose upstream gradients are known only later:
 * grad[n, v] = grad_loss[n] * d loss[n] / d s_v, from spec_distill's stats of the
 * same logits, teacher, temperature and weights.  Arguments as there; stats and
 * grad_loss [N] fp32 are inputs.  A row whose row_weight or grad_loss is 0 (or
 * their product) is not read and its gradient is 0, whatever the other is.
 * grad may be student_logits itself.
 */
SPEC_API spec_status spec_distill_backward(const void *student_logits, spec_dtype dtype, int N, int V, const int32_t *top_ids,
                                           const float *top_logits, int K, const float *top_lse, float temperature,
                                           const float *row_weight, const float *stats, const float *grad_loss, void *grad,
                                           uint32_t *dev_status, void *stream);

/*
 * Penalties for repeated tokens, biases and grammar masks on the logits that a
 * verify or a draw then takes.  Row n of sequence b scores what follows node n
 * of the draft, so it counts the sequence's history and the drafted tokens on
 * node n's own path, which differ from row to row:
 *   x = logits[b, n, t] in fp32, then in this order, each step rounded to fp32:
 *   bias        x += the sum of the bias values whose id is t (in slot order)
 *   repetition  if t is in the history or on the path: x = x > 0 ? x / r : x * r
 *   frequency   x -= f * c,  c = how often t is among the generated tokens and on the path
 *   presence    x -= p  if c > 0
 *   mask        x = -inf  if t's bit in allowed is 0 (whatever x is, NaN too)
 * and out[b, n, t] = x in the logits' type.
 *   logits [B, N, V] fp32 or bf16: a verify's target rows.  A linear draft of K
 *          tokens has N = K + 1 and mask NULL; rows without a draft have N = 1.
 *   tokens [B, L] int32: the history, prompt first; -1 is no token.  NULL with L = 0: none.
 *   prompt_len, total_len [B] int32: tokens[b, 0 .. prompt_len) are the prompt's, up to
 *          total_len the generated ones, the token that the step started from (the
 *          root) among them.  NULL: 0, and L.
 *   node_tokens [B, N] int32: column 0 (the root) is ignored, -1 is no token; row b of
 *          spec_mtp_plug's in_tokens has this form.  NULL: no drafted tokens.
 *   mask   [N, ceil(N/32)]: node n's path as spec_tree_mask gives it (bit 0 is
 *          ignored); NULL: a chain, nodes 1 .. n.
 *   repetition r > 0, frequency f, presence p: [B] fp32, finite, or NULL (1, 0, 0).
 *          A sequence with r = 1 and f = p = 0 has its history left unread.
 *   bias_ids, bias [B, M]: int32 (-1: an empty slot), fp32.  NULL with M = 0: none.
 *   allowed [B, N, ceil(V/32)] uint32: bit (t % 32) of word t / 32 of a row; NULL: all.
 *   out    [B, N, V]: it may be logits itself (then only what changes is written), and
 *          must not overlap it otherwise (SPEC_ERR_INVALID_ARG).
 *   dev_status  SPEC_DEV_BAD_TOKEN, SPEC_DEV_BAD_LENGTH (taken as the nearest length
 *          in [0, L], the prompt's at most total_len), SPEC_DEV_BAD_PARAM.
 * 1 <= N <= SPEC_MAX_NODES, 0 <= M <= SPEC_MAX_BIASES, 0 <= L < 2^24.  No workspace; one
 * launch; the same result every time.  For inference: there is no call for its gradient.
 */
SPEC_API spec_status spec_adjust_logits(const void *logits, spec_dtype dtype, int B, int N, int V, const int32_t *tokens, int L,
                                        const int32_t *prompt_len, const int32_t *total_len, const int32_t *node_tokens,
                                        const uint32_t *mask, const float *repetition, const float *frequency,
                                        const float *presence, const int32_t *bias_ids, const float *bias, int M,
                                        const uint32_t *allowed, void *out, uint32_t *dev_status, void *stream);
#define SPEC_MAX_NODES  1024 /* N of spec_adjust_logits and spec_tree_attention */
#define SPEC_MAX_BIASES 1024 /* M of spec_adjust_logits */

/*
 * A paged cache of keys and values, as the three calls below take it (a HOST
 * struct, read during the call; its pointers are device memory).  A token at
 * position i of sequence b lies in page page_table[b, i / page_size], in slot
 * i % page_size of every head.  In 8 bits each (token, head) row of D values x has
 * one power of two 2^e, kept as the byte e + 127: with e the least whole number
 * such that max |x| <= 448 * 2^e, -110 <= e <= 120 (in fp16 also e >= -24), the values
 * are x / 2^e rounded to e4m3, to nearest even (at the type's end, e = 120 and
 * in fp16 e = 8, at most 240, since 256 * 2^e would be read back as an infinity).  A row with an infinity or a NaN has byte 255 and reads as NaN.
 * Powers of two lose nothing in a floating format and make what is read back exact.
 */
typedef struct spec_cache {
    void *k, *v;               /* [pages, kv_heads, page_size, head_dim], 16-byte aligned */
    uint8_t *k_scale, *v_scale; /* [pages, kv_heads, page_size] with SPEC_E4M3, else NULL */
    const int32_t *page_table; /* [B, table_width] */
    spec_dtype dtype;          /* SPEC_E4M3, or the type of the keys and values themselves */
    int pages, page_size;      /* page_size 16, 32, 64, 128 or 256 */
    int kv_heads, head_dim;    /* head_dim 64 or 128 */
    int table_width;
} spec_cache;

/*
 * Writes keys and values of a batch into the cache: what a prompt, a step, or the
 * accepted path of a verified draft adds to each sequence's context.
 *   k, v     [B, N, kv_heads, head_dim] of `dtype` (SPEC_BF16 or SPEC_F16); strides (host, 4
 *            entries: k's batch and token strides in elements, then v's; multiples of 8, an axis of one
 *            entry's does not matter) or NULL for contiguous; 16-byte aligned.
 *   select   [B, S] int32: row i of sequence b is token select[b, i] (spec_verify_tree's
 *            path_nodes with S = max_depth + 1); a negative entry writes nothing, and one that start or count
 *            leaves out is not looked at.  NULL: S = N, row i is token i.
 *   start    [B] int32: row i goes to position start[b] + i; a sequence with a negative start is left out.
 *   count    [B] int32: only rows i < count[b] (above S: S, below 0: none); NULL: all S.
 *            spec_verify_linear's num_emitted, when u_bonus was given, counts the accepted rows (the root's among them).
 * No length is advanced: the layers of a model call this with the same start.
 * Two rows that name one slot leave it unspecified, unless they are the same row (in 8 bits it may hold one's values and the
 * other's power of two): a page that sequences share is not appended to.  k and v must not overlap the cache.  dev_status: SPEC_DEV_BAD_LENGTH (a
 * position behind the table, or an entry of select not below N), SPEC_DEV_BAD_PAGE; such a row
 * is not written.  B * S <= INT_MAX / 64; positions below 2^30; kv_heads <= 1024.  No workspace; one launch.
 */
SPEC_API spec_status spec_cache_append(const void *k, const void *v, spec_dtype dtype, int B, int N, const long long *strides,
                                       const int32_t *select, int S, const int32_t *start, const int32_t *count,
                                       const spec_cache *cache, uint32_t *dev_status, void *stream);

/*
 * Reads positions start[b] .. start[b] + count[b] - 1 of every sequence back:
 *   k, v [B, S, kv_heads, head_dim] of `dtype` (output, contiguous, 16-byte aligned): row i is
 *        position start[b] + i; rows from count[b] on are left as they were.  With SPEC_E4M3
 *        each value is q * 2^e, rounded to `dtype` (exactly, but for fp16 below 2^-14, and past fp16's
 *        range where the cache was written from bf16: an infinity).
 *   start, count, dev_status as in spec_cache_append (such a row is left as it was).
 */
SPEC_API spec_status spec_cache_read(const spec_cache *cache, int B, int S, const int32_t *start, const int32_t *count, void *k,
                                     void *v, spec_dtype dtype, uint32_t *dev_status, void *stream);

/*
 * Attention of drafted tokens: the N nodes of each sequence's draft (N = 1: plain
 * decoding) attend to the sequence's cached context and to the nodes on their own
 * path ("Speculative-Decoding / Medusa" blog, section 三: the tree is verified in
 * one target pass under a mask that keeps its paths apart), for query head h of key head
 * g = h / (heads / kv_heads):
 *   s_j = scale * q[b, n, h] . k_j,   out[b, n, h] = sum_j exp(s_j) v_j / sum_j exp(s_j)
 * over the positions j < context_lens[b] of the cache and the nodes m with bit m set in mask
 * row n.  A row that sees nothing gives 0, and lse -inf.  A key or value that a row does not
 * see has no part in it, whatever it holds.
 *   q [B, N, heads, head_dim], k, v [B, N, kv_heads, head_dim] of `dtype` (SPEC_BF16 or
 *          SPEC_F16): the nodes' own, not in the cache yet (spec_cache_append adds the accepted
 *          ones); strides (host, 6 entries: q's batch and token strides in elements, k's, v's;
 *          multiples of 8, above 0 and below 2^38, an axis of one entry's does not matter) or NULL for contiguous;
 *          16-byte aligned.  With shared_len q's batch stride is N times its token stride, or B or N is 1
 *          (else SPEC_ERR_UNSUPPORTED).
 *   cache  of `dtype` or SPEC_E4M3.  Positions may differ in their key heads' scales.
 *   context_lens [B] int32; a sequence with a negative length is left out, its rows of out
 *          and lse as they were.
 *   shared_len  the first shared_len positions hold the same keys and values in every
 *          sequence (a common prompt): they are read through sequence 0's page table, once for
 *          the whole batch, also where sequence 0 is left out.  0: nothing is shared.  Every context_lens[b] >= 0 is then at least
 *          shared_len (SPEC_DEV_BAD_LENGTH where it is not, and that sequence's rows are unspecified).
 *   mask   [N, ceil(N/32)] as spec_tree_mask gives it; NULL: a chain, nodes 0 .. n.
 *   scale  finite, > 0.
 *   out    [B, N, heads, head_dim] of `dtype`, contiguous, 16-byte aligned; overlaps nothing that is read
 *          (SPEC_ERR_INVALID_ARG for q, k and v).
 *   lse    [B, N, heads] fp32 or NULL: log sum_j exp(s_j).
 *   dev_status  SPEC_DEV_BAD_LENGTH, SPEC_DEV_BAD_PAGE: that sequence's rows are unspecified (a bad page
 *          of the shared positions: all rows); SPEC_DEV_TIMEOUT.
 *   workspace  spec_workspace_bytes_attention() bytes (43 MB with head_dim 128, 22 MB with 64, and with shared_len 8 bytes more
 *          for each value of out), 16-byte aligned; its content before a call does not matter.
 * Scores, sums and the weighted sums are fp32; exp(s_j - m), the weight of v_j in the matrix
 * product, is rounded to `dtype` (off by up to 2^-8 of itself in bf16, 2^-11 in fp16, errors that the sum averages).
 * For inference: there is no call for its gradient.
 * 1 <= N <= SPEC_MAX_NODES; heads a multiple of kv_heads, at most 128 times it.  Positions below 2^30, and at most
 * INT_MAX tiles of 128 keys (by the table's width).  Two launches.  The same result every time.
 */
SPEC_API size_t spec_workspace_bytes_attention(int B, int N, int heads, int kv_heads, int head_dim, int shared_len);
SPEC_API spec_status spec_tree_attention(const void *q, const void *k, const void *v, spec_dtype dtype, int B, int N, int heads,
                                         const long long *strides, const spec_cache *cache, const int32_t *context_lens,
                                         int shared_len, const uint32_t *mask, float scale, void *out, float *lse,
                                         uint32_t *dev_status, void *workspace, size_t workspace_bytes, void *stream);

/*
 * spec_verify_linear with the library's own workspace.  The pages describe no
 * such call: it exists for callers that cannot allocate device memory at the
 * point where they verify -- e.g. a host program embedded in an inference
 * engine whose memory pool already owns the device, or a decode loop that must
 * not call cudaMalloc / cudaFree between steps because cudaFree synchronises
 * the whole device.  It allocates nothing (no cudaMalloc, no cudaFree, no
 * allocating library routine).
 *
 * The workspace is one statically sized array per device, compiled into the
 * library: SPEC_STATIC_WORKSPACE_BYTES bytes.  Shapes whose
 * spec_workspace_bytes_linear(B, K, V, dtype) exceeds that are rejected with
 * SPEC_ERR_WORKSPACE (spec_last_error() gives both sizes); use
 * spec_verify_linear with a workspace of your own for those.
 *
 * First call on each device: it looks up the array's device address
 * (cudaGetSymbolAddress, with that device current; this may also load the
 * library's kernels onto the device) and keeps it for the life of the
 * process.  Make one call on every device you will use before you begin any
 * stream capture on it.  Resetting a device (cudaDeviceReset) after that
 * first call is not supported: the kept address would name memory of the
 * destroyed context.
 *
 * Every call clears the part of the array it uses with cudaMemsetAsync on
 * `stream` before its kernel, so no earlier call's leftovers matter.  There is
 * ONE array per device and process: calls that may overlap in time (different
 * streams, or host threads without ordering) race on it and give wrong
 * results.  Issue them on one stream, or use spec_verify_linear.
 *
 * Arguments, outputs and errors are those of spec_verify_linear, without
 * `workspace` and `workspace_bytes`.
 */
#define SPEC_STATIC_WORKSPACE_BYTES (16u << 20)

SPEC_API spec_status spec_verify_linear_static(const void *target_logits, const void *draft_logits,
                                      spec_dtype dtype, int B, int K, int V,
                                      const int32_t *draft_tokens, const float *u_accept,
                                      const float *u_bonus, float temperature,
                                      int32_t *accept_len, int32_t *out_tokens, int32_t *num_emitted,
                                      float *probs_out, uint32_t *dev_status, void *stream);

/* Static text for a status code. */
SPEC_API const char *spec_status_string(spec_status status);

/* Detail of the last error returned on the calling host thread ("" if none). */
SPEC_API const char *spec_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H */
