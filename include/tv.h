/*
 * tv.h -- C ABI of the tree-speculative-verification library for gated-DeltaNet hybrids.
 *
 * One verify round of a hybrid model (qwen35-tree-spec post, §七 完整验证流程) runs a draft
 * tree, given by a parents[] array, through two kinds of layers:
 *
 *   - gated-DeltaNet (GDN) layers, where every node i gets its own recurrent state
 *         S_i = alpha_i * S_p @ (I - beta_i k_i k_i^T) + beta_i v_i k_i^T,   o_i = S_i q_i
 *     evolved from its parent p (the committed state S_0 for a root), either by
 *     depth-by-depth fork/checkpoint (same post, §四) or by the TreeWY form, which keeps a
 *     small pseudo-value matrix instead of per-node states (TreeWY: Speculative Verification
 *     for Gated DeltaNet Hybrids, abstract);
 *   - full-attention layers, where every node attends to the committed KV prefix plus its
 *     ancestors plus itself at RoPE position prefix_len + depth (handbook chapter
 *     投机解码进阶：树形草稿与 EAGLE, §实现, forward_with_mask and tree_mask);
 *
 * then commits the accepted path: the GDN state goes back to the last accepted node's state
 * (qwen35-tree-spec §五 用途 2) and the accepted nodes' KV moves to the contiguous slots after
 * the prefix, or whole blocks of it are taken over through the block table (handbook chapter,
 * note after the listing: the KV is reused, not recomputed).
 *
 * Conventions for every call below
 * --------------------------------
 *  - Pointers are DEVICE pointers owned by the caller, unless a comment says otherwise; the
 *    library allocates no memory.  Every tensor is dense, row-major (last index fastest) with
 *    the shape written beside it, and its base address is 16-byte aligned.
 *  - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy default stream).
 *    The return value reports only what the host can see before launch: TV_OK, or
 *    TV_ERR_INVALID_ARG (null/misaligned pointer, non-positive or inconsistent size),
 *    TV_ERR_UNSUPPORTED (a size or dtype outside the supported set) or TV_ERR_CUDA (a launch
 *    failed; tv_last_cuda_error() then holds the CUDA error code).  Nothing is launched when
 *    the return value is not TV_OK.
 *  - Data-dependent errors (a malformed tree, a bad accepted path, a block table that is too
 *    short or points outside the cache) are written per sequence to the device array
 *    err[B] (0 = that sequence is fine, else a TV_ERR_* code).  A failed sequence's outputs
 *    are left unwritten; the other sequences are unaffected.  No kernel traps or waits
 *    without bound.  Read err after synchronising the stream.
 *  - parents[b][i] is -1 (node i follows the committed state directly: a root) or an
 *    earlier node index (-1 <= parents[i] < i); anything else is TV_ERR_BAD_TREE.
 *  - Sizes: 1 <= N <= TV_MAX_NODES nodes per tree, every sequence of a call has N nodes.
 *  - dtype codes: TV_F32 (fp32) or TV_BF16 (bf16, round-to-nearest-even on store).
 *    Arithmetic is fp32 throughout.
 */
#ifndef TV_H_
#define TV_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(__GNUC__)
#define TV_API __attribute__((visibility("default")))
#else
#define TV_API
#endif

struct CUstream_st;
typedef struct CUstream_st* tv_stream_t; /* same type as cudaStream_t */

enum tv_status {
  TV_OK = 0,
  TV_ERR_INVALID_ARG = -1,
  TV_ERR_BAD_TREE = -2,
  TV_ERR_BAD_PATH = -3,
  TV_ERR_UNSUPPORTED = -4,
  TV_ERR_CUDA = -5,
  TV_ERR_TIMEOUT = -6,
  TV_ERR_CAPACITY = -7,     /* block table too short for prefix_len + N slots */
  TV_ERR_BAD_BLOCK = -8,    /* a block-table entry outside [0, num_blocks), or (compaction)
                               two logical blocks of the tree's window on one physical block */
  TV_ERR_SCRATCH = -9,      /* tv_tree_attn_static: the call needs more than
                               TV_STATIC_SCRATCH_BYTES of scratch */
  TV_ERR_BAD_SEQLEN = -10,  /* packed prompts: cu_seqlens decreases, leaves [0, T], or holds a
                               prompt longer than max_len */
  TV_ERR_BAD_PROBS = -11    /* tv_accept_sample: no token has a positive probability */
};

enum tv_dtype { TV_F32 = 0, TV_BF16 = 1 };
enum tv_mode { TV_MODE_FORK = 0, TV_MODE_WY = 1 };

#define TV_MAX_NODES 256
#define TV_BLOCK_SIZE 16
#define TV_STATIC_SCRATCH_BYTES (64u << 20) /* scratch array of tv_tree_attn_static: 64 MiB */

/* Human-readable name of a tv_status code (static string, never NULL). */
TV_API const char* tv_status_string(int status);

/* CUDA error code (cudaError_t value) of the last call that returned TV_ERR_CUDA on this
 * host thread, or 0. */
TV_API int tv_last_cuda_error(void);

/* Library ABI version: major * 10000 + minor * 100 + patch. */
TV_API int tv_version(void);

/* ------------------------------------------------------------------------------------------
 * tv_tree_prepare -- topology of B draft trees.
 *
 * Source: handbook chapter 树形草稿与 EAGLE, §实现, `depths` (depth 0 for a root, parent's
 * depth + 1 otherwise) and `tree_mask` (node i sees itself and every ancestor).
 *
 *   parents   [B, N] int32          in
 *   depth     [B, N] int32          out: depth of every node
 *   mask_bits [B, N, W] uint32      out: W = ceil(N / 32); bit (j % 32) of word j / 32 of row
 *                                   i is 1 iff node j is i or an ancestor of i
 *   paths     [B, N, path_cap] int32  out, optional (NULL: not written): row i is the root-to-i
 *                                   path (handbook §实现: the nodes a draft token's branch
 *                                   passes through), root first, then -1 up to path_cap entries
 *   path_cap  entries per path row, >= 1 when paths is given (depth + 1 entries are needed)
 *   max_depth [B] int32             out, optional (NULL: not written): the deepest node's depth
 *   err       [B] int32             out: 0, TV_ERR_BAD_TREE, or TV_ERR_UNSUPPORTED when a node's
 *                                   depth + 1 exceeds path_cap (depth, mask_bits and max_depth
 *                                   are still written; that sequence's paths are unspecified)
 * Outputs of a sequence whose tree is malformed are unspecified.  Returns TV_ERR_INVALID_ARG for
 * a null or misaligned required pointer, a misaligned optional one, or path_cap < 1 with paths.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_tree_prepare(const int32_t* parents, int B, int N, int32_t* depth, uint32_t* mask_bits,
                           int32_t* paths, int path_cap, int32_t* max_depth, int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_gdn_tree_verify_fork -- one GDN layer over B draft trees, fork/checkpoint mode.
 *
 * Source: qwen35-tree-spec §四 (Fork/Checkpoint, 逐深度处理): every node evolves from its
 * parent's snapshot (S_0 for a root) and its own snapshot is kept for the commit step; the
 * per-node semantics is exactly the root-to-node path replay of the gated delta rule above.
 * The kernel keeps each node's state in fp32 on chip and walks the tree depth-first, so each
 * parent state is read from HBM once (S_0) and each node's snapshot is written once.
 *
 *   q, k        [B, N, H, dk]  io_dtype      in
 *   v           [B, N, H, dv]  io_dtype      in
 *   alpha, beta [B, N, H]      fp32          in  (decay in (0,1], write strength)
 *   S0          [B, H, dv, dk] state_dtype   in  committed state (row = value index)
 *   parents     [B, N]         int32         in
 *   q_scale                                      o_i = S_i (q_scale * q_i)
 *   out         [B, N, H, dv]  io_dtype      out o_i
 *   node_states [B, N, H, dv, dk] state_dtype out S_i of every node (the checkpoints)
 *   err         [B] int32                    out 0 or TV_ERR_BAD_TREE
 * Supported: dk, dv in {64, 128}; (io, state) in {(F32,F32), (BF16,BF16), (BF16,F32)}.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_gdn_tree_verify_fork(const void* q, const void* k, const void* v, const float* alpha,
                            const float* beta, const void* S0, const int32_t* parents, int B,
                            int N, int H, int dk, int dv, int io_dtype, int state_dtype,
                            float q_scale, void* out, void* node_states, int32_t* err,
                            tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_gdn_tree_verify_wy -- one GDN layer over B draft trees, TreeWY mode.
 *
 * Source: TreeWY abstract -- all node outputs from one triangular solve over a small
 * pseudo-value matrix, no per-node states.  Reading of the algebra (not on the page): with
 * gamma_i the product of alpha along the root-to-node path P(i), Gamma_ij = gamma_i/gamma_j,
 * and the pseudo-value w_i = beta_i (v_i - alpha_i S_parent k_i),
 *     S_i = gamma_i S_0 + sum_{j in P(i)} Gamma_ij w_j k_j^T,
 *     (I + diag(beta)(A o Gamma o K K^T)) W = diag(beta)(V - diag(gamma) K S_0^T),
 *     O = diag(gamma) (q_scale Q) S_0^T + (M o Gamma o (q_scale Q) K^T) W,
 * A the strict-ancestor mask, M = A + I the tree mask.  The system is unit lower triangular
 * because parents[i] < i; it is solved along ancestor lists (each row of A has depth(i)
 * nonzeros).
 *
 *   inputs as tv_gdn_tree_verify_fork
 *   out         [B, N, H, dv]  io_dtype   out o_i
 *   pseudo_v    [B, N, H, dv]  fp32       out W (w_i per node and head)
 *   log_gamma   [B, N, H]      fp32       out log(gamma_i)
 *   err         [B] int32                 out 0, TV_ERR_BAD_TREE, or TV_ERR_UNSUPPORTED if
 *                                         the sum over nodes of (depth+1) exceeds 4096
 * Supported: dk, dv in {64, 128}; (io, state) as for fork.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_gdn_tree_verify_wy(const void* q, const void* k, const void* v, const float* alpha,
                          const float* beta, const void* S0, const int32_t* parents, int B,
                          int N, int H, int dk, int dv, int io_dtype, int state_dtype,
                          float q_scale, void* out, float* pseudo_v, float* log_gamma,
                          int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_gdn_tree_verify_wy_lazy -- TreeWY verify with the previous round's commit fused in.
 *
 * Source: TreeWY abstract (only the accepted state is rebuilt on commit).  The previous
 * round's WY commit (see tv_gdn_commit, TV_MODE_WY) is applied to S0 while it is staged for
 * this round's contraction, saving that commit's separate pass over the state:
 *   S0[b] <- gamma_a S0[b] + sum_r Gamma_{a,path[r]} w_{path[r]} k_{path[r]}^T   (written back)
 * then this round is verified exactly as tv_gdn_tree_verify_wy.  The committed S0 and all
 * outputs equal tv_gdn_commit followed by tv_gdn_tree_verify_wy, bit for bit.
 *
 *   prev_path [B, Lmax], prev_len [B]         the previous round's accepted paths (1 <= len
 *                                             <= min(Lmax, prev_N, 16))
 *   prev_parents [B, prev_N]                  the previous round's trees (the path's links are
 *                                             checked)
 *   prev_pseudo_v [B, prev_N, H, dv] fp32, prev_log_gamma [B, prev_N, H] fp32, prev_k
 *   [B, prev_N, H, dk]                        the previous round's W, log(gamma) and keys; they
 *                                             may share memory with this round's pseudo_v /
 *                                             log_gamma outputs
 *   S0                                        in/out
 *   other arguments as tv_gdn_tree_verify_wy
 *   err [B]  0, TV_ERR_BAD_TREE, TV_ERR_BAD_PATH (previous path invalid: the sequence is
 *            skipped, S0[b] untouched) or TV_ERR_UNSUPPORTED as tv_gdn_tree_verify_wy
 * Supported: bf16 I/O and state, dk = dv = 128, N <= 240 (else TV_ERR_UNSUPPORTED).
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_gdn_tree_verify_wy_lazy(const int32_t* prev_path, const int32_t* prev_len, int Lmax,
                                      const int32_t* prev_parents, int prev_N, const float* prev_pseudo_v,
                                      const float* prev_log_gamma, const void* prev_k, const void* q,
                                      const void* k, const void* v, const float* alpha, const float* beta,
                                      void* S0, const int32_t* parents, int B, int N, int H, int dk, int dv,
                                      int io_dtype, int state_dtype, float q_scale, void* out,
                                      float* pseudo_v, float* log_gamma, int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_gdn_commit -- write the accepted node's state back into S_0.
 *
 * Source: qwen35-tree-spec §五 用途 2 and §七 Step 4 (restore the state of the last accepted
 * token, drop the other snapshots); TreeWY abstract (rebuild only the accepted state).
 * The accepted path of sequence b is accepted_path[b][0 .. accepted_len[b]-1]: path[0] a
 * root and path[r] a child of path[r-1]; 1 <= accepted_len[b] <= Lmax.
 *
 *   mode = TV_MODE_FORK:  S0[b] <- node_states[b, path[L-1]]
 *   mode = TV_MODE_WY:    S0[b] <- gamma_a S0[b] + sum_r Gamma_{a,path[r]} w_{path[r]} k_{path[r]}^T
 *                         (a = path[L-1]), from pseudo_v, log_gamma and k of the verify call
 *
 *   accepted_path [B, Lmax] int32   in
 *   accepted_len  [B] int32         in
 *   parents       [B, N] int32      in  (to check the path)
 *   node_states   [B,N,H,dv,dk] state_dtype in  (fork mode; may be NULL in WY mode)
 *   pseudo_v      [B,N,H,dv] fp32, log_gamma [B,N,H] fp32, k [B,N,H,dk] io_dtype
 *                                   in  (WY mode; may be NULL in fork mode)
 *   S0            [B,H,dv,dk] state_dtype   in/out
 *   err           [B] int32         out 0, TV_ERR_BAD_TREE or TV_ERR_BAD_PATH (S0[b] untouched)
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_gdn_commit(int mode, const int32_t* accepted_path, const int32_t* accepted_len, int Lmax,
                  const int32_t* parents, const void* node_states, const float* pseudo_v,
                  const float* log_gamma, const void* k, void* S0, int B, int N, int H, int dk,
                  int dv, int io_dtype, int state_dtype, int32_t* err, tv_stream_t stream);

/* tv_gdn_commit_layers -- the commit of a whole stack of independent layers in one launch.
 * Every layer commits the same accepted paths (the path, its length and the parents are shared),
 * once the target has accepted them; the per-layer tensors lie back to back, layer first:
 *   S0 [layers, B, H, dv, dk]; fork: node_states [layers, B, N, H, dv, dk]; TreeWY:
 *   pseudo_v [layers, B, N, H, dv], log_gamma [layers, B, N, H], k [layers, B, N, H, dk].
 * The result for each layer equals tv_gdn_commit on that layer's slices.  err [B] reports the
 * shared path check.  layers >= 1; layers * B * H must fit in an int.  The pages have no
 * counterpart: layers are independent at commit time, so one launch serves them all. */
TV_API int tv_gdn_commit_layers(int mode, const int32_t* accepted_path, const int32_t* accepted_len, int Lmax,
                                const int32_t* parents, const void* node_states, const float* pseudo_v,
                                const float* log_gamma, const void* k, void* S0, int layers, int B, int N, int H,
                                int dk, int dv, int io_dtype, int state_dtype, int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_gdn_tree_verify_fork_ws -- fork mode in two passes, with a workspace.
 *
 * Same results and layouts as tv_gdn_tree_verify_fork (outputs and every node's snapshot),
 * computed differently: a TreeWY pass (TreeWY abstract: one triangular solve gives every
 * node's output and pseudo-value w_i = beta_i (v_i - alpha_i S_parent k_i)) writes the outputs
 * and w into the workspace; then every snapshot is materialized from its parent's along the
 * depth-first walk, S_i = alpha_i S_parent + w_i k_i^T -- the gated delta update
 * (qwen35-tree-spec §四) with its S_parent k_i term taken from the solve.
 *
 *   workspace   device scratch of at least tv_gdn_fork_workspace_size(B, N, H, dv) bytes,
 *               16-byte aligned, owned by the caller; contents on entry are ignored.  Calls
 *               that share a workspace must not overlap in time.
 *   err [B]     0, TV_ERR_BAD_TREE, or TV_ERR_UNSUPPORTED (also when the sum over nodes of
 *               (depth + 1) exceeds 4096, the TreeWY limit)
 * ---------------------------------------------------------------------------------------- */
TV_API size_t tv_gdn_fork_workspace_size(int B, int N, int H, int dv);
TV_API int tv_gdn_tree_verify_fork_ws(const void* q, const void* k, const void* v, const float* alpha,
                                      const float* beta, const void* S0, const int32_t* parents, int B, int N,
                                      int H, int dk, int dv, int io_dtype, int state_dtype, float q_scale,
                                      void* out, void* node_states, void* workspace, size_t workspace_bytes,
                                      int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_gdn_fork_materialize -- the snapshot pass of tv_gdn_tree_verify_fork_ws as a call of its
 * own, so that it can run on a second stream.
 *
 * Source: the gated delta update of qwen35-tree-spec §四, S_i = alpha_i S_parent + w_i k_i^T,
 * with w_i from a TreeWY verify (TreeWY abstract).  Every output of fork mode, and w, come from
 * tv_gdn_tree_verify_wy on the same q, k, v, alpha, beta, S0 and parents; this call writes
 * node_states exactly as tv_gdn_tree_verify_fork_ws does.  Nothing downstream of the outputs
 * needs the snapshots until the commit, so a caller may run this pass on its own stream (after
 * an event recorded behind the verify) while the next layer's verify runs on the first.
 *
 *   k, alpha, S0, parents   as tv_gdn_tree_verify_fork (read)
 *   pseudo_v     [B, N, H, dv] fp32, the w written by tv_gdn_tree_verify_wy (read)
 *   node_states  [B, N, H, dv, dk] state_dtype, 16-byte aligned (written)
 *   err [B]      in: the verify's per-sequence status -- a sequence with err != 0 is skipped
 *                and its snapshots are left untouched; out: unchanged for the others unless
 *                the depth-first schedule fails (TV_ERR_UNSUPPORTED)
 *   max_ctas_per_sm  0: as many resident CTAs per SM as fit; > 0: at most that many, which
 *                leaves registers and shared memory for kernels of other streams
 * Returns TV_ERR_INVALID_ARG for null or misaligned pointers, B, N or H < 1, or a negative
 * max_ctas_per_sm; TV_ERR_UNSUPPORTED for sizes or dtypes without a kernel.
 * The paper has no counterpart of the split: it is a scheduling choice of this library.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_gdn_fork_materialize(const void* k, const float* alpha, const void* S0, const int32_t* parents,
                                   const float* pseudo_v, int B, int N, int H, int dk, int dv, int io_dtype,
                                   int state_dtype, int max_ctas_per_sm, void* node_states, int32_t* err,
                                   tv_stream_t stream);

/* tv_gdn_fork_materialize_selective -- the same pass keeping only the selected snapshots
 * (qwen35-tree-spec §六, 选择性 Fork): node i keeps its snapshot iff confidence[b][i] <=
 * threshold, at slot s of node_states [B, capacity, H, dv, dk], slots numbered in node order,
 * exactly as tv_gdn_tree_verify_fork_selective; its outputs come from the preceding
 * tv_gdn_tree_verify_wy.  slot [B, N] int32 out (-1: no snapshot).  A sequence that keeps
 * more than capacity snapshots reports TV_ERR_CAPACITY in err and keeps none; a sequence the
 * verify rejected (err != 0 on entry) keeps none either (all its slots -1).  The commit is
 * tv_gdn_commit_selective.  Argument errors as tv_gdn_fork_materialize, plus a null
 * confidence or slot, a non-finite threshold, or capacity outside [1, N]. */
TV_API int tv_gdn_fork_materialize_selective(const void* k, const float* alpha, const void* S0,
                                             const int32_t* parents, const float* pseudo_v,
                                             const float* confidence, float threshold, int capacity, int B,
                                             int N, int H, int dk, int dv, int io_dtype, int state_dtype,
                                             int max_ctas_per_sm, void* node_states, int32_t* slot, int32_t* err,
                                             tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_gdn_tree_verify_fork_selective / tv_gdn_commit_selective -- fork mode with selective
 * snapshots.
 *
 * Source: qwen35-tree-spec §六, 选择性 Fork: a node whose draft confidence is above a
 * threshold (0.95 on the page) is processed without keeping a snapshot -- it is almost
 * surely accepted, so it needs no rollback point -- which cuts the snapshot count.
 *
 * Verify: as tv_gdn_tree_verify_fork, except that node i keeps its snapshot only if
 * confidence[b][i] <= threshold.  Kept snapshots are numbered 0, 1, ... in node order:
 *   confidence   [B, N] fp32                 in
 *   node_states  [B, capacity, H, dv, dk]    out snapshot of the node with slot s at index s
 *   slot         [B, N] int32                out snapshot index of each node, -1 if none (all
 *                                            -1 for a sequence that reports an error)
 *   err          [B] int32                   out 0, TV_ERR_BAD_TREE, TV_ERR_UNSUPPORTED, or
 *                                            TV_ERR_CAPACITY (more than capacity kept; the
 *                                            sequence is skipped)
 *   1 <= capacity <= N.
 * Commit: S0[b] <- state of the last accepted node, resumed from the deepest node of the
 * accepted path that kept a snapshot (S0[b] itself if none did) and replayed along the rest of
 * the path with k, v, alpha, beta of the verify call.  Path rules and err as tv_gdn_commit
 * (fork mode).
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_gdn_tree_verify_fork_selective(const void* q, const void* k, const void* v, const float* alpha,
                                             const float* beta, const void* S0, const int32_t* parents,
                                             const float* confidence, float threshold, int capacity, int B,
                                             int N, int H, int dk, int dv, int io_dtype, int state_dtype,
                                             float q_scale, void* out, void* node_states, int32_t* slot,
                                             int32_t* err, tv_stream_t stream);
TV_API int tv_gdn_commit_selective(const int32_t* accepted_path, const int32_t* accepted_len, int Lmax,
                                   const int32_t* parents, const void* node_states, const int32_t* slot,
                                   int capacity, const void* k, const void* v, const float* alpha,
                                   const float* beta, void* S0, int B, int N, int H, int dk, int dv,
                                   int io_dtype, int state_dtype, int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_tree_attn -- tree-masked GQA attention over a paged KV prefix.
 *
 * Source: handbook chapter 树形草稿与 EAGLE, §实现, forward_with_mask: q and k of the new
 * nodes are rotated (RoPE) at position prefix_len + depth; keys/values are the cached prefix
 * followed by the nodes'; node i sees the whole prefix, its ancestors and itself; query head
 * h reads KV head h / (Hq / Hkv); softmax scale sm_scale (pass 1/sqrt(hd) for the default).
 * RoPE reading: rotate-half pairs (x_c, x_{c+hd/2}), angle pos * rope_theta^(-2c/hd), over the
 * full head dim.  Cached prefix keys are stored already rotated.
 *
 * The call first writes each node's rotated key and its value into the cache at logical slot
 * prefix_len[b] + i, then attends over logical slots [0, prefix_len[b] + N).
 *
 *   q            [B, N, Hq, hd]  bf16     in  (not rotated)
 *   k_new, v_new [B, N, Hkv, hd] bf16     in  (k not rotated)
 *   k_cache, v_cache [num_blocks, Hkv, block_size, hd] bf16  in/out
 *   block_table  [B, max_blocks] int32    in  logical slot s of sequence b lives in block
 *                                         block_table[b][s / block_size], row s % block_size
 *   prefix_len   [B] int32                in
 *   parents      [B, N] int32             in
 *   out          [B, N, Hq, hd] bf16      out
 *   workspace    device scratch of at least tv_tree_attn_workspace_size(...) bytes, 256-byte
 *                aligned, owned by the caller; contents on entry are ignored.  Calls that
 *                share a workspace must not overlap in time.
 *   err          [B] int32                out 0, TV_ERR_BAD_TREE, TV_ERR_CAPACITY
 *                                         (prefix_len + N > max_blocks * block_size or
 *                                         prefix_len < 0), TV_ERR_BAD_BLOCK, or TV_ERR_TIMEOUT
 *                                         (a bounded device wait gave up; that sequence's
 *                                         outputs are then unspecified)
 * Supported: hd in {64, 128, 256}; block_size = 16; Hq a multiple of Hkv; B <= 65535.
 * ---------------------------------------------------------------------------------------- */
TV_API size_t tv_tree_attn_workspace_size(int B, int N, int Hq, int Hkv, int hd, int max_blocks,
                                   int block_size);

TV_API int tv_tree_attn(const void* q, const void* k_new, const void* v_new, void* k_cache,
                 void* v_cache, int num_blocks, const int32_t* block_table, int max_blocks,
                 const int32_t* prefix_len, const int32_t* parents, int B, int N, int Hq,
                 int Hkv, int hd, int block_size, float rope_theta, float sm_scale, void* out,
                 void* workspace, size_t workspace_bytes, int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_tree_attn_static -- tv_tree_attn without a workspace and without any allocation.
 *
 * The pages have no counterpart: this is a deployment variant of tv_tree_attn, for callers
 * that cannot hand the library a workspace (e.g. code that must not allocate).  Arguments,
 * layouts, results and the err codes are those of tv_tree_attn; the workspace is replaced by
 * one device array of TV_STATIC_SCRATCH_BYTES (64 MiB) owned by the library.
 *
 *  - Size limit: when tv_tree_attn_workspace_size(B, N, Hq, Hkv, hd, max_blocks, block_size)
 *    exceeds TV_STATIC_SCRATCH_BYTES the call returns TV_ERR_SCRATCH before any CUDA call
 *    and launches nothing; use tv_tree_attn with a workspace for such sizes.
 *  - Argument errors: every host-side check of tv_tree_attn (null or misaligned pointers,
 *    sizes) runs before any CUDA call, as does the size limit below.
 *  - Set-up: the first call in each CUDA context looks up the array's device address
 *    (cudaGetSymbolAddress; a failure returns TV_ERR_CUDA) and caches it with that context.
 *    That lookup may load a module, so make the first call on each device in set-up code,
 *    before any stream capture.  A call made in a new context of the device (e.g. after
 *    cudaDeviceReset) looks the address up again: the old one died with the old context.
 *  - Shared state: the scratch is one array per device for the whole process.  Its contents
 *    persist between calls; nothing in it has to start at zero (every call writes each
 *    scratch entry it reads).  Two calls whose execution overlaps on the same device (other
 *    streams, other host threads) race on it: serialise them, e.g. on one stream.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_tree_attn_static(const void* q, const void* k_new, const void* v_new, void* k_cache,
                        void* v_cache, int num_blocks, const int32_t* block_table, int max_blocks,
                        const int32_t* prefix_len, const int32_t* parents, int B, int N, int Hq,
                        int Hkv, int hd, int block_size, float rope_theta, float sm_scale,
                        void* out, int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_kv_compact -- keep the accepted path's KV, in place.
 *
 * Source: handbook chapter 树形草稿与 EAGLE, note after the listing (the accepted nodes' KV
 * was computed at the right positions during verification and is moved to the sequence's
 * contiguous slots; rejected slots become void) and qwen35-tree-spec §七 Step 4.
 * For r < L = accepted_len[b]: logical slot prefix_len[b] + r receives what logical slot
 * prefix_len[b] + path[r] held before the call (every source is read before any write), for
 * K and V and all KV heads.  Slots at or past the new length are left as they are.
 *
 *   k_cache, v_cache [num_blocks, Hkv, block_size, hd] bf16   in/out
 *   block_table [B, max_blocks] int32, prefix_len [B] int32, parents [B, N] int32   in
 *   accepted_path [B, Lmax] int32, accepted_len [B] int32                            in
 *   slot_map    [B, Lmax] int32   out physical source slot (block * block_size + row) of
 *                                 each kept entry, -1 for r >= L
 *   new_len     [B] int32         out prefix_len + L (prefix_len on error)
 *   err         [B] int32         out 0, TV_ERR_BAD_TREE, TV_ERR_BAD_PATH, TV_ERR_CAPACITY
 *                                 or TV_ERR_BAD_BLOCK
 * Precondition, checked: the table entries of the logical blocks that hold slots prefix_len ..
 * prefix_len + N - 1 (the window every source and destination lies in) are distinct physical
 * blocks.  Were two of them the same block, a store could overwrite a source before it is read;
 * such a sequence reports TV_ERR_BAD_BLOCK and is skipped.
 * Supported: hd in {64, 128, 256}; block_size = 16.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_kv_compact(void* k_cache, void* v_cache, int num_blocks, const int32_t* block_table,
                  int max_blocks, const int32_t* prefix_len, const int32_t* parents, int N,
                  const int32_t* accepted_path, const int32_t* accepted_len, int Lmax, int B,
                  int Hkv, int hd, int block_size, int32_t* slot_map, int32_t* new_len,
                  int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_kv_compact_remap -- keep the accepted path's KV, exchanging whole blocks of the block
 * table where that replaces moving them.
 *
 * Source: handbook chapter 树形草稿与 EAGLE, note after the listing (the accepted nodes' slots
 * are compacted to the sequence's positions, or only the block table is updated).  Reading,
 * per sequence with P = prefix_len[b], L = accepted_len[b], block size 16:
 *  - a logical block m with 16 m >= P that holds kept entries (P + r for r < L), all of which
 *    come from logical slot P + r + 16 j for one j >= 1, takes block m + j's physical block:
 *    entries m and m + j of the table row are exchanged, in ascending m;
 *  - every other kept entry r is moved: physical slot (new row, P + r) receives what physical
 *    slot (old row, P + path[r]) held before the call.  Every source is read before any
 *    write; an entry already in place is not written.
 * Read through block_table_out, logical slots [0, P + L) then hold what tv_kv_compact leaves
 * in them read through block_table.  The new row is a permutation of the old one; entries of
 * blocks holding prefix slots are unchanged.  Slots at or past the new length are void.
 *
 *   k_cache, v_cache [num_blocks, Hkv, block_size, hd] bf16     in/out
 *   block_table     [B, max_blocks] int32   in   the rows before the call
 *   block_table_out [B, max_blocks] int32   out  the rows after the exchanges (a copy of the
 *                                                row for a sequence with an error); must not
 *                                                overlap block_table (TV_ERR_INVALID_ARG)
 *   prefix_len, parents, accepted_path, accepted_len, slot_map, new_len, err: as for
 *                                                tv_kv_compact (slot_map under the old rows)
 *   remapped        [B] int32               out  exchanges made (0 on error)
 * Precondition, checked as for tv_kv_compact: the window's table entries are distinct (an
 * exchange of two entries naming one block would lose none but move data twice);
 * TV_ERR_BAD_BLOCK otherwise, the row copied unchanged.
 * Supported: hd in {64, 128, 256}; block_size = 16; N <= TV_MAX_NODES.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_kv_compact_remap(void* k_cache, void* v_cache, int num_blocks, const int32_t* block_table,
                        int32_t* block_table_out, int max_blocks, const int32_t* prefix_len,
                        const int32_t* parents, int N, const int32_t* accepted_path,
                        const int32_t* accepted_len, int Lmax, int B, int Hkv, int hd, int block_size,
                        int32_t* slot_map, int32_t* new_len, int32_t* remapped, int32_t* err,
                        tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_accept_walk -- greedy acceptance of B draft trees, on the device.
 *
 * Source: handbook chapter 树形草稿与 EAGLE, §实现, tree_speculative_generate: from node 0,
 * while the target model's token at the current node equals the draft token of one of its
 * children, step to the lowest-numbered such child; the target's token at the last accepted
 * node is the next token.  The walk also stops once Lmax nodes are accepted.  Its output feeds
 * tv_gdn_commit and tv_kv_compact without a host round trip.
 *
 *   parents        [B, N] int32   in
 *   draft_tokens   [B, N] int32   in  token proposed at each node
 *   target_tokens  [B, N] int32   in  token the target model chose at each node (its argmax)
 *   accepted_path  [B, Lmax] int32 out path[0] = 0, path[r] a child of path[r-1]; -1 past the
 *                                      length
 *   accepted_len   [B] int32      out 1 <= len <= Lmax (0 on error)
 *   next_token     [B] int32      out target_tokens[b][path[len-1]] (-1 on error)
 *   err            [B] int32      out 0 or TV_ERR_BAD_TREE
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_accept_walk(const int32_t* parents, const int32_t* draft_tokens, const int32_t* target_tokens,
                          int B, int N, int Lmax, int32_t* accepted_path, int32_t* accepted_len,
                          int32_t* next_token, int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_linear_attn_prompt -- linear attention with a decay over whole prompts.
 *
 * The pages have no counterpart: they verify draft trees from a committed state.  This call
 * makes such a state from a prompt, for layers whose recurrence decays without a delta
 * correction -- the gated delta rule above with its (I - beta k k^T) left out:
 *     S_t = alpha_t S_{t-1} + v_t k_t^T,     o_t = S_t (q_scale q_t),
 * S [dv, dk] with the value index as its row, as everywhere in this library.
 *
 * B prompts lie back to back: prompt b is tokens cu_seqlens[b] .. cu_seqlens[b+1] - 1 of T.  A
 * prompt may be empty (its S is then its S0).  Query and key heads may be shared: value head h
 * reads query and key head h / (H / Hk).
 *
 *   q, k        [T, Hk, dk] io_dtype   in   token t's heads start at q + t * q_stride (elements);
 *   v           [T, H, dv]  io_dtype   in   k_stride, v_stride, out_stride alike: slices of one
 *                                           projection's output need no copy
 *   alpha       fp32                   in   decay in [0, 1] of token t, head h at
 *                                           alpha[t * alpha_stride + h]; alpha_stride 0: [H], one
 *                                           decay for each head
 *   S0          [B, H, dv, dk] state_dtype  in   state before the prompt; NULL: zero
 *   cu_seqlens  [B + 1] int32          in
 *   max_len     an upper bound of the prompts' lengths (T serves; closer is faster).  Long prompts
 *               are cut into segments that run side by side; where depends on the sizes and max_len,
 *               and with it the order of some sums: results of calls that agree in those are equal
 *               bit for bit
 *   out         [T, H, dv]  io_dtype   out  rows of no prompt are not written
 *   S           [B, H, dv, dk] state_dtype  out  state after the prompt; may be S0 itself
 *   workspace   device scratch of at least tv_linear_attn_workspace_size(...) bytes, 16-byte
 *               aligned (may be NULL when that is 0); contents on entry are ignored.  Calls that
 *               share a workspace must not overlap in time.
 *   err         [B] int32              out  0, or TV_ERR_BAD_SEQLEN in every entry when cu_seqlens
 *                                           decreases, leaves [0, T] or holds a prompt longer than
 *                                           max_len (nothing else is written then); or
 *                                           TV_ERR_TIMEOUT (a bounded device wait gave up; that
 *                                           prompt's outputs are then unspecified)
 * Rounding: products accumulate in fp32; bf16 operands that are themselves sums or scaled
 * (scores, decayed keys, states) enter the matrix units as a bf16 pair, value and remainder, the
 * keys of an fp32 state in three parts.  From chunk to chunk a state is carried in 32 bits, and the
 * matrix units, which cut what they add to an accumulator, add to its small remainder only.  An
 * fp32 state of bf16 inputs is off by at most 1e-6 of its norm, whatever its length, its decays and
 * the share of tokens that add to it (measured: 5e-7 after 32768 tokens); what is left of an S0 to
 * which nothing was added, decayed to e^-x of itself, by x * 1e-7 more.
 * fp32 inputs are walked token by token, and a state takes in each with one rounding to nearest: off
 * by 3e-7 after some thousand tokens of mixed decays, by 1.1e-6 after 8192 and 2.2e-6 after 32768
 * that do not decay; decays themselves cost nothing (a state to which nothing is added: 1e-7).
 * Values beyond 2^106 may overflow there.
 * The states are not a gated delta rule's: no tv_gdn_* call takes them.
 * A non-finite input makes later tokens of its prompt and head non-finite, and may make earlier
 * ones of the same 128-token chunk so; other prompts are not touched.
 * Supported: dk, dv in {64, 128}; H a multiple of Hk; (io, state) as tv_gdn_tree_verify_fork.
 * Strides: at least the dense row (Hk * dk or H * dv; alpha H or 0) and whole multiples of 16
 * bytes (alpha: any), else TV_ERR_INVALID_ARG.  B * H <= 2^24.
 * ---------------------------------------------------------------------------------------- */
TV_API size_t tv_linear_attn_workspace_size(int B, int T, int max_len, int H, int dk, int dv, int io_dtype);
TV_API int tv_linear_attn_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, const float* alpha, int64_t alpha_stride, const void* S0,
                                 const int32_t* cu_seqlens, int B, int T, int max_len, int Hk, int H, int dk, int dv,
                                 int io_dtype, int state_dtype, float q_scale, void* out, int64_t out_stride, void* S,
                                 void* workspace, size_t workspace_bytes, int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_linear_attn_step -- the same recurrence for one new token of every sequence.
 *
 * S <- alpha S + v k^T in place, out = S (q_scale q).  The output uses the fp32 state before its
 * rounding to state_dtype.
 *
 *   q, k        [B, Hk, dk] io_dtype, v [B, H, dv] io_dtype   in   strides as tv_linear_attn_prompt
 *   alpha       [B, H] (alpha_stride) or [H] (alpha_stride 0) fp32   in
 *   live        [B] int32, optional (NULL: all)   in   a sequence with live[b] = 0 is skipped: its
 *               state and output rows are left as they are (rows of a padded batch)
 *   out         [B, H, dv] io_dtype               out
 *   S           [B, H, dv, dk] state_dtype        in/out
 * Supported sizes and types as tv_linear_attn_prompt.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_linear_attn_step(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                               int64_t v_stride, const float* alpha, int64_t alpha_stride, const int32_t* live, int B,
                               int Hk, int H, int dk, int dv, int io_dtype, int state_dtype, float q_scale, void* out,
                               int64_t out_stride, void* S, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_gated_rmsnorm -- a mixer's output, normalised per head and multiplied by its gate.
 *
 * With n(x) = x / sqrt(mean(x^2) + eps) * (weight_offset + weight) over the d columns of a head and
 * silu(g) = g / (1 + exp(-g)):
 *     gate_first = 0:  out = n(x) silu(gate)          gate_first = 1:  out = n(x silu(gate))
 *
 *   x, gate, out  [rows, H, d] io_dtype   row r starts at x + r * x_stride (elements); gate may be
 *                 NULL (factor 1); out may be x itself
 *   weight        [d] io_dtype, or NULL (out is not scaled by a weight, and weight_offset is not used)
 * Arithmetic is fp32, rounded once on store.  silu(g) of gates below -87.3, at most 1e-36, is 0.  Any d from 1 to 32768 and any stride of at least H * d;
 * base addresses need only their element's alignment.  rows * H <= 2^31 - 256.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_gated_rmsnorm(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride,
                            const void* weight, int rows, int H, int d, int io_dtype, float eps, float weight_offset,
                            int gate_first, void* out, int64_t out_stride, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_residual_rmsnorm -- a block's output into the residual stream, and the next block's norm.
 *
 *     t   = y, or n(y) with post_weight          (the norm after the block)
 *     r   = residual + scale * gate * t          (gate NULL: 1)
 *     residual_out = r,  out = n(r) with weight  (the norm before the next block)
 * n as above, over the D columns; out is taken from the fp32 r before its rounding.
 *
 *   y, gate, out             [rows, D] io_dtype; out may be NULL (weight is then ignored)
 *   residual, residual_out   [rows, D] residual_dtype
 *   post_weight, weight      [D] io_dtype; post_weight NULL: no norm after the block; weight NULL: n
 *                            without a weight
 * residual_out may be residual itself, and out may be y itself.  Supported: (io, residual) in
 * {(F32,F32), (BF16,BF16), (BF16,F32)}; 1 <= D <= 32768; strides of at least D elements; base
 * addresses need only their element's alignment.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_residual_rmsnorm(const void* y, int64_t y_stride, const void* residual, int64_t residual_stride,
                               const void* post_weight, const void* gate, int64_t gate_stride, float scale,
                               const void* weight, int rows, int D, int io_dtype, int residual_dtype, float eps,
                               float weight_offset, void* residual_out, int64_t residual_out_stride, void* out,
                               int64_t out_stride, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_qk_norm_rope -- norms of queries and keys per head, their rotation by position, and the new
 * keys and values into the paged cache, in one pass.
 *
 * What lies between a softmax layer's projections and its attention.  For every head of q and k
 *     y = x / sqrt(mean(x^2) + eps) * (weight_offset + weight)      (norm = 0: y = x)
 * over its hd columns, then the first rotary_dim columns are rotated as in tv_tree_attn: pairs
 * (y_c, y_{c + rotary_dim/2}) by the angle position * rope_theta^(-2c/rotary_dim).  The i-th new
 * token of sequence b has position prefix_len[b] + i and goes to that logical slot of the cache;
 * values are copied as they are.  Angles are formed from whole turns in 64-bit fixed point, exact
 * to 2^-27 of a turn for every position below 2^31.
 *
 *   q            [T, Hq, hd], k, v [T, Hkv, hd] io_dtype  in   token t's heads start at
 *                q + t * q_stride (elements); k_stride, v_stride and the output strides alike
 *   q_weight, k_weight [hd] io_dtype, or NULL (no weight, and weight_offset is not used)
 *   cu_seqlens   [B + 1] int32  in   sequence b's new tokens are cu_seqlens[b] .. cu_seqlens[b+1]-1;
 *                NULL: one token for each sequence, T = B
 *   prefix_len   [B] int32      in   tokens before the new ones; may be NULL (zero) without a cache
 *   live         [B] int32, optional (NULL: all)  in   a sequence with live[b] = 0 is skipped, its
 *                rows of every output left as they are
 *   q_out        [T, Hq, hd]  io_dtype  out  may be q itself
 *   k_out        [T, Hkv, hd] io_dtype  out  optional (NULL: not written); may be k itself
 *   k_cache, v_cache [num_blocks, Hkv, block_size, hd] bf16  out  optional, both or neither (then v,
 *                block_table, num_blocks, max_blocks and block_size are not used); at least one of
 *                k_out and the caches is given.  The blocks that new tokens go to belong to one
 *                sequence each
 *   block_table  [B, max_blocks] int32   in
 *   err          [B] int32   out  0, TV_ERR_BAD_SEQLEN in every entry (cu_seqlens decreases or leaves
 *                [0, T]; nothing else is written), TV_ERR_CAPACITY (prefix_len + tokens passes the
 *                block table, or 2^31 - 1; prefix_len < 0) or TV_ERR_BAD_BLOCK (a block that a new
 *                token goes to); a failed sequence's rows are left as they are
 * Rows of no sequence are not written.  Arithmetic is fp32, rounded once on store.  Supported: hd in
 * {64, 128, 256}; rotary_dim a multiple of 16 from 0 (no rotation) to hd; block_size = 16; io F32 or
 * BF16, the caches with BF16 only.  rope_theta >= 1.  Strides: at least the dense row and whole
 * multiples of 16 bytes.  With rotary_dim = 0 and no cache it makes the norms alone, as before
 * tv_tree_attn, which rotates itself.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                           int64_t v_stride, const void* q_weight, const void* k_weight, const int32_t* cu_seqlens,
                           const int32_t* prefix_len, const int32_t* live, int B, int T, int Hq, int Hkv, int hd,
                           int rotary_dim, int io_dtype, int norm, float eps, float weight_offset, float rope_theta,
                           void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride, void* k_cache,
                           void* v_cache, int num_blocks, const int32_t* block_table, int max_blocks, int block_size,
                           int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_window_attn_prompt -- GQA attention of new tokens over the paged cache, within a window.
 *
 * Whole prompts, later parts of them, or drafted chains: the n new tokens of a sequence stand at
 * positions prefix_len .. prefix_len + n - 1, and their keys and values already lie in the cache
 * (tv_qk_norm_rope puts them there).  The query at position p sees key j <= p if
 *     p - j < window (window = 0: every j),   or   j < sinks (a few first tokens that stay visible);
 * query head h reads KV head h / (Hq / Hkv); o = sum_j softmax_j(sm_scale q . k_j) v_j.
 *
 *   q            [T, Hq, hd] bf16  in   rotated; token t's heads start at q + t * q_stride (elements)
 *   k_cache, v_cache [num_blocks, Hkv, block_size, hd] bf16   in
 *   block_table  [B, max_blocks] int32   in   entries of blocks that no query of the call sees are not
 *                read (blocks behind the window may have been given back)
 *   cu_seqlens   [B + 1] int32     in   sequence b's new tokens; it may have none
 *   prefix_len   [B] int32         in   tokens before the new ones
 *   max_len      an upper bound of the numbers of new tokens (T serves; closer is faster)
 *   out          [T, Hq, hd] bf16  out  strided like q; rows of no sequence are not written
 *   workspace    device scratch of at least tv_window_attn_workspace_size(...) bytes, 16-byte
 *                aligned (may be NULL when that is 0); contents on entry are ignored.  Calls that
 *                share a workspace must not overlap in time.
 *   err          [B] int32         out  0, TV_ERR_BAD_SEQLEN in every entry (nothing else is written
 *                then), TV_ERR_CAPACITY (prefix_len + tokens passes the block table; prefix_len < 0),
 *                TV_ERR_BAD_BLOCK (a block that some query sees is outside the cache), or
 *                TV_ERR_TIMEOUT (a bounded device wait gave up; that sequence's outputs are then
 *                unspecified)
 * Scores, softmax statistics and sums are fp32; the weights enter the product with the values as bf16.  Outputs are off by
 * 0.0016 to 0.0024 of their norm, 0.0017 of it the store's rounding, at any length of the context.  With at most 16 query rows
 * (max_len times query heads of a KV head) weights are summed as rounded, otherwise before: within that error, a query's
 * output depends on which.
 * Results depend on the lengths of all sequences (where work is cut), on no other's data.  A non-finite key or value that
 * some query sees may reach other queries of its sequence and KV head; one that no query of the
 * sequence sees reaches none.
 * Supported: hd in {64, 128, 256}; block_size = 16; Hq a multiple of Hkv, Hq / Hkv <= 128; window and
 * sinks from 0; sequences up to 2^30 tokens (max_blocks <= 2^26); num_blocks * Hkv <= 2^29;
 * B * Hkv <= 2^24.  Strides: at least the dense row and whole multiples of 16 bytes.
 * ---------------------------------------------------------------------------------------- */
TV_API size_t tv_window_attn_workspace_size(int B, int T, int max_len, int Hq, int Hkv, int hd, int max_blocks,
                                            int block_size, int window, int sinks);
TV_API int tv_window_attn_prompt(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                                 int num_blocks, const int32_t* block_table, int max_blocks,
                                 const int32_t* cu_seqlens, const int32_t* prefix_len, int B, int T, int max_len,
                                 int Hq, int Hkv, int hd, int block_size, int window, int sinks, float sm_scale,
                                 void* out, int64_t out_stride, void* workspace, size_t workspace_bytes, int32_t* err,
                                 tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_window_attn_step -- the same attention for one new token of every sequence.
 *
 * The token of sequence b stands at position prefix_len[b]; its key and value lie in the cache.
 *
 *   q, out       [B, Hq, hd] bf16, strided as tv_window_attn_prompt
 *   live         [B] int32, optional (NULL: all)   in   a sequence with live[b] = 0 is skipped: its
 *                output row is left as it is, its err is 0 (rows of a padded batch)
 *   workspace    of at least tv_window_attn_workspace_size(B, B, 1, ...) bytes
 *   err          [B] int32   out  0, TV_ERR_CAPACITY, TV_ERR_BAD_BLOCK or TV_ERR_TIMEOUT
 * Everything else as tv_window_attn_prompt.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_window_attn_step(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache,
                               int num_blocks, const int32_t* block_table, int max_blocks, const int32_t* prefix_len,
                               const int32_t* live, int B, int Hq, int Hkv, int hd, int block_size, int window,
                               int sinks, float sm_scale, void* out, int64_t out_stride, void* workspace,
                               size_t workspace_bytes, int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_accept_sample -- acceptance of B draft trees by probabilities, on the device.
 *
 * The sampled counterpart of tv_accept_walk: the accepted tokens and the one after them are
 * distributed as if the target model had drawn them, given uniform random numbers.  From node 0 the
 * walk tests the children of the last accepted node in ascending order.  With p = target_probs[node]
 * and, as the tokens are refused one after another, R_0 = p and M_0 = 1:
 *   draft_probs given (every child's token was drawn from q = draft_probs[node]):
 *     accept child c with token x if uniforms[c] * q(x) * M_k < R_k(x), else
 *     R_{k+1} = max(R_k - M_k q, 0),  M_{k+1} = sum R_{k+1};
 *     where that sum is 0, R and M start again from p and 1;
 *   draft_probs NULL (children are chosen, not drawn, and distinct):
 *     accept if uniforms[c] * M_k < R_k(x), else R_{k+1} = R_k with R(x) = 0, M_{k+1} = M_k - R_k(x).
 * Without a child accepted, or once Lmax nodes are, next_token is the smallest x with
 *     R(0) + ... + R(x) > uniforms[0] * sum R        (R is p where nothing was refused, or sum R = 0).
 * Probabilities are taken as they are, negative ones and NaN as 0.  A token outside [0, V) is never
 * accepted.  All sums, and products of numbers above 2^-100, are carried to 2^-44 or better.  A chain is a tree too, and N = 1
 * draws one token from target_probs.
 *
 *   parents, draft_tokens [B, N] int32     in   as tv_accept_walk
 *   target_probs   [B, N, V] probs_dtype   in   row i: the target's probabilities after node i
 *   draft_probs    [B, N, V] probs_dtype   in   row i: what node i's children were drawn from; or NULL
 *   uniforms       [B, N] fp32             in   in [0, 1); entry 0 draws the next token
 *   accepted_path  [B, Lmax], accepted_len [B], next_token [B] int32   out   as tv_accept_walk
 *   err            [B] int32               out  0, TV_ERR_BAD_TREE, or TV_ERR_BAD_PROBS when the row
 *                                               that the next token is drawn from has no positive
 *                                               entry (path -1, length 0, next_token -1 for both)
 * Supported: N <= TV_MAX_NODES, V <= 2^24, probs F32 or BF16.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_accept_sample(const int32_t* parents, const int32_t* draft_tokens, const void* target_probs,
                            const void* draft_probs, const float* uniforms, int B, int N, int V, int Lmax,
                            int probs_dtype, int32_t* accepted_path, int32_t* accepted_len, int32_t* next_token,
                            int32_t* err, tv_stream_t stream);

/* ------------------------------------------------------------------------------------------
 * tv_test_bounded_wait -- test support for the bounded device waits.
 *
 * The pages have no counterpart: this checks a property of the library.  Every wait of the
 * tensor-core kernels on a shared-memory mbarrier (copies landed, MMAs done) gives up after a
 * bounded number of polls, and the kernel then reports TV_ERR_TIMEOUT in err[b] and returns.
 * This call launches one thread that runs that same wait on a barrier nothing arrives on (no
 * copy or MMA is in flight), so a test can make it run out:
 *   max_polls   polls before giving up; 0 = the limit the library's kernels use
 *   arrive      nonzero: the thread arrives on the barrier first, so the wait succeeds
 *   status      [1] int32 out   TV_OK or TV_ERR_TIMEOUT
 *   elapsed_ns  [1] int64 out   device time the wait took (the %globaltimer clock)
 * Returns TV_ERR_INVALID_ARG for a null or misaligned pointer.
 * ---------------------------------------------------------------------------------------- */
TV_API int tv_test_bounded_wait(unsigned max_polls, int arrive, int32_t* status, int64_t* elapsed_ns,
                                tv_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* TV_H_ */
