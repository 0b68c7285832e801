// C ABI entry points (declared in include/tv.h): host-side argument checks, then the
// launchers of the individual kernels.  Nothing here allocates device memory.
#include <math.h>
#include <stdint.h>

#include "tv.h"
#include "tv_internal.h"

namespace tv {

int device_sm_count() {
  static int cached[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 148;
  if (dev < 64 && cached[dev] > 0) return cached[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) n = 148;
  if (dev < 64) cached[dev] = n;
  return n;
}

}  // namespace tv

namespace {

thread_local int g_last_cuda = 0;

int cuda_status(cudaError_t e) {
  if (e == cudaSuccess) return TV_OK;
  g_last_cuda = static_cast<int>(e);
  return TV_ERR_CUDA;
}

}  // namespace

int tv::cuda_status_of(cudaError_t e) { return cuda_status(e); }

namespace {

bool a16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool a4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool dim_ok(int d) { return d == 64 || d == 128; }

// (io, state) pairs with a kernel: (F32,F32), (BF16,BF16), (BF16,F32).
int gdn_dtypes(int io, int state) {
  if ((io == TV_F32 && state == TV_F32) || (io == TV_BF16 && state == TV_BF16) ||
      (io == TV_BF16 && state == TV_F32))
    return TV_OK;
  if ((io != TV_F32 && io != TV_BF16) || (state != TV_F32 && state != TV_BF16)) return TV_ERR_INVALID_ARG;
  return TV_ERR_UNSUPPORTED;
}

int gdn_common(const void* q, const void* k, const void* v, const float* alpha, const float* beta,
               const void* S0, const int32_t* parents, int B, int N, int H, int dk, int dv, int io,
               int state, float q_scale, const void* out, const int32_t* err) {
  if (!a16(q) || !a16(k) || !a4(v) || !a4(alpha) || !a4(beta) || !a16(S0) || !a4(parents) || !a4(out) ||
      !a4(err))
    return TV_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || H < 1 || !isfinite(q_scale)) return TV_ERR_INVALID_ARG;
  if (N > TV_MAX_NODES || !dim_ok(dk) || !dim_ok(dv)) return TV_ERR_UNSUPPORTED;
  return gdn_dtypes(io, state);
}

}  // namespace

extern "C" {

const char* tv_status_string(int status) {
  switch (status) {
    case TV_OK: return "ok";
    case TV_ERR_INVALID_ARG: return "invalid argument";
    case TV_ERR_BAD_TREE: return "malformed tree (parents[i] must be -1 or an earlier node)";
    case TV_ERR_BAD_PATH: return "accepted path is not a root-to-node path";
    case TV_ERR_UNSUPPORTED: return "unsupported size or dtype";
    case TV_ERR_CUDA: return "CUDA launch error";
    case TV_ERR_TIMEOUT: return "device wait timed out";
    case TV_ERR_CAPACITY: return "block table too short for prefix_len + N slots";
    case TV_ERR_BAD_BLOCK: return "block-table entry outside the cache";
    case TV_ERR_BAD_SEQLEN: return "cu_seqlens decreases, leaves [0, T] or holds a prompt longer than max_len";
    case TV_ERR_BAD_PROBS: return "no token has a positive probability";
    case TV_ERR_SCRATCH: return "request needs more than the static scratch of TV_STATIC_SCRATCH_BYTES";
    default: return "unknown status";
  }
}

int tv_last_cuda_error(void) { return g_last_cuda; }

int tv_version(void) { return 100; }

int tv_tree_prepare(const int32_t* parents, int B, int N, int32_t* depth, uint32_t* mask_bits, int32_t* paths,
                    int path_cap, int32_t* max_depth, int32_t* err, tv_stream_t stream) {
  if (!a4(parents) || !a4(depth) || !a4(mask_bits) || !a4(err) || B < 1 || N < 1) return TV_ERR_INVALID_ARG;
  if ((paths != nullptr && (!a4(paths) || path_cap < 1)) || (max_depth != nullptr && !a4(max_depth)))
    return TV_ERR_INVALID_ARG;
  if (N > TV_MAX_NODES) return TV_ERR_UNSUPPORTED;
  return cuda_status(tv::launch_tree_prepare(parents, B, N, depth, mask_bits, paths, paths ? path_cap : 0, max_depth,
                                             err, stream));
}

int tv_gdn_tree_verify_fork(const void* q, const void* k, const void* v, const float* alpha,
                            const float* beta, const void* S0, const int32_t* parents, int B, int N,
                            int H, int dk, int dv, int io_dtype, int state_dtype, float q_scale,
                            void* out, void* node_states, int32_t* err, tv_stream_t stream) {
  int st = gdn_common(q, k, v, alpha, beta, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, q_scale,
                      out, err);
  if (st != TV_OK) return st;
  if (!a16(node_states)) return TV_ERR_INVALID_ARG;
  tv::GdnArgs a{q, k, v, alpha, beta, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, q_scale, out, err};
  const tv::ForkSelect all{nullptr, 0.f, N, nullptr};
  return cuda_status(tv::launch_gdn_fork(a, node_states, all, stream));
}

size_t tv_gdn_fork_workspace_size(int B, int N, int H, int dv) {
  if (B < 1 || N < 1 || H < 1 || dv < 1) return 0;
  const size_t pv = ((size_t)B * N * H * dv * 4 + 255) & ~(size_t)255;
  const size_t lg = ((size_t)B * N * H * 4 + 255) & ~(size_t)255;
  return pv + lg;
}

int tv_gdn_tree_verify_fork_ws(const void* q, const void* k, const void* v, const float* alpha, const float* beta,
                               const void* S0, const int32_t* parents, int B, int N, int H, int dk, int dv,
                               int io_dtype, int state_dtype, float q_scale, void* out, void* node_states,
                               void* workspace, size_t workspace_bytes, int32_t* err, tv_stream_t stream) {
  int st = gdn_common(q, k, v, alpha, beta, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, q_scale,
                      out, err);
  if (st != TV_OK) return st;
  if (!a16(node_states) || !a16(workspace)) return TV_ERR_INVALID_ARG;
  if (workspace_bytes < tv_gdn_fork_workspace_size(B, N, H, dv)) return TV_ERR_INVALID_ARG;
  float* pv = static_cast<float*>(workspace);
  float* lg = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                       (((size_t)B * N * H * dv * 4 + 255) & ~(size_t)255));
  tv::GdnArgs a{q, k, v, alpha, beta, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, q_scale, out, err};
  return cuda_status(tv::launch_gdn_fork_two_pass(a, node_states, pv, lg, stream));
}

int tv_gdn_fork_materialize(const void* k, const float* alpha, const void* S0, const int32_t* parents,
                            const float* pseudo_v, int B, int N, int H, int dk, int dv, int io_dtype,
                            int state_dtype, int max_ctas_per_sm, void* node_states, int32_t* err,
                            tv_stream_t stream) {
  if (!a16(k) || !a4(alpha) || !a16(S0) || !a4(parents) || !a16(pseudo_v) || !a16(node_states) || !a4(err))
    return TV_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || H < 1 || max_ctas_per_sm < 0) return TV_ERR_INVALID_ARG;
  if (N > TV_MAX_NODES || !dim_ok(dk) || !dim_ok(dv)) return TV_ERR_UNSUPPORTED;
  const int st = gdn_dtypes(io_dtype, state_dtype);
  if (st != TV_OK) return st;
  // q, v, beta and out are not read by this pass.
  tv::GdnArgs a{nullptr, k, nullptr, alpha, nullptr, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, 1.f,
                nullptr, err};
  const tv::ForkSelect all{nullptr, 0.f, N, nullptr};
  return cuda_status(tv::launch_gdn_fork_materialize(a, node_states, pseudo_v, all, max_ctas_per_sm, stream));
}

int tv_gdn_fork_materialize_selective(const void* k, const float* alpha, const void* S0, const int32_t* parents,
                                      const float* pseudo_v, const float* confidence, float threshold, int capacity,
                                      int B, int N, int H, int dk, int dv, int io_dtype, int state_dtype,
                                      int max_ctas_per_sm, void* node_states, int32_t* slot, int32_t* err,
                                      tv_stream_t stream) {
  if (!a16(k) || !a4(alpha) || !a16(S0) || !a4(parents) || !a16(pseudo_v) || !a16(node_states) || !a4(err) ||
      !a4(confidence) || !a4(slot))
    return TV_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || H < 1 || max_ctas_per_sm < 0 || !isfinite(threshold) || capacity < 1 || capacity > N)
    return TV_ERR_INVALID_ARG;
  if (N > TV_MAX_NODES || !dim_ok(dk) || !dim_ok(dv)) return TV_ERR_UNSUPPORTED;
  const int st = gdn_dtypes(io_dtype, state_dtype);
  if (st != TV_OK) return st;
  tv::GdnArgs a{nullptr, k, nullptr, alpha, nullptr, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, 1.f,
                nullptr, err};
  const tv::ForkSelect sel{confidence, threshold, capacity, slot};
  return cuda_status(tv::launch_gdn_fork_materialize(a, node_states, pseudo_v, sel, max_ctas_per_sm, stream));
}

int tv_gdn_tree_verify_fork_selective(const void* q, const void* k, const void* v, const float* alpha,
                                      const float* beta, const void* S0, const int32_t* parents,
                                      const float* confidence, float threshold, int capacity, int B, int N,
                                      int H, int dk, int dv, int io_dtype, int state_dtype, float q_scale,
                                      void* out, void* node_states, int32_t* slot, int32_t* err,
                                      tv_stream_t stream) {
  int st = gdn_common(q, k, v, alpha, beta, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, q_scale,
                      out, err);
  if (st != TV_OK) return st;
  if (!a4(confidence) || !a4(slot) || !isfinite(threshold) || capacity < 1 || capacity > N)
    return TV_ERR_INVALID_ARG;
  if (!a16(node_states)) return TV_ERR_INVALID_ARG;
  tv::GdnArgs a{q, k, v, alpha, beta, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, q_scale, out, err};
  const tv::ForkSelect sel{confidence, threshold, capacity, slot};
  return cuda_status(tv::launch_gdn_fork(a, node_states, sel, stream));
}

int tv_gdn_tree_verify_wy(const void* q, const void* k, const void* v, const float* alpha,
                          const float* beta, const void* S0, const int32_t* parents, int B, int N,
                          int H, int dk, int dv, int io_dtype, int state_dtype, float q_scale, void* out,
                          float* pseudo_v, float* log_gamma, int32_t* err, tv_stream_t stream) {
  int st = gdn_common(q, k, v, alpha, beta, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, q_scale,
                      out, err);
  if (st != TV_OK) return st;
  if (!a4(pseudo_v) || !a4(log_gamma)) return TV_ERR_INVALID_ARG;
  tv::GdnArgs a{q, k, v, alpha, beta, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, q_scale, out, err};
  return cuda_status(tv::launch_gdn_wy(a, pseudo_v, log_gamma, stream));
}

int tv_gdn_tree_verify_wy_lazy(const int32_t* prev_path, const int32_t* prev_len, int Lmax,
                               const int32_t* prev_parents, int prev_N, const float* prev_pseudo_v,
                               const float* prev_log_gamma, const void* prev_k, const void* q, const void* k,
                               const void* v, const float* alpha, const float* beta, void* S0,
                               const int32_t* parents, int B, int N, int H, int dk, int dv, int io_dtype,
                               int state_dtype, float q_scale, void* out, float* pseudo_v, float* log_gamma,
                               int32_t* err, tv_stream_t stream) {
  int st = gdn_common(q, k, v, alpha, beta, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, q_scale,
                      out, err);
  if (st != TV_OK) return st;
  if (!a4(pseudo_v) || !a4(log_gamma) || !a4(prev_path) || !a4(prev_len) || !a4(prev_parents) ||
      !a4(prev_pseudo_v) || !a4(prev_log_gamma) || !a16(prev_k) || Lmax < 1 || prev_N < 1)
    return TV_ERR_INVALID_ARG;
  if (prev_N > TV_MAX_NODES) return TV_ERR_UNSUPPORTED;
  tv::GdnArgs a{q, k, v, alpha, beta, S0, parents, B, N, H, dk, dv, io_dtype, state_dtype, q_scale, out, err};
  if (!tv::gdn_wy_tc_supported(a) || !tv::gdn_wy_lazy_fits(N)) return TV_ERR_UNSUPPORTED;
  const tv::WyLazy lz{prev_path, prev_len, Lmax, prev_N, prev_parents, prev_pseudo_v, prev_log_gamma, prev_k};
  return cuda_status(tv::launch_gdn_wy_tc(a, pseudo_v, log_gamma, lz, stream));
}

int tv_gdn_commit_layers(int mode, const int32_t* accepted_path, const int32_t* accepted_len, int Lmax,
                         const int32_t* parents, const void* node_states, const float* pseudo_v,
                         const float* log_gamma, const void* k, void* S0, int layers, int B, int N, int H, int dk,
                         int dv, int io_dtype, int state_dtype, int32_t* err, tv_stream_t stream) {
  if (!a4(accepted_path) || !a4(accepted_len) || !a4(parents) || !a16(S0) || !a4(err)) return TV_ERR_INVALID_ARG;
  if (layers < 1 || B < 1 || N < 1 || H < 1 || Lmax < 1) return TV_ERR_INVALID_ARG;
  if ((long long)layers * B * H > 0x7fffffffLL) return TV_ERR_UNSUPPORTED;
  if (mode == TV_MODE_FORK) {
    if (!a16(node_states)) return TV_ERR_INVALID_ARG;
  } else if (mode == TV_MODE_WY) {
    if (!a4(pseudo_v) || !a4(log_gamma) || !a16(k)) return TV_ERR_INVALID_ARG;
  } else {
    return TV_ERR_INVALID_ARG;
  }
  if (N > TV_MAX_NODES || !dim_ok(dk) || !dim_ok(dv)) return TV_ERR_UNSUPPORTED;
  int st = gdn_dtypes(io_dtype, state_dtype);
  if (st != TV_OK) return st;
  tv::CommitArgs a{mode, accepted_path, accepted_len, Lmax, parents, node_states, pseudo_v, log_gamma, k,
                   S0, B, N, H, dk, dv, io_dtype, state_dtype, err};
  a.layers = layers;
  if (mode == TV_MODE_FORK) a.pseudo_v = nullptr, a.log_gamma = nullptr, a.k = nullptr;
  else a.node_states = nullptr;
  return cuda_status(tv::launch_gdn_commit(a, stream));
}

int tv_gdn_commit(int mode, const int32_t* accepted_path, const int32_t* accepted_len, int Lmax,
                  const int32_t* parents, const void* node_states, const float* pseudo_v,
                  const float* log_gamma, const void* k, void* S0, int B, int N, int H, int dk, int dv,
                  int io_dtype, int state_dtype, int32_t* err, tv_stream_t stream) {
  return tv_gdn_commit_layers(mode, accepted_path, accepted_len, Lmax, parents, node_states, pseudo_v, log_gamma, k,
                              S0, 1, B, N, H, dk, dv, io_dtype, state_dtype, err, stream);
}

int tv_gdn_commit_selective(const int32_t* accepted_path, const int32_t* accepted_len, int Lmax,
                            const int32_t* parents, const void* node_states, const int32_t* slot, int capacity,
                            const void* k, const void* v, const float* alpha, const float* beta, void* S0, int B,
                            int N, int H, int dk, int dv, int io_dtype, int state_dtype, int32_t* err,
                            tv_stream_t stream) {
  if (!a4(accepted_path) || !a4(accepted_len) || !a4(parents) || !a16(S0) || !a4(err) || !a16(node_states) ||
      !a4(slot) || !a16(k) || !a4(v) || !a4(alpha) || !a4(beta))
    return TV_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || H < 1 || Lmax < 1 || capacity < 1 || capacity > N) return TV_ERR_INVALID_ARG;
  if (N > TV_MAX_NODES || !dim_ok(dk) || !dim_ok(dv)) return TV_ERR_UNSUPPORTED;
  int st = gdn_dtypes(io_dtype, state_dtype);
  if (st != TV_OK) return st;
  tv::CommitArgs a{TV_MODE_FORK, accepted_path, accepted_len, Lmax, parents, node_states, nullptr, nullptr, k,
                   S0, B, N, H, dk, dv, io_dtype, state_dtype, err};
  const tv::ReplayArgs r{slot, capacity, v, alpha, beta};
  return cuda_status(tv::launch_gdn_commit_replay(a, r, stream));
}

size_t tv_tree_attn_workspace_size(int B, int N, int Hq, int Hkv, int hd, int max_blocks, int block_size) {
  if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || hd < 1 || max_blocks < 1 || block_size < 1) return 0;
  return tv::attn_workspace_size(B, N, Hq, Hkv, hd, max_blocks, block_size);
}

}  // extern "C"

int tv::tree_attn_check_args(const void* q, const void* k_new, const void* v_new, const void* k_cache,
                             const void* v_cache, int num_blocks, const int32_t* block_table, int max_blocks,
                             const int32_t* prefix_len, const int32_t* parents, int B, int N, int Hq, int Hkv,
                             int hd, int block_size, float rope_theta, float sm_scale, const void* out,
                             const int32_t* err) {
  if (!a16(q) || !a16(k_new) || !a16(v_new) || !a16(k_cache) || !a16(v_cache) || !a4(block_table) ||
      !a4(prefix_len) || !a4(parents) || !a16(out) || !a4(err))
    return TV_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || num_blocks < 1 || max_blocks < 1 ||
      !(rope_theta > 0.f) || !isfinite(rope_theta) || !isfinite(sm_scale))
    return TV_ERR_INVALID_ARG;
  if (N > TV_MAX_NODES || (hd != 64 && hd != 128 && hd != 256) || block_size != TV_BLOCK_SIZE)
    return TV_ERR_UNSUPPORTED;
  if (B > 65535) return TV_ERR_UNSUPPORTED;
  return TV_OK;
}

extern "C" {

int tv_tree_attn(const void* q, const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                 int num_blocks, const int32_t* block_table, int max_blocks, const int32_t* prefix_len,
                 const int32_t* parents, int B, int N, int Hq, int Hkv, int hd, int block_size,
                 float rope_theta, float sm_scale, void* out, void* workspace, size_t workspace_bytes,
                 int32_t* err, tv_stream_t stream) {
  const int st = tv::tree_attn_check_args(q, k_new, v_new, k_cache, v_cache, num_blocks, block_table, max_blocks,
                                          prefix_len, parents, B, N, Hq, Hkv, hd, block_size, rope_theta,
                                          sm_scale, out, err);
  if (st != TV_OK) return st;
  if (!a16(workspace)) return TV_ERR_INVALID_ARG;
  if (workspace_bytes < tv::attn_workspace_size(B, N, Hq, Hkv, hd, max_blocks, block_size))
    return TV_ERR_INVALID_ARG;
  tv::AttnArgs a{q, k_new, v_new, k_cache, v_cache, num_blocks, block_table, max_blocks, prefix_len, parents,
                 B, N, Hq, Hkv, hd, block_size, rope_theta, sm_scale, out, err};
  return cuda_status(tv::launch_tree_attn(a, workspace, workspace_bytes, stream));
}

int tv_kv_compact(void* k_cache, void* v_cache, int num_blocks, const int32_t* block_table, int max_blocks,
                  const int32_t* prefix_len, const int32_t* parents, int N, const int32_t* accepted_path,
                  const int32_t* accepted_len, int Lmax, int B, int Hkv, int hd, int block_size,
                  int32_t* slot_map, int32_t* new_len, int32_t* err, tv_stream_t stream) {
  if (!a16(k_cache) || !a16(v_cache) || !a4(block_table) || !a4(prefix_len) || !a4(parents) ||
      !a4(accepted_path) || !a4(accepted_len) || !a4(slot_map) || !a4(new_len) || !a4(err))
    return TV_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || Hkv < 1 || Lmax < 1 || num_blocks < 1 || max_blocks < 1) return TV_ERR_INVALID_ARG;
  if (N > TV_MAX_NODES || (hd != 64 && hd != 128 && hd != 256) || block_size != TV_BLOCK_SIZE)
    return TV_ERR_UNSUPPORTED;
  tv::CompactArgs a{k_cache, v_cache, num_blocks, block_table, max_blocks, prefix_len, parents, N,
                    accepted_path, accepted_len, Lmax, B, Hkv, hd, block_size, slot_map, new_len, err};
  return cuda_status(tv::launch_kv_compact(a, stream));
}

int tv_kv_compact_remap(void* k_cache, void* v_cache, int num_blocks, const int32_t* block_table,
                        int32_t* block_table_out, int max_blocks, const int32_t* prefix_len,
                        const int32_t* parents, int N, const int32_t* accepted_path,
                        const int32_t* accepted_len, int Lmax, int B, int Hkv, int hd, int block_size,
                        int32_t* slot_map, int32_t* new_len, int32_t* remapped, int32_t* err,
                        tv_stream_t stream) {
  if (!a16(k_cache) || !a16(v_cache) || !a4(block_table) || !a4(block_table_out) || !a4(prefix_len) ||
      !a4(parents) || !a4(accepted_path) || !a4(accepted_len) || !a4(slot_map) || !a4(new_len) ||
      !a4(remapped) || !a4(err))
    return TV_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || Hkv < 1 || Lmax < 1 || num_blocks < 1 || max_blocks < 1) return TV_ERR_INVALID_ARG;
  {
    const uintptr_t in0 = reinterpret_cast<uintptr_t>(block_table);
    const uintptr_t out0 = reinterpret_cast<uintptr_t>(block_table_out);
    const uintptr_t bytes = (uintptr_t)B * (uintptr_t)max_blocks * sizeof(int32_t);
    if (in0 < out0 + bytes && out0 < in0 + bytes) return TV_ERR_INVALID_ARG;
  }
  if (N > TV_MAX_NODES || (hd != 64 && hd != 128 && hd != 256) || block_size != TV_BLOCK_SIZE)
    return TV_ERR_UNSUPPORTED;
  tv::CompactArgs a{k_cache, v_cache, num_blocks, block_table, max_blocks, prefix_len, parents, N,
                    accepted_path, accepted_len, Lmax, B, Hkv, hd, block_size, slot_map, new_len, err,
                    block_table_out, remapped};
  return cuda_status(tv::launch_kv_compact_remap(a, stream));
}

int tv_accept_walk(const int32_t* parents, const int32_t* draft_tokens, const int32_t* target_tokens, int B,
                   int N, int Lmax, int32_t* accepted_path, int32_t* accepted_len, int32_t* next_token,
                   int32_t* err, tv_stream_t stream) {
  if (!a4(parents) || !a4(draft_tokens) || !a4(target_tokens) || !a4(accepted_path) || !a4(accepted_len) ||
      !a4(next_token) || !a4(err))
    return TV_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || Lmax < 1) return TV_ERR_INVALID_ARG;
  if (N > TV_MAX_NODES) return TV_ERR_UNSUPPORTED;
  tv::AcceptArgs a{parents, draft_tokens, target_tokens, B, N, Lmax, accepted_path, accepted_len, next_token, err};
  return cuda_status(tv::launch_accept_walk(a, stream));
}

size_t tv_linear_attn_workspace_size(int B, int T, int max_len, int H, int dk, int dv, int io_dtype) {
  if (B < 1 || T < 0 || max_len < 0 || H < 1 || !dim_ok(dk) || !dim_ok(dv)) return 0;
  return tv::linear_attn_workspace_size(B, T, max_len, H, dk, dv, io_dtype);
}

}  // extern "C"

namespace {

// Types, sizes and the token strides shared by the prompt and the single-token call.
int linear_attn_common(int64_t q_stride, int64_t k_stride, int64_t v_stride, int64_t alpha_stride, int64_t out_stride,
                       int Hk, int H, int dk, int dv, int io, int state, float q_scale) {
  if (Hk < 1 || H < 1 || H % Hk || !isfinite(q_scale)) return TV_ERR_INVALID_ARG;
  if (!dim_ok(dk) || !dim_ok(dv)) return TV_ERR_UNSUPPORTED;
  const int st = gdn_dtypes(io, state);
  if (st != TV_OK) return st;
  const int64_t per16 = io == TV_BF16 ? 8 : 4, qk = (int64_t)Hk * dk, vo = (int64_t)H * dv;
  if (q_stride < qk || k_stride < qk || v_stride < vo || out_stride < vo || q_stride % per16 || k_stride % per16 ||
      v_stride % per16 || out_stride % per16 || (alpha_stride != 0 && alpha_stride < H))
    return TV_ERR_INVALID_ARG;
  return TV_OK;
}

}  // namespace

extern "C" {

int tv_linear_attn_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                          int64_t v_stride, const float* alpha, int64_t alpha_stride, const void* S0,
                          const int32_t* cu_seqlens, int B, int T, int max_len, int Hk, int H, int dk, int dv,
                          int io_dtype, int state_dtype, float q_scale, void* out, int64_t out_stride, void* S,
                          void* workspace, size_t workspace_bytes, int32_t* err, tv_stream_t stream) {
  // With no token at all (T = 0) the token tensors may be null.
  if (T > 0 && (!a16(q) || !a16(k) || !a16(v) || !a4(alpha) || !a16(out))) return TV_ERR_INVALID_ARG;
  if ((S0 != nullptr && !a16(S0)) || !a16(S) || !a4(cu_seqlens) || !a4(err) || B < 1 || T < 0 || max_len < 0)
    return TV_ERR_INVALID_ARG;
  const int st = linear_attn_common(q_stride, k_stride, v_stride, alpha_stride, out_stride, Hk, H, dk, dv, io_dtype,
                                    state_dtype, q_scale);
  if (st != TV_OK) return st;
  if ((long long)B * H > (1 << 24)) return TV_ERR_UNSUPPORTED;
  if (max_len > T) max_len = T;
  const size_t need = tv::linear_attn_workspace_size(B, T, max_len, H, dk, dv, io_dtype);
  if (need > 0 && (!a16(workspace) || workspace_bytes < need)) return TV_ERR_INVALID_ARG;
  tv::LinAttnArgs a{q, k, v, q_stride, k_stride, v_stride, alpha, alpha_stride, S0, cu_seqlens,
                    B, T, max_len, Hk, H, dk, dv, io_dtype, state_dtype, q_scale, out, out_stride, S, err,
                    0, nullptr, nullptr};
  if (need > 0) {
    a.seg_len = tv::linear_attn_segment(B, T, max_len, H, dk, dv, io_dtype);
    const size_t segments = (size_t)B + T / a.seg_len;
    a.slots = static_cast<float*>(workspace);
    a.decay = reinterpret_cast<float2*>(a.slots + segments * H * dv * dk);
  }
  return cuda_status(tv::launch_linear_attn_prompt(a, stream));
}

int tv_linear_attn_step(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                        int64_t v_stride, const float* alpha, int64_t alpha_stride, const int32_t* live, int B, int Hk,
                        int H, int dk, int dv, int io_dtype, int state_dtype, float q_scale, void* out,
                        int64_t out_stride, void* S, tv_stream_t stream) {
  if (!a16(q) || !a16(k) || !a16(v) || !a4(alpha) || !a16(out) || !a16(S) || (live != nullptr && !a4(live)) || B < 1)
    return TV_ERR_INVALID_ARG;
  const int st = linear_attn_common(q_stride, k_stride, v_stride, alpha_stride, out_stride, Hk, H, dk, dv, io_dtype,
                                    state_dtype, q_scale);
  if (st != TV_OK) return st;
  if ((long long)B * H > (1 << 24)) return TV_ERR_UNSUPPORTED;
  tv::LinStepArgs a{q, k, v, q_stride, k_stride, v_stride, alpha, alpha_stride, live, B, Hk, H, dk, dv,
                    io_dtype, state_dtype, q_scale, out, out_stride, S};
  return cuda_status(tv::launch_linear_attn_step(a, stream));
}

}  // extern "C"

namespace {

constexpr int kNormMax = 32768;  // widest row: five 8-column vectors for each of 832 threads, at any offset

bool el(const void* p, int dtype) {  // aligned to its element
  return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (dtype == TV_F32 ? 3u : 1u)) == 0;
}

}  // namespace

extern "C" {

int tv_gated_rmsnorm(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, const void* weight,
                     int rows, int H, int d, int io_dtype, float eps, float weight_offset, int gate_first, void* out,
                     int64_t out_stride, tv_stream_t stream) {
  if (io_dtype != TV_F32 && io_dtype != TV_BF16) return TV_ERR_INVALID_ARG;
  if (rows < 0 || H < 1 || d < 1 || !(eps >= 0.f) || !isfinite(eps) || !isfinite(weight_offset) || gate_first < 0 ||
      gate_first > 1)
    return TV_ERR_INVALID_ARG;
  // Row numbers are ints, and the last block counts up to 31 past the last one.
  if (d > kNormMax || (long long)rows * H > 0x7fffff00LL) return TV_ERR_UNSUPPORTED;
  if (rows == 0) return TV_OK;
  const int64_t row = (int64_t)H * d;
  if (!el(x, io_dtype) || !el(out, io_dtype) || (gate != nullptr && !el(gate, io_dtype)) ||
      (weight != nullptr && !el(weight, io_dtype)) || x_stride < row || out_stride < row ||
      (gate != nullptr && gate_stride < row))
    return TV_ERR_INVALID_ARG;
  tv::GatedNormArgs a{x, gate, weight, out, x_stride, gate_stride, out_stride, rows, H, d, io_dtype, eps,
                      weight_offset, gate_first};
  return cuda_status(tv::launch_gated_rmsnorm(a, stream));
}

int tv_residual_rmsnorm(const void* y, int64_t y_stride, const void* residual, int64_t residual_stride,
                        const void* post_weight, const void* gate, int64_t gate_stride, float scale,
                        const void* weight, int rows, int D, int io_dtype, int residual_dtype, float eps,
                        float weight_offset, void* residual_out, int64_t residual_out_stride, void* out,
                        int64_t out_stride, tv_stream_t stream) {
  const int st = gdn_dtypes(io_dtype, residual_dtype);
  if (st != TV_OK) return st;
  if (rows < 0 || D < 1 || !(eps >= 0.f) || !isfinite(eps) || !isfinite(weight_offset) || !isfinite(scale))
    return TV_ERR_INVALID_ARG;
  if (D > kNormMax) return TV_ERR_UNSUPPORTED;
  if (rows == 0) return TV_OK;
  if (!el(y, io_dtype) || !el(residual, residual_dtype) || !el(residual_out, residual_dtype) ||
      (post_weight != nullptr && !el(post_weight, io_dtype)) || (gate != nullptr && !el(gate, io_dtype)) ||
      (weight != nullptr && !el(weight, io_dtype)) || (out != nullptr && !el(out, io_dtype)) || y_stride < D ||
      residual_stride < D || residual_out_stride < D || (gate != nullptr && gate_stride < D) ||
      (out != nullptr && out_stride < D))
    return TV_ERR_INVALID_ARG;
  tv::ResidualNormArgs a{y, residual, post_weight, gate, weight, residual_out, out, y_stride, residual_stride,
                         gate_stride, residual_out_stride, out_stride, rows, D, io_dtype, residual_dtype, scale, eps,
                         weight_offset};
  return cuda_status(tv::launch_residual_rmsnorm(a, stream));
}

}  // extern "C"

namespace {

// Sizes and the row strides shared by the calls over a paged cache of 16-token blocks; rows in whole 16 bytes.
bool rows_ok(int64_t stride, int64_t row, int dtype) {
  return stride >= row && stride % (dtype == TV_BF16 ? 8 : 4) == 0;
}
bool head_ok(int hd) { return hd == 64 || hd == 128 || hd == 256; }

int window_attn_common(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache, int num_blocks,
                       const int32_t* block_table, int max_blocks, const int32_t* prefix_len, int B, int Hq, int Hkv,
                       int hd, int block_size, int window, int sinks, float sm_scale, const void* out,
                       int64_t out_stride, const int32_t* err) {
  if (!a16(q) || !a16(k_cache) || !a16(v_cache) || !a4(block_table) || !a4(prefix_len) || !a16(out) || !a4(err))
    return TV_ERR_INVALID_ARG;
  if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv || num_blocks < 1 || max_blocks < 1 || window < 0 || sinks < 0 ||
      !isfinite(sm_scale))
    return TV_ERR_INVALID_ARG;
  if (!head_ok(hd) || block_size != TV_BLOCK_SIZE || Hq / Hkv > 128 || max_blocks > (1 << 26)) return TV_ERR_UNSUPPORTED;
  if (Hq > (1 << 16) || (long long)B * Hkv > (1 << 24) || (long long)num_blocks * Hkv > (1 << 29))
    return TV_ERR_UNSUPPORTED;
  if (!rows_ok(q_stride, (int64_t)Hq * hd, TV_BF16) || !rows_ok(out_stride, (int64_t)Hq * hd, TV_BF16))
    return TV_ERR_INVALID_ARG;
  return TV_OK;
}

}  // namespace

extern "C" {

int tv_qk_norm_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                    const void* q_weight, const void* k_weight, const int32_t* cu_seqlens, const int32_t* prefix_len,
                    const int32_t* live, int B, int T, int Hq, int Hkv, int hd, int rotary_dim, int io_dtype, int norm,
                    float eps, float weight_offset, float rope_theta, void* q_out, int64_t q_out_stride, void* k_out,
                    int64_t k_out_stride, void* k_cache, void* v_cache, int num_blocks, const int32_t* block_table,
                    int max_blocks, int block_size, int32_t* err, tv_stream_t stream) {
  const bool cache = k_cache != nullptr || v_cache != nullptr;
  if (io_dtype != TV_F32 && io_dtype != TV_BF16) return TV_ERR_INVALID_ARG;
  if (B < 1 || T < 0 || Hq < 1 || Hkv < 1 || norm < 0 || norm > 1 || !(eps >= 0.f) || !isfinite(eps) ||
      !isfinite(weight_offset) || rotary_dim < 0 || rotary_dim > hd ||
      (rotary_dim > 0 && (!(rope_theta >= 1.f) || !isfinite(rope_theta))) || (cu_seqlens == nullptr && T != B))
    return TV_ERR_INVALID_ARG;
  if (!head_ok(hd) || rotary_dim % 16 || Hq > (1 << 16) || Hkv > (1 << 16)) return TV_ERR_UNSUPPORTED;
  if (cache && (block_size != TV_BLOCK_SIZE || io_dtype != TV_BF16 || max_blocks > (1 << 26))) return TV_ERR_UNSUPPORTED;
  if ((cu_seqlens != nullptr && !a4(cu_seqlens)) || (prefix_len != nullptr && !a4(prefix_len)) ||
      (live != nullptr && !a4(live)) || (q_weight != nullptr && !a16(q_weight)) ||
      (k_weight != nullptr && !a16(k_weight)) || !a4(err))
    return TV_ERR_INVALID_ARG;
  if (cache && (!a16(k_cache) || !a16(v_cache) || !a4(block_table) || prefix_len == nullptr || num_blocks < 1 ||
                max_blocks < 1))
    return TV_ERR_INVALID_ARG;
  if (!cache && k_out == nullptr) return TV_ERR_INVALID_ARG;
  const int64_t qrow = (int64_t)Hq * hd, krow = (int64_t)Hkv * hd;
  // With no token at all (T = 0) the token tensors may be null.
  if (T > 0 && (!a16(q) || !a16(k) || !a16(q_out) || (cache && !a16(v)) || (k_out != nullptr && !a16(k_out))))
    return TV_ERR_INVALID_ARG;
  if (!rows_ok(q_stride, qrow, io_dtype) || !rows_ok(k_stride, krow, io_dtype) ||
      !rows_ok(q_out_stride, qrow, io_dtype) || (cache && !rows_ok(v_stride, krow, io_dtype)) ||
      (k_out != nullptr && !rows_ok(k_out_stride, krow, io_dtype)))
    return TV_ERR_INVALID_ARG;
  tv::QkRopeArgs a{q, k, v, q_stride, k_stride, v_stride, q_weight, k_weight, cu_seqlens, prefix_len, live,
                   B, T, Hq, Hkv, hd, rotary_dim, io_dtype, norm, eps, weight_offset, rope_theta,
                   q_out, k_out, q_out_stride, k_out_stride, k_cache, v_cache, num_blocks, block_table, max_blocks, err};
  return cuda_status(tv::launch_qk_norm_rope(a, stream));
}

size_t tv_window_attn_workspace_size(int B, int T, int max_len, int Hq, int Hkv, int hd, int max_blocks,
                                     int block_size, int window, int sinks) {
  if (B < 1 || T < 0 || max_len < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || !head_ok(hd) || max_blocks < 1 ||
      max_blocks > (1 << 26) || block_size != TV_BLOCK_SIZE || window < 0 || sinks < 0 || Hq / Hkv > 128)
    return 0;
  return tv::window_attn_workspace_size(B, T, max_len < T ? max_len : T, Hq, Hkv, hd, max_blocks, window, sinks);
}

int tv_window_attn_prompt(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache, int num_blocks,
                          const int32_t* block_table, int max_blocks, const int32_t* cu_seqlens,
                          const int32_t* prefix_len, int B, int T, int max_len, int Hq, int Hkv, int hd,
                          int block_size, int window, int sinks, float sm_scale, void* out, int64_t out_stride,
                          void* workspace, size_t workspace_bytes, int32_t* err, tv_stream_t stream) {
  if (T < 0 || max_len < 0 || !a4(cu_seqlens)) return TV_ERR_INVALID_ARG;
  // With no token at all (T = 0) the token tensors may be null.
  const int st = window_attn_common(T > 0 ? q : k_cache, q_stride, k_cache, v_cache, num_blocks, block_table,
                                    max_blocks, prefix_len, B, Hq, Hkv, hd, block_size, window, sinks, sm_scale,
                                    T > 0 ? out : k_cache, out_stride, err);
  if (st != TV_OK) return st;
  if (max_len > T) max_len = T;
  const size_t need = tv::window_attn_workspace_size(B, T, max_len, Hq, Hkv, hd, max_blocks, window, sinks);
  if (need > 0 && (!a16(workspace) || workspace_bytes < need)) return TV_ERR_INVALID_ARG;
  tv::WinAttnArgs a{q, q_stride, k_cache, v_cache, num_blocks, block_table, max_blocks, cu_seqlens, prefix_len, nullptr,
                    B, T, max_len, Hq, Hkv, hd, window, sinks, sm_scale, out, out_stride, err};
  return cuda_status(tv::launch_window_attn(a, workspace, stream));
}

int tv_window_attn_step(const void* q, int64_t q_stride, const void* k_cache, const void* v_cache, int num_blocks,
                        const int32_t* block_table, int max_blocks, const int32_t* prefix_len, const int32_t* live,
                        int B, int Hq, int Hkv, int hd, int block_size, int window, int sinks, float sm_scale,
                        void* out, int64_t out_stride, void* workspace, size_t workspace_bytes, int32_t* err,
                        tv_stream_t stream) {
  if (live != nullptr && !a4(live)) return TV_ERR_INVALID_ARG;
  const int st = window_attn_common(q, q_stride, k_cache, v_cache, num_blocks, block_table, max_blocks, prefix_len, B,
                                    Hq, Hkv, hd, block_size, window, sinks, sm_scale, out, out_stride, err);
  if (st != TV_OK) return st;
  const size_t need = tv::window_attn_workspace_size(B, B, 1, Hq, Hkv, hd, max_blocks, window, sinks);
  if (need > 0 && (!a16(workspace) || workspace_bytes < need)) return TV_ERR_INVALID_ARG;
  tv::WinAttnArgs a{q, q_stride, k_cache, v_cache, num_blocks, block_table, max_blocks, nullptr, prefix_len, live,
                    B, B, 1, Hq, Hkv, hd, window, sinks, sm_scale, out, out_stride, err};
  return cuda_status(tv::launch_window_attn(a, workspace, stream));
}

int tv_accept_sample(const int32_t* parents, const int32_t* draft_tokens, const void* target_probs,
                     const void* draft_probs, const float* uniforms, int B, int N, int V, int Lmax, int probs_dtype,
                     int32_t* accepted_path, int32_t* accepted_len, int32_t* next_token, int32_t* err,
                     tv_stream_t stream) {
  if (probs_dtype != TV_F32 && probs_dtype != TV_BF16) return TV_ERR_INVALID_ARG;
  if (!a4(parents) || !a4(draft_tokens) || !a16(target_probs) || (draft_probs != nullptr && !a16(draft_probs)) ||
      !a4(uniforms) || !a4(accepted_path) || !a4(accepted_len) || !a4(next_token) || !a4(err))
    return TV_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || V < 1 || Lmax < 1) return TV_ERR_INVALID_ARG;
  if (N > TV_MAX_NODES || V > (1 << 24) || B > (1 << 24)) return TV_ERR_UNSUPPORTED;
  tv::SampleArgs a{parents, draft_tokens, target_probs, draft_probs, uniforms, B, N, V, Lmax, probs_dtype,
                   accepted_path, accepted_len, next_token, err};
  return cuda_status(tv::launch_accept_sample(a, stream));
}

}  // extern "C"
