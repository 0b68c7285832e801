"""Python binding of the CUDA library ``_lib/libtv.so`` (argument marshalling only).

Every function has the name of the C entry point it calls (``include/tv.h``), takes torch
tensors that live on the GPU, and passes their data pointers, sizes and dtype codes.  All of
the work runs in the library's kernels; there is no CPU fallback.  Importing this package
raises ``ImportError`` when the library has not been built
(``python tree_speculative_verification_gdn_gb300/_build.py``).

Non-OK return codes raise :class:`TVError`.  Per-sequence, data-dependent errors land in the
caller's ``err`` tensor (read it after synchronising).
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libtv.so")

# Status codes and enums of include/tv.h.
TV_OK = 0
TV_ERR_INVALID_ARG = -1
TV_ERR_BAD_TREE = -2
TV_ERR_BAD_PATH = -3
TV_ERR_UNSUPPORTED = -4
TV_ERR_CUDA = -5
TV_ERR_TIMEOUT = -6
TV_ERR_CAPACITY = -7
TV_ERR_BAD_BLOCK = -8
TV_ERR_SCRATCH = -9
TV_ERR_BAD_SEQLEN = -10
TV_ERR_BAD_PROBS = -11
TV_F32 = 0
TV_BF16 = 1
TV_MODE_FORK = 0
TV_MODE_WY = 1
TV_MAX_NODES = 256
TV_BLOCK_SIZE = 16
TV_STATIC_SCRATCH_BYTES = 64 << 20

EXPORTED = ("tv_status_string", "tv_last_cuda_error", "tv_version", "tv_tree_prepare",
            "tv_gdn_tree_verify_fork", "tv_gdn_tree_verify_wy", "tv_gdn_commit",
            "tv_tree_attn_workspace_size", "tv_tree_attn", "tv_tree_attn_static", "tv_kv_compact",
            "tv_accept_walk", "tv_gdn_tree_verify_fork_selective", "tv_gdn_commit_selective",
            "tv_gdn_tree_verify_wy_lazy", "tv_gdn_fork_workspace_size", "tv_gdn_tree_verify_fork_ws",
            "tv_gdn_fork_materialize", "tv_gdn_fork_materialize_selective", "tv_gdn_commit_layers",
            "tv_kv_compact_remap", "tv_linear_attn_workspace_size", "tv_linear_attn_prompt",
            "tv_linear_attn_step", "tv_gated_rmsnorm", "tv_residual_rmsnorm", "tv_qk_norm_rope",
            "tv_window_attn_workspace_size", "tv_window_attn_prompt", "tv_window_attn_step", "tv_accept_sample",
            "tv_test_bounded_wait")

_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_Z = ctypes.c_size_t
_L = ctypes.c_int64

_SIGNATURES = {
    "tv_status_string": (ctypes.c_char_p, [_I]),
    "tv_last_cuda_error": (_I, []),
    "tv_version": (_I, []),
    "tv_tree_prepare": (_I, [_P, _I, _I, _P, _P, _P, _I, _P, _P, _P]),
    "tv_gdn_tree_verify_fork": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P]),
    "tv_gdn_tree_verify_wy": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _P, _P]),
    "tv_gdn_commit": (_I, [_I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _P, _P]),
    "tv_gdn_commit_layers": (_I, [_I, _P, _P, _I, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P]),
    "tv_tree_attn_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I]),
    "tv_tree_attn": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _P, _P, _Z,
                          _P, _P]),
    "tv_tree_attn_static": (_I, [_P, _P, _P, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _P,
                                 _P, _P]),
    "tv_gdn_tree_verify_fork_selective": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _I, _I,
                                              _F, _P, _P, _P, _P, _P]),
    "tv_gdn_commit_selective": (_I, [_P, _P, _I, _P, _P, _P, _I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I,
                                    _P, _P]),
    "tv_gdn_tree_verify_wy_lazy": (_I, [_P, _P, _I, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I,
                                       _I, _I, _I, _F, _P, _P, _P, _P, _P]),
    "tv_gdn_fork_workspace_size": (_Z, [_I, _I, _I, _I]),
    "tv_gdn_tree_verify_fork_ws": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _P, _Z,
                                       _P, _P]),
    "tv_gdn_fork_materialize": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    "tv_gdn_fork_materialize_selective": (_I, [_P, _P, _P, _P, _P, _P, _F, _I, _I, _I, _I, _I, _I, _I, _I, _I,
                                               _P, _P, _P, _P]),
    "tv_accept_walk": (_I, [_P, _P, _P, _I, _I, _I, _P, _P, _P, _P, _P]),
    "tv_kv_compact": (_I, [_P, _P, _I, _P, _I, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P]),
    "tv_kv_compact_remap": (_I, [_P, _P, _I, _P, _P, _I, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                                 _P]),
    "tv_linear_attn_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I]),
    "tv_linear_attn_prompt": (_I, [_P, _L, _P, _L, _P, _L, _P, _L, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F,
                                   _P, _L, _P, _P, _Z, _P, _P]),
    "tv_linear_attn_step": (_I, [_P, _L, _P, _L, _P, _L, _P, _L, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _L, _P,
                                 _P]),
    "tv_gated_rmsnorm": (_I, [_P, _L, _P, _L, _P, _I, _I, _I, _I, _F, _F, _I, _P, _L, _P]),
    "tv_residual_rmsnorm": (_I, [_P, _L, _P, _L, _P, _P, _L, _F, _P, _I, _I, _I, _I, _F, _F, _P, _L, _P, _L, _P]),
    "tv_qk_norm_rope": (_I, [_P, _L, _P, _L, _P, _L, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _F, _F, _P,
                             _L, _P, _L, _P, _P, _I, _P, _I, _I, _P, _P]),
    "tv_window_attn_workspace_size": (_Z, [_I, _I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "tv_window_attn_prompt": (_I, [_P, _L, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _L,
                                   _P, _Z, _P, _P]),
    "tv_window_attn_step": (_I, [_P, _L, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _L, _P, _Z, _P,
                                 _P]),
    "tv_accept_sample": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "tv_test_bounded_wait": (_I, [ctypes.c_uint, _I, _P, _P, _P]),
}


class TVError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.tv_status_string(status).decode()
        if status == TV_ERR_CUDA:
            msg += f" (cudaError {lib.tv_last_cuda_error()})"
        super().__init__(f"{where}: {msg} [{status}]")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it first with "
                          "python tree_speculative_verification_gdn_gb300/_build.py or "
                          "__graft_entry__.build()")
    handle = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(handle, name)
        fn.restype = res
        fn.argtypes = args
    return handle


lib = _load()

_DTYPES = {torch.float32: TV_F32, torch.bfloat16: TV_BF16}


def _ptr(t):
    if t is None:
        return None
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("tensors passed to the library must be contiguous CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _refuse(name: str, t, shape, dtype):
    if not t.is_cuda:
        raise ValueError("tensors passed to the library must be CUDA tensors")
    raise ValueError(f"{name}: expected {tuple(shape)} {dtype}, got {tuple(t.shape)} {t.dtype}")


def _whole(name: str, t, shape, dtype):
    """Pointer of a dense tensor.  The library sees pointers and sizes only: a tensor of another
    shape or type is caught here."""
    if t is None:
        return None
    if t.shape != shape or t.dtype != dtype or not t.is_cuda:
        _refuse(name, t, shape, dtype)
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous CUDA tensors")
    return t.data_ptr()


def _rows(name: str, t, shape, dtype, row: int):
    """Pointer and row stride (elements) of a tensor whose rows -- everything past the first
    dimension, ``row`` elements -- are dense; the rows themselves may lie apart, as in a slice of a
    projection."""
    if t is None:
        return None, row
    if t.shape != shape or t.dtype != dtype or not t.is_cuda:
        _refuse(name, t, shape, dtype)
    if t.is_contiguous():
        return t.data_ptr(), row
    dense = 1
    for n, stride in zip(reversed(t.shape[1:]), reversed(t.stride()[1:])):
        if n != 1 and stride != dense:
            raise ValueError("the rows of tensors passed to the library must be dense")
        dense *= n
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else row


# The current device without torch's check that CUDA is up (it is, where a tensor lies on it).
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
# The current stream's handle without building a Stream object (3 us of a small call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, where: str) -> None:
    if status != TV_OK:
        raise TVError(status, where)


def status_string(status: int) -> str:
    return lib.tv_status_string(status).decode()


def tv_tree_prepare(parents, depth, mask_bits, err, paths=None, max_depth=None, stream=None) -> None:
    """parents [B,N] int32 -> depth [B,N] int32, mask_bits [B,N,ceil(N/32)] int32 (bit pattern
    of uint32 words), err [B] int32; optionally paths [B,N,cap] int32 (root-to-node, -1 padded)
    and max_depth [B] int32."""
    B, N = parents.shape
    cap = paths.shape[-1] if paths is not None else 0
    _check(lib.tv_tree_prepare(_ptr(parents), B, N, _ptr(depth), _ptr(mask_bits), _ptr(paths), cap,
                               _ptr(max_depth), _ptr(err), _stream(stream)), "tv_tree_prepare")


def tv_gdn_tree_verify_fork(q, k, v, alpha, beta, S0, parents, out, node_states, err,
                            q_scale: float = 1.0, stream=None) -> None:
    B, N, H, dk = q.shape
    dv = v.shape[-1]
    _check(lib.tv_gdn_tree_verify_fork(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0), _ptr(parents), B, N, H, dk, dv,
        _DTYPES[q.dtype], _DTYPES[S0.dtype], float(q_scale), _ptr(out), _ptr(node_states), _ptr(err),
        _stream(stream)), "tv_gdn_tree_verify_fork")


def tv_gdn_fork_workspace_size(B, N, H, dv) -> int:
    return int(lib.tv_gdn_fork_workspace_size(B, N, H, dv))


def tv_gdn_tree_verify_fork_ws(q, k, v, alpha, beta, S0, parents, out, node_states, workspace, err,
                               q_scale: float = 1.0, stream=None) -> None:
    """Fork mode in two passes (TreeWY outputs and w, then the snapshots) with a workspace."""
    B, N, H, dk = q.shape
    dv = v.shape[-1]
    _check(lib.tv_gdn_tree_verify_fork_ws(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0), _ptr(parents), B, N, H, dk, dv,
        _DTYPES[q.dtype], _DTYPES[S0.dtype], float(q_scale), _ptr(out), _ptr(node_states), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(err), _stream(stream)), "tv_gdn_tree_verify_fork_ws")


def tv_gdn_fork_materialize(k, alpha, S0, parents, pseudo_v, node_states, err, max_ctas_per_sm: int = 0,
                            stream=None) -> None:
    """Every fork-mode snapshot from the w of a preceding tv_gdn_tree_verify_wy (same inputs)."""
    B, N, H, dk = k.shape
    dv = pseudo_v.shape[-1]
    _check(lib.tv_gdn_fork_materialize(
        _ptr(k), _ptr(alpha), _ptr(S0), _ptr(parents), _ptr(pseudo_v), B, N, H, dk, dv, _DTYPES[k.dtype],
        _DTYPES[S0.dtype], int(max_ctas_per_sm), _ptr(node_states), _ptr(err), _stream(stream)),
        "tv_gdn_fork_materialize")


def tv_gdn_fork_materialize_selective(k, alpha, S0, parents, pseudo_v, confidence, threshold: float, node_states,
                                      slot, err, max_ctas_per_sm: int = 0, stream=None) -> None:
    """The selected fork-mode snapshots (confidence <= threshold) from the w of a preceding
    tv_gdn_tree_verify_wy: node_states [B, capacity, H, dv, dk], slot [B, N] int32."""
    B, N, H, dk = k.shape
    dv = pseudo_v.shape[-1]
    _check(lib.tv_gdn_fork_materialize_selective(
        _ptr(k), _ptr(alpha), _ptr(S0), _ptr(parents), _ptr(pseudo_v), _ptr(confidence), float(threshold),
        node_states.shape[1], B, N, H, dk, dv, _DTYPES[k.dtype], _DTYPES[S0.dtype], int(max_ctas_per_sm),
        _ptr(node_states), _ptr(slot), _ptr(err), _stream(stream)), "tv_gdn_fork_materialize_selective")


def tv_gdn_tree_verify_fork_selective(q, k, v, alpha, beta, S0, parents, confidence, threshold: float, out,
                                      node_states, slot, err, q_scale: float = 1.0, stream=None) -> None:
    """Fork mode keeping snapshots only of nodes with confidence <= threshold: node_states
    [B, capacity, H, dv, dk] (capacity = node_states.shape[1]), slot [B, N] int32."""
    B, N, H, dk = q.shape
    dv = v.shape[-1]
    _check(lib.tv_gdn_tree_verify_fork_selective(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0), _ptr(parents), _ptr(confidence),
        float(threshold), node_states.shape[1], B, N, H, dk, dv, _DTYPES[q.dtype], _DTYPES[S0.dtype],
        float(q_scale), _ptr(out), _ptr(node_states), _ptr(slot), _ptr(err), _stream(stream)),
        "tv_gdn_tree_verify_fork_selective")


def tv_gdn_commit_selective(accepted_path, accepted_len, parents, node_states, slot, k, v, alpha, beta, S0, err,
                            stream=None) -> None:
    """Commit after tv_gdn_tree_verify_fork_selective (replays from the deepest kept snapshot)."""
    B, H, dv, dk = S0.shape
    N = parents.shape[1]
    _check(lib.tv_gdn_commit_selective(
        _ptr(accepted_path), _ptr(accepted_len), accepted_path.shape[1], _ptr(parents), _ptr(node_states),
        _ptr(slot), node_states.shape[1], _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0), B, N, H, dk, dv,
        _DTYPES[k.dtype], _DTYPES[S0.dtype], _ptr(err), _stream(stream)), "tv_gdn_commit_selective")


def tv_gdn_tree_verify_wy_lazy(prev_path, prev_len, prev_parents, prev_pseudo_v, prev_log_gamma, prev_k,
                               q, k, v, alpha, beta, S0, parents, out, pseudo_v, log_gamma, err,
                               q_scale: float = 1.0, stream=None) -> None:
    """The previous round's TreeWY commit applied to S0 (in place) inside this round's verify."""
    B, N, H, dk = q.shape
    dv = v.shape[-1]
    _check(lib.tv_gdn_tree_verify_wy_lazy(
        _ptr(prev_path), _ptr(prev_len), prev_path.shape[1], _ptr(prev_parents), prev_parents.shape[1],
        _ptr(prev_pseudo_v), _ptr(prev_log_gamma), _ptr(prev_k), _ptr(q), _ptr(k), _ptr(v), _ptr(alpha),
        _ptr(beta), _ptr(S0), _ptr(parents), B, N, H, dk, dv, _DTYPES[q.dtype], _DTYPES[S0.dtype],
        float(q_scale), _ptr(out), _ptr(pseudo_v), _ptr(log_gamma), _ptr(err), _stream(stream)),
        "tv_gdn_tree_verify_wy_lazy")


def tv_gdn_tree_verify_wy(q, k, v, alpha, beta, S0, parents, out, pseudo_v, log_gamma, err,
                          q_scale: float = 1.0, stream=None) -> None:
    B, N, H, dk = q.shape
    dv = v.shape[-1]
    _check(lib.tv_gdn_tree_verify_wy(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(S0), _ptr(parents), B, N, H, dk, dv,
        _DTYPES[q.dtype], _DTYPES[S0.dtype], float(q_scale), _ptr(out), _ptr(pseudo_v), _ptr(log_gamma),
        _ptr(err), _stream(stream)), "tv_gdn_tree_verify_wy")


def tv_gdn_commit(mode: int, accepted_path, accepted_len, parents, S0, err, *, node_states=None,
                  pseudo_v=None, log_gamma=None, k=None, io_dtype=None, N=None, stream=None) -> None:
    """Fork mode reads ``node_states``; WY mode reads ``pseudo_v``, ``log_gamma`` and ``k``."""
    B, H, dv, dk = S0.shape
    Lmax = accepted_path.shape[1]
    N = parents.shape[1] if N is None else N
    io = _DTYPES[k.dtype] if k is not None else (_DTYPES[io_dtype] if io_dtype is not None else
                                                  _DTYPES[S0.dtype])
    _check(lib.tv_gdn_commit(
        int(mode), _ptr(accepted_path), _ptr(accepted_len), Lmax, _ptr(parents), _ptr(node_states),
        _ptr(pseudo_v), _ptr(log_gamma), _ptr(k), _ptr(S0), B, N, H, dk, dv, io, _DTYPES[S0.dtype],
        _ptr(err), _stream(stream)), "tv_gdn_commit")


def tv_gdn_commit_layers(mode: int, accepted_path, accepted_len, parents, S0, err, *, node_states=None,
                         pseudo_v=None, log_gamma=None, k=None, io_dtype=None, N=None, stream=None) -> None:
    """One launch commits every layer: S0 [layers, B, H, dv, dk] and the mode's per-layer tensors
    with a leading layer dimension; path, lengths, parents and err are shared by the layers."""
    layers, B, H, dv, dk = S0.shape
    Lmax = accepted_path.shape[1]
    N = parents.shape[1] if N is None else N
    io = _DTYPES[k.dtype] if k is not None else (_DTYPES[io_dtype] if io_dtype is not None else
                                                  _DTYPES[S0.dtype])
    _check(lib.tv_gdn_commit_layers(
        int(mode), _ptr(accepted_path), _ptr(accepted_len), Lmax, _ptr(parents), _ptr(node_states),
        _ptr(pseudo_v), _ptr(log_gamma), _ptr(k), _ptr(S0), layers, B, N, H, dk, dv, io, _DTYPES[S0.dtype],
        _ptr(err), _stream(stream)), "tv_gdn_commit_layers")


def tv_tree_attn_workspace_size(B, N, Hq, Hkv, hd, max_blocks, block_size=TV_BLOCK_SIZE) -> int:
    return int(lib.tv_tree_attn_workspace_size(B, N, Hq, Hkv, hd, max_blocks, block_size))


def tv_tree_attn(q, k_new, v_new, k_cache, v_cache, block_table, prefix_len, parents, out,
                 workspace, err, rope_theta: float, sm_scale: float | None = None, stream=None) -> None:
    B, N, Hq, hd = q.shape
    Hkv = k_new.shape[2]
    num_blocks, _, bs, _ = k_cache.shape
    max_blocks = block_table.shape[1]
    scale = hd ** -0.5 if sm_scale is None else sm_scale
    _check(lib.tv_tree_attn(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), num_blocks, _ptr(block_table),
        max_blocks, _ptr(prefix_len), _ptr(parents), B, N, Hq, Hkv, hd, bs, float(rope_theta), float(scale),
        _ptr(out), _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err),
        _stream(stream)), "tv_tree_attn")


def tv_tree_attn_static(q, k_new, v_new, k_cache, v_cache, block_table, prefix_len, parents, out,
                        err, rope_theta: float, sm_scale: float | None = None, stream=None) -> None:
    """``tv_tree_attn`` on the library's static scratch (no workspace, no allocation).  Raises
    TVError with TV_ERR_SCRATCH when the call needs more than TV_STATIC_SCRATCH_BYTES."""
    B, N, Hq, hd = q.shape
    Hkv = k_new.shape[2]
    num_blocks, _, bs, _ = k_cache.shape
    max_blocks = block_table.shape[1]
    scale = hd ** -0.5 if sm_scale is None else sm_scale
    _check(lib.tv_tree_attn_static(
        _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_cache), _ptr(v_cache), num_blocks, _ptr(block_table),
        max_blocks, _ptr(prefix_len), _ptr(parents), B, N, Hq, Hkv, hd, bs, float(rope_theta), float(scale),
        _ptr(out), _ptr(err), _stream(stream)), "tv_tree_attn_static")


def tv_kv_compact(k_cache, v_cache, block_table, prefix_len, parents, accepted_path, accepted_len,
                  slot_map, new_len, err, stream=None) -> None:
    num_blocks, Hkv, bs, hd = k_cache.shape
    B, max_blocks = block_table.shape
    N = parents.shape[1]
    Lmax = accepted_path.shape[1]
    _check(lib.tv_kv_compact(
        _ptr(k_cache), _ptr(v_cache), num_blocks, _ptr(block_table), max_blocks, _ptr(prefix_len),
        _ptr(parents), N, _ptr(accepted_path), _ptr(accepted_len), Lmax, B, Hkv, hd, bs, _ptr(slot_map),
        _ptr(new_len), _ptr(err), _stream(stream)), "tv_kv_compact")


def tv_kv_compact_remap(k_cache, v_cache, block_table, block_table_out, prefix_len, parents, accepted_path,
                        accepted_len, slot_map, new_len, remapped, err, stream=None) -> None:
    """Compaction that exchanges whole blocks of ``block_table`` where it can (result rows in
    ``block_table_out``) and moves the other kept entries; ``remapped [B]`` counts exchanges."""
    num_blocks, Hkv, bs, hd = k_cache.shape
    B, max_blocks = block_table.shape
    N = parents.shape[1]
    Lmax = accepted_path.shape[1]
    _check(lib.tv_kv_compact_remap(
        _ptr(k_cache), _ptr(v_cache), num_blocks, _ptr(block_table), _ptr(block_table_out), max_blocks,
        _ptr(prefix_len), _ptr(parents), N, _ptr(accepted_path), _ptr(accepted_len), Lmax, B, Hkv, hd, bs,
        _ptr(slot_map), _ptr(new_len), _ptr(remapped), _ptr(err), _stream(stream)), "tv_kv_compact_remap")


def tv_accept_walk(parents, draft_tokens, target_tokens, accepted_path, accepted_len, next_token, err,
                   stream=None) -> None:
    """parents, draft_tokens, target_tokens [B,N] int32 -> accepted_path [B,Lmax], accepted_len [B],
    next_token [B], err [B] (all int32)."""
    B, N = parents.shape
    _check(lib.tv_accept_walk(_ptr(parents), _ptr(draft_tokens), _ptr(target_tokens), B, N, accepted_path.shape[1],
                              _ptr(accepted_path), _ptr(accepted_len), _ptr(next_token), _ptr(err), _stream(stream)),
           "tv_accept_walk")


def tv_linear_attn_workspace_size(B, T, max_len, H, dk, dv, io_dtype=torch.bfloat16) -> int:
    return int(lib.tv_linear_attn_workspace_size(B, T, max_len, H, dk, dv, _DTYPES[io_dtype]))


def _alpha(alpha, n, H):
    """One decay per head, [H], or per token and head, [n, H]."""
    if alpha.dim() == 1:
        return _whole("alpha", alpha, (H,), torch.float32), 0
    return _rows("alpha", alpha, (n, H), torch.float32, H)


def tv_linear_attn_prompt(q, k, v, alpha, cu_seqlens, out, S, err, S0=None, max_len: int | None = None,
                          workspace=None, q_scale: float = 1.0, stream=None) -> None:
    """S_t = alpha_t S_{t-1} + v_t k_t^T, out_t = S_t (q_scale q_t) over packed prompts: q, k
    [T, Hk, dk] and v, out [T, H, dv] (token stride free, so slices of one projection serve), alpha
    [T, H] or [H] fp32, cu_seqlens [B + 1] int32, S (and S0, which may be S) [B, H, dv, dk].
    Without a ``workspace`` one is taken from torch's allocator when the call needs it."""
    T, H, dv = v.shape
    Hk, dk = q.shape[1:]
    B = cu_seqlens.shape[0] - 1
    io, state, keys, values, states = v.dtype, S.dtype, (T, Hk, dk), (T, H, dv), (B, H, dv, dk)
    pq, sq = _rows("q", q, keys, io, Hk * dk)
    pk, sk = _rows("k", k, keys, io, Hk * dk)
    pv, sv = _rows("v", v, values, io, H * dv)
    po, so = _rows("out", out, values, io, H * dv)
    pa, sa = _alpha(alpha, T, H)
    max_len = T if max_len is None else int(max_len)
    size = 0
    if workspace is None:
        size = lib.tv_linear_attn_workspace_size(B, T, max_len, H, dk, dv, _DTYPES[io])
        if size:
            if stream is None:
                workspace = torch.empty(size, dtype=torch.uint8, device=v.device)
            else:
                with torch.cuda.stream(stream):
                    workspace = torch.empty(size, dtype=torch.uint8, device=v.device)
    else:
        size = workspace.numel() * workspace.element_size()
    _check(lib.tv_linear_attn_prompt(
        pq, sq, pk, sk, pv, sv, pa, sa, _whole("S0", S0, states, state),
        _whole("cu_seqlens", cu_seqlens, (B + 1,), torch.int32), B, T, max_len, Hk, H, dk, dv, _DTYPES[io],
        _DTYPES[state], q_scale, po, so, _whole("S", S, states, state), _ptr(workspace), size,
        _whole("err", err, (B,), torch.int32), _stream(stream)), "tv_linear_attn_prompt")


def tv_linear_attn_step(q, k, v, alpha, S, out, live=None, q_scale: float = 1.0, stream=None) -> None:
    """One token of every sequence: S [B, H, dv, dk] in place; q, k [B, Hk, dk], v, out [B, H, dv],
    alpha [B, H] or [H]; sequences with live[b] = 0 are left alone."""
    B, H, dv = v.shape
    Hk, dk = q.shape[1:]
    io, state, keys, values = v.dtype, S.dtype, (B, Hk, dk), (B, H, dv)
    pq, sq = _rows("q", q, keys, io, Hk * dk)
    pk, sk = _rows("k", k, keys, io, Hk * dk)
    pv, sv = _rows("v", v, values, io, H * dv)
    po, so = _rows("out", out, values, io, H * dv)
    pa, sa = _alpha(alpha, B, H)
    _check(lib.tv_linear_attn_step(
        pq, sq, pk, sk, pv, sv, pa, sa, _whole("live", live, (B,), torch.int32), B, Hk, H, dk, dv, _DTYPES[io],
        _DTYPES[state], q_scale, po, so, _whole("S", S, (B, H, dv, dk), state), _stream(stream)), "tv_linear_attn_step")


def tv_gated_rmsnorm(x, gate, weight, out, eps: float, gate_first: bool = False, weight_offset: float = 0.0,
                     stream=None) -> None:
    """x, gate, out [rows, H, d] (row stride free): rmsnorm over d, times silu(gate); with
    ``gate_first`` the norm is taken of x * silu(gate).  gate and weight [d] may be None."""
    shape, io = x.shape, x.dtype
    rows, H, d = shape
    px, sx = _rows("x", x, shape, io, H * d)
    pg, sg = _rows("gate", gate, shape, io, H * d)
    po, so = _rows("out", out, shape, io, H * d)
    _check(lib.tv_gated_rmsnorm(px, sx, pg, sg, _whole("weight", weight, (d,), io), rows, H, d, _DTYPES[io], eps,
                                weight_offset, int(gate_first), po, so, _stream(stream)), "tv_gated_rmsnorm")


def tv_residual_rmsnorm(y, residual, residual_out, eps: float, out=None, weight=None, post_weight=None, gate=None,
                        scale: float = 1.0, weight_offset: float = 0.0, stream=None) -> None:
    """residual_out = residual + scale * gate * (y, or rmsnorm(y) with post_weight); out (optional) =
    rmsnorm(residual_out) with weight.  All [rows, D] (row stride free), weights [D]."""
    shape, io, res = y.shape, y.dtype, residual.dtype
    rows, D = shape
    py, sy = _rows("y", y, shape, io, D)
    pr, sr = _rows("residual", residual, shape, res, D)
    pg, sg = _rows("gate", gate, shape, io, D)
    pro, sro = _rows("residual_out", residual_out, shape, res, D)
    po, so = _rows("out", out, shape, io, D)
    _check(lib.tv_residual_rmsnorm(py, sy, pr, sr, _whole("post_weight", post_weight, (D,), io), pg, sg, scale,
                                   _whole("weight", weight, (D,), io), rows, D, _DTYPES[io], _DTYPES[res], eps,
                                   weight_offset, pro, sro, po, so, _stream(stream)), "tv_residual_rmsnorm")


def _scratch(size: int, device, stream):
    """``size`` bytes from torch's allocator for a call on ``stream``; None for none."""
    if not size:
        return None
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _room(workspace, device: int):
    """Pointer and bytes of a caller's workspace on the current device."""
    if workspace.is_cuda and workspace.get_device() != device:
        raise ValueError(f"workspace lies on {workspace.device} while cuda:{device} is the current device")
    return _ptr(workspace), workspace.numel() * workspace.element_size()


def _dense(t, shape, dtype, device: int, name: str):
    """Pointer of a dense tensor on the current device (the calls launch on its stream)."""
    if t is None:
        return None
    if t.dtype is dtype and t.get_device() == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _refuse_here(name, t, shape, dtype, device)


def _heads(t, shape, dtype, device: int, row: int, name: str):
    """Pointer and token stride of [tokens, heads, hd] on the current device, the tokens' rows dense."""
    if t is None:
        return None, row
    if t.dtype is dtype and t.get_device() == device and t.shape == shape:
        apart, head, column = t.stride()
        if column == 1 and head == shape[2]:
            return t.data_ptr(), apart if shape[0] > 1 else row
        return _rows(name, t, shape, dtype, row)
    _refuse_here(name, t, shape, dtype, device)


def _refuse_here(name: str, t, shape, dtype, device: int):
    if t.is_cuda and t.get_device() != device:
        raise ValueError(f"{name} lies on {t.device} while cuda:{device} is the current device")
    if t.shape == shape and t.dtype == dtype and t.is_cuda:
        raise ValueError(f"{name}: tensors passed to the library must be contiguous")
    _refuse(name, t, shape, dtype)


def _current(t, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name}: tensors passed to the library must be CUDA tensors")
    return _current_device()


def tv_qk_norm_rope(q, k, q_out, prefix_len, err, *, k_out=None, v=None, k_cache=None, v_cache=None, block_table=None,
                    cu_seqlens=None, live=None, q_weight=None, k_weight=None, norm: bool = True, eps: float = 1e-6,
                    weight_offset: float = 0.0, rotary_dim: int | None = None, rope_theta: float = 10000.0,
                    stream=None) -> None:
    """rmsnorm of q [T, Hq, hd] and k [T, Hkv, hd] per head (``norm``), rotated over the first ``rotary_dim``
    columns (default: all) by the position prefix_len [B] + index in the sequence; queries to ``q_out``, keys to
    ``k_out`` and, with v as it is, to the paged ``k_cache``, ``v_cache`` [num_blocks, Hkv, 16, hd] through
    ``block_table`` [B, max_blocks].  Sequences are packed by ``cu_seqlens`` [B + 1], or one token each without it.
    Token strides are free.  ``prefix_len`` may be None (zero) without a cache; ``live`` [B] skips rows."""
    shape, io, device, whole = q.shape, q.dtype, _current(q, "q"), torch.int32
    T, Hq, hd = shape
    Hkv = k.shape[1]
    B = T if cu_seqlens is None else cu_seqlens.shape[0] - 1
    if io not in _DTYPES:
        _refuse("q", q, shape, "float32 or bfloat16")
    keys = (T, Hkv, hd)
    pq, sq = _heads(q, shape, io, device, Hq * hd, "q")
    pk, sk = _heads(k, keys, io, device, Hkv * hd, "k")
    pqo, sqo = _heads(q_out, shape, io, device, Hq * hd, "q_out")
    pko, sko = _heads(k_out, keys, io, device, Hkv * hd, "k_out")
    pv, sv, pkc, pvc, ptab, blocks, most, bs = None, Hkv * hd, None, None, None, 0, 0, 0
    if k_cache is not None or v_cache is not None:
        if k_cache is None or v_cache is None or v is None or block_table is None:
            raise ValueError("k_cache, v_cache, v and block_table go together")
        blocks, _, bs, _ = k_cache.shape
        most = block_table.shape[1]
        cache = (blocks, Hkv, bs, hd)
        pv, sv = _heads(v, keys, io, device, Hkv * hd, "v")
        pkc = _dense(k_cache, cache, torch.bfloat16, device, "k_cache")
        pvc = _dense(v_cache, cache, torch.bfloat16, device, "v_cache")
        ptab = _dense(block_table, (B, most), whole, device, "block_table")
    _check(lib.tv_qk_norm_rope(
        pq, sq, pk, sk, pv, sv, _dense(q_weight, (hd,), io, device, "q_weight"),
        _dense(k_weight, (hd,), io, device, "k_weight"), _dense(cu_seqlens, (B + 1,), whole, device, "cu_seqlens"),
        _dense(prefix_len, (B,), whole, device, "prefix_len"), _dense(live, (B,), whole, device, "live"), B, T, Hq, Hkv, hd,
        hd if rotary_dim is None else rotary_dim, _DTYPES[io], norm, eps, weight_offset, rope_theta, pqo, sqo, pko, sko, pkc,
        pvc, blocks, ptab, most, bs, _dense(err, (B,), whole, device, "err"), _stream(stream)), "tv_qk_norm_rope")


def tv_window_attn_workspace_size(B, T, max_len, Hq, Hkv, hd, max_blocks, window: int = 0, sinks: int = 0,
                                  block_size=TV_BLOCK_SIZE) -> int:
    return int(lib.tv_window_attn_workspace_size(B, T, max_len, Hq, Hkv, hd, max_blocks, block_size, window, sinks))


def tv_window_attn_prompt(q, k_cache, v_cache, block_table, cu_seqlens, prefix_len, out, err, window: int = 0,
                          sinks: int = 0, max_len: int | None = None, workspace=None, sm_scale: float | None = None,
                          stream=None) -> None:
    """Attention of the new tokens q [T, Hq, hd] bf16, packed by cu_seqlens [B + 1] and standing behind prefix_len [B]
    tokens, over the paged cache that already holds their keys: key j for the query at position p if j <= p and
    (p - j < window, or j < sinks); window 0: every j <= p.  out [T, Hq, hd]; token strides free.  Without a
    ``workspace`` one is taken from torch's allocator when the call needs it."""
    device, bf, whole = _current(q, "q"), torch.bfloat16, torch.int32
    tokens, cache = q.shape, k_cache.shape
    T, Hq, hd = tokens
    blocks, Hkv, bs, _ = cache
    B, most = block_table.shape
    if cache[3] != hd:
        raise ValueError(f"k_cache: expected heads of {hd} columns, got {cache[3]}")
    max_len = T if max_len is None else int(max_len)
    if workspace is None:
        size = lib.tv_window_attn_workspace_size(B, T, max_len, Hq, Hkv, hd, most, bs, window, sinks)
        workspace = _scratch(size, q.device, stream)
        room = None if workspace is None else workspace.data_ptr()
    else:
        room, size = _room(workspace, device)
    pq, sq = _heads(q, tokens, bf, device, Hq * hd, "q")
    po, so = _heads(out, tokens, bf, device, Hq * hd, "out")
    _check(lib.tv_window_attn_prompt(
        pq, sq, _dense(k_cache, cache, bf, device, "k_cache"), _dense(v_cache, cache, bf, device, "v_cache"), blocks,
        _dense(block_table, (B, most), whole, device, "block_table"), most,
        _dense(cu_seqlens, (B + 1,), whole, device, "cu_seqlens"), _dense(prefix_len, (B,), whole, device, "prefix_len"), B, T,
        max_len, Hq, Hkv, hd, bs, window, sinks, hd ** -0.5 if sm_scale is None else sm_scale, po, so, room, size,
        _dense(err, (B,), whole, device, "err"), _stream(stream)), "tv_window_attn_prompt")


def tv_window_attn_step(q, k_cache, v_cache, block_table, prefix_len, out, err, window: int = 0, sinks: int = 0,
                        live=None, workspace=None, sm_scale: float | None = None, stream=None) -> None:
    """The same for one new token of every sequence, q and out [B, Hq, hd], at position prefix_len [B]; sequences with
    live[b] = 0 are left alone."""
    device, bf, whole = _current(q, "q"), torch.bfloat16, torch.int32
    tokens, cache = q.shape, k_cache.shape
    B, Hq, hd = tokens
    blocks, Hkv, bs, _ = cache
    most = block_table.shape[1]
    if cache[3] != hd:
        raise ValueError(f"k_cache: expected heads of {hd} columns, got {cache[3]}")
    if workspace is None:
        size = lib.tv_window_attn_workspace_size(B, B, 1, Hq, Hkv, hd, most, bs, window, sinks)
        workspace = _scratch(size, q.device, stream)
        room = None if workspace is None else workspace.data_ptr()
    else:
        room, size = _room(workspace, device)
    pq, sq = _heads(q, tokens, bf, device, Hq * hd, "q")
    po, so = _heads(out, tokens, bf, device, Hq * hd, "out")
    _check(lib.tv_window_attn_step(
        pq, sq, _dense(k_cache, cache, bf, device, "k_cache"), _dense(v_cache, cache, bf, device, "v_cache"), blocks,
        _dense(block_table, (B, most), whole, device, "block_table"), most,
        _dense(prefix_len, (B,), whole, device, "prefix_len"), _dense(live, (B,), whole, device, "live"), B, Hq, Hkv, hd, bs,
        window, sinks, hd ** -0.5 if sm_scale is None else sm_scale, po, so, room, size,
        _dense(err, (B,), whole, device, "err"), _stream(stream)), "tv_window_attn_step")


def tv_accept_sample(parents, draft_tokens, target_probs, draft_probs, uniforms, accepted_path, accepted_len, next_token,
                     err, stream=None) -> None:
    """Acceptance by probabilities: parents, draft_tokens [B, N] int32, target_probs and draft_probs [B, N, V] (fp32 or
    bf16; draft_probs None: the drafted tokens were chosen, not drawn), uniforms [B, N] fp32 in [0, 1) -> accepted_path
    [B, Lmax], accepted_len [B], next_token [B], err [B] (all int32)."""
    device, io, whole = _current(target_probs, "target_probs"), target_probs.dtype, torch.int32
    B, N, V = target_probs.shape
    Lmax, tree, one = accepted_path.shape[1], (B, N), (B,)
    if io not in _DTYPES:
        _refuse("target_probs", target_probs, target_probs.shape, "float32 or bfloat16")
    _check(lib.tv_accept_sample(
        _dense(parents, tree, whole, device, "parents"), _dense(draft_tokens, tree, whole, device, "draft_tokens"),
        _dense(target_probs, (B, N, V), io, device, "target_probs"), _dense(draft_probs, (B, N, V), io, device, "draft_probs"),
        _dense(uniforms, tree, torch.float32, device, "uniforms"), B, N, V, Lmax, _DTYPES[io],
        _dense(accepted_path, (B, Lmax), whole, device, "accepted_path"), _dense(accepted_len, one, whole, device, "accepted_len"),
        _dense(next_token, one, whole, device, "next_token"), _dense(err, one, whole, device, "err"), _stream(stream)),
        "tv_accept_sample")


def tv_test_bounded_wait(max_polls: int, arrive: bool, status, elapsed_ns, stream=None) -> None:
    """One thread waits on a shared-memory barrier with the library's bounded wait (nothing
    arrives unless ``arrive``): status [1] int32 gets TV_OK or TV_ERR_TIMEOUT, elapsed_ns [1]
    int64 the device time of the wait.  max_polls 0 = the limit the kernels use."""
    _check(lib.tv_test_bounded_wait(int(max_polls), int(bool(arrive)), _ptr(status), _ptr(elapsed_ns),
                                    _stream(stream)), "tv_test_bounded_wait")
