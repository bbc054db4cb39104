"""Batched speculative-verify causal depthwise conv1d update on GB300 (sm_103a).

Thin Python binding over the C ABI in ``include/convverify.h`` (library built in-tree by
``spec_decode_verify_gb300.build``).  This module only marshals torch tensors into pointers and
element strides; every step of the computation runs in the library's CUDA kernels.  There is no
CPU path: CPU tensors are rejected and a missing library raises.

    conv_verify(x, conv_state, weight, bias, out, window, layout=..., qk_channels=..., head_dim=...)
    conv_commit(conv_state, window, accept_len, layout=..., T=..., width=..., x=...)
    conv_prefill(x, conv_state, weight, bias, out, cu_seqlens, max_seqlen=..., qk_channels=..., head_dim=...)

and the operators that follow the conv in a hybrid layer:

    linattn_prefill(q, k, v, log_decay, state, out, cu_seqlens, max_seqlen=...)
    linattn_step(q, k, v, log_decay, state, out, prev=LinattnDrafts(...), update_state=...)
    linattn_commit(LinattnDrafts(...), state)
    block_norm(y, out, gate=..., group=..., post_weight=..., residual=..., residual_out=..., pre_weight=...)

and those of its attention layers, with the acceptance of the drafts:

    cache = PagedCache(k, v, page_table, held=..., refs=...)
    qk_norm_rope(q, k, q_out, cos_sin=..., q_weight=..., k_weight=..., v=v, cache=cache, cache_len=...)
    tree_attention(q, out, cache, cache_len, parent=...)
    draft_verify(probs, tokens, uniforms, accept_len, out_tokens, draft_probs=..., parent=..., path=...)
    cache_compact(cache, cache_len, path, accept_len, new_len=...)
    cache_reserve(cache, n_tokens, cache_len=...), cache_fork(cache, src_idx, dst_idx, n_tokens), cache_free(cache, n_tokens)
"""
from __future__ import annotations

import ctypes
import os
import struct
from typing import Optional

__all__ = ["conv_verify", "conv_commit", "conv_prefill", "verify_plan", "status_string", "load_library", "library_path",
           "CvError", "DENSE", "DEDUP", "HISTORY", "RECOMPUTE", "SEQ_BAD_SLOT", "SEQ_BAD_OFFSET", "SEQ_BAD_ACCEPT",
           "SEQ_TIMEOUT", "SEQ_BAD_SPAN", "SEQ_BAD_TREE", "linattn_prefill", "linattn_step", "linattn_commit",
           "linattn_workspace", "LinattnDrafts", "block_norm", "PagedCache", "tree_attention",
           "tree_attention_workspace", "draft_verify", "qk_norm_rope", "cache_compact", "cache_reserve", "cache_fork", "cache_free",
           "SEQ_BAD_LENGTH", "SEQ_BAD_PAGE", "SEQ_BAD_TOKEN", "SEQ_BAD_PROBS", "SEQ_NO_PAGES", "SEQ_BAD_POSITION",
           "SEQ_SHARED_PAGE"]

_PKG = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_PKG, "_build", "libconvverify.so")

DENSE, DEDUP, HISTORY, RECOMPUTE = 1, 2, 3, 4
F32, BF16 = 0, 1
SEQ_BAD_SLOT, SEQ_BAD_OFFSET, SEQ_BAD_ACCEPT, SEQ_TIMEOUT, SEQ_BAD_SPAN, SEQ_BAD_TREE = 1, 2, 4, 8, 16, 32
SEQ_BAD_LENGTH, SEQ_BAD_PAGE, SEQ_BAD_TOKEN, SEQ_BAD_PROBS, SEQ_NO_PAGES, SEQ_BAD_POSITION, SEQ_SHARED_PAGE = 64, 128, 256, 512, 1024, 2048, 4096
MAX_T = 128
ERR_WORKSPACE = -13

c_i32, c_i64, c_vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p


class VerifyArgs(ctypes.Structure):
    """Mirror of cv_verify_args."""
    _fields_ = [
        ("n_seq", c_i32), ("T", c_i32), ("dim", c_i32), ("width", c_i32), ("qk_channels", c_i32),
        ("head_dim", c_i32), ("dtype", c_i32), ("l2_eps", ctypes.c_float),
        ("x", c_vp), ("x_seq_stride", c_i64), ("x_tok_stride", c_i64),
        ("out", c_vp), ("out_seq_stride", c_i64), ("out_tok_stride", c_i64),
        ("conv_state", c_vp), ("n_slots", c_i32), ("state_cols", c_i32),
        ("state_slot_stride", c_i64), ("state_ch_stride", c_i64),
        ("cache_idx", c_vp), ("state_off", c_vp), ("weight", c_vp), ("bias", c_vp),
        ("window", c_vp), ("window_layout", c_i32), ("wait_polls", c_i32),
        ("win_seq_stride", c_i64), ("win_step_stride", c_i64), ("win_ch_stride", c_i64), ("win_col_stride", c_i64),
        ("err", c_vp), ("state_dtype", c_i32), ("parent", c_vp), ("cu_draft", c_vp), ("total_tokens", c_i32),
        ("state_col_stride", c_i64),
    ]


class CommitArgs(ctypes.Structure):
    """Mirror of cv_commit_args."""
    _fields_ = [
        ("n_seq", c_i32), ("T", c_i32), ("dim", c_i32), ("width", c_i32), ("dtype", c_i32), ("n_slots", c_i32),
        ("conv_state", c_vp), ("state_slot_stride", c_i64), ("state_ch_stride", c_i64),
        ("state_cols", c_i32), ("window_layout", c_i32), ("cache_idx", c_vp), ("window", c_vp),
        ("win_seq_stride", c_i64), ("win_step_stride", c_i64), ("win_ch_stride", c_i64), ("win_col_stride", c_i64),
        ("accept_len", c_vp), ("err", c_vp), ("x", c_vp), ("x_seq_stride", c_i64), ("x_tok_stride", c_i64),
        ("cu_draft", c_vp), ("total_tokens", c_i32), ("wait_polls", c_i32),
    ]


class PrefillArgs(ctypes.Structure):
    """Mirror of cv_prefill_args."""
    _fields_ = [
        ("n_seq", c_i32), ("dim", c_i32), ("width", c_i32), ("qk_channels", c_i32), ("head_dim", c_i32),
        ("dtype", c_i32), ("l2_eps", ctypes.c_float), ("total_tokens", c_i32), ("max_seqlen", c_i32),
        ("x", c_vp), ("x_tok_stride", c_i64), ("out", c_vp), ("out_tok_stride", c_i64), ("cu_seqlens", c_vp),
        ("conv_state", c_vp), ("n_slots", c_i32), ("state_cols", c_i32), ("state_slot_stride", c_i64),
        ("state_ch_stride", c_i64), ("cache_idx", c_vp), ("has_initial_state", c_vp), ("weight", c_vp),
        ("bias", c_vp), ("err", c_vp),
    ]


class LaunchPlan(ctypes.Structure):
    """Mirror of cv_launch_plan."""
    _fields_ = [("grid_x", c_i32), ("grid_y", c_i32), ("threads", c_i32), ("smem_bytes", c_i32),
                ("channels_per_block", c_i32), ("path", c_i32), ("stages", c_i32), ("token_groups", c_i32)]


class LinattnTokens(ctypes.Structure):
    """Mirror of cv_linattn_tokens."""
    _fields_ = [
        ("T", c_i32), ("total_tokens", c_i32), ("cu", c_vp), ("q", c_vp), ("k", c_vp), ("v", c_vp),
        ("q_seq_stride", c_i64), ("q_tok_stride", c_i64), ("q_head_stride", c_i64),
        ("k_seq_stride", c_i64), ("k_tok_stride", c_i64), ("k_head_stride", c_i64),
        ("v_seq_stride", c_i64), ("v_tok_stride", c_i64), ("v_head_stride", c_i64),
        ("log_decay", c_vp), ("decay_seq_stride", c_i64), ("decay_tok_stride", c_i64),
        ("gain", c_vp), ("gain_seq_stride", c_i64), ("gain_tok_stride", c_i64),
    ]


class LinattnArgs(ctypes.Structure):
    """Mirror of cv_linattn_args."""
    _fields_ = [
        ("n_seq", c_i32), ("n_heads", c_i32), ("n_qk_heads", c_i32), ("dk", c_i32), ("dv", c_i32), ("dtype", c_i32),
        ("scale", ctypes.c_float), ("n_slots", c_i32), ("tok", LinattnTokens), ("skip", c_vp), ("out", c_vp),
        ("out_seq_stride", c_i64), ("out_tok_stride", c_i64), ("out_head_stride", c_i64), ("state", c_vp),
        ("state_slot_stride", c_i64), ("state_head_stride", c_i64), ("cache_idx", c_vp), ("has_initial_state", c_vp),
        ("err", c_vp), ("prev", LinattnTokens), ("accept_len", c_vp), ("update_state", c_i32), ("wait_polls", c_i32), ("workspace", c_vp),
        ("workspace_bytes", c_i64),
    ]


class NormArgs(ctypes.Structure):
    """Mirror of cv_norm_args."""
    _fields_ = [
        ("rows", c_i64), ("dim", c_i32), ("group", c_i32), ("dtype", c_i32), ("residual_dtype", c_i32),
        ("gate_act", c_i32), ("gate_first", c_i32), ("eps", ctypes.c_float), ("scale", ctypes.c_float),
        ("y", c_vp), ("y_stride", c_i64), ("gate", c_vp), ("gate_stride", c_i64), ("post_weight", c_vp),
        ("residual", c_vp), ("residual_stride", c_i64), ("residual_out", c_vp), ("residual_out_stride", c_i64),
        ("channel_scale", c_vp), ("pre_weight", c_vp), ("out", c_vp), ("out_stride", c_i64),
    ]


class Cache(ctypes.Structure):
    """Mirror of cv_cache."""
    _fields_ = [
        ("k", c_vp), ("v", c_vp),
        ("k_layer_stride", c_i64), ("k_page_stride", c_i64), ("k_row_stride", c_i64), ("k_head_stride", c_i64),
        ("v_layer_stride", c_i64), ("v_page_stride", c_i64), ("v_row_stride", c_i64), ("v_head_stride", c_i64),
        ("n_layers", c_i32), ("n_pages", c_i32), ("page_size", c_i32), ("n_kv_heads", c_i32), ("head_dim", c_i32),
        ("n_slots", c_i32), ("max_pages", c_i32), ("dtype", c_i32), ("page_table", c_vp), ("table_stride", c_i64),
        ("held", c_vp), ("refs", c_vp),
    ]


class TreeAttentionArgs(ctypes.Structure):
    """Mirror of cv_tree_attention_args."""
    _fields_ = [
        ("n_seq", c_i32), ("T", c_i32), ("n_heads", c_i32), ("total_tokens", c_i32), ("scale", ctypes.c_float),
        ("wait_polls", c_i32), ("cache", Cache), ("q", c_vp), ("q_seq_stride", c_i64), ("q_tok_stride", c_i64),
        ("q_head_stride", c_i64), ("out", c_vp), ("out_seq_stride", c_i64), ("out_tok_stride", c_i64),
        ("out_head_stride", c_i64), ("cu_draft", c_vp), ("parent", c_vp), ("cache_len", c_vp), ("cache_idx", c_vp),
        ("err", c_vp), ("workspace", c_vp), ("workspace_bytes", c_i64),
    ]


class DraftVerifyArgs(ctypes.Structure):
    """Mirror of cv_draft_verify_args."""
    _fields_ = [
        ("n_seq", c_i32), ("T", c_i32), ("vocab", c_i32), ("dtype", c_i32), ("total_tokens", c_i32), ("probs", c_vp),
        ("probs_seq_stride", c_i64), ("probs_tok_stride", c_i64), ("draft_probs", c_vp), ("draft_seq_stride", c_i64),
        ("draft_tok_stride", c_i64), ("tokens", c_vp), ("parent", c_vp), ("uniforms", c_vp), ("cu_draft", c_vp),
        ("cache_idx", c_vp), ("accept_len", c_vp), ("accept_node", c_vp), ("path", c_vp), ("out_tokens", c_vp), ("err", c_vp),
    ]


class QkNormRopeArgs(ctypes.Structure):
    """Mirror of cv_qk_norm_rope_args."""
    _fields_ = [
        ("n_seq", c_i32), ("T", c_i32), ("n_heads", c_i32), ("n_kv_heads", c_i32), ("head_dim", c_i32), ("dtype", c_i32),
        ("total_tokens", c_i32), ("rot_dim", c_i32), ("pairs", c_i32), ("norm", c_i32), ("n_positions", c_i32),
        ("eps", ctypes.c_float),
        ("q", c_vp), ("q_seq_stride", c_i64), ("q_tok_stride", c_i64), ("q_head_stride", c_i64),
        ("q_out", c_vp), ("q_out_seq_stride", c_i64), ("q_out_tok_stride", c_i64), ("q_out_head_stride", c_i64),
        ("k", c_vp), ("k_seq_stride", c_i64), ("k_tok_stride", c_i64), ("k_head_stride", c_i64),
        ("k_out", c_vp), ("k_out_seq_stride", c_i64), ("k_out_tok_stride", c_i64), ("k_out_head_stride", c_i64),
        ("v", c_vp), ("v_seq_stride", c_i64), ("v_tok_stride", c_i64), ("v_head_stride", c_i64),
        ("q_weight", c_vp), ("k_weight", c_vp), ("cos_sin", c_vp), ("cos_sin_stride", c_i64), ("positions", c_vp), ("cu", c_vp),
        ("cache_len", c_vp), ("cache_idx", c_vp), ("cache", Cache), ("err", c_vp),
    ]


class CacheCompactArgs(ctypes.Structure):
    """Mirror of cv_cache_compact_args."""
    _fields_ = [("n_seq", c_i32), ("T", c_i32), ("cache", Cache), ("cache_len", c_vp), ("path", c_vp), ("accept_len", c_vp),
                ("cache_idx", c_vp), ("new_len", c_vp), ("err", c_vp)]


class CachePagesArgs(ctypes.Structure):
    """Mirror of cv_cache_pages_args."""
    _fields_ = [("n_seq", c_i32), ("cache", Cache), ("idx", c_vp), ("src_idx", c_vp), ("n_tokens", c_vp), ("err", c_vp),
                ("cache_len", c_vp)]


class CvError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} (status {status})")
        self.status = status


_lib = None


def load_library(path: Optional[str] = None):
    """Load the CUDA library (raises if it has not been built: there is no fallback)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or library_path
    if not os.path.exists(p):
        raise RuntimeError(f"CUDA library not built: {p} is missing (python -m spec_decode_verify_gb300.build)")
    lib = ctypes.CDLL(p)
    lib.cv_conv_verify.argtypes = [ctypes.POINTER(VerifyArgs), c_vp]
    lib.cv_conv_verify.restype = c_i32
    lib.cv_conv_commit.argtypes = [ctypes.POINTER(CommitArgs), c_vp]
    lib.cv_conv_commit.restype = c_i32
    lib.cv_conv_prefill.argtypes = [ctypes.POINTER(PrefillArgs), c_vp]
    lib.cv_conv_prefill.restype = c_i32
    lib.cv_verify_plan.argtypes = [ctypes.POINTER(VerifyArgs), ctypes.POINTER(LaunchPlan)]
    lib.cv_verify_plan.restype = c_i32
    lib.cv_linattn_prefill.argtypes = [ctypes.POINTER(LinattnArgs), c_vp]
    lib.cv_linattn_prefill.restype = c_i32
    lib.cv_linattn_workspace.argtypes = [ctypes.POINTER(LinattnArgs), ctypes.POINTER(c_i64)]
    lib.cv_linattn_workspace.restype = c_i32
    lib.cv_linattn_step.argtypes = [ctypes.POINTER(LinattnArgs), c_vp]
    lib.cv_linattn_step.restype = c_i32
    lib.cv_block_norm.argtypes = [ctypes.POINTER(NormArgs), c_vp]
    lib.cv_block_norm.restype = c_i32
    for name, args in (("cv_tree_attention", TreeAttentionArgs), ("cv_draft_verify", DraftVerifyArgs),
                       ("cv_qk_norm_rope", QkNormRopeArgs), ("cv_cache_compact", CacheCompactArgs),
                       ("cv_cache_reserve", CachePagesArgs), ("cv_cache_fork", CachePagesArgs), ("cv_cache_free", CachePagesArgs)):
        getattr(lib, name).argtypes = [ctypes.POINTER(args), c_vp]
        getattr(lib, name).restype = c_i32
    lib.cv_tree_attention_workspace.argtypes = [ctypes.POINTER(TreeAttentionArgs), ctypes.POINTER(c_i64)]
    lib.cv_tree_attention_workspace.restype = c_i32
    lib.cv_status_string.argtypes = [c_i32]
    lib.cv_status_string.restype = ctypes.c_char_p
    lib.cv_abi_version.argtypes = []
    lib.cv_abi_version.restype = c_i32
    if path is None:
        _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().cv_status_string(int(status)).decode()


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}: expected bfloat16 or float32")


def _dev_ptr(t, name, required=True):
    if t is None:
        if required:
            raise ValueError(f"{name} is required")
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    return t.data_ptr()


def _need_shape(t, name, shape):
    """Shapes are checked here because the library sees only pointers: a buffer smaller than the
    sizes describe would be read or written past its end."""
    if t is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_int32(t, name, n=None, shape=None):
    """An int32 device array: contiguous, of the given shape, or holding at least n elements."""
    if t is None:
        return
    import torch
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor")
    if shape is not None:
        _need_shape(t, name, shape)
    if n is not None and t.numel() < n:
        raise ValueError(f"{name} needs at least {n} elements, got {t.numel()}")


def _layout_code(layout) -> int:
    if layout in (DENSE, "dense"):
        return DENSE
    if layout in (DEDUP, "dedup"):
        return DEDUP
    if layout in (HISTORY, "history"):
        return HISTORY
    if layout in (RECOMPUTE, "recompute"):
        return RECOMPUTE
    raise ValueError(f"unknown window layout {layout!r}")


def _window_strides(window, layout: int):
    if layout in (HISTORY, RECOMPUTE) or window is None:  # no window buffer
        return 0, 0, 0, 0
    s = window.stride()
    if layout == DENSE:  # [n_seq, T, dim, W-1]
        return s[0], s[1], s[2], s[3]
    return s[0], s[2], s[1], s[2]  # dedup row [n_seq, dim, T+W-2]: step stride = column stride


def _stream_ptr(stream) -> Optional[int]:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_current_stream = _current_device = None


def _one_device(*tensors) -> None:
    """Raise unless all of a call's tensors are on the current CUDA device, which is the one that the library plans for
    and launches on: a pointer of another device would be a bad address there."""
    dev = None
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:
                    raise ValueError("every tensor of a call must be a CUDA tensor (there is no CPU path)")
                if dev is not None:
                    raise ValueError(f"the tensors of a call must be on one device, got cuda:{dev} and cuda:{d}")
                dev = d
    if dev is not None and dev != (_current_device or _load_device())():
        raise ValueError(f"the tensors are on cuda:{dev}, but the current device is cuda:{_current_device()}")


def _load_device():
    global _current_device
    import torch
    _current_device = torch._C._cuda_getDevice
    return _current_device


def _stream_of(stream, t) -> int:
    """The handle of ``stream``, by default torch's current stream on the device of ``t``."""
    if stream is None:
        global _current_stream
        if _current_stream is None:
            import torch
            _current_stream = torch._C._cuda_getCurrentRawStream
        return _current_stream(t.get_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def make_verify_args(x, conv_state, weight, bias, out, window, *, layout, qk_channels, head_dim,
                     l2_eps=1e-6, cache_idx=None, state_off=None, err=None, parent=None, wait_polls=0,
                     cu_draft=None, T=None, check_device=True) -> VerifyArgs:
    """Build cv_verify_args from tensors.

    x [n_seq, T, dim] (channel stride 1, any seq/token strides), conv_state [n_slots, dim, S]
    (column stride 1; it may have the other dtype than x: mixed dtypes), weight [dim, W] contiguous,
    bias [dim] or None, out [n_seq, T, dim] (channel stride 1), window dense [n_seq, T, dim, W-1] or
    dedup [n_seq, dim, T+W-2] (any strides, the dtype of conv_state), or
    None with layout "history" (conv_state [n_slots, dim, S >= T+W-2] then receives the snapshot
    row and the next call reads at state_off = accept_len - 1) or "recompute" (outputs only; the
    commit rebuilds the state from x), cache_idx / state_off / err int32 [n_seq] or None, parent int32
    [n_seq, T] contiguous (tree verify, dense layout) or None.  wait_polls: the limit of the
    pipelined kernel's bounded waits (0 = the default; see cv_verify_args).

    Packed ragged drafts: cu_draft int32 [n_seq + 1]; x and out are then [total_tokens, dim] (token
    stride free, channel stride 1), sequence s owning rows cu_draft[s] .. cu_draft[s+1]-1, and T
    (required) is the largest draft count, the T of the window buffer."""
    lay = _layout_code(layout)
    ptr = _dev_ptr if check_device else (lambda t, n, required=True: None if t is None else t.data_ptr())
    varlen = cu_draft is not None
    if x.dim() != (2 if varlen else 3) or conv_state.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [n_seq, T, dim] ([total_tokens, dim] with cu_draft), conv_state "
                         "[n_slots, dim, S] and weight [dim, W]")
    if varlen:
        if T is None:
            raise ValueError("packed drafts need T, the largest draft count")
        _need_int32(cu_draft, "cu_draft")
        if cu_draft.dim() != 1 or cu_draft.shape[0] < 1:
            raise ValueError("cu_draft must be [n_seq + 1]")
        n_seq, (total, dim) = cu_draft.shape[0] - 1, x.shape
        T = int(T)
    else:
        n_seq, T, dim = x.shape
        total = 0
    W = weight.shape[1]
    _need_shape(out, "out", x.shape)
    _need_shape(weight, "weight", (dim, W))
    _need_shape(bias, "bias", (dim,))
    if conv_state.shape[1] != dim:
        raise ValueError(f"conv_state must have dim = {dim} channels, got {conv_state.shape[1]}")
    if lay == DENSE:
        _need_shape(window, "window", (n_seq, T, dim, W - 1))
    elif lay == DEDUP:
        _need_shape(window, "window", (n_seq, dim, T + W - 2))
    for t, name in ((cache_idx, "cache_idx"), (state_off, "state_off"), (err, "err")):
        _need_int32(t, name, n=n_seq)
    _need_int32(parent, "parent", shape=(n_seq, T))
    if x.stride(-1) != 1 or out.stride(-1) != 1:
        raise ValueError("x and out need a unit innermost stride")
    # conv_state: columns contiguous, or (history layout) column-major rows [n_slots, S, dim] seen
    # as [n_slots, dim, S]; the library checks which strides it accepts
    st_col = 1 if conv_state.shape[2] == 1 else conv_state.stride(2)
    if not weight.is_contiguous() or (bias is not None and not bias.is_contiguous()):
        raise ValueError("weight and bias must be contiguous")
    ws = _window_strides(window, lay)
    if check_device:
        _one_device(x, conv_state, weight, bias, out, window, cache_idx, state_off, err, parent, cu_draft)
    return VerifyArgs(
        n_seq=n_seq, T=T, dim=dim, width=W, qk_channels=qk_channels, head_dim=head_dim, dtype=_dtype_code(x),
        l2_eps=l2_eps, x=ptr(x, "x", total > 0 or not varlen), x_seq_stride=0 if varlen else x.stride(0),
        x_tok_stride=x.stride(-2), out=ptr(out, "out", total > 0 or not varlen),
        out_seq_stride=0 if varlen else out.stride(0), out_tok_stride=out.stride(-2),
        conv_state=ptr(conv_state, "conv_state"), n_slots=conv_state.shape[0], state_cols=conv_state.shape[2],
        state_slot_stride=conv_state.stride(0), state_ch_stride=conv_state.stride(1),
        cache_idx=ptr(cache_idx, "cache_idx", False), state_off=ptr(state_off, "state_off", False),
        weight=ptr(weight, "weight"), bias=ptr(bias, "bias", False),
        window=ptr(window, "window", lay not in (HISTORY, RECOMPUTE)),
        window_layout=lay, wait_polls=int(wait_polls), win_seq_stride=ws[0], win_step_stride=ws[1], win_ch_stride=ws[2],
        win_col_stride=ws[3], err=ptr(err, "err", False),
        state_dtype=0 if conv_state.dtype == x.dtype else _dtype_code(conv_state) + 1,
        parent=ptr(parent, "parent", False), cu_draft=ptr(cu_draft, "cu_draft", False), total_tokens=total,
        state_col_stride=st_col)


def conv_verify(x, conv_state, weight, bias, out, window, *, layout, qk_channels, head_dim, l2_eps=1e-6,
                cache_idx=None, state_off=None, err=None, parent=None, wait_polls=0, cu_draft=None, T=None,
                stream=None) -> None:
    """Queue one batched verify on ``stream`` (default: torch's current stream).

    Writes out, window, conv_state (and err); raises CvError on an invalid argument.  With layout
    "history" pass window=None: the snapshots go into the state rows."""
    for t in (weight, out):
        if t.dtype != x.dtype:
            raise TypeError("x, weight and out must share one dtype")
    if window is not None and window.dtype != conv_state.dtype:
        raise TypeError("window must have the dtype of conv_state")
    _dtype_code(conv_state)
    if bias is not None and bias.dtype != x.dtype:
        raise TypeError("bias must have the dtype of x")
    a = make_verify_args(x, conv_state, weight, bias, out, window, layout=layout, qk_channels=qk_channels,
                         head_dim=head_dim, l2_eps=l2_eps, cache_idx=cache_idx, state_off=state_off, err=err,
                         parent=parent, wait_polls=wait_polls, cu_draft=cu_draft, T=T)
    rc = load_library().cv_conv_verify(ctypes.byref(a), _stream_ptr(stream))
    if rc != 0:
        raise CvError(rc, "cv_conv_verify")


def verify_plan(x, conv_state, weight, bias, out, window, *, layout, qk_channels, head_dim, l2_eps=1e-6,
                cache_idx=None, state_off=None, err=None, parent=None, cu_draft=None, T=None) -> LaunchPlan:
    """The launch cv_conv_verify would make (validates without touching the GPU)."""
    a = make_verify_args(x, conv_state, weight, bias, out, window, layout=layout, qk_channels=qk_channels,
                         head_dim=head_dim, l2_eps=l2_eps, cache_idx=cache_idx, state_off=state_off, err=err,
                         parent=parent, cu_draft=cu_draft, T=T, check_device=False)
    pl = LaunchPlan()
    rc = load_library().cv_verify_plan(ctypes.byref(a), ctypes.byref(pl))
    if rc != 0:
        raise CvError(rc, "cv_verify_plan")
    return pl


def make_commit_args(conv_state, window, accept_len, *, layout, T, width, cache_idx=None, err=None,
                     x=None, cu_draft=None, total_tokens=None, wait_polls=0, check_device=True) -> CommitArgs:
    """Build cv_commit_args.  Layout "recompute": window is None and x is the verify's input
    [n_seq, T, dim] (channel stride 1).  cu_draft: the matching verify's packed draft spans (x is
    then [total_tokens, dim]); accept_len[s] must lie in 1..T_s."""
    lay = _layout_code(layout)
    if x is not None and x.stride(-1) != 1:
        raise ValueError("x needs a unit channel stride")
    varlen = cu_draft is not None
    if varlen:
        _need_int32(cu_draft, "cu_draft", n=accept_len.shape[0] + 1)
        if total_tokens is None:
            total_tokens = x.shape[0] if x is not None else 0
    ptr = _dev_ptr if check_device else (lambda t, n, required=True: None if t is None else t.data_ptr())
    ws = _window_strides(window, lay)
    if conv_state.dim() != 3 or conv_state.stride(2) != 1:
        raise ValueError("conv_state must be [n_slots, dim, S] with a unit column stride")
    _need_int32(accept_len, "accept_len")
    if accept_len.dim() != 1:
        raise ValueError("accept_len must be [n_seq]")
    n_seq, dim = accept_len.shape[0], conv_state.shape[1]
    for t, name in ((cache_idx, "cache_idx"), (err, "err")):
        _need_int32(t, name, n=n_seq)
    if lay == DENSE:
        _need_shape(window, "window", (n_seq, T, dim, width - 1))
    elif lay == DEDUP:
        _need_shape(window, "window", (n_seq, dim, T + width - 2))
    elif varlen:
        if x is None or x.dim() != 2 or x.shape[1] != dim or x.shape[0] != total_tokens:
            raise ValueError(f"x must be [total_tokens, {dim}] with packed drafts")
    else:
        _need_shape(x, "x", (n_seq, T, dim))
    if check_device:
        _one_device(conv_state, window, accept_len, cache_idx, err, x, cu_draft)
    return CommitArgs(
        n_seq=accept_len.shape[0], T=T, dim=conv_state.shape[1], width=width, dtype=_dtype_code(conv_state),
        n_slots=conv_state.shape[0], conv_state=ptr(conv_state, "conv_state"),
        state_slot_stride=conv_state.stride(0), state_ch_stride=conv_state.stride(1),
        state_cols=conv_state.shape[2], window_layout=lay, cache_idx=ptr(cache_idx, "cache_idx", False),
        window=ptr(window, "window", lay != RECOMPUTE), win_seq_stride=ws[0], win_step_stride=ws[1],
        win_ch_stride=ws[2], win_col_stride=ws[3], accept_len=ptr(accept_len, "accept_len"),
        err=ptr(err, "err", False), x=ptr(x, "x", lay == RECOMPUTE and not (varlen and total_tokens == 0)),
        x_seq_stride=x.stride(0) if x is not None and not varlen else 0,
        x_tok_stride=x.stride(-2) if x is not None else 0,
        cu_draft=ptr(cu_draft, "cu_draft", False), total_tokens=int(total_tokens or 0), wait_polls=int(wait_polls))


def conv_commit(conv_state, window, accept_len, *, layout, T, width, cache_idx=None, err=None, x=None,
                cu_draft=None, total_tokens=None, wait_polls=0, stream=None) -> None:
    """Queue the commit: conv_state[slot] <- snapshot accept_len[s]-1 of sequence s (rebuilt from the
    kept window and x with layout "recompute")."""
    for t in (window, x):
        if t is not None and t.dtype != conv_state.dtype:
            raise TypeError("window / x and conv_state must share one dtype")
    a = make_commit_args(conv_state, window, accept_len, layout=layout, T=T, width=width, cache_idx=cache_idx,
                         err=err, x=x, cu_draft=cu_draft, total_tokens=total_tokens, wait_polls=wait_polls)
    rc = load_library().cv_conv_commit(ctypes.byref(a), _stream_ptr(stream))
    if rc != 0:
        raise CvError(rc, "cv_conv_commit")


def make_prefill_args(x, conv_state, weight, bias, out, cu_seqlens, *, max_seqlen, qk_channels, head_dim,
                      l2_eps=1e-6, cache_idx=None, has_initial_state=None, err=None, check_device=True) -> PrefillArgs:
    """Build cv_prefill_args from tensors.

    x, out [total_tokens, dim] (channel stride 1, any token stride), conv_state [n_slots, dim, S]
    (column stride 1), weight [dim, W] contiguous, bias [dim] or None, cu_seqlens int32
    [n_seq + 1], cache_idx / has_initial_state / err int32 [n_seq] or None; max_seqlen bounds
    every sequence's length (host int)."""
    ptr = _dev_ptr if check_device else (lambda t, n, required=True: None if t is None else t.data_ptr())
    if x.dim() != 2 or conv_state.dim() != 3 or weight.dim() != 2:
        raise ValueError("x must be [total_tokens, dim], conv_state [n_slots, dim, S] and weight [dim, W]")
    total, dim = x.shape
    _need_shape(out, "out", x.shape)
    _need_shape(weight, "weight", (dim, weight.shape[1]))
    _need_shape(bias, "bias", (dim,))
    if conv_state.shape[1] != dim:
        raise ValueError(f"conv_state must have dim = {dim} channels, got {conv_state.shape[1]}")
    _need_int32(cu_seqlens, "cu_seqlens")
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [n_seq + 1]")
    for t, name in ((cache_idx, "cache_idx"), (has_initial_state, "has_initial_state"), (err, "err")):
        _need_int32(t, name, n=cu_seqlens.shape[0] - 1)
    if x.stride(1) != 1 or out.stride(1) != 1 or conv_state.stride(2) != 1:
        raise ValueError("x, out and conv_state need a unit innermost stride")
    if not weight.is_contiguous() or (bias is not None and not bias.is_contiguous()):
        raise ValueError("weight and bias must be contiguous")
    if check_device:
        _one_device(x, conv_state, weight, bias, out, cu_seqlens, cache_idx, has_initial_state, err)
    return PrefillArgs(
        n_seq=cu_seqlens.shape[0] - 1, dim=dim, width=weight.shape[1], qk_channels=qk_channels, head_dim=head_dim,
        dtype=_dtype_code(x), l2_eps=l2_eps, total_tokens=total, max_seqlen=int(max_seqlen),
        x=ptr(x, "x", total > 0), x_tok_stride=x.stride(0), out=ptr(out, "out", total > 0),
        out_tok_stride=out.stride(0), cu_seqlens=ptr(cu_seqlens, "cu_seqlens"),
        conv_state=ptr(conv_state, "conv_state"), n_slots=conv_state.shape[0], state_cols=conv_state.shape[2],
        state_slot_stride=conv_state.stride(0), state_ch_stride=conv_state.stride(1),
        cache_idx=ptr(cache_idx, "cache_idx", False), has_initial_state=ptr(has_initial_state, "has_initial_state", False),
        weight=ptr(weight, "weight"), bias=ptr(bias, "bias", False), err=ptr(err, "err", False))


def conv_prefill(x, conv_state, weight, bias, out, cu_seqlens, *, max_seqlen, qk_channels, head_dim, l2_eps=1e-6,
                 cache_idx=None, has_initial_state=None, err=None, stream=None) -> None:
    """Queue one packed variable-length prefill on ``stream`` (default: torch's current stream).

    Writes out, conv_state (and err); raises CvError on an invalid argument."""
    for t in (x, conv_state, weight, out):
        if t.dtype != x.dtype:
            raise TypeError("x, conv_state, weight and out must share one dtype")
    if bias is not None and bias.dtype != x.dtype:
        raise TypeError("bias must have the dtype of x")
    a = make_prefill_args(x, conv_state, weight, bias, out, cu_seqlens, max_seqlen=max_seqlen, qk_channels=qk_channels,
                          head_dim=head_dim, l2_eps=l2_eps, cache_idx=cache_idx, has_initial_state=has_initial_state,
                          err=err)
    rc = load_library().cv_conv_prefill(ctypes.byref(a), _stream_ptr(stream))
    if rc != 0:
        raise CvError(rc, "cv_conv_prefill")


class LinattnDrafts:
    """Drafts of an earlier linattn_step and how many of each sequence's were accepted.

    k [n_seq, T, n_qk_heads, dk], v [n_seq, T, n_heads, dv], log_decay fp32 [n_seq, T, n_heads], gain
    like log_decay or None; with cu_draft (int32 [n_seq + 1]) packed rows [total, ...] instead, T then
    being the largest count (required).  accept_len int32 [n_seq]: 0 .. the sequence's draft count."""
    __slots__ = ("k", "v", "log_decay", "gain", "accept_len", "cu_draft", "T")

    def __init__(self, k, v, log_decay, accept_len, *, gain=None, cu_draft=None, T=None):
        self.k, self.v, self.log_decay, self.gain, self.accept_len = k, v, log_decay, gain, accept_len
        self.cu_draft, self.T = cu_draft, T


# cv_linattn_tokens and cv_linattn_args as the struct module writes them: one call fills all fields
_TOKENS = "iiQQQQ9qQ2qQ2q"
_LINATTN = struct.Struct("<6ifi" + _TOKENS + "QQ3qQ2qQQQ" + _TOKENS + "QiiQq")
_NO_TOKENS = (0,) * 21
_NORM = struct.Struct("<q6i2fQqQqQQqQqQQQq")


def _pointer(t, name) -> int:
    if t is None:
        raise ValueError(f"{name} is required")
    return t.data_ptr()


def _index_array(t, name, n) -> int:
    """Pointer of an int32 array of at least n elements, or 0."""
    if t is None:
        return 0
    if t.dtype is not _i32 or t.numel() < n or not t.is_contiguous():
        _need_int32(t, name, n=n)
    return t.data_ptr()


# torch's types, looked up once (the package does not import torch by itself)
_f32 = _bf16 = _i32 = None


def _load_types():
    global _f32, _bf16, _i32
    import torch
    _bf16, _i32, _f32 = torch.bfloat16, torch.int32, torch.float32
    return _f32


def _linattn_tokens(q, k, v, log_decay, gain, cu, T, n_seq, what) -> tuple:
    """The fields of cv_linattn_tokens for [n_seq, T, heads, d] rows, or packed [total, heads, d] rows with
    cu."""
    f32 = _f32 or _load_types()
    packed = cu is not None
    nd = 3 if packed else 4
    ks, vs, gs = k.shape, v.shape, log_decay.shape
    if len(ks) != nd or len(vs) != nd or len(gs) != nd - 1 or (q is not None and q.shape != ks):
        raise ValueError(f"{what}: q and k must agree, and q, k and v be [n_seq, T, heads, d] and log_decay "
                         "[n_seq, T, heads], or [total, ...] with packed rows")
    if ks[:-2] != vs[:-2] or gs != vs[:-1] or (gain is not None and gain.shape != gs):
        raise ValueError(f"{what}: q, k, v, log_decay and gain must have the same rows, and log_decay and gain the heads "
                         f"of v: {tuple(ks)}, {tuple(vs)}, {tuple(gs)}")
    dt = k.dtype
    if v.dtype is not dt or (q is not None and q.dtype is not dt):
        raise TypeError("q, k and v must share one dtype")
    if log_decay.dtype is not f32 or (gain is not None and gain.dtype is not f32):
        raise TypeError("log_decay and gain must be float32")
    kt, vt, gt = k.stride(), v.stride(), log_decay.stride()
    qt = q.stride() if q is not None else kt
    bt = gain.stride() if gain is not None else gt
    if (kt[-1] != 1 or qt[-1] != 1) and ks[-1] > 1 or vt[-1] != 1 and vs[-1] > 1:
        raise ValueError("q, k and v need a unit innermost stride")
    if gs[-1] > 1 and (gt[-1] != 1 or bt[-1] != 1):
        raise ValueError("log_decay and gain need a unit innermost stride")
    if packed:
        if cu.dtype is not _i32 or cu.shape != (n_seq + 1,) or not cu.is_contiguous():
            _need_int32(cu, "cu", shape=(n_seq + 1,))
        if T is None:
            raise ValueError(f"{what}: packed rows need T, the largest count")
        total = vs[0]
        qt, kt, vt, gt, bt = (0, qt[0], qt[1]), (0, kt[0], kt[1]), (0, vt[0], vt[1]), (0, gt[0]), (0, bt[0])
    else:
        if vs[0] != n_seq:
            raise ValueError(f"{what}: {n_seq} sequences expected, got {vs[0]}")
        if T is not None and T != vs[1]:
            raise ValueError(f"{what}: T = {T} but the rows hold {vs[1]} tokens")
        T, total = vs[1], 0
    return (int(T), total, cu.data_ptr() if packed else 0, q.data_ptr() if q is not None else 0, k.data_ptr(), v.data_ptr(),
            qt[0], qt[1], qt[2], kt[0], kt[1], kt[2], vt[0], vt[1], vt[2], log_decay.data_ptr(), gt[0], gt[1],
            gain.data_ptr() if gain is not None else 0, bt[0], bt[1])


def make_linattn_args(q, k, v, log_decay, state, out, *, n_seq, gain=None, skip=None, scale=None, cu=None, T=None,
                      prev=None, update_state=False, cache_idx=None, has_initial_state=None, err=None,
                      workspace=None, wait_polls=0, check_device=True) -> LinattnArgs:
    """Build cv_linattn_args (see linattn_prefill and linattn_step; q None: no tokens, prev alone)."""
    f32 = _f32 or _load_types()
    ss, st = state.shape, state.stride()
    if len(ss) != 4 or state.dtype is not f32:
        raise ValueError("state must be float32 [n_slots, n_heads, dk, dv]")
    n_slots, H, dk, dv = ss
    if (dv > 1 and st[3] != 1) or (dk > 1 and st[2] != dv):
        raise ValueError("the [dk, dv] state of a head must be contiguous")
    first = q if q is not None else prev.k
    nq = first.shape[-2]
    tok, o, os = _NO_TOKENS, 0, (0, 0, 0)
    if q is not None:
        tok = _linattn_tokens(q, k, v, log_decay, gain, cu, T, n_seq, "tokens")
        if q.shape[-1] != dk or v.shape[-2] != H or v.shape[-1] != dv:
            raise ValueError(f"heads of q|k [.., {q.shape[-1]}] and v {tuple(v.shape[-2:])} do not fit the state {tuple(ss)}")
        if out.shape != v.shape or out.dtype is not v.dtype or (out.stride(-1) != 1 and dv > 1):
            raise ValueError("out needs the shape and dtype of v and a unit innermost stride")
        o, os = _pointer(out, "out"), out.stride()
        os = (0, os[0], os[1]) if cu is not None else os
    sk = 0
    if skip is not None:
        _need_shape(skip, "skip", (H,))
        if skip.dtype is not f32 or not skip.is_contiguous():
            raise ValueError("skip must be contiguous float32")
        sk = skip.data_ptr()
    old, accept = _NO_TOKENS, 0
    if prev is not None:
        pk, pv = prev.k, prev.v
        old = _linattn_tokens(None, pk, pv, prev.log_decay, prev.gain, prev.cu_draft, prev.T, n_seq,
                              "previous drafts")
        if pk.dtype is not first.dtype or pk.shape[-2] != nq or pk.shape[-1] != dk or pv.shape[-2] != H or pv.shape[-1] != dv:
            raise ValueError("the previous drafts must have the dtype, heads and head sizes of the tokens")
        if prev.accept_len is None:
            raise ValueError("accept_len is required")
        accept = _index_array(prev.accept_len, "accept_len", n_seq)
    ws, ws_bytes = 0, 0
    if workspace is not None:
        ws, ws_bytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    if check_device:  # written out, since a call of one token notices a loop (0.5 us of 11)
        dev = state.get_device()
        if not (dev >= 0 and (_current_device or _load_device())() == dev and
                (q is None or q.get_device() == k.get_device() == v.get_device() == log_decay.get_device() == out.get_device() == dev) and
                (gain is None or gain.get_device() == dev) and (skip is None or skip.get_device() == dev) and
                (cu is None or cu.get_device() == dev) and (cache_idx is None or cache_idx.get_device() == dev) and
                (has_initial_state is None or has_initial_state.get_device() == dev) and
                (err is None or err.get_device() == dev) and (workspace is None or workspace.get_device() == dev) and
                (prev is None or prev.k.get_device() == prev.v.get_device() == prev.log_decay.get_device() ==
                 prev.accept_len.get_device() == dev and (prev.gain is None or prev.gain.get_device() == dev) and
                 (prev.cu_draft is None or prev.cu_draft.get_device() == dev))):
            _one_device(state, q, k, v, log_decay, out, gain, skip, cu, cache_idx, has_initial_state, err, workspace,
                        *((prev.k, prev.v, prev.log_decay, prev.gain, prev.cu_draft, prev.accept_len) if prev is not None else ()))
    return LinattnArgs.from_buffer_copy(_LINATTN.pack(
        n_seq, H, nq, dk, dv, BF16 if first.dtype is _bf16 else _dtype_code(first), dk ** -0.5 if scale is None else scale, n_slots, *tok, sk, o, os[0], os[1],
        os[2], state.data_ptr(), st[0], st[1], _index_array(cache_idx, "cache_idx", n_seq),
        _index_array(has_initial_state, "has_initial_state", n_seq), _index_array(err, "err", n_seq), *old, accept, 1 if update_state else 0, wait_polls, ws, ws_bytes))


def linattn_workspace(q, k, v, log_decay, state, out, cu_seqlens, *, max_seqlen, **kw) -> int:
    """Bytes of workspace linattn_prefill needs for these arguments on the current device (0 = none)."""
    a = make_linattn_args(q, k, v, log_decay, state, out, n_seq=cu_seqlens.shape[0] - 1, cu=cu_seqlens, T=max_seqlen,
                          check_device=False, **kw)
    return _linattn_workspace(a)


def _linattn_workspace(a: LinattnArgs) -> int:
    n = c_i64(0)
    rc = load_library().cv_linattn_workspace(ctypes.byref(a), ctypes.byref(n))
    if rc != 0:
        raise CvError(rc, "cv_linattn_workspace")
    return n.value


def linattn_prefill(q, k, v, log_decay, state, out, cu_seqlens, *, max_seqlen, gain=None, skip=None, scale=None,
                    cache_idx=None, has_initial_state=None, err=None, workspace=None, wait_polls=0, stream=None) -> None:
    """Queue linear attention with a decay for each head over packed prompts (cv_linattn_prefill).

    q, k [total, n_qk_heads, dk], v and out [total, n_heads, dv] (innermost stride 1, the others free:
    slices of one conv output will do), log_decay and gain fp32 [total, n_heads], skip fp32 [n_heads],
    state fp32 [n_slots, n_heads, dk, dv], cu_seqlens int32 [n_seq + 1], max_seqlen a host bound on the
    lengths; scale defaults to dk**-0.5.  Writes out, state (and err).  workspace: a uint8 buffer of
    linattn_workspace bytes; by default torch's allocator gives one for the call.  wait_polls: the limit of the
    kernel's bounded waits (0: the default; negative: none, a wait gives up at once)."""
    if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
        raise ValueError("cu_seqlens must be [n_seq + 1]")
    a = make_linattn_args(q, k, v, log_decay, state, out, n_seq=cu_seqlens.shape[0] - 1, gain=gain, skip=skip,
                          scale=scale, cu=cu_seqlens, T=max_seqlen, cache_idx=cache_idx,
                          has_initial_state=has_initial_state, err=err, workspace=workspace, wait_polls=wait_polls)
    lib, on = load_library(), _stream_of(stream, q)
    rc = lib.cv_linattn_prefill(ctypes.byref(a), on)
    if rc == ERR_WORKSPACE and workspace is None:  # nothing was launched: this call needs one
        import torch
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            raise ValueError("pass workspace with a raw stream handle")
        need = _linattn_workspace(a)
        # from the stream's own pool: a block freed on another stream may still be in use there
        with torch.cuda.stream(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), need
        rc = lib.cv_linattn_prefill(ctypes.byref(a), on)
    if rc != 0:
        raise CvError(rc, "cv_linattn_prefill")


def linattn_step(q, k, v, log_decay, state, out, *, gain=None, skip=None, scale=None, update_state=True, prev=None,
                 cache_idx=None, has_initial_state=None, cu_draft=None, T=None, err=None, stream=None) -> None:
    """Queue one step of the same recurrence (cv_linattn_step): T new tokens for each sequence.

    q, k [n_seq, T, n_qk_heads, dk], v and out [n_seq, T, n_heads, dv], log_decay and gain fp32
    [n_seq, T, n_heads]; with cu_draft packed rows [total, ...], T then being the largest count.
    prev (LinattnDrafts): the state is first advanced over the accepted drafts of the previous step.
    update_state False leaves the state there (a verify: pass these tokens as prev next time, or to
    linattn_commit); True leaves it after the new tokens (decoding)."""
    n_seq = cu_draft.shape[0] - 1 if cu_draft is not None else q.shape[0]
    a = make_linattn_args(q, k, v, log_decay, state, out, n_seq=n_seq, gain=gain, skip=skip, scale=scale, cu=cu_draft,
                          T=T, prev=prev, update_state=update_state, cache_idx=cache_idx,
                          has_initial_state=has_initial_state, err=err)
    rc = load_library().cv_linattn_step(ctypes.byref(a), _stream_of(stream, q))
    if rc != 0:
        raise CvError(rc, "cv_linattn_step")


def linattn_commit(drafts: LinattnDrafts, state, *, cache_idx=None, has_initial_state=None, err=None,
                   stream=None) -> None:
    """Queue the commit alone: the state advanced over each sequence's accepted drafts."""
    n_seq = drafts.accept_len.shape[0]
    a = make_linattn_args(None, None, None, None, state, None, n_seq=n_seq, prev=drafts, cache_idx=cache_idx,
                          has_initial_state=has_initial_state, err=err)
    rc = load_library().cv_linattn_step(ctypes.byref(a), _stream_of(stream, state))
    if rc != 0:
        raise CvError(rc, "cv_linattn_step")


def make_norm_args(y, out, *, gate=None, gate_act=None, gate_first=False, group=0, post_weight=None, residual=None,
                   residual_out=None, scale=1.0, channel_scale=None, pre_weight=None, eps=1e-6,
                   check_device=True) -> NormArgs:
    """Build cv_norm_args (see block_norm)."""
    shape = y.shape
    if len(shape) != 2:
        raise ValueError("y must be [rows, dim]")
    rows, dim = shape
    dt = y.dtype
    f32 = _f32 or _load_types()
    act = 0 if gate_act in (None, "silu") else 1 if gate_act == "sigmoid" else None
    if act is None:
        raise ValueError(f"unknown gate activation {gate_act!r}")

    def row(t, name, like):  # pointer and row stride
        if t is None:
            return 0, 0
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        st = t.stride()
        if st[1] != 1 and dim > 1:
            raise ValueError(f"{name} needs a unit channel stride")
        if like and t.dtype is not dt:
            raise TypeError("y, gate and out must share one dtype")
        return t.data_ptr(), st[0]

    def vec(t, name, n):
        if t is None:
            return 0
        if t.dim() != 1 or t.shape[0] != n or t.dtype is not dt or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous [{n}] and have the dtype of y")
        return t.data_ptr()

    if residual is None:
        if out is None or residual_out is not None or channel_scale is not None or pre_weight is not None:
            raise ValueError("without a residual, out is required and residual_out, channel_scale and pre_weight "
                             "have no meaning")
    elif residual_out is None or residual_out.dtype is not residual.dtype:
        raise ValueError("residual needs residual_out of its dtype")
    if check_device:
        dev = y.get_device()
        if not (dev >= 0 and (_current_device or _load_device())() == dev and (out is None or out.get_device() == dev) and
                (gate is None or gate.get_device() == dev) and (post_weight is None or post_weight.get_device() == dev) and
                (residual is None or residual.get_device() == residual_out.get_device() == dev) and
                (channel_scale is None or channel_scale.get_device() == dev) and
                (pre_weight is None or pre_weight.get_device() == dev)):
            _one_device(y, out, gate, residual, residual_out, post_weight, channel_scale, pre_weight)
    code = BF16 if dt is _bf16 else _dtype_code(y)
    return NormArgs.from_buffer_copy(_NORM.pack(
        rows, dim, group, code, code if residual is None else F32 if residual.dtype is f32 else _dtype_code(residual), act, 1 if gate_first else 0, eps, scale,
        *row(y, "y", True), *row(gate, "gate", True), vec(post_weight, "post_weight", group),
        *row(residual, "residual", False), *row(residual_out, "residual_out", False),
        vec(channel_scale, "channel_scale", dim), vec(pre_weight, "pre_weight", dim), *row(out, "out", True)))


def block_norm(y, out, *, gate=None, gate_act=None, gate_first=False, group=0, post_weight=None, residual=None,
               residual_out=None, scale=1.0, channel_scale=None, pre_weight=None, eps=1e-6, stream=None) -> None:
    """Queue the norms around a block with its gate and scaled residual (cv_block_norm).

    y [rows, dim] is gated by gate (gate_act "silu" or "sigmoid"; before the norm with gate_first, else
    after) and RMS-normed over groups of ``group`` channels (0: not at all) with post_weight [group].
    Without residual, out receives that.  With residual (fp32 or the dtype of y), residual_out receives
    residual + scale * channel_scale * that, and out (may be None) its RMS norm over the row with
    pre_weight [dim].  Row strides are free, channels contiguous; out may be y or gate, and residual_out
    may be residual."""
    a = make_norm_args(y, out, gate=gate, gate_act=gate_act, gate_first=gate_first, group=group,
                       post_weight=post_weight, residual=residual, residual_out=residual_out, scale=scale,
                       channel_scale=channel_scale, pre_weight=pre_weight, eps=eps)
    rc = load_library().cv_block_norm(ctypes.byref(a), _stream_of(stream, y))
    if rc != 0:
        raise CvError(rc, "cv_block_norm")


# cv_cache and the structs around it as the struct module writes them
_CACHE = struct.Struct("<2Q8q8iQq2Q")
_IN = f"{_CACHE.size}s"
_TREE_ATTENTION = struct.Struct("<4ifi" + _IN + "Q3qQ3q4QQQq")
_DRAFT_VERIFY = struct.Struct("<5i4xQ2qQ2q5Q5Q")
_QK_NORM_ROPE = struct.Struct("<11if" + 5 * "Q3q" + "3Qq4Q" + _IN + "Q")
_COMPACT = struct.Struct("<2i" + _IN + "6Q")
_PAGES = struct.Struct("<i4x" + _IN + "5Q")
_NO_CACHE = bytes(_CACHE.size)


class PagedCache:
    """A cache of K and V in pages (cv_cache): position x of slot r is row x % page_size of page page_table[r, x // page_size].

    k, v [n_pages, page_size, n_kv_heads, head_dim], or [n_layers, n_pages, ...] for cache_compact and cache_fork (innermost
    stride 1, the others free, one dtype); page_table int32 [n_slots, max_pages], entries past those in use may be
    anything.  held int32 [n_slots] (pages of each slot) and refs int32 [n_pages] (slots that hold each page, 0 = free) are
    needed by cache_reserve, cache_fork and cache_free; with refs, qk_norm_rope and cache_compact write into no page that more than one slot
    holds (SEQ_SHARED_PAGE): a slot that was forked shares full pages and is not to be written before their end.  Made once for the tensors, which it keeps; layer(i) is the cache
    of one layer.  A call raises ValueError where one of them has been given other memory since (set_, resize_, .data): the handle is then
    to be made again."""
    __slots__ = ("_k", "_v", "_page_table", "_held", "_refs", "_packed", "_at", "_device", "_dtype", "_code", "_heads", "_d", "_layers")

    def __init__(self, k, v, page_table, *, held=None, refs=None):
        if k.dim() not in (4, 5) or v.shape != k.shape:
            raise ValueError("k and v must be [n_pages, page_size, n_kv_heads, head_dim] or [n_layers, n_pages, ...] alike, got "
                             f"{tuple(k.shape)} and {tuple(v.shape)}")
        if v.dtype is not k.dtype:
            raise TypeError("k and v must share one dtype")
        dtype = _dtype_code(k)
        if k.shape[-1] > 1 and (k.stride(-1) != 1 or v.stride(-1) != 1):
            raise ValueError("k and v need a unit innermost stride")
        _load_types()
        if page_table.dim() != 2 or page_table.dtype is not _i32 or (page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("page_table must be int32 [n_slots, max_pages] with a unit innermost stride")
        _need_int32(held, "held", shape=(page_table.shape[0],))
        _need_int32(refs, "refs", shape=(k.shape[-4],))
        self._k, self._v, self._page_table, self._held, self._refs = k, v, page_table, held, refs
        devices = {x.get_device() for x in self._tensors() if x is not None}
        self._device = devices.pop() if len(devices) == 1 else None
        self._dtype, self._code, self._heads, self._d, self._layers = k.dtype, dtype, k.shape[-2], k.shape[-1], k.dim() == 5
        ks, vs = k.stride()[-5:-1], v.stride()[-5:-1]
        if k.dim() == 4:
            ks, vs = (0, *ks), (0, *vs)
        rows = page_table.stride(0) if page_table.shape[0] > 1 else page_table.shape[1]
        self._at = self._addresses()
        self._packed = _CACHE.pack(
            k.data_ptr(), v.data_ptr(), *ks, *vs, k.shape[0] if k.dim() == 5 else 1, *k.shape[-4:], *page_table.shape, dtype,
            page_table.data_ptr(), rows, held.data_ptr() if held is not None else 0,
            refs.data_ptr() if refs is not None else 0)

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    page_table = property(lambda self: self._page_table)
    held = property(lambda self: self._held)
    refs = property(lambda self: self._refs)

    def layer(self, i) -> "PagedCache":
        """The cache of layer i of [n_layers, ...] tensors."""
        return PagedCache(self._k[i], self._v[i], self._page_table, held=self._held, refs=self._refs)

    def _tensors(self):
        return self._k, self._v, self._page_table, self._held, self._refs

    def _addresses(self):
        held, refs = self._held, self._refs
        return (self._k.data_ptr(), self._v.data_ptr(), self._page_table.data_ptr(), held.data_ptr() if held is not None else 0,
                refs.data_ptr() if refs is not None else 0)

    def _args(self) -> bytes:
        """cv_cache of the tensors, as long as their memory is what it was."""
        if self._addresses() != self._at:
            raise ValueError("a tensor of the cache has other memory than when the PagedCache was made: make it again")
        return self._packed


def _one_layer(cache) -> None:
    if cache._layers:
        raise ValueError("this call takes the cache of one layer (PagedCache.layer)")


def _exactly(t, name, shape) -> int:
    """Pointer of a contiguous int32 array of the given shape, or 0."""
    if t is None:
        return 0
    if t.dtype is not _i32 or t.shape != shape or not t.is_contiguous():
        _need_int32(t, name, shape=shape)
    return t.data_ptr()


def _lead(shape, cu, T, name):
    """(n_seq, T, total, lead) of [n_seq, T, ...] rows, or [total, ...] with cu."""
    if cu is None:
        if len(shape) < 2:
            raise ValueError(f"{name} must be [n_seq, T, ...]")
        if T is not None and T != shape[1]:
            raise ValueError(f"T = {T} but {name} holds {shape[1]} tokens a sequence")
        return shape[0], shape[1], 0, shape[:2]
    n = cu.shape
    if len(n) != 1 or n[0] < 1:
        raise ValueError("the cumulative counts must be [n_seq + 1]")
    if cu.dtype is not _i32 or not cu.is_contiguous():
        _need_int32(cu, "the cumulative counts")
    if T is None:
        raise ValueError("packed rows need T, the largest count")
    return n[0] - 1, int(T), shape[0], shape[:1]


def make_tree_attention_args(q, out, cache, cache_len, *, parent=None, scale=None, cu_draft=None, T=None, cache_idx=None, err=None,
                             workspace=None, wait_polls=0, check_device=True) -> TreeAttentionArgs:
    """Build cv_tree_attention_args (see tree_attention)."""
    if cache._layers:
        _one_layer(cache)
    qs, d, dt = q.shape, cache._d, cache._dtype
    if len(qs) != (4 if cu_draft is None else 3):
        raise ValueError("q must be [n_seq, T, n_heads, head_dim], or [total, n_heads, head_dim] with cu_draft")
    n, T, total, lead = _lead(qs, cu_draft, T, "q")
    if out is None or out.shape != qs or qs[-1] != d:
        raise ValueError(f"q and out must have one shape and heads of {d} channels")
    if q.dtype is not dt or out.dtype is not dt:
        raise TypeError(f"q and out must have the dtype of the cache, {dt}")
    qt, ot = q.stride(), out.stride()
    if d > 1 and (qt[-1] != 1 or ot[-1] != 1):
        raise ValueError("q and out need a unit innermost stride")
    if cu_draft is not None:
        qt, ot = (0, *qt), (0, *ot)
    ws, ws_bytes = (workspace.data_ptr(), workspace.numel() * workspace.element_size()) if workspace is not None else (0, 0)
    if cache_len is None:
        raise ValueError("cache_len is required")
    if check_device:  # written out, since a call of one token notices a loop
        dev = cache._device
        if not (dev is not None and dev >= 0 and (_current_device or _load_device())() == dev and
                q.get_device() == out.get_device() == cache_len.get_device() == dev and
                (parent is None or parent.get_device() == dev) and (cu_draft is None or cu_draft.get_device() == dev) and
                (cache_idx is None or cache_idx.get_device() == dev) and (err is None or err.get_device() == dev) and
                (workspace is None or workspace.get_device() == dev)):
            _one_device(q, out, *cache._tensors(), cache_len, parent, cu_draft, cache_idx, err, workspace)
    return TreeAttentionArgs.from_buffer_copy(_TREE_ATTENTION.pack(
        n, T, qs[-2], total, d ** -0.5 if scale is None else scale, wait_polls, cache._args(), q.data_ptr(), qt[0], qt[1], qt[2],
        out.data_ptr(), ot[0], ot[1], ot[2], cu_draft.data_ptr() if cu_draft is not None else 0,
        _exactly(parent, "parent", lead), _index_array(cache_len, "cache_len", n), _index_array(cache_idx, "cache_idx", n),
        _index_array(err, "err", n), ws, ws_bytes))


def tree_attention_workspace(q, out, cache, cache_len, **kw) -> int:
    """Bytes of workspace tree_attention needs for these arguments on the current device (0 = none)."""
    return _attention_workspace(make_tree_attention_args(q, out, cache, cache_len, check_device=False, **kw))


def _attention_workspace(a: TreeAttentionArgs) -> int:
    n = c_i64(0)
    rc = load_library().cv_tree_attention_workspace(ctypes.byref(a), ctypes.byref(n))
    if rc != 0:
        raise CvError(rc, "cv_tree_attention_workspace")
    return n.value


def tree_attention(q, out, cache, cache_len, *, parent=None, scale=None, cu_draft=None, T=None, cache_idx=None, err=None,
                   workspace=None, wait_polls=0, stream=None) -> None:
    """Queue attention of drafted tokens over a paged cache (cv_tree_attention).

    q, out [n_seq, T, n_heads, head_dim], or with cu_draft (int32 [n_seq + 1]) packed [total, n_heads, head_dim] rows, T then
    being the largest count; dtype of the cache, innermost stride 1, the others free.  cache_len int32 [n_seq]: tokens
    before the drafts, whose own K and V stand at positions cache_len .. cache_len + T - 1 already (qk_norm_rope writes
    them there).  parent int32 like q's rows: a draft attends to the cached tokens, its ancestors and itself; without parent
    to all drafts before it.  scale defaults to head_dim**-0.5.  Writes out (and err).  workspace: a uint8 buffer of
    tree_attention_workspace bytes; by default torch's allocator gives one for the call."""
    a = make_tree_attention_args(q, out, cache, cache_len, parent=parent, scale=scale, cu_draft=cu_draft, T=T,
                                 cache_idx=cache_idx, err=err, workspace=workspace, wait_polls=wait_polls)
    lib, on = load_library(), _stream_of(stream, q)
    rc = lib.cv_tree_attention(ctypes.byref(a), on)
    if rc == ERR_WORKSPACE and workspace is None:  # nothing was launched: this call needs one
        import torch
        if stream is not None and not isinstance(stream, torch.cuda.Stream):
            raise ValueError("pass workspace with a raw stream handle")
        need = _attention_workspace(a)
        # from the stream's own pool: a block freed on another stream may still be in use there
        with torch.cuda.stream(stream):
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        a.workspace, a.workspace_bytes = workspace.data_ptr(), need
        rc = lib.cv_tree_attention(ctypes.byref(a), on)
    if rc != 0:
        raise CvError(rc, "cv_tree_attention")


def make_draft_verify_args(probs, tokens, uniforms, accept_len, out_tokens, *, draft_probs=None, parent=None, path=None,
                           accept_node=None, cu_draft=None, T=None, cache_idx=None, err=None,
                           check_device=True) -> DraftVerifyArgs:
    """Build cv_draft_verify_args (see draft_verify)."""
    f32 = _f32 or _load_types()
    ps = probs.shape
    if len(ps) != (3 if cu_draft is None else 2):
        raise ValueError("probs must be [n_seq, T, vocab], or [total, vocab] with cu_draft")
    n, T, total, lead = _lead(ps, cu_draft, T, "probs")
    V, dt = ps[-1], probs.dtype
    pt = qt = probs.stride()
    if draft_probs is not None:
        qt = draft_probs.stride()
        if draft_probs.shape != ps or draft_probs.dtype is not dt:
            raise ValueError("draft_probs must have the shape and dtype of probs")
    if V > 1 and (pt[-1] != 1 or qt[-1] != 1):
        raise ValueError("probs and draft_probs need a unit innermost stride")
    if cu_draft is not None:
        pt, qt = (0, *pt), (0, *qt)
    if tokens is None or accept_len is None or out_tokens is None:
        raise ValueError("tokens, accept_len and out_tokens are required")
    if uniforms.dtype is not f32 or uniforms.shape != (n, T + 1) or not uniforms.is_contiguous():
        raise ValueError(f"uniforms must be contiguous float32 [{n}, {T + 1}]")
    if check_device:
        dev = probs.get_device()
        if not (dev >= 0 and (_current_device or _load_device())() == dev and
                tokens.get_device() == uniforms.get_device() == accept_len.get_device() == out_tokens.get_device() == dev and
                (draft_probs is None or draft_probs.get_device() == dev) and (parent is None or parent.get_device() == dev) and
                (path is None or path.get_device() == dev) and (accept_node is None or accept_node.get_device() == dev) and
                (cu_draft is None or cu_draft.get_device() == dev) and (cache_idx is None or cache_idx.get_device() == dev) and
                (err is None or err.get_device() == dev)):
            _one_device(probs, tokens, uniforms, accept_len, out_tokens, draft_probs, parent, path, accept_node, cu_draft, cache_idx, err)
    return DraftVerifyArgs.from_buffer_copy(_DRAFT_VERIFY.pack(
        n, T, V, BF16 if dt is _bf16 else _dtype_code(probs), total, probs.data_ptr(), pt[0], pt[1],
        draft_probs.data_ptr() if draft_probs is not None else 0, qt[0], qt[1], _exactly(tokens, "tokens", lead),
        _exactly(parent, "parent", lead), uniforms.data_ptr(), cu_draft.data_ptr() if cu_draft is not None else 0,
        _index_array(cache_idx, "cache_idx", n), _index_array(accept_len, "accept_len", n),
        _index_array(accept_node, "accept_node", n), _exactly(path, "path", (n, T)), _exactly(out_tokens, "out_tokens", (n, T)),
        _index_array(err, "err", n)))


def draft_verify(probs, tokens, uniforms, accept_len, out_tokens, *, draft_probs=None, parent=None, path=None, accept_node=None,
                 cu_draft=None, T=None, cache_idx=None, err=None, stream=None) -> None:
    """Queue the verification of drafted tokens (cv_draft_verify): which of them stand, and the token sampled after them.

    probs [n_seq, T, vocab] (bf16 or fp32): the target's distribution after each draft; tokens int32 [n_seq, T], token 0 the
    last step's; uniforms fp32 [n_seq, T + 1] in [0, 1): one for each draft's choice among its children, and the last for the
    new token.  draft_probs like probs (a chain only): row t is what token t was drawn from.  parent int32 [n_seq, T] for
    trees.  With cu_draft packed rows ([total, vocab], [total]), T being the largest count.  Writes accept_len int32
    [n_seq] (1 .. T: for conv_commit and LinattnDrafts of a chain), accept_node (1 + the last accepted token's index: for
    conv_commit of a tree), path int32 [n_seq, T] (for cache_compact), out_tokens int32 [n_seq, T] (this step's tokens: the
    accepted ones after token 0 and the new one, then -1), and err."""
    a = make_draft_verify_args(probs, tokens, uniforms, accept_len, out_tokens, draft_probs=draft_probs, parent=parent, path=path,
                               accept_node=accept_node, cu_draft=cu_draft, T=T, cache_idx=cache_idx, err=err)
    rc = load_library().cv_draft_verify(ctypes.byref(a), _stream_of(stream, probs))
    if rc != 0:
        raise CvError(rc, "cv_draft_verify")


def make_qk_norm_rope_args(q, k, q_out, *, k_out=None, v=None, cos_sin=None, q_weight=None, k_weight=None, norm=True, eps=1e-6,
                           pairs=False, positions=None, cache=None, cache_len=None, cu_seqlens=None, max_seqlen=None,
                           cache_idx=None, err=None, check_device=True) -> QkNormRopeArgs:
    """Build cv_qk_norm_rope_args (see qk_norm_rope)."""
    f32 = _f32 or _load_types()
    qs, dt = q.shape, q.dtype
    batch = cu_seqlens is None
    if len(qs) != (4 if batch else 3):
        raise ValueError("q must be [n_seq, T, n_heads, head_dim], or [total, n_heads, head_dim] with cu_seqlens")
    n, T, total, lead = _lead(qs, cu_seqlens, None if batch else max_seqlen, "q")
    if batch and max_seqlen is not None and max_seqlen < T:
        raise ValueError(f"max_seqlen = {max_seqlen} but q holds {T} tokens a sequence")
    d = qs[-1]
    if q_out is None or q_out.shape != qs:
        raise ValueError("q_out must have the shape of q")
    kv, ks = 0, None
    if k is not None:
        ks = k.shape
        kv = ks[-2]
        if ks[:-2] != lead or ks[-1] != d:
            raise ValueError(f"k must be [{', '.join(map(str, lead))}, heads, {d}], got {tuple(ks)}")
        if k_out is None and cache is None:
            raise ValueError("k needs k_out or a cache to be written to")
    if (k_out is not None and k_out.shape != ks) or (v is not None and v.shape != ks):
        raise ValueError("k_out and v must have the shape of k")
    packed = _NO_CACHE
    if cache is not None:
        if cache._layers:
            _one_layer(cache)
        if cache._heads != kv or cache._d != d or cache._dtype is not dt:
            raise ValueError("the cache must have the kv heads, head size and dtype of k")
        packed = cache._args()
        if cache_len is None:
            raise ValueError("cache_len is required")
    elif v is not None:
        raise ValueError("v needs a cache to be written to")

    def rows(t, name):  # pointer and (sequence, token, head) strides
        if t is None:
            return 0, 0, 0, 0
        if t.dtype is not dt:
            raise TypeError(f"{name} must have the dtype of q")
        st = t.stride()
        if st[-1] != 1 and d > 1:
            raise ValueError(f"{name} needs a unit innermost stride")
        return (t.data_ptr(), st[0], st[1], st[2]) if batch else (t.data_ptr(), 0, st[0], st[1])

    def weight(t, name):
        if t is None:
            return 0
        if t.dtype is not dt or t.shape != (d,) or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous [{d}] and have the dtype of q")
        return t.data_ptr()

    cs, cs_row, rot, n_pos = 0, 0, 0, 0
    if cos_sin is not None:
        if cos_sin.dtype is not f32 or cos_sin.dim() != 2 or (cos_sin.shape[1] > 1 and cos_sin.stride(1) != 1):
            raise ValueError("cos_sin must be float32 [n_positions, rot_dim] with a unit innermost stride")
        n_pos, rot = cos_sin.shape
        cs, cs_row = cos_sin.data_ptr(), cos_sin.stride(0) if n_pos > 1 else rot
        if positions is None and cache_len is None:
            raise ValueError("the rotation needs positions, or cache_len")
    if check_device:
        dev = q.get_device()
        if not (dev >= 0 and (_current_device or _load_device())() == dev and q_out.get_device() == dev and
                (k is None or k.get_device() == dev) and (k_out is None or k_out.get_device() == dev) and
                (v is None or v.get_device() == dev) and (cos_sin is None or cos_sin.get_device() == dev) and
                (q_weight is None or q_weight.get_device() == dev) and (k_weight is None or k_weight.get_device() == dev) and
                (positions is None or positions.get_device() == dev) and (cache_len is None or cache_len.get_device() == dev) and
                (cu_seqlens is None or cu_seqlens.get_device() == dev) and (cache_idx is None or cache_idx.get_device() == dev) and
                (err is None or err.get_device() == dev) and (cache is None or cache._device == dev)):
            _one_device(q, k, q_out, k_out, v, cos_sin, q_weight, k_weight, positions, cache_len, cu_seqlens, cache_idx, err,
                        *(cache._tensors() if cache is not None else ()))
    return QkNormRopeArgs.from_buffer_copy(_QK_NORM_ROPE.pack(
        n, T, qs[-2], kv, d, BF16 if dt is _bf16 else _dtype_code(q), total, rot, 1 if pairs else 0, 1 if norm else 0, n_pos, eps,
        *rows(q, "q"), *rows(q_out, "q_out"), *rows(k, "k"), *rows(k_out, "k_out"), *rows(v, "v"), weight(q_weight, "q_weight"),
        weight(k_weight, "k_weight"), cs, cs_row, _exactly(positions, "positions", lead),
        cu_seqlens.data_ptr() if cu_seqlens is not None else 0, _index_array(cache_len, "cache_len", n),
        _index_array(cache_idx, "cache_idx", n), packed, _index_array(err, "err", n)))


def qk_norm_rope(q, k, q_out, *, k_out=None, v=None, cos_sin=None, q_weight=None, k_weight=None, norm=True, eps=1e-6, pairs=False,
                 positions=None, cache=None, cache_len=None, cu_seqlens=None, max_seqlen=None, cache_idx=None, err=None,
                 stream=None) -> None:
    """Queue the norms of query and key heads and their rotation by position (cv_qk_norm_rope).

    q, q_out [n_seq, T, n_heads, head_dim] and k, k_out, v [n_seq, T, n_kv_heads, head_dim], or with cu_seqlens packed [total, ...]
    rows, max_seqlen then bounding the lengths; innermost stride 1, the others free (slices of one projection will do).  Every head
    is RMS-normed with q_weight or k_weight [head_dim] (norm False: not at all) and its first cos_sin.shape[1] channels rotated:
    cos_sin fp32 [n_positions, rot_dim], a row's cosines then its sines; pairs: neighbouring channels turn together, else
    channel i and i + rot_dim/2.  positions int32 like q's rows, by default cache_len + t.  With cache, K and V go to positions
    cache_len + t of the sequences' pages.  q_out may be q and k_out may be k."""
    a = make_qk_norm_rope_args(q, k, q_out, k_out=k_out, v=v, cos_sin=cos_sin, q_weight=q_weight, k_weight=k_weight, norm=norm,
                               eps=eps, pairs=pairs, positions=positions, cache=cache, cache_len=cache_len, cu_seqlens=cu_seqlens,
                               max_seqlen=max_seqlen, cache_idx=cache_idx, err=err)
    rc = load_library().cv_qk_norm_rope(ctypes.byref(a), _stream_of(stream, q))
    if rc != 0:
        raise CvError(rc, "cv_qk_norm_rope")


def make_cache_compact_args(cache, cache_len, path, accept_len, *, new_len=None, cache_idx=None, err=None,
                            check_device=True) -> CacheCompactArgs:
    """Build cv_cache_compact_args (see cache_compact)."""
    if path.dim() != 2:
        raise ValueError("path must be int32 [n_seq, T]")
    if cache_len is None or accept_len is None:
        raise ValueError("cache_len and accept_len are required")
    n, T = path.shape
    if check_device:
        dev = cache._device
        if not (dev is not None and dev >= 0 and (_current_device or _load_device())() == dev and
                path.get_device() == cache_len.get_device() == accept_len.get_device() == dev and
                (new_len is None or new_len.get_device() == dev) and (cache_idx is None or cache_idx.get_device() == dev) and
                (err is None or err.get_device() == dev)):
            _one_device(path, *cache._tensors(), cache_len, accept_len, new_len, cache_idx, err)
    return CacheCompactArgs.from_buffer_copy(_COMPACT.pack(
        n, T, cache._args(), _index_array(cache_len, "cache_len", n), _exactly(path, "path", (n, T)),
        _index_array(accept_len, "accept_len", n), _index_array(cache_idx, "cache_idx", n), _index_array(new_len, "new_len", n),
        _index_array(err, "err", n)))


def cache_compact(cache, cache_len, path, accept_len, *, new_len=None, cache_idx=None, err=None, stream=None) -> None:
    """Queue the move of each sequence's accepted path to its place in the cache (cv_cache_compact): row cache_len + path[s, i]
    of every layer's K and V goes to cache_len + i, i < accept_len[s].  path int32 [n_seq, T] as draft_verify leaves it.  new_len
    int32 [n_seq] receives cache_len + accept_len; it may not be cache_len itself."""
    a = make_cache_compact_args(cache, cache_len, path, accept_len, new_len=new_len, cache_idx=cache_idx, err=err)
    rc = load_library().cv_cache_compact(ctypes.byref(a), _stream_of(stream, path))
    if rc != 0:
        raise CvError(rc, "cv_cache_compact")


def make_cache_pages_args(cache, n_seq, *, idx=None, src_idx=None, n_tokens=None, err=None, cache_len=None,
                          check_device=True) -> CachePagesArgs:
    """Build cv_cache_pages_args (see cache_reserve, cache_fork and cache_free)."""
    if cache._held is None or cache._refs is None:
        raise ValueError("the cache needs held and refs")
    if check_device:
        dev = cache._device
        if not (dev is not None and dev >= 0 and (_current_device or _load_device())() == dev and
                (idx is None or idx.get_device() == dev) and (src_idx is None or src_idx.get_device() == dev) and
                (n_tokens is None or n_tokens.get_device() == dev) and (err is None or err.get_device() == dev) and
                (cache_len is None or cache_len.get_device() == dev)):
            _one_device(*cache._tensors(), idx, src_idx, n_tokens, err, cache_len)
    return CachePagesArgs.from_buffer_copy(_PAGES.pack(
        n_seq, cache._args(), _exactly(idx, "cache_idx", (n_seq,)), _exactly(src_idx, "src_idx", (n_seq,)),
        _exactly(n_tokens, "n_tokens", (n_seq,)), _index_array(err, "err", n_seq), _index_array(cache_len, "cache_len", n_seq)))


def cache_reserve(cache, n_tokens, *, cache_len=None, cache_idx=None, err=None, stream=None) -> None:
    """Queue the growth of slots (cv_cache_reserve): slot cache_idx[s] (default s) gets pages for n_tokens[s] tokens in all, the free
    pages with the lowest numbers, sequences in order.  With cache_len int32 [n_seq], the tokens that the slot has, positions cache_len[s] ..
    n_tokens[s] - 1 stand in pages of its own: one that another slot holds too is replaced by a copy (every layer), which a slot needs
    that was trimmed into pages shared by a fork."""
    a = make_cache_pages_args(cache, n_tokens.shape[0], idx=cache_idx, n_tokens=n_tokens, err=err, cache_len=cache_len)
    rc = load_library().cv_cache_reserve(ctypes.byref(a), _stream_of(stream, n_tokens))
    if rc != 0:
        raise CvError(rc, "cv_cache_reserve")


def cache_fork(cache, src_idx, dst_idx, n_tokens, *, err=None, stream=None) -> None:
    """Queue forks (cv_cache_fork): slot dst_idx[s], which holds no pages, gets the first n_tokens[s] tokens of slot src_idx[s]: full
    pages shared, the rest of the last one copied (every layer)."""
    a = make_cache_pages_args(cache, n_tokens.shape[0], idx=dst_idx, src_idx=src_idx, n_tokens=n_tokens, err=err)
    rc = load_library().cv_cache_fork(ctypes.byref(a), _stream_of(stream, n_tokens))
    if rc != 0:
        raise CvError(rc, "cv_cache_fork")


def cache_free(cache, n_tokens=None, *, cache_idx=None, err=None, stream=None) -> None:
    """Queue the release of pages (cv_cache_free): slot cache_idx[s] (default s) keeps those of its first n_tokens[s] tokens
    (default 0: none).  A page is free again once no slot holds it.  The last page kept may be shared with a fork: before more tokens are
    written there, cache_reserve with cache_len makes it the slot's own."""
    if n_tokens is None and cache_idx is None:
        n = cache.page_table.shape[0]
    else:
        n = (n_tokens if n_tokens is not None else cache_idx).shape[0]
    a = make_cache_pages_args(cache, n, idx=cache_idx, n_tokens=n_tokens, err=err)
    rc = load_library().cv_cache_free(ctypes.byref(a), _stream_of(stream, cache.page_table))
    if rc != 0:
        raise CvError(rc, "cv_cache_free")
