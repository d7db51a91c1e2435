"""Python binding of the GB300 ManifoldKV-style KV-cache compressor.

Thin ctypes marshalling over the C ABI in ``include/mkv.h`` (``libmkv.so``,
built in-tree by ``geometric_kv_cache_gb300.build``). Every step of the path
runs in the library's CUDA kernels; this module only turns torch tensors into
pointers and sizes, passes the current CUDA stream, and raises on a non-OK
status. There is no CPU fallback: without the compiled library, or without a
CUDA device, the calls raise.

Functions carry the C names (``mkv_centroid``, ``mkv_score``,
``mkv_select_topk``, ``mkv_compact``, ``mkv_compress``, ...). ``compress`` is
a convenience wrapper that allocates the outputs and the workspace with torch.
"""
from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

from . import build as _build

MKV_OK = 0
MKV_ERR_INVALID_ARG = 1
MKV_ERR_UNSUPPORTED = 2
MKV_ERR_WORKSPACE = 3
MKV_ERR_CUDA = 4
MKV_ERR_DEVICE = 5

MKV_DEV_BAD_SEQ_LEN = 0x1
MKV_DEV_BAD_N_KEEP = 0x2
MKV_DEV_INTERNAL = 0x4
MKV_DEV_TIMEOUT = 0x8
MKV_DEV_BAD_PAGE = 0x10
MKV_DEV_NO_PAGES = 0x20
MKV_DEV_BAD_PARENT = 0x40
MKV_DEV_BAD_TOKENS = 0x80
MKV_DEV_BAD_INDEX = 0x100

MKV_MODE_L2 = 0
MKV_MODE_COSINE = 1
_MODES = {"l2": MKV_MODE_L2, "cosine": MKV_MODE_COSINE, MKV_MODE_L2: MKV_MODE_L2, MKV_MODE_COSINE: MKV_MODE_COSINE}

MKV_ROPE_HALF = 0
MKV_ROPE_INTERLEAVED = 1
_ROPE_LAYOUTS = {"half": MKV_ROPE_HALF, "interleaved": MKV_ROPE_INTERLEAVED, MKV_ROPE_HALF: MKV_ROPE_HALF,
                 MKV_ROPE_INTERLEAVED: MKV_ROPE_INTERLEAVED}
_ROPE_SCALINGS = {"plain": 0, "linear": 1, "by_parts": 2, 0: 0, 1: 1, 2: 2}

HEAD_DIM = 128

# Every symbol include/mkv.h declares (checked by the tests).
EXPORTED = (
    "mkv_num_keep", "mkv_num_windows", "mkv_workspace_size", "mkv_centroid", "mkv_score",
    "mkv_select_topk", "mkv_compact", "mkv_compress", "mkv_compress_num_stages",
    "mkv_compress_profiled", "mkv_compress_host", "mkv_device_status", "mkv_status_string",
    "mkv_compress_noalloc", "mkv_compress_single_pass", "mkv_set_single_pass", "mkv_layer_budgets",
    "mkv_inject_stalled_windows", "mkv_window_means", "mkv_num_keep_quota", "mkv_select_quota",
    "mkv_compress_quota", "mkv_oja_workspace_size", "mkv_oja_score", "mkv_compress_oja", "mkv_oja_score_profiled",
    "mkv_compress_inplace", "mkv_set_head_groups", "mkv_set_fused", "mkv_centroid_score",
    "mkv_inject_stalled_fused", "mkv_set_head_group_ring", "mkv_head_group_plan", "mkv_set_oja_pair",
    "mkv_page_workspace_size", "mkv_page_update", "mkv_page_compact", "mkv_rope_append", "mkv_rope_frequencies",
    "mkv_attention_workspace_size", "mkv_paged_attention",
)


class MkvShape(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("t_max", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32), ("seq_lens", ctypes.c_void_p)]


class MkvPagePool(ctypes.Structure):
    _fields_ = [("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("k_pages", ctypes.c_void_p), ("v_pages", ctypes.c_void_p)]


class MkvPageLists(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("heads", ctypes.c_int32), ("max_pages", ctypes.c_int32),
                ("table", ctypes.c_void_p), ("lens", ctypes.c_void_p)]


class MkvNewTokens(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int32), ("q_heads", ctypes.c_int32), ("q_start", ctypes.c_void_p)]


# mkv_dtype of each supported cache element type
DTYPES = {torch.bfloat16: 0, torch.float8_e4m3fn: 1}


class MKVError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {mkv_status_string(status)}")


_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB_PATH


def load(build_if_missing: bool = True):
    """Load libmkv.so (building it first if it is missing and nvcc exists)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.LIB_PATH
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(f"{path} is missing: run geometric_kv_cache_gb300.build.build_library()")
            _build.build_library()
        lib = ctypes.CDLL(path)
        i32, u32, f64, vp, sz = ctypes.c_int32, ctypes.c_uint32, ctypes.c_double, ctypes.c_void_p, ctypes.c_size_t
        i64, f32 = ctypes.c_int64, ctypes.c_float
        sig = {
            "mkv_num_keep": (i32, [i32, f64]),
            "mkv_num_windows": (i32, [i32, i32]),
            "mkv_workspace_size": (sz, [MkvShape, i32]),
            "mkv_centroid": (i32, [vp, MkvShape, i32, vp, vp, sz, vp]),
            "mkv_score": (i32, [vp, vp, MkvShape, i32, i32, vp, vp, sz, vp]),
            "mkv_select_topk": (i32, [vp, MkvShape, f64, vp, vp, vp, sz, vp]),
            "mkv_compact": (i32, [vp, vp, vp, vp, MkvShape, f64, vp, i32, vp, vp, vp, vp, vp, sz, vp]),
            "mkv_compress": (i32, [vp, vp, MkvShape, f64, vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            "mkv_compress_num_stages": (i32, []),
            "mkv_compress_single_pass": (i32, [MkvShape, i32, i32]),
            "mkv_set_single_pass": (i32, [i32]),
            "mkv_set_head_groups": (i32, [i32]),
            "mkv_set_head_group_ring": (i32, [i32]),
            "mkv_head_group_plan": (i32, [MkvShape, i32, i32, ctypes.POINTER(i32)]),
            "mkv_set_fused": (i32, [i32, i32]),
            "mkv_set_oja_pair": (i32, [i32]),
            "mkv_centroid_score": (i32, [vp, MkvShape, i32, i32, vp, vp, vp, sz, vp]),
            "mkv_layer_budgets": (i32, [vp, i32, f64, f64, ctypes.c_int64, vp, vp]),
            "mkv_inject_stalled_windows": (i32, [vp, vp, MkvShape, f64, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            "mkv_inject_stalled_fused": (i32, [vp, vp, MkvShape, f64, i32, i32, vp, vp, vp, vp, i32, vp, sz, vp]),
            "mkv_compress_profiled": (i32, [vp, vp, MkvShape, f64, vp, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp,
                                            ctypes.POINTER(vp), i32]),
            "mkv_compress_host": (i32, [vp, vp, vp, vp, MkvShape, f64, i32, i32, i32, vp, vp, vp, vp,
                                        vp, vp, vp, vp, vp, sz, vp]),
            "mkv_device_status": (i32, [vp, vp, ctypes.POINTER(u32)]),
            "mkv_compress_noalloc": (i32, [vp, vp, MkvShape, f64, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp]),
            "mkv_status_string": (ctypes.c_char_p, [i32]),
            "mkv_window_means": (i32, [vp, MkvShape, i32, vp, vp, vp, sz, vp]),
            "mkv_oja_workspace_size": (sz, [MkvShape, i32]),
            "mkv_compress_inplace": (i32, [vp, vp, MkvShape, f64, vp, i32, i32, vp, vp, vp, sz, vp]),
            "mkv_oja_score": (i32, [vp, vp, vp, MkvShape, i32, i32, vp, vp, sz, vp]),
            "mkv_oja_score_profiled": (i32, [vp, vp, vp, MkvShape, i32, i32, vp, vp, sz, vp, ctypes.POINTER(vp), i32]),
            "mkv_compress_oja": (i32, [vp, vp, vp, vp, MkvShape, i32, i32, f64, vp, i32, vp, vp, vp, vp, vp, sz,
                                       vp]),
            "mkv_num_keep_quota": (i32, [i32, f64, i32]),
            "mkv_select_quota": (i32, [vp, MkvShape, f64, i32, i32, vp, vp, vp, sz, vp]),
            "mkv_compress_quota": (i32, [vp, vp, MkvShape, f64, i32, i32, i32, vp, vp, vp, vp, vp, sz, vp]),
            "mkv_page_workspace_size": (sz, [MkvPagePool, MkvPageLists]),
            "mkv_page_update": (i32, [MkvPagePool, MkvPageLists, vp, vp, vp, MkvPageLists, vp, vp, sz, vp]),
            "mkv_page_compact": (i32, [MkvPagePool, MkvPageLists, vp, vp, i32, vp, vp, vp, i32, vp, MkvPageLists, vp,
                                       vp, sz, vp]),
            "mkv_rope_append": (i32, [vp, i64, vp, i64, vp, i64, MkvNewTokens, vp, vp, i32, i32, f32, vp, MkvPagePool,
                                      MkvPageLists, f32, f32, vp, sz, vp]),
            "mkv_rope_frequencies": (i32, [i32, f64, i32, f64, i32, f64, f64, vp]),
            "mkv_attention_workspace_size": (sz, [MkvPagePool, MkvPageLists, MkvNewTokens, i32, i32]),
            "mkv_paged_attention": (i32, [vp, i64, MkvNewTokens, i32, MkvPagePool, MkvPageLists, i32, f32, f32, f32,
                                          i32, i32, vp, i64, vp, vp, sz, vp]),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


# ------------------------------------------------------------------ helpers --

def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _check(status: int, where: str):
    if status != MKV_OK:
        raise MKVError(status, where)


def _cache_types(*ts):
    """The cache tensors of one call (K, V and the compacted outputs) share one
    element type: the library reads them all with the shape's dtype."""
    types = {t.dtype for t in ts if t is not None}
    if len(types) > 1 or not types <= set(DTYPES):
        raise ValueError("K, V and the output caches must share one dtype: bf16 or float8_e4m3fn")


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors passed to the CUDA library must live on a CUDA device")
        if t is not None and not t.is_contiguous():
            raise ValueError("tensors passed to the CUDA library must be contiguous")


def shape_of(K: torch.Tensor, seq_lens: Optional[torch.Tensor] = None) -> MkvShape:
    """mkv_shape of a [batch, heads, t_max, head_dim] bf16 or float8_e4m3fn cache."""
    if K.dim() != 4 or K.dtype not in DTYPES:
        raise ValueError("K must be a bf16 or float8_e4m3fn tensor [batch, heads, t_max, head_dim]")
    if seq_lens is not None and (seq_lens.dtype != torch.int32 or seq_lens.numel() != K.shape[0]):
        raise ValueError("seq_lens must be int32 [batch]")
    b, h, t, d = K.shape
    return MkvShape(b, h, t, d, DTYPES[K.dtype], None if seq_lens is None else seq_lens.data_ptr())


def mkv_status_string(status: int) -> str:
    return load().mkv_status_string(int(status)).decode()


def mkv_num_keep(T: int, ratio: float) -> int:
    return int(load().mkv_num_keep(int(T), float(ratio)))


def mkv_num_windows(t_max: int, window: int) -> int:
    return int(load().mkv_num_windows(int(t_max), int(window)))


def mkv_workspace_size(shape: MkvShape, window: int = 0) -> int:
    return int(load().mkv_workspace_size(shape, int(window)))


def mkv_compress_num_stages() -> int:
    return int(load().mkv_compress_num_stages())


def mkv_compress_single_pass(shape: MkvShape, window: int = 0, mode="l2") -> int:
    """1 if mkv_compress reads K once for this shape on the current device."""
    return int(load().mkv_compress_single_pass(shape, int(window), _MODES[mode]))


def mkv_set_single_pass(enable: bool) -> bool:
    """Allow or forbid the single-pass centroid + score kernel; returns the
    previous setting."""
    return bool(load().mkv_set_single_pass(1 if enable else 0))


def mkv_set_head_groups(enable: bool) -> bool:
    """Allow or forbid the head-group kernel; returns the previous setting."""
    return bool(load().mkv_set_head_groups(1 if enable else 0))


def mkv_set_head_group_ring(enable: bool) -> bool:
    """Allow or forbid the copy-ring form of the head-group kernel (bf16,
    head dim 128); returns the previous setting."""
    return bool(load().mkv_set_head_group_ring(1 if enable else 0))


def mkv_head_group_plan(shape, window: int, mode) -> Optional[dict]:
    """The head-group plan on the current device (groups, CTAs per group,
    windows per unit, copy ring), or None when head groups do not apply."""
    out = (ctypes.c_int32 * 4)()
    if load().mkv_head_group_plan(shape, int(window), _MODES[mode], out) != 0:
        return None
    return {"groups": out[0], "gsize": out[1], "windows_per_unit": out[2], "ring": bool(out[3])}


def mkv_set_oja_pair(enable: bool) -> bool:
    """Run the OjaKV contraction (n_query <= 128) on pairs of CTAs (tcgen05
    cta_group::2, 256 tokens per MMA) or on one CTA per SM; returns the
    previous setting."""
    return bool(load().mkv_set_oja_pair(1 if enable else 0))


def mkv_set_fused(scorer_ctas: int, select_ctas: int = 0) -> int:
    """When mkv_compress runs the fused whole-path kernel: scorer_ctas < 0 on
    its own shape rule (the default), > 0 wherever it applies with that scorer
    budget (select_ctas > 0 sets the selector CTAs), 0 never. Returns the
    previous scorer setting."""
    return int(load().mkv_set_fused(int(scorer_ctas), int(select_ctas)))


def mkv_layer_budgets(sensitivity, r: float, gamma: float, total: int, cap):
    """Per-layer kept-token budgets (host helper). Returns (status, budgets)
    with budgets an int32 list of one entry per layer; status 1 means the caps
    absorb the whole total."""
    import array
    sv = array.array("d", [float(x) for x in sensitivity])
    cp = array.array("i", [int(x) for x in cap])
    out = array.array("i", [0] * len(sv))
    if len(cp) != len(sv):
        raise ValueError("one cap per layer is required")
    st = load().mkv_layer_budgets(ctypes.c_void_p(sv.buffer_info()[0]), len(sv), float(r), float(gamma), int(total),
                                  ctypes.c_void_p(cp.buffer_info()[0]), ctypes.c_void_p(out.buffer_info()[0]))
    if st < 0:
        raise MKVError(MKV_ERR_INVALID_ARG, "mkv_layer_budgets")
    return int(st), list(out)


def workspace_for(K: torch.Tensor, window: int = 0, seq_lens=None) -> torch.Tensor:
    """A zeroed workspace (uint8, 256-byte aligned by the caching allocator)."""
    n = mkv_workspace_size(shape_of(K, seq_lens), window)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=K.device)


# -------------------------------------------------------------- entry points --

def mkv_centroid(K, window, C, workspace, seq_lens=None, stream=None):
    _need_cuda(K, C, workspace, seq_lens)
    _check(load().mkv_centroid(_ptr(K), shape_of(K, seq_lens), int(window), _ptr(C), _ptr(workspace),
                               workspace.numel(), _stream(stream)), "mkv_centroid")


def mkv_window_means(X, window, mean, workspace, radius=None, seq_lens=None, stream=None):
    """Cluster summaries of a bf16 cache X (keys or values): fp32 window means
    [batch, heads, nw, 128] and, optionally, fp32 radii [batch, heads, nw]."""
    _need_cuda(X, mean, radius, workspace, seq_lens)
    _check(load().mkv_window_means(_ptr(X), shape_of(X, seq_lens), int(window), _ptr(mean), _ptr(radius),
                                   _ptr(workspace), workspace.numel(), _stream(stream)), "mkv_window_means")


def mkv_centroid_score(K, window, mode, C, S, workspace, seq_lens=None, stream=None):
    """Steps a1 + a2 as mkv_compress runs them (C and S as mkv_centroid / mkv_score write them)."""
    _need_cuda(K, C, S, workspace, seq_lens)
    _check(load().mkv_centroid_score(_ptr(K), shape_of(K, seq_lens), int(window), _MODES[mode], _ptr(C), _ptr(S),
                                     _ptr(workspace), workspace.numel(), _stream(stream)), "mkv_centroid_score")


def mkv_score(K, C, window, mode, S, workspace, seq_lens=None, stream=None):
    _need_cuda(K, C, S, workspace, seq_lens)
    _check(load().mkv_score(_ptr(K), _ptr(C), shape_of(K, seq_lens), int(window), _MODES[mode], _ptr(S),
                            _ptr(workspace), workspace.numel(), _stream(stream)), "mkv_score")


def mkv_select_topk(S, shape: MkvShape, ratio, cut, workspace, n_keep=None, stream=None):
    _need_cuda(S, cut, workspace, n_keep)
    _check(load().mkv_select_topk(_ptr(S), shape, float(ratio), _ptr(n_keep), _ptr(cut), _ptr(workspace),
                                  workspace.numel(), _stream(stream)), "mkv_select_topk")


def mkv_compact(S, cut, K, V, shape: MkvShape, ratio, keep_stride, idx, kept, K_out, V_out, workspace,
                n_keep=None, stream=None):
    _need_cuda(S, cut, K, V, idx, kept, K_out, V_out, workspace, n_keep)
    _cache_types(K, V, K_out, V_out)
    _check(load().mkv_compact(_ptr(S), _ptr(cut), _ptr(K), _ptr(V), shape, float(ratio), _ptr(n_keep),
                              int(keep_stride), _ptr(idx), _ptr(kept), _ptr(K_out), _ptr(V_out), _ptr(workspace),
                              workspace.numel(), _stream(stream)), "mkv_compact")


def mkv_compress(K, V, ratio, mode, window, keep_stride, K_out, V_out, idx, kept, workspace, seq_lens=None,
                 n_keep=None, stream=None):
    _need_cuda(K, V, K_out, V_out, idx, kept, workspace, seq_lens, n_keep)
    _cache_types(K, V, K_out, V_out)
    _check(load().mkv_compress(_ptr(K), _ptr(V), shape_of(K, seq_lens), float(ratio), _ptr(n_keep), _MODES[mode],
                               int(window), int(keep_stride), _ptr(K_out), _ptr(V_out), _ptr(idx), _ptr(kept),
                               _ptr(workspace), workspace.numel(), _stream(stream)), "mkv_compress")


def mkv_num_keep_quota(T: int, ratio: float, window: int) -> int:
    return int(load().mkv_num_keep_quota(int(T), float(ratio), int(window)))


def mkv_select_quota(S, shape: MkvShape, ratio, window, keep_stride, idx, kept, workspace, stream=None):
    _need_cuda(S, idx, kept, workspace)
    _check(load().mkv_select_quota(_ptr(S), shape, float(ratio), int(window), int(keep_stride), _ptr(idx),
                                   _ptr(kept), _ptr(workspace), workspace.numel(), _stream(stream)),
           "mkv_select_quota")


def mkv_compress_quota(K, V, ratio, mode, window, keep_stride, K_out, V_out, idx, kept, workspace, seq_lens=None,
                       stream=None):
    _need_cuda(K, V, K_out, V_out, idx, kept, workspace, seq_lens)
    _cache_types(K, V, K_out, V_out)
    _check(load().mkv_compress_quota(_ptr(K), _ptr(V), shape_of(K, seq_lens), float(ratio), _MODES[mode],
                                     int(window), int(keep_stride), _ptr(K_out), _ptr(V_out), _ptr(idx),
                                     _ptr(kept), _ptr(workspace), workspace.numel(), _stream(stream)),
           "mkv_compress_quota")


def mkv_oja_workspace_size(shape: MkvShape, n_query: int) -> int:
    return int(load().mkv_oja_workspace_size(shape, int(n_query)))


def oja_workspace_for(K: torch.Tensor, n_query: int, seq_lens=None) -> torch.Tensor:
    n = mkv_oja_workspace_size(shape_of(K, seq_lens), n_query)
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=K.device)


def mkv_oja_score(K, Q, U, S, workspace, seq_lens=None, stream=None):
    """OjaKV-style reconstruction-error scores: K [B, H, T, 128] bf16,
    Q [B, H, n_query, 128] bf16, U [B, H, 128, rank] fp32 -> S [B, H, T]."""
    _need_cuda(K, Q, U, S, workspace, seq_lens)
    _check(load().mkv_oja_score(_ptr(K), _ptr(Q), _ptr(U), shape_of(K, seq_lens), int(Q.shape[-2]),
                                int(U.shape[-1]), _ptr(S), _ptr(workspace), workspace.numel(), _stream(stream)),
           "mkv_oja_score")


def mkv_oja_score_profiled(K, Q, U, S, workspace, events, seq_lens=None, stream=None):
    """mkv_oja_score with three torch.cuda.Event objects recorded around its
    two kernels (query projection, contraction)."""
    _need_cuda(K, Q, U, S, workspace, seq_lens)
    s = torch.cuda.current_stream() if stream is None else stream
    for e in events:
        e.record(s)  # creates the event handles lazily; re-recorded below
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(load().mkv_oja_score_profiled(_ptr(K), _ptr(Q), _ptr(U), shape_of(K, seq_lens), int(Q.shape[-2]),
                                         int(U.shape[-1]), _ptr(S), _ptr(workspace), workspace.numel(),
                                         _stream(s), arr, len(events)), "mkv_oja_score_profiled")


def mkv_compress_oja(K, V, Q, U, ratio, keep_stride, K_out, V_out, idx, kept, workspace, seq_lens=None, n_keep=None,
                     stream=None):
    _need_cuda(K, V, Q, U, K_out, V_out, idx, kept, workspace, seq_lens, n_keep)
    _check(load().mkv_compress_oja(_ptr(K), _ptr(V), _ptr(Q), _ptr(U), shape_of(K, seq_lens), int(Q.shape[-2]),
                                   int(U.shape[-1]), float(ratio), _ptr(n_keep), int(keep_stride), _ptr(K_out),
                                   _ptr(V_out), _ptr(idx), _ptr(kept), _ptr(workspace), workspace.numel(),
                                   _stream(stream)), "mkv_compress_oja")


def mkv_compress_inplace(K, V, ratio, mode, window, workspace, idx=None, kept=None, seq_lens=None, n_keep=None,
                         stream=None):
    """Compress K and V in place: rows [0, kept) of every head become the
    kept rows; idx [B, H, t_max] and kept [B, H] are optional outputs."""
    _need_cuda(K, V, idx, kept, workspace, seq_lens, n_keep)
    _cache_types(K, V)
    _check(load().mkv_compress_inplace(_ptr(K), _ptr(V), shape_of(K, seq_lens), float(ratio), _ptr(n_keep),
                                       _MODES[mode], int(window), _ptr(idx), _ptr(kept), _ptr(workspace),
                                       workspace.numel(), _stream(stream)), "mkv_compress_inplace")


def mkv_compress_profiled(K, V, ratio, mode, window, keep_stride, K_out, V_out, idx, kept, workspace, events,
                          seq_lens=None, n_keep=None, stream=None):
    """mkv_compress with torch.cuda.Event objects recorded around each kernel."""
    _need_cuda(K, V, K_out, V_out, idx, kept, workspace, seq_lens, n_keep)
    _cache_types(K, V, K_out, V_out)
    st = torch.cuda.current_stream() if stream is None else stream
    for e in events:
        if not e.cuda_event:  # torch creates the CUDA event on its first record
            e.record(st)
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(load().mkv_compress_profiled(_ptr(K), _ptr(V), shape_of(K, seq_lens), float(ratio), _ptr(n_keep),
                                        _MODES[mode], int(window), int(keep_stride), _ptr(K_out), _ptr(V_out),
                                        _ptr(idx), _ptr(kept), _ptr(workspace), workspace.numel(), _stream(stream),
                                        arr, len(events)), "mkv_compress_profiled")


def mkv_compress_host(hK, hV, dK, dV, ratio, mode, window, keep_stride, dK_out, dV_out, d_idx, d_kept,
                      hK_out, hV_out, h_idx, h_kept, workspace, seq_lens=None, stream=None):
    """Host-resident cache: H2D copies, compress and D2H copies in one call."""
    _need_cuda(dK, dV, dK_out, dV_out, d_idx, d_kept, workspace, seq_lens)
    _cache_types(hK, hV, dK, dV, dK_out, dV_out, hK_out, hV_out)
    for t in (hK, hV, hK_out, hV_out, h_idx, h_kept):
        if t is not None and (t.is_cuda or not t.is_contiguous()):
            raise ValueError("host buffers must be contiguous CPU tensors (pinned for asynchrony)")
    _check(load().mkv_compress_host(_ptr(hK), _ptr(hV), _ptr(dK), _ptr(dV), shape_of(dK, seq_lens), float(ratio),
                                    _MODES[mode], int(window), int(keep_stride), _ptr(dK_out), _ptr(dV_out),
                                    _ptr(d_idx), _ptr(d_kept), _ptr(hK_out), _ptr(hV_out), _ptr(h_idx),
                                    _ptr(h_kept), _ptr(workspace), workspace.numel(), _stream(stream)),
           "mkv_compress_host")


def mkv_compress_noalloc(K, V, ratio, mode, window, keep_stride, K_out, V_out, idx, kept, status_out=None,
                         seq_lens=None, n_keep=None, stream=None):
    """mkv_compress without a workspace, for callers that cannot allocate
    device memory: the library uses its own fixed 32 MiB scratch array, so
    problems needing more scratch than that raise MKV_ERR_UNSUPPORTED, and
    calls must not overlap on the GPU. ``status_out`` (int32/uint32 [1] on
    the device, optional) receives the call's device status bits."""
    _need_cuda(K, V, K_out, V_out, idx, kept, status_out, seq_lens, n_keep)
    _cache_types(K, V, K_out, V_out)
    _check(load().mkv_compress_noalloc(_ptr(K), _ptr(V), shape_of(K, seq_lens), float(ratio), _ptr(n_keep),
                                       _MODES[mode], int(window), int(keep_stride), _ptr(K_out), _ptr(V_out),
                                       _ptr(idx), _ptr(kept), _ptr(status_out), _stream(stream)),
           "mkv_compress_noalloc")


def mkv_inject_stalled_windows(K, V, ratio, mode, window, keep_stride, K_out, V_out, idx, kept, workspace,
                               seq_lens=None, stream=None):
    """Failure injection: the single-pass kernel with no window ever
    completing; every wait between CTAs must run out (MKV_DEV_TIMEOUT)."""
    _need_cuda(K, V, K_out, V_out, idx, kept, workspace, seq_lens)
    _cache_types(K, V, K_out, V_out)
    _check(load().mkv_inject_stalled_windows(_ptr(K), _ptr(V), shape_of(K, seq_lens), float(ratio), _MODES[mode],
                                             int(window), int(keep_stride), _ptr(K_out), _ptr(V_out), _ptr(idx),
                                             _ptr(kept), _ptr(workspace), workspace.numel(), _stream(stream)),
           "mkv_inject_stalled_windows")


def mkv_inject_stalled_fused(K, V, ratio, mode, keep_stride, K_out, V_out, idx, kept, stage, workspace,
                             seq_lens=None, stream=None):
    """Failure injection: the fused whole-path kernel with one wait that
    cannot end (stage 0: scorer group 0's barrier; stage 1: head 0's select);
    it must run out (MKV_DEV_TIMEOUT) and the rest of the launch drain."""
    _need_cuda(K, V, K_out, V_out, idx, kept, workspace, seq_lens)
    _cache_types(K, V, K_out, V_out)
    _check(load().mkv_inject_stalled_fused(_ptr(K), _ptr(V), shape_of(K, seq_lens), float(ratio), _MODES[mode],
                                           int(keep_stride), _ptr(K_out), _ptr(V_out), _ptr(idx), _ptr(kept),
                                           int(stage), _ptr(workspace), workspace.numel(), _stream(stream)),
           "mkv_inject_stalled_fused")


# --------------------------------------------------------------- paged caches --

# (The checks below run on every step of a serving loop: plain comparisons, no
# temporary objects.)

def _on_device(ts) -> int:
    """The one CUDA device of a call's tensors, which must be the current one
    (the launches go to a stream of the current device)."""
    dev = torch._C._cuda_getDevice() if torch.cuda.is_initialized() else -2
    for t in ts:
        if t is not None and t.get_device() != dev:
            if not t.is_cuda:
                raise ValueError("tensors passed to the CUDA library must live on a CUDA device")
            if dev == -2 and t.get_device() == torch.cuda.current_device():
                dev = t.get_device()
                continue
            raise ValueError("tensors of one call must live on one CUDA device, the current one")
    return dev


def _raw_stream(stream, dev) -> int:
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _int32(t, shape, what):
    if t is not None and (t.dtype is not torch.int32 or t.shape != shape or not t.is_contiguous()):
        raise ValueError(f"{what} must be a contiguous int32 tensor {list(shape)}")


def _at(t):
    return None if t is None else t.data_ptr()


def _workspace(ws):
    if ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous uint8 tensor")


def pool_of(k_pages: torch.Tensor, v_pages: torch.Tensor) -> MkvPagePool:
    """mkv_page_pool of two [n_pages, page_size, head_dim] bf16 or float8_e4m3fn tensors."""
    dtype, shape = DTYPES.get(k_pages.dtype), k_pages.shape
    if len(shape) != 3 or dtype is None:
        raise ValueError("k_pages must be a bf16 or float8_e4m3fn tensor [n_pages, page_size, head_dim]")
    if v_pages.shape != shape or v_pages.dtype is not k_pages.dtype:
        raise ValueError("k_pages and v_pages must have one shape and dtype")
    if not (k_pages.is_contiguous() and v_pages.is_contiguous()):
        raise ValueError("k_pages and v_pages must be contiguous")
    n, p, d = shape
    return MkvPagePool(n, p, d, dtype, k_pages.data_ptr(), v_pages.data_ptr())


def lists_of(table: torch.Tensor, lens: Optional[torch.Tensor] = None) -> MkvPageLists:
    """mkv_page_lists of table int32 [batch, heads, max_pages] and lens int32 [batch, heads]."""
    shape = table.shape
    if len(shape) != 3:
        raise ValueError("table must be an int32 tensor [batch, heads, max_pages]")
    b, h, m = shape
    _int32(table, shape, "table")
    _int32(lens, (b, h), "lens")
    return MkvPageLists(b, h, m, table.data_ptr(), None if lens is None else lens.data_ptr())


def _token_rows(t, heads, d, n_tokens, what):
    """Stride (elements) between the tokens of a bf16 [n_tokens, heads, d] tensor, whose tokens may lie apart."""
    if t.dtype is not torch.bfloat16 or t.shape != (n_tokens, heads, d):
        raise ValueError(f"{what} must be a bf16 tensor [{n_tokens}, {heads}, {d}]")
    if n_tokens == 0:
        return heads * d
    s0, s1, s2 = t.stride()
    if (heads > 1 and s1 != d) or s2 != 1:
        raise ValueError(f"the heads of one token of {what} must be contiguous")
    return heads * d if n_tokens == 1 else s0


def page_workspace_for(k_pages: torch.Tensor, table: torch.Tensor) -> torch.Tensor:
    """A zeroed workspace for mkv_page_update, mkv_page_compact and mkv_rope_append."""
    n = int(load().mkv_page_workspace_size(pool_of(k_pages, k_pages), lists_of(table)))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=k_pages.device)


def mkv_page_update(k_pages, v_pages, table, lens, refs, table_out, lens_out, refs_out, workspace, parent=None,
                    n_new=None, stream=None):
    """Page lists after a step: row b continues row parent[b] (-1: it ends; None: itself) and grows by n_new[b]
    tokens. table int32 [batch, heads, max_pages], lens int32 [batch, heads], refs int32 [n_pages]; parent and n_new
    int32 [batch]. Full pages are shared, partly filled last pages copied for all but one child. With parent None,
    table_out and lens_out may be table and lens; refs_out may always be refs."""
    dev = _on_device((k_pages, v_pages, table, lens, refs, table_out, lens_out, refs_out, workspace, parent, n_new))
    pool, src, dst = pool_of(k_pages, v_pages), lists_of(table, lens), lists_of(table_out, lens_out)
    _int32(refs, (pool.n_pages,), "refs")
    _int32(refs_out, (pool.n_pages,), "refs_out")
    _int32(parent, (src.batch,), "parent")
    _int32(n_new, (src.batch,), "n_new")
    _workspace(workspace)
    _check((_lib or load()).mkv_page_update(pool, src, refs.data_ptr(), _at(parent), _at(n_new), dst, refs_out.data_ptr(),
                                            workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev)),
           "mkv_page_update")


def mkv_page_compact(k_pages, v_pages, table, lens, refs, idx, kept, table_out, lens_out, refs_out, workspace, K=None,
                     V=None, seq_lens=None, stream=None):
    """Compaction in pages: list h keeps its tokens idx[h][:kept[h]] in new pages, its old pages lose a holder. idx
    int32 [batch, heads, n] (None: the first kept tokens, not the same as n = 0), kept int32 [batch, heads], as mkv_compress writes them.
    With K and V [batch, heads, t_max, head_dim] (and seq_lens) the tokens come from that contiguous cache instead."""
    dev = _on_device((k_pages, v_pages, table, lens, refs, idx, kept, table_out, lens_out, refs_out, workspace, K, V,
                      seq_lens))
    pool, src, dst = pool_of(k_pages, v_pages), lists_of(table, lens), lists_of(table_out, lens_out)
    _int32(refs, (pool.n_pages,), "refs")
    _int32(refs_out, (pool.n_pages,), "refs_out")
    _int32(kept, (src.batch, src.heads), "kept")
    if idx is not None:
        _int32(idx, (src.batch, src.heads, idx.shape[-1]), "idx")
    _workspace(workspace)
    t_max = 0
    if (K is None) != (V is None) or (K is None and seq_lens is not None):
        raise ValueError("K and V come together (and seq_lens only with them)")
    if K is not None:
        if K.dtype is not k_pages.dtype or V.dtype is not k_pages.dtype:
            raise ValueError("K, V and the pages must share one dtype: bf16 or float8_e4m3fn")
        t_max = K.shape[2] if K.dim() == 4 else 0
        if K.shape != (src.batch, src.heads, t_max, pool.head_dim) or V.shape != K.shape:
            raise ValueError("K and V must be [batch, heads, t_max, head_dim] of the lists' sizes")
        if not (K.is_contiguous() and V.is_contiguous()):
            raise ValueError("tensors passed to the CUDA library must be contiguous")
        _int32(seq_lens, (src.batch,), "seq_lens")
    # (a tensor without elements has no address, and to the library NULL means that there is none at all)
    some = workspace.data_ptr()
    _check((_lib or load()).mkv_page_compact(pool, src, refs.data_ptr(), None if idx is None else idx.data_ptr() or some,
                                             0 if idx is None else idx.shape[-1], kept.data_ptr(),
                                             None if K is None else K.data_ptr() or some,
                                             None if V is None else V.data_ptr() or some, t_max, _at(seq_lens), dst,
                                             refs_out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                             _raw_stream(stream, dev)), "mkv_page_compact")


def mkv_rope_frequencies(rot_dim: int, theta: float, scaling="plain", scale: float = 1.0, original_len: int = 0,
                         low_turns: float = 0.0, high_turns: float = 0.0) -> torch.Tensor:
    """Rotary frequencies (host helper): fp32 [rot_dim / 2] on the CPU. scaling "plain", "linear" (all divided by
    scale) or "by_parts" (pairs of fewer than low_turns turns over original_len positions divided by scale, pairs of
    more than high_turns kept, a ramp between)."""
    out = torch.empty(max(int(rot_dim) // 2, 0), dtype=torch.float32)
    st = load().mkv_rope_frequencies(int(rot_dim), float(theta), _ROPE_SCALINGS[scaling], float(scale),
                                     int(original_len), float(low_turns), float(high_turns), _ptr(out))
    if st != 0:
        raise MKVError(MKV_ERR_INVALID_ARG, "mkv_rope_frequencies")
    return out


def mkv_rope_append(Q, K, V, positions, inv_freq, k_pages, v_pages, table, lens, q_start, Q_out, workspace,
                    layout="half", factor: float = 1.0, k_scale: float = 1.0, v_scale: float = 1.0, stream=None):
    """Rotary positions of a step's new tokens: Q [n_tokens, q_heads, d] turned into Q_out, K [n_tokens, heads, d]
    turned into the pages, V into the pages (all bf16; tokens may lie apart, as in a fused projection). Row b's tokens
    are [q_start[b], q_start[b + 1]) and the last ones of its lists. inv_freq fp32 [rot_dim / 2] on the device."""
    dev = _on_device((Q, K, V, positions, inv_freq, k_pages, v_pages, table, lens, q_start, Q_out, workspace))
    pool, lists = pool_of(k_pages, v_pages), lists_of(table, lens)
    if Q.dim() != 3:
        raise ValueError("Q must be a bf16 tensor [n_tokens, q_heads, head_dim]")
    n, hq, d = Q.shape[0], Q.shape[1], pool.head_dim
    qs = _token_rows(Q, hq, d, n, "Q")
    ks, vs = _token_rows(K, lists.heads, d, n, "K"), _token_rows(V, lists.heads, d, n, "V")
    _token_rows(Q_out, hq, d, n, "Q_out")
    if not Q_out.is_contiguous():
        raise ValueError("Q_out must be contiguous")
    _int32(positions, (n,), "positions")
    _int32(q_start, (lists.batch + 1,), "q_start")
    if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be a contiguous fp32 tensor [rot_dim / 2]")
    _workspace(workspace)
    _check((_lib or load()).mkv_rope_append(
        Q.data_ptr(), qs, K.data_ptr(), ks, V.data_ptr(), vs, MkvNewTokens(n, hq, q_start.data_ptr()), positions.data_ptr(),
        inv_freq.data_ptr(), 2 * inv_freq.shape[0], _ROPE_LAYOUTS[layout], factor, Q_out.data_ptr(), pool, lists, k_scale,
        v_scale, workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev)), "mkv_rope_append")


def attention_workspace_for(Q, k_pages, table, max_q: int, max_len: int) -> torch.Tensor:
    """A zeroed workspace for mkv_paged_attention on these shapes."""
    n = int(load().mkv_attention_workspace_size(pool_of(k_pages, k_pages), lists_of(table),
                                                MkvNewTokens(Q.shape[0], Q.shape[1], None), int(max_q), int(max_len)))
    return torch.zeros(max(n, 256), dtype=torch.uint8, device=Q.device)


def mkv_paged_attention(Q, k_pages, v_pages, table, lens, q_start, max_q: int, max_len: int, O, workspace,
                        scale: Optional[float] = None, k_scale: float = 1.0, v_scale: float = 1.0, window: int = 0,
                        sinks: int = 0, lse=None, stream=None):
    """Attention of new tokens Q bf16 [n_tokens, q_heads, d] over the paged cache, into O (like Q) and, if given, lse
    fp32 [n_tokens, q_heads]. Row b's tokens are [q_start[b], q_start[b + 1]) and the last ones of its lists; each sees
    the tokens up to its own, with window > 0 the last `window` of them and the first `sinks`. max_q and max_len bound
    the rows' new tokens and the lists' lengths. scale defaults to 1 / sqrt(d)."""
    dev = _on_device((Q, k_pages, v_pages, table, lens, q_start, O, workspace, lse))
    pool, lists = pool_of(k_pages, v_pages), lists_of(table, lens)
    if Q.dim() != 3:
        raise ValueError("Q must be a bf16 tensor [n_tokens, q_heads, head_dim]")
    n, hq, d = Q.shape[0], Q.shape[1], pool.head_dim
    qs, os_ = _token_rows(Q, hq, d, n, "Q"), _token_rows(O, hq, d, n, "O")
    _int32(q_start, (lists.batch + 1,), "q_start")
    if max(max_q, max_len, window, sinks) > 0x7FFFFFFF:
        raise ValueError("max_q, max_len, window and sinks are 32-bit numbers")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (n, hq) or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous fp32 tensor [n_tokens, q_heads]")
    _workspace(workspace)
    _check((_lib or load()).mkv_paged_attention(
        Q.data_ptr(), qs, MkvNewTokens(n, hq, q_start.data_ptr()), max_q, pool, lists, max_len,
        d ** -0.5 if scale is None else scale, k_scale, v_scale, window, sinks, O.data_ptr(), os_, _at(lse),
        workspace.data_ptr(), workspace.numel(), _raw_stream(stream, dev)), "mkv_paged_attention")


def mkv_device_status(workspace, stream=None) -> int:
    """Synchronise, return the status bits of ``workspace`` and clear them."""
    bits = ctypes.c_uint32(0)
    st = load().mkv_device_status(_ptr(workspace), _stream(stream), ctypes.byref(bits))
    if st not in (MKV_OK, MKV_ERR_DEVICE):
        raise MKVError(st, "mkv_device_status")
    return int(bits.value)


# ---------------------------------------------------------------- convenience --

def compress(K, V, ratio: float, mode="l2", window: int = 0, seq_lens=None, n_keep=None,
             keep_stride: Optional[int] = None, workspace=None, stream=None):
    """Compress a bf16 cache [batch, heads, t_max, 128]; returns
    (K_out, V_out, idx, kept) with K_out/V_out [batch, heads, keep_stride, 128]."""
    if keep_stride is None:
        keep_stride = mkv_num_keep(K.shape[2], ratio) if n_keep is None else int(n_keep.max().item())
    b, h = K.shape[0], K.shape[1]
    K_out = torch.empty((b, h, keep_stride, K.shape[3]), dtype=K.dtype, device=K.device)
    V_out = torch.empty_like(K_out)
    idx = torch.empty((b, h, keep_stride), dtype=torch.int32, device=K.device)
    kept = torch.empty((b, h), dtype=torch.int32, device=K.device)
    ws = workspace if workspace is not None else workspace_for(K, window, seq_lens)
    mkv_compress(K, V, ratio, mode, window, keep_stride, K_out, V_out, idx, kept, ws, seq_lens, n_keep, stream)
    return K_out, V_out, idx, kept
