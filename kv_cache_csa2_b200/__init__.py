"""Python binding of libcsa2 (the CSA2 hot path on B200).

Argument marshalling only: every step of the path runs in the CUDA kernels of
``libcsa2.so``; PyTorch supplies device memory and streams.  The functions
carry the C ABI's names (include/csa2.h) and take torch CUDA tensors.  If the
library is not built, importing works but the first call raises.
"""
from __future__ import annotations

import ctypes
import os

__all__ = [
    "CSA2Error", "lib", "lib_path", "FULL", "REINDEX", "REUSE", "KV_BF16", "KV_FP4", "ACT_RELU",
    "ACT_IDENTITY", "csa2_compress", "csa2_index_scores", "csa2_select_topk", "csa2_select_topk_noalloc",
    "csa2_index_topk",
    "csa2_sparse_attn", "csa2_sparse_attn_swa", "csa2_dense_attn", "csa2_compress_hca",
    "csa2_index_scores_fp4", "csa2_index_topk_fp4",
    "csa2_fp4_pack", "csa2_fp4_unpack", "Group", "csa2_device_error",
    "KV_F16", "Rope", "PagedKv", "csa2_qk_norm_rope", "csa2_paged_append", "csa2_paged_decode_attn",
    "csa2_paged_window_attn",
    "launch_counts", "reset_launch_counts", "set_fault", "set_device_wait", "EXPORTED_SYMBOLS",
]

FULL, REINDEX, REUSE = 0, 1, 2
KV_BF16, KV_FP4, KV_F16 = 0, 1, 2
ACT_RELU, ACT_IDENTITY = 0, 1
_MODE = {"full": FULL, "reindex": REINDEX, "reuse": REUSE, FULL: FULL, REINDEX: REINDEX,
         REUSE: REUSE}

_P, _I, _I64, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class CSA2Kv(ctypes.Structure):
    _fields_ = [("fmt", _I), ("data", _P), ("scales", _P), ("n", _I64), ("dim", _I)]


class CSA2GroupDesc(ctypes.Structure):
    _fields_ = [("B", _I), ("Q", _I), ("N", _I64), ("D", _I), ("Ha", _I), ("Hi", _I), ("d", _I),
                ("k", _I), ("P", _I), ("scale", _F), ("kv_fmt", _I), ("act", _I),
                ("n_layers", _I), ("modes", ctypes.POINTER(_I))]


class CSA2LayerIO(ctypes.Structure):
    _fields_ = [("kv", CSA2Kv), ("index_k", _P), ("n_visible", _P), ("q_index", _P),
                ("w_index", _P), ("q_attn", _P), ("out", _P), ("lse", _P),
                ("swa_kv", _P), ("swa_rows", _I64), ("swa_end", _P), ("swa_window", _I)]


class CSA2Heads(ctypes.Structure):
    _fields_ = [("data", _P), ("heads", _I), ("token_stride", _I64), ("head_stride", _I64)]


class CSA2Rope(ctypes.Structure):
    _fields_ = [("inv_freq", _P), ("half", _I), ("offset", _I), ("interleaved", _I), ("inverse", _I)]


class CSA2PagedKv(ctypes.Structure):
    _fields_ = [("fmt", _I), ("k", _P), ("v", _P), ("k_scales", _P), ("v_scales", _P), ("n_pages", _I64),
                ("page_stride", _I64), ("token_stride", _I64), ("head_stride", _I64), ("page_size", _I),
                ("heads", _I), ("dim", _I), ("B", _I), ("max_pages", _I), ("table_stride", _I64),
                ("table", _P), ("lens", _P), ("max_len", _I64)]


_HEADS, _ROPE, _PAGED = ctypes.POINTER(CSA2Heads), ctypes.POINTER(CSA2Rope), ctypes.POINTER(CSA2PagedKv)

# name -> (restype, argtypes); every symbol include/csa2.h declares
_SIGS = {
    "csa2_compress": (_I, [_P, _P, _P, _I, _I64, _I, _I, _I, _P, _I64, _P]),
    "csa2_index_scores": (_I, [_P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _I, _I, _P, _P]),
    "csa2_select_topk_workspace": (_SZ, [_I64, _I64, _I]),
    "csa2_select_topk": (_I, [_P, _I64, _I64, _I, _P, _P, _P, _SZ, _P]),
    "csa2_select_topk_noalloc": (_I, [_P, _I64, _I64, _I, _P, _P, _P]),
    "csa2_index_topk_workspace": (_SZ, [_I, _I, _I64, _I, _I, _I]),
    "csa2_index_topk": (_I, [_I, _P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _I, _I, _P, _P, _I, _I,
                             _P, _SZ, _P]),
    "csa2_sparse_attn_workspace": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "csa2_sparse_attn": (_I, [_I, _P, ctypes.POINTER(CSA2Kv), _P, _I, _I, _I, _I, _F, _P, _P, _P,
                              _SZ, _P]),
    "csa2_index_scores_fp4": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _I, _I, _P, _P]),
    "csa2_index_topk_fp4": (_I, [_I, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I64, _P, _P, _I, _I, _P, _P,
                                 _I, _I, _P, _SZ, _P]),
    "csa2_sparse_attn_swa_workspace": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "csa2_sparse_attn_swa": (_I, [_I, _P, ctypes.POINTER(CSA2Kv), _P, _I, _I, _I, _I, _F, _P, _I64,
                                  _P, _I, _P, _P, _P, _SZ, _P]),
    "csa2_dense_attn_workspace": (_SZ, [_I, _I, _I, _I, _I64, _I]),
    "csa2_dense_attn": (_I, [_P, ctypes.POINTER(CSA2Kv), _P, _I, _I, _I, _F, _P, _P, _P, _SZ, _P]),
    "csa2_compress_hca": (_I, [_P, _P, _P, _I, _I64, _I, _I, _P, _I64, _P]),
    "csa2_fp4_pack": (_I, [_P, _I64, _I, _P, _P, _P]),
    "csa2_fp4_unpack": (_I, [_P, _P, _I64, _I, _P, _P]),
    "csa2_qk_norm_rope": (_I, [_I, _HEADS, _P, _HEADS, _HEADS, _P, _HEADS, _I64, _I, _F, _P, _ROPE, _P]),
    "csa2_paged_append": (_I, [_I, _HEADS, _HEADS, _P, _P, _I64, _ROPE, _PAGED, _P]),
    "csa2_paged_decode_attn_workspace": (_SZ, [_PAGED, _I, _I, _I, _I]),
    "csa2_paged_decode_attn": (_I, [_HEADS, _PAGED, _F, _I, _I, _I, _P, _P, _P, _SZ, _P]),
    "csa2_paged_window_attn": (_I, [_HEADS, _P, _I64, _PAGED, _F, _I, _I, _P, _P, _P]),
    "csa2_group_create": (_I, [ctypes.POINTER(_P), ctypes.POINTER(CSA2GroupDesc)]),
    "csa2_group_layer": (_I, [_P, _I, ctypes.POINTER(CSA2LayerIO), _P]),
    "csa2_group_selection": (_I, [_P, ctypes.POINTER(_P), ctypes.POINTER(_P)]),
    "csa2_group_copy_selection": (_I, [_P, _P, _P, _P]),
    "csa2_group_destroy": (None, [_P]),
    "csa2_status_string": (ctypes.c_char_p, [_I]),
    "csa2_last_error": (ctypes.c_char_p, []),
    "csa2_device_error": (_I, [_P]),
    "csa2_launch_counts": (_I, [ctypes.POINTER(_I64), _I]),
    "csa2_reset_launch_counts": (None, []),
    "csa2_set_fault": (_I, [ctypes.c_char_p]),
    "csa2_set_device_wait": (_I, [ctypes.c_uint64, _I]),
    "csa2_timing_enable": (_I, [_I]),
    "csa2_kernel_times": (_I, [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_I64), _I]),
    "csa2_timing_reset": (None, []),
    "csa2_version": (_I, []),
}
EXPORTED_SYMBOLS = tuple(_SIGS)

_LIB = None


def lib_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "libcsa2.so")


def lib():
    """Load libcsa2.so (raises if it is missing: there is no fallback path)."""
    global _LIB
    if _LIB is None:
        path = lib_path()
        if not os.path.exists(path):
            raise ImportError(f"{path} is not built; run `python -m kv_cache_csa2_b200.build`")
        L = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


class CSA2Error(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{lib().csa2_status_string(status).decode()}: {msg}")
        self.status = status


def _check(status: int) -> None:
    if status != 0:
        raise CSA2Error(status, lib().csa2_last_error().decode(errors="replace"))


def _torch():
    import torch
    return torch


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    torch = _torch()
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _need(t, dtype, ndim, name):
    torch = _torch()
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype != dtype or t.dim() != ndim or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous CUDA {dtype} with {ndim} dims, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t


# ------------------------------------------------------------------ (a1)
def csa2_compress(c, z, bias, m: int, has_left_halo: bool = False, out=None,
                  out_batch_stride: int = 0, stream=None):
    """Compress raw tokens (c bf16 / z f32 [B, T+halo, D], bias f32 [2m, D]) into entries."""
    torch = _torch()
    _need(c, torch.bfloat16, 3, "c")
    _need(z, torch.float32, 3, "z")
    _need(bias, torch.float32, 2, "bias")
    B, t_in, D = c.shape
    T = t_in - (m if has_left_halo else 0)
    if out is None:
        out = torch.empty(B, T // m, D, dtype=torch.bfloat16, device=c.device)
    _check(lib().csa2_compress(_ptr(c), _ptr(z), _ptr(bias), B, T, D, m, int(has_left_halo),
                               _ptr(out), out_batch_stride, _stream(stream)))
    return out


# ------------------------------------------------------------------ (a2, a3)
def csa2_index_scores(q, w, k, n_visible=None, pool=None, act: int = ACT_RELU, out=None,
                      stream=None):
    torch = _torch()
    _need(q, torch.bfloat16, 4, "q")
    _need(w, torch.float32, 3, "w")
    _need(k, torch.bfloat16, 3, "k")
    B, Q, H, d = q.shape
    N = k.shape[1]
    P = pool.shape[2] if pool is not None else 0
    if pool is not None:
        _need(pool, torch.int32, 3, "pool")
    if n_visible is not None:
        _need(n_visible, torch.int32, 2, "n_visible")
    if out is None:
        out = torch.empty(B, Q, P if pool is not None else N, dtype=torch.float32, device=q.device)
    _check(lib().csa2_index_scores(_ptr(q), _ptr(w), _ptr(k), B, Q, H, d, N, _ptr(n_visible),
                                   _ptr(pool), P, act, _ptr(out), _stream(stream)))
    return out


def csa2_index_scores_fp4(q_codes, q_scales, w, k_codes, k_scales, n_visible=None, pool=None,
                          act: int = ACT_RELU, out=None, stream=None):
    """FP4 indexer: q codes/scales [B,Q,H,d/2]/[B,Q,H,d/16], K codes/scales
    [B,N,d/2]/[B,N,d/16] (csa2_fp4_pack's format); returns bf16 scores."""
    torch = _torch()
    _need(q_codes, torch.uint8, 4, "q_codes")
    _need(k_codes, torch.uint8, 3, "k_codes")
    _need(w, torch.float32, 3, "w")
    B, Q, H, d2 = q_codes.shape
    N = k_codes.shape[1]
    P = pool.shape[2] if pool is not None else 0
    if out is None:
        out = torch.empty(B, Q, P if pool is not None else N, dtype=torch.bfloat16, device=q_codes.device)
    _check(lib().csa2_index_scores_fp4(_ptr(q_codes), _ptr(q_scales), _ptr(w), _ptr(k_codes),
                                       _ptr(k_scales), B, Q, H, 2 * d2, N, _ptr(n_visible), _ptr(pool),
                                       P, act, _ptr(out), _stream(stream)))
    return out


def csa2_index_topk_fp4(mode, q_codes, q_scales, w, k_codes, k_scales, k_top: int, n_visible=None,
                        pool_in=None, pool_size: int = 0, act: int = ACT_RELU, stream=None):
    """Scores (FP4 indexer, bf16) + selection for one Full / Reindex layer."""
    torch = _torch()
    mode = _MODE[mode]
    B, Q, H, d2 = q_codes.shape
    N = k_codes.shape[1]
    P_in = pool_in.shape[2] if pool_in is not None else 0
    topk = torch.empty(B, Q, k_top, dtype=torch.int32, device=q_codes.device)
    pool = (torch.empty(B, Q, pool_size, dtype=torch.int32, device=q_codes.device)
            if pool_size > 0 else None)
    nb = lib().csa2_index_topk_workspace(B, Q, N, P_in, k_top, pool_size)
    ws = _workspace(nb, q_codes.device)
    _check(lib().csa2_index_topk_fp4(mode, _ptr(q_codes), _ptr(q_scales), _ptr(w), _ptr(k_codes),
                                     _ptr(k_scales), B, Q, H, 2 * d2, N, _ptr(n_visible),
                                     _ptr(pool_in), P_in, k_top, _ptr(topk), _ptr(pool), pool_size,
                                     act, _ptr(ws), nb, _stream(stream)))
    return topk, pool


def _workspace(nbytes, device):
    torch = _torch()
    if nbytes == 0:
        return None
    return torch.empty(int(nbytes), dtype=torch.uint8, device=device)


def csa2_select_topk(scores, count: int, ids=None, out=None, stream=None):
    """Top-`count` positions of each row of scores [..., L] (ascending, -1 padded)."""
    torch = _torch()
    L = scores.shape[-1]
    rows = scores.numel() // max(L, 1)
    if out is None:
        out = torch.empty(*scores.shape[:-1], count, dtype=torch.int32, device=scores.device)
    nb = lib().csa2_select_topk_workspace(rows, L, count)
    ws = _workspace(nb, scores.device)
    _check(lib().csa2_select_topk(_ptr(scores), rows, L, count, _ptr(ids), _ptr(out), _ptr(ws),
                                  nb, _stream(stream)))
    return out


def csa2_select_topk_noalloc(scores, count: int, ids=None, out=None, stream=None):
    """csa2_select_topk with the library's static scratch (no workspace is allocated)."""
    torch = _torch()
    L = scores.shape[-1]
    rows = scores.numel() // max(L, 1)
    if out is None:
        out = torch.empty(*scores.shape[:-1], count, dtype=torch.int32, device=scores.device)
    _check(lib().csa2_select_topk_noalloc(_ptr(scores), rows, L, count, _ptr(ids), _ptr(out),
                                          _stream(stream)))
    return out


def csa2_index_topk(mode, q, w, k, k_top: int, n_visible=None, pool_in=None, pool_size: int = 0,
                    act: int = ACT_RELU, stream=None):
    """Scores + selection for one Full / Reindex layer.  Returns (topk, pool or None)."""
    torch = _torch()
    mode = _MODE[mode]
    B, Q, H, d = q.shape
    N = k.shape[1]
    P_in = pool_in.shape[2] if pool_in is not None else 0
    topk = torch.empty(B, Q, k_top, dtype=torch.int32, device=q.device)
    pool = (torch.empty(B, Q, pool_size, dtype=torch.int32, device=q.device)
            if pool_size > 0 else None)
    nb = lib().csa2_index_topk_workspace(B, Q, N, P_in, k_top, pool_size)
    ws = _workspace(nb, q.device)
    _check(lib().csa2_index_topk(mode, _ptr(q), _ptr(w), _ptr(k), B, Q, H, d, N, _ptr(n_visible),
                                 _ptr(pool_in), P_in, k_top, _ptr(topk), _ptr(pool), pool_size,
                                 act, _ptr(ws), nb, _stream(stream)))
    return topk, pool


# ------------------------------------------------------------------ (a4)
def make_kv(kv, scales=None):
    """csa2_kv for a bf16 [B, n, D] tensor, or FP4 codes uint8 [B, n, D/2] + scales [B, n, D/16]."""
    if scales is None:
        return CSA2Kv(KV_BF16, kv.data_ptr(), None, kv.shape[1], kv.shape[2])
    return CSA2Kv(KV_FP4, kv.data_ptr(), scales.data_ptr(), kv.shape[1], kv.shape[2] * 2)


def csa2_sparse_attn(q, kv, topk, scale: float, kv_scales=None, mode=FULL, out=None, lse=None,
                     stream=None):
    torch = _torch()
    _need(q, torch.bfloat16, 4, "q")
    _need(topk, torch.int32, 3, "topk")
    B, Q, Ha, D = q.shape
    k = topk.shape[2]
    desc = make_kv(kv, kv_scales)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Q, Ha, dtype=torch.float32, device=q.device)
    nb = lib().csa2_sparse_attn_workspace(B, Q, Ha, D, k, desc.fmt)
    ws = _workspace(nb, q.device)
    _check(lib().csa2_sparse_attn(_MODE[mode], _ptr(q), ctypes.byref(desc), _ptr(topk), B, Q, Ha,
                                  k, scale, _ptr(out), _ptr(lse), _ptr(ws), nb, _stream(stream)))
    return out, lse


def csa2_sparse_attn_swa(q, kv, topk, scale: float, win, win_end, W: int = 128, kv_scales=None,
                         mode=FULL, out=None, lse=None, stream=None):
    """Sparse attention with the layer's sliding-window branch in the same
    softmax: win bf16 [B, R, D] window rows, win_end int32 [B, Q]."""
    torch = _torch()
    _need(q, torch.bfloat16, 4, "q")
    _need(topk, torch.int32, 3, "topk")
    _need(win, torch.bfloat16, 3, "win")
    _need(win_end, torch.int32, 2, "win_end")
    B, Q, Ha, D = q.shape
    k = topk.shape[2]
    desc = make_kv(kv, kv_scales)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Q, Ha, dtype=torch.float32, device=q.device)
    nb = lib().csa2_sparse_attn_swa_workspace(B, Q, Ha, D, k, desc.fmt)
    ws = _workspace(nb, q.device)
    _check(lib().csa2_sparse_attn_swa(_MODE[mode], _ptr(q), ctypes.byref(desc), _ptr(topk), B, Q,
                                      Ha, k, scale, _ptr(win), win.shape[1], _ptr(win_end), W,
                                      _ptr(out), _ptr(lse), _ptr(ws), nb, _stream(stream)))
    return out, lse


def csa2_dense_attn(q, kv, scale: float, n_visible=None, kv_scales=None, out=None, lse=None,
                    stream=None):
    """HCA attention: every query attends to entries [0, n_visible) of its sequence."""
    torch = _torch()
    _need(q, torch.bfloat16, 4, "q")
    if n_visible is not None:
        _need(n_visible, torch.int32, 2, "n_visible")
    B, Q, Ha, D = q.shape
    desc = make_kv(kv, kv_scales)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, Q, Ha, dtype=torch.float32, device=q.device)
    nb = lib().csa2_dense_attn_workspace(B, Q, Ha, D, desc.n, desc.fmt)
    ws = _workspace(nb, q.device)
    _check(lib().csa2_dense_attn(_ptr(q), ctypes.byref(desc), _ptr(n_visible), B, Q, Ha, scale,
                                 _ptr(out), _ptr(lse), _ptr(ws), nb, _stream(stream)))
    return out, lse


def csa2_compress_hca(c, z, bias, m: int, out=None, out_batch_stride: int = 0, stream=None):
    """HCA compression of raw tokens (c bf16 / z f32 [B, T, D], bias f32 [m, D])."""
    torch = _torch()
    _need(c, torch.bfloat16, 3, "c")
    _need(z, torch.float32, 3, "z")
    _need(bias, torch.float32, 2, "bias")
    B, T, D = c.shape
    if out is None:
        out = torch.empty(B, T // m, D, dtype=torch.bfloat16, device=c.device)
    _check(lib().csa2_compress_hca(_ptr(c), _ptr(z), _ptr(bias), B, T, D, m, _ptr(out),
                                   out_batch_stride, _stream(stream)))
    return out


# ------------------------------------------------------------------ (a5)
def csa2_fp4_pack(x, stream=None):
    torch = _torch()
    rows, D = x.reshape(-1, x.shape[-1]).shape
    codes = torch.empty(*x.shape[:-1], D // 2, dtype=torch.uint8, device=x.device)
    scales = torch.empty(*x.shape[:-1], D // 16, dtype=torch.uint8, device=x.device)
    _check(lib().csa2_fp4_pack(_ptr(x), rows, D, _ptr(codes), _ptr(scales), _stream(stream)))
    return codes, scales


def csa2_fp4_unpack(codes, scales, stream=None):
    torch = _torch()
    D = codes.shape[-1] * 2
    rows = codes.numel() // (D // 2)
    x = torch.empty(*codes.shape[:-1], D, dtype=torch.bfloat16, device=codes.device)
    _check(lib().csa2_fp4_unpack(_ptr(codes), _ptr(scales), rows, D, _ptr(x), _stream(stream)))
    return x


# ------------------------------------------------------------------ (p)
# The calls of this part run on their tensors' device and, with `stream`, on
# that stream: results and scratch memory are then allocated for it, and the
# inputs are marked as in use by it.

def _elsewhere(fn, dev, tensors, stream, args):
    """A call made again with its device and stream current (its arguments in order)."""
    torch = _torch()
    if dev < 0:
        raise ValueError(f"{fn.__name__}: expected CUDA tensors")
    if stream is None:
        with torch.cuda.device(dev):
            return fn(*args)
    if stream.device.index != dev:
        raise ValueError(f"{fn.__name__}: a stream of device {stream.device.index} with tensors on {dev}")
    if stream != torch.cuda.current_stream(dev):
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
    with torch.cuda.stream(stream):
        return fn(*args)


def _same_device(fn, dev, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{fn.__name__}: tensors on devices {dev} and {t.get_device()}")


def _raw_stream(dev):
    return _torch()._C._cuda_getCurrentRawStream(dev)


def _rows(t, name, dtype=None):
    """csa2_heads of a [T, heads, D] tensor with adjacent channels."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dim() != 3 or (t.dtype != dtype if dtype is not None else t.dtype not in _dtype_ids()):
        raise ValueError(f"{name}: expected {dtype or 'bfloat16 or float16'} [T, heads, D], got {t.dtype} "
                         f"{tuple(t.shape)}")
    T, H, D = t.shape
    ts, hs, cs = t.stride()
    if H <= 1:
        hs = D
    if T <= 1:
        ts = H * hs
    if (cs != 1 and D > 1) or ts <= 0 or hs <= 0:
        raise ValueError(f"{name}: channels must be adjacent and rows distinct, got strides {t.stride()}")
    return CSA2Heads(t.data_ptr(), H, ts, hs)


def _rows_out(t, out, name, T, H, D):
    """An output of t's shape (allocated when None) and its rows."""
    if out is None:
        out = t.new_empty((T, H, D))
        return out, CSA2Heads(out.data_ptr(), H, H * D, D)
    if out.shape != t.shape:
        raise ValueError(f"{name}: {tuple(out.shape)} for {tuple(t.shape)}")
    return out, _rows(out, name, t.dtype)


def _ints(t, name, n):
    """The address of a contiguous int32 tensor of n values."""
    if t is None or t.dtype is not _torch().int32 or t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        got = None if t is None else (t.dtype, tuple(t.shape))
        raise ValueError(f"{name}: expected contiguous int32 ({n},), got {got}")
    return t.data_ptr()


class Rope:
    """A position rotation: pair i of channels [offset, offset + 2 * half) turns
    by pos * inv_freq[i] (inv_freq f32 CUDA [half]); pairs (i, i + half), or
    neighbours when interleaved; inverse turns back."""

    def __init__(self, inv_freq, offset: int = 0, interleaved: bool = False, inverse: bool = False):
        torch = _torch()
        _need(inv_freq, torch.float32, 1, "inv_freq")
        self.inv_freq = inv_freq
        self.device = inv_freq.get_device()
        self.desc = CSA2Rope(inv_freq.data_ptr(), inv_freq.numel(), offset, int(interleaved), int(inverse))
        self.ref = ctypes.byref(self.desc)


class PagedKv:
    """A paged cache: k (and v; None: values are the key rows) [n_pages,
    page_size, heads, D] bf16 / f16 with adjacent channels, or uint8 FP4 codes
    [n_pages, page_size, heads, D/2] with scales [n_pages, page_size, heads, D/16];
    table int32 [B, max_pages], lens int32 [B] (device; the program updates them
    in place).  max_len: a bound of lens it knows (0: what the table holds); a
    decode call is cut into chunks by it, so give it where the table is long."""

    def __init__(self, k, table, lens, v=None, k_scales=None, v_scales=None, max_len: int = 0):
        torch = _torch()
        if k is None or k.dim() != 4 or not k.is_cuda:
            raise ValueError("k: expected a CUDA tensor [n_pages, page_size, heads, D]")
        fmts = {torch.bfloat16: KV_BF16, torch.float16: KV_F16, torch.uint8: KV_FP4}
        if k.dtype not in fmts:
            raise ValueError(f"k: unknown cache type {k.dtype}")
        fmt = fmts[k.dtype]
        fp4 = fmt == KV_FP4
        if v is k:
            v, v_scales = None, None
        n_pages, page, heads, width = k.shape
        dim = 2 * width if fp4 else width
        strides = self._strides(k, "k", 2 if fp4 else 1, dim)
        if v is not None and (v.dtype != k.dtype or v.shape != k.shape or self._strides(v, "v", 2 if fp4 else 1, dim) != strides):
            raise ValueError("v: type, shape and strides must be k's")
        for s, x, name in ((k_scales, k, "k_scales"), (v_scales, v, "v_scales")):
            if (s is not None) != (fp4 and x is not None):
                raise ValueError(f"{name}: scales belong to an FP4 cache's rows, and only to them")
            if s is not None and (s.dtype != torch.uint8 or tuple(s.shape) != (n_pages, page, heads, dim // 16) or
                                  self._strides(s, name, 16, dim) != strides):
                raise ValueError(f"{name}: expected uint8 [n_pages, page_size, heads, D/16] laid out like {name[0]}")
        if table is None or table.dtype != torch.int32 or table.dim() != 2 or (table.shape[1] > 1 and table.stride(1) != 1):
            raise ValueError("table: expected int32 [B, max_pages]")
        B, max_pages = table.shape
        _ints(lens, "lens", B)
        if B > 1 and table.stride(0) < max_pages:
            raise ValueError("table: rows overlap")
        self.k, self.v, self.k_scales, self.v_scales, self.table, self.lens = k, v, k_scales, v_scales, table, lens
        self.tensors = (k, v, k_scales, v_scales, table, lens)
        if len({t.get_device() for t in self.tensors if t is not None}) != 1:
            raise ValueError("the cache's tensors must be on one device")
        self.device = k.get_device()
        self.dtype = torch.bfloat16 if fp4 else k.dtype
        self._workspaces = {}
        self.heads, self.dim, self.B = heads, dim, B
        self.desc = CSA2PagedKv(fmt, k.data_ptr(), None if v is None else v.data_ptr(),
                                None if k_scales is None else k_scales.data_ptr(),
                                None if v_scales is None else v_scales.data_ptr(), n_pages, strides[0], strides[1],
                                strides[2], page, heads, dim, B, max_pages,
                                table.stride(0) if B > 1 else max_pages, table.data_ptr(), lens.data_ptr(), max_len)
        self.ref = ctypes.byref(self.desc)

    def decode_workspace(self, Hq, window=0, sinks=0, chunk=0):
        """Bytes of scratch a csa2_paged_decode_attn call takes (depends on the shapes only)."""
        key = (Hq, window, sinks, chunk)
        nb = self._workspaces.get(key)
        if nb is None:
            with _torch().cuda.device(self.device):
                nb = self._workspaces[key] = lib().csa2_paged_decode_attn_workspace(self.ref, *key)
        return nb

    @staticmethod
    def _strides(t, name, unit, dim):
        """(page, token, head) strides in channels; dimensions of one element count as dense."""
        n, page, heads, width = t.shape
        st = [x * unit for x in t.stride()]
        if heads <= 1:
            st[2] = dim
        if page <= 1:
            st[1] = heads * st[2]
        if n <= 1:
            st[0] = page * st[1]
        if (width > 1 and t.stride(3) != 1) or min(st[:3]) < dim:
            raise ValueError(f"{name}: channels must be adjacent and rows distinct, got strides {t.stride()}")
        return tuple(st[:3])


_DTYPE_ID = {}


def _dtype_ids():
    if not _DTYPE_ID:
        torch = _torch()
        _DTYPE_ID.update({torch.bfloat16: 0, torch.float16: 1})
    return _DTYPE_ID


def _weight(w, name, D):
    if w is None:
        return None
    if w.dtype is not _torch().float32 or w.dim() != 1 or w.shape[0] != D or not w.is_contiguous():
        raise ValueError(f"{name}: expected contiguous float32 ({D},), got {w.dtype} {tuple(w.shape)}")
    return w.data_ptr()


def csa2_qk_norm_rope(q, k, positions=None, q_weight=None, k_weight=None, eps: float = 1e-6, rope=None, q_out=None,
                      k_out=None, stream=None):
    """RMS norm of every head row (weight f32 [D] or None) and its rotation to
    positions[t] (int32 [T]); q, k [T, heads, D] bf16 / f16 (either may be None).
    q_out / k_out may be q / k (in place).  Returns (q_out, k_out)."""
    torch = _torch()
    x = q if q is not None else k
    if x is None:
        raise ValueError("csa2_qk_norm_rope: neither q nor k given")
    dev = x.get_device()
    _same_device(csa2_qk_norm_rope, dev, q, k, positions, q_weight, k_weight, q_out, k_out)
    if rope is not None and rope.device != dev:
        raise ValueError(f"csa2_qk_norm_rope: rotation on device {rope.device}, tensors on {dev}")
    if dev < 0 or stream is not None or dev != torch.cuda.current_device():
        return _elsewhere(csa2_qk_norm_rope, dev, (q, k, positions, q_weight, k_weight, q_out, k_out,
                                                   None if rope is None else rope.inv_freq), stream,
                          (q, k, positions, q_weight, k_weight, eps, rope, q_out, k_out))
    dtype = x.dtype
    xr = _rows(x, "q" if x is q else "k")
    T, _, D = x.shape
    qa = qo = ka = ko = None
    if q is not None:
        q_out, r = _rows_out(q, q_out, "q_out", T, xr.heads, D)
        qa, qo = ctypes.byref(xr), ctypes.byref(r)
    if k is not None:
        if k.shape[0] != T or k.shape[2] != D:
            raise ValueError(f"k: {tuple(k.shape)} beside {T} rows of {D} channels")
        kr = xr if x is k else _rows(k, "k", dtype)
        k_out, r2 = _rows_out(k, k_out, "k_out", T, kr.heads, D)
        ka, ko = ctypes.byref(kr), ctypes.byref(r2)
    st = lib().csa2_qk_norm_rope(_dtype_ids()[dtype], qa, _weight(q_weight, "q_weight", D), qo, ka,
                                 _weight(k_weight, "k_weight", D), ko, T, D, eps,
                                 None if positions is None else _ints(positions, "positions", T),
                                 None if rope is None else rope.ref, _raw_stream(dev))
    if st:
        _check(st)
    return q_out if q is not None else None, k_out if k is not None else None


def csa2_paged_append(cache, k, v, seq, pos, rope=None, stream=None):
    """Write rows k (rotated to pos when `rope`), v [T, heads, D] to tokens pos[t] of
    sequences seq[t] (int32 [T]; seq -1: skip) of a PagedKv; v None for a shared cache."""
    dev = cache.device
    _same_device(csa2_paged_append, dev, k, v, seq, pos)
    if rope is not None and rope.device != dev:
        raise ValueError(f"csa2_paged_append: rotation on device {rope.device}, cache on {dev}")
    if stream is not None or dev != _torch().cuda.current_device():
        return _elsewhere(csa2_paged_append, dev, (k, v, seq, pos, None if rope is None else rope.inv_freq) + cache.tensors,
                          stream, (cache, k, v, seq, pos, rope))
    kr = _rows(k, "k", cache.dtype)
    T = k.shape[0]
    if k.shape[2] != cache.dim or (v is not None and v.shape != k.shape):
        raise ValueError(f"k, v: {tuple(k.shape)}, {None if v is None else tuple(v.shape)} for a cache of width {cache.dim}")
    st = lib().csa2_paged_append(_dtype_ids()[cache.dtype], ctypes.byref(kr),
                                 None if v is None else ctypes.byref(_rows(v, "v", cache.dtype)), _ints(seq, "seq", T),
                                 _ints(pos, "pos", T), T, None if rope is None else rope.ref, cache.ref, _raw_stream(dev))
    if st:
        _check(st)


def _attn_out(q, out, lse):
    if out is None:
        out = q.new_empty(q.shape)
    elif out.dtype != q.dtype or out.shape != q.shape or not out.is_contiguous():
        raise ValueError(f"out: expected contiguous {q.dtype} {tuple(q.shape)}")
    if lse is None:
        lse = q.new_empty(q.shape[:2], dtype=_torch().float32)
    elif lse.dtype != _torch().float32 or lse.shape != q.shape[:2] or not lse.is_contiguous():
        raise ValueError(f"lse: expected contiguous float32 {tuple(q.shape[:2])}")
    return out, lse


def _fits(name, *counts):
    """Counts that a 32-bit argument would cut to other counts are refused."""
    for x in counts:
        if not -0x80000000 <= x <= 0x7fffffff:
            raise ValueError(f"{name}: {x} is past 32 bits")


def csa2_paged_decode_attn(q, cache, scale: float, window: int = 0, sinks: int = 0, chunk: int = 0, out=None, lse=None,
                           stream=None):
    """Attention of one new token per sequence (q [B, Hq, D], at position lens[b] - 1)
    over a PagedKv: the last `window` tokens (0: all) and the first `sinks`."""
    _fits("csa2_paged_decode_attn", window, sinks, chunk)
    dev = cache.device
    _same_device(csa2_paged_decode_attn, dev, q, out, lse)
    if stream is not None or dev != _torch().cuda.current_device():
        return _elsewhere(csa2_paged_decode_attn, dev, (q, out, lse) + cache.tensors, stream,
                          (q, cache, scale, window, sinks, chunk, out, lse))
    rows = _rows(q, "q", cache.dtype)
    B, Hq, D = q.shape
    if B != cache.B or D != cache.dim:
        raise ValueError(f"q: {tuple(q.shape)} for a cache of {cache.B} sequences of width {cache.dim}")
    out, lse = _attn_out(q, out, lse)
    nb = cache.decode_workspace(Hq, window, sinks, chunk)
    ws = q.new_empty(nb, dtype=_torch().uint8) if nb else None
    st = lib().csa2_paged_decode_attn(ctypes.byref(rows), cache.ref, scale, window, sinks, chunk, out.data_ptr(),
                                      lse.data_ptr(), ws.data_ptr() if nb else None, nb, _raw_stream(dev))
    if st:
        _check(st)
    return out, lse


def csa2_paged_window_attn(q, cu_q, cache, scale: float, window: int = 0, sinks: int = 0, out=None, lse=None,
                           stream=None):
    """Causal attention of a prompt chunk: sequence b's new tokens are rows
    cu_q[b]..cu_q[b+1] of q [T, Hq, D], the last at position lens[b] - 1."""
    _fits("csa2_paged_window_attn", window, sinks)
    dev = cache.device
    _same_device(csa2_paged_window_attn, dev, q, cu_q, out, lse)
    if stream is not None or dev != _torch().cuda.current_device():
        return _elsewhere(csa2_paged_window_attn, dev, (q, cu_q, out, lse) + cache.tensors, stream,
                          (q, cu_q, cache, scale, window, sinks, out, lse))
    rows = _rows(q, "q", cache.dtype)
    T, _, D = q.shape
    if D != cache.dim:
        raise ValueError(f"q: {tuple(q.shape)} for a cache of width {cache.dim}")
    out, lse = _attn_out(q, out, lse)
    st = lib().csa2_paged_window_attn(ctypes.byref(rows), _ints(cu_q, "cu_q", cache.B + 1), T, cache.ref, scale, window,
                                      sinks, out.data_ptr(), lse.data_ptr(), _raw_stream(dev))
    if st:
        _check(st)
    return out, lse


# ------------------------------------------------------------------ (a6)
class Group:
    """A CSA2 layer group (Full / Reindex / Reuse modes) driven through the C ABI."""

    def __init__(self, B, Q, N, D, Ha, Hi, d, k, modes, P=0, scale=None, kv_fmt=KV_BF16,
                 act=ACT_RELU):
        self.modes = [_MODE[m] for m in modes]
        arr = (_I * len(self.modes))(*self.modes)
        self._modes_arr = arr
        desc = CSA2GroupDesc(B, Q, N, D, Ha, Hi, d, k, P,
                             (D ** -0.5) if scale is None else scale, kv_fmt, act,
                             len(self.modes), arr)
        h = _P()
        _check(lib().csa2_group_create(ctypes.byref(h), ctypes.byref(desc)))
        self._h = h
        self.desc = desc

    def layer(self, i, q_attn, out, lse=None, kv=None, kv_scales=None, index_k=None,
              q_index=None, w_index=None, n_visible=None, swa=None, stream=None):
        """swa: optional (win bf16 [B, R, D], win_end int32 [B, Q], W), this
        layer's own sliding-window rows."""
        io = CSA2LayerIO()
        if kv is not None:
            io.kv = make_kv(kv, kv_scales)
        io.index_k = _ptr(index_k)
        io.n_visible = _ptr(n_visible)
        io.q_index = _ptr(q_index)
        io.w_index = _ptr(w_index)
        io.q_attn = _ptr(q_attn)
        io.out = _ptr(out)
        io.lse = _ptr(lse)
        if swa is not None:
            win, win_end, W = swa
            io.swa_kv = _ptr(win)
            io.swa_rows = win.shape[1]
            io.swa_end = _ptr(win_end)
            io.swa_window = W
        _check(lib().csa2_group_layer(self._h, i, ctypes.byref(io), _stream(stream)))

    def selection(self):
        t, p = _P(), _P()
        _check(lib().csa2_group_selection(self._h, ctypes.byref(t), ctypes.byref(p)))
        return t.value, p.value

    def copy_selection(self, stream=None):
        """(topk [B,Q,k], pool [B,Q,P] or None) copies of the current selection."""
        torch = _torch()
        d = self.desc
        topk = torch.empty(d.B, d.Q, d.k, dtype=torch.int32, device="cuda")
        pool = torch.empty(d.B, d.Q, d.P, dtype=torch.int32, device="cuda") if d.P > 0 else None
        _check(lib().csa2_group_copy_selection(self._h, _ptr(topk), _ptr(pool), _stream(stream)))
        return topk, pool

    def close(self):
        if getattr(self, "_h", None) and self._h.value:
            lib().csa2_group_destroy(self._h)
            self._h = _P()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------------ errors, counters
def csa2_device_error(stream=None):
    """Synchronise and raise if a kernel recorded a device-side error."""
    _check(lib().csa2_device_error(_stream(stream)))


LAUNCH_KINDS = ("compress", "index_scores", "topk", "attn", "attn_combine", "fp4_pack",
                "fp4_unpack", "other", "index_pool")


def launch_counts() -> dict:
    arr = (_I64 * len(LAUNCH_KINDS))()
    lib().csa2_launch_counts(arr, len(LAUNCH_KINDS))
    return dict(zip(LAUNCH_KINDS, arr))


def reset_launch_counts() -> None:
    lib().csa2_reset_launch_counts()


def timing_enable(on: bool) -> None:
    """Bracket every library launch with CUDA events (instrumentation)."""
    _check(lib().csa2_timing_enable(int(bool(on))))


def timing_reset() -> None:
    lib().csa2_timing_reset()


def kernel_times() -> dict:
    """{kind: (total_ms, timed_launches)} since the last timing_reset()."""
    n = len(LAUNCH_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (_I64 * n)()
    lib().csa2_kernel_times(ms, cnt, n)
    return {k: (ms[i], cnt[i]) for i, k in enumerate(LAUNCH_KINDS)}


def set_fault(kind: str) -> None:
    _check(lib().csa2_set_fault(kind.encode()))


def set_device_wait(limit_ns: int = 0, unreachable: bool = False) -> None:
    """Bound of the cross-CTA device waits (0 = default, 1 s); `unreachable`
    makes each such wait run out (a test of the error path)."""
    _check(lib().csa2_set_device_wait(int(limit_ns), int(bool(unreachable))))
