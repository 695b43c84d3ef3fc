"""Python binding of libcsa.so, the CSA/HCA attention layer for one B200.

Argument marshalling only: every function here checks tensor shapes, dtypes
and devices, passes raw device pointers and the current CUDA stream to the C
ABI declared in ``include/csa.h`` and raises ``CsaError`` on a non-OK status.
All arithmetic runs in the library's CUDA kernels; there is no fallback.

The functions carry the C names: ``csa_compress``, ``csa_index_topk``,
``csa_sparse_attn``, ``hca_attn`` and the decode-cache calls
(``CsaCache`` wraps ``csa_cache_layout`` / ``csa_cache_store_entries`` /
``csa_cache_write_rows`` / ``csa_decode_step``), ``csa_qk_norm_rope``,
``csa_window_attn``, the 4-bit key/value cache (``csa_kv4_cache``,
``csa_kv4_store``, ``csa_kv4_fetch``, ``csa_kv4_decode_attn``) and the blocks
of paged caches (``csa_blocks_copy``, ``csa_blocks_fork``,
``csa_blocks_free``, ``csa_blocks_compact``).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libcsa.so")

CSA_OK, CSA_ERR_INVALID_ARG, CSA_ERR_UNSUPPORTED, CSA_ERR_WORKSPACE, CSA_ERR_CUDA, \
    CSA_ERR_TIMEOUT = 0, -1, -2, -3, -4, -5
CSA_F32, CSA_BF16 = 0, 1

EXPORTED = (
    "csa_status_string", "csa_last_error", "csa_abi_version", "csa_check", "csa_selftest_wait",
    "csa_compress",
    "csa_index_topk_workspace", "csa_index_topk", "csa_index_topk_noalloc", "csa_sparse_attn",
    "hca_attn",
    "csa_cache_layout", "csa_cache_store_entries", "csa_cache_write_rows",
    "csa_decode_workspace", "csa_decode_step",
    "csa_norm_rope_rows", "csa_compress_norm_rope", "csa_sparse_attn_norm_rope",
    "hca_attn_norm_rope", "csa_index_topk_lowp_workspace", "csa_index_topk_lowp",
    "csa_grouped_out_proj_workspace", "csa_grouped_out_proj",
    "csa_paged_cache_layout", "csa_paged_cache_store_entries", "csa_paged_cache_write_rows",
    "csa_paged_decode_step",
    "csa_qk_norm_rope", "csa_window_attn",
    "csa_kv4_block_bytes", "csa_kv4_store", "csa_kv4_fetch", "csa_kv4_decode_workspace",
    "csa_kv4_decode_attn",
    "csa_blocks_copy", "csa_blocks_fork", "csa_blocks_free", "csa_blocks_compact",
)
CSA_INDEX_FP8_QK, CSA_INDEX_BF16_SCORES = 1, 2


class CsaError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{status_string(status)}: {detail}")


class CacheDesc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("capacity", ctypes.c_int64), ("c", ctypes.c_int32),
                ("rope_dims", ctypes.c_int32), ("c_i", ctypes.c_int32), ("m", ctypes.c_int32),
                ("window", ctypes.c_int32), ("nh", ctypes.c_int32), ("nh_i", ctypes.c_int32),
                ("k", ctypes.c_int32), ("is_hca", ctypes.c_int32)]


class CacheLayout(ctypes.Structure):
    _fields_ = [(nm, ctypes.c_size_t) for nm in (
        "entry_fp8", "entry_scale", "entry_rope", "ikey_fp8", "ikey_scale", "window", "state",
        "istate", "total_bytes")]


class Rows(ctypes.Structure):
    _fields_ = [(nm, ctypes.c_void_p) for nm in (
        "ca", "cb", "za", "zb", "ica", "icb", "iza", "izb", "kv_win")]


class DecodeParams(ctypes.Structure):
    _fields_ = [("ba", ctypes.c_void_p), ("bb", ctypes.c_void_p), ("iba", ctypes.c_void_p),
                ("ibb", ctypes.c_void_p), ("sink", ctypes.c_void_p), ("scale", ctypes.c_float),
                ("sel_out", ctypes.c_void_p), ("scores_out", ctypes.c_void_p)]


class Paging(ctypes.Structure):
    _fields_ = [("block_tokens", ctypes.c_int32), ("num_blocks", ctypes.c_int64),
                ("max_blocks", ctypes.c_int64), ("block_table", ctypes.c_void_p)]


class NormRope(ctypes.Structure):
    _fields_ = [("gamma", ctypes.c_void_p), ("eps", ctypes.c_float),
                ("rope_dims", ctypes.c_int32), ("rope_base", ctypes.c_float)]


class QkRope(ctypes.Structure):
    _fields_ = [("q_gamma", ctypes.c_void_p), ("k_gamma", ctypes.c_void_p),
                ("per_head", ctypes.c_int32), ("eps", ctypes.c_float),
                ("rope_dims", ctypes.c_int32), ("rope_base", ctypes.c_float),
                ("halves", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("sections", ctypes.c_int32 * 4)]


class Kv4Desc(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("batch", ctypes.c_int64), ("max_blocks", ctypes.c_int64),
                ("num_blocks", ctypes.c_int64), ("nkv", ctypes.c_int32), ("c", ctypes.c_int32),
                ("block_tokens", ctypes.c_int32)]


class BlockRegion(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("block_bytes", ctypes.c_size_t)]


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded libcsa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python -m compressed_sparse_attention_11_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, \
        ctypes.c_float
    sig = {
        "csa_status_string": (ctypes.c_char_p, [i32]),
        "csa_last_error": (ctypes.c_char_p, []),
        "csa_abi_version": (i32, []),
        "csa_check": (i32, [vp]),
        "csa_selftest_wait": (i32, [ctypes.c_uint32, i32, vp]),
        "csa_compress": (i32, [vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, i32, i32, vp, vp]),
        "csa_index_topk_workspace": (sz, [i64, i64, i32, i32, i32, i32]),
        "csa_index_topk": (i32, [vp, vp, vp, i64, i64, i32, i32, i32, i32, i32, vp, vp, sz, vp]),
        "csa_index_topk_noalloc": (i32, [vp, vp, vp, i64, i64, i32, i32, i32, i32, i32, vp, vp]),
        "csa_sparse_attn": (i32, [vp, vp, vp, i32, vp, i32, vp, f32, i64, i64, i32, i32, i32,
                                  i32, vp, vp]),
        "hca_attn": (i32, [vp, vp, vp, i32, vp, f32, i64, i64, i32, i32, i32, i32, vp, vp]),
        "csa_cache_layout": (i32, [ctypes.POINTER(CacheDesc), ctypes.POINTER(CacheLayout)]),
        "csa_cache_store_entries": (i32, [ctypes.POINTER(CacheDesc), vp, i64, i64, vp, vp, i32,
                                          vp]),
        "csa_cache_write_rows": (i32, [ctypes.POINTER(CacheDesc), vp, i64, i64,
                                       ctypes.POINTER(Rows), vp]),
        "csa_decode_workspace": (sz, [ctypes.POINTER(CacheDesc)]),
        "csa_decode_step": (i32, [ctypes.POINTER(CacheDesc), vp, vp, ctypes.POINTER(Rows),
                                  ctypes.POINTER(DecodeParams), vp, vp, vp, vp, vp, sz, vp]),
        "csa_norm_rope_rows": (i32, [vp, i64, i64, i32, i32, i64, ctypes.POINTER(NormRope), i32,
                                     vp, vp]),
        "csa_compress_norm_rope": (i32, [vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, i32, i32,
                                         ctypes.POINTER(NormRope), vp, vp]),
        "csa_sparse_attn_norm_rope": (i32, [vp, vp, vp, i32, vp, i32, vp, f32, i64, i64, i32, i32,
                                            i32, i32, ctypes.POINTER(NormRope), vp, vp]),
        "hca_attn_norm_rope": (i32, [vp, vp, vp, i32, vp, f32, i64, i64, i32, i32, i32, i32,
                                     ctypes.POINTER(NormRope), vp, vp]),
        "csa_paged_cache_layout": (i32, [ctypes.POINTER(CacheDesc), ctypes.POINTER(Paging),
                                         ctypes.POINTER(CacheLayout)]),
        "csa_paged_cache_store_entries": (i32, [ctypes.POINTER(CacheDesc), ctypes.POINTER(Paging),
                                                vp, i64, i64, vp, vp, i32, vp]),
        "csa_paged_cache_write_rows": (i32, [ctypes.POINTER(CacheDesc), ctypes.POINTER(Paging), vp,
                                             i64, i64, ctypes.POINTER(Rows), vp]),
        "csa_paged_decode_step": (i32, [ctypes.POINTER(CacheDesc), ctypes.POINTER(Paging), vp, vp,
                                        ctypes.POINTER(Rows), ctypes.POINTER(DecodeParams), vp, vp,
                                        vp, vp, vp, sz, vp]),
        "csa_grouped_out_proj_workspace": (sz, [i64, i32, i32]),
        "csa_grouped_out_proj": (i32, [vp, i64, i32, i32, i32, i32, i32, vp, vp, vp, sz, vp, vp]),
        "csa_qk_norm_rope": (i32, [vp, i64, vp, i64, i64, i32, i32, i32, vp,
                                   ctypes.POINTER(QkRope), i32, vp, i64, vp, i64, vp]),
        "csa_window_attn": (i32, [vp, i64, vp, i64, vp, i64, i64, i64, vp, f32, i64, i64, i64, i32,
                                  i32, i32, i32, vp, vp]),
        "csa_kv4_block_bytes": (sz, [i32, i32, i32]),
        "csa_kv4_store": (i32, [ctypes.POINTER(Kv4Desc), vp, i64, vp, vp, i64, vp, i64, i32, vp]),
        "csa_kv4_fetch": (i32, [ctypes.POINTER(Kv4Desc), vp, i64, vp, i32, vp, vp, vp]),
        "csa_kv4_decode_workspace": (sz, [i32, i32, i32]),
        "csa_kv4_decode_attn": (i32, [ctypes.POINTER(Kv4Desc), vp, vp, i32, i64, i64, vp, f32, vp,
                                      vp, sz, vp]),
        "csa_blocks_copy": (i32, [ctypes.POINTER(BlockRegion), i32, i64, vp, vp, i64, vp, vp]),
        "csa_blocks_fork": (i32, [vp, i64, i64, vp, vp, vp, vp, i32, i32, vp, vp, vp, vp]),
        "csa_blocks_free": (i32, [vp, i64, i64, i64, vp, i32, vp, vp, vp, vp]),
        "csa_blocks_compact": (i32, [vp, i64, i64, i64, vp, vp, vp, vp, vp]),
        "csa_index_topk_lowp_workspace": (sz, [i64, i64, i32, i32, i32, i32, i32]),
        "csa_index_topk_lowp": (i32, [vp, vp, vp, i64, i64, i32, i32, i32, i32, i32, i32, vp, vp,
                                      sz, vp]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def status_string(status: int) -> str:
    return lib().csa_status_string(int(status)).decode()


def _check(status: int):
    if status != CSA_OK:
        raise CsaError(status, lib().csa_last_error().decode())


def csa_check(device=None):
    """Synchronises the current stream and raises if a kernel gave up a bounded wait."""
    _check(lib().csa_check(torch.cuda.current_stream(device).cuda_stream))


def selftest_wait(limit_us: int, arrive: bool, device=None) -> int:
    """Runs the library's bounded-wait self-test on the current stream and
    returns the status csa_check reports afterwards (CSA_OK when the barrier
    was completed, CSA_ERR_TIMEOUT when the wait gave up)."""
    L = lib()
    stream = torch.cuda.current_stream(device).cuda_stream
    _check(L.csa_selftest_wait(int(limit_us), 1 if arrive else 0, stream))
    return int(L.csa_check(stream))


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return CSA_F32
    if t.dtype == torch.bfloat16:
        return CSA_BF16
    raise ValueError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(t: torch.Tensor) -> int:
    return torch.cuda.current_stream(t.device).cuda_stream


# ------------------------------------------------------------------ prefill ---

def csa_compress(ca, cb, za, zb, ba, bb, m: int, out: Optional[torch.Tensor] = None):
    """Compress [B, n, c] streams into [B, n//m, c] entries.

    CSA (overlapped) when ``cb`` is given, HCA (single stream) when ``cb``,
    ``zb`` and ``bb`` are None.
    """
    overlap = 1 if cb is not None else 0
    B, n, c = ca.shape
    if out is None:
        out = torch.empty((B, n // m, c), dtype=ca.dtype, device=ca.device)
    _check(lib().csa_compress(_ptr(ca), _ptr(cb), _ptr(za), _ptr(zb), _ptr(ba), _ptr(bb), B, n,
                              c, m, overlap, _dt(ca), _ptr(out), _stream(ca)))
    return out


def csa_index_topk_workspace(batch: int, n: int, nh_i: int, c_i: int, m: int, k: int) -> int:
    return int(lib().csa_index_topk_workspace(batch, n, nh_i, c_i, m, k))


def csa_index_topk(q_i, w_i, k_i, m: int, k: int, ws: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None):
    """Top-k entry indices [B, n, k] int32 (ascending, -1 padded)."""
    B, n, H, ci = q_i.shape
    need = csa_index_topk_workspace(B, n, H, ci, m, k)
    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=q_i.device)
    if out is None:
        out = torch.empty((B, n, k), dtype=torch.int32, device=q_i.device)
    _check(lib().csa_index_topk(_ptr(q_i), _ptr(w_i), _ptr(k_i), B, n, H, ci, m, k, _dt(q_i),
                                _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                _stream(q_i)))
    return out


def csa_index_topk_noalloc(q_i, w_i, k_i, m: int, k: int, out: Optional[torch.Tensor] = None):
    """csa_index_topk using the library's built-in score scratch (no workspace).

    For callers that cannot allocate device memory; limited to
    batch * n * (n // m) <= 2**21 scores, and concurrent calls race."""
    B, n, H, ci = q_i.shape
    if out is None:
        out = torch.empty((B, n, k), dtype=torch.int32, device=q_i.device)
    _check(lib().csa_index_topk_noalloc(_ptr(q_i), _ptr(w_i), _ptr(k_i), B, n, H, ci, m, k,
                                        _dt(q_i), _ptr(out), _stream(q_i)))
    return out


def csa_index_topk_lowp(q_i, w_i, k_i, m: int, k: int, fp8_qk: bool = True,
                        bf16_scores: bool = True, ws: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None):
    """The indexer + top-k with FP8 query/key scoring and / or bf16-stored
    scores: indices [B, n, k] int32 (ascending, -1 padded)."""
    B, n, H, ci = q_i.shape
    flags = (CSA_INDEX_FP8_QK if fp8_qk else 0) | (CSA_INDEX_BF16_SCORES if bf16_scores else 0)
    need = int(lib().csa_index_topk_lowp_workspace(B, n, H, ci, m, k, flags))
    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=q_i.device)
    if out is None:
        out = torch.empty((B, n, k), dtype=torch.int32, device=q_i.device)
    _check(lib().csa_index_topk_lowp(_ptr(q_i), _ptr(w_i), _ptr(k_i), B, n, H, ci, m, k, _dt(q_i),
                                     flags, _ptr(out), _ptr(ws), ws.numel() * ws.element_size(),
                                     _stream(q_i)))
    return out


def csa_sparse_attn(q, kv_comp, idx, kv_win, window: int, sink, scale: float, m: int,
                    out: Optional[torch.Tensor] = None):
    B, n, nh, c = q.shape
    if out is None:
        out = torch.empty_like(q)
    _check(lib().csa_sparse_attn(_ptr(q), _ptr(kv_comp), _ptr(idx), idx.shape[-1], _ptr(kv_win),
                                 window, _ptr(sink), float(scale), B, n, nh, c, m, _dt(q),
                                 _ptr(out), _stream(q)))
    return out


def hca_attn(q, kv_comp, kv_win, window: int, sink, scale: float, m_heavy: int,
             out: Optional[torch.Tensor] = None):
    B, n, nh, c = q.shape
    if out is None:
        out = torch.empty_like(q)
    _check(lib().hca_attn(_ptr(q), _ptr(kv_comp), _ptr(kv_win), window, _ptr(sink), float(scale),
                          B, n, nh, c, m_heavy, _dt(q), _ptr(out), _stream(q)))
    return out


# ------------------------------------------------- RMSNorm and partial RoPE ---

ROPE_BASE = 10000.0
NORM_EPS = 1e-6


def _norm_rope(gamma, eps: float, rope_dims: int, rope_base: float) -> NormRope:
    if gamma is None or gamma.dtype != torch.float32:
        raise ValueError("gamma must be a float32 tensor")
    return NormRope(_ptr(gamma), float(eps), int(rope_dims), float(rope_base))


def csa_norm_rope_rows(x, gamma, pos_mul: int = 1, eps: float = NORM_EPS, rope_dims: int = 64,
                       rope_base: float = ROPE_BASE, out: Optional[torch.Tensor] = None):
    """RMSNorm + rotation of the trailing dims of every row of x [B, n, c] or
    [B, n, heads, c]; row t turns for position t * pos_mul (out may be x)."""
    B, n = x.shape[0], x.shape[1]
    heads = x.shape[2] if x.dim() == 4 else 1
    c = x.shape[-1]
    if out is None:
        out = torch.empty_like(x)
    nr = _norm_rope(gamma, eps, rope_dims, rope_base)
    _check(lib().csa_norm_rope_rows(_ptr(x), B, n, heads, c, int(pos_mul), ctypes.byref(nr),
                                    _dt(x), _ptr(out), _stream(x)))
    return out


def csa_compress_norm_rope(ca, cb, za, zb, ba, bb, m: int, gamma, eps: float = NORM_EPS,
                           rope_dims: int = 64, rope_base: float = ROPE_BASE,
                           out: Optional[torch.Tensor] = None):
    """csa_compress with each entry i RMSNorm-ed and rotated for position m * i."""
    overlap = 1 if cb is not None else 0
    B, n, c = ca.shape
    if out is None:
        out = torch.empty((B, n // m, c), dtype=ca.dtype, device=ca.device)
    nr = _norm_rope(gamma, eps, rope_dims, rope_base)
    _check(lib().csa_compress_norm_rope(_ptr(ca), _ptr(cb), _ptr(za), _ptr(zb), _ptr(ba),
                                        _ptr(bb), B, n, c, m, overlap, _dt(ca), ctypes.byref(nr),
                                        _ptr(out), _stream(ca)))
    return out


def csa_sparse_attn_norm_rope(q, kv_comp, idx, kv_win, window: int, sink, scale: float, m: int,
                              q_gamma, eps: float = NORM_EPS, rope_dims: int = 64,
                              rope_base: float = ROPE_BASE, out: Optional[torch.Tensor] = None):
    """csa_sparse_attn with the query norm + rotation and the output rotation
    by -t; kv_comp and kv_win must already be normed and rotated."""
    B, n, nh, c = q.shape
    if out is None:
        out = torch.empty_like(q)
    nr = _norm_rope(q_gamma, eps, rope_dims, rope_base)
    _check(lib().csa_sparse_attn_norm_rope(_ptr(q), _ptr(kv_comp), _ptr(idx), idx.shape[-1],
                                           _ptr(kv_win), window, _ptr(sink), float(scale), B, n,
                                           nh, c, m, _dt(q), ctypes.byref(nr), _ptr(out),
                                           _stream(q)))
    return out


def hca_attn_norm_rope(q, kv_comp, kv_win, window: int, sink, scale: float, m_heavy: int,
                       q_gamma, eps: float = NORM_EPS, rope_dims: int = 64,
                       rope_base: float = ROPE_BASE, out: Optional[torch.Tensor] = None):
    """hca_attn with the query norm + rotation and the output rotation by -t."""
    B, n, nh, c = q.shape
    if out is None:
        out = torch.empty_like(q)
    nr = _norm_rope(q_gamma, eps, rope_dims, rope_base)
    _check(lib().hca_attn_norm_rope(_ptr(q), _ptr(kv_comp), _ptr(kv_win), window, _ptr(sink),
                                    float(scale), B, n, nh, c, m_heavy, _dt(q), ctypes.byref(nr),
                                    _ptr(out), _stream(q)))
    return out


# ------------------------------------------------------ output projection ---

def csa_grouped_out_proj(o, w1, w2, ws: Optional[torch.Tensor] = None,
                         out: Optional[torch.Tensor] = None):
    """Grouped output projection: o [rows, nh, c] (or [B, n, nh, c]) with
    w1 [G, d_g, nh/G * c] and w2 [d, G * d_g] -> y [rows, d] (bf16)."""
    nh, c = o.shape[-2], o.shape[-1]
    rows = o.numel() // (nh * c)
    G, dg = w1.shape[0], w1.shape[1]
    d = w2.shape[0]
    need = int(lib().csa_grouped_out_proj_workspace(rows, G, dg))
    if ws is None:
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=o.device)
    if out is None:
        out = torch.empty(o.shape[:-2] + (d,), dtype=o.dtype, device=o.device)
    if o.dtype != torch.bfloat16 or w1.dtype != torch.bfloat16 or w2.dtype != torch.bfloat16:
        raise ValueError("the grouped output projection takes bfloat16 tensors")
    _check(lib().csa_grouped_out_proj(_ptr(o), rows, nh, c, G, dg, d, _ptr(w1), _ptr(w2),
                                      _ptr(ws), ws.numel() * ws.element_size(), _ptr(out),
                                      _stream(o)))
    return out


# --------------------------------------- head norms, window, 4-bit cache, blocks ---

# These calls take microseconds on the GPU, so their marshalling is kept short:
# one device query per tensor, a single strides pass for dense tensors, and the
# library's functions looked up once.

def _call(fn, dev: int, *args):
    """fn(*args, current stream of device ``dev``) with that device current."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        _check(status)


def _device(t: torch.Tensor) -> int:
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must live on a CUDA device")
    return dev


def _dense(t: Optional[torch.Tensor], dev: int, dtype, name: str, numel: int = -1):
    """Pointer of a dense tensor of the given type on device ``dev`` (None: NULL)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}")
    if t.get_device() != dev:
        _device(t)
        raise ValueError(f"{name} must live on cuda:{dev}")
    if numel >= 0 and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _like(x: torch.Tensor) -> torch.Tensor:
    """A dense tensor of x's shape and type (a third of torch.empty's host time)."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _tokens_view(x: torch.Tensor, name: str):
    """(tokens, stride) of x [..., heads, c] whose heads are dense and whose
    leading dims step by one token stride (elements)."""
    shape = x.shape
    heads, c = shape[-2], shape[-1]
    if x.is_contiguous():
        return (x.numel() // (heads * c) if heads and c else 0), heads * c
    strides = x.stride()
    if (c > 1 and strides[-1] != 1) or (heads > 1 and strides[-2] != c):
        raise ValueError(f"the heads of {name} must be dense")
    tokens, step = 1, 0
    for size, st in zip(shape[-3::-1], strides[-3::-1]):
        if size == 1:
            continue
        if tokens == 1:
            step = st
        elif st != step * tokens:
            raise ValueError(f"the tokens of {name} must step by one stride")
        tokens *= size
    return tokens, (step if tokens > 1 else heads * c)


def _per_head(gamma: torch.Tensor, heads: int, c: int, name: str) -> int:
    """0 for a weight [c], 1 for [heads, c]."""
    dims, n = gamma.dim(), gamma.numel()
    if dims == 1 and n == c:
        return 0
    if dims == 2 and n == heads * c and gamma.size(1) == c:
        return 1
    raise ValueError(f"{name} must be [c] or [heads, c]")


def csa_qk_norm_rope(q, k, pos, q_gamma=None, k_gamma=None, eps: float = NORM_EPS,
                     rope_dims: int = 64, rope_base: float = ROPE_BASE, halves: bool = False,
                     sections=None, q_out: Optional[torch.Tensor] = None,
                     k_out: Optional[torch.Tensor] = None):
    """RMSNorm (weight [c], or [heads, c] for one per head; None: no norm) and
    rotation of the trailing dims of q [..., nh, c] and k [..., nkv, c] in one
    pass; either may be None.  ``pos``: int64 [...] as the leading dims (or
    these flattened), or [axes, ...] with ``sections`` = the pairs of each
    axis.  q and k may be views with one token stride (of a packed
    projection); q_out and k_out may be q and k.  Returns (q_out, k_out)."""
    ref = q if q is not None else k
    if ref is None:
        raise ValueError("q or k must be given")
    dev, dt, dtype, shape = _device(ref), _dt(ref), ref.dtype, tuple(ref.shape)
    lead, c = shape[:-2], shape[-1]
    qp = kp = qop = kop = qg = kg = None
    qs = ks = qos = kos = nh = nkv = 0
    per_head = None
    if q is not None:
        nh = shape[-2]
        tokens, qs = _tokens_view(q, "q")
        if q_out is None:
            q_out, qos = _like(q), nh * c
        else:
            if q_out.shape != q.shape or q_out.dtype != dtype or q_out.get_device() != dev:
                raise ValueError("q_out must be like q")
            qos = _tokens_view(q_out, "q_out")[1]
        qp, qop = q.data_ptr(), q_out.data_ptr()
        if q_gamma is not None:
            qg = _dense(q_gamma, dev, torch.float32, "q_gamma")
            per_head = _per_head(q_gamma, nh, c, "q_gamma")
    if k is not None:
        shape = tuple(k.shape)
        nkv = shape[-2]
        tokens, ks = _tokens_view(k, "k")
        if shape[:-2] != lead or shape[-1] != c or k.dtype != dtype or k.get_device() != dev:
            raise ValueError("q and k must have the same leading dims, head dim, dtype and device")
        if k_out is None:
            k_out, kos = _like(k), nkv * c
        else:
            if k_out.shape != k.shape or k_out.dtype != dtype or k_out.get_device() != dev:
                raise ValueError("k_out must be like k")
            kos = _tokens_view(k_out, "k_out")[1]
        kp, kop = k.data_ptr(), k_out.data_ptr()
        if k_gamma is not None:
            kg = _dense(k_gamma, dev, torch.float32, "k_gamma")
            one = _per_head(k_gamma, nkv, c, "k_gamma")
            if per_head is not None and per_head != one:
                raise ValueError("q_gamma and k_gamma must both be [c] or both be [heads, c]")
            per_head = one
    p = QkRope(qg, kg, per_head or 0, eps, rope_dims, rope_base, 1 if halves else 0)
    axes = 1
    if sections is None:
        p.sections[0] = rope_dims // 2
    else:
        axes = len(sections)
        if not 1 <= axes <= 4:
            raise ValueError("1 to 4 sections")
        for i, n in enumerate(sections):
            p.sections[i] = n
    p.axes = axes
    pp = None
    if rope_dims and pos is not None:
        pp = _dense(pos, dev, torch.int64, "pos")
        shape = tuple(pos.shape)
        if axes > 1 or shape != lead:
            one = shape[1:] if shape[:1] == (axes,) else shape if axes == 1 else None
            if one != lead and one != (tokens,):
                raise ValueError("pos must have the leading dims of q and k, behind one of the axes "
                                 "where there are sections")
    _call(lib().csa_qk_norm_rope, dev, qp, qs, kp, ks, tokens, nh, nkv, c, pp, ctypes.byref(p), dt,
          qop, qos, kop, kos)
    return q_out if q is not None else None, k_out if k is not None else None


def csa_window_attn(q, k, v, window: int, first: int = 0, sink=None, scale: float = 1.0,
                    out: Optional[torch.Tensor] = None):
    """Causal attention over the last ``window`` tokens and the first ``first``
    ones: q [B, n_q, nh, c], k and v [B, n_k, nkv, c] (query i at position
    n_k - n_q + i; views with one token stride), or v None and k [B, n, c]:
    shared rows, each its own value.  Returns [B, n_q, nh, c]."""
    if v is None and k.dim() == 3:
        k = k.unsqueeze(2)
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, n_q, nh, c] and k [B, n_k, nkv, c]")
    dev, dt, dtype = _device(q), _dt(q), q.dtype
    B, nq, nh, c = q.shape
    _, nk, nkv, ck = k.shape
    if k.shape[0] != B or ck != c or k.dtype != dtype or k.get_device() != dev:
        raise ValueError("k must be [B, n_k, nkv, c] of q's dtype and device")
    vp, vs = None, 0
    if v is not None:
        if v.shape != k.shape or v.dtype != dtype or v.get_device() != dev:
            raise ValueError("v must be like k")
        vp, vs = v.data_ptr(), _tokens_view(v, "v")[1]
    if out is None:
        out = _like(q)
    elif out.shape != q.shape:
        raise ValueError("out must be like q")
    _call(lib().csa_window_attn, dev, q.data_ptr(), _tokens_view(q, "q")[1], k.data_ptr(),
          _tokens_view(k, "k")[1], vp, vs, window, first,
          _dense(sink, dev, torch.float32, "sink", nh), scale, B, nq, nk, nh, nkv, c, dt,
          _dense(out, dev, dtype, "out"))
    return out


def csa_kv4_block_bytes(nkv: int, c: int, block_tokens: int = 128) -> int:
    return int(lib().csa_kv4_block_bytes(nkv, c, block_tokens))


def csa_kv4_cache(num_blocks: int, nkv: int, c: int, block_tokens: int = 128,
                  device="cuda") -> torch.Tensor:
    """An empty 4-bit key/value cache: uint8 [num_blocks, nkv, block_tokens / 16, 18 c + 32]
    (c = 64 or 128)."""
    n = csa_kv4_block_bytes(nkv, c, block_tokens)
    if n == 0:
        raise ValueError("c must be 64 or 128, nkv >= 1 and block_tokens a multiple of 16")
    return torch.zeros((num_blocks, nkv, block_tokens // 16, 18 * c + 32), dtype=torch.uint8,
                       device=device)


def _kv4_desc(cache: torch.Tensor, block_table: torch.Tensor):
    """(device, descriptor, nkv, c) of a cache and its block table."""
    if cache.dim() != 4 or block_table.dim() != 2:
        raise ValueError("cache must be a uint8 [num_blocks, nkv, block_tokens / 16, bytes] tensor "
                         "and block_table an int32 [batch, max_blocks] tensor")
    nb, nkv, tiles, by = cache.shape
    c = (by - 32) // 18
    if by != 18 * c + 32:
        raise ValueError("the last dim of cache must be 18 c + 32 bytes")
    dev = _device(cache)
    return dev, Kv4Desc(_dense(cache, dev, torch.uint8, "cache"),
                        _dense(block_table, dev, torch.int32, "block_table"), *block_table.shape,
                        nb, nkv, c, 16 * tiles), nkv, c


def csa_kv4_store(cache, block_table, pos, k, v, count: Optional[torch.Tensor] = None):
    """Stores k and v [B, n, nkv, c] (bf16 or fp32, views with one token
    stride) in 4 bits at positions pos[b] + i; count: int32 [B] rows to store."""
    dev, d, nkv, c = _kv4_desc(cache, block_table)
    if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype or k.get_device() != dev \
            or v.get_device() != dev or k.shape[2] != nkv or k.shape[3] != c \
            or k.shape[0] != block_table.shape[0]:
        raise ValueError("k and v must be [batch, n, nkv, c] on the cache's device")
    B, n = k.shape[0], k.shape[1]
    _call(lib().csa_kv4_store, dev, ctypes.byref(d), _dense(pos, dev, torch.int64, "pos", B), n,
          _dense(count, dev, torch.int32, "count", B), k.data_ptr(), _tokens_view(k, "k")[1],
          v.data_ptr(), _tokens_view(v, "v")[1], _dt(k))


def csa_kv4_fetch(cache, block_table, pos, n: int, count: Optional[torch.Tensor] = None,
                  dtype=torch.bfloat16):
    """The stored rows of positions pos[b] .. pos[b] + n - 1 as k, v [B, n, nkv, c]
    (zeros from row count[b] on and where the block is absent)."""
    dev, d, nkv, c = _kv4_desc(cache, block_table)
    B = block_table.shape[0]
    k = torch.empty((B, n, nkv, c), dtype=dtype, device=cache.device)
    v = torch.empty((B, n, nkv, c), dtype=dtype, device=cache.device)
    _call(lib().csa_kv4_fetch, dev, ctypes.byref(d), _dense(pos, dev, torch.int64, "pos", B), n,
          _dense(count, dev, torch.int32, "count", B), _dt(k), k.data_ptr(), v.data_ptr())
    return k, v


def csa_kv4_decode_workspace(nh: int, nkv: int, c: int) -> int:
    return int(lib().csa_kv4_decode_workspace(nh, nkv, c))


def csa_kv4_decode_attn(q, cache, block_table, pos, scale: float, window: int = 0, first: int = 0,
                        sink=None, ws: Optional[torch.Tensor] = None,
                        out: Optional[torch.Tensor] = None):
    """Attention of one query token per sequence, q [B, nh, c] bf16 at position
    pos[b] (already stored), over the 4-bit cache: every token, or with
    ``window`` the last ``window`` and the first ``first`` ones."""
    dev, d, nkv, c = _kv4_desc(cache, block_table)
    if q.dim() != 3 or q.shape[0] != block_table.shape[0] or q.shape[2] != c:
        raise ValueError("q must be a bfloat16 [batch, nh, c] tensor on the cache's device")
    B, nh, _ = q.shape
    qp = _dense(q, dev, torch.bfloat16, "q")
    if out is None:
        out = _like(q)
    if ws is None:
        if dev == torch._C._cuda_getDevice():
            need = lib().csa_kv4_decode_workspace(nh, nkv, c)
        else:
            with torch.cuda.device(dev):
                need = lib().csa_kv4_decode_workspace(nh, nkv, c)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    elif ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("ws must be a dense tensor on the cache's device")
    _call(lib().csa_kv4_decode_attn, dev, ctypes.byref(d),
          _dense(pos, dev, torch.int64, "pos", B), qp, nh, window, first,
          _dense(sink, dev, torch.float32, "sink", nh), scale,
          _dense(out, dev, torch.bfloat16, "out", B * nh * c), ws.data_ptr(), ws.nbytes)
    return out


def csa_blocks_copy(regions, src, dst, count: Optional[torch.Tensor] = None):
    """In every region (a dense tensor [num_blocks, ...]) block dst[i] becomes a
    copy of block src[i] (int32 lists on the device; ids outside the pool are
    skipped; count: int32, count[0] pairs).  No block may be a destination
    twice, nor both a source and a destination."""
    if not regions:
        return
    if len(regions) > 16:
        raise ValueError("at most 16 regions")
    dev, nb = _device(regions[0]), regions[0].shape[0]
    arr = (BlockRegion * len(regions))()
    for a, r in zip(arr, regions):
        if r.shape[0] != nb or r.get_device() != dev or not r.is_contiguous():
            raise ValueError("regions must be dense and have the same blocks and device")
        a.base, a.block_bytes = r.data_ptr(), r.nbytes // nb if nb else 0
    n = src.numel()
    if count is not None and count.numel() < 1:
        raise ValueError("count must have an element")
    _call(lib().csa_blocks_copy, dev, arr, len(regions), nb,
          _dense(src, dev, torch.int32, "src"), _dense(dst, dev, torch.int32, "dst", n), n,
          _dense(count, dev, torch.int32, "count"))


def _table(table: torch.Tensor, out: Optional[torch.Tensor]):
    if table.dim() != 2:
        raise ValueError("table must be an int32 [rows, max_blocks] tensor")
    dev = _device(table)
    if out is None:
        out = _like(table)
    elif out.shape != table.shape:
        raise ValueError("table_out must be like table")
    return dev, _dense(table, dev, torch.int32, "table"), *table.shape, \
        _dense(out, dev, torch.int32, "table_out"), out


def csa_blocks_fork(table, src, dst, tokens, fresh, block_tokens: int = 128,
                    table_out: Optional[torch.Tensor] = None):
    """Row dst[i] of the new table forks the first tokens[i] (int64) tokens of row
    src[i]: whole blocks are shared, a partly filled last block becomes
    fresh[i].  Returns (table_out, copy_src, copy_dst); the copies (for
    csa_blocks_copy, once per cache) are -1 where there is nothing to copy."""
    dev, tp, rows, mb, op, out = _table(table, table_out)
    n = src.numel()
    cs, cd = table.new_empty((2, n)).unbind()
    i32 = torch.int32
    _call(lib().csa_blocks_fork, dev, tp, rows, mb, _dense(src, dev, i32, "src"),
          _dense(dst, dev, i32, "dst", n), _dense(tokens, dev, torch.int64, "tokens", n),
          _dense(fresh, dev, i32, "fresh", n), n, block_tokens, op, cs.data_ptr(), cd.data_ptr())
    return out, cs, cd


def csa_blocks_free(table, seqs, num_blocks: int, table_out: Optional[torch.Tensor] = None):
    """Rows ``seqs`` (int32) of the new table are -1.  Returns (table_out, freed,
    nfreed): the blocks no row names any more, ascending (int32 [num_blocks],
    -1 padded), and how many (int32 [1])."""
    dev, tp, rows, mb, op, out = _table(table, table_out)
    freed, n = table.new_empty(num_blocks), table.new_empty(1)
    _call(lib().csa_blocks_free, dev, tp, rows, mb, num_blocks,
          _dense(seqs, dev, torch.int32, "seqs"), seqs.numel(), op, freed.data_ptr(), n.data_ptr())
    return out, freed, n


def csa_blocks_compact(table, num_blocks: int, table_out: Optional[torch.Tensor] = None):
    """The blocks in use move to the low end of the pool.  Returns (table_out,
    copy_src, copy_dst, counts): the moves (int32 [num_blocks], -1 padded; for
    csa_blocks_copy with count=counts, once per cache) and counts = [moves,
    blocks in use]."""
    dev, tp, rows, mb, op, out = _table(table, table_out)
    cs, cd = table.new_empty((2, num_blocks)).unbind()
    counts = table.new_empty(2)
    _call(lib().csa_blocks_compact, dev, tp, rows, mb, num_blocks, op, cs.data_ptr(),
          cd.data_ptr(), counts.data_ptr())
    return out, cs, cd, counts


# ------------------------------------------------------------------- decode ---

class CsaCache:
    """A caller-owned decode cache (one layer, ``batch`` sequences).

    With ``block_table`` (int32 [batch, max_blocks] on the device) the
    compressed entries live in a paged pool of ``num_blocks`` blocks of
    ``block_tokens`` raw tokens each (the classical cache; capacity becomes
    max_blocks * block_tokens // m); the window ring and the compressor tail
    stay per sequence."""

    def __init__(self, batch: int, capacity: int, c: int, rope_dims: int, m: int, window: int,
                 nh: int, is_hca: bool, c_i: int = 0, nh_i: int = 0, k: int = 0,
                 device="cuda", block_table: Optional[torch.Tensor] = None,
                 block_tokens: int = 128, num_blocks: int = 0):
        self.paging = None
        if block_table is not None:
            if block_table.dtype != torch.int32 or block_table.dim() != 2:
                raise ValueError("block_table must be an int32 [batch, max_blocks] tensor")
            self.block_table = block_table
            capacity = block_table.shape[1] * (block_tokens // m)
            self.paging = Paging(int(block_tokens), int(num_blocks), int(block_table.shape[1]),
                                 _ptr(block_table))
        self.desc = CacheDesc(batch, capacity, c, rope_dims, c_i, m, window, nh, nh_i, k,
                              1 if is_hca else 0)
        self.layout = CacheLayout()
        if self.paging is not None:
            _check(lib().csa_paged_cache_layout(ctypes.byref(self.desc), ctypes.byref(self.paging),
                                                ctypes.byref(self.layout)))
        else:
            _check(lib().csa_cache_layout(ctypes.byref(self.desc), ctypes.byref(self.layout)))
        self.buffer = torch.zeros(self.layout.total_bytes, dtype=torch.uint8, device=device)
        ws = int(lib().csa_decode_workspace(ctypes.byref(self.desc)))
        self.workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=device)

    # views of the regions (for tests and inspection)
    def region(self, name: str, dtype, shape):
        off = getattr(self.layout, name)
        nbytes = int(torch.tensor(shape).prod().item()) * torch.empty((), dtype=dtype).element_size()
        return self.buffer[off:off + nbytes].view(dtype).view(*shape)

    def entries(self):
        """The entry regions as [batch, capacity, ...] (gathered through the
        block table when paged; absent blocks read as zeros)."""
        d = self.desc
        B, cap = d.batch, d.capacity
        rows = B * cap
        if self.paging is not None:
            epb = self.paging.block_tokens // d.m
            rows = self.paging.num_blocks * epb
        out = dict(codes=self.region("entry_fp8", torch.uint8, (rows, d.c - d.rope_dims)),
                   scale=self.region("entry_scale", torch.float32, (rows,)),
                   rope=self.region("entry_rope", torch.bfloat16, (rows, d.rope_dims)))
        if not d.is_hca:
            out["icodes"] = self.region("ikey_fp8", torch.uint8, (rows, d.c_i))
            out["iscale"] = self.region("ikey_scale", torch.float32, (rows,))
        if self.paging is None:
            return {k: v.view(B, cap, *v.shape[1:]) for k, v in out.items()}
        bt = self.block_table.long()
        s = torch.arange(cap, device=bt.device)
        blk = bt[:, s // epb]                                       # [B, cap]
        ok = (blk >= 0) & (blk < self.paging.num_blocks)
        row = torch.where(ok, blk * epb + (s % epb)[None, :], torch.zeros_like(blk))
        res = {}
        for k, v in out.items():
            g = v[row.reshape(-1)].reshape(B, cap, *v.shape[1:]).clone()
            g[~ok] = 0
            res[k] = g
        return res

    def copy_blocks(self, src, dst, count: Optional[torch.Tensor] = None):
        """Copies blocks of the paged pool (csa_blocks_copy over every entry region)."""
        if self.paging is None:
            raise ValueError("only a paged cache has blocks")
        d, nb = self.desc, self.paging.num_blocks
        epb = self.paging.block_tokens // d.m
        regions = [self.region("entry_fp8", torch.uint8, (nb, epb * (d.c - d.rope_dims))),
                   self.region("entry_scale", torch.float32, (nb, epb)),
                   self.region("entry_rope", torch.bfloat16, (nb, epb * d.rope_dims))]
        if not d.is_hca:
            regions += [self.region("ikey_fp8", torch.uint8, (nb, epb * d.c_i)),
                        self.region("ikey_scale", torch.float32, (nb, epb))]
        csa_blocks_copy(regions, src, dst, count)

    def copy_sequences(self, src, dst, count: Optional[torch.Tensor] = None):
        """Copies what the cache keeps per sequence (window ring and compressor
        state; without paging the entries too) of sequences src to dst."""
        d, B = self.desc, self.desc.batch
        regions = [self.region("window", torch.bfloat16, (B, d.window * d.c)),
                   self.region("state", torch.bfloat16, (B, (2 if d.is_hca else 8) * d.m * d.c))]
        if not d.is_hca:
            regions.append(self.region("istate", torch.bfloat16, (B, 8 * d.m * d.c_i)))
        if self.paging is None:
            cap = d.capacity
            regions += [self.region("entry_fp8", torch.uint8, (B, cap * (d.c - d.rope_dims))),
                        self.region("entry_scale", torch.float32, (B, cap)),
                        self.region("entry_rope", torch.bfloat16, (B, cap * d.rope_dims))]
            if not d.is_hca:
                regions += [self.region("ikey_fp8", torch.uint8, (B, cap * d.c_i)),
                            self.region("ikey_scale", torch.float32, (B, cap))]
        csa_blocks_copy(regions, src, dst, count)

    def store_entries(self, first: int, kv, ikey=None):
        count = kv.shape[1]
        if self.paging is not None:
            _check(lib().csa_paged_cache_store_entries(
                ctypes.byref(self.desc), ctypes.byref(self.paging), _ptr(self.buffer), first,
                count, _ptr(kv), _ptr(ikey), _dt(kv), _stream(self.buffer)))
            return
        _check(lib().csa_cache_store_entries(ctypes.byref(self.desc), _ptr(self.buffer), first,
                                             count, _ptr(kv), _ptr(ikey), _dt(kv),
                                             _stream(self.buffer)))

    @staticmethod
    def _rows(rows: dict) -> Rows:
        r = Rows()
        for nm in ("ca", "cb", "za", "zb", "ica", "icb", "iza", "izb", "kv_win"):
            t = rows.get(nm)
            if t is not None and t.dtype != torch.bfloat16:
                raise ValueError(f"row stream {nm} must be bfloat16")
            setattr(r, nm, _ptr(t))
        return r

    def write_rows(self, first_pos: int, rows: dict):
        count = rows["kv_win"].shape[1]
        r = self._rows(rows)
        if self.paging is not None:
            _check(lib().csa_paged_cache_write_rows(
                ctypes.byref(self.desc), ctypes.byref(self.paging), _ptr(self.buffer), first_pos,
                count, ctypes.byref(r), _stream(self.buffer)))
            return
        _check(lib().csa_cache_write_rows(ctypes.byref(self.desc), _ptr(self.buffer), first_pos,
                                          count, ctypes.byref(r), _stream(self.buffer)))

    def decode_step(self, pos, rows: dict, biases: dict, sink, scale: float, q, q_i=None,
                    w_i=None, out: Optional[torch.Tensor] = None,
                    sel_out: Optional[torch.Tensor] = None,
                    scores_out: Optional[torch.Tensor] = None):
        """One token per sequence at positions ``pos`` (int64 [B] on device).

        ``rows``: per-stream [B, dim] bf16 tensors; ``biases``: ba, bb, iba, ibb
        fp32; returns out [B, nh, c] bf16.  ``sel_out`` (CSA, optional, int32
        [B, k] on device) receives the selected entry indices; ``scores_out``
        (CSA, optional, fp32 [B, capacity] on device) the indexer scores."""
        if out is None:
            out = torch.empty_like(q)
        r = self._rows({k: v for k, v in rows.items()})
        if sel_out is not None and (sel_out.dtype != torch.int32 or not sel_out.is_contiguous()
                                    or sel_out.numel() != self.desc.batch * self.desc.k):
            raise ValueError("sel_out must be a contiguous int32 [batch, k] tensor")
        if scores_out is not None and (
                scores_out.dtype != torch.float32 or not scores_out.is_contiguous()
                or scores_out.numel() != self.desc.batch * self.desc.capacity):
            raise ValueError("scores_out must be a contiguous float32 [batch, capacity] tensor")
        p = DecodeParams(_ptr(biases.get("ba")), _ptr(biases.get("bb")), _ptr(biases.get("iba")),
                         _ptr(biases.get("ibb")), _ptr(sink), float(scale), _ptr(sel_out),
                         _ptr(scores_out))
        if pos.dtype != torch.int64:
            raise ValueError("pos must be int64")
        if self.paging is not None:
            _check(lib().csa_paged_decode_step(
                ctypes.byref(self.desc), ctypes.byref(self.paging), _ptr(self.buffer), _ptr(pos),
                ctypes.byref(r), ctypes.byref(p), _ptr(q), _ptr(q_i), _ptr(w_i), _ptr(out),
                _ptr(self.workspace), self.workspace.numel(), _stream(q)))
            return out
        _check(lib().csa_decode_step(ctypes.byref(self.desc), _ptr(self.buffer), _ptr(pos),
                                     ctypes.byref(r), ctypes.byref(p), _ptr(q), _ptr(q_i),
                                     _ptr(w_i), _ptr(out), _ptr(self.workspace),
                                     self.workspace.numel(), _stream(q)))
        return out
