"""Thin ctypes binding of libqsa.so (include/qsa.h): argument marshalling only.

Every call takes torch tensors that already live on the GPU and passes their device
pointers and the stream handle to the C ABI; every step of the decode path runs in
the library's CUDA kernels. There is no fallback: if libqsa.so is missing or cannot be
loaded, importing the binding's library raises.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import c_float, c_int32, c_int64, c_size_t, c_void_p

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqsa.so")

QSA_OK = 0
STATUS_NAMES = {0: "QSA_OK", 1: "QSA_ERR_INVALID_ARG", 2: "QSA_ERR_CAPACITY", 3: "QSA_ERR_STATE",
                4: "QSA_ERR_CUDA", 5: "QSA_ERR_UNSUPPORTED", 6: "QSA_ERR_BAD_INDEX",
                7: "QSA_ERR_TIMEOUT"}
(QSA_BUF_KV, QSA_BUF_IDX, QSA_BUF_POOLED, QSA_BUF_WORKSPACE, QSA_BUF_MAX_CELLS, QSA_BUF_SCORE_STRIDE,
 QSA_BUF_KV_SCALES, QSA_BUF_POOLED_SCALES) = range(8)
QSA_KV_F16, QSA_KV_FP8 = 0, 1
QSA_SCAN_TENSOR, QSA_SCAN_CUDA_CORES = 0, 1
QSA_POOLED_F16, QSA_POOLED_FP8 = 0, 1
QSA_INPUTS_ORDERED, QSA_INPUTS_EARLY = 0, 1
QSA_MAX_QUERIES = 4
QSA_MAX_DRAFTS = 64
QSA_PAGE_F16, QSA_PAGE_FP8, QSA_PAGE_INT4 = range(3)
QSA_PAGED_BUF_PAGES, QSA_PAGED_BUF_SCALES = 0, 1


class QsaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


class QsaConfig(ctypes.Structure):
    _fields_ = [("n_layers", c_int32), ("max_ctx", c_int32), ("d_idx", c_int32),
                ("n_idx_heads", c_int32), ("top_k_tokens", c_int32), ("n_q_heads", c_int32),
                ("n_kv_heads", c_int32), ("head_dim", c_int32), ("rope_base", c_float),
                ("rms_eps", c_float), ("rope_dims", c_int32), ("rope_interleaved", c_int32),
                ("rope_pos_stride", c_int32), ("rope_pos_offset", c_int32), ("kv_format", c_int32),
                ("scan_kind", c_int32), ("pooled_format", c_int32), ("early_inputs", c_int32)]


class QsaLayerBuffers(ctypes.Structure):
    _fields_ = [("k_cache", c_void_p), ("v_cache", c_void_p), ("idx_cache", c_void_p),
                ("pooled_cache", c_void_p), ("rms_gain", c_void_p), ("workspace", c_void_p),
                ("kv_scales", c_void_p), ("pooled_scales", c_void_p)]


class QsaPagedKv(ctypes.Structure):
    _fields_ = [("n_pages", c_int32), ("page_size", c_int32), ("n_kv_heads", c_int32), ("head_dim", c_int32),
                ("format", c_int32), ("reserved", c_int32), ("page_stride", c_int64), ("scale_stride", c_int64),
                ("k_pages", c_void_p), ("v_pages", c_void_p), ("k_scales", c_void_p), ("v_scales", c_void_p)]


_P = c_void_p
_I = c_int32
_L = c_int64
_F = c_float
_Z = c_size_t
_KV = ctypes.POINTER(QsaPagedKv)
# name -> (restype, argtypes); must list every function include/qsa.h declares
SIGNATURES = {
    "qsa_buffer_bytes": (c_size_t, [ctypes.POINTER(QsaConfig), _I]),
    "qsa_create": (_I, [ctypes.POINTER(QsaConfig), ctypes.POINTER(_P)]),
    "qsa_destroy": (None, [_P]),
    "qsa_last_error": (ctypes.c_char_p, [_P]),
    "qsa_bind_layer": (_I, [_P, _I, ctypes.POINTER(QsaLayerBuffers), _P]),
    "qsa_restore_layer": (_I, [_P, _I, _I, _I, _P]),
    "qsa_read_layer_state": (_I, [_P, _I, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I), _I, _P]),
    "qsa_append_token": (_I, [_P, _I, _P, _P, _P, _P]),
    "qsa_append_tokens": (_I, [_P, _I, _I, _P, _P, _P, _P]),
    "qsa_update_pooled_cache": (_I, [_P, _I, _P]),
    "qsa_decode_append": (_I, [_P, _I, _P, _P, _P, _P]),
    "qsa_invalidate_pooled_cache": (_I, [_P, _I, _I, _P]),
    "qsa_index_topk": (_I, [_P, _I, _P, _P, _P, _P, _P, _P]),
    "qsa_index_scores": (_I, [_P, _I, _P, _P, _P, _P]),
    "qsa_select_topk": (_I, [_P, _I, _P, _P, _P, _P]),
    "qsa_gather_kv": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _P]),
    "qsa_sparse_attend": (_I, [_P, _I, _P, _P, _P, _P, _P]),
    "qsa_sparse_attend_selected": (_I, [_P, _I, _P, _P, _P, _P, _P]),
    "qsa_sparse_attend_noalloc": (_I, [_P, _P, _P, _I, _P, _P, _P, _I, _I, _I, _I, _P]),
    "qsa_index_topk_multi": (_I, [_P, _I, _I, _P, _P, _P, _P, _P, _P]),
    "qsa_sparse_attend_selected_multi": (_I, [_P, _I, _I, _P, _P, _P, _P, _P]),
    "qsa_rollback": (_I, [_P, _I, _I, _P]),
    "qsa_layer_bytes": (c_size_t, [ctypes.POINTER(QsaConfig), _I]),
    "qsa_n_ctx": (_I, [_P, _I]),
    "qsa_get_device_status": (_I, [_P, ctypes.POINTER(_I)]),
    "qsa_decode_step": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "qsa_cp_index_candidates": (_I, [_P, _I, _P, _P, _I, _I, _P, _P, _P, _P]),
    "qsa_cp_select": (_I, [_P, _P, _I, _I, _P, _P, _P]),
    "qsa_cp_attend_partial": (_I, [_P, _I, _P, _P, _P, _I, _P, _P, _P]),
    "qsa_cp_merge": (_I, [_P, _P, _I, _I, _I, _P, _P]),
    "qsa_rollback_rejected": (_I, [_P, _I, _I, _P, _P]),
    "qsa_verify_drafts": (_I, [_P, _L, _P, _L, _P, _P, _P, _I, _I, _I, _P, _P, _P, _P]),
    "qsa_paged_bytes": (c_size_t, [_KV, _I]),
    "qsa_paged_write": (_I, [_KV, _P, _P, _L, _I, _P, _I, _I, _P, _P, _P, _P]),
    "qsa_paged_read": (_I, [_KV, _P, _P, _L, _I, _P, _I, _I, _P, _P, _P, _P]),
    "qsa_paged_workspace_bytes": (c_size_t, [_KV, _I, _I]),
    "qsa_paged_attend": (_I, [_KV, _P, _L, _I, _I, _P, _I, _I, _P, _F, _P, _P, _P, _Z, _P, _P]),
}

_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libqsa.so (or the library QSA_LIBRARY names, e.g. the checked build) and
    declare its signatures. Raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or os.environ.get("QSA_LIBRARY") or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(f"{p} is missing: build it with `python -m sparse_attention_decode_02_b200.build`")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib


def _ptr(t):
    """Device pointer of a torch tensor (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("tensors passed to the QSA library must live on the GPU")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the QSA library must be contiguous")
    return t.data_ptr()


_raw_stream = None


def _stream(stream):
    """Handle of `stream` (default: the current one of the current device)."""
    global _raw_stream
    if stream is not None:
        return getattr(stream, "cuda_stream", stream)
    if _raw_stream is None:
        import torch
        # the handle itself where torch gives it, without a Stream object around it (3 us a call)
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _raw_stream = (lambda: raw(torch._C._cuda_getDevice())) if raw and torch.cuda.is_initialized() else \
            (lambda: torch.cuda.current_stream().cuda_stream)
    return _raw_stream()


def make_config(n_layers, max_ctx, d_idx, n_idx_heads, top_k_tokens, n_q_heads, n_kv_heads, head_dim,
                rope_base=10000.0, rms_eps=1e-6, rope_dims=0, rope_interleaved=False, rope_pos_stride=4,
                rope_pos_offset=0, kv_format=QSA_KV_F16, scan_kind=QSA_SCAN_TENSOR,
                pooled_format=QSA_POOLED_F16, early_inputs=QSA_INPUTS_ORDERED) -> QsaConfig:
    return QsaConfig(n_layers, max_ctx, d_idx, n_idx_heads, top_k_tokens, n_q_heads, n_kv_heads, head_dim,
                     rope_base, rms_eps, rope_dims, int(bool(rope_interleaved)), rope_pos_stride, rope_pos_offset,
                     kv_format, scan_kind, pooled_format, early_inputs)


def buffer_bytes(cfg: QsaConfig, which: int) -> int:
    return int(load_library().qsa_buffer_bytes(ctypes.byref(cfg), which))


class Qsa:
    """One library context (qsa_ctx) on the current CUDA device. Method names follow the C ABI."""

    def __init__(self, cfg: QsaConfig):
        self.lib = load_library()
        self.cfg = cfg
        h = c_void_p()
        st = self.lib.qsa_create(ctypes.byref(cfg), ctypes.byref(h))
        if st != QSA_OK:
            raise QsaError(st, "qsa_create rejected the configuration")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            self.lib.qsa_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _check(self, st):
        if st != QSA_OK:
            msg = self.lib.qsa_last_error(self.handle)
            raise QsaError(st, msg.decode() if msg else "")

    def buffer_bytes(self, which: int) -> int:
        return buffer_bytes(self.cfg, which)

    def bind_layer(self, layer, k_cache, v_cache, idx_cache, pooled_cache, workspace, rms_gain=None,
                   kv_scales=None, pooled_scales=None, stream=None):
        b = QsaLayerBuffers(_ptr(k_cache), _ptr(v_cache), _ptr(idx_cache), _ptr(pooled_cache),
                            _ptr(rms_gain), _ptr(workspace), _ptr(kv_scales), _ptr(pooled_scales))
        self._check(self.lib.qsa_bind_layer(self.handle, layer, ctypes.byref(b), _stream(stream)))

    def restore_layer(self, layer, n_ctx, n_pooled, stream=None):
        self._check(self.lib.qsa_restore_layer(self.handle, layer, n_ctx, n_pooled, _stream(stream)))

    def read_layer_state(self, layer, clear=False, stream=None):
        n, p, s = c_int32(), c_int32(), c_int32()
        self._check(self.lib.qsa_read_layer_state(self.handle, layer, ctypes.byref(n), ctypes.byref(p),
                                                  ctypes.byref(s), int(clear), _stream(stream)))
        return n.value, p.value, s.value

    def append_token(self, layer, k, v, idx_key, stream=None):
        self._check(self.lib.qsa_append_token(self.handle, layer, _ptr(k), _ptr(v), _ptr(idx_key),
                                              _stream(stream)))

    def append_tokens(self, layer, k, v, idx_key, stream=None):
        self._check(self.lib.qsa_append_tokens(self.handle, layer, int(k.shape[0]), _ptr(k), _ptr(v),
                                               _ptr(idx_key), _stream(stream)))

    def decode_append(self, layer, k, v, idx_key, stream=None):
        self._check(self.lib.qsa_decode_append(self.handle, layer, _ptr(k), _ptr(v), _ptr(idx_key), _stream(stream)))

    def update_pooled_cache(self, layer, stream=None):
        self._check(self.lib.qsa_update_pooled_cache(self.handle, layer, _stream(stream)))

    def invalidate_pooled_cache(self, layer, from_block, stream=None):
        self._check(self.lib.qsa_invalidate_pooled_cache(self.handle, layer, from_block, _stream(stream)))

    def index_topk(self, layer, q_idx, w, sel_blocks, n_sel, scores=None, stream=None):
        self._check(self.lib.qsa_index_topk(self.handle, layer, _ptr(q_idx), _ptr(w), _ptr(sel_blocks),
                                            _ptr(n_sel), _ptr(scores), _stream(stream)))

    def index_scores(self, layer, q_idx, w, scores, stream=None):
        self._check(self.lib.qsa_index_scores(self.handle, layer, _ptr(q_idx), _ptr(w), _ptr(scores),
                                              _stream(stream)))

    def select_topk(self, layer, scores, sel_blocks, n_sel, stream=None):
        self._check(self.lib.qsa_select_topk(self.handle, layer, _ptr(scores), _ptr(sel_blocks), _ptr(n_sel),
                                             _stream(stream)))

    def gather_kv(self, layer, sel_blocks, n_sel, cells, n_cells, k_compact=None, v_compact=None,
                  stream=None):
        self._check(self.lib.qsa_gather_kv(self.handle, layer, _ptr(sel_blocks), _ptr(n_sel), _ptr(cells),
                                           _ptr(n_cells), _ptr(k_compact), _ptr(v_compact), _stream(stream)))

    def sparse_attend_selected(self, layer, q, sel_blocks, n_sel, out, stream=None):
        self._check(self.lib.qsa_sparse_attend_selected(self.handle, layer, _ptr(q), _ptr(sel_blocks), _ptr(n_sel),
                                                        _ptr(out), _stream(stream)))

    def sparse_attend(self, layer, q, cells, n_cells, out, stream=None):
        self._check(self.lib.qsa_sparse_attend(self.handle, layer, _ptr(q), _ptr(cells), _ptr(n_cells),
                                               _ptr(out), _stream(stream)))

    def index_topk_multi(self, layer, q_idx, w, sel_blocks, n_sel, scores=None, stream=None):
        """T = q_idx.shape[0] queries (the last T tokens) in one scan and one selection."""
        self._check(self.lib.qsa_index_topk_multi(self.handle, layer, int(q_idx.shape[0]), _ptr(q_idx), _ptr(w),
                                                  _ptr(sel_blocks), _ptr(n_sel), _ptr(scores), _stream(stream)))

    def sparse_attend_selected_multi(self, layer, q, sel_blocks, n_sel, out, stream=None):
        self._check(self.lib.qsa_sparse_attend_selected_multi(self.handle, layer, int(q.shape[0]), _ptr(q),
                                                              _ptr(sel_blocks), _ptr(n_sel), _ptr(out),
                                                              _stream(stream)))

    def rollback(self, layer, n_keep, stream=None):
        self._check(self.lib.qsa_rollback(self.handle, layer, int(n_keep), _stream(stream)))

    def rollback_rejected(self, layer, n_drafts, n_accepted, stream=None):
        """Of the n_drafts newest tokens keep the first n_accepted (a device i32)."""
        self._check(self.lib.qsa_rollback_rejected(self.handle, layer, int(n_drafts), _ptr(n_accepted),
                                                   _stream(stream)))

    def decode_step(self, layer, k, v, idx_key, q_idx, w, q, sel_blocks, n_sel, out, stream=None):
        """The whole hot path of one decode step of one layer in one ABI call."""
        self._check(self.lib.qsa_decode_step(self.handle, layer, _ptr(k), _ptr(v), _ptr(idx_key), _ptr(q_idx),
                                             _ptr(w), _ptr(q), _ptr(sel_blocks), _ptr(n_sel), _ptr(out),
                                             _stream(stream)))

    def cp_index_candidates(self, layer, q_idx, w, n_global, block_base, cand_scores, cand_blocks, n_cand,
                            stream=None):
        """A context-parallel shard's scan (query at global position n_global - 1) and its
        local top-K as fixed-size slots of scores and global block ids."""
        self._check(self.lib.qsa_cp_index_candidates(self.handle, layer, _ptr(q_idx), _ptr(w), int(n_global),
                                                     int(block_base), _ptr(cand_scores), _ptr(cand_blocks),
                                                     _ptr(n_cand), _stream(stream)))

    def cp_attend_partial(self, layer, q, sel_blocks, n_sel, block_base, out, lse, stream=None):
        """A context-parallel shard's attention over its part of the global selection:
        normalised output and per-head log-sum-exp."""
        self._check(self.lib.qsa_cp_attend_partial(self.handle, layer, _ptr(q), _ptr(sel_blocks), _ptr(n_sel),
                                                   int(block_base), _ptr(out), _ptr(lse), _stream(stream)))

    def n_ctx(self, layer) -> int:
        """Tokens in the layer's caches (synchronises the device)."""
        n = self.lib.qsa_n_ctx(self.handle, layer)
        if n < 0:
            raise QsaError(1, f"qsa_n_ctx failed for layer {layer}")
        return n

    def device_status(self) -> int:
        """First non-zero device status word over the bound layers (synchronises the device)."""
        st = c_int32()
        self._check(self.lib.qsa_get_device_status(self.handle, ctypes.byref(st)))
        return st.value


def cp_select(cand_scores, cand_blocks, n_shards, k_blocks, sel_blocks, n_sel, stream=None):
    """qsa_cp_select: the global top-K of every shard's candidate slots."""
    st = load_library().qsa_cp_select(_ptr(cand_scores), _ptr(cand_blocks), int(n_shards), int(k_blocks),
                                      _ptr(sel_blocks), _ptr(n_sel), _stream(stream))
    if st != QSA_OK:
        raise QsaError(st, "qsa_cp_select failed")


def cp_merge(o_parts, lse_parts, n_shards, n_q_heads, head_dim, out, stream=None):
    """qsa_cp_merge: the exact merge of the shards' attention partials."""
    st = load_library().qsa_cp_merge(_ptr(o_parts), _ptr(lse_parts), int(n_shards), int(n_q_heads), int(head_dim),
                                     _ptr(out), _stream(stream))
    if st != QSA_OK:
        raise QsaError(st, "qsa_cp_merge failed")


def sparse_attend_noalloc(q, k_cache, v_cache, n_ctx, cells, n_cells, out, n_q_heads, n_kv_heads, head_dim,
                          top_k_tokens, stream=None):
    """qsa_sparse_attend_noalloc: attention with the library's fixed scratch array (no
    context, no workspace). Raises QsaError with the returned status on failure."""
    st = load_library().qsa_sparse_attend_noalloc(_ptr(q), _ptr(k_cache), _ptr(v_cache), int(n_ctx), _ptr(cells),
                                                  _ptr(n_cells), _ptr(out), n_q_heads, n_kv_heads, head_dim,
                                                  top_k_tokens, _stream(stream))
    if st != QSA_OK:
        raise QsaError(st, "qsa_sparse_attend_noalloc failed")


class _Types:
    """torch's types, looked up once: the calls below check their arguments in a few attribute reads."""
    f16 = f32 = i32 = u8 = e4m3 = device = None

    @classmethod
    def load(cls):
        import torch
        cls.f16, cls.f32, cls.i32, cls.u8, cls.e4m3 = (torch.float16, torch.float32, torch.int32, torch.uint8,
                                                       torch.float8_e4m3fn)
        cls.device = staticmethod(torch.cuda.current_device)


def _bad(name, t, dtype, shape):
    want = " x ".join("?" if w is None else str(w) for w in shape)
    raise ValueError(f"{name} must be a {dtype} tensor of shape [{want}] on the current device, "
                     f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _arg(name, t, dtype, shape, device):
    """Device pointer of a contiguous argument of this type and shape on the current device."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        _bad(name, t, dtype, shape)
    return t.data_ptr()


def _rows_stride(name, t, dtype, shape, device):
    """Elements between the rows of an argument whose last dims are contiguous rows and whose
    leading dims (shape[:2] of 3 or 4) lie evenly apart; 0 if packed."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != device:
        _bad(name, t, dtype, shape)
    if t.is_contiguous():
        return 0
    st, row = t.stride(), 1
    for n, d in zip(reversed(shape[2:]), reversed(st[2:])):
        if n > 1 and d != row:
            raise ValueError(f"rows of {name} must be contiguous")
        row *= n
    step = st[1] if shape[1] > 1 else st[0] if shape[0] > 1 else row
    if step < row or (shape[0] > 1 and shape[1] > 1 and st[0] != shape[1] * step):
        raise ValueError(f"rows of {name} must be equally far apart")
    return step


class PagedKV:
    """A paged K/V cache over tensors the caller owns (qsa_paged_kv):
    k_pages, v_pages [n_pages, n_kv_heads, page_size, row] with rows of head_dim f16 values
    (QSA_PAGE_F16), head_dim e4m3 codes (QSA_PAGE_FP8, a one-byte type) or head_dim/2 bytes of
    4-bit codes (QSA_PAGE_INT4); k_scales, v_scales [n_pages, n_kv_heads, page_size] f32
    (FP8) or [n_pages, n_kv_heads, page_size, head_dim/32] f16 (INT4). Pages may lie apart
    (a layer's part of one pool: stride(0) larger than a page), the rest is contiguous."""

    def __init__(self, k_pages, v_pages, page_format, k_scales=None, v_scales=None):
        if _Types.f32 is None:
            _Types.load()
        self.lib = load_library()
        self._attend = self.lib.qsa_paged_attend
        self.tensors = (k_pages, v_pages, k_scales, v_scales)  # kept alive with the descriptor
        if page_format not in (QSA_PAGE_F16, QSA_PAGE_FP8, QSA_PAGE_INT4):
            raise ValueError("page_format must be QSA_PAGE_F16, QSA_PAGE_FP8 or QSA_PAGE_INT4")
        if k_pages.dim() != 4:
            raise ValueError("k_pages must be [n_pages, n_kv_heads, page_size, row]")
        n, heads, page, row = k_pages.shape
        if n < 1:
            raise QsaError(1, "a paged cache has at least one page")
        self.head_dim = 2 * row if page_format == QSA_PAGE_INT4 else row
        self.n_kv_heads, self.device = heads, k_pages.get_device()
        types = {QSA_PAGE_F16: (_Types.f16,), QSA_PAGE_FP8: (_Types.u8, _Types.e4m3), QSA_PAGE_INT4: (_Types.u8,)}
        want = [("k_pages", k_pages, types[page_format], (n, heads, page, row)),
                ("v_pages", v_pages, (k_pages.dtype,), (n, heads, page, row))]
        if page_format == QSA_PAGE_F16:
            k_scales = v_scales = None
        elif k_scales is None or v_scales is None:
            raise ValueError("this page format has scales")
        else:
            fp8 = page_format == QSA_PAGE_FP8
            shape = (n, heads, page) if fp8 else (n, heads, page, self.head_dim // 32)
            kind = _Types.f32 if fp8 else _Types.f16
            want += [("k_scales", k_scales, (kind,), shape), ("v_scales", v_scales, (kind,), shape)]
        for name, t, kinds, shape in want:
            if t.dtype not in kinds or t.shape != shape:
                _bad(name, t, " or ".join(map(str, kinds)), shape)

        def stride(a, b):  # bytes between pages; pages themselves contiguous
            if a is None:
                return 0
            for t in (a, b):
                if not t.is_cuda or t.get_device() != self.device:
                    raise ValueError("pages and scales must live on one GPU")
                if not t[0].is_contiguous() or (n > 1 and (t.stride(0) != a.stride(0) or t.stride(0) < t[0].numel())):
                    raise ValueError("pages must be contiguous and K and V pages equally far apart")
            return a.stride(0) * a.element_size() if n > 1 else 0

        addr = [None if t is None else t.data_ptr() for t in (k_pages, v_pages, k_scales, v_scales)]
        self.desc = QsaPagedKv(n, page, heads, self.head_dim, page_format, 0, stride(k_pages, v_pages),
                               stride(k_scales, v_scales), *addr)
        self._ref = ctypes.byref(self.desc)
        if self.lib.qsa_paged_bytes(self._ref, QSA_PAGED_BUF_PAGES) == 0:
            raise QsaError(5, "no such paged cache: page_size 16..256 (a power of two), head_dim 64 or 128")

    def _rows(self, k, v, block_table, first, row_start, status):
        a = k if k is not None else v
        if a is None:
            raise ValueError("k and v must not both be None")
        dev = self._device()
        n_rows, shape = a.shape[0], (1, a.shape[0], self.n_kv_heads, self.head_dim)
        stride = _rows_stride("k", a[None], _Types.f16, shape, dev) if not a.is_contiguous() or a.dim() != 3 else 0
        for name, t in (("k", k), ("v", v)):
            if t is not None and (t.dtype != _Types.f16 or t.shape != shape[1:] or t.get_device() != dev or
                                  (t is not a and t.stride() != a.stride() and n_rows > 0)):
                _bad(name, t, _Types.f16, shape[1:])
        n_seqs, width = block_table.shape
        return (k.data_ptr() if k is not None else None, v.data_ptr() if v is not None else None, stride, n_rows,
                _arg("block_table", block_table, _Types.i32, (n_seqs, width), dev), width, n_seqs,
                _arg("first", first, _Types.i32, (n_seqs,), dev),
                _arg("row_start", row_start, _Types.i32, (n_seqs + 1,), dev),
                None if status is None else _arg("status", status, _Types.i32, (1,), dev))

    def _device(self):
        """The current device, which must be the cache's."""
        dev = _Types.device()
        if dev != self.device:
            raise ValueError(f"the cache lives on cuda:{self.device}, the current device is cuda:{dev}")
        return dev

    def write(self, k, v, block_table, first, row_start, status=None, stream=None):
        """qsa_paged_write: stores rows k, v [n_rows, n_kv_heads, head_dim] f16 (rows may lie apart)."""
        if k is None or v is None:
            raise ValueError("k and v must be tensors")
        args = self._rows(k, v, block_table, first, row_start, status)
        st = self.lib.qsa_paged_write(self._ref, *args, _stream(stream))
        if st != QSA_OK:
            raise QsaError(st, "qsa_paged_write failed")

    def read(self, k, v, block_table, first, row_start, status=None, stream=None):
        """qsa_paged_read: rows back as f16 values, into k and v (either may be None)."""
        args = self._rows(k, v, block_table, first, row_start, status)
        st = self.lib.qsa_paged_read(self._ref, *args, _stream(stream))
        if st != QSA_OK:
            raise QsaError(st, "qsa_paged_read failed")

    def workspace_bytes(self, n_q_heads, n_queries=1) -> int:
        """Bytes of the workspace of attend() with these heads and queries."""
        n = int(self.lib.qsa_paged_workspace_bytes(self._ref, n_q_heads, n_queries))
        if n == 0:
            raise QsaError(5, "n_q_heads / n_kv_heads must be 1..8 and n_queries 1..4")
        return n

    def attend(self, q, block_table, seq_lens, out, workspace, lse=None, sm_scale=0.0, status=None, stream=None):
        """qsa_paged_attend: q [n_seqs, n_queries, n_q_heads, head_dim] f16 (query rows may lie
        apart evenly), out the same f32, lse [n_seqs, n_queries, n_q_heads] f32, status one i32."""
        shape = q.shape
        n_seqs, n_queries, n_q_heads, dim = shape
        dev = self._device()
        if dim != self.head_dim:
            _bad("q", q, _Types.f16, (n_seqs, n_queries, n_q_heads, self.head_dim))
        stride = _rows_stride("q", q, _Types.f16, shape, dev)
        width = block_table.shape[-1]
        if workspace.get_device() != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous on the current device")
        st = self._attend(
            self._ref, q.data_ptr(), stride, n_queries, n_q_heads,
            _arg("block_table", block_table, _Types.i32, (n_seqs, width), dev), width, n_seqs,
            _arg("seq_lens", seq_lens, _Types.i32, (n_seqs,), dev), sm_scale, _arg("out", out, _Types.f32, shape, dev),
            None if lse is None else _arg("lse", lse, _Types.f32, shape[:3], dev), workspace.data_ptr(),
            workspace.nbytes, None if status is None else _arg("status", status, _Types.i32, (1,), dev),
            _stream(stream))
        if st != QSA_OK:
            raise QsaError(st, "qsa_paged_attend failed")


def alloc_paged_kv(n_pages, page_size, n_kv_heads, head_dim, page_format=QSA_PAGE_F16, device="cuda") -> PagedKV:
    """Allocates the buffers of a paged cache with torch (`.tensors`: k and v pages, k and v scales)."""
    import torch
    row, kind = {QSA_PAGE_F16: (head_dim, torch.float16), QSA_PAGE_FP8: (head_dim, torch.uint8),
                 QSA_PAGE_INT4: (head_dim // 2, torch.uint8)}[page_format]
    pages = [torch.zeros(n_pages, n_kv_heads, page_size, row, dtype=kind, device=device) for _ in range(2)]
    scales = [None, None]
    if page_format == QSA_PAGE_FP8:
        scales = [torch.ones(n_pages, n_kv_heads, page_size, device=device) for _ in range(2)]
    elif page_format == QSA_PAGE_INT4:
        scales = [torch.zeros(n_pages, n_kv_heads, page_size, head_dim // 32, dtype=torch.float16, device=device)
                  for _ in range(2)]
    return PagedKV(*pages, page_format, *scales)


def verify_drafts(target_probs, draft_probs, draft_tokens, uniforms, n_accepted, next_token, n_drafts=None, status=None,
                  stream=None):
    """qsa_verify_drafts: target_probs [n_seqs, max_drafts + 1, vocab] f32, draft_probs [n_seqs,
    max_drafts, vocab] f32 or None (rows of both may lie apart evenly), draft_tokens [n_seqs,
    max_drafts] i32, uniforms [n_seqs, max_drafts + 1] f32 -> n_accepted, next_token [n_seqs] i32."""
    if _Types.f32 is None:
        _Types.load()
    dev, shape = _Types.device(), target_probs.shape
    n_seqs, rows, vocab = shape
    k = rows - 1
    t_stride = _rows_stride("target_probs", target_probs, _Types.f32, shape, dev)
    d_ptr, d_stride = None, 0
    if draft_probs is not None and k > 0:
        d_stride = _rows_stride("draft_probs", draft_probs, _Types.f32, (n_seqs, k, vocab), dev)
        d_ptr = draft_probs.data_ptr()
    st = load_library().qsa_verify_drafts(
        target_probs.data_ptr(), t_stride, d_ptr, d_stride,
        _arg("draft_tokens", draft_tokens, _Types.i32, (n_seqs, k), dev),
        None if n_drafts is None else _arg("n_drafts", n_drafts, _Types.i32, (n_seqs,), dev),
        _arg("uniforms", uniforms, _Types.f32, (n_seqs, rows), dev), n_seqs, k, vocab,
        _arg("n_accepted", n_accepted, _Types.i32, (n_seqs,), dev),
        _arg("next_token", next_token, _Types.i32, (n_seqs,), dev),
        None if status is None else _arg("status", status, _Types.i32, (1,), dev), _stream(stream))
    if st != QSA_OK:
        raise QsaError(st, "qsa_verify_drafts failed")


def alloc_layer(cfg: QsaConfig, device="cuda"):
    """Allocate one layer's buffers with torch (the caller owns them). With QSA_KV_FP8 the
    K/V caches are uint8 e4m3 codes and `kv_scales` holds the per-row K and V scales."""
    import torch
    fp8 = cfg.kv_format == QSA_KV_FP8
    kv_dtype = torch.uint8 if fp8 else torch.float16
    shape = (cfg.max_ctx, cfg.n_kv_heads, cfg.head_dim)
    bufs = {
        "k_cache": torch.zeros(shape, dtype=kv_dtype, device=device),
        "v_cache": torch.zeros(shape, dtype=kv_dtype, device=device),
        "idx_cache": torch.zeros(cfg.max_ctx, cfg.d_idx, dtype=torch.float16, device=device),
        "pooled_cache": torch.zeros(cfg.max_ctx // 4, cfg.d_idx, device=device,
                                    dtype=torch.uint8 if cfg.pooled_format == QSA_POOLED_FP8 else torch.float16),
        "workspace": torch.zeros(buffer_bytes(cfg, QSA_BUF_WORKSPACE), dtype=torch.uint8, device=device),
    }
    assert bufs["k_cache"].numel() * bufs["k_cache"].element_size() == buffer_bytes(cfg, QSA_BUF_KV)
    if fp8:
        bufs["kv_scales"] = torch.zeros(cfg.max_ctx, cfg.n_kv_heads, 2, dtype=torch.float32, device=device)
    if cfg.pooled_format == QSA_POOLED_FP8:
        bufs["pooled_scales"] = torch.zeros(cfg.max_ctx // 4, dtype=torch.float32, device=device)
    assert bufs["pooled_cache"].numel() * bufs["pooled_cache"].element_size() == buffer_bytes(cfg, QSA_BUF_POOLED)
    return bufs


def alloc_multi_outputs(cfg: QsaConfig, n_queries: int, device="cuda"):
    """Outputs of a multi-query step: per-query selections, counts, scores and attention."""
    import torch
    k_blocks = cfg.top_k_tokens // 4
    return {
        "sel": torch.zeros(n_queries, k_blocks, dtype=torch.int32, device=device),
        "n_sel": torch.zeros(n_queries, dtype=torch.int32, device=device),
        "scores": torch.zeros(n_queries, buffer_bytes(cfg, QSA_BUF_SCORE_STRIDE), dtype=torch.float32,
                              device=device),
        "out": torch.zeros(n_queries, cfg.n_q_heads, cfg.head_dim, dtype=torch.float32, device=device),
    }


def alloc_step_outputs(cfg: QsaConfig, device="cuda"):
    """Per-step output buffers: selected blocks, cells, counts and the attention output."""
    import torch
    k_blocks = cfg.top_k_tokens // 4
    return {
        "sel": torch.zeros(k_blocks, dtype=torch.int32, device=device),
        "n_sel": torch.zeros(4, dtype=torch.int32, device=device),
        "cells": torch.zeros(4 * k_blocks + 3, dtype=torch.int32, device=device),
        "n_cells": torch.zeros(4, dtype=torch.int32, device=device),
        "out": torch.zeros(cfg.n_q_heads, cfg.head_dim, dtype=torch.float32, device=device),
    }
