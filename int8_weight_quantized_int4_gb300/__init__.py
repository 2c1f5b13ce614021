"""Python binding of libqgemm (include/qgemm.h): the GB300 weight-quantized
linear layer.  Argument marshalling only -- every computing step runs in the
library's CUDA kernels; there is no CPU or PyTorch fallback.  PyTorch supplies
device memory and the current CUDA stream.

Entry points (same names as the C ABI):
    qpack_w4(codes, scales) -> packed        qpack_w8(codes, scales) -> packed
    quant_act_int8(x) -> (xq, xs)
    qgemm_w4a16(x, packed, N, K) -> y        qgemm_w4a8(xq, xs, packed, N, K) -> y
    qgemm_w4a8_fused(x, packed, N, K) -> y
    qgemm_w8a16(x, packed, N, K) -> y
    embed_gather_w8(ids, packed, V, D) -> out        topk_logits(logits, k) -> (vals, idx)
    kv_append(k, v, k_pages, v_pages, page_table, seq_lens, cu_tokens)
    attn_paged(q, k_pages, v_pages, page_table, seq_lens, cu_tokens) -> out
    kv_copy_pages(pairs, *pools)                     KvPool: pages of sequences, on the host
    token_logprobs(logits, tokens, k) -> TokenLogprobs
    attn_tree(q, k_pages, v_pages, page_table, seq_lens, cu_tokens, parents) -> out
    sample_tokens(logits, u, temperature, top_k, top_p, min_p) -> SampledTokens
    tree_accept(tokens, drawn, parents, cu_tokens, max_path) -> TreePath
    kv_keep_path(path, count, page_table, seq_lens, cu_tokens, *pools) -> new lengths
"""
from __future__ import annotations

import ctypes
import math
import os
import struct
import threading
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqgemm.so")

QW_OK = 0
QW_ERR_INVALID_ARG = -1
QW_ERR_UNSUPPORTED_SHAPE = -2
QW_ERR_ALIGNMENT = -3
QW_ERR_WORKSPACE = -4
QW_ERR_ARCH = -5
QW_ERR_CUDA = -6
QW_ERR_TIMEOUT = -7
QW_ERR_BAD_CODES = -8
QW_ERR_BAD_INDEX = -9
QW_ERR_NO_PAGES = -10
QW_ERR_HOST_MEMORY = -11
QW_KV_F16, QW_KV_BF16, QW_KV_INT8 = 0, 1, 2
QW_F16, QW_BF16, QW_F32 = 0, 1, 2
MODE_W4A16, MODE_W4A8, MODE_W8A16, MODE_W4A8_FUSED = 0, 1, 2, 3

# every function the header declares: name -> (restype, argtypes)
_p, _i, _sz, _ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_longlong


class Plan(ctypes.Structure):
    _fields_ = [("bn", _i), ("token_tiles", _i), ("row_tiles", _i), ("groups", _i),
                ("tiles", _ll), ("chunks", _ll), ("grid", _i), ("stream_k", _i), ("stages", _i),
                ("smem_bytes", _i), ("ws_bytes", _sz), ("ws_zero_bytes", _sz),
                ("act_stages", _i), ("act_block", _i), ("fused", _i), ("decode_teams", _i),
                ("decode_row_blocks", _i)]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [("k", _p), ("v", _p), ("k_scale", _p), ("v_scale", _p), ("dtype", _i), ("num_pages", _i),
                ("page", _i), ("Hkv", _i), ("d", _i), ("page_stride", _ll), ("head_stride", _ll),
                ("token_stride", _ll)]


class KvBatchDesc(ctypes.Structure):
    _fields_ = [("page_table", _p), ("seq_lens", _p), ("cu_tokens", _p), ("B", _i), ("max_pages", _i)]


class PagePoolDesc(ctypes.Structure):
    _fields_ = [("base", _p), ("layers", _i), ("num_pages", _i), ("layer_stride", _ll), ("page_stride", _ll),
                ("page_bytes", _ll)]


class RowPoolDesc(ctypes.Structure):
    _fields_ = [("base", _p), ("layers", _i), ("num_pages", _i), ("heads", _i), ("row_bytes", _i),
                ("layer_stride", _ll), ("page_stride", _ll), ("head_stride", _ll), ("token_stride", _ll)]


class SamplingDesc(ctypes.Structure):
    _fields_ = [("temperature", ctypes.c_float), ("top_p", ctypes.c_float), ("min_p", ctypes.c_float), ("top_k", _i),
                ("temperatures", _p), ("top_ps", _p), ("min_ps", _p), ("top_ks", _p)]


_ip = ctypes.POINTER(ctypes.c_int)

SIGNATURES = {
    "qpack_w4_bytes": (_sz, [_i, _i]),
    "qpack_w8_bytes": (_sz, [_i, _i]),
    "qpack_w4": (_i, [_p, _p, _i, _i, _p, _p]),
    "qpack_w8": (_i, [_p, _p, _i, _i, _p, _p]),
    "quant_act_int8": (_i, [_p, _i, _i, _p, _p, _p]),
    "qgemm_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "qgemm_workspace_zero_bytes": (_sz, [_i, _i, _i, _i]),
    "qgemm_w4a16": (_i, [_p, _p, _i, _i, _i, _p, _p, _sz, _p]),
    "qgemm_w4a8": (_i, [_p, _p, _p, _i, _i, _i, _p, _p, _sz, _p]),
    "qgemm_w4a8_fused": (_i, [_p, _p, _i, _i, _i, _p, _p, _sz, _p]),
    "embed_gather_w8": (_i, [_p, _i, _p, _i, _i, _p, _p]),
    "topk_workspace_bytes": (_sz, [_i, _i, _i]),
    "topk_workspace_zero_bytes": (_sz, [_i, _i, _i]),
    "topk_logits": (_i, [_p, _i, _i, _i, _p, _p, _p, _sz, _p]),
    "qgemm_w8a16": (_i, [_p, _p, _i, _i, _i, _p, _p, _sz, _p]),
    "qgemm_w4a16_noalloc": (_i, [_p, _p, _i, _i, _i, _p, _p]),
    "qgemm_lm_head_topk_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "qgemm_lm_head_topk_workspace_zero_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "qgemm_lm_head_topk": (_i, [_i, _p, _p, _i, _i, _i, _i, _p, _p, _p, _p, _sz, _p]),
    "attn_int8qk_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "attn_int8qk_workspace_layout": (_i, [_i, _i, _i, _i, _i, ctypes.POINTER(ctypes.c_size_t)]),
    "attn_int8qk_prefill": (_i, [_p, _p, _p, _i, _i, _i, _i, _i, _p, _p, _sz, _p]),
    "kv_append": (_i, [ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), _p, _p, _i, _ll, _ll, _ll, _ll, _p]),
    "kv_copy_pages": (_i, [ctypes.POINTER(PagePoolDesc), _i, _p, _i, _p]),
    "attn_paged_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "attn_paged_workspace_zero_bytes": (_sz, [_i, _i, _i, _i]),
    "attn_paged": (_i, [ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), _p, _i, _i, _ll, _ll, _i, _i, _i,
                        ctypes.c_float, _p, _p, _p, _sz, _p]),
    "kv_pool_create": (_i, [_i, _i, ctypes.POINTER(_p)]),
    "kv_pool_destroy": (None, [_p]),
    "kv_pool_add": (_i, [_p, _ip]),
    "kv_pool_extend": (_i, [_p, _i, _i, _p, _ip]),
    "kv_pool_truncate": (_i, [_p, _i, _i]),
    "kv_pool_fork": (_i, [_p, _i, _ip]),
    "kv_pool_free": (_i, [_p, _i]),
    "kv_pool_compact": (_i, [_p, _p, _i, _ip]),
    "kv_pool_table": (_i, [_p, _p, _i, _i, _p, _p]),
    "kv_pool_pages": (_i, [_p, _i, _ip, _ip]),
    "kv_pool_free_pages": (_i, [_p]),
    "token_logprobs_workspace_bytes": (_sz, [_i, _i, _i, _i]),
    "token_logprobs_workspace_zero_bytes": (_sz, [_i, _i, _i, _i]),
    "token_logprobs": (_i, [_p, _i, _i, _i, _ll, _p, _i, _i, _i, _p, _p, _p, _p, _p, _p, _sz, _p]),
    "attn_tree_workspace_bytes": (_sz, [_i, _i, _i]),
    "attn_tree": (_i, [ctypes.POINTER(KvCacheDesc), ctypes.POINTER(KvBatchDesc), _p, _p, _i, _i, _ll, _ll, _i, _i, _i,
                       ctypes.c_float, _p, _p, _p, _sz, _p]),
    "sample_tokens": (_i, [_p, _i, _i, _i, _ll, _p, ctypes.POINTER(SamplingDesc), _p, _p, _p]),
    "tree_accept": (_i, [_p, _p, _p, _p, _i, _i, _i, _p, _p, _p, _p]),
    "kv_keep_path": (_i, [ctypes.POINTER(RowPoolDesc), _i, ctypes.POINTER(KvBatchDesc), _i, _i, _p, _p, _i, _p, _p]),
    "qw_last_error_string": (ctypes.c_char_p, []),
    "qw_device_error": (_i, [_p]),
    "qw_num_kernel_launches": (_ll, []),
    "qw_stream_capture_id": (ctypes.c_ulonglong, [_p]),
    "qw_set_option": (_i, [_i, _i]),
    "qw_get_option": (_i, [_i]),
    "qw_diag_mma_peak": (_i, [_i, _i, _i, _i, _p, ctypes.POINTER(ctypes.c_double), _p]),
    "qw_diag_tc_probe": (_i, [_i, _i, _i, _i, _i, _i, _p, _i, _p]),
    "qw_diag_f8f6f4_gemm": (_i, [_p, _p, _i, _i, _p, _p]),
    "qw_plan": (_i, [_i, _i, _i, _i, _i, ctypes.POINTER(Plan)]),
    "qw_plan_segments": (_i, [ctypes.POINTER(Plan), _i, _i, _p, _p, _p, _p]),
    "qw_plan_row_blocks": (_i, [ctypes.POINTER(Plan), _i, _p, _p]),
}

_lib = None
_lock = threading.Lock()


class QgemmError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"qgemm error {code}: {msg}")
        self.code = code


def lib():
    """Load libqgemm.so (built by build.py / __graft_entry__.build()); raise if absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise ImportError(f"{LIB_PATH} is missing: build it with "
                                  "`python -c 'import __graft_entry__ as g; g.build()'`")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in SIGNATURES.items():
                f = getattr(L, name)
                f.restype = res
                f.argtypes = args
            _lib = L
    return _lib


def _check(rc: int):
    if rc != QW_OK:
        raise QgemmError(rc, lib().qw_last_error_string().decode())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _need(t, dtype, name, ndim=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions")


def _need_shape(t, shape, name):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _need_packed(packed, nbytes, like, name="packed"):
    """A packed weight buffer: a contiguous uint8 CUDA tensor on `like`'s device holding at
    least the nbytes the layout needs for the given shape (the kernels read all of them)."""
    _need(packed, torch.uint8, name)
    if packed.device != like.device:
        raise ValueError(f"{name} is on {packed.device}, the activations on {like.device}")
    if nbytes <= 0:
        return                          # an unsupported shape: the library rejects it
    if packed.numel() < nbytes:
        raise ValueError(f"{name} holds {packed.numel()} bytes, the layout needs {nbytes}")


# ------------------------------------------------------------------ packing --
def qpack_w4_bytes(N: int, K: int) -> int:
    return int(lib().qpack_w4_bytes(N, K))


def qpack_w8_bytes(N: int, K: int) -> int:
    return int(lib().qpack_w8_bytes(N, K))


def _pack(bits, codes, scales, out=None):
    _need(codes, torch.int8, "codes", 2)
    _need(scales, torch.float16, "scales", 2)
    N, K = codes.shape
    nbytes = (qpack_w4_bytes if bits == 4 else qpack_w8_bytes)(N, K)
    _need_shape(scales, (N, K // 128), "scales")
    if out is None:
        out = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=codes.device)
    elif nbytes > 0:
        _need_packed(out, nbytes, codes, "out")
    fn = lib().qpack_w4 if bits == 4 else lib().qpack_w8
    with torch.cuda.device(codes.device):
        _check(fn(_ptr(codes), _ptr(scales), N, K, _ptr(out), _stream(codes)))
    return out


def qpack_w4(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None):
    """int4 codes int8 [N,K] in [-8,7] + signed fp16 scales [N,K/128] -> packed uint8 buffer."""
    return _pack(4, codes, scales, out)


def qpack_w8(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor | None = None):
    """int8 codes [N,K] + signed fp16 scales [N,K/128] -> packed uint8 buffer."""
    return _pack(8, codes, scales, out)


# ------------------------------------------------------- activation quant --
def quant_act_int8(x: torch.Tensor, xq: torch.Tensor | None = None, xs: torch.Tensor | None = None):
    """fp16 [M,K] -> (int8 codes [M,K], binary32 per-token scales [M])."""
    _need(x, torch.float16, "x", 2)
    M, K = x.shape
    if xq is None:
        xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    _need(xq, torch.int8, "xq", 2)
    _need_shape(xq, (M, K), "xq")
    if xs is None:
        xs = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(xs, torch.float32, "xs", 1)
    _need_shape(xs, (M,), "xs")
    with torch.cuda.device(x.device):
        _check(lib().quant_act_int8(_ptr(x), M, K, _ptr(xq), _ptr(xs), _stream(x)))
    return xq, xs


# -------------------------------------------------------------- workspace --
def workspace_bytes(mode: int, M: int, N: int, K: int) -> int:
    return int(lib().qgemm_workspace_bytes(mode, M, N, K))


def _raw_stream(index):
    return torch.cuda.current_stream(index).cuda_stream


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _raw_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


_is_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", torch.cuda.is_current_stream_capturing)


def _capture_id(index):
    """A number of the graph being captured on device `index`'s current stream, 0 without one."""
    if index == _current_device() and not _is_capturing():
        return 0
    return int(lib().qw_stream_capture_id(_raw_stream(index)))


class Workspace:
    """A zero-initialised device workspace that grows on demand (one per stream).  Each kind of
    call has a buffer of its own in it, whose layout the others do not know.

    A buffer that a graph was captured with stays allocated as long as the Workspace lives,
    whatever later calls need; the Workspace has to outlive the graph.  A capture that finds no
    large enough buffer gets one of its own from the graph's memory, zero-filled at every
    replay (a call of the same sizes before the capture saves that)."""

    def __init__(self, device=None):
        self.device = torch.device(device or "cuda")
        self.buf = None                     # the buffer of the latest call
        self._bufs = {}                     # by kind of call: [buffer, its leading zero bytes], held by no graph
        self._index = self.device.index if self.device.type == "cuda" else -1    # -1: host memory
        self._held = []                     # buffers that graphs were captured with,
        self._fixed = {}                    # the newest of them by (kind, zero bytes)
        self._own = (0, {})                 # the latest capture and the buffers of its own, likewise

    def get(self, mode: int, M: int, N: int, K: int):
        with torch.cuda.device(self.device):
            need = workspace_bytes(mode, M, N, K)
        return self.get_bytes(need)

    def get_bytes(self, need: int, kind: str = "gemm", zero: int = 0):
        """A buffer of at least `need` bytes for calls of a kind (zero-filled when it is made).
        zero: the leading bytes that the call finds and leaves zero, for kinds where they depend
        on its sizes; what a smaller call has written there is zero-filled again."""
        if need == 0:
            return None, 0
        index = self._index
        capture = _capture_id(_current_device() if index is None else index) if index != -1 else 0
        entry = self._bufs.get(kind)
        if entry is not None and entry[0].numel() < need:
            entry = None
        if capture and entry is not None and entry[1] == zero:
            buf = self._fixed[kind, zero] = self._bufs.pop(kind)[0]
            self._held.append(buf)
        elif entry is None or capture or entry[1] < zero:
            buf = self._fixed.get((kind, zero))
            if buf is None or buf.numel() < need:
                if capture:
                    if self._own[0] != capture:
                        self._own = (capture, {})
                    buf = self._own[1].get((kind, zero))
                    if buf is None or buf.numel() < need:
                        buf = self._own[1][kind, zero] = self._zeros(need)
                    return buf, buf.numel()
                if entry is None:
                    entry = self._bufs[kind] = [self._zeros(need), zero]
                buf = entry[0]
                buf[entry[1]:zero].zero_()
                entry[1] = zero
        else:
            buf, entry[1] = entry[0], zero
        self.buf = buf
        return buf, buf.numel()

    def _zeros(self, n):
        return torch.zeros(n, dtype=torch.uint8, device=self.device)

    def zero(self):
        """Zero-fill the buffers again (needed after a call that ended in QW_ERR_TIMEOUT)."""
        for x in [x for x, _ in self._bufs.values()] + self._held:
            x.zero_()


_default_ws = {}


def _ws_for(t, mode, M, N, K, ws):
    if ws is None:
        key = (t.device, torch.cuda.current_stream(t.device).cuda_stream)
        ws = _default_ws.setdefault(key, Workspace(t.device))
    return ws.get(mode, M, N, K)


# ------------------------------------------------------------------ GEMMs --
def _out(y, M, N, dev):
    if y is None:
        return torch.empty((M, N), dtype=torch.float16, device=dev)
    _need(y, torch.float16, "y", 2)
    if tuple(y.shape) != (M, N):
        raise ValueError("y has the wrong shape")
    return y


def qgemm_w4a16(x, packed, N: int, K: int, y=None, ws: Workspace | None = None):
    """y[M,N] = x[M,K] . W^T with W int4 group-128 (packed by qpack_w4), fp16 out."""
    _need(x, torch.float16, "x", 2)
    M = x.shape[0]
    if x.shape[1] != K:
        raise ValueError("x.shape[1] != K")
    y = _out(y, M, N, x.device)
    if M and N:
        _need_packed(packed, qpack_w4_bytes(N, K), x)
    wbuf, wbytes = _ws_for(x, MODE_W4A16, M, N, K, ws)
    with torch.cuda.device(x.device):
        _check(lib().qgemm_w4a16(_ptr(x), _ptr(packed), M, N, K, _ptr(y), _ptr(wbuf), wbytes,
                                 _stream(x)))
    return y


def qgemm_w4a8(xq, xs, packed, N: int, K: int, y=None, ws: Workspace | None = None):
    """y[M,N] = xs[m] * (xq[M,K] . W^T) with int8 per-token activations, int4 weights."""
    _need(xq, torch.int8, "xq", 2)
    _need(xs, torch.float32, "xs", 1)
    M = xq.shape[0]
    if xq.shape[1] != K or xs.shape[0] != M:
        raise ValueError("shape mismatch")
    y = _out(y, M, N, xq.device)
    if M and N:
        _need_packed(packed, qpack_w4_bytes(N, K), xq)
    wbuf, wbytes = _ws_for(xq, MODE_W4A8, M, N, K, ws)
    with torch.cuda.device(xq.device):
        _check(lib().qgemm_w4a8(_ptr(xq), _ptr(xs), _ptr(packed), M, N, K, _ptr(y), _ptr(wbuf),
                                wbytes, _stream(xq)))
    return y


def qgemm_w4a8_fused(x, packed, N: int, K: int, y=None, ws: Workspace | None = None):
    """The W4A8 layer from fp16 activations: bit-identical to qgemm_w4a8 applied to
    quant_act_int8(x).  Small decode batches quantize inside the row-block GEMM; otherwise
    the quantizer writes fp16 codes that the GEMM reads as fp16 tiles."""
    _need(x, torch.float16, "x", 2)
    M = x.shape[0]
    if x.shape[1] != K:
        raise ValueError("x.shape[1] != K")
    y = _out(y, M, N, x.device)
    if M and N:
        _need_packed(packed, qpack_w4_bytes(N, K), x)
    wbuf, wbytes = _ws_for(x, MODE_W4A8_FUSED, M, N, K, ws)
    with torch.cuda.device(x.device):
        _check(lib().qgemm_w4a8_fused(_ptr(x), _ptr(packed), M, N, K, _ptr(y), _ptr(wbuf), wbytes,
                                      _stream(x)))
    return y


def qgemm_w8a16(x, packed, N: int, K: int, y=None, ws: Workspace | None = None):
    """y[M,N] = x[M,K] . W^T with W int8 group-128 (packed by qpack_w8), fp16 out."""
    _need(x, torch.float16, "x", 2)
    M = x.shape[0]
    if x.shape[1] != K:
        raise ValueError("x.shape[1] != K")
    y = _out(y, M, N, x.device)
    if M and N:
        _need_packed(packed, qpack_w8_bytes(N, K), x)
    wbuf, wbytes = _ws_for(x, MODE_W8A16, M, N, K, ws)
    with torch.cuda.device(x.device):
        _check(lib().qgemm_w8a16(_ptr(x), _ptr(packed), M, N, K, _ptr(y), _ptr(wbuf), wbytes,
                                 _stream(x)))
    return y


def embed_gather_w8(ids, packed, V: int, D: int, out=None):
    """out[t] = the dequantized row ids[t] of an int8 group-128 table [V, D] packed by
    qpack_w8: fp16(code * scale).  ids int32 [T] on the device."""
    _need(ids, torch.int32, "ids", 1)
    T = ids.shape[0]
    if out is None:
        out = torch.empty((T, D), dtype=torch.float16, device=ids.device)
    _need(out, torch.float16, "out", 2)
    _need_shape(out, (T, D), "out")
    if T:
        _need_packed(packed, qpack_w8_bytes(V, D), ids)
    with torch.cuda.device(ids.device):
        _check(lib().embed_gather_w8(_ptr(ids), T, _ptr(packed), V, D, _ptr(out), _stream(ids)))
    return out


def attn_int8qk_prefill(q, k, v, out=None, ws: Workspace | None = None):
    """int8-QK causal prefill attention: q [T,Hq,d], k and v [S,Hkv,d] fp16 on the device
    (the T queries are the context's last T positions) -> out [T,Hq,d] fp16."""
    _need(q, torch.float16, "q", 3)
    _need(k, torch.float16, "k", 3)
    _need(v, torch.float16, "v", 3)
    T, Hq, d = q.shape
    S, Hkv, dk = k.shape
    if dk != d or tuple(v.shape) != (S, Hkv, d):
        raise ValueError("k and v must be [S, Hkv, d] with q's d")
    if out is None:
        out = torch.empty((T, Hq, d), dtype=torch.float16, device=q.device)
    _need(out, torch.float16, "out", 3)
    _need_shape(out, (T, Hq, d), "out")
    if ws is None:
        key = (q.device, torch.cuda.current_stream(q.device).cuda_stream, "attn")
        ws = _default_ws.setdefault(key, Workspace(q.device))
    with torch.cuda.device(q.device):
        wbuf, wbytes = ws.get_bytes(int(lib().attn_int8qk_workspace_bytes(T, S, Hq, Hkv, d)), "int8qk")
        _check(lib().attn_int8qk_prefill(_ptr(q), _ptr(k), _ptr(v), T, S, Hq, Hkv, d, _ptr(out), _ptr(wbuf),
                                         wbytes, _stream(q)))
    return out


def attn_int8qk_intermediates(ws: Workspace, T: int, S: int, Hq: int, Hkv: int, d: int = 256):
    """Views into the workspace of the last attn_int8qk_prefill call with these sizes:
    (query codes [Hq,T,d], query scales [Hq,T], key codes [Hkv,S,d], key scales [Hkv,S],
    V^T [Hkv,d,S]); codes as fp16 tensors holding the int8 values."""
    off = (ctypes.c_size_t * 6)()
    _check(lib().attn_int8qk_workspace_layout(T, S, Hq, Hkv, d, off))
    b = ws._bufs["int8qk"][0] if "int8qk" in ws._bufs else ws._fixed["int8qk", 0]

    def view(o, n, dt, shape):
        return b[o:o + n * torch.tensor([], dtype=dt).element_size()].view(dt).view(shape)
    return (view(off[0], Hq * T * d, torch.float16, (Hq, T, d)), view(off[1], Hq * T, torch.float32, (Hq, T)),
            view(off[2], Hkv * S * d, torch.float16, (Hkv, S, d)), view(off[3], Hkv * S, torch.float32, (Hkv, S)),
            view(off[4], Hkv * d * S, torch.float16, (Hkv, d, S)))


def qgemm_lm_head_topk(mode: int, x, packed, N: int, K: int, k: int, y=None, vals=None, idx=None,
                       ws: Workspace | None = None):
    """The lm_head (MODE_W4A16 on qpack_w4 bytes or MODE_W8A16 on qpack_w8 bytes) with the
    top-k of each row fused in: returns (y [M,N] fp16 logits, vals [M,k] fp16, idx [M,k] int32),
    y bit-identical to the plain GEMM and (vals, idx) equal to topk_logits(y, k)."""
    _need(x, torch.float16, "x", 2)
    M = x.shape[0]
    if x.shape[1] != K:
        raise ValueError("x.shape[1] != K")
    y = _out(y, M, N, x.device)
    if vals is None:
        vals = torch.empty((M, k), dtype=torch.float16, device=x.device)
    if idx is None:
        idx = torch.empty((M, k), dtype=torch.int32, device=x.device)
    _need(vals, torch.float16, "vals", 2)
    _need(idx, torch.int32, "idx", 2)
    _need_shape(vals, (M, k), "vals")
    _need_shape(idx, (M, k), "idx")
    if M and N:
        _need_packed(packed, (qpack_w8_bytes if mode == MODE_W8A16 else qpack_w4_bytes)(N, K), x)
    if ws is None:
        key = (x.device, torch.cuda.current_stream(x.device).cuda_stream, "lm_head_topk")
        ws = _default_ws.setdefault(key, Workspace(x.device))
    with torch.cuda.device(x.device):
        need = int(lib().qgemm_lm_head_topk_workspace_bytes(mode, M, N, K, k))
        wbuf, wbytes = ws.get_bytes(need, "lm_head_topk",
                                    int(lib().qgemm_lm_head_topk_workspace_zero_bytes(mode, M, N, K, k)))
        _check(lib().qgemm_lm_head_topk(mode, _ptr(x), _ptr(packed), M, N, K, k, _ptr(y), _ptr(vals),
                                        _ptr(idx), _ptr(wbuf), wbytes, _stream(x)))
    return y, vals, idx


def topk_logits(logits, k: int):
    """Per row the k largest logits (largest first, ties to the smaller index):
    returns (values fp16 [M,k], indices int32 [M,k])."""
    _need(logits, torch.float16, "logits", 2)
    M, N = logits.shape
    vals = torch.empty((M, k), dtype=torch.float16, device=logits.device)
    idx = torch.empty((M, k), dtype=torch.int32, device=logits.device)
    key = (logits.device, torch.cuda.current_stream(logits.device).cuda_stream, "topk")
    ws = _default_ws.setdefault(key, Workspace(logits.device))
    with torch.cuda.device(logits.device):
        buf, nbytes = ws.get_bytes(int(lib().topk_workspace_bytes(M, N, k)), "topk",
                                   int(lib().topk_workspace_zero_bytes(M, N, k)))
        _check(lib().topk_logits(_ptr(logits), M, N, k, _ptr(vals), _ptr(idx), _ptr(buf), nbytes,
                                 _stream(logits)))
    return vals, idx


# ------------------------------------------------------------ paged cache --
# These calls run once a layer and token, so their marshalling is kept short: device indices
# instead of device objects, descriptors packed by struct (native layout, as the C structs),
# the raw handle of the current stream.
_KV_TYPES = {torch.float16: QW_KV_F16, torch.bfloat16: QW_KV_BF16, torch.int8: QW_KV_INT8}
_ACT_TYPES = (torch.float16, torch.bfloat16, torch.float16)       # by cache type
_pack_cache = struct.Struct("@PPPPiiiiiqqq").pack
_pack_batch = struct.Struct("@PPPii").pack
_pack_pool = struct.Struct("@Piiqqq").pack
assert struct.calcsize("@PPPPiiiiiqqq") == ctypes.sizeof(KvCacheDesc)
assert struct.calcsize("@PPPii0q") == ctypes.sizeof(KvBatchDesc)
assert struct.calcsize("@Piiqqq") == ctypes.sizeof(PagePoolDesc)
_pack_rows = struct.Struct("@Piiiiqqqq").pack
_pack_sampling = struct.Struct("@fffiPPPP").pack
assert struct.calcsize("@Piiiiqqqq") == ctypes.sizeof(RowPoolDesc)
assert struct.calcsize("@fffiPPPP") == ctypes.sizeof(SamplingDesc)
_i32, _f32 = torch.int32, torch.float32
_INT_MAX = 0x7fffffff


def _int(x):
    """x as a C int; ctypes would take it modulo 2^32."""
    if not -_INT_MAX <= x <= _INT_MAX:
        raise ValueError(f"{x} is outside the 32-bit range")
    return x


_step = {}


def _step_fn(name):
    """The entry point with its descriptors taken as packed bytes."""
    fn = _step.get(name)
    if fn is None:
        lib()
        fn = getattr(ctypes.CDLL(LIB_PATH), name)
        fn.restype, args = SIGNATURES[name]
        fn.argtypes = [ctypes.c_char_p if isinstance(x, type) and issubclass(x, ctypes._Pointer) else x for x in args]
        _step[name] = fn
    return fn


def _run(index, fn, *args):
    """fn(*args) with device `index` current; raises on an error code."""
    if index == _current_device():
        rc = fn(*args)
    else:
        with torch.cuda.device(index):
            rc = fn(*args)
    if rc:
        _check(rc)


def _scratch(ws, index, stream, kind, query, *args):
    """(buffer, pointer, bytes) of `ws`, or of the default workspace of this kind of call and
    stream.  The caller keeps the buffer until its call is enqueued."""
    if ws is None:
        ws = _default_ws.get((index, stream, kind))
        if ws is None:
            ws = _default_ws.setdefault((index, stream, kind), Workspace(torch.device("cuda", index)))
    if index == _current_device():
        need = query(*args)
    else:
        with torch.cuda.device(index):
            need = query(*args)
    buf, nbytes = ws.get_bytes(need, kind)
    return buf, (None if buf is None else buf.data_ptr()), nbytes


def _strides(t):
    """The strides, 0 for dimensions of one element, where they mean nothing."""
    return tuple(0 if n == 1 else st for n, st in zip(t.shape[:-1], t.stride())) + t.stride()[-1:]


def _kv_cache(k_pages, v_pages, k_scale, v_scale, index):
    """(packed descriptor, cache type, Hkv, d) of one layer's cache, [pages, Hkv, page, d]."""
    dtype = _KV_TYPES.get(k_pages.dtype)
    if dtype is None or v_pages.dtype is not k_pages.dtype:
        raise TypeError("k_pages and v_pages must both be float16, bfloat16 or int8")
    if index < 0 or v_pages.get_device() != index:
        raise TypeError("k_pages and v_pages must be CUDA tensors on one device")
    shape, stride = k_pages.shape, k_pages.stride()
    if len(shape) != 4 or v_pages.shape != shape:
        raise ValueError("k_pages and v_pages must have one shape [pages, Hkv, page, d]")
    if 1 in shape:
        stride = _strides(k_pages)
    if (_strides(v_pages) if 1 in shape else v_pages.stride()) != stride or stride[3] != 1:
        raise ValueError("k_pages and v_pages must have the same strides, the last dimension contiguous")
    ks = vs = 0
    pages, heads, page, d = shape
    if dtype == QW_KV_INT8:
        for s, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            _need(s, torch.float32, name, 3)
            if s.shape != shape[:3] or s.get_device() != index:
                raise ValueError(f"{name} must be {tuple(shape[:3])} on the cache's device")
        ks, vs = k_scale.data_ptr(), v_scale.data_ptr()
    elif k_scale is not None or v_scale is not None:
        raise ValueError("only an int8 cache has scales")
    return (_pack_cache(k_pages.data_ptr(), v_pages.data_ptr(), ks, vs, dtype, pages, page, heads, d, stride[0],
                        stride[1], stride[2]), dtype, heads, d)


def _kv_batch(table, lens, cu, index):
    """The packed descriptor of a batch."""
    if not (table.dtype is lens.dtype is cu.dtype is _i32):
        raise ValueError("page_table, seq_lens and cu_tokens must be int32")
    if not (table.get_device() == lens.get_device() == cu.get_device() == index):
        raise ValueError("page_table, seq_lens and cu_tokens must be on the cache's device")
    if table.dim() != 2 or not (table.is_contiguous() and lens.is_contiguous() and cu.is_contiguous()):
        raise ValueError("page_table [B, max_pages], seq_lens [B] and cu_tokens [B + 1] must be contiguous")
    B, width = table.shape
    if lens.dim() != 1 or cu.dim() != 1 or lens.shape[0] != B or cu.shape[0] != B + 1:
        raise ValueError("page_table [B, max_pages], seq_lens [B] and cu_tokens [B + 1] disagree")
    return _pack_batch(table.data_ptr(), lens.data_ptr(), cu.data_ptr(), B, width)


def _rows(t, name, dtype, d, index, heads):
    """Checks new tokens' rows [T, heads, d] (strided, d contiguous); returns (T, heads, strides)."""
    want = _ACT_TYPES[dtype]
    if t.dtype is not want or t.get_device() != index:
        raise TypeError(f"{name} must be {want} on the cache's device, got {t.dtype} on {t.device}")
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, heads, {d}]")
    T, h, dt = t.shape
    st, sh, sd = t.stride() if T > 1 and h > 1 else _strides(t)
    if dt != d or (heads and h != heads) or sd != 1:
        raise ValueError(f"{name} must be [T, {heads or 'Hq'}, {d}] with the last dimension contiguous")
    return T, h, st, sh


def kv_append(k, v, k_pages, v_pages, page_table, seq_lens, cu_tokens, k_scale=None, v_scale=None):
    """Writes the new tokens' k and v [T, Hkv, d] into their pages (k_pages, v_pages
    [pages, Hkv, page, d]; an int8 cache has scales [pages, Hkv, page] float32 and quantizes
    each row).  Sequence b's new tokens are rows cu_tokens[b] .. cu_tokens[b + 1] - 1 and its
    last positions; seq_lens counts them already."""
    index = k_pages.get_device()
    cache, dtype, heads, d = _kv_cache(k_pages, v_pages, k_scale, v_scale, index)
    batch = _kv_batch(page_table, seq_lens, cu_tokens, index)
    T, _, kt, kh = _rows(k, "k", dtype, d, index, heads)
    Tv, _, vt, vh = _rows(v, "v", dtype, d, index, heads)
    if Tv != T:
        raise ValueError("k and v must have the same number of tokens")
    _run(index, _step_fn("kv_append"), cache, batch, k.data_ptr(), v.data_ptr(), T, kt, kh, vt, vh, _raw_stream(index))


def kv_copy_pages(pairs, *pools):
    """For every (source, destination) of pairs (int32 [n, 2], device): copies the page in
    each pool and layer.  A pool is a tensor whose leading dimensions are [pages] or
    [layers, pages] -- 4 or 5 dimensions for K and V, 3 or 4 (float32) for the scales of an
    int8 cache -- and whose pages are dense.  No page may be a destination twice, nor both a
    source and a destination."""
    index = pairs.get_device()
    if pairs.dtype is not _i32 or index < 0:
        raise TypeError("pairs must be an int32 CUDA tensor")
    if pairs.dim() != 2 or pairs.shape[1] != 2 or not pairs.is_contiguous():
        raise ValueError("pairs must be a contiguous [n, 2]")
    if not 1 <= len(pools) <= 4:
        raise ValueError("one to four pools")
    desc = b""
    for i, x in enumerate(pools):
        if x.get_device() != index:
            raise ValueError(f"pool {i} is on {x.device}, the pairs on {pairs.device}")
        shape, stride, es = x.shape, x.stride(), x.element_size()
        lead = len(shape) - (2 if x.dtype is _f32 else 3)
        if lead != 1 and lead != 2:
            raise ValueError(f"pool {i}: [pages, ...] or [layers, pages, ...] before a page's dimensions")
        dense = 1
        for st, n in sorted(zip(stride[lead:], shape[lead:])):
            if n != 1 and st != dense:
                raise ValueError(f"pool {i}: a page must be one dense block")
            dense *= n
        layers, pages = shape[0] if lead == 2 else 1, shape[lead - 1]
        desc += _pack_pool(x.data_ptr(), layers, pages, stride[0] * es if layers > 1 else 0,
                           (stride[lead - 1] if pages > 1 else dense) * es, dense * es)
    _run(index, _step_fn("kv_copy_pages"), desc, len(pools), pairs.data_ptr(), pairs.shape[0], _raw_stream(index))


def attn_paged(q, k_pages, v_pages, page_table, seq_lens, cu_tokens, max_new: int = 1, window: int = 0, sinks: int = 0,
               scale: float | None = None, k_scale=None, v_scale=None, out=None, lse=None,
               ws: Workspace | None = None):
    """Attention of the new tokens q [T, Hq, d] over the paged cache, which holds them
    already: out [T, Hq, d].  The token at position i sees keys j <= i and, with window > 0,
    j > i - window or j < sinks.  max_new: the most new tokens of a sequence (a hint).
    scale: 1 / sqrt(d) unless given.  lse: a float32 [T, Hq] tensor to fill with the log of
    the sum of exponentials; then (out, lse) is returned."""
    index = k_pages.get_device()
    cache, dtype, heads, d = _kv_cache(k_pages, v_pages, k_scale, v_scale, index)
    batch = _kv_batch(page_table, seq_lens, cu_tokens, index)
    T, Hq, qt, qh = _rows(q, "q", dtype, d, index, 0)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device)
    elif out.dtype is not q.dtype or out.shape != q.shape or out.get_device() != index or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {q.dtype} tensor {tuple(q.shape)} on the cache's device")
    if lse is not None and (lse.dtype is not _f32 or lse.shape != (T, Hq) or lse.get_device() != index
                            or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor {(T, Hq)} on the cache's device")
    if max(max_new, window, sinks) > _INT_MAX or min(max_new, window, sinks) < 0:
        max_new, window, sinks = (max(min(x, _INT_MAX), -1) for x in (max_new, window, sinks))   # -1: refused below
    stream = _raw_stream(index)
    buf, pbuf, nbytes = _scratch(ws, index, stream, "paged", _step_fn("attn_paged_workspace_bytes"), d, Hq, heads,
                                 max_new)
    _run(index, _step_fn("attn_paged"), cache, batch, q.data_ptr(), T, Hq, qt, qh, max_new, window, sinks,
         d ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(), pbuf, nbytes,
         stream)
    return out if lse is None else (out, lse)


class KvPool:
    """Which pages hold which sequence (host side, include/qgemm.h kv_pool_*).  Sequences are
    small integers.  Copies come back as [source, destination] lists; enqueue them with
    kv_copy_pages before the step writes its tokens."""

    def __init__(self, num_pages: int, page: int):
        h = ctypes.c_void_p()
        _check(lib().kv_pool_create(_int(num_pages), _int(page), ctypes.byref(h)))
        self._h = h
        self.num_pages, self.page = num_pages, page

    def __del__(self):
        h, self._h = getattr(self, "_h", None), None
        if h:
            lib().kv_pool_destroy(h)

    def add(self) -> int:
        s = ctypes.c_int()
        _check(lib().kv_pool_add(self._h, ctypes.byref(s)))
        return s.value

    def extend(self, seq: int, n_tokens: int) -> list:
        """Lengthens the sequence; returns the pages to copy first: [] or [[src, dst]]."""
        pair, n = (ctypes.c_int32 * 2)(), ctypes.c_int()
        _check(lib().kv_pool_extend(self._h, _int(seq), _int(n_tokens), pair, ctypes.byref(n)))
        return [list(pair)] if n.value else []

    def truncate(self, seq: int, length: int):
        _check(lib().kv_pool_truncate(self._h, _int(seq), _int(length)))

    def fork(self, seq: int) -> int:
        s = ctypes.c_int()
        _check(lib().kv_pool_fork(self._h, _int(seq), ctypes.byref(s)))
        return s.value

    def free(self, seq: int):
        _check(lib().kv_pool_free(self._h, _int(seq)))

    def compact(self, most: int | None = None) -> list:
        """Moves live pages into the lowest free ones; returns the pages to copy."""
        cap = self.num_pages if most is None else min(most, self.num_pages)
        pairs, n = (ctypes.c_int32 * (2 * max(cap, 1)))(), ctypes.c_int()
        _check(lib().kv_pool_compact(self._h, pairs, _int(cap), ctypes.byref(n)))
        return [[pairs[2 * i], pairs[2 * i + 1]] for i in range(n.value)]

    def length(self, seq: int) -> int:
        n = ctypes.c_int()
        _check(lib().kv_pool_pages(self._h, _int(seq), ctypes.byref(n), None))
        return n.value

    def pages(self, seq: int) -> int:
        n = ctypes.c_int()
        _check(lib().kv_pool_pages(self._h, _int(seq), None, ctypes.byref(n)))
        return n.value

    def free_pages(self) -> int:
        n = int(lib().kv_pool_free_pages(self._h))
        if n < 0:
            _check(n)
        return n

    def table(self, seqs, max_pages: int | None = None, pin: bool = False):
        """CPU int32 tensors (page_table [B, max_pages], seq_lens [B]) of the sequences."""
        seqs = [_int(int(s)) for s in seqs]
        width = max([self.pages(s) for s in seqs], default=0) if max_pages is None else max_pages
        table = torch.empty((len(seqs), width), dtype=torch.int32, pin_memory=pin)
        lens = torch.empty((len(seqs),), dtype=torch.int32, pin_memory=pin)
        ids = (ctypes.c_int32 * max(len(seqs), 1))(*seqs)
        _check(lib().kv_pool_table(self._h, ids, len(seqs), width, table.data_ptr(), lens.data_ptr()))
        return table, lens


# ------------------------------------------------------- token probabilities --
class TokenLogprobs(NamedTuple):
    logprob: torch.Tensor               # [M, C] (or [M]) of the given tokens
    entropy: torch.Tensor               # [M]
    lse: torch.Tensor                   # [M] logsumexp
    top_logprob: torch.Tensor | None    # [M, k], most likely first
    top_idx: torch.Tensor | None        # [M, k] int32


_LOGIT_TYPES = {torch.float16: QW_F16, torch.bfloat16: QW_BF16, torch.float32: QW_F32}


def token_logprobs(logits, tokens, k: int = 0, ws: Workspace | None = None) -> TokenLogprobs:
    """Log probabilities of given tokens (int32 or int64 [M] or [M, C]), entropy, logsumexp
    and the k (<= 64) most likely tokens of each row of logits [M, N] (fp16, bf16 or float32;
    rows may be strided), in one pass over the logits."""
    dtype = _LOGIT_TYPES.get(logits.dtype)
    index = logits.get_device()
    if dtype is None or index < 0:
        raise TypeError("logits must be a float16, bfloat16 or float32 CUDA tensor")
    if logits.dim() != 2:
        raise ValueError("logits must be [M, N] with contiguous rows")
    M, N = logits.shape
    row, col = logits.stride()
    if col != 1 and N > 1:
        raise ValueError("logits must be [M, N] with contiguous rows")
    tt = tokens.dtype
    if tt is not torch.int64 and tt is not _i32 or tokens.get_device() != index:
        raise TypeError("tokens must be int32 or int64 on the logits' device")
    shape = tokens.shape
    if len(shape) not in (1, 2) or shape[0] != M or not tokens.is_contiguous():
        raise ValueError("tokens must be a contiguous [M] or [M, C]")
    C = 1 if len(shape) == 1 else shape[1]
    if k < 0:
        raise ValueError("k must not be negative")
    dev, empty = logits.device, torch.empty
    entropy, lse = empty(M, dtype=_f32, device=dev), empty(M, dtype=_f32, device=dev)
    logprob = empty(shape, dtype=_f32, device=dev)
    top = idx = ptop = pidx = None
    if k:
        top, idx = empty((M, k), dtype=_f32, device=dev), empty((M, k), dtype=_i32, device=dev)
        ptop, pidx = top.data_ptr(), idx.data_ptr()
    stream = _raw_stream(index)
    buf, pbuf, nbytes = _scratch(ws, index, stream, "logprobs", _step_fn("token_logprobs_workspace_bytes"), M, N, k,
                                 dtype)
    _run(index, _step_fn("token_logprobs"), logits.data_ptr(), dtype, M, N, row, tokens.data_ptr(),
         4 if tt is _i32 else 8, C, k, logprob.data_ptr(), entropy.data_ptr(), lse.data_ptr(), ptop, pidx, pbuf, nbytes,
         stream)
    return TokenLogprobs(logprob, entropy, lse, top, idx)


# ------------------------------------------------- trees of drafted tokens --
def _need_ints(index, *named):
    """Raises for what is no contiguous int32 vector of the given length on device `index`; named: (tensor, name, length)."""
    for t, name, n in named:
        if t.dtype is not _i32 or t.get_device() != index or index < 0:
            raise TypeError(f"{name} must be int32 on one CUDA device with the others, got {t.dtype} on {t.device}")
        if t.shape != (n,) or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous [{n}], got {tuple(t.shape)}")


def attn_tree(q, k_pages, v_pages, page_table, seq_lens, cu_tokens, parents, max_nodes: int = 64, window: int = 0,
              sinks: int = 0, scale: float | None = None, k_scale=None, v_scale=None, out=None, lse=None,
              ws: Workspace | None = None):
    """attn_paged for new tokens that are the nodes of a tree: parents (int32 [T]) gives each
    node's parent as its place among the sequence's new tokens, an earlier one, or -1.  A node sees
    the keys before the tree, its ancestors and itself; window counts positions, a node's being
    the first node's slot plus its depth.  max_nodes (<= 256): at least the nodes of any sequence."""
    index = k_pages.get_device()
    cache, dtype, heads, d = _kv_cache(k_pages, v_pages, k_scale, v_scale, index)
    batch = _kv_batch(page_table, seq_lens, cu_tokens, index)
    T, Hq, qt, qh = _rows(q, "q", dtype, d, index, 0)
    if parents.dtype is not _i32 or parents.get_device() != index or parents.shape != (T,) or not parents.is_contiguous():
        _need_ints(index, (parents, "parents", T))
    if out is None:
        out = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device)
    elif out.dtype is not q.dtype or out.shape != q.shape or out.get_device() != index or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {q.dtype} tensor {tuple(q.shape)} on the cache's device")
    if lse is not None and (lse.dtype is not _f32 or lse.shape != (T, Hq) or lse.get_device() != index
                            or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor {(T, Hq)} on the cache's device")
    if max(max_nodes, window, sinks) > _INT_MAX or min(max_nodes, window, sinks) < 0:
        max_nodes, window, sinks = (max(min(x, _INT_MAX), -1) for x in (max_nodes, window, sinks))   # -1: refused below
    stream = _raw_stream(index)
    buf, pbuf, nbytes = _scratch(ws, index, stream, "tree", _step_fn("attn_tree_workspace_bytes"), d, Hq, heads)
    _run(index, _step_fn("attn_tree"), cache, batch, parents.data_ptr(), q.data_ptr(), T, Hq, qt, qh, max_nodes, window,
         sinks, d ** -0.5 if scale is None else scale, out.data_ptr(), None if lse is None else lse.data_ptr(), pbuf,
         nbytes, stream)
    return out if lse is None else (out, lse)


class SampledTokens(NamedTuple):
    token: torch.Tensor                 # [M] int32
    logprob: torch.Tensor               # [M] of its share of what the filters leave


def _setting(x, name, dtype, M, index):
    """(number, pointer) of a sampler's setting: a number, or a tensor of one a row."""
    if not isinstance(x, torch.Tensor):
        return (_int(int(x)) if dtype is _i32 else x), 0
    if x.dtype is not dtype or x.get_device() != index:
        raise TypeError(f"{name} must be a number, or {dtype} on the logits' device")
    if x.shape != (M,) or not x.is_contiguous():
        raise ValueError(f"{name} must be a number or a contiguous [{M}]")
    return 0, x.data_ptr()


def sample_tokens(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0) -> SampledTokens:
    """Draws a token from each row of logits [M, N] (fp16, bf16 or float32; rows may be strided)
    with the uniform numbers u (float32 [M], in [0, 1)).  temperature (0: the most likely), top_k
    (0: off), top_p (1: off, of what top_k leaves) and min_p (0: off, a share of the most likely
    token's probability) are numbers, or tensors of one a row (float32; top_k int32)."""
    dtype = _LOGIT_TYPES.get(logits.dtype)
    index = logits.get_device()
    if dtype is None or index < 0:
        raise TypeError("logits must be a float16, bfloat16 or float32 CUDA tensor")
    shape = logits.shape
    if len(shape) != 2:
        raise ValueError("logits must be [M, N] with contiguous rows")
    M, N = shape
    row, col = logits.stride()
    if col != 1 and N > 1:
        raise ValueError("logits must be [M, N] with contiguous rows")
    if u.dtype is not _f32 or u.get_device() != index:
        raise TypeError("u must be float32 on the logits' device")
    if u.shape != shape[:1] or not u.is_contiguous():
        raise ValueError(f"u must be a contiguous [{M}]")
    t, pt = _setting(temperature, "temperature", _f32, M, index)
    k, pk = _setting(top_k, "top_k", _i32, M, index)
    p, pp = _setting(top_p, "top_p", _f32, M, index)
    m, pm = _setting(min_p, "min_p", _f32, M, index)
    logprob = torch.empty_like(u)
    token = torch.empty_like(u, dtype=_i32)
    _run(index, _step_fn("sample_tokens"), logits.data_ptr(), dtype, M, N, row if M > 1 else 0, u.data_ptr(),
         _pack_sampling(t, p, m, k, pt, pp, pm, pk), token.data_ptr(), logprob.data_ptr(), _raw_stream(index))
    return SampledTokens(token, logprob)


class TreePath(NamedTuple):
    path: torch.Tensor                  # [B, max_path] int32, the accepted nodes, -1 behind them
    count: torch.Tensor                 # [B] int32, their number
    next_token: torch.Tensor            # [B] int32, the token drawn at the last of them


def tree_accept(tokens, drawn, parents, cu_tokens, max_path: int) -> TreePath:
    """The path of each sequence's tree that the drawn tokens accept: node 0, and after a node
    its first child whose token is the one drawn at the node.  tokens, drawn, parents int32 [T]."""
    index = tokens.get_device()
    shape, cu = tokens.shape, cu_tokens.shape
    if not (tokens.dtype is drawn.dtype is parents.dtype is cu_tokens.dtype is _i32 and shape == drawn.shape == parents.shape
            and index == drawn.get_device() == parents.get_device() == cu_tokens.get_device() >= 0
            and len(shape) == len(cu) == 1 and cu[0] > 0 and tokens.is_contiguous() and drawn.is_contiguous()
            and parents.is_contiguous() and cu_tokens.is_contiguous()):
        T = shape[0] if len(shape) else 0
        _need_ints(index, (tokens, "tokens", T), (drawn, "drawn", T), (parents, "parents", T),
                   (cu_tokens, "cu_tokens", max(cu[0] if len(cu) else 1, 1)))
    if not 1 <= max_path <= _INT_MAX:
        raise ValueError("max_path must be positive")
    B, dev, empty = cu[0] - 1, tokens.device, torch.empty
    path, count, following = empty((B, max_path), dtype=_i32, device=dev), empty(B, dtype=_i32, device=dev), empty(B, dtype=_i32, device=dev)
    _run(index, _step_fn("tree_accept"), tokens.data_ptr(), drawn.data_ptr(), parents.data_ptr(), cu_tokens.data_ptr(), B,
         shape[0], max_path, path.data_ptr(), count.data_ptr(), following.data_ptr(), _raw_stream(index))
    return TreePath(path, count, following)


def kv_keep_path(path, count, page_table, seq_lens, cu_tokens, *pools):
    """Moves the rows of each sequence's accepted nodes (path int32 [B, max_path], count int32
    [B], as tree_accept gives them) together behind the tokens before the tree, in every layer of
    the pools: K and V [pages, Hkv, page, d] or [layers, pages, Hkv, page, d] (any strides with d
    contiguous), the scales of an int8 cache [(layers,) pages, Hkv, page] float32.  seq_lens
    counts all nodes; returns the lengths that remain, int32 [B]."""
    index = path.get_device()
    if index < 0 or path.dtype is not _i32:
        raise TypeError("path must be an int32 CUDA tensor")
    batch = _kv_batch(page_table, seq_lens, cu_tokens, index)
    shape = path.shape
    if len(shape) != 2 or shape[0] != page_table.shape[0] or not path.is_contiguous():
        raise ValueError("path must be a contiguous [B, max_path]")
    if count.dtype is not _i32 or count.get_device() != index or count.shape != shape[:1] or not count.is_contiguous():
        _need_ints(index, (count, "count", shape[0]))
    if len(pools) > 4:
        raise ValueError("at most four pools")
    desc, page = [], 0
    for i, x in enumerate(pools):
        if x.get_device() != index:
            raise ValueError(f"pool {i} is on {x.device}, the path on {path.device}")
        dims, es = x.shape, x.element_size()
        if x.dtype is _f32:                       # scales: a row is one number
            if 1 in dims:
                stride = _strides(x.unsqueeze(-1))[:-1]
            else:
                stride = x.stride()
            row = 1
        else:
            stride = _strides(x) if 1 in dims else x.stride()
            if len(dims) < 4 or stride[-1] != 1 and dims[-1] != 1:
                raise ValueError(f"pool {i}: [(layers,) pages, Hkv, page, d] with d contiguous")
            row, dims, stride = dims[-1], dims[:-1], stride[:-1]
        if len(dims) == 4:
            layers, pages, heads, tokens = dims
            sl, sp, sh, st = stride
        elif len(dims) == 3:
            layers, (pages, heads, tokens) = 1, dims
            sl, (sp, sh, st) = 0, stride
        else:
            raise ValueError(f"pool {i}: [(layers,) pages, Hkv, page, ...]")
        if page and tokens != page:
            raise ValueError(f"pool {i} has pages of {tokens} tokens, the others of {page}")
        page = tokens
        desc.append(_pack_rows(x.data_ptr(), layers, pages, heads, row * es, sl * es, sp * es, sh * es, st * es))
    lens = torch.empty_like(count)
    _run(index, _step_fn("kv_keep_path"), b"".join(desc) or None, len(desc), batch, _INT_MAX, page or 1, path.data_ptr(),
         count.data_ptr(), shape[1], lens.data_ptr(), _raw_stream(index))
    return lens


def qgemm_w4a16_noalloc(x, packed, N: int, K: int, y=None):
    """qgemm_w4a16 with the library's built-in scratch instead of a workspace (for
    callers that cannot allocate device memory; see include/qgemm.h)."""
    _need(x, torch.float16, "x", 2)
    M = x.shape[0]
    if x.shape[1] != K:
        raise ValueError("x.shape[1] != K")
    y = _out(y, M, N, x.device)
    if M and N:
        _need_packed(packed, qpack_w4_bytes(N, K), x)
    with torch.cuda.device(x.device):
        _check(lib().qgemm_w4a16_noalloc(_ptr(x), _ptr(packed), M, N, K, _ptr(y), _stream(x)))
    return y


# -------------------------------------------------------------- diagnostics --
def device_error(stream=None) -> int:
    """Wait for the work enqueued on `stream` (default: the current stream of the current
    device), then return and clear the device error word of the current device."""
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(lib().qw_device_error(ctypes.c_void_p(stream.cuda_stream)))


QW_OPT_WEIGHTS_IMMUTABLE = 1


def set_weights_immutable(flag: bool = True):
    """Declare that packed weights are never written by the kernel that directly
    precedes a GEMM on its stream, letting each GEMM stream its weights while the
    preceding kernel finishes (see include/qgemm.h)."""
    _check(lib().qw_set_option(QW_OPT_WEIGHTS_IMMUTABLE, 1 if flag else 0))


QW_OPT_WAIT_LIMIT_US = 2
DEFAULT_WAIT_LIMIT_US = 4_000_000


def set_wait_limit_us(us: int | None = None):
    """Test hook: the time limit of every wait inside the GEMM kernels and attn_tree's launched
    from now on, in microseconds (None restores the 4 s default).  A kernel whose wait runs past
    it ends early with QW_ERR_TIMEOUT in the device error word."""
    _check(lib().qw_set_option(QW_OPT_WAIT_LIMIT_US, DEFAULT_WAIT_LIMIT_US if us is None else int(us)))


def num_kernel_launches() -> int:
    return int(lib().qw_num_kernel_launches())


# ----------------------------------------------------- measurement tools --
MMA_KINDS = {"f16": 0, "s8": 1, "e4m3": 2, "s4": 3}


def diag_mma_peak(kind: str, ctas: int, iters: int, chains: int = 8, device=None):
    """Launch the mma.sync rate (chains=8) or latency (chains=1) microbenchmark on the
    current stream; returns (ops of the launch, sink tensor).  The caller times it."""
    dev = torch.device(device or "cuda")
    sink = torch.empty(ctas * 256, dtype=torch.float32, device=dev)
    ops = ctypes.c_double(0.0)
    with torch.cuda.device(dev):
        _check(lib().qw_diag_mma_peak(MMA_KINDS[kind], ctas, iters, chains, _ptr(sink), ctypes.byref(ops),
                                      _stream(sink)))
    return ops.value, sink


def diag_tc_probe(kind: int, a_tmem: bool, n: int, issuers: int, chunks: int, window: int, grid: int,
                  device=None):
    """tcgen05.mma timing probe; returns the device tensor [grid, 4, 4] (issue ns, wait ns,
    total ns, chunks) -- read it after synchronizing."""
    dev = torch.device(device or "cuda")
    out = torch.zeros((grid, 4, 4), dtype=torch.int64, device=dev)
    with torch.cuda.device(dev):
        _check(lib().qw_diag_tc_probe(kind, 1 if a_tmem else 0, n, issuers, chunks, window, _ptr(out), grid,
                                      _stream(out)))
    return out


def diag_f8f6f4_gemm(a_e4m3, b_e4m3, a_tmem: bool):
    """d [128, 16] fp32 = a [128, K] . b [16, K]^T on tcgen05 kind::f8f6f4 (e4m3 bytes as uint8)."""
    _need(a_e4m3, torch.uint8, "a", 2)
    _need(b_e4m3, torch.uint8, "b", 2)
    K = a_e4m3.shape[1]
    if tuple(a_e4m3.shape) != (128, K) or tuple(b_e4m3.shape) != (16, K):
        raise ValueError("a must be [128, K] and b [16, K]")
    d = torch.empty((128, 16), dtype=torch.float32, device=a_e4m3.device)
    with torch.cuda.device(a_e4m3.device):
        _check(lib().qw_diag_f8f6f4_gemm(_ptr(a_e4m3), _ptr(b_e4m3), K, 1 if a_tmem else 0, _ptr(d),
                                         _stream(a_e4m3)))
    return d


def plan(mode: int, M: int, N: int, K: int, num_sms: int) -> Plan:
    p = Plan()
    _check(lib().qw_plan(mode, M, N, K, num_sms, ctypes.byref(p)))
    return p


def plan_segments(p: Plan, cta: int):
    n = lib().qw_plan_segments(ctypes.byref(p), cta, 0, None, None, None, None)
    if n < 0:
        _check(n)
    tile = (ctypes.c_longlong * max(n, 1))()
    g0 = (ctypes.c_int * max(n, 1))()
    g1 = (ctypes.c_int * max(n, 1))()
    slot = (ctypes.c_int * max(n, 1))()
    lib().qw_plan_segments(ctypes.byref(p), cta, n, tile, g0, g1, slot)
    return [(tile[i], g0[i], g1[i], slot[i]) for i in range(n)]


def plan_row_blocks(p: Plan, cta: int):
    """Under a row-block plan: the 16-row blocks (begin, end) CTA `cta` computes."""
    b, e = ctypes.c_int(), ctypes.c_int()
    _check(lib().qw_plan_row_blocks(ctypes.byref(p), cta, ctypes.byref(b), ctypes.byref(e)))
    return b.value, e.value
