"""Thin Python binding over the C ABI of ``libnvfp4skinny.so`` (ctypes).

Argument marshalling only: every step of the computation runs in the
library's CUDA kernels.  PyTorch supplies device memory and streams.  There is
no fallback: if the shared library is missing, ``load()`` raises.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np
import torch

from .build import LIB

NVFP4_GATED = 1
NVFP4_ROUTE_SOFTMAX_ALL = 1
NVFP4_KV_BF16 = 0
NVFP4_KV_E4M3 = 1
NVFP4_ROPE_INTERLEAVED = 1
NVFP4_ROPE_INVERSE = 2
KV_MAPS_BYTES = 1024
COUNTER_BYTES = 4096  # arrival counters at the start of an attention workspace
LAYOUT_VERSION = 2

STATUS = {0: "ok", 1: "null pointer", 2: "bad shape", 3: "misaligned pointer",
          4: "workspace missing or too small", 5: "weight layout version or flags mismatch", 6: "CUDA error"}

EXPORTS = (
    "nvfp4_status_string", "nvfp4_layout_version", "nvfp4_device_error", "nvfp4_repacked_bytes",
    "nvfp4_quantize_workspace_bytes", "nvfp4_quantize", "nvfp4_repack", "nvfp4_gemm_workspace_bytes",
    "nvfp4_gemm", "moe_route_topk", "moe_ffn_workspace_bytes", "moe_ffn_grouped",
    "lm_head_workspace_bytes", "lm_head_argmax", "lm_head_argmax_noalloc", "nvfp4_plan_info",
    "lm_head_sample", "moe_route_topk_ex", "lm_head_sample_ex", "nvfp4_plan_check", "moe_router_logits",
    "nvfp4_repack_host", "nvfp4_quantize_act", "nvfp4_gemm_w4a4", "lm_head_argmax_w4a4", "moe_forward", "nvfp4_selftest_wait_timeout",
    "rope_frequencies", "rope_apply", "kv_append", "kv_cache_maps", "paged_attention_workspace_bytes", "paged_attention",
    "paged_attention_plan_check",
)


class NVFP4Error(RuntimeError):
    def __init__(self, call: str, status: int):
        super().__init__(f"{call} failed: {STATUS.get(status, status)} ({status})")
        self.status = status


class CWeight(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("global_scale", ctypes.c_void_p), ("n", ctypes.c_int32),
                ("k", ctypes.c_int32), ("num_matrices", ctypes.c_int32), ("flags", ctypes.c_uint32),
                ("layout_version", ctypes.c_uint32)]


@dataclass
class Weight:
    """A repacked NVFP4 weight living on the GPU (owns its tensors)."""
    data: torch.Tensor          # uint8, repacked tiles
    global_scale: torch.Tensor  # float32 [num_matrices]
    n: int
    k: int
    num_matrices: int = 1
    flags: int = 0

    def c(self) -> CWeight:
        return CWeight(self.data.data_ptr(), self.global_scale.data_ptr(), self.n, self.k,
                       self.num_matrices, self.flags, LAYOUT_VERSION)

    @property
    def nbytes_algorithmic(self) -> int:
        """Bytes the method must read: n*k/2 nibbles + n*k/16 scales per matrix."""
        return self.num_matrices * (self.n * self.k // 2 + self.n * self.k // 16)


class CKVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("num_pages", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32),
                ("dtype", ctypes.c_uint32), ("maps", ctypes.c_void_p)]


class CBatch(ctypes.Structure):
    _fields_ = [("cu_tokens", ctypes.c_void_p), ("kv_len", ctypes.c_void_p), ("page_table", ctypes.c_void_p),
                ("n_seqs", ctypes.c_int32), ("max_pages", ctypes.c_int32), ("max_new", ctypes.c_int32)]


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


def _need_int32(value: int, what: str):
    """ctypes cuts an integer to the 32 bits of its parameter without a word."""
    if not -2 ** 31 <= value < 2 ** 31:
        raise ValueError(f"{what}: beyond 32 bits")


class KVCache:
    """A paged key/value cache on the GPU: pools [num_pages, n_kv_heads, page_size, head_dim] of bf16, or of
    float8_e4m3fn holding value / scale with fp32 scales per kv head (None: ones).  Pages may be strided (k and v
    in one pool); the rest is contiguous.  Keeps its tensors and its TMA descriptors; make it once per pool."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor = None, v_scale: torch.Tensor = None):
        _need(k.dim() == 4 and k.shape == v.shape and k.dtype == v.dtype and k.stride() == v.stride(),
              "k and v: pools of one shape, type and layout, [num_pages, n_kv_heads, page_size, head_dim]")
        _need(k.is_cuda and v.device == k.device, "k and v: pools on one GPU")
        _need(k.dtype in (torch.bfloat16, torch.float8_e4m3fn), "k and v: bf16 or float8_e4m3fn")
        pages, heads, page, dim = k.shape
        _need(k.stride()[1:] == (page * dim, dim, 1), "the heads of a page have to be contiguous")
        for s in (k_scale, v_scale):
            _need(s is None or (s.dtype == torch.float32 and s.shape == (heads,) and s.is_contiguous()
                                and s.device == k.device), "scales: contiguous fp32 [n_kv_heads] on the cache's GPU")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_kv_heads, self.page_size, self.head_dim, self.device = heads, page, dim, k.device
        stride = k.stride(0) if pages > 1 else heads * page * dim
        self.c = CKVCache(k.data_ptr(), v.data_ptr(), _ptr(k_scale), _ptr(v_scale), stride, pages, page, heads, dim,
                          NVFP4_KV_BF16 if k.dtype == torch.bfloat16 else NVFP4_KV_E4M3)
        self.ref = ctypes.byref(self.c)
        self._maps = ctypes.create_string_buffer(KV_MAPS_BYTES + 128)
        at = -(-ctypes.addressof(self._maps) // 128) * 128
        st = load().lib.kv_cache_maps(self.ref, at)
        if st:
            raise NVFP4Error("kv_cache_maps", st)
        self.c.maps = at


class Batch:
    """The sequences of an attention call: cu_tokens int32 [n_seqs + 1], kv_len int32 [n_seqs] (new tokens
    included), page_table int32 [n_seqs, max_pages], and max_new, a bound on the new tokens of any sequence.
    Keeps its tensors alive; their contents may change between calls (a captured graph reads them anew)."""

    def __init__(self, cu_tokens: torch.Tensor, kv_len: torch.Tensor, page_table: torch.Tensor, max_new: int):
        n = kv_len.shape[0]
        _need(page_table.dim() == 2 and cu_tokens.shape == (n + 1,) and kv_len.shape == (n,)
              and page_table.shape[0] == n, "cu_tokens [n_seqs + 1], kv_len [n_seqs], page_table [n_seqs, max_pages]")
        for x in (cu_tokens, kv_len, page_table):
            _need(x.dtype == torch.int32 and x.is_contiguous() and x.is_cuda and x.device == kv_len.device,
                  "cu_tokens, kv_len, page_table: contiguous int32 on one GPU")
        _need_int32(max_new, "max_new")
        self.cu_tokens, self.kv_len, self.page_table, self.max_new = cu_tokens, kv_len, page_table, int(max_new)
        self.n_seqs, self.device = n, kv_len.device
        self.c = CBatch(cu_tokens.data_ptr(), kv_len.data_ptr(), page_table.data_ptr(), n, page_table.shape[1],
                        self.max_new)
        self.ref = ctypes.byref(self.c)


_P = ctypes.c_void_p
_I = ctypes.c_int32
_SZ = ctypes.c_size_t
_I64 = ctypes.c_int64


def _sig(lib):
    lib.nvfp4_status_string.restype = ctypes.c_char_p
    lib.nvfp4_status_string.argtypes = [ctypes.c_int]
    lib.nvfp4_layout_version.restype = ctypes.c_uint32
    lib.nvfp4_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), _I]
    lib.nvfp4_repacked_bytes.restype = _SZ
    lib.nvfp4_repacked_bytes.argtypes = [_I, _I, _I]
    lib.nvfp4_quantize_workspace_bytes.restype = _SZ
    lib.nvfp4_quantize_workspace_bytes.argtypes = [_I]
    lib.nvfp4_quantize.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]
    lib.nvfp4_repack.argtypes = [_P, _P, _I, _I, _I, ctypes.c_uint32, _P, _P]
    lib.nvfp4_gemm_workspace_bytes.restype = _SZ
    lib.nvfp4_gemm_workspace_bytes.argtypes = [_I, _I, _I]
    lib.nvfp4_gemm.argtypes = [ctypes.POINTER(CWeight), _P, _I, _P, _P, _SZ, _P]
    lib.moe_route_topk.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _P]
    lib.moe_route_topk_ex.argtypes = [_P, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P]
    lib.moe_route_topk_ex.restype = ctypes.c_int
    lib.moe_ffn_workspace_bytes.restype = _SZ
    lib.moe_ffn_workspace_bytes.argtypes = [_I, _I, _I, _I, _I]
    lib.moe_ffn_grouped.argtypes = [_P, _I, _I, _P, _P, _P, ctypes.POINTER(CWeight), ctypes.POINTER(CWeight),
                                    ctypes.POINTER(CWeight), ctypes.POINTER(CWeight), _P, _P, _SZ, _P]
    lib.lm_head_workspace_bytes.restype = _SZ
    lib.lm_head_workspace_bytes.argtypes = [_I, _I]
    lib.lm_head_argmax.argtypes = [ctypes.POINTER(CWeight), _P, _I, _P, _P, _P, _SZ, _P]
    lib.lm_head_argmax_noalloc.argtypes = [ctypes.POINTER(CWeight), _P, _I, _P, _P, _P]
    lib.lm_head_sample.argtypes = [ctypes.POINTER(CWeight), _P, _I, ctypes.c_float, ctypes.c_uint64, _P, _P, _P, _SZ,
                                   _P]
    lib.lm_head_sample.restype = ctypes.c_int
    lib.nvfp4_plan_info.argtypes = [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_int32), _I]
    lib.nvfp4_plan_info.restype = ctypes.c_int
    lib.nvfp4_plan_check.argtypes = [_I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_int32), _I]
    lib.nvfp4_plan_check.restype = ctypes.c_int
    lib.lm_head_sample_ex.argtypes = [ctypes.POINTER(CWeight), _P, _I, ctypes.c_float, ctypes.c_float, ctypes.c_uint64,
                                      _P, _P, _P, _SZ, _P]
    lib.lm_head_sample_ex.restype = ctypes.c_int
    lib.moe_router_logits.argtypes = [ctypes.POINTER(CWeight), _P, _I, _P, ctypes.c_float, _P, _P, _SZ, _P]
    lib.moe_router_logits.restype = ctypes.c_int
    lib.moe_forward.argtypes = [_P, _P, _I, _I, _I, _P, _P, _P, _P, _P, ctypes.POINTER(CWeight),
                                ctypes.POINTER(CWeight), ctypes.POINTER(CWeight), ctypes.POINTER(CWeight), _P, _P, _SZ,
                                _P]
    lib.moe_forward.restype = ctypes.c_int
    lib.nvfp4_selftest_wait_timeout.argtypes = [ctypes.c_int64, _P]
    lib.nvfp4_selftest_wait_timeout.restype = ctypes.c_int
    lib.nvfp4_quantize_act.argtypes = [_P, _I, _I, _P, _P, _P, _P, _SZ, _P]
    lib.nvfp4_quantize_act.restype = ctypes.c_int
    lib.nvfp4_gemm_w4a4.argtypes = [ctypes.POINTER(CWeight), _P, _P, _P, _I, _P, _P, _SZ, _P]
    lib.nvfp4_gemm_w4a4.restype = ctypes.c_int
    lib.lm_head_argmax_w4a4.argtypes = [ctypes.POINTER(CWeight), _P, _P, _P, _I, _P, _P, _P, _SZ, _P]
    lib.lm_head_argmax_w4a4.restype = ctypes.c_int
    lib.nvfp4_repack_host.argtypes = [_P, _P, _I, _I, _I, ctypes.c_uint32, _P, _SZ]
    lib.nvfp4_repack_host.restype = ctypes.c_int
    lib.rope_frequencies.argtypes = [_I] + [ctypes.c_double] * 5 + [_P]
    lib.rope_frequencies.restype = ctypes.c_int
    lib.rope_apply.argtypes = [_P, _I64, _I, _I, _I, _P, _P, _I, ctypes.c_float, _I, _P, _I64, _P]
    lib.rope_apply.restype = ctypes.c_int
    lib.kv_append.argtypes = [_P, _P, _I64, _P, _I64, _I, _P, _P, _P, _I, ctypes.c_float, _I, _P, _I64, _I, _P, _I64,
                              _P]
    lib.kv_append.restype = ctypes.c_int
    lib.kv_cache_maps.argtypes = [_P, _P]
    lib.kv_cache_maps.restype = ctypes.c_int
    lib.paged_attention_workspace_bytes.restype = _SZ
    lib.paged_attention_workspace_bytes.argtypes = [_I] * 6
    lib.paged_attention.argtypes = [_P, _P, _P, _I64, _I, _I, ctypes.c_float, ctypes.c_float, _I, _P, _I64, _P, _P,
                                    _SZ, _P]
    lib.paged_attention.restype = ctypes.c_int
    lib.paged_attention_plan_check.argtypes = [_P, _P, _I, _I, _I, _I, ctypes.POINTER(ctypes.c_int32), _I]
    lib.paged_attention_plan_check.restype = ctypes.c_int
    for name in ("nvfp4_quantize", "nvfp4_repack", "nvfp4_gemm", "moe_route_topk", "moe_ffn_grouped",
                 "lm_head_argmax", "lm_head_argmax_noalloc", "nvfp4_device_error"):
        getattr(lib, name).restype = ctypes.c_int


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _ptr(t):
    return None if t is None else t.data_ptr()


def _raw_stream(stream, device) -> int:
    """The stream's handle; the current stream of `device` without building a Stream object."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


_current_device = getattr(torch._C, "_cuda_getDevice", None)  # (a CPU build of torch can still import the package)


def _on_current(device, stream):
    """The library launches on the current device; a default stream's handle is the same on every one."""
    if device.type != "cuda" or device.index != _current_device():
        raise ValueError(f"tensors on {device}: they have to be on the current GPU (torch.cuda.device(...) makes it so)")
    if stream is not None and stream.device_index != device.index:
        raise ValueError("stream: of another GPU than the tensors")


def _is_capturing(stream) -> bool:
    """Whether a stream is being captured into a graph."""
    with torch.cuda.stream(stream):
        return torch.cuda.is_current_stream_capturing()


def _empty(shape, dtype, device, stream):
    """An output, allocated on the stream that writes it: memory that another stream's work may still use is not
    written before that work is done."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _used_on(stream, *tensors):
    """Tensors that a call on an explicitly given stream uses: their memory is not given away before that stream is
    done with it."""
    for x in tensors:
        if x is not None:
            x.record_stream(stream)


def _rows(x: torch.Tensor, what: str, device) -> int:
    """Rows of heads [tokens, heads, dim]: the row stride in elements."""
    shape = x.shape
    if len(shape) == 3 and x.dtype is torch.bfloat16 and x.device == device:
        row, head, one = x.stride()
        if one == 1 and (head == shape[2] or shape[1] == 1):
            return row if shape[0] > 1 else shape[1] * shape[2]
    raise ValueError(f"{what}: bf16 [tokens, heads, dim] on the call's GPU, the heads of a token contiguous")


def _index(x: torch.Tensor, n: int, dtype, what: str, device) -> int:
    if x.dtype is dtype and x.shape == (n,) and x.device == device and (n < 2 or x.stride(0) == 1):
        return x.data_ptr()
    raise ValueError(f"{what}: contiguous {dtype} [{n}] on the call's GPU")


class Library:
    """The loaded C ABI; methods take CUDA tensors and enqueue on the current stream."""

    def __init__(self, path: str = LIB):
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -m nvfp4_w4a16_moe_skinny_gb300.build` "
                               "(there is no CPU fallback)")
        self.path = path
        self.lib = ctypes.CDLL(path)
        _sig(self.lib)
        self._ws = {}
        self._attention_bytes = {}  # attention workspaces: their sizes by the sizes of a call,
        self._attention_ws = {}     # and one for each (device, stream)

    # -------------------------------------------------------------- plumbing
    def _check(self, call, st):
        if st != 0:
            raise NVFP4Error(call, st)

    def workspace(self, key, nbytes: int, device) -> torch.Tensor:
        """A per-(call kind, device) workspace, zero-filled once at allocation."""
        cur = self._ws.get((key, device))
        if cur is None or cur.numel() < nbytes:
            cur = torch.zeros(max(nbytes, 16), dtype=torch.uint8, device=device)
            self._ws[(key, device)] = cur
        return cur

    def device_error(self, clear: bool = True) -> int:
        v = ctypes.c_uint32(0)
        self._check("nvfp4_device_error", self.lib.nvfp4_device_error(ctypes.byref(v), int(clear)))
        return v.value

    def selftest_wait_timeout(self, limit_cycles: int, stream=None):
        """Run the bounded-wait self-test (a wait that runs out after limit_cycles)."""
        self._check("nvfp4_selftest_wait_timeout", self.lib.nvfp4_selftest_wait_timeout(int(limit_cycles),
                                                                                        _stream(stream)))

    def repacked_bytes(self, n, k, num_matrices=1) -> int:
        return self.lib.nvfp4_repacked_bytes(n, k, num_matrices)

    # -------------------------------------------------------------- offline
    def quantize(self, w: torch.Tensor, stream=None):
        """fp32 [E, n, k] or [n, k] on the GPU -> canonical (nibbles, scales, global_scale)."""
        squeeze = w.dim() == 2
        w3 = w.unsqueeze(0) if squeeze else w
        w3 = w3.contiguous()
        e, n, k = w3.shape
        nib = torch.empty((e, n, k // 2), dtype=torch.uint8, device=w.device)
        sc = torch.empty((e, n, k // 16), dtype=torch.uint8, device=w.device)
        g = torch.empty((e,), dtype=torch.float32, device=w.device)
        ws = torch.empty((max(1, self.lib.nvfp4_quantize_workspace_bytes(e)),), dtype=torch.uint8, device=w.device)
        self._check("nvfp4_quantize", self.lib.nvfp4_quantize(
            w3.data_ptr(), e, n, k, nib.data_ptr(), sc.data_ptr(), g.data_ptr(), ws.data_ptr(), ws.numel(),
            _stream(stream)))
        if squeeze:
            return nib[0], sc[0], g
        return nib, sc, g

    def repack(self, nib: torch.Tensor, sc: torch.Tensor, gscale: torch.Tensor, gated: bool = False,
               stream=None) -> Weight:
        nib3 = nib.unsqueeze(0) if nib.dim() == 2 else nib
        sc3 = sc.unsqueeze(0) if sc.dim() == 2 else sc
        e, n, kh = nib3.shape
        k = 2 * kh
        out = torch.empty((self.repacked_bytes(n, k, e),), dtype=torch.uint8, device=nib.device)
        flags = NVFP4_GATED if gated else 0
        self._check("nvfp4_repack", self.lib.nvfp4_repack(
            nib3.contiguous().data_ptr(), sc3.contiguous().data_ptr(), e, n, k, flags, out.data_ptr(),
            _stream(stream)))
        return Weight(out, gscale.reshape(-1).contiguous().float(), n, k, e, flags)

    def repack_host(self, nib: np.ndarray, sc: np.ndarray, gated: bool = False) -> np.ndarray:
        """The host-memory repack: canonical u8 [E, n, k/2] / [E, n, k/16] (or 2-D) numpy
        arrays -> the repacked bytes (u8 numpy)."""
        nib3 = np.ascontiguousarray(nib.reshape((-1,) + nib.shape[-2:]), np.uint8)
        sc3 = np.ascontiguousarray(sc.reshape((-1,) + sc.shape[-2:]), np.uint8)
        e, n, kh = nib3.shape
        k = 2 * kh
        out = np.empty((self.repacked_bytes(n, k, e),), dtype=np.uint8)
        self._check("nvfp4_repack_host", self.lib.nvfp4_repack_host(
            nib3.ctypes.data, sc3.ctypes.data, e, n, k, NVFP4_GATED if gated else 0, out.ctypes.data, out.nbytes))
        return out

    def prepare(self, w: torch.Tensor, gated: bool = False, stream=None) -> Weight:
        """quantize + repack of fp32 weights already on the GPU."""
        nib, sc, g = self.quantize(w, stream)
        return self.repack(nib, sc, g, gated, stream)

    # -------------------------------------------------------------- hot path
    def gemm(self, w: Weight, x: torch.Tensor, y: torch.Tensor = None, stream=None) -> torch.Tensor:
        m = x.shape[0]
        if y is None:
            y = torch.empty((m, w.n), dtype=torch.bfloat16, device=x.device)
        nbytes = self.lib.nvfp4_gemm_workspace_bytes(m, w.n, w.k)
        ws = self.workspace("gemm", nbytes, x.device)
        cw = w.c()
        self._check("nvfp4_gemm", self.lib.nvfp4_gemm(
            ctypes.byref(cw), x.data_ptr(), m, y.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
        return y

    def lm_head_argmax(self, w: Weight, x: torch.Tensor, out=None, stream=None):
        m = x.shape[0]
        if out is None:
            out = (torch.empty((m,), dtype=torch.float32, device=x.device),
                   torch.empty((m,), dtype=torch.int32, device=x.device))
        nbytes = self.lib.lm_head_workspace_bytes(m, w.n)
        ws = self.workspace("lm_head", nbytes, x.device)
        cw = w.c()
        self._check("lm_head_argmax", self.lib.lm_head_argmax(
            ctypes.byref(cw), x.data_ptr(), m, out[0].data_ptr(), out[1].data_ptr(), ws.data_ptr(), ws.numel(),
            _stream(stream)))
        return out

    # -------------------------------------------------------------- W4A4
    def quantize_act(self, x: torch.Tensor, out=None, stream=None):
        """bf16 activations [m, k] -> NVFP4 per token row: (codes u8 [m, k/2], scales u8
        [m, k/16], global scales fp32 [m])."""
        m, k = x.shape
        if out is None:
            out = (torch.empty((m, k // 2), dtype=torch.uint8, device=x.device),
                   torch.empty((m, k // 16), dtype=torch.uint8, device=x.device),
                   torch.empty((m,), dtype=torch.float32, device=x.device))
        ws = self.workspace("quantize_act", max(16, self.lib.nvfp4_quantize_workspace_bytes(m)), x.device)
        self._check("nvfp4_quantize_act", self.lib.nvfp4_quantize_act(
            x.data_ptr(), m, k, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), ws.data_ptr(), ws.numel(),
            _stream(stream)))
        return out

    def gemm_w4a4(self, w: Weight, xq, y: torch.Tensor = None, stream=None) -> torch.Tensor:
        codes, scales, g = xq
        m = codes.shape[0]
        if y is None:
            y = torch.empty((m, w.n), dtype=torch.bfloat16, device=codes.device)
        ws = self.workspace("gemm", self.lib.nvfp4_gemm_workspace_bytes(m, w.n, w.k), codes.device)
        cw = w.c()
        self._check("nvfp4_gemm_w4a4", self.lib.nvfp4_gemm_w4a4(
            ctypes.byref(cw), codes.data_ptr(), scales.data_ptr(), g.data_ptr(), m, y.data_ptr(), ws.data_ptr(),
            ws.numel(), _stream(stream)))
        return y

    def lm_head_argmax_w4a4(self, w: Weight, xq, out=None, stream=None):
        codes, scales, g = xq
        m = codes.shape[0]
        if out is None:
            out = (torch.empty((m,), dtype=torch.float32, device=codes.device),
                   torch.empty((m,), dtype=torch.int32, device=codes.device))
        ws = self.workspace("lm_head", self.lib.lm_head_workspace_bytes(m, w.n), codes.device)
        cw = w.c()
        self._check("lm_head_argmax_w4a4", self.lib.lm_head_argmax_w4a4(
            ctypes.byref(cw), codes.data_ptr(), scales.data_ptr(), g.data_ptr(), m, out[0].data_ptr(),
            out[1].data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
        return out

    def lm_head_sample(self, w: Weight, x: torch.Tensor, temperature: float, seed: int, out=None, stream=None,
                       softcap: float = 0.0):
        """Gumbel-max sample per token row (temperature 0: greedy): returns (max key, token).
        softcap > 0 applies cap * tanh(logit / cap) to every logit first."""
        m = x.shape[0]
        if out is None:
            out = (torch.empty((m,), dtype=torch.float32, device=x.device),
                   torch.empty((m,), dtype=torch.int32, device=x.device))
        ws = self.workspace("lm_head", self.lib.lm_head_workspace_bytes(m, w.n), x.device)
        cw = w.c()
        if softcap:
            self._check("lm_head_sample_ex", self.lib.lm_head_sample_ex(
                ctypes.byref(cw), x.data_ptr(), m, float(softcap), float(temperature), int(seed) & (2 ** 64 - 1),
                out[0].data_ptr(), out[1].data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
        else:
            self._check("lm_head_sample", self.lib.lm_head_sample(
                ctypes.byref(cw), x.data_ptr(), m, float(temperature), int(seed) & (2 ** 64 - 1), out[0].data_ptr(),
                out[1].data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
        return out

    def plan_lm_head_sample(self, w: Weight, x: torch.Tensor, temperature: float, seed: int, max_key, token,
                            stream=None):
        """lm_head_sample as a zero-argument callable (arguments marshalled once)."""
        m = x.shape[0]
        ws = self.workspace("lm_head", self.lib.lm_head_workspace_bytes(m, w.n), x.device)
        cw = w.c()
        args = (ctypes.byref(cw), x.data_ptr(), m, float(temperature), int(seed) & (2 ** 64 - 1), max_key.data_ptr(),
                token.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
        fn = self.lib.lm_head_sample

        def run():
            st = fn(*args)
            if st:
                raise NVFP4Error("lm_head_sample", st)
        run.keep = (cw, ws)
        return run

    def router_logits(self, w: Weight, x: torch.Tensor, gate_scale: torch.Tensor = None, eps: float = 1e-6,
                      out: torch.Tensor = None, stream=None) -> torch.Tensor:
        """Router logits: the unweighted RMSNorm of W . x times the per-expert scale (fp32 [m, n_experts])."""
        m = x.shape[0]
        if out is None:
            out = torch.empty((m, w.n), dtype=torch.float32, device=x.device)
        ws = self.workspace("gemm", self.lib.nvfp4_gemm_workspace_bytes(m, w.n, w.k), x.device)
        cw = w.c()
        self._check("moe_router_logits", self.lib.moe_router_logits(
            ctypes.byref(cw), x.data_ptr(), m, _ptr(gate_scale), float(eps), out.data_ptr(), ws.data_ptr(), ws.numel(),
            _stream(stream)))
        return out

    def route_topk(self, logits: torch.Tensor, top_k: int, out=None, stream=None, softmax_all: bool = False,
                   expert_scale: torch.Tensor = None):
        m, e = logits.shape
        if out is None:
            dev = logits.device
            out = (torch.empty((m, top_k), dtype=torch.int32, device=dev),
                   torch.empty((m, top_k), dtype=torch.float32, device=dev),
                   torch.empty((e + 1,), dtype=torch.int32, device=dev),
                   torch.empty((m * top_k,), dtype=torch.int32, device=dev))
        ids, probs, offsets, pairs = out
        if not softmax_all and expert_scale is None:
            self._check("moe_route_topk", self.lib.moe_route_topk(
                logits.data_ptr(), m, e, top_k, ids.data_ptr(), probs.data_ptr(), offsets.data_ptr(),
                pairs.data_ptr(), _stream(stream)))
        else:
            self._check("moe_route_topk_ex", self.lib.moe_route_topk_ex(
                logits.data_ptr(), m, e, top_k, NVFP4_ROUTE_SOFTMAX_ALL if softmax_all else 0,
                expert_scale.data_ptr() if expert_scale is not None else None, ids.data_ptr(), probs.data_ptr(),
                offsets.data_ptr(), pairs.data_ptr(), _stream(stream)))
        return out

    def moe_ffn(self, x, top_k, probs, offsets, pairs, gate_up: Weight, down: Weight, shared_gate_up: Weight = None,
                shared_down: Weight = None, out=None, stream=None):
        m, d = x.shape
        inter = down.k
        if out is None:
            out = torch.empty((m, d), dtype=torch.bfloat16, device=x.device)
        nbytes = self.lib.moe_ffn_workspace_bytes(m, top_k, gate_up.num_matrices, d, inter)
        ws = self.workspace("moe", nbytes, x.device)
        cg, cd = gate_up.c(), down.c()
        sg = ctypes.byref(shared_gate_up.c()) if shared_gate_up is not None else None
        sd = ctypes.byref(shared_down.c()) if shared_down is not None else None
        self._check("moe_ffn_grouped", self.lib.moe_ffn_grouped(
            x.data_ptr(), m, top_k, probs.data_ptr(), offsets.data_ptr(), pairs.data_ptr(), ctypes.byref(cg),
            ctypes.byref(cd), sg, sd, out.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream)))
        return out

    # -------------------------------------------------------------- attention side
    def rope_frequencies(self, rot_dim: int, theta: float = 10000.0, factor: float = 1.0, trained_context: float = 0.0,
                         slow: float = 1.0, fast: float = 32.0, device=None) -> torch.Tensor:
        """Radians a position for each rotated pair, fp64 [rot_dim / 2] (on `device`, if given).  factor > 1 stretches
        them: all of them (trained_context 0), or those that make fewer than `fast` turns over the trained context,
        wholly below `slow` turns."""
        _need_int32(rot_dim, "rot_dim")
        out = torch.empty((max(0, rot_dim) // 2,), dtype=torch.float64)
        self._check("rope_frequencies", self.lib.rope_frequencies(rot_dim, theta, factor, trained_context, slow, fast,
                                                                  out.data_ptr() or None))
        return out if device is None else out.to(device)

    def rope_apply(self, x: torch.Tensor, positions: torch.Tensor, inv_freq: torch.Tensor, interleaved: bool = False,
                   amplitude: float = 1.0, inverse: bool = False, out: torch.Tensor = None, stream=None) -> torch.Tensor:
        """Rotary positions on the first 2 * len(inv_freq) values of every head of x [tokens, heads, dim]; out may be x.
        inverse rotates back, which is the gradient's way through the rotation."""
        dev = x.device
        if dev.index != _current_device() or stream is not None:
            _on_current(dev, stream)
        stride = _rows(x, "x", dev)
        tokens, heads, dim = x.shape
        pairs = inv_freq.shape[0]
        if out is None:
            out = _empty((tokens, heads, dim), torch.bfloat16, dev, stream)
            out_stride = heads * dim
        else:
            _need(out.shape == x.shape, "out: the shape of x")
            out_stride = _rows(out, "out", dev)
        st = self.lib.rope_apply(
            x.data_ptr(), stride, tokens, heads, dim, _index(positions, tokens, torch.int32, "positions", dev),
            _index(inv_freq, pairs, torch.float64, "inv_freq", dev), 2 * pairs, amplitude,
            (NVFP4_ROPE_INTERLEAVED if interleaved else 0) | (NVFP4_ROPE_INVERSE if inverse else 0), out.data_ptr(),
            out_stride, _raw_stream(stream, dev))
        if st:
            raise NVFP4Error("rope_apply", st)
        if stream is not None:
            _used_on(stream, x, positions, inv_freq, out)
        return out

    def kv_append(self, cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                  positions: torch.Tensor = None, inv_freq: torch.Tensor = None, interleaved: bool = False,
                  amplitude: float = 1.0, q: torch.Tensor = None, q_out: torch.Tensor = None, stream=None):
        """Write k (rotated, if inv_freq is given) and v [tokens, n_kv_heads, dim] to slots int64 [tokens] of the cache
        (negative: skipped) and return the rotated q (None without q); q_out may be q."""
        dev = cache.device
        if dev.index != _current_device() or stream is not None:
            _on_current(dev, stream)
        tokens, heads, dim = k.shape
        _need(k.shape == v.shape and heads == cache.n_kv_heads and dim == cache.head_dim,
              "k and v: [tokens, n_kv_heads, head_dim] of the cache")
        pos = freq = None
        rot = 0
        if inv_freq is not None:
            _need(positions is not None, "positions are needed with inv_freq")
            rot = 2 * inv_freq.shape[0]
            freq = _index(inv_freq, inv_freq.shape[0], torch.float64, "inv_freq", dev)
            pos = _index(positions, tokens, torch.int32, "positions", dev)
        q_ptr = out_ptr = None
        q_heads = q_stride = out_stride = 0
        if q is not None:
            q_heads = q.shape[1]
            _need(q.shape == (tokens, q_heads, dim), "q: [tokens, heads, head_dim] of the cache")
            q_ptr, q_stride = q.data_ptr(), _rows(q, "q", dev)
            if q_out is None:
                q_out = _empty((tokens, q_heads, dim), torch.bfloat16, dev, stream)
                out_stride = q_heads * dim
            else:
                _need(q_out.shape == q.shape, "q_out: the shape of q")
                out_stride = _rows(q_out, "q_out", dev)
            out_ptr = q_out.data_ptr()
        st = self.lib.kv_append(
            cache.ref, k.data_ptr(), _rows(k, "k", dev), v.data_ptr(), _rows(v, "v", dev), tokens,
            _index(slots, tokens, torch.int64, "slots", dev), pos, freq, rot, amplitude,
            NVFP4_ROPE_INTERLEAVED if interleaved else 0, q_ptr, q_stride, q_heads, out_ptr, out_stride,
            _raw_stream(stream, dev))
        if st:
            raise NVFP4Error("kv_append", st)
        if stream is not None:
            _used_on(stream, k, v, slots, positions, inv_freq, q, q_out, cache.k, cache.v, cache.k_scale, cache.v_scale)
        return q_out

    def paged_attention(self, q: torch.Tensor, cache: KVCache, batch: Batch, scale: float = None, softcap: float = 0.0,
                        window: int = 0, out: torch.Tensor = None, lse: torch.Tensor = None, with_lse: bool = False,
                        stream=None):
        """Attention of the batch's new tokens q [tokens, heads, dim] over their sequences' cached keys (scale: 1 /
        sqrt(dim)): out, or (out, log-sum-exp fp32 [tokens, heads]) with with_lse."""
        dev = cache.device
        if dev.index != _current_device() or stream is not None:
            _on_current(dev, stream)
        stride = _rows(q, "q", dev)
        shape = q.shape
        tokens, heads, dim = shape
        if dim != cache.head_dim or batch.device != dev:
            raise ValueError("q: [tokens, heads, head_dim] of the cache; the batch on its GPU")
        if not -2 ** 31 <= window < 2 ** 31:
            raise ValueError("window: beyond 32 bits")
        if out is None:
            out = _empty(shape, torch.bfloat16, dev, stream)
            out_stride = heads * dim
        else:
            _need(out.shape == shape, "out: the shape of q")
            out_stride = _rows(out, "out", dev)
        lse_ptr = None
        if lse is not None:
            _need(lse.shape == (tokens, heads) and lse.dtype is torch.float32 and lse.is_contiguous()
                  and lse.device == dev, "lse: contiguous fp32 [tokens, heads]")
            lse_ptr = lse.data_ptr()
        elif with_lse:
            lse = _empty((tokens, heads), torch.float32, dev, stream)
            lse_ptr = lse.data_ptr()
        raw = _raw_stream(stream, dev)
        sizes = (tokens, batch.n_seqs, batch.max_new, heads, cache.n_kv_heads, dim)
        nbytes = self._attention_bytes.get(sizes)
        if nbytes is None:
            if len(self._attention_bytes) > 4096:
                self._attention_bytes.clear()
            nbytes = self._attention_bytes[sizes] = self.lib.paged_attention_workspace_bytes(*sizes)
        ws, ws_ptr, ws_bytes = self._stream_workspace(nbytes, dev, raw, stream)
        st = self.lib.paged_attention(
            cache.ref, batch.ref, q.data_ptr(), stride, tokens, heads, dim ** -0.5 if scale is None else scale, softcap,
            window, out.data_ptr(), out_stride, lse_ptr, ws_ptr, ws_bytes, raw)
        if st:
            raise NVFP4Error("paged_attention", st)
        if stream is not None:
            _used_on(stream, q, out, lse, cache.k, cache.v, cache.k_scale, cache.v_scale, batch.cu_tokens, batch.kv_len,
                     batch.page_table)
        return (out, lse) if with_lse else out

    def _stream_workspace(self, nbytes: int, device, raw: int, stream):
        """(tensor, address, bytes) of an attention workspace.  Each (device, stream) has its own: calls on different
        streams may overlap.  It is allocated, and its counters cleared, on the stream that uses it, so that one that
        is outgrown is not reused under a running call.  A captured call gets one from its graph's pool, which lives
        and dies with the graph and whose counters are cleared at every replay."""
        key = (device.index, raw)
        cur = self._attention_ws.get(key)
        capturing = torch.cuda.is_current_stream_capturing() if stream is None else _is_capturing(stream)
        if cur is not None and cur[2] >= nbytes and not capturing:
            return cur
        with torch.cuda.stream(torch.cuda.current_stream(device) if stream is None else stream):
            ws = torch.empty(max(nbytes, COUNTER_BYTES), dtype=torch.uint8, device=device)
            ws[:COUNTER_BYTES].zero_()
            cur = (ws, ws.data_ptr(), ws.numel())
            if not capturing:
                self._attention_ws[key] = cur
        return cur

    # -------------------------------------------------------------- call plans
    # Zero-argument callables with every ctypes argument built once, for timed
    # loops where per-call Python marshalling would otherwise show up.
    def plan_gemm(self, w: Weight, x: torch.Tensor, y: torch.Tensor, stream=None):
        m = x.shape[0]
        ws = self.workspace("gemm", self.lib.nvfp4_gemm_workspace_bytes(m, w.n, w.k), x.device)
        cw = w.c()
        args = (ctypes.byref(cw), x.data_ptr(), m, y.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
        fn = self.lib.nvfp4_gemm

        def run():
            st = fn(*args)
            if st:
                raise NVFP4Error("nvfp4_gemm", st)
        run.keep = (cw, ws)
        return run

    def plan_quantize_act(self, x: torch.Tensor, out, stream=None):
        """nvfp4_quantize_act as a zero-argument callable into `out` = (codes, scales, g)."""
        m, k = x.shape
        ws = self.workspace("quantize_act", max(16, self.lib.nvfp4_quantize_workspace_bytes(m)), x.device)
        args = (x.data_ptr(), m, k, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr(), ws.data_ptr(),
                ws.numel(), _stream(stream))
        fn = self.lib.nvfp4_quantize_act

        def run():
            st = fn(*args)
            if st:
                raise NVFP4Error("nvfp4_quantize_act", st)
        run.keep = (ws,)
        return run

    def plan_gemm_w4a4(self, w: Weight, xq, y: torch.Tensor, stream=None):
        codes, scales, g = xq
        m = codes.shape[0]
        ws = self.workspace("gemm", self.lib.nvfp4_gemm_workspace_bytes(m, w.n, w.k), codes.device)
        cw = w.c()
        args = (ctypes.byref(cw), codes.data_ptr(), scales.data_ptr(), g.data_ptr(), m, y.data_ptr(), ws.data_ptr(),
                ws.numel(), _stream(stream))
        fn = self.lib.nvfp4_gemm_w4a4

        def run():
            st = fn(*args)
            if st:
                raise NVFP4Error("nvfp4_gemm_w4a4", st)
        run.keep = (cw, ws)
        return run

    def plan_lm_head_w4a4(self, w: Weight, xq, max_logit: torch.Tensor, argmax: torch.Tensor, stream=None):
        codes, scales, g = xq
        m = codes.shape[0]
        ws = self.workspace("lm_head", self.lib.lm_head_workspace_bytes(m, w.n), codes.device)
        cw = w.c()
        args = (ctypes.byref(cw), codes.data_ptr(), scales.data_ptr(), g.data_ptr(), m, max_logit.data_ptr(),
                argmax.data_ptr(), ws.data_ptr(), ws.numel(), _stream(stream))
        fn = self.lib.lm_head_argmax_w4a4

        def run():
            st = fn(*args)
            if st:
                raise NVFP4Error("lm_head_argmax_w4a4", st)
        run.keep = (cw, ws)
        return run

    def plan_lm_head(self, w: Weight, x: torch.Tensor, max_logit: torch.Tensor, argmax: torch.Tensor, stream=None):
        m = x.shape[0]
        ws = self.workspace("lm_head", self.lib.lm_head_workspace_bytes(m, w.n), x.device)
        cw = w.c()
        args = (ctypes.byref(cw), x.data_ptr(), m, max_logit.data_ptr(), argmax.data_ptr(), ws.data_ptr(),
                ws.numel(), _stream(stream))
        fn = self.lib.lm_head_argmax

        def run():
            st = fn(*args)
            if st:
                raise NVFP4Error("lm_head_argmax", st)
        run.keep = (cw, ws)
        return run

    def moe_forward(self, x, logits, top_k, gate_up: Weight, down: Weight, shared_gate_up: Weight = None,
                    shared_down: Weight = None, route_out=None, out=None, stream=None, softmax_all: bool = False,
                    expert_scale: torch.Tensor = None):
        """The MoE layer in one C call (router + grouped FFN): returns (out, (ids, probs, offsets, pairs))."""
        m, d = x.shape
        e = logits.shape[1]
        dev = x.device
        if route_out is None:
            route_out = (torch.empty((m, top_k), dtype=torch.int32, device=dev),
                         torch.empty((m, top_k), dtype=torch.float32, device=dev),
                         torch.empty((e + 1,), dtype=torch.int32, device=dev),
                         torch.empty((m * top_k,), dtype=torch.int32, device=dev))
        if out is None:
            out = torch.empty((m, d), dtype=torch.bfloat16, device=dev)
        ws = self.workspace("moe", self.lib.moe_ffn_workspace_bytes(m, top_k, gate_up.num_matrices, d, down.k), dev)
        cg, cd = gate_up.c(), down.c()
        sg = shared_gate_up.c() if shared_gate_up is not None else None
        sd = shared_down.c() if shared_down is not None else None
        ids, probs, offsets, pairs = route_out
        self._check("moe_forward", self.lib.moe_forward(
            x.data_ptr(), logits.data_ptr(), m, top_k, NVFP4_ROUTE_SOFTMAX_ALL if softmax_all else 0,
            _ptr(expert_scale), ids.data_ptr(), probs.data_ptr(), offsets.data_ptr(), pairs.data_ptr(),
            ctypes.byref(cg), ctypes.byref(cd), ctypes.byref(sg) if sg is not None else None,
            ctypes.byref(sd) if sd is not None else None, out.data_ptr(), ws.data_ptr(), ws.numel(),
            _stream(stream)))
        return out, route_out

    def plan_moe(self, x, logits, top_k, gate_up: Weight, down: Weight, shared_gate_up: Weight, shared_down: Weight,
                 route_out, out, stream=None):
        """The MoE layer (moe_forward: router + grouped FFN in one C call) as a zero-argument callable."""
        m, d = x.shape
        e = logits.shape[1]
        ids, probs, offsets, pairs = route_out
        ws = self.workspace("moe", self.lib.moe_ffn_workspace_bytes(m, top_k, gate_up.num_matrices, d, down.k),
                            x.device)
        cg, cd = gate_up.c(), down.c()
        sg = shared_gate_up.c() if shared_gate_up is not None else None
        sd = shared_down.c() if shared_down is not None else None
        s = _stream(stream)
        args = (x.data_ptr(), logits.data_ptr(), m, top_k, 0, None, ids.data_ptr(), probs.data_ptr(),
                offsets.data_ptr(), pairs.data_ptr(), ctypes.byref(cg), ctypes.byref(cd),
                ctypes.byref(sg) if sg is not None else None, ctypes.byref(sd) if sd is not None else None,
                out.data_ptr(), ws.data_ptr(), ws.numel(), s)
        fn = self.lib.moe_forward

        def run():
            st = fn(*args)
            if st:
                raise NVFP4Error("moe_forward", st)
        run.keep = (cg, cd, sg, sd, ws)
        return run


_LIB = None


def load(path: str = LIB) -> Library:
    global _LIB
    if _LIB is None or _LIB.path != path:
        _LIB = Library(path)
    return _LIB
