"""Thin ctypes binding of libtq (include/tq.h) for PyTorch tensors.

Argument marshalling only: every step of encode, query preparation, scoring
and top-k runs in the library's CUDA kernels.  Tensors are passed as raw
device pointers with the caller's current CUDA stream.  If the shared
library is missing this module raises at load time; there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtq.so")

TQ_F32, TQ_BF16, TQ_F16 = 0, 1, 2
ROTATIONS = {"auto": 0, "hadamard": 1, "haar": 2}
STATUS = {0: "ok", 1: "invalid argument", 2: "unsupported configuration",
          3: "misaligned pointer or leading dimension", 4: "out of memory",
          5: "CUDA error", 6: "workspace missing or too small",
          7: "request exceeds the fixed internal scratch buffer",
          8: "a kernel gave up a bounded wait; the outputs of that call are not valid"}

_lib = None


class TQError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} failed: {STATUS.get(code, code)} (status {code})")
        self.code = code


class _Info(ctypes.Structure):
    _fields_ = [("d", ctypes.c_int), ("b", ctypes.c_int), ("w", ctypes.c_int), ("m", ctypes.c_int),
                ("rotation", ctypes.c_int), ("device", ctypes.c_int), ("seed", ctypes.c_uint64),
                ("code_bytes", ctypes.c_size_t), ("sign_bytes", ctypes.c_size_t),
                ("coord_mse", ctypes.c_double)]


class _Rows(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("signs", ctypes.c_void_p), ("norms", ctypes.c_void_p)]


def lib() -> ctypes.CDLL:
    """Load libtq.so from the package directory (raises if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libtq.so not built at {LIB_PATH}; run "
                          "`python online_vector_quantization_tq_b200/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, u64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t
    rows = ctypes.POINTER(_Rows)
    sigs = {
        "tq_status_string": (ctypes.c_char_p, [i32]),
        "tq_codebook": (i32, [i32, i32, i32, u64, i32, ctypes.POINTER(vp)]),
        "tq_codebook_host": (i32, [i32, i32, i32, u64, i32, ctypes.POINTER(vp)]),
        "tq_codebook_mse": (i32, [i32, i32, u64, i32, ctypes.POINTER(vp)]),
        "tq_codebook_mse_host": (i32, [i32, i32, u64, i32, ctypes.POINTER(vp)]),
        "tq_destroy": (None, [vp]),
        "tq_info": (i32, [vp, ctypes.POINTER(_Info)]),
        "tq_code_bytes": (sz, [vp]),
        "tq_set_qjl_onthefly": (i32, [vp, i32]),
        "tq_attend_workspace_bytes": (sz, [vp, i64, i64, i64]),
        "tq_attend": (i32, [vp, vp, i64, i64, i64, ctypes.c_float, vp, vp, i64, i64, i64, vp, i64, vp, sz, vp]),
        "tq_attend_prompt": (i32, [vp, i32, vp, i64, vp, i64, vp, i64, i64, vp, i64, i64, i64, ctypes.c_float, vp, i64,
                                   vp]),
        "tq_paged_store": (i32, [vp, vp, rows, rows, vp, i64, i64, rows, rows, i64, i32, vp]),
        "tq_attend_paged_workspace_bytes": (sz, [vp, vp, i64, i64, i64, i64, i64, i64, i32]),
        "tq_attend_paged": (i32, [vp, vp, i32, vp, i64, i64, vp, i64, i64, i64, i64, rows, rows, i64, i32, vp, i64,
                                  i64, vp, ctypes.c_float, vp, i64, vp, sz, vp]),
        "tq_qjl_matrix": (i32, [vp, vp, vp]),
        "tq_codebook_get": (i32, [vp, vp, vp, vp]),
        "tq_tables_get": (i32, [vp, vp, vp, vp]),
        "tq_encode": (i32, [vp, vp, i32, i64, i64, vp, i64, vp, vp, vp, i64, vp]),
        "tq_encode_workspace_bytes": (sz, [vp, i64]),
        "tq_encode_ws": (i32, [vp, vp, i32, i64, i64, vp, i64, vp, vp, vp, i64, vp, sz, vp]),
        "tq_prepare_queries": (i32, [vp, vp, i64, i64, vp, i64, vp, vp, vp]),
        "tq_score_workspace_bytes": (sz, [vp, i64]),
        "tq_score": (i32, [vp, vp, i64, i64, i64, vp, vp, vp, vp, i64, vp, i32, vp, sz, vp]),
        "tq_score_prepare": (i32, [vp, vp, i64, i64, i64, vp, vp, sz, vp]),
        "tq_score_prepared": (i32, [vp, i64, i64, vp, vp, vp, i64, vp, i32, vp, sz, vp]),
        "tq_topk_workspace_bytes": (sz, [vp, i64, i64, i32]),
        "tq_topk": (i32, [vp, vp, i64, i64, vp, vp, vp, i64, i32, vp, vp, vp, sz, vp]),
        "tq_score_noalloc": (i32, [vp, vp, i64, i64, i64, vp, vp, vp, vp, i64, vp, i32, vp]),
        "tq_rerank": (i32, [vp, i64, i64, vp, i32, i64, i64, i32, vp, i32, i32, vp, vp, vp]),
        "tq_outlier_workspace_bytes": (sz, [i64, i32]),
        "tq_outlier_channels": (i32, [vp, i32, i64, i64, i32, i64, i32, vp, vp, vp, sz, vp]),
        "tq_sync_check": (i32, [vp, vp]),
        "tq_selftest_timeout": (i32, [vp, vp]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(fn: str, code: int):
    if code != 0:
        raise TQError(fn, code)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype(x: torch.Tensor) -> int:
    if x.dtype == torch.float32:
        return TQ_F32
    if x.dtype == torch.bfloat16:
        return TQ_BF16
    raise TypeError(f"unsupported dtype {x.dtype}")


def _ld(x: torch.Tensor) -> int:
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with unit stride in the last dimension")
    return x.stride(0)


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A result that a call on `stream` writes.  torch hands memory out, and
    takes it back, in the order of one stream: what another than the current
    one writes has to come from its own memory, and the current one, whose
    tensor it looks like to the caller, has to be done with it before it is
    reused."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(t.device))
    return t


def _like(y: torch.Tensor, stream) -> torch.Tensor:
    """_empty of y's shape and type, in half the host's time where it is the current stream's."""
    if stream is None:
        return torch.empty_like(y, memory_format=torch.contiguous_format)
    return _empty(y.shape, y.dtype, y.device, stream)


def _workspace(nbytes: int, device, stream=None) -> torch.Tensor:
    """Scratch of a call on `stream`, from that stream's memory (see _empty)."""
    n = max(int(nbytes), 16)
    if stream is None:
        return torch.empty(n, dtype=torch.uint8, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=torch.uint8, device=device)


@dataclass
class Encoded:
    codes: torch.Tensor   # uint8 [n, code_bytes]
    signs: torch.Tensor   # uint8 [n, sign_bytes]
    norms: torch.Tensor   # float32 [n, 2]: ||x||, gamma

    def check(self):
        """The library reads and writes whole packed rows back to back: every
        array must be row-contiguous (a strided view would be read as if it
        were not)."""
        for name in ("codes", "signs", "norms"):
            t = getattr(self, name)
            if t.numel() and not t.is_contiguous():
                raise ValueError(f"Encoded.{name} must be contiguous (got strides {t.stride()})")
        return self


def _packed(name: str, t: torch.Tensor, dtype, shape: tuple):
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {shape} (got {t.dtype} {tuple(t.shape)})")
    if not t.is_contiguous() and t.numel():
        raise ValueError(f"{name} must be contiguous (got strides {t.stride()})")


@dataclass
class PagedCache:
    """Packed rows of a cache's keys, or of its values, in pages (include/tq.h:
    tq_rows).  Page p holds page_size tokens of every KV head."""
    codes: torch.Tensor   # uint8 [npages, kv_heads, page_size, code_bytes]
    signs: torch.Tensor   # uint8 [npages, kv_heads, page_size, sign_bytes]
    norms: torch.Tensor   # float32 [npages, kv_heads, page_size, 2]

    def check(self, q: "Quantizer"):
        """Shapes, types and contiguity that the library relies on: it reads and
        writes whole rows of q's quantizer."""
        if self.codes.dim() != 4:
            raise ValueError(f"PagedCache.codes must have 4 dimensions (got {self.codes.dim()})")
        lead = self.codes.shape[:3]
        _packed("PagedCache.codes", self.codes, torch.uint8, (*lead, q.code_bytes))
        if q.sign_bytes or self.signs is not None:
            _packed("PagedCache.signs", self.signs, torch.uint8, (*lead, q.sign_bytes))
        _packed("PagedCache.norms", self.norms, torch.float32, (*lead, 2))
        return self


class Quantizer:
    """Owned tq_quantizer handle."""

    def __init__(self, handle: ctypes.c_void_p):
        self._h = handle
        info = _Info()
        _check("tq_info", lib().tq_info(self._h, ctypes.byref(info)))
        self.d, self.b, self.w, self.m = info.d, info.b, info.w, info.m
        self.rotation = {1: "hadamard", 2: "haar"}[info.rotation]
        self.device_index = info.device
        self.seed = info.seed
        self.code_bytes, self.sign_bytes = info.code_bytes, info.sign_bytes
        self.coord_mse = info.coord_mse

    @property
    def handle(self):
        return self._h

    def close(self):
        if self._h:
            lib().tq_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def codebook(self):
        import numpy as np
        L = 1 << self.w
        c = np.zeros(L)
        t = np.zeros(L - 1)
        mse = ctypes.c_double()
        _check("tq_codebook_get", lib().tq_codebook_get(
            self._h, c.ctypes.data_as(ctypes.c_void_p), t.ctypes.data_as(ctypes.c_void_p), ctypes.byref(mse)))
        return c, t, mse.value

    def tables(self):
        """(R fp32 [d,d], diagonal signs int8 [3,d] or None, S fp16 bits uint16 [m,d])."""
        import numpy as np
        r = np.zeros((self.d, self.d), dtype=np.float32)
        diag = np.zeros((3, self.d), dtype=np.int8)
        s = np.zeros((self.m, self.d), dtype=np.uint16)
        _check("tq_tables_get", lib().tq_tables_get(
            self._h, r.ctypes.data_as(ctypes.c_void_p), diag.ctypes.data_as(ctypes.c_void_p),
            s.ctypes.data_as(ctypes.c_void_p)))
        return r, (diag if self.rotation == "hadamard" else None), s

    def empty_encoded(self, n: int, device="cuda", stream=None) -> Encoded:
        return Encoded(_empty((n, self.code_bytes), torch.uint8, device, stream),
                       _empty((n, self.sign_bytes), torch.uint8, device, stream),
                       _empty((n, 2), torch.float32, device, stream))

    def empty_paged(self, npages: int, kv_heads: int, page_size: int, device="cuda") -> PagedCache:
        lead = (npages, kv_heads, page_size)
        return PagedCache(torch.empty(lead + (self.code_bytes,), dtype=torch.uint8, device=device),
                          torch.empty(lead + (self.sign_bytes,), dtype=torch.uint8, device=device),
                          torch.empty(lead + (2,), dtype=torch.float32, device=device))


def tq_codebook(d: int, b: int, m: int = 0, seed: int = 0, rotation: str = "auto") -> Quantizer:
    h = ctypes.c_void_p()
    _check("tq_codebook", lib().tq_codebook(d, b, m, seed, ROTATIONS[rotation], ctypes.byref(h)))
    return Quantizer(h)


def tq_codebook_host(d: int, b: int, m: int = 0, seed: int = 0, rotation: str = "auto") -> Quantizer:
    h = ctypes.c_void_p()
    _check("tq_codebook_host", lib().tq_codebook_host(d, b, m, seed, ROTATIONS[rotation], ctypes.byref(h)))
    return Quantizer(h)


def tq_codebook_mse(d: int, b: int, seed: int = 0, rotation: str = "auto") -> Quantizer:
    """TurboQuant-MSE quantizer: all b bits to the codebook, no QJL sign bits."""
    h = ctypes.c_void_p()
    _check("tq_codebook_mse", lib().tq_codebook_mse(d, b, seed, ROTATIONS[rotation], ctypes.byref(h)))
    return Quantizer(h)


def tq_codebook_mse_host(d: int, b: int, seed: int = 0, rotation: str = "auto") -> Quantizer:
    h = ctypes.c_void_p()
    _check("tq_codebook_mse_host", lib().tq_codebook_mse_host(d, b, seed, ROTATIONS[rotation], ctypes.byref(h)))
    return Quantizer(h)


def tq_encode(q: Quantizer, x: torch.Tensor, out: Encoded | None = None, chan: torch.Tensor | None = None,
              chan_rows: int = 0, out_stride: int = 1, workspace: torch.Tensor | None = None,
              stream=None) -> Encoded:
    n = x.shape[0]
    if out is None:
        out = q.empty_encoded(n, x.device, stream)
    out.check()
    if chan is not None and chan.dtype != torch.int32:
        raise TypeError("chan must be int32")
    L = lib()
    args = (q.handle, _ptr(x), _dtype(x), n, _ld(x), _ptr(chan), chan_rows,
            _ptr(out.codes), _ptr(out.signs), _ptr(out.norms), out_stride)
    if workspace is None:
        ws = L.tq_encode_workspace_bytes(q.handle, n)
        if ws:
            workspace = _workspace(ws, x.device, stream)
    if workspace is None:
        _check("tq_encode", L.tq_encode(*args, _stream(stream)))
    else:
        _check("tq_encode_ws", L.tq_encode_ws(*args, _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


def tq_prepare_queries(q: Quantizer, y: torch.Tensor, ychan: torch.Tensor | None = None, ychan_rows: int = 0,
                       stream=None):
    nq = y.shape[0]
    ytil = _empty((nq, q.d), torch.float32, y.device, stream)
    p = _empty((nq, q.m), torch.float32, y.device, stream)
    _check("tq_prepare_queries", lib().tq_prepare_queries(
        q.handle, _ptr(y), nq, _ld(y), _ptr(ychan), ychan_rows, _ptr(ytil), _ptr(p), _stream(stream)))
    return ytil, p


def score_workspace(q: Quantizer, nq: int, device="cuda") -> torch.Tensor:
    return _workspace(lib().tq_score_workspace_bytes(q.handle, nq), device)


def tq_score(q: Quantizer, y: torch.Tensor, groups: int, G: int, enc: Encoded, keys_per_group: int,
             out: torch.Tensor | None = None, accumulate: bool = False, ychan: torch.Tensor | None = None,
             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    enc.check()
    if out is None:
        out = _empty((groups * G, keys_per_group), torch.float32, y.device, stream)
    if workspace is None:
        workspace = _workspace(lib().tq_score_workspace_bytes(q.handle, groups * G), y.device, stream)
    _check("tq_score", lib().tq_score(
        q.handle, _ptr(y), groups, G, _ld(y), _ptr(ychan), _ptr(enc.codes), _ptr(enc.signs), _ptr(enc.norms),
        keys_per_group, _ptr(out), int(bool(accumulate)), _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


def tq_score_prepare(q: Quantizer, y: torch.Tensor, groups: int, G: int, workspace: torch.Tensor | None = None,
                     ychan: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Query half of tq_score: writes the prepared queries into `workspace`
    (allocated when None) and returns it, for tq_score_prepared."""
    if workspace is None:
        nbytes = max(lib().tq_score_workspace_bytes(q.handle, groups * G), 16)
        workspace = _empty(nbytes, torch.uint8, y.device, stream)
    _check("tq_score_prepare", lib().tq_score_prepare(
        q.handle, _ptr(y), groups, G, _ld(y), _ptr(ychan), _ptr(workspace), workspace.numel(), _stream(stream)))
    return workspace


def tq_score_prepared(q: Quantizer, groups: int, G: int, enc: Encoded, keys_per_group: int,
                      workspace: torch.Tensor, out: torch.Tensor | None = None, accumulate: bool = False,
                      stream=None) -> torch.Tensor:
    """Key half of tq_score against the queries tq_score_prepare wrote into
    `workspace`."""
    enc.check()
    if out is None:
        out = _empty((groups * G, keys_per_group), torch.float32, enc.codes.device, stream)
    _check("tq_score_prepared", lib().tq_score_prepared(
        q.handle, groups, G, _ptr(enc.codes), _ptr(enc.signs), _ptr(enc.norms), keys_per_group, _ptr(out),
        int(bool(accumulate)), _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


def topk_workspace(q: Quantizer, nq: int, n: int, k: int, device="cuda") -> torch.Tensor:
    return _workspace(lib().tq_topk_workspace_bytes(q.handle, nq, n, k), device)


def tq_topk(q: Quantizer, y: torch.Tensor, enc: Encoded, k: int, n: int | None = None,
            workspace: torch.Tensor | None = None, out=None, stream=None):
    """(scores fp32 [nq, k], key indices int64 [nq, k]); `out` may give both."""
    nq = y.shape[0]
    enc.check()
    n = enc.codes.shape[0] if n is None else n
    if out is None:
        vals = _empty((nq, k), torch.float32, y.device, stream)
        idx = _empty((nq, k), torch.int64, y.device, stream)
    else:
        vals, idx = out
    if workspace is None:
        workspace = _workspace(lib().tq_topk_workspace_bytes(q.handle, nq, n, k), y.device, stream)
    _check("tq_topk", lib().tq_topk(
        q.handle, _ptr(y), nq, _ld(y), _ptr(enc.codes), _ptr(enc.signs), _ptr(enc.norms), n, k,
        _ptr(vals), _ptr(idx), _ptr(workspace), workspace.numel(), _stream(stream)))
    return vals, idx


def tq_attend(qv: Quantizer, logits: torch.Tensor, groups: int, G: int, venc: Encoded, keys_per_group: int,
              scale: float, key_base: int = 0, nkeys: int | None = None, out: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Attention over a quantized KV cache: softmax(scale * logits) times the
    TurboQuant-MSE reconstructions of the values (venc, encoded by qv), one
    row of d floats per query (groups*G rows)."""
    venc.check()
    n = keys_per_group - key_base if nkeys is None else nkeys
    if out is None:
        out = _empty((groups * G, qv.d), torch.float32, logits.device, stream)
    if workspace is None:
        workspace = _workspace(lib().tq_attend_workspace_bytes(qv.handle, groups, G, n), logits.device, stream)
    _check("tq_attend", lib().tq_attend(
        qv.handle, _ptr(logits), _ld(logits), groups, G, float(scale), _ptr(venc.codes),
        _ptr(venc.norms), keys_per_group, key_base, n, _ptr(out), _ld(out), _ptr(workspace), workspace.numel(),
        _stream(stream)))
    return out


def _dtype16(x: torch.Tensor) -> int:
    if x.dtype == torch.bfloat16:
        return TQ_BF16
    if x.dtype == torch.float16:
        return TQ_F16
    raise TypeError(f"unsupported dtype {x.dtype}")


def _ld_rows(x: torch.Tensor) -> int:
    """_ld, but a single row's stride (which torch leaves open) does not count."""
    if x.shape[0] == 1 and x.dim() == 2:
        if x.stride(1) == 1 or x.shape[1] <= 1:
            return x.shape[1]
    return _ld(x)


def _rows(t) -> _Rows:
    signs = t.signs
    return _Rows(t.codes.data_ptr(), 0 if signs is None else signs.data_ptr(), t.norms.data_ptr())


def _one_device(q: Quantizer, names: str, *tensors) -> int:
    """The device of the tensors (None among them passes), which has to be a
    CUDA device, the same for all that are not empty, and the quantizer's."""
    found = -1
    for i, t in enumerate(tensors):
        if t is None:
            continue
        dev = t.get_device()
        if (dev != found or dev < 0) and t.numel():
            if dev < 0 or found >= 0:
                raise ValueError(f"{names.split()[i]} must be a CUDA tensor" + (f" of device {found}" if found >= 0 else ""))
            found = dev
    if found >= 0 and found != q.device_index and q.device_index >= 0:
        raise ValueError(f"the tensors are on device {found}, the quantizer on device {q.device_index}")
    return found


def _raw_stream(stream, device: int):
    """`stream`, or the current one of the tensors' device."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device) if device >= 0 else None


def _vector(t: torch.Tensor, dtype, name: str, length: int | None = None) -> torch.Tensor:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if t.dim() != 1 or not t.is_contiguous() or (length is not None and t.numel() != length):
        raise ValueError(f"{name} must be a contiguous 1-D tensor" + ("" if length is None else f" of {length}"))
    return t


def _check_caches(qk: Quantizer, qv: Quantizer, kcache: PagedCache, vcache: PagedCache):
    """(npages, kv_heads, page_size) that both arrays agree on."""
    kcache.check(qk)
    vcache.check(qv)
    lead = kcache.codes.shape[:3]
    if lead != vcache.codes.shape[:3]:
        raise ValueError("kcache and vcache must have the same pages, KV heads and page size")
    if kcache.codes.get_device() < 0 and kcache.codes.numel():
        raise ValueError("kcache must be CUDA tensors")
    return lead


def tq_attend_prompt(q: Quantizer, y: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     scale: float, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Causal attention of packed prompts on raw rows: y [tokens, heads*d], k
    and v [tokens, kv_heads*d] (bf16 or fp16; views of one projection's output
    will do), sequence i the tokens cu_seqlens[i] to cu_seqlens[i+1] (int32).
    q, any quantizer, gives d and the device.  Rows of out for tokens of no
    sequence are not written."""
    if y.dim() != 2 or k.dim() != 2 or k.shape != v.shape or k.shape[0] != y.shape[0]:
        raise ValueError("y, k and v must be 2-D with the same tokens, k and v of one shape")
    (total, wide), narrow, d, dtype = y.shape, k.shape[1], q.d, y.dtype
    if narrow == 0 or narrow % d != 0 or wide == 0 or wide % narrow != 0:
        raise ValueError(f"y must have a whole number of heads of {d} for each KV head of k and v")
    if k.dtype != dtype or v.dtype != dtype:
        raise TypeError("y, k and v must have one type")
    _vector(cu_seqlens, torch.int32, "cu_seqlens")
    nseq = cu_seqlens.shape[0] - 1
    if nseq < 0:
        raise ValueError("cu_seqlens must have one entry more than there are sequences")
    if out is None:
        out = _like(y, stream)
    elif out.dtype != dtype or out.shape != y.shape:
        raise ValueError("out must have y's shape and type")
    device = _one_device(q, "y k v cu_seqlens out", y, k, v, cu_seqlens, out)
    _check("tq_attend_prompt", lib().tq_attend_prompt(
        q.handle, _dtype16(y), y.data_ptr(), _ld_rows(y), k.data_ptr(), _ld_rows(k), v.data_ptr(), _ld_rows(v), total,
        cu_seqlens.data_ptr(), nseq, wide // d, narrow // d, scale, out.data_ptr(), _ld_rows(out),
        _raw_stream(stream, device)))
    return out


def tq_paged_store(qk: Quantizer, qv: Quantizer, kenc: Encoded, venc: Encoded, slots: torch.Tensor,
                   kcache: PagedCache, vcache: PagedCache, stream=None) -> None:
    """Store encoded keys and values of new tokens (row t*kv_heads + h: token
    t, head h) into the pages, token t at slot slots[t] = page*page_size +
    offset (int64; a slot outside the cache stores nothing)."""
    npages, kv_heads, page_size = _check_caches(qk, qv, kcache, vcache)
    _vector(slots, torch.int64, "slots")
    tokens = slots.shape[0]
    n = tokens * kv_heads
    for q, e, name in ((qk, kenc, "kenc"), (qv, venc, "venc")):
        _packed(name + ".codes", e.codes, torch.uint8, (n, q.code_bytes))
        if q.sign_bytes:
            _packed(name + ".signs", e.signs, torch.uint8, (n, q.sign_bytes))
        _packed(name + ".norms", e.norms, torch.float32, (n, 2))
    device = _one_device(qk, "slots kenc.codes kenc.norms venc.codes venc.norms kcache.codes kcache.norms vcache.codes "
                             "vcache.norms kenc.signs kcache.signs venc.signs vcache.signs", slots, kenc.codes,
                         kenc.norms, venc.codes, venc.norms, kcache.codes, kcache.norms, vcache.codes, vcache.norms,
                         kenc.signs, kcache.signs, venc.signs, vcache.signs)
    _check("tq_paged_store", lib().tq_paged_store(
        qk.handle, qv.handle, _rows(kenc), _rows(venc), slots.data_ptr(), tokens, kv_heads, _rows(kcache),
        _rows(vcache), npages, page_size, _raw_stream(stream, device)))


def attend_paged_workspace(qk: Quantizer, qv: Quantizer, total_q: int, nseq: int, heads: int, kv_heads: int,
                           max_new: int, max_pages: int, page_size: int, device="cuda") -> torch.Tensor:
    return _workspace(lib().tq_attend_paged_workspace_bytes(
        qk.handle, qv.handle, total_q, nseq, heads, kv_heads, max_new, max_pages, page_size), device)


def tq_attend_paged(qk: Quantizer, qv: Quantizer, y: torch.Tensor, q_start: torch.Tensor, kcache: PagedCache,
                    vcache: PagedCache, page_table: torch.Tensor, kv_len: torch.Tensor, max_new: int, scale: float,
                    out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """Causal attention of new tokens over a paged quantized cache: y [tokens,
    heads*d] (bf16 or fp16), sequence i's new tokens q_start[i] to q_start[i+1]
    (at most max_new), its pages page_table[i], its keys kv_len[i] (the new
    tokens' last among them)."""
    npages, kv_heads, page_size = _check_caches(qk, qv, kcache, vcache)
    ldy, d = _ld_rows(y), qk.d
    total_q, wide = y.shape
    if kv_heads == 0 or wide % (d * kv_heads) != 0:
        raise ValueError(f"y must have a whole number of heads of {d} for each of {kv_heads} KV heads")
    heads = wide // d
    _vector(kv_len, torch.int32, "kv_len")
    nseq = kv_len.shape[0]
    _vector(q_start, torch.int32, "q_start", nseq + 1)
    if page_table.dtype != torch.int32 or page_table.dim() != 2 or page_table.shape[0] != nseq:
        raise TypeError(f"page_table must be an int32 tensor of {nseq} rows")
    if out is None:
        out = _like(y, stream)
    elif out.dtype != y.dtype or out.shape != y.shape:
        raise ValueError("out must have y's shape and type")
    max_pages = page_table.shape[1]
    if workspace is None:
        workspace = _workspace(lib().tq_attend_paged_workspace_bytes(
            qk.handle, qv.handle, total_q, nseq, heads, kv_heads, max_new, max_pages, page_size), y.device, stream)
    device = _one_device(qk, "y q_start kv_len page_table out workspace kcache.codes kcache.norms vcache.codes "
                             "vcache.norms kcache.signs", y, q_start, kv_len, page_table, out, workspace, kcache.codes,
                         kcache.norms, vcache.codes, vcache.norms, kcache.signs)
    _check("tq_attend_paged", lib().tq_attend_paged(
        qk.handle, qv.handle, _dtype16(y), y.data_ptr(), ldy, total_q, q_start.data_ptr(), nseq, max_new, heads,
        kv_heads, _rows(kcache), _rows(vcache), npages, page_size, page_table.data_ptr(), _ld_rows(page_table),
        max_pages, kv_len.data_ptr(), scale, out.data_ptr(), _ld_rows(out), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _raw_stream(stream, device)))
    return out


def tq_set_qjl_onthefly(q: Quantizer, enable: bool = True) -> None:
    """Generate the QJL matrix S from the seed inside the kernels that can
    (see include/tq.h) instead of reading the stored table."""
    _check("tq_set_qjl_onthefly", lib().tq_set_qjl_onthefly(q.handle, int(bool(enable))))


def tq_qjl_matrix(q: Quantizer, device="cuda", stream=None) -> torch.Tensor:
    """S (m x d fp16 bit patterns as int16, row-major) generated on the
    device from the quantizer seed."""
    out = _empty((q.m, q.d), torch.int16, device, stream)
    _check("tq_qjl_matrix", lib().tq_qjl_matrix(q.handle, _ptr(out), _stream(stream)))
    return out


def tq_rerank(y: torch.Tensor, x: torch.Tensor, cand: torch.Tensor, k: int, out=None, stream=None):
    """Second stage of two-stage retrieval: exact <y, x> of every candidate
    key (cand: int64 [nq, kc], e.g. tq_topk's indices) against the raw rows
    x, and the k best per query: (scores fp32 [nq, k], keys int64 [nq, k])."""
    nq, kc = cand.shape
    if out is None:
        vals = _empty((nq, k), torch.float32, y.device, stream)
        idx = _empty((nq, k), torch.int64, y.device, stream)
    else:
        vals, idx = out
    if cand.dtype != torch.int64 or not cand.is_contiguous():
        raise TypeError("cand must be a contiguous int64 tensor")
    _check("tq_rerank", lib().tq_rerank(
        _ptr(y), nq, _ld(y), _ptr(x), _dtype(x), x.shape[0], _ld(x), x.shape[1], _ptr(cand), kc, k,
        _ptr(vals), _ptr(idx), _stream(stream)))
    return vals, idx


def tq_outlier_channels(x: torch.Tensor, groups: int, rows_per_group: int, count: int, stream=None):
    """Per group, the `count` highest-mean-square channels and the rest (both
    ascending int32 tensors on x's device)."""
    dim = x.shape[1]
    sel = _empty((groups, count), torch.int32, x.device, stream)
    rest = _empty((groups, dim - count), torch.int32, x.device, stream)
    ws = _workspace(lib().tq_outlier_workspace_bytes(groups, dim), x.device, stream)
    _check("tq_outlier_channels", lib().tq_outlier_channels(
        _ptr(x), _dtype(x), groups, rows_per_group, dim, _ld(x), count, _ptr(sel), _ptr(rest),
        _ptr(ws), ws.numel(), _stream(stream)))
    return sel, rest


def tq_sync_check(q: "Quantizer", stream=None) -> None:
    """Synchronize `stream` and raise TQError (status 8) if a kernel of q gave
    up a bounded wait since the last check (its outputs are not valid)."""
    _check("tq_sync_check", lib().tq_sync_check(q.handle, _stream(stream)))


def tq_selftest_timeout(q: "Quantizer", stream=None) -> None:
    """Launch a kernel whose wait runs out (about 2 s): tests the failure path."""
    _check("tq_selftest_timeout", lib().tq_selftest_timeout(q.handle, _stream(stream)))
