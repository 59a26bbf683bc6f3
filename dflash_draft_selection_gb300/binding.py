"""ctypes binding of libdflash2.so: torch CUDA tensors in, pointers out.

Every function here has the name of the C entry point it calls (without the
``dflash2_`` prefix) and does argument marshalling only: shapes are read from
the tensors, outputs are allocated when not passed in, and the call is made on
the current CUDA stream.  Nothing is computed in Python; if the library cannot
be loaded the call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdflash2.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_WORKSPACE = 0, 1, 2, 3, 4
F32, BF16 = 0, 1
ST_OK, ST_NAN, ST_BAD_Q, ST_BAD_PARAMS, ST_UNSUPPORTED = 0, 1, 2, 3, 4
VERIFY_TRUST_Q = 1
NC = 16
SHARD_LIST = 64

SAMPLING_DTYPE = np.dtype([("temperature", "<f4"), ("top_k", "<i4"), ("top_p", "<f4")])

_lib = None
_lock = threading.Lock()


ATTN_CAUSAL, ATTN_WEIGHTS = 1, 2


class _CacheRecord(ctypes.Structure):
    """dflash2_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("weight", ctypes.c_void_p), ("pos", ctypes.c_void_p),
                ("num_pages", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("slot_stride", ctypes.c_int64), ("Hkv", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("d", ctypes.c_int32), ("dt", ctypes.c_int32)]


class _Weight4Record(ctypes.Structure):
    """dflash2_weight4."""
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("code_stride", ctypes.c_int64),
                ("side_stride", ctypes.c_int64), ("group", ctypes.c_int32), ("side_dt", ctypes.c_int32)]


class DFlash2Error(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn}: {_status_string(code)} (status {code})")


def load_library():
    """Load libdflash2.so (built in-tree by the package's build step)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise OSError(f"{LIB_PATH} is missing: build it with `python -m dflash_draft_selection_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32, u32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
        L.dflash2_topk16_workspace_bytes.argtypes = [i64]
        L.dflash2_topk16_workspace_bytes.restype = sz
        L.dflash2_topk16.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, vp, vp, vp, sz, vp]
        L.dflash2_topk16_noalloc.argtypes = [vp, i32, i64, i64, i64, vp, i64, vp, vp, vp, vp]
        L.dflash2_topk16_shard.argtypes = [vp, i32, i64, i64, i64, i64, i64, vp, i64, vp, vp, vp, vp, vp, sz, vp]
        L.dflash2_topk16_merge.argtypes = [i32, i64, vp, vp, vp, vp, i64, vp, i64, vp, vp, vp, vp]
        L.dflash2_lmhead_topk16_workspace_bytes.argtypes = [i64, i64]
        L.dflash2_lmhead_topk16_workspace_bytes.restype = sz
        L.dflash2_lmhead_topk16.argtypes = [vp, vp, i64, i64, i64, vp, i64, vp, vp, vp, vp, sz, vp]
        L.dflash2_ctx_gate.argtypes = [vp, i32, i64, i64, vp, i32, vp, vp]
        L.dflash2_pair_score_walk.argtypes = [i64, i32, vp, vp, vp, vp, vp, i32, i64, i32, vp, vp, vp, vp, vp,
                                              vp, vp, vp]
        L.dflash2_verify_workspace_bytes.argtypes = [i64, i32]
        L.dflash2_verify_workspace_bytes.restype = sz
        L.dflash2_verify.argtypes = [vp, i32, i64, i32, i64, i64, vp, vp, vp, vp, vp, vp, vp, u32, vp, vp, vp,
                                     vp, sz, vp]
        L.dflash2_conv2tap.argtypes = [vp, vp, vp, vp, i32, i64, i32, i64, i32, vp, vp]
        L.dflash2_dynconv2tap.argtypes = [vp, vp, vp, i32, i64, i32, i64, i32, vp, vp, vp]
        f32 = ctypes.c_float
        L.dflash2_rope_append.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, i32, vp, i64,
                                          i32, vp, i32, vp, i32, vp, vp, f32, vp, vp, vp]
        L.dflash2_paged_attn_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i32]
        L.dflash2_paged_attn_workspace_bytes.restype = sz
        L.dflash2_paged_attn.argtypes = [vp, vp, i32, vp, vp, vp, vp, i64, i32, i32, f32, i32, u32, vp, vp, vp, sz,
                                         vp]
        L.dflash2_kv_evict_workspace_bytes.argtypes = [i64, i32, i64, i32]
        L.dflash2_kv_evict_workspace_bytes.restype = sz
        L.dflash2_kv_evict.argtypes = [vp, vp, i32, vp, vp, i64, i32, i32, i32, vp, vp, sz, vp]
        L.dflash2_quant4.argtypes = [vp, i32, i64, vp, vp]
        L.dflash2_dequant4.argtypes = [vp, vp, i32, i64, vp]
        L.dflash2_linear4_workspace_bytes.argtypes = [i32, i64, i64, i64]
        L.dflash2_linear4_workspace_bytes.restype = sz
        L.dflash2_linear4.argtypes = [vp, i32, i64, i64, vp, vp, i32, i64, vp, sz, vp]
        L.dflash2_linear4_rounded.argtypes = L.dflash2_linear4.argtypes
        L.dflash2_sample.argtypes = [vp, i32, i64, i64, i64, vp, vp, i64, vp, vp, vp, vp]
        L.dflash2_status_string.argtypes = [i32]
        L.dflash2_status_string.restype = ctypes.c_char_p
        L.dflash2_device_error.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
        L.dflash2_test_hold.argtypes = [vp, i64]
        for fn in ("dflash2_topk16", "dflash2_topk16_noalloc", "dflash2_topk16_shard", "dflash2_topk16_merge",
                   "dflash2_lmhead_topk16",
                   "dflash2_ctx_gate", "dflash2_pair_score_walk",
                   "dflash2_verify", "dflash2_conv2tap", "dflash2_dynconv2tap", "dflash2_device_error",
                   "dflash2_test_hold", "dflash2_rope_append", "dflash2_paged_attn", "dflash2_kv_evict",
                   "dflash2_quant4", "dflash2_dequant4", "dflash2_linear4", "dflash2_linear4_rounded", "dflash2_sample"):
            getattr(L, fn).restype = i32
        _lib = L
        return _lib


def _status_string(code: int) -> str:
    try:
        return load_library().dflash2_status_string(code).decode()
    except OSError:
        return "library not loaded"


def _check(fn: str, code: int):
    if code != OK:
        raise DFlash2Error(fn, code)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return BF16
    if dt == torch.float32:
        return F32
    raise TypeError(f"unsupported dtype {dt}")


def _here(cache, what: str = "cache") -> int:
    """The index of a cache's (or weights') device, which has to be the current one: a call launches there."""
    dev = cache._dev
    if torch._C._cuda_getDevice() != dev:
        raise ValueError(f"the {what} lies on cuda:{dev}, which is not the current device")
    return dev


def _int32(B: int, name: str, t, dev: int):
    """A per-request array: contiguous int32 [B] on GPU `dev` (None passes).  Returns its address."""
    if t is None:
        return None
    if t.dtype is not torch.int32 or t.shape != (B,) or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: contiguous int32 [{B}] on the cache's GPU")
    return t.data_ptr()


def _page_table(t: torch.Tensor, B: int, dev: int):
    """Address and pages per request of a page table."""
    shape = t.shape
    if t.dtype is not torch.int32 or len(shape) != 2 or shape[0] != B or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"page_table: contiguous int32 [{B}, pages] on the cache's GPU")
    return t.data_ptr(), shape[1]


def _heads(name: str, t: torch.Tensor, dt, B: int, T: int, H: int, d: int, dev: int):
    """Address and token stride of [B, T, H, d] with contiguous heads and one stride from token to token."""
    if t.dtype is not dt or t.shape != (B, T, H, d) or t.get_device() != dev:
        raise ValueError(f"{name}: {dt} [{B}, {T}, {H}, {d}] on the cache's GPU")
    s0, s1, s2, s3 = t.stride()
    if (s3 != 1 and d > 1) or (s2 != d and H > 1) or (B > 1 and T > 1 and s0 != T * s1):
        raise ValueError(f"{name}: contiguous heads and one stride from token to token")
    return t.data_ptr(), s1 if T > 1 else (s0 if B > 1 else H * d)


def _dense(name: str, t, dt, shape, dev: int, owner: str = "cache"):
    """Address of a contiguous tensor of a type and shape on GPU `dev` (None passes)."""
    if t is None:
        return None
    if t.dtype is not dt or t.shape != shape or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: contiguous {dt} {list(shape)} on the {owner}'s GPU")
    return t.data_ptr()


def _count(name: str, n: int) -> int:
    """A number that C takes in 32 bits (ctypes would drop the others)."""
    if not -2 ** 31 <= n < 2 ** 31:
        raise ValueError(f"{name}: {n} does not fit 32 bits")
    return n


def _scratch(ws, dev: int):
    """Address and size of a workspace."""
    if ws.buf.get_device() != dev:
        raise ValueError("ws: a workspace on the GPU of the other tensors")
    return ws.buf.data_ptr(), ws.buf.numel()


def _raw_stream(dev: int) -> int:
    """The current stream of a device as a number (torch.cuda.current_stream without its object)."""
    return torch._C._cuda_getCurrentRawStream(dev)


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("dflash2 tensors must be CUDA tensors")


def sampling_params(temperature, top_k, top_p, n: int | None = None, device="cuda") -> torch.Tensor:
    """Pack per-request sampling parameters into the C record layout (12 bytes each) on `device`."""
    if n is None:
        n = np.broadcast(np.asarray(temperature), np.asarray(top_k), np.asarray(top_p)).size
    rec = np.zeros(n, dtype=SAMPLING_DTYPE)
    rec["temperature"] = temperature
    rec["top_k"] = top_k
    rec["top_p"] = top_p
    return torch.from_numpy(rec.view(np.uint8).copy()).to(device)


def _params_from(params, device):
    if params is None or isinstance(params, torch.Tensor):
        return params
    rec = np.ascontiguousarray(np.asarray(params, dtype=SAMPLING_DTYPE))
    return torch.from_numpy(rec.view(np.uint8).copy()).to(device)


class Workspace:
    """A zero-filled device workspace, reusable across calls of one kind: for one entry point and set of sizes, or for
    calls of paged_attn and kv_evict of any sizes that fit.  What a call needs zero it leaves zero; ``buf.zero_()``
    before the workspace goes to another kind of call."""

    def __init__(self, nbytes: int, device="cuda"):
        self.buf = torch.zeros(max(int(nbytes), 16), dtype=torch.uint8, device=device)

    @property
    def nbytes(self) -> int:
        return self.buf.numel()

    def ptr(self):
        return ctypes.c_void_p(self.buf.data_ptr())

    @staticmethod
    def for_topk16(rows: int, device="cuda") -> "Workspace":
        return Workspace(load_library().dflash2_topk16_workspace_bytes(rows), device)

    @staticmethod
    def for_lmhead(rows: int, V: int, device="cuda") -> "Workspace":
        return Workspace(load_library().dflash2_lmhead_topk16_workspace_bytes(rows, V), device)

    @staticmethod
    def for_verify(B: int, K: int, device="cuda") -> "Workspace":
        return Workspace(load_library().dflash2_verify_workspace_bytes(B, K), device)

    @staticmethod
    def for_paged_attn(B: int, T: int, Hq: int, Hkv: int, d: int, dtype, device="cuda") -> "Workspace":
        return Workspace(load_library().dflash2_paged_attn_workspace_bytes(B, T, Hq, Hkv, d, _dtype_code(dtype)),
                         device)

    @staticmethod
    def for_linear4(rows: int, N: int, K: int, dtype=torch.bfloat16, device="cuda") -> "Workspace":
        return Workspace(load_library().dflash2_linear4_workspace_bytes(_dtype_code(dtype), rows, N, K), device)

    @staticmethod
    def for_kv_evict(B: int, Hkv: int, capacity: int, budget: int, device="cuda") -> "Workspace":
        """capacity: the slots a request's page table can hold (pages * page size)."""
        return Workspace(load_library().dflash2_kv_evict_workspace_bytes(B, Hkv, capacity, budget), device)


class KVCache:
    """A paged key-value cache: k and v [num_pages, Hkv, page_size, d] (bf16 or f32), of any strides with
    contiguous rows of d (a [num_pages, page_size, Hkv, d] pool is passed transposed), and the optional side
    arrays weight (f32) and pos (i32), contiguous [num_pages, Hkv, page_size].  Holds views, copies nothing.  A call
    takes tensors of the cache's device, which has to be the current one."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, weight: torch.Tensor | None = None,
                 pos: torch.Tensor | None = None):
        _need_cuda(k, v, weight, pos)
        if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v: one shape [num_pages, Hkv, page_size, d], one type and one layout, rows of d "
                             "contiguous")
        for name, t, dt in (("weight", weight, torch.float32), ("pos", pos, torch.int32)):
            if t is not None and (t.dtype != dt or t.shape != k.shape[:3] or not t.is_contiguous()):
                raise ValueError(f"{name}: contiguous {dt} [num_pages, Hkv, page_size]")
        if any(t is not None and t.device != k.device for t in (v, weight, pos)):
            raise ValueError("a cache's tensors lie on one device")
        self.k, self.v, self.weight, self.pos = k, v, weight, pos
        self.num_pages, self.Hkv, self.page_size, self.d = k.shape
        self.device, self.dtype, self._dev = k.device, k.dtype, k.get_device()
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self._rec = _CacheRecord(ptr(k), ptr(v), ptr(weight), ptr(pos), self.num_pages, k.stride(0), k.stride(1),
                                 k.stride(2), self.Hkv, self.page_size, self.d, _dtype(k))
        self._ref = ctypes.byref(self._rec)

    @staticmethod
    def empty(num_pages: int, Hkv: int, page_size: int, d: int, dtype=torch.bfloat16, weights: bool = False,
              positions: bool = False, device="cuda") -> "KVCache":
        """Uninitialised pages (weights and positions zero)."""
        kv = torch.empty(2, num_pages, Hkv, page_size, d, dtype=dtype, device=device)
        side = (num_pages, Hkv, page_size)
        return KVCache(kv[0], kv[1], torch.zeros(side, device=device) if weights else None,
                       torch.zeros(side, dtype=torch.int32, device=device) if positions else None)


class Weight4:
    """A matrix [N, K] held in 4 bits: codes uint8 [N, bytes] (two to a byte, the even column in the low half; bytes a
    multiple of 16 that covers K), scale [N, groups] (bf16 or f32) and the optional zero points of the same type (8
    without).  Rows may lie apart, rows themselves are contiguous, so slices of rows are taken as they are.  Holds
    views, copies nothing.  A call takes tensors of the codes' device, which has to be the current one."""

    def __init__(self, codes: torch.Tensor, scale: torch.Tensor, zero: torch.Tensor | None = None,
                 K: int | None = None, group: int = 128):
        _need_cuda(codes, scale, zero)
        if codes.dim() != 2 or codes.dtype is not torch.uint8 or (codes.stride(1) != 1 and codes.shape[1] > 1):
            raise ValueError("codes: uint8 [N, bytes] with contiguous rows")
        N = codes.shape[0]
        K = 2 * codes.shape[1] if K is None else K
        if group not in (32, 64, 128) or K < 1:
            raise ValueError("groups of 32, 64 or 128 and at least one column")
        if codes.shape[1] < -(-K // 32) * 16:
            raise ValueError(f"codes: {K} columns take {-(-K // 32) * 16} bytes a row")
        G = -(-K // group)
        _dtype(scale)
        for name, t in (("scale", scale), ("zero", zero)):
            if t is not None and (t.dtype is not scale.dtype or t.shape != (N, G) or t.device != codes.device or
                                  (t.stride(1) != 1 and G > 1)):
                raise ValueError(f"{name}: {scale.dtype} [{N}, {G}] with contiguous rows, beside the codes")
        if zero is not None and N > 1 and zero.stride(0) != scale.stride(0):
            raise ValueError("scale and zero: one distance from row to row")
        self.codes, self.scale, self.zero = codes, scale, zero
        self.N, self.K, self.group = N, K, group
        self.device, self._dev = codes.device, codes.get_device()
        ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
        self._rec = _Weight4Record(ptr(codes), ptr(scale), ptr(zero), N, K,
                                   codes.stride(0) if N > 1 else -(-codes.shape[1] // 16) * 16,
                                   scale.stride(0) if N > 1 else G, group, _dtype(scale))
        self._ref = ctypes.byref(self._rec)

    @staticmethod
    def empty(N: int, K: int, group: int = 128, zero: bool = False, dtype=torch.bfloat16, device="cuda") -> "Weight4":
        """Uninitialised codes, scales and (with zero) zero points."""
        side = lambda: torch.empty(N, -(-K // group), dtype=dtype, device=device)  # noqa: E731
        return Weight4(torch.empty(N, -(-K // 32) * 16, dtype=torch.uint8, device=device), side(),
                       side() if zero else None, K, group)


# ------------------------------------------------------------------ calls ----
def topk16(logits: torch.Tensor, params=None, rows_per_param: int = 1, V: int | None = None, ws=None, out=None):
    """dflash2_topk16.  logits [rows, ld] (bf16/f32).  Returns (cand_idx, cand_U, lse)."""
    L = load_library()
    _need_cuda(logits)
    assert logits.dim() == 2 and logits.stride(1) == 1
    rows, ld = logits.shape[0], logits.stride(0)
    V = logits.shape[1] if V is None else V
    dev = logits.device
    if out is None:
        out = (torch.empty(rows, NC, dtype=torch.int32, device=dev),
               torch.empty(rows, NC, dtype=torch.float32, device=dev),
               torch.empty(rows, dtype=torch.float32, device=dev))
    cand_idx, cand_U, lse = out
    if ws is None:
        ws = Workspace.for_topk16(rows, dev)
    p = _params_from(params, dev)
    _check("dflash2_topk16", L.dflash2_topk16(_ptr(logits), _dtype(logits), rows, V, ld, _ptr(p), rows_per_param,
                                              _ptr(cand_idx), _ptr(cand_U), _ptr(lse), ws.ptr(), ws.nbytes,
                                              _stream(dev)))
    return cand_idx, cand_U, lse


def topk16_noalloc(logits: torch.Tensor, params=None, rows_per_param: int = 1, V: int | None = None, out=None):
    """dflash2_topk16_noalloc: topk16 with the library's own fixed scratch.  Returns (cand_idx, cand_U, lse)."""
    L = load_library()
    _need_cuda(logits)
    assert logits.dim() == 2 and logits.stride(1) == 1
    rows, ld = logits.shape[0], logits.stride(0)
    V = logits.shape[1] if V is None else V
    dev = logits.device
    if out is None:
        out = (torch.empty(rows, NC, dtype=torch.int32, device=dev),
               torch.empty(rows, NC, dtype=torch.float32, device=dev),
               torch.empty(rows, dtype=torch.float32, device=dev))
    cand_idx, cand_U, lse = out
    p = _params_from(params, dev)
    _check("dflash2_topk16_noalloc",
           L.dflash2_topk16_noalloc(_ptr(logits), _dtype(logits), rows, V, ld, _ptr(p), rows_per_param,
                                    _ptr(cand_idx), _ptr(cand_U), _ptr(lse), _stream(dev)))
    return cand_idx, cand_U, lse


def topk16_shard(logits: torch.Tensor, id_offset: int, V_total: int, params=None, rows_per_param: int = 1,
                 V: int | None = None, ws=None, out=None):
    """dflash2_topk16_shard: one vocabulary slice's partial.  logits [rows, ld] hold tokens id_offset.. .
    Returns (part_idx [rows, 64] i32, part_z [rows, 64] f32, part_m [rows] f32, part_s [rows] f32)."""
    L = load_library()
    _need_cuda(logits)
    assert logits.dim() == 2 and logits.stride(1) == 1
    rows, ld = logits.shape[0], logits.stride(0)
    V = logits.shape[1] if V is None else V
    dev = logits.device
    if out is None:
        out = (torch.empty(rows, SHARD_LIST, dtype=torch.int32, device=dev),
               torch.empty(rows, SHARD_LIST, dtype=torch.float32, device=dev),
               torch.empty(rows, dtype=torch.float32, device=dev), torch.empty(rows, dtype=torch.float32, device=dev))
    pi, pz, pm, ps = out
    if ws is None:
        ws = Workspace.for_topk16(rows, dev)
    p = _params_from(params, dev)
    _check("dflash2_topk16_shard",
           L.dflash2_topk16_shard(_ptr(logits), _dtype(logits), rows, V, ld, id_offset, V_total, _ptr(p),
                                  rows_per_param, _ptr(pi), _ptr(pz), _ptr(pm), _ptr(ps), ws.ptr(), ws.nbytes,
                                  _stream(dev)))
    return pi, pz, pm, ps


def topk16_merge(part_idx, part_z, part_m, part_s, V_total: int, params=None, rows_per_param: int = 1, out=None):
    """dflash2_topk16_merge: partials stacked [S, rows, 64] / [S, rows].  Returns (cand_idx, cand_U, lse)."""
    L = load_library()
    _need_cuda(part_idx, part_z, part_m, part_s)
    for t in (part_idx, part_z, part_m, part_s):
        assert t.is_contiguous()
    S, rows = part_idx.shape[0], part_idx.shape[1]
    dev = part_idx.device
    if out is None:
        out = (torch.empty(rows, NC, dtype=torch.int32, device=dev),
               torch.empty(rows, NC, dtype=torch.float32, device=dev),
               torch.empty(rows, dtype=torch.float32, device=dev))
    cand_idx, cand_U, lse = out
    p = _params_from(params, dev)
    _check("dflash2_topk16_merge",
           L.dflash2_topk16_merge(S, rows, _ptr(part_idx), _ptr(part_z), _ptr(part_m), _ptr(part_s), V_total,
                                  _ptr(p), rows_per_param, _ptr(cand_idx), _ptr(cand_U), _ptr(lse), _stream(dev)))
    return cand_idx, cand_U, lse


def lmhead_topk16(h: torch.Tensor, W: torch.Tensor, params=None, rows_per_param: int = 1, ws=None, out=None):
    """dflash2_lmhead_topk16: h [rows, hidden] bf16, W [V, hidden] bf16.  Returns (cand_idx, cand_U, lse)."""
    L = load_library()
    _need_cuda(h, W)
    assert h.dtype == torch.bfloat16 and W.dtype == torch.bfloat16 and h.is_contiguous() and W.is_contiguous()
    rows, hidden = h.shape
    V = W.shape[0]
    dev = h.device
    if out is None:
        out = (torch.empty(rows, NC, dtype=torch.int32, device=dev),
               torch.empty(rows, NC, dtype=torch.float32, device=dev),
               torch.empty(rows, dtype=torch.float32, device=dev))
    cand_idx, cand_U, lse = out
    if ws is None:
        ws = Workspace.for_lmhead(rows, V, dev)
    p = _params_from(params, dev)
    _check("dflash2_lmhead_topk16",
           L.dflash2_lmhead_topk16(_ptr(h), _ptr(W), rows, hidden, V, _ptr(p), rows_per_param, _ptr(cand_idx),
                                   _ptr(cand_U), _ptr(lse), ws.ptr(), ws.nbytes, _stream(dev)))
    return cand_idx, cand_U, lse


def ctx_gate(h: torch.Tensor, Wg: torch.Tensor, out=None):
    """dflash2_ctx_gate.  h [n, hidden], Wg [D, hidden] (same dtype).  Returns gate [n, D] f32."""
    L = load_library()
    _need_cuda(h, Wg)
    assert h.is_contiguous() and Wg.is_contiguous() and h.dtype == Wg.dtype
    n, hidden = h.shape
    D = Wg.shape[0]
    gate = torch.empty(n, D, dtype=torch.float32, device=h.device) if out is None else out
    _check("dflash2_ctx_gate", L.dflash2_ctx_gate(_ptr(h), _dtype(h), n, hidden, _ptr(Wg), D, _ptr(gate),
                                                  _stream(h.device)))
    return gate


def pair_score_walk(cand_idx, cand_U, last_tok, A, Bt, gate, params=None, u_walk=None, out=None):
    """dflash2_pair_score_walk.  cand_idx/cand_U [B, K, 16], gate [B, K, D], A/Bt [V, D].

    Returns (path_tok [B,K], path_slot [B,K], q_sel [B,K,16], scores [B,K,16,16]).
    """
    L = load_library()
    _need_cuda(cand_idx, cand_U, last_tok, A, Bt, gate)
    B, K = cand_idx.shape[0], cand_idx.shape[1]
    V, D = A.shape
    dev = cand_idx.device
    if out is None:
        out = (torch.empty(B, K, dtype=torch.int32, device=dev), torch.empty(B, K, dtype=torch.int32, device=dev),
               torch.empty(B, K, NC, dtype=torch.float32, device=dev),
               torch.empty(B, K, NC, NC, dtype=torch.float32, device=dev))
    path_tok, path_slot, q_sel, scores = out
    p = _params_from(params, dev)
    _check("dflash2_pair_score_walk",
           L.dflash2_pair_score_walk(B, K, _ptr(cand_idx), _ptr(cand_U), _ptr(last_tok), _ptr(A), _ptr(Bt),
                                     _dtype(A), V, D, _ptr(gate), _ptr(p), _ptr(u_walk), _ptr(path_tok),
                                     _ptr(path_slot), _ptr(q_sel), _ptr(scores), _stream(dev)))
    return path_tok, path_slot, q_sel, scores


def verify(tlogits, path_tok, cand_idx, q_sel, path_slot, params=None, u_acc=None, u_res=None, ws=None,
           trusted: bool = False, V: int | None = None, out=None):
    """dflash2_verify.  tlogits [B*(K+1), ld].  Returns (accept_len [B], out_tok [B, K+1], status [B])."""
    L = load_library()
    _need_cuda(tlogits, path_tok, cand_idx, q_sel, path_slot)
    B, K = path_tok.shape
    assert tlogits.dim() == 2 and tlogits.stride(1) == 1 and tlogits.shape[0] == B * (K + 1)
    ld = tlogits.stride(0)
    V = tlogits.shape[1] if V is None else V
    dev = tlogits.device
    if ws is None:
        ws = Workspace.for_verify(B, K, dev)
    if out is None:
        out = (torch.empty(B, dtype=torch.int32, device=dev), torch.empty(B, K + 1, dtype=torch.int32, device=dev),
               torch.empty(B, dtype=torch.int32, device=dev))
    accept_len, out_tok, status = out
    p = _params_from(params, dev)
    _check("dflash2_verify",
           L.dflash2_verify(_ptr(tlogits), _dtype(tlogits), B, K, V, ld, _ptr(path_tok), _ptr(cand_idx),
                            _ptr(q_sel), _ptr(path_slot), _ptr(p), _ptr(u_acc), _ptr(u_res),
                            VERIFY_TRUST_Q if trusted else 0, _ptr(accept_len), _ptr(out_tok), _ptr(status),
                            ws.ptr(), ws.nbytes, _stream(dev)))
    return accept_len, out_tok, status


def conv2tap(x, k0, k1, x_prev, group: int = 1, out=None):
    """dflash2_conv2tap.  x [B, T, H], k0/k1 [B, T, H/group], x_prev [B, H].  Returns y [B, T, H]."""
    L = load_library()
    _need_cuda(x, k0, k1, x_prev)
    B, T, H = x.shape
    y = torch.empty_like(x) if out is None else out
    _check("dflash2_conv2tap", L.dflash2_conv2tap(_ptr(x), _ptr(k0), _ptr(k1), _ptr(x_prev), _dtype(x), B, T, H,
                                                  group, _ptr(y), _stream(x.device)))
    return y


def dynconv2tap(x, x_prev, Wd, group: int = 1, out=None):
    """dflash2_dynconv2tap.  x [B, T, H], x_prev [B, H], Wd [H/group, H].  Returns (taps [B, T, H/group]
    f32, y [B, T, H])."""
    L = load_library()
    _need_cuda(x, x_prev, Wd)
    B, T, H = x.shape
    if out is None:
        out = (torch.empty(B, T, H // group, dtype=torch.float32, device=x.device), torch.empty_like(x))
    taps, y = out
    _check("dflash2_dynconv2tap", L.dflash2_dynconv2tap(_ptr(x), _ptr(x_prev), _ptr(Wd), _dtype(x), B, T, H, group,
                                                        _ptr(taps), _ptr(y), _stream(x.device)))
    return taps, y


def rope_append(q, k, v, cos_sin, pos_ids, cache: KVCache, page_table, kv_len, pair_axis=None,
                interleaved: bool = False, q_norm=None, k_norm=None, eps: float = 1e-6, q_len=None, seq_pos=None,
                out=None):
    """dflash2_rope_append.  q [B, T, Hq, d], k and v [B, T, Hkv, d] of the cache's type (slices of a fused
    projection are taken as they are); cos_sin [n_pos, rot] f32; pos_ids [axes, B, T] int32; pair_axis [rot / 2]
    uint8; kv_len [B] int32, the slots in use before the call.  Returns (rotated q [B, T, Hq, d], kv_len + q_len)."""
    B, T, Hq, d = q.shape
    dt, Hkv, dev = cache.dtype, cache.Hkv, _here(cache)
    if d != cache.d:
        raise ValueError(f"q: heads of {cache.d}")
    qp, qs = _heads("q", q, dt, B, T, Hq, d, dev)
    kp, ks = _heads("k", k, dt, B, T, Hkv, d, dev)
    vp, vs = _heads("v", v, dt, B, T, Hkv, d, dev)
    n_pos, rot = cos_sin.shape
    axes = pos_ids.shape[0]
    table, pages = _page_table(page_table, B, dev)
    if out is None:
        out = (torch.empty((B, T, Hq, d), dtype=dt, device=q.device), torch.empty_like(kv_len))
    q_out, kv_len_out = out
    _check("dflash2_rope_append",
           (_lib or load_library()).dflash2_rope_append(
               cache._ref, table, pages, _int32(B, "kv_len", kv_len, dev), _int32(B, "q_len", q_len, dev),
               _int32(B, "seq_pos", seq_pos, dev), qp, kp, vp, qs, ks, vs, B, T, Hq,
               _dense("cos_sin", cos_sin, torch.float32, (n_pos, rot), dev), n_pos, rot,
               _dense("pos_ids", pos_ids, torch.int32, (axes, B, T), dev), axes,
               _dense("pair_axis", pair_axis, torch.uint8, (rot // 2,), dev), interleaved,
               _dense("q_norm", q_norm, dt, (d,), dev), _dense("k_norm", k_norm, dt, (d,), dev), eps,
               _dense("out", q_out, dt, (B, T, Hq, d), dev), _int32(B, "out", kv_len_out, dev), _raw_stream(dev)))
    return out


def paged_attn(q, cache: KVCache, page_table, kv_len, scale: float | None = None, causal: bool = True,
               window: int = 0, q_len=None, seq_pos=None, add_weights: bool = False, ws=None, out=None):
    """dflash2_paged_attn.  q [B, T, Hq, d] of the cache's type; kv_len [B] int32, the slots in use with the block's
    own among them; scale 1 / sqrt(d) unless given; add_weights adds every cached key's softmax weight to
    cache.weight (of all the block's tokens, before a verify has rejected any).  Returns (out [B, T, Hq, d], lse [B, T, Hq] f32)."""
    B, T, Hq, d = shape = q.shape
    dt, dev = cache.dtype, _here(cache)
    if d != cache.d:
        raise ValueError(f"q: heads of {cache.d}")
    table, pages = _page_table(page_table, B, dev)
    if ws is None:
        ws = Workspace.for_paged_attn(B, T, Hq, cache.Hkv, d, dt, q.device)
    if out is None:
        out = (torch.empty_like(q), torch.empty((B, T, Hq), dtype=torch.float32, device=q.device))
    o, lse = out
    _check("dflash2_paged_attn",
           (_lib or load_library()).dflash2_paged_attn(
               cache._ref, table, pages, _int32(B, "kv_len", kv_len, dev), _int32(B, "q_len", q_len, dev),
               _int32(B, "seq_pos", seq_pos, dev), _dense("q", q, dt, shape, dev), B, T, Hq,
               d ** -0.5 if scale is None else scale, _count("window", window),
               (ATTN_CAUSAL if causal else 0) | (ATTN_WEIGHTS if add_weights else 0), _dense("out", o, dt, shape, dev),
               _dense("out", lse, torch.float32, (B, T, Hq), dev), *_scratch(ws, dev), _raw_stream(dev)))
    return out


def kv_evict(cache: KVCache, page_table, kv_len, budget: int, recent: int = 0, sink: int = 0, seq_len=None, ws=None,
             out=None):
    """dflash2_kv_evict.  Every head keeps `budget` slots of a request that has more: those of the `recent` newest and
    `sink` first positions, then the most attended.  Returns min(kv_len, budget) [B] int32."""
    B, dev = kv_len.shape[0], _here(cache)
    table, pages = _page_table(page_table, B, dev)
    _count("budget", budget)
    if ws is None:
        ws = Workspace.for_kv_evict(B, cache.Hkv, pages * cache.page_size, budget, kv_len.device)
    if out is None:
        out = torch.empty_like(kv_len)
    _check("dflash2_kv_evict",
           (_lib or load_library()).dflash2_kv_evict(
               cache._ref, table, pages, _int32(B, "kv_len", kv_len, dev), _int32(B, "seq_len", seq_len, dev), B, budget,
               _count("recent", recent), _count("sink", sink), _int32(B, "out", out, dev), *_scratch(ws, dev),
               _raw_stream(dev)))
    return out


def _rows(name: str, t, shape, dev: int):
    """Address and row stride of a matrix with contiguous rows on GPU `dev`."""
    if t.dim() != 2 or tuple(t.shape) != shape or t.get_device() != dev or (t.stride(1) != 1 and shape[1] > 1):
        raise ValueError(f"{name}: [{shape[0]}, {shape[1]}] with contiguous rows on the weights' GPU")
    return t.data_ptr(), t.stride(0) if shape[0] > 1 else max(shape[1], 1)


def quant4(W: torch.Tensor, group: int = 128, zero: bool = False, dtype=torch.bfloat16, out=None) -> Weight4:
    """dflash2_quant4.  W [N, K] (bf16/f32, contiguous rows).  Returns its Weight4 (scales of `dtype`), or fills
    `out`."""
    L = load_library()
    _need_cuda(W)
    if W.dim() != 2:
        raise ValueError("W: [N, K]")
    if out is None:
        out = Weight4.empty(W.shape[0], W.shape[1], group, zero, dtype, W.device)
    dev = _here(out, "weights")
    p, ld = _rows("W", W, (out.N, out.K), dev)
    _check("dflash2_quant4", L.dflash2_quant4(p, _dtype(W), ld, out._ref, _raw_stream(dev)))
    return out


def dequant4(w: Weight4, dtype=torch.bfloat16, out=None) -> torch.Tensor:
    """dflash2_dequant4.  Returns [N, K] of `dtype`, or fills `out` (contiguous rows)."""
    L = load_library()
    dev = _here(w, "weights")
    if out is None:
        out = torch.empty(w.N, w.K, dtype=dtype, device=w.device)
    p, ld = _rows("out", out, (w.N, w.K), dev)
    _check("dflash2_dequant4", L.dflash2_dequant4(w._ref, p, _dtype(out), ld, _raw_stream(dev)))
    return out


def linear4(x: torch.Tensor, w: Weight4, dtype=None, ws=None, out=None, rounded: bool = False) -> torch.Tensor:
    """dflash2_linear4.  x [rows, K] (bf16/f32, contiguous rows).  Returns x . W^T [rows, N] of x's type or float32, or
    fills `out` (contiguous rows, any distance from row to row).  With rounded, dflash2_linear4_rounded: many rows of bf16
    may be taken on weights rounded to bf16, which is faster."""
    dev = _here(w, "weights")
    rows = x.shape[0]
    xp, xs = _rows("x", x, (rows, w.K), dev)
    if out is None:
        out = torch.empty((rows, w.N), dtype=x.dtype if dtype is None else dtype, device=x.device)
    yp, ys = _rows("out", out, (rows, w.N), dev)
    L, dt = _lib or load_library(), _dtype(x)
    if ws is None:
        need = L.dflash2_linear4_workspace_bytes(dt, rows, w.N, w.K)
        buf = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
        scratch = (buf.data_ptr(), need) if need else (None, 0)
    else:
        scratch = _scratch(ws, dev)
    call = L.dflash2_linear4_rounded if rounded else L.dflash2_linear4
    _check("dflash2_linear4", call(xp, dt, rows, xs, w._ref, yp, _dtype(out), ys, *scratch, _raw_stream(dev)))
    return out


def sample(logits: torch.Tensor, u: torch.Tensor, params=None, min_p=None, rows_per_param: int = 1,
           V: int | None = None, out=None):
    """dflash2_sample.  logits [rows, ld] (bf16/f32), u [rows] f32 uniforms, min_p [n] f32 for the n = ceil(rows /
    rows_per_param) entries of params (or alone: greedy).  Returns (token [rows] int32, prob [rows] f32)."""
    _need_cuda(logits, u, min_p)
    rows, dev = logits.shape[0], logits.get_device()
    if torch._C._cuda_getDevice() != dev:
        raise ValueError(f"the logits lie on cuda:{dev}, which is not the current device")
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits: [rows, ld] with contiguous rows")
    _count("rows_per_param", rows_per_param)
    n = -(-rows // max(rows_per_param, 1))
    p = _params_from(params, logits.device)
    if p is not None and (p.get_device() != dev or not p.is_contiguous() or
                          p.numel() * p.element_size() < 12 * n):
        raise ValueError(f"params: {n} records on the logits' GPU")
    if out is None:
        out = (torch.empty(rows, dtype=torch.int32, device=logits.device),
               torch.empty(rows, dtype=torch.float32, device=logits.device))
    token, prob = out
    ld = logits.stride(0)
    if rows <= 1:                                        # a single row's stride says nothing
        ld = -(-logits.shape[1] * logits.element_size() // 16) * 16 // logits.element_size()
    V = logits.shape[1] if V is None else V
    if V > logits.shape[1]:
        raise ValueError("V: more entries than a row has")
    f32 = torch.float32
    _check("dflash2_sample",
           (_lib or load_library()).dflash2_sample(
               logits.data_ptr(), _dtype(logits), rows, V, ld, None if p is None else p.data_ptr(),
               _dense("min_p", min_p, f32, (n,), dev, "logits"), rows_per_param, _dense("u", u, f32, (rows,), dev, "logits"),
               _dense("out", token, torch.int32, (rows,), dev, "logits"), _dense("out", prob, f32, (rows,), dev, "logits"),
               _raw_stream(dev)))
    return out


def device_error(clear: bool = False) -> int:
    """The library's device error word (synchronises the device)."""
    L = load_library()
    code = ctypes.c_uint32(0)
    _check("dflash2_device_error", L.dflash2_device_error(ctypes.byref(code), int(clear)))
    return code.value


def test_hold(flag=None, max_cycles: int = 0):
    """dflash2_test_hold: with `flag` (a CUDA int32 tensor of one element) set, later scan
    kernels wait on it for at most `max_cycles` before their first copy; None switches it off."""
    L = load_library()
    _need_cuda(flag)
    _check("dflash2_test_hold", L.dflash2_test_hold(_ptr(flag), int(max_cycles) if flag is not None else 0))
