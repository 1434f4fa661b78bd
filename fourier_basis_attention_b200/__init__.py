"""Python binding of the Fourier-approximated KV cache library (sm_100a).

Argument marshalling only: every step of the hot path runs in the CUDA kernels of
``libfourier_attention.so`` behind the C ABI declared in ``include/fourier_attention.h``.
PyTorch is used for device memory and streams. The functions keep the C names:

    fa_plan_init, fa_plan_reserve, fa_build_basis, fa_compress, fa_decode_workspace_size,
    fa_decode_describe, fa_decode, fa_decode_noalloc, fa_append, fa_dim_sensitivity_workspace_size,
    fa_dim_sensitivity, fa_select_dims, fa_device_status, fa_last_error

and, over a paged full-precision cache,

    fa_rope_init, fa_rope, fa_paged_append, fa_paged_attend_workspace_size, fa_paged_attend,
    fa_paged_weights, fa_evict_workspace_size, fa_evict

There is no CPU fallback: if the shared library is missing or fails to load, importing
this package raises.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np

from . import _build

HEAD_DIM = 128
MAX_KV_HEADS = 64
MAX_K_DECODE = 2047
FA_OK, FA_ERR_INVALID, FA_ERR_UNSUPPORTED, FA_ERR_CUDA, FA_ERR_DEVICE = range(5)
FA_BF16, FA_F32 = 0, 1
(FA_SPLIT_NONE, FA_SPLIT_CUDA_CORES, FA_SPLIT_TC_TOKEN_MAJOR, FA_SPLIT_WARP_MMA,
 FA_SPLIT_TC_CLUSTER) = range(5)

EXPORTED = ("fa_plan_init", "fa_plan_reserve", "fa_build_basis", "fa_compress",
            "fa_decode_workspace_size", "fa_decode", "fa_decode_noalloc", "fa_append",
            "fa_dim_sensitivity_workspace_size", "fa_dim_sensitivity", "fa_select_dims",
            "fa_device_status", "fa_watchdog_selftest", "fa_last_error", "fa_decode_describe",
            "fa_rope_init", "fa_rope", "fa_paged_append", "fa_paged_attend_workspace_size",
            "fa_paged_attend", "fa_paged_weights", "fa_evict_workspace_size", "fa_evict")
MAX_Q_HEADS = 1024
ROPE_SCALINGS = {"plain": 0, "linear": 1, "ntk": 2, "bands": 3, "yarn": 4}
NOISE_SCALE = 0.1
NOALLOC_SCRATCH_BYTES = 16 << 20


class FaError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


class fa_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "D", "L", "S", "R", "k")]


_H = MAX_KV_HEADS


class fa_plan(ctypes.Structure):
    _fields_ = [
        ("shape", fa_shape),
        ("S", ctypes.c_int32), ("R", ctypes.c_int32), ("M", ctypes.c_int32),
        ("kk", ctypes.c_int32), ("G", ctypes.c_int32), ("phi_ld", ctypes.c_int32),
        ("e_token_major", ctypes.c_int32), ("P", ctypes.c_int32), ("recent_head", ctypes.c_int32),
        ("dc", ctypes.c_int32 * _H), ("de", ctypes.c_int32 * _H),
        ("dc_ld", ctypes.c_int32 * _H), ("de_ld", ctypes.c_int32 * _H),
        ("e_pitch", ctypes.c_int32 * _H),
        ("c_off", ctypes.c_int64 * _H), ("e_off", ctypes.c_int64 * _H),
        ("c_batch", ctypes.c_int64), ("e_batch", ctypes.c_int64),
        ("f_elems", ctypes.c_int64), ("e_elems", ctypes.c_int64), ("c_elems", ctypes.c_int64),
        ("perm", (ctypes.c_uint8 * HEAD_DIM) * _H),
    ]


class fa_decode_info(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("split_kernel", "num_splits", "cluster", "launches")]


SPLIT_KERNELS = {0: "none (no middle span)", 1: "CUDA cores (decode_main_kernel)",
                 2: "tcgen05, token-major E (decode_tc_kernel)",
                 3: "warp MMA (decode_hmma_kernel)",
                 4: "tcgen05, slot-split cluster (decode_cl_kernel)"}


class fa_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("F_K", "F_V", "E_K", "E_V", "C_K", "C_V")]


class fa_paged_shape(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hkv", "D", "page_size", "num_pages",
                                              "max_pages", "total_q", "max_q", "max_kv")]


class fa_paged_cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("K", "V", "page_table", "q_start", "kv_len")]


class fa_rope_config(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_int32) for n in ("rot_dim", "interleaved", "scaling",
                                               "original_len")]
                + [(n, ctypes.c_double) for n in ("base", "factor", "low", "high", "magnitude")])


class fa_rope_plan(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("magnitude", ctypes.c_float), ("reserved", ctypes.c_int32),
                ("turns", ctypes.c_uint64 * (HEAD_DIM // 2))]


def _load() -> ctypes.CDLL:
    path = _build.LIB
    if os.environ.get("FA_SKIP_BUILD") != "1":
        path = _build.build()
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing; run fourier_basis_attention_b200._build.build()")
    return configure(ctypes.CDLL(path))


def configure(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Declare the C signatures on a loaded copy of the library."""
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.fa_plan_init.argtypes = [ctypes.POINTER(fa_shape), P, ctypes.POINTER(fa_plan)]
    lib.fa_plan_reserve.argtypes = [ctypes.POINTER(fa_plan), I32]
    lib.fa_build_basis.argtypes = [I32, I32, I32, I32, P, I64, P]
    lib.fa_append.argtypes = [ctypes.POINTER(fa_plan), P, P, ctypes.POINTER(fa_cache), P]
    lib.fa_dim_sensitivity_workspace_size.argtypes = [ctypes.POINTER(fa_shape)]
    lib.fa_dim_sensitivity_workspace_size.restype = SZ
    lib.fa_dim_sensitivity.argtypes = [ctypes.POINTER(fa_shape), P, P, P, P, P, SZ, P]
    lib.fa_select_dims.argtypes = [P, I32, I32, P]
    lib.fa_compress.argtypes = [ctypes.POINTER(fa_plan), P, P, P, ctypes.POINTER(fa_cache), P]
    lib.fa_decode_workspace_size.argtypes = [ctypes.POINTER(fa_plan), I32]
    lib.fa_decode_workspace_size.restype = SZ
    lib.fa_decode_describe.argtypes = [ctypes.POINTER(fa_plan), I32, ctypes.POINTER(fa_decode_info)]
    lib.fa_decode.argtypes = [ctypes.POINTER(fa_plan), P, ctypes.POINTER(fa_cache), P, I32, P, SZ,
                              I32, P]
    lib.fa_decode_noalloc.argtypes = [ctypes.POINTER(fa_plan), P, ctypes.POINTER(fa_cache), P, I32,
                                      I32, P]
    lib.fa_device_status.argtypes = [P]
    lib.fa_watchdog_selftest.argtypes = [ctypes.c_uint32, P]
    SH, CA = ctypes.POINTER(fa_paged_shape), ctypes.POINTER(fa_paged_cache)
    RP, F32 = ctypes.POINTER(fa_rope_plan), ctypes.c_float
    lib.fa_rope_init.argtypes = [ctypes.POINTER(fa_rope_config), RP]
    lib.fa_rope.argtypes = [RP, I32, I32, I32, P, P, ctypes.POINTER(I64), P, ctypes.POINTER(I64),
                            I32, I32, P]
    lib.fa_paged_append.argtypes = [SH, CA, RP, P, P, I64, P, I64, P, I64, P, I64, P]
    lib.fa_paged_attend_workspace_size.argtypes = [SH, I32]
    lib.fa_paged_attend_workspace_size.restype = SZ
    lib.fa_paged_attend.argtypes = [SH, CA, P, I64, F32, I32, P, I64, P, P, SZ, P]
    lib.fa_paged_weights.argtypes = [SH, CA, P, I64, F32, I32, P, P, I64, P]
    lib.fa_evict_workspace_size.argtypes = [SH, I32]
    lib.fa_evict_workspace_size.restype = SZ
    lib.fa_evict.argtypes = [SH, CA, P, I64, I32, I32, I32, SH, CA, P, I64, P, P, P, SZ, P]
    lib.fa_last_error.argtypes = []
    lib.fa_last_error.restype = ctypes.c_char_p
    for name in ("fa_plan_init", "fa_plan_reserve", "fa_build_basis", "fa_compress", "fa_decode",
                 "fa_decode_noalloc", "fa_append", "fa_dim_sensitivity", "fa_select_dims",
                 "fa_device_status", "fa_watchdog_selftest", "fa_decode_describe", "fa_rope_init",
                 "fa_rope", "fa_paged_append", "fa_paged_attend", "fa_paged_weights", "fa_evict"):
        getattr(lib, name).restype = ctypes.c_int
    return lib


LIB = _load()
LIB_PATH = _build.LIB


def fa_last_error() -> str:
    return LIB.fa_last_error().decode()


def _check(code: int) -> None:
    if code != FA_OK:
        raise FaError(code, fa_last_error())


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


# ----------------------------------------------------------------------------- C entry points

def fa_plan_init(B, Hq, Hkv, L, S, R, k, mask, D=HEAD_DIM) -> fa_plan:
    """Host-side plan of one layer. ``mask``: uint8-like [Hkv, 128], nonzero = compressed."""
    m = np.ascontiguousarray(np.asarray(mask) != 0, dtype=np.uint8)
    if m.shape != (Hkv, D):
        raise FaError(FA_ERR_INVALID, f"mask shape {m.shape} != ({Hkv}, {D})")
    shape = fa_shape(B, Hq, Hkv, D, L, S, R, k)
    plan = fa_plan()
    _check(LIB.fa_plan_init(ctypes.byref(shape), m.ctypes.data, ctypes.byref(plan)))
    return plan


def fa_plan_reserve(plan: fa_plan, L_max: int) -> fa_plan:
    """Room for tokens appended while decoding: basis period P = L_max - S - R (in place)."""
    _check(LIB.fa_plan_reserve(ctypes.byref(plan), int(L_max)))
    return plan


def fa_build_basis(M: int, k: int, phiT, ld: int | None = None, normalized: bool = False,
                   stream=None) -> None:
    """Fill device tensor ``phiT`` ([k, ld], bf16 or fp32) with the transposed basis
    (``normalized=False``: the unit-amplitude table fa_compress reads)."""
    import torch
    dtype = FA_BF16 if phiT.dtype == torch.bfloat16 else FA_F32
    if ld is None:
        ld = phiT.shape[-1]
    _check(LIB.fa_build_basis(M, k, dtype, int(bool(normalized)), _ptr(phiT), ld,
                              _stream(stream)))


def fa_compress(plan: fa_plan, K, V, phiT, cache: "Cache", stream=None) -> None:
    _check(LIB.fa_compress(ctypes.byref(plan), _ptr(K), _ptr(V), _ptr(phiT),
                           ctypes.byref(cache.c), _stream(stream)))


def fa_decode_workspace_size(plan: fa_plan, num_splits: int = 0) -> int:
    return int(LIB.fa_decode_workspace_size(ctypes.byref(plan), num_splits))


def fa_decode_describe(plan: fa_plan, num_splits: int = 0) -> fa_decode_info:
    """How fa_decode runs this plan: split kernel, split count, cluster size, launches."""
    info = fa_decode_info()
    _check(LIB.fa_decode_describe(ctypes.byref(plan), num_splits, ctypes.byref(info)))
    return info


def fa_decode(plan: fa_plan, q, cache: "Cache", out, workspace, num_splits: int = 0,
              stream=None) -> None:
    """One decode step; ``out`` is a [B, Hq, 128] fp32 or bf16 device tensor."""
    import torch
    out_dtype = FA_F32 if out.dtype == torch.float32 else FA_BF16
    nbytes = workspace.numel() * workspace.element_size()
    _check(LIB.fa_decode(ctypes.byref(plan), _ptr(q), ctypes.byref(cache.c), _ptr(out),
                         out_dtype, _ptr(workspace), nbytes, num_splits, _stream(stream)))


def fa_decode_noalloc(plan: fa_plan, q, cache: "Cache", out, num_splits: int = 0,
                      stream=None) -> None:
    """fa_decode without a workspace argument, for callers that cannot allocate device
    memory: the library's own fixed scratch array is used (see the C header)."""
    import torch
    out_dtype = FA_F32 if out.dtype == torch.float32 else FA_BF16
    _check(LIB.fa_decode_noalloc(ctypes.byref(plan), _ptr(q), ctypes.byref(cache.c), _ptr(out),
                                 out_dtype, num_splits, _stream(stream)))


def fa_append(plan: fa_plan, k_new, v_new, cache: "Cache", stream=None) -> None:
    """Append one token per sequence (k_new, v_new: bf16 [B, Hkv, 128]); advances ``plan``."""
    _check(LIB.fa_append(ctypes.byref(plan), _ptr(k_new), _ptr(v_new), ctypes.byref(cache.c),
                         _stream(stream)))


def fa_dim_sensitivity_workspace_size(B, Hq, Hkv, L) -> int:
    return LIB.fa_dim_sensitivity_workspace_size(ctypes.byref(fa_shape(B, Hq, Hkv, HEAD_DIM, L, 0, 0, 1)))


def fa_dim_sensitivity(q, K, noise, scores, workspace, stream=None) -> None:
    """Sensitivity scores [Hkv, 128] (fp32, device) of every head dim under value noise.
    q: bf16 [B, Hq, 128]; K, noise: bf16 [B, Hkv, L, 128]."""
    B, Hkv, L, D = K.shape
    shape = fa_shape(B, q.shape[1], Hkv, D, L, 0, 0, 1)
    _check(LIB.fa_dim_sensitivity(ctypes.byref(shape), _ptr(q), _ptr(K), _ptr(noise), _ptr(scores),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream)))


def fa_select_dims(scores, n_compressed: int) -> np.ndarray:
    """Host: uint8 mask [Hkv, 128] compressing the n_compressed lowest-score dims per KV head."""
    sc = np.ascontiguousarray(np.asarray(scores, dtype=np.float32))
    Hkv = sc.shape[0]
    mask = np.zeros((Hkv, HEAD_DIM), dtype=np.uint8)
    _check(LIB.fa_select_dims(sc.ctypes.data, Hkv, int(n_compressed), mask.ctypes.data))
    return mask


# ------------------------------------------------------------------- paged full-precision cache

def _invalid(msg: str):
    raise FaError(FA_ERR_INVALID, msg)


_torch = None  # held from the first call on, so that later ones do not look it up


def _import_torch():
    global _torch
    import torch as _torch
    return _torch


def _device() -> int:
    return (_torch or _import_torch()).cuda.current_device()


def _raw_stream(stream, device: int):
    if stream is None:
        return _torch._C._cuda_getCurrentRawStream(device)
    return getattr(stream, "cuda_stream", stream)


def _int32(**values) -> None:
    """Refuse whole numbers that ctypes would cut to other ones."""
    for name, n in values.items():
        if not -2 ** 31 <= n < 2 ** 31:
            _invalid(f"{name}={n} does not fit 32 bits")


def _softmax(window: int, scale: float) -> None:
    if not -2 ** 31 <= window < 2 ** 31:
        _int32(window=window)
    if 0.0 < abs(scale) < 1e-37:  # fp32 would make 0 of it, which picks 1 / sqrt(128)
        raise FaError(FA_ERR_UNSUPPORTED, f"scale={scale} is outside [1e-20, 1e20]")


def _here(pages, name: str = "the batch") -> int:
    """The current device, where the pointers that a PagedBatch or PagedCache holds must lie."""
    device = _device()
    if pages.device != device:
        _invalid(f"{name} is on cuda:{pages.device}, not on the current CUDA device")
    return device


def _why(t, name: str, dtype, shape, device: int, dense: int):
    """Raise for a tensor that _tensor refused."""
    import torch
    if not isinstance(t, torch.Tensor):
        _invalid(f"{name} is not a tensor")
    if t.dtype != dtype:
        _invalid(f"{name} has dtype {t.dtype}, needs {dtype}")
    if t.dim() != len(shape) or any(n is not None and n != m for n, m in zip(shape, t.shape)):
        _invalid(f"{name} has shape {tuple(t.shape)}, needs {tuple(shape)}")
    if not t.is_cuda or t.get_device() != device:
        _invalid(f"{name} is on {t.device}, not on the current CUDA device")
    _invalid(f"{name}: the last {dense} axes must be dense, strides are {t.stride()}")


def _tensor(t, name: str, dtype, shape: tuple, device: int) -> int:
    """Data pointer of a dense tensor of this type and shape on the current device."""
    try:
        if (t.dtype is dtype and t.shape == shape and t.get_device() == device
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    return _why(t, name, dtype, shape, device, len(shape))


def _rows(t, name: str, shape: tuple, device: int):
    """(pointer, elements between tokens) of a bf16 [tokens, heads, 128] tensor whose heads
    are dense."""
    try:
        if t.dtype is _torch.bfloat16 and t.shape == shape and t.get_device() == device:
            st = t.stride()
            if st[2] == 1 and (st[1] == HEAD_DIM or shape[1] == 1) or not t.numel():
                return t.data_ptr(), st[0] if shape[0] > 1 else shape[1] * HEAD_DIM
    except AttributeError:
        pass
    return _why(t, name, _torch.bfloat16, shape, device, 2)


class PagedCache:
    """Pools of pages: K, V bf16 [num_pages, Hkv, page_size, 128], page_table int32
    [B, max_pages]. Keeps the tensors; a dense [B, Hkv, L, 128] tensor is a pool of B pages
    (``PagedCache.dense``)."""

    def __init__(self, K, V, page_table):
        import torch
        for t, name, dtype, dims in ((K, "K", torch.bfloat16, 4), (V, "V", torch.bfloat16, 4),
                                     (page_table, "page_table", torch.int32, 2)):
            if not isinstance(t, torch.Tensor) or t.dim() != dims:
                _why(t, name, dtype, (None,) * dims, -1, dims)
        device = self.device = _device() if K.is_cuda else -2
        shape = (*K.shape[:3], HEAD_DIM)
        self.pointers = (_tensor(K, "K", torch.bfloat16, shape, device),
                         _tensor(V, "V", torch.bfloat16, shape, device),
                         _tensor(page_table, "page_table", torch.int32, tuple(page_table.shape), device))
        self.K, self.V, self.page_table = K, V, page_table
        self.num_pages, self.Hkv, self.page_size = K.shape[:3]
        self.B, self.max_pages = page_table.shape

    @classmethod
    def dense(cls, K, V):
        """The dense [B, Hkv, L, 128] tensors that fa_compress reads: page b is sequence b."""
        import torch
        table = torch.arange(K.shape[0], dtype=torch.int32, device=K.device)
        return cls(K, V, table[:, None].contiguous())


class PagedBatch:
    """A batch over a PagedCache: q_start int32 [B + 1], kv_len int32 [B] (device, read when a
    call runs) and the bounds that size the launches. max_kv = None: all the table holds."""

    def __init__(self, cache: PagedCache, Hq: int, q_start, kv_len, total_q: int, max_q: int,
                 max_kv: int | None = None):
        import torch
        device = self.device = _here(cache, "the cache")
        starts = _tensor(q_start, "q_start", torch.int32, (cache.B + 1,), device)
        lens = _tensor(kv_len, "kv_len", torch.int32, (cache.B,), device)
        self.cache, self.q_start, self.kv_len = cache, q_start, kv_len
        self.Hq, self.total_q = Hq, total_q
        if max_kv is None:
            max_kv = cache.max_pages * cache.page_size
        self.max_kv = max_kv
        _int32(Hq=Hq, total_q=total_q, max_q=max_q, max_kv=max_kv)
        self.shape = fa_paged_shape(cache.B, Hq, cache.Hkv, HEAD_DIM, cache.page_size,
                                    cache.num_pages, cache.max_pages, total_q, max_q, max_kv)
        self.c = fa_paged_cache(*cache.pointers, starts, lens)
        self.refs = ctypes.byref(self.shape), ctypes.byref(self.c)
        # shapes of q, of k and v, of lse
        self.q_shape, self.kv_shape = (total_q, Hq, HEAD_DIM), (total_q, cache.Hkv, HEAD_DIM)
        self.lse_shape = (total_q, Hq)


def fa_rope_init(rot_dim: int = HEAD_DIM, base: float = 10000.0, interleaved: bool = False,
                 scaling: str = "plain", factor: float = 1.0, low: float = 1.0, high: float = 4.0,
                 original_len: int = 0, magnitude: float = 0.0) -> fa_rope_plan:
    """Host-side plan of a rotation (see the C header for the scalings)."""
    if scaling not in ROPE_SCALINGS:
        _invalid(f"unknown scaling {scaling!r}")
    _int32(rot_dim=rot_dim, original_len=original_len)
    config = fa_rope_config(rot_dim, int(bool(interleaved)), ROPE_SCALINGS[scaling], original_len,
                            base, factor, low, high, magnitude)
    plan = fa_rope_plan()
    _check(LIB.fa_rope_init(ctypes.byref(config), ctypes.byref(plan)))
    return plan


_STRIDE3 = ctypes.c_int64 * 3


def fa_rope(rope: fa_rope_plan, x, positions, out, transpose: bool = False, stream=None) -> None:
    """Rotate x (bf16 or fp32 [B, T, H, 128], any strides of the first three axes) at int32
    positions [B, T] into ``out``; ``transpose``: the transposed map, its gradient."""
    torch = _torch or _import_torch()
    dtype = FA_BF16
    if x.dtype is not torch.bfloat16:
        dtype = FA_F32
        if x.dtype is not torch.float32:
            _invalid(f"x has dtype {x.dtype}, needs bfloat16 or float32")
    shape = x.shape
    if len(shape) != 4 or shape[3] != HEAD_DIM:
        _invalid(f"x has shape {tuple(shape)}, needs [B, T, H, 128]")
    if not x.is_cuda:
        _invalid(f"x is on {x.device}, not on the current CUDA device")
    device = _device()
    xs, ys = x.stride(), out.stride()
    if x.get_device() != device:
        _why(x, "x", x.dtype, shape, device, 1)
    if out.dtype is not x.dtype or out.shape != shape or out.get_device() != device:
        _why(out, "out", x.dtype, shape, device, 1)
    if (xs[3] != 1 or ys[3] != 1) and x.numel():
        _invalid(f"the last axis of x and out must be dense, strides are {xs} and {ys}")
    B, T, H, _ = shape
    pp = _tensor(positions, "positions", torch.int32, (B, T), device)
    _check(LIB.fa_rope(rope, B, T, H, pp, x.data_ptr(), _STRIDE3(xs[0], xs[1], xs[2]), out.data_ptr(),
                       _STRIDE3(ys[0], ys[1], ys[2]), dtype, 1 if transpose else 0,
                       _raw_stream(stream, device)))


def fa_paged_append(batch: PagedBatch, k, v, q=None, q_out=None, rope: fa_rope_plan | None = None,
                    positions=None, stream=None) -> None:
    """Write the new tokens k, v (bf16 [total_q, Hkv, 128]) into the pages; with ``rope`` k, and
    q into q_out (bf16 [total_q, Hq, 128]), are rotated, at the cache index or ``positions``."""
    device = _here(batch)
    pq = pqo = pp = None
    qs = qos = 0
    if q is not None:
        pq, qs = _rows(q, "q", batch.q_shape, device)
    if q_out is not None:
        pqo, qos = _rows(q_out, "q_out", batch.q_shape, device)
    if positions is not None:
        pp = _tensor(positions, "positions", _torch.int32, (batch.total_q,), device)
    pk, ks = _rows(k, "k", batch.kv_shape, device)
    pv, vs = _rows(v, "v", batch.kv_shape, device)
    _check(LIB.fa_paged_append(*batch.refs, rope, pp, pq, qs, pqo, qos, pk, ks, pv, vs,
                               _raw_stream(stream, device)))


def fa_paged_attend_workspace_size(batch: PagedBatch, window: int = 0) -> int:
    _softmax(window, 0.0)
    return LIB.fa_paged_attend_workspace_size(batch.refs[0], window)


def _workspace(workspace, device: int):
    if workspace is None:
        return None, 0
    if workspace.get_device() != device:
        _invalid(f"workspace is on {workspace.device}, not on the current CUDA device")
    if not workspace.is_contiguous():
        _invalid("workspace must be contiguous")
    return workspace.data_ptr() or None, workspace.numel() * workspace.element_size()


def fa_paged_attend(batch: PagedBatch, q, out, workspace=None, lse=None, window: int = 0,
                    scale: float = 0.0, stream=None) -> None:
    """Causal attention of the new tokens q (bf16 [total_q, Hq, 128], rotated) over the pages,
    their own keys included, into ``out`` (same shape); lse: fp32 [total_q, Hq] or None."""
    device = _here(batch)
    _softmax(window, scale)
    pq, qs = _rows(q, "q", batch.q_shape, device)
    po, os_ = _rows(out, "out", batch.q_shape, device)
    pl = None if lse is None else _tensor(lse, "lse", _torch.float32, batch.lse_shape, device)
    ws, size = _workspace(workspace, device)
    _check(LIB.fa_paged_attend(*batch.refs, pq, qs, scale, window, po, os_, pl, ws, size,
                               _raw_stream(stream, device)))


def fa_paged_weights(batch: PagedBatch, q, lse, weights, window: int = 0, scale: float = 0.0,
                     stream=None) -> None:
    """Add to ``weights`` (fp32 [B, Hkv, >= max_kv]) what each key gets from the batch's
    queries; ``lse`` as fa_paged_attend wrote it for the same arguments."""
    device = _here(batch)
    _softmax(window, scale)
    pq, qs = _rows(q, "q", batch.q_shape, device)
    pl = _tensor(lse, "lse", _torch.float32, batch.lse_shape, device)
    pw, ld = _wide(weights, "weights", batch.cache, device)
    _check(LIB.fa_paged_weights(*batch.refs, pq, qs, scale, window, pl, pw, ld,
                                _raw_stream(stream, device)))


def _wide(t, name: str, cache: PagedCache, device: int):
    """(pointer, last size) of a dense fp32 [B, Hkv, any] tensor."""
    last = t.shape[-1] if isinstance(t, _torch.Tensor) and t.dim() == 3 else None
    return _tensor(t, name, _torch.float32, (cache.B, cache.Hkv, last), device), last


def fa_evict_workspace_size(batch: PagedBatch, keep: int) -> int:
    _int32(keep=keep)
    return LIB.fa_evict_workspace_size(batch.refs[0], keep)


def fa_evict(batch: PagedBatch, weights, keep: int, dst: PagedCache, index, dst_len, workspace=None,
             sink: int = 0, recent: int = 0, dst_weights=None, stream=None) -> None:
    """Keep at most ``keep`` tokens a sequence and KV head (the first ``sink``, the last
    ``recent``, then those of the largest ``weights``) and move them into the pages of ``dst``.
    index: int32 [B, Hkv, keep]; dst_len: int32 [B]; dst_weights: fp32 [B, Hkv, >= keep] or None."""
    c, device = batch.cache, _here(batch)
    _here(dst, "dst")
    _int32(keep=keep, sink=sink, recent=recent)
    pw, wld = _wide(weights, "weights", c, device)
    pi = _tensor(index, "index", _torch.int32, (c.B, c.Hkv, keep), device)
    pn = _tensor(dst_len, "dst_len", _torch.int32, (c.B,), device)
    pd, ld = (None, 0) if dst_weights is None else _wide(dst_weights, "dst_weights", c, device)
    ws, size = _workspace(workspace, device)
    # the table may have room for more tokens than a shape can state: it holds `keep` or what it can
    room = min(dst.max_pages * dst.page_size, keep)
    shape = fa_paged_shape(dst.B, dst.Hkv, dst.Hkv, HEAD_DIM, dst.page_size, dst.num_pages,
                           dst.max_pages, 0, 0, room)
    cache = fa_paged_cache(*dst.pointers, None, None)
    _check(LIB.fa_evict(*batch.refs, pw, wld, keep, sink, recent, ctypes.byref(shape),
                        ctypes.byref(cache), pd, ld, pi, pn, ws, size, _raw_stream(stream, device)))


def fa_device_status(stream=None) -> None:
    _check(LIB.fa_device_status(_stream(stream)))


def fa_watchdog_selftest(wait_ns: int = 20_000_000, stream=None) -> None:
    """Launch a kernel whose bounded wait must expire (see the C header)."""
    _check(LIB.fa_watchdog_selftest(wait_ns, _stream(stream)))


# ----------------------------------------------------------------------------- marshalling helpers

class Cache:
    """Device buffers of one layer's hybrid cache (allocated by torch) + the C struct.
    F and E are bf16, C is fp32 (see fa_plan in the header)."""

    def __init__(self, plan: fa_plan, device="cuda"):
        import torch
        bf = torch.bfloat16
        self.plan = plan
        self.F_K = torch.empty(max(plan.f_elems, 8), dtype=bf, device=device)
        self.F_V = torch.empty_like(self.F_K)
        self.E_K = torch.empty(max(plan.e_elems, 8), dtype=bf, device=device)
        self.E_V = torch.empty_like(self.E_K)
        self.C_K = torch.empty(max(plan.c_elems, 8), dtype=torch.float32, device=device)
        self.C_V = torch.empty_like(self.C_K)
        self.c = fa_cache(*(t.data_ptr() for t in (self.F_K, self.F_V, self.E_K, self.E_V,
                                                  self.C_K, self.C_V)))

    # views in the documented layouts (for tests and callers that inspect the cache)
    def F(self, which: str):
        """[B, Hkv, S + R, 128]: sink rows, then the recent ring (oldest at S + recent_head)."""
        p = self.plan
        t = self.F_K if which == "K" else self.F_V
        return t[:p.f_elems].view(p.shape.B, p.shape.Hkv, p.S + p.R, HEAD_DIM)

    def F_tokens(self, which: str):
        """[B, Hkv, S + R, 128]: the sink rows, then the recent rows in token order (the ring
        rotated so that its oldest row comes first). A copy, not a view."""
        import torch
        p = self.plan
        F = self.F(which)
        if p.R == 0 or p.recent_head == 0:
            return F.clone()
        idx = list(range(p.S)) + [p.S + (p.recent_head + a) % p.R for a in range(p.R)]
        return F[:, :, torch.tensor(idx, device=F.device)]

    def E(self, which: str, b: int, g: int):
        return self.E_raw(which, b, g)[:, :self.plan.de[g]]

    def C(self, which: str, b: int, g: int):
        p = self.plan
        t = self.C_K if which == "K" else self.C_V
        off = b * p.c_batch + p.c_off[g]
        return t[off:off + p.kk * p.dc_ld[g]].view(p.kk, p.dc_ld[g])[:, :p.dc[g]]

    def E_raw(self, which: str, b: int, g: int):
        """[M, de_ld] view of KV head (b, g)'s middle rows (strided when E is token-major)."""
        p = self.plan
        t = self.E_K if which == "K" else self.E_V
        off = b * p.e_batch + p.e_off[g]
        return t.as_strided((p.M, p.de_ld[g]), (p.e_pitch[g], 1), t.storage_offset() + off)

    def C_raw(self, which: str, b: int, g: int):
        p = self.plan
        t = self.C_K if which == "K" else self.C_V
        off = b * p.c_batch + p.c_off[g]
        return t[off:off + p.kk * p.dc_ld[g]].view(p.kk, p.dc_ld[g])


def basis_table(plan: fa_plan, device="cuda", stream=None):
    """Allocate and fill the bf16 basis table (period P) fa_compress reads (None if M == 0)."""
    import torch
    if plan.M == 0:
        return None
    phiT = torch.empty(plan.shape.k, plan.phi_ld, dtype=torch.bfloat16, device=device)
    fa_build_basis(plan.P, plan.shape.k, phiT, plan.phi_ld, normalized=False, stream=stream)
    return phiT


def perm_lists(plan: fa_plan, g: int):
    """(compressed dims, retained dims) of KV head g, as the plan derived them."""
    perm = np.frombuffer(bytes(plan.perm[g]), dtype=np.uint8).astype(np.int64)
    return perm[:plan.dc[g]], perm[plan.dc[g]:]
