"""GB300 sparse multi-head attention: Python binding of ``libgtattn.so``.

A thin ctypes layer over the C ABI declared in ``include/gtattn.h``: each
function has the C entry point's name and arguments, takes torch CUDA tensors
(or raw device pointers as ints) and raises :class:`GtattnError` on a non-OK
status.  It only marshals arguments; every step runs in the library's CUDA
kernels.  There is no CPU fallback: without the built library (or without a
GPU) the calls raise.

    out[i,h,:] = sum_{e in row i} softmax_e(scale * q_i . k_j) v_j

over a CSR graph keyed by destination (row i attends over
indices[indptr[i]:indptr[i+1]]); empty rows give zeros.
"""
from __future__ import annotations

import ctypes
import os
import threading

from ._build import LIB, build

__all__ = [
    "GtattnError", "Plan", "build", "load", "gtattn_fwd", "gtattn_fwd_plan", "gtattn_fwd_probs", "gtattn_fwd_bias", "gtattn_fwd_weighted", "gtattn_bwd", "gtattn_fwd_ndh",
    "gtattn_fwd_noalloc", "gtattn_fwd_host", "gtattn_fwd_proj", "gtattn_device_errors", "gtattn_bwd_plan",
    "gtattn_fwd_plan_stats", "gtattn_csr_build",
    "gtattn_plan_destroy", "gtattn_plan_get_info", "gtattn_coo_to_csr",
    "gtattn_csr_validate", "gtattn_status_string", "gtattn_profile_enable", "gtattn_profile_read",
    "sparse_mha", "GTATTN_F32", "GTATTN_BF16", "GTATTN_BF16_OUT_F32",
    "GTATTN_KERNEL_AUTO", "GTATTN_KERNEL_VECTOR", "GTATTN_KERNEL_GENERIC", "GTATTN_KERNEL_NARROW",
    "Cache", "gtattn_cache_slots", "gtattn_cache_append", "gtattn_cache_select", "gtattn_fwd_cache",
    "EXPORTED_SYMBOLS",
]

GTATTN_OK, GTATTN_ERR_INVALID_ARG, GTATTN_ERR_BAD_CSR, GTATTN_ERR_UNSUPPORTED = 0, 1, 2, 3
GTATTN_ERR_CUDA, GTATTN_ERR_NO_MEMORY, GTATTN_ERR_TIMEOUT = 4, 5, 6
GTATTN_F32, GTATTN_BF16, GTATTN_BF16_OUT_F32 = 0, 1, 2
GTATTN_KERNEL_AUTO, GTATTN_KERNEL_VECTOR, GTATTN_KERNEL_GENERIC, GTATTN_KERNEL_NARROW = 0, 1, 2, 3

EXPORTED_SYMBOLS = (
    "gtattn_status_string", "gtattn_last_error", "gtattn_csr_build", "gtattn_plan_destroy",
    "gtattn_plan_get_info", "gtattn_fwd", "gtattn_fwd_plan", "gtattn_fwd_probs",
    "gtattn_coo_to_csr", "gtattn_csr_validate", "gtattn_profile_enable", "gtattn_profile_read",
    "gtattn_fwd_noalloc", "gtattn_fwd_host", "gtattn_fwd_bias", "gtattn_fwd_weighted", "gtattn_bwd",
    "gtattn_fwd_ndh", "gtattn_fwd_proj", "gtattn_device_errors", "gtattn_bwd_plan", "gtattn_fwd_plan_stats",
    "gtattn_cache_slots", "gtattn_cache_append", "gtattn_cache_select", "gtattn_fwd_cache",
)
KCAT_NAMES = ("bin", "rows", "combine", "softmax", "dense", "gemm", "cache")


class GtattnError(RuntimeError):
    def __init__(self, status: int, what: str, detail: str = ""):
        self.status = status
        msg = f"{what}: {gtattn_status_string(status)} ({status})"
        if detail:
            msg += f": {detail}"
        super().__init__(msg)


class PlanOpts(ctypes.Structure):
    _fields_ = [("long_row_min", ctypes.c_int32), ("chunk_edges", ctypes.c_int32),
                ("detect_dense", ctypes.c_int32), ("kernel", ctypes.c_int32), ("wait_cycles", ctypes.c_int32),
                ("test_stall", ctypes.c_int32)]


class PlanInfo(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("nnz", ctypes.c_int64), ("n_long_rows", ctypes.c_int32),
                ("n_chunks", ctypes.c_int32), ("n_dense_blocks", ctypes.c_int32),
                ("n_dense_rows", ctypes.c_int32), ("n_empty_rows", ctypes.c_int32),
                ("max_degree", ctypes.c_int32), ("n_buckets", ctypes.c_int32),
                ("bucket_rows", ctypes.c_int32 * 64), ("device_error", ctypes.c_int32)]

    def as_dict(self):
        d = {k: getattr(self, k) for k, _ in self._fields_ if k != "bucket_rows"}
        d["bucket_rows"] = list(self.bucket_rows)[: self.n_buckets]
        return d


class Profile(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_int32 * 8), ("groups", ctypes.c_int32 * 8),
                ("ms", ctypes.c_double * 8)]


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k8", ctypes.c_void_p), ("v8", ctypes.c_void_p), ("kscale", ctypes.c_void_p),
                ("vscale", ctypes.c_void_p), ("kmean", ctypes.c_void_p), ("pages", ctypes.c_int32),
                ("page", ctypes.c_int32), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def load(path: str | None = None):
    """Load ``libgtattn.so`` (building it first if it is missing) and
    declare the C signatures.  Raises if it cannot be built or loaded."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB
        if not os.path.exists(p):
            build()
        lib = ctypes.CDLL(p)
        vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        sig = {
            "gtattn_status_string": ([i32], ctypes.c_char_p),
            "gtattn_last_error": ([], ctypes.c_char_p),
            "gtattn_csr_build": ([vp, vp, i64, i64, vp, vp, vp], i32),
            "gtattn_plan_destroy": ([vp], i32),
            "gtattn_plan_get_info": ([vp, vp], i32),
            "gtattn_fwd": ([vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, i32, vp], i32),
            "gtattn_fwd_plan": ([vp, vp, vp, vp, vp, vp, vp, i32, i32, f32, i32, vp], i32),
            "gtattn_fwd_probs": ([vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, i32, vp], i32),
            "gtattn_fwd_bias": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, i32, vp], i32),
            "gtattn_fwd_weighted": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, i32, vp], i32),
            "gtattn_bwd": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, i32, vp], i32),
            "gtattn_fwd_ndh": ([vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, i32, vp], i32),
            "gtattn_coo_to_csr": ([vp, vp, i64, i64, vp, vp, vp], i32),
            "gtattn_csr_validate": ([vp, vp, i64, i64, vp], i32),
            "gtattn_fwd_noalloc": ([vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, i32, vp], i32),
            "gtattn_fwd_host": ([vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, f32, i32, vp], i32),
            "gtattn_fwd_proj": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i32, i32, i32, i32, i32, f32,
                                 i32, vp], i32),
            "gtattn_device_errors": ([vp, i32], i32),
            "gtattn_bwd_plan": ([vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, f32, i32, vp], i32),
            "gtattn_fwd_plan_stats": ([vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, f32, i32, vp], i32),
            "gtattn_cache_slots": ([vp, vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, i32, vp], i32),
            "gtattn_cache_append": ([vp, vp, vp, vp, i64, i32, vp], i32),
            "gtattn_cache_select": ([vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, i32, vp], i32),
            "gtattn_fwd_cache": ([vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, i32, f32, i32, vp], i32),
            "gtattn_profile_enable": ([i32], i32),
            "gtattn_profile_read": ([vp, i32], i32),
        }
        for name, (args, res) in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
        return lib


def gtattn_status_string(status: int) -> str:
    try:
        return load().gtattn_status_string(int(status)).decode()
    except OSError:
        return str(status)


# --------------------------------------------------------------------------
# marshalling helpers
# --------------------------------------------------------------------------
def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if x.numel() and not x.is_cuda:
            raise ValueError("expected a CUDA tensor")
        if not x.is_contiguous():
            raise ValueError("expected a contiguous tensor")
        return x.data_ptr() or None
    raise TypeError(f"cannot take a device pointer of {type(x)}")


def _host_ptr(x):
    """Pointer of a contiguous host (CPU) tensor, or None."""
    if x is None:
        return None
    if getattr(x, "is_cuda", False):
        raise ValueError("expected a host (CPU) tensor")
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return x.data_ptr() or None


def _stream(stream):
    if stream is None:
        import torch
        # (the raw handle: building a torch.cuda.Stream for it costs 3 us a call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(q, out=None):
    """gtattn_dtype of (Q, out): fp32/fp32, bf16/bf16 or bf16/fp32."""
    import torch
    if q.dtype == torch.float32 and (out is None or out.dtype == torch.float32):
        return GTATTN_F32
    if q.dtype == torch.bfloat16 and (out is None or out.dtype == torch.bfloat16):
        return GTATTN_BF16
    if q.dtype == torch.bfloat16 and out.dtype == torch.float32:
        return GTATTN_BF16_OUT_F32
    raise ValueError(f"unsupported dtypes {q.dtype} -> {None if out is None else out.dtype}")


def _check(status, what):
    if status != GTATTN_OK:
        detail = load().gtattn_last_error().decode() if status == GTATTN_ERR_CUDA else ""
        raise GtattnError(status, what, detail)


# --------------------------------------------------------------------------
# the C entry points
# --------------------------------------------------------------------------
def gtattn_fwd(indptr, indices, Q, K, V, out, N, nnz, H, D, scale, dtype, stream=None):
    _check(load().gtattn_fwd(_ptr(indptr), _ptr(indices), _ptr(Q), _ptr(K), _ptr(V), _ptr(out),
                             int(N), int(nnz), int(H), int(D), float(scale), int(dtype),
                             _stream(stream)), "gtattn_fwd")


def gtattn_fwd_noalloc(indptr, indices, Q, K, V, out, N, nnz, H, D, scale, dtype, stream=None):
    """gtattn_fwd for callers that cannot allocate device memory: temporaries
    live in the library's fixed 32 MiB device array (see include/gtattn.h for
    the size limit and why overlapping calls race)."""
    _check(load().gtattn_fwd_noalloc(_ptr(indptr), _ptr(indices), _ptr(Q), _ptr(K), _ptr(V), _ptr(out),
                                     int(N), int(nnz), int(H), int(D), float(scale), int(dtype),
                                     _stream(stream)), "gtattn_fwd_noalloc")


def gtattn_fwd_host(indptr, indices, Q, K, V, out, N, nnz, H, D, scale, dtype, stream=None):
    """gtattn_fwd on host (CPU, preferably pinned) tensors: copies in,
    computes and copies the output back, overlapped, ordered on `stream`;
    `out` is complete once `stream` has passed the call."""
    _check(load().gtattn_fwd_host(_host_ptr(indptr), _host_ptr(indices), _host_ptr(Q), _host_ptr(K),
                                  _host_ptr(V), _host_ptr(out),
                                  int(N), int(nnz), int(H), int(D), float(scale), int(dtype),
                                  _stream(stream)), "gtattn_fwd_host")


def gtattn_fwd_proj(indptr, indices, X, Wqkv, bqkv, Wo, bo, Y, N, nnz, F_in, H, D, F_out, scale, dtype,
                    heads_inner=False, qkv=None, attn=None, stream=None):
    """The attention block with its projections: q, k, v = X Wqkv^T + bqkv
    (weights of the three maps stacked, nn.Linear layout), the sparse
    attention, Y = o Wo^T + bo.  bqkv / bo: fp32 device tensors or None;
    qkv ([3, N, H, D]) and attn ([N, H, D]) optionally receive the
    intermediates; heads_inner: SparseMHA's feature order (d*H + h)."""
    _check(load().gtattn_fwd_proj(_ptr(indptr), _ptr(indices), _ptr(X), _ptr(Wqkv), _ptr(bqkv), _ptr(Wo), _ptr(bo),
                                  _ptr(Y), _ptr(qkv), _ptr(attn), int(N), int(nnz), int(F_in), int(H), int(D),
                                  int(F_out), 1 if heads_inner else 0, float(scale), int(dtype), _stream(stream)),
           "gtattn_fwd_proj")


def gtattn_bwd_plan(plan, indptr, indices, Q, K, V, dO, dQ, dK, dV, H, D, scale, dtype, O=None, stats=None,
                    stream=None):
    """gtattn_bwd on a plan's binning; the plan keeps the source-major
    pattern built by its first backward call.  O and stats: the fp32 output
    and row statistics of gtattn_fwd_plan_stats (both or neither); given,
    the forward is not recomputed."""
    _check(load().gtattn_bwd_plan(plan.handle if isinstance(plan, Plan) else plan, _ptr(indptr), _ptr(indices),
                                  _ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(stats), _ptr(dO), _ptr(dQ), _ptr(dK),
                                  _ptr(dV), int(H), int(D), float(scale), int(dtype), _stream(stream)),
           "gtattn_bwd_plan")


def gtattn_device_errors(reset: bool = True) -> int:
    """Error codes recorded on the current device by the plan-less
    tensor-core kernels (1: a bounded wait gave up); synchronises."""
    code = ctypes.c_int(0)
    _check(load().gtattn_device_errors(ctypes.byref(code), 1 if reset else 0), "gtattn_device_errors")
    return code.value


def gtattn_fwd_plan(plan, indptr, indices, Q, K, V, out, H, D, scale, dtype, stream=None):
    _check(load().gtattn_fwd_plan(plan.handle if isinstance(plan, Plan) else plan, _ptr(indptr),
                                  _ptr(indices), _ptr(Q), _ptr(K), _ptr(V), _ptr(out), int(H), int(D),
                                  float(scale), int(dtype), _stream(stream)), "gtattn_fwd_plan")


def gtattn_fwd_plan_stats(plan, indptr, indices, Q, K, V, out, stats, H, D, scale, dtype, stream=None):
    """gtattn_fwd_plan that also writes the rows' log2-sum-exp (fp32 [N, H])."""
    _check(load().gtattn_fwd_plan_stats(plan.handle if isinstance(plan, Plan) else plan, _ptr(indptr),
                                        _ptr(indices), _ptr(Q), _ptr(K), _ptr(V), _ptr(out), _ptr(stats), int(H),
                                        int(D), float(scale), int(dtype), _stream(stream)),
           "gtattn_fwd_plan_stats")


def gtattn_fwd_probs(indptr, indices, Q, K, V, out, logits, probs, N, nnz, H, D, scale, dtype,
                     stream=None):
    _check(load().gtattn_fwd_probs(_ptr(indptr), _ptr(indices), _ptr(Q), _ptr(K), _ptr(V), _ptr(out),
                                   _ptr(logits), _ptr(probs), int(N), int(nnz), int(H), int(D),
                                   float(scale), int(dtype), _stream(stream)), "gtattn_fwd_probs")


def gtattn_fwd_bias(indptr, indices, Q, K, V, bias, out, N, nnz, H, D, scale, dtype, logits=None, probs=None,
                    stream=None):
    """Forward with a per-edge, per-head additive bias (fp32 [nnz, H] device
    tensor); logits/probs (optional) select the unfused path."""
    _check(load().gtattn_fwd_bias(_ptr(indptr), _ptr(indices), _ptr(Q), _ptr(K), _ptr(V), _ptr(bias), _ptr(out),
                                  _ptr(logits), _ptr(probs), int(N), int(nnz), int(H), int(D), float(scale),
                                  int(dtype), _stream(stream)), "gtattn_fwd_bias")


def gtattn_fwd_weighted(indptr, indices, values, Q, K, V, out, N, nnz, H, D, scale, dtype, logits=None, probs=None,
                        stream=None):
    """Forward on a weighted adjacency (values: fp32 [nnz] device tensor, A's
    stored values); logits/probs (optional) select the unfused path."""
    _check(load().gtattn_fwd_weighted(_ptr(indptr), _ptr(indices), _ptr(values), _ptr(Q), _ptr(K), _ptr(V),
                                      _ptr(out), _ptr(logits), _ptr(probs), int(N), int(nnz), int(H), int(D),
                                      float(scale), int(dtype), _stream(stream)), "gtattn_fwd_weighted")


def gtattn_bwd(indptr, indices, Q, K, V, dO, dQ, dK, dV, N, nnz, H, D, scale, dtype, stream=None):
    """Gradients of sum(out * dO) with respect to Q, K, V (fp32 device tensors
    dQ, dK, dV, overwritten)."""
    _check(load().gtattn_bwd(_ptr(indptr), _ptr(indices), _ptr(Q), _ptr(K), _ptr(V), _ptr(dO), _ptr(dQ), _ptr(dK),
                             _ptr(dV), int(N), int(nnz), int(H), int(D), float(scale), int(dtype), _stream(stream)),
           "gtattn_bwd")


def gtattn_fwd_ndh(indptr, indices, Q, K, V, out, N, nnz, H, D, scale, dtype, stream=None):
    """gtattn_fwd on head-innermost [N, D, H] tensors."""
    _check(load().gtattn_fwd_ndh(_ptr(indptr), _ptr(indices), _ptr(Q), _ptr(K), _ptr(V), _ptr(out), int(N), int(nnz),
                                 int(H), int(D), float(scale), int(dtype), _stream(stream)), "gtattn_fwd_ndh")


def gtattn_csr_build(indptr, indices, N, nnz, opts=None, stream=None):
    """Returns a raw plan handle (int); prefer :class:`Plan`."""
    h = ctypes.c_void_p()
    o = ctypes.byref(opts) if opts is not None else None
    _check(load().gtattn_csr_build(_ptr(indptr), _ptr(indices), int(N), int(nnz), o, ctypes.byref(h),
                                   _stream(stream)), "gtattn_csr_build")
    return h.value


def gtattn_plan_destroy(handle):
    _check(load().gtattn_plan_destroy(handle), "gtattn_plan_destroy")


def gtattn_plan_get_info(handle) -> dict:
    info = PlanInfo()
    _check(load().gtattn_plan_get_info(handle, ctypes.byref(info)), "gtattn_plan_get_info")
    return info.as_dict()


def gtattn_coo_to_csr(src, dst, nnz, N, indptr, indices, stream=None):
    _check(load().gtattn_coo_to_csr(_ptr(src), _ptr(dst), int(nnz), int(N), _ptr(indptr), _ptr(indices),
                                    _stream(stream)), "gtattn_coo_to_csr")


def gtattn_csr_validate(indptr, indices, N, nnz, stream=None) -> bool:
    """True for a well-formed CSR, False for GTATTN_ERR_BAD_CSR; raises otherwise."""
    st = load().gtattn_csr_validate(_ptr(indptr), _ptr(indices), int(N), int(nnz), _stream(stream))
    if st == GTATTN_ERR_BAD_CSR:
        return False
    _check(st, "gtattn_csr_validate")
    return True


def gtattn_profile_enable(on: bool = True):
    _check(load().gtattn_profile_enable(int(bool(on))), "gtattn_profile_enable")


def gtattn_profile_read(reset: bool = True) -> dict:
    """Per-category kernel launches and summed CUDA-event milliseconds
    recorded while profiling was enabled."""
    pr = Profile()
    _check(load().gtattn_profile_read(ctypes.byref(pr), int(bool(reset))), "gtattn_profile_read")
    return {name: dict(launches=pr.launches[k], groups=pr.groups[k], ms=pr.ms[k])
            for k, name in enumerate(KCAT_NAMES)}


class Plan:
    """Owns a plan built by ``gtattn_csr_build`` (freed on close/GC)."""

    def __init__(self, indptr, indices, N=None, nnz=None, long_row_min=0, chunk_edges=0,
                 detect_dense=False, kernel=GTATTN_KERNEL_AUTO, wait_cycles=0, test_stall=False,
                 stream=None):
        N = int(indptr.numel() - 1) if N is None else int(N)
        nnz = int(indices.numel()) if nnz is None else int(nnz)
        self.opts = PlanOpts(int(long_row_min), int(chunk_edges), int(bool(detect_dense)), int(kernel),
                             int(wait_cycles), int(bool(test_stall)))
        self.handle = gtattn_csr_build(indptr, indices, N, nnz, self.opts, stream)
        self.N, self.nnz = N, nnz
        self._keep = (indptr, indices)

    def info(self) -> dict:
        return gtattn_plan_get_info(self.handle)

    def close(self):
        if getattr(self, "handle", None):
            gtattn_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# --------------------------------------------------------------------------
# the 8-bit K/V cache
# --------------------------------------------------------------------------
class Cache:
    """A K/V cache held in 8 bits (``gtattn_cache``): the tensors it is made of.

    k8, v8: e4m3 codes [pages, Hkv, page, D] (torch.float8_e4m3fn or uint8);
    kscale, vscale: fp32 [pages, Hkv]; kmean: bf16 [pages, Hkv, D] or None.
    Any of them may be None where no call needs it (k8, or kmean and
    ``page``, give the sizes).  The tensors stay the caller's: calls write
    into them, and the object keeps them alive."""

    def __init__(self, k8, v8, kscale, vscale, kmean=None, page=None):
        import torch
        if k8 is not None:
            pages, Hkv, tokens, D = k8.shape
            if page is not None and int(page) != tokens:
                raise ValueError(f"page is {page}, the tiles hold {tokens} tokens")
        elif kmean is not None and page is not None:
            (pages, Hkv, D), tokens = kmean.shape, int(page)
        else:
            raise ValueError("give k8, or kmean and page")
        codes = (torch.float8_e4m3fn, torch.uint8)
        dev = None
        for name, x, shape, dtypes in (("k8", k8, (pages, Hkv, tokens, D), codes),
                                       ("v8", v8, (pages, Hkv, tokens, D), codes),
                                       ("kscale", kscale, (pages, Hkv), (torch.float32,)),
                                       ("vscale", vscale, (pages, Hkv), (torch.float32,)),
                                       ("kmean", kmean, (pages, Hkv, D), (torch.bfloat16,))):
            if x is None:
                continue
            if tuple(x.shape) != shape or x.dtype not in dtypes:
                raise ValueError(f"{name}: expected {shape} of {dtypes[0]}, got {tuple(x.shape)} of {x.dtype}")
            if dev is not None and x.device != dev:
                raise ValueError(f"{name} is on {x.device}, the cache on {dev}")
            dev = x.device
        self.k8, self.v8, self.kscale, self.vscale, self.kmean = k8, v8, kscale, vscale, kmean
        self.pages, self.Hkv, self.page, self.D = pages, Hkv, tokens, D
        self.device = dev
        self._struct = _CacheStruct(_ptr(k8), _ptr(v8), _ptr(kscale), _ptr(vscale), _ptr(kmean), pages, tokens, Hkv, D)
        self._ref = ctypes.addressof(self._struct)
        self._dev = dev.index if dev.type == "cuda" else -1

    @classmethod
    def empty(cls, pages, Hkv, D, page=64, device="cuda", means=True):
        """A cache of unused pages (``means``: with the page means that
        gtattn_cache_select reads)."""
        import torch
        tile = (int(pages), int(Hkv), int(page), int(D))
        k8, v8 = (torch.zeros(tile, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn) for _ in range(2))
        ks, vs = (torch.zeros(tile[:2], dtype=torch.float32, device=device) for _ in range(2))
        km = torch.zeros(tile[0], tile[1], tile[3], dtype=torch.bfloat16, device=device) if means else None
        return cls(k8, v8, ks, vs, km)


def _arg(x, name, least, dtypes, dev):
    """Device pointer of a contiguous CUDA tensor on device ``dev`` with at
    least ``least`` elements of one of ``dtypes`` (ints pass as pointers)."""
    if x is None or isinstance(x, int):
        return x
    if x.dtype in dtypes and x.numel() >= least and x.is_contiguous() and x.get_device() == dev:
        return x.data_ptr() or None
    if x.dtype not in dtypes:
        raise ValueError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {x.dtype}")
    n = x.numel()
    if n < least:
        raise ValueError(f"{name}: expected at least {least} elements, got {n}")
    if n and x.get_device() != dev:
        raise ValueError(f"{name} is on {x.device}, the call runs on cuda:{dev}")
    if not x.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return x.data_ptr() or None


_types_of = None       # gtattn_dtype -> (input, output) torch dtypes; None -> int32's; as tuples for _arg


def _call(cache, dtype, stream):
    """(library, current device, int32, input and output types, stream) of a
    cache call; the cache has to be on the current device."""
    global _types_of
    import torch
    if _types_of is None:
        f, b = (torch.float32,), (torch.bfloat16,)
        _types_of = {None: (None, None), GTATTN_F32: (f, f), GTATTN_BF16: (b, b), GTATTN_BF16_OUT_F32: (b, f),
                     "i32": (torch.int32,)}
    if dtype not in _types_of:
        raise GtattnError(GTATTN_ERR_INVALID_ARG, "dtype")
    dev = torch.cuda.current_device()
    if cache is not None and cache._dev != dev:
        raise ValueError(f"the cache is on {cache.device}, the call runs on cuda:{dev}")
    ti, to = _types_of[dtype]
    s = torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)
    return _lib or load(), dev, _types_of["i32"], ti, to, s


def gtattn_cache_slots(length, add, table, free_pages, new_length, tok_off, slots, counts, S, max_pages, n_free, T, page,
                       stream=None):
    """Pages and slots for the tokens that S requests add: takes pages from
    ``free_pages`` into ``table`` [S, max_pages], writes ``new_length`` [S],
    ``tok_off`` [S+1], ``slots`` [T] (-1: no place) and ``counts`` [3] (pages
    taken, rows, requests refused); all int32 CUDA tensors."""
    lib, dev, i, _, _, stream = _call(None, None, stream)
    _check(lib.gtattn_cache_slots(
        _arg(length, "length", S, i, dev), _arg(add, "add", S, i, dev), _arg(table, "table", S * max_pages, i, dev),
        _arg(free_pages, "free_pages", n_free, i, dev), _arg(new_length, "new_length", S, i, dev),
        _arg(tok_off, "tok_off", S + 1, i, dev), _arg(slots, "slots", T, i, dev), _arg(counts, "counts", 3, i, dev),
        S, max_pages, n_free, T, page, stream), "gtattn_cache_slots")


def gtattn_cache_append(cache, K, V, slots, T, dtype, stream=None):
    """Stores the keys and values [T, Hkv, D] of T tokens in the cache's
    ``slots`` (int32 [T], as gtattn_cache_slots lists them), in 8 bits."""
    lib, dev, i, t, _, stream = _call(cache, dtype, stream)
    n = T * cache.Hkv * cache.D
    _check(lib.gtattn_cache_append(cache._ref, _arg(K, "K", n, t, dev), _arg(V, "V", n, t, dev),
                                   _arg(slots, "slots", T, i, dev), T, dtype, stream), "gtattn_cache_append")


def gtattn_cache_select(cache, Q, table, length, tok_off, sel, S, T, max_pages, H, n_sel, dtype, stream=None):
    """The pages each row and K/V head reads: its own and the n_sel - 1
    earlier ones whose mean key scores highest; ``sel`` [T, Hkv, n_sel]
    int32, ascending, -1 where there are fewer."""
    lib, dev, i, t, _, stream = _call(cache, dtype, stream)
    _check(lib.gtattn_cache_select(
        cache._ref, _arg(Q, "Q", T * H * cache.D, t, dev), _arg(table, "table", S * max_pages, i, dev),
        _arg(length, "length", S, i, dev), _arg(tok_off, "tok_off", S + 1, i, dev),
        _arg(sel, "sel", T * cache.Hkv * n_sel, i, dev), S, T, max_pages, H, n_sel, dtype, stream),
        "gtattn_cache_select")


def gtattn_fwd_cache(cache, Q, table, length, tok_off, out, S, T, max_pages, H, scale, dtype, sel=None, n_sel=0,
                     stream=None):
    """Attention of T new rows Q [T, H, D] over the cache: all tokens of
    their request up to each row's position, or those in the pages ``sel``
    ([T, Hkv, n_sel] int32) names."""
    lib, dev, i, ti, to, stream = _call(cache, dtype, stream)
    n = T * H * cache.D
    _check(lib.gtattn_fwd_cache(
        cache._ref, _arg(Q, "Q", n, ti, dev), _arg(table, "table", S * max_pages, i, dev),
        _arg(length, "length", S, i, dev), _arg(tok_off, "tok_off", S + 1, i, dev),
        _arg(sel, "sel", T * cache.Hkv * n_sel, i, dev), _arg(out, "out", n, to, dev), S, T, max_pages, H, n_sel, scale,
        dtype, stream), "gtattn_fwd_cache")


def sparse_mha(indptr, indices, Q, K, V, scale=None, out=None, plan=None, stream=None):
    """Convenience wrapper: allocates ``out`` and calls ``gtattn_fwd`` (or
    ``gtattn_fwd_plan`` when a :class:`Plan` is given)."""
    import torch
    N, H, D = Q.shape
    if scale is None:
        scale = 1.0 / float(D) ** 0.5
    if out is None:
        out = torch.empty_like(Q)
    dt = _dtype_code(Q, out)
    if plan is not None:
        gtattn_fwd_plan(plan, indptr, indices, Q, K, V, out, H, D, scale, dt, stream)
    else:
        gtattn_fwd(indptr, indices, Q, K, V, out, N, indices.numel(), H, D, scale, dt, stream)
    return out
