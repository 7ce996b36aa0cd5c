"""Python binding of libbskv: CSR-indexed sparse and paged attention on one GB300.

A thin ctypes layer over the C ABI declared in include/bskv.h. Functions carry the
C names; they marshal torch tensors into pointers, strides and the current CUDA
stream, allocate outputs and workspaces with torch when the caller does not pass
them, and raise on any non-OK status. Every step of the computation runs in the
library's CUDA kernels; there is no CPU fallback. Importing works without a GPU
(plans are host code), but the library must have been built (``build()``).
"""

import ctypes
import os

import torch

from . import build as _build

__all__ = [
    "BskvError", "Plan", "load_library", "build",
    "bskv_version", "bskv_last_error_message",
    "bskv_plan_decode", "bskv_plan_bsr", "bskv_plan_mla_sparse",
    "bskv_run_decode", "bskv_run_decode_partial", "bskv_decode_merge", "bskv_run_decode_noalloc",
    "bskv_run_bsr", "bskv_run_mla_sparse",
    "bskv_plan_decode_fp4", "bskv_run_decode_fp4",
    "bskv_quantize_fp4_append_paged", "bskv_dequantize_fp4_paged",
    "bskv_plan_attn_weights", "bskv_run_attn_weights", "bskv_run_attn_weights_fp4",
    "bskv_plan_evict", "bskv_run_evict", "bskv_run_evict_fp4",
    "PageTable", "bskv_build_page_table", "bskv_norm_rope_append_paged", "bskv_block_bounds_paged",
    "bskv_plan_decode_blocks", "bskv_run_select_blocks", "bskv_run_decode_blocks",
    "bskv_rope_quantize_fp8", "bskv_merge_states",
    "bskv_get_device_status", "bskv_set_debug_force_timeout",
]

FP16, BF16, FP32, E4M3, INT32, INT64 = range(6)
STATUS = {0: "OK", 1: "ERR_INVALID_ARG", 2: "ERR_UNSUPPORTED", 3: "ERR_WORKSPACE_TOO_SMALL",
          4: "ERR_CUDA", 5: "ERR_TIMEOUT", 6: "ERR_DEVICE_INDEX"}

_DT = {torch.float16: FP16, torch.bfloat16: BF16, torch.float32: FP32, torch.int32: INT32,
       torch.int64: INT64}
if hasattr(torch, "float8_e4m3fn"):
    _DT[torch.float8_e4m3fn] = E4M3


class BskvError(RuntimeError):
    def __init__(self, fn, code, msg):
        super().__init__("%s -> %s: %s" % (fn, STATUS.get(code, code), msg))
        self.code = code
        self.status = STATUS.get(code, str(code))


_lib = None
_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_I64P = ctypes.POINTER(ctypes.c_int64)
_I32P = ctypes.POINTER(ctypes.c_int32)

_SIGS = {
    "bskv_version": ([], _I32),
    "bskv_last_error_message": ([], ctypes.c_char_p),
    "bskv_plan_decode": ([_I32P, _I32P, _I32P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                          _I32, ctypes.POINTER(_P)], _I32),
    "bskv_plan_bsr": ([_I32P, _I32P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                       ctypes.POINTER(_P)], _I32),
    "bskv_plan_prefill_paged": ([_I32P, _I32P, _I32P, _I32P, _I32, _I32, _I32, _I32, _I32,
                                 _I32, _I32, _I32, _I32, ctypes.POINTER(_P)], _I32),
    "bskv_run_prefill_paged": ([_P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _F, _P], _I32),
    "bskv_plan_bsr_variable": ([_P, _I32P, _I32P, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                _I32, ctypes.POINTER(_P)], _I32),
    "bskv_run_bsr_variable": ([_P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _F, _P],
                              _I32),
    "bskv_plan_bsr_masked": ([_I32P, _I32P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                              ctypes.POINTER(_P)], _I32),
    "bskv_run_bsr_masked": ([_P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _SZ, _P, _I64P, _P, _F,
                             _P], _I32),
    "bskv_plan_mla_sparse": ([_I32P, _I32, _I32, _I32, _I32, _I32, ctypes.POINTER(_P)], _I32),
    "bskv_plan_mla_paged": ([_I32P, _I32P, _I32P, _I32, _I32, _I32, _I32, _I32,
                             ctypes.POINTER(_P)], _I32),
    "bskv_plan_destroy": ([_P], _I32),
    "bskv_plan_metadata": ([_P, ctypes.POINTER(_I32P), _I64P], _I32),
    "bskv_plan_workspace_sizes": ([_P, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)], _I32),
    "bskv_plan_upload": ([_P, _P, _SZ, _P], _I32),
    "bskv_run_decode": ([_P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _F, _P, _SZ, _P], _I32),
    "bskv_run_decode_partial": ([_P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _F, _P, _SZ, _P], _I32),
    "bskv_decode_merge": ([_P, _P, _I64P, _P, _P, _SZ, _P], _I32),
    "bskv_run_decode_noalloc": ([_P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _F, _P], _I32),
    "bskv_run_bsr": ([_P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _F, _P, _SZ, _P], _I32),
    "bskv_run_mla_sparse": ([_P, _P, _P, _I64, _P, _F, _F, _P, _P, _P, _SZ, _P], _I32),
    "bskv_run_mla_paged": ([_P, _P, _P, _F, _F, _P, _P, _P, _SZ, _P], _I32),
    "bskv_rope_quantize_fp8": ([_P, _I64P, _P, _I64P, _P, _I64, _I32, _P, _I64P, _P, _I64P,
                                _P, _I64, _P, _I64, _P, _I64, _P, _I64, _P, _I64,
                                _I32, _P, _I32, _I64, _I32, _F, _F, _P], _I32),
    "bskv_rope_quantize_fp8_append_paged": ([_P, _I64P, _P, _I64P, _P, _I64, _I32, _P, _I64P,
                                             _P, _I64P, _P, _I64, _P, _I64, _P, _I64, _P, _P,
                                             _P, _P, _I32, _I32, _I64, _P,
                                             _I32, _P, _I32, _I64, _I32, _F, _F, _P], _I32),
    "bskv_plan_decode_fp4": ([_I32P, _I32P, _I32P, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                              _I32, ctypes.POINTER(_P)], _I32),
    "bskv_run_decode_fp4": ([_P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _F, _P, _SZ, _P],
                            _I32),
    "bskv_quantize_fp4_append_paged": ([_P, _I64P, _P, _I64P, _I32, _I64, _I32, _I32, _P, _P, _P,
                                        _P, _I32, _I32, _I64, _P, _I64P, _P, _I64P, _P], _I32),
    "bskv_dequantize_fp4_paged": ([_P, _I64P, _P, _I64P, _P, _P, _P, _P, _I32, _I32, _I64, _P,
                                   _I64P, _P, _I64P, _I32, _I64, _I32, _I32, _P], _I32),
    "bskv_plan_attn_weights": ([_I32P, _I32P, _I32P, _I32P, _I32, _I32, _I32, _I32, _I32, _I32,
                                _I32, _I32, _I32, ctypes.POINTER(_P)], _I32),
    "bskv_run_attn_weights": ([_P, _P, _I64P, _P, _I64P, _P, _P, _I64P, _F, _F, _P], _I32),
    "bskv_run_attn_weights_fp4": ([_P, _P, _I64P, _P, _I64P, _P, _I64P, _P, _P, _I64P, _F, _F, _P],
                                  _I32),
    "bskv_plan_evict": ([_I32P, _I32P, _I32P, _I32P, _I32, _I32, _I32P, _I32P, _I32, _I32, _I32,
                         _I32, _I32, _I32, ctypes.POINTER(_P)], _I32),
    "bskv_run_evict": ([_P, _P, _I64P, _I32, _P, _I64P, _P, _P], _I32),
    "bskv_run_evict_fp4": ([_P, _P, _I64P, _I32, _P, _I64P, _P, _I64P, _P, _P], _I32),
    "bskv_build_page_table": ([_P, _P, _I32, _I32, _P, _I64, _I32, _I32, _P, _I32, _P, _P, _P, _P, _I64,
                               _P, _P, _P, _P, _P, _I64, _P], _I32),
    "bskv_norm_rope_append_paged": ([_P, _P, _P, _P, _P, _P, _I32, _I64, _I32, _I32, _I32, _P,
                                     _P, _F, _P, _I32, _I64, _I32, _I32, _P, _P, _P, _P, _P, _I32, _I32,
                                     _I64, _P, _P, _P, _P, _P], _I32),
    "bskv_block_bounds_paged": ([_P, _P, _I32, _I32, _I32, _I32, _I64, _P, _P, _I64, _P, _P, _P,
                                 _I32, _P, _P, _P], _I32),
    "bskv_plan_decode_blocks": ([_I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32, _I32,
                                 ctypes.POINTER(_P)], _I32),
    "bskv_run_select_blocks": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _SZ, _P], _I32),
    "bskv_run_decode_blocks": ([_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _F,
                                _P, _SZ, _P], _I32),
    "bskv_merge_states": ([_P, _P, _I64, _I32, _I32, _I32, _P, _I32, _P, _P], _I32),
    "bskv_get_device_status": ([_I32P, _I32], _I32),
    "bskv_set_debug_force_timeout": ([_I32], _I32),
}


def build(force=False):
    """Compile libbskv.so for sm_103a in-tree (nvcc) and load it."""
    global _lib
    _build.build(force=force)
    _lib = None
    return load_library()


def load_library():
    """Load libbskv.so; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_build.LIB):
        raise RuntimeError("libbskv.so is missing (%s): build it with "
                           "block_sparse_kv_gb300.build() first" % _build.LIB)
    lib = ctypes.CDLL(_build.LIB)
    for name, (args, res) in _SIGS.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(fn, code):
    if code != 0:
        msg = load_library().bskv_last_error_message().decode(errors="replace")
        raise BskvError(fn, code, msg)


def _i32_array(x):
    t = torch.as_tensor(x, dtype=torch.int32).contiguous().cpu()
    return t, t.data_ptr()


def _ptr(t):
    return None if t is None else t.data_ptr()


def _strides(*vals):
    return (ctypes.c_int64 * len(vals))(*[int(v) for v in vals])


def _stream(t=None):
    dev = t.device if t is not None and t.is_cuda else None
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)  # of an initialised CUDA
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _capturing(device):
    """Whether the device's current stream is being captured."""
    if torch.cuda.current_device() == device.index:
        return torch.cuda.is_current_stream_capturing()
    with torch.cuda.device(device):
        return torch.cuda.is_current_stream_capturing()


def _num_sms(device=None):
    if torch.cuda.is_available():
        d = torch.cuda.current_device() if device is None else torch.device(device).index or 0
        return torch.cuda.get_device_properties(d).multi_processor_count
    raise RuntimeError("num_sms must be given when no GPU is visible")


def bskv_version():
    return load_library().bskv_version()


def bskv_last_error_message():
    return load_library().bskv_last_error_message().decode(errors="replace")


class Plan:
    """Host plan handle plus (after upload) its device workspaces.

    A run on another stream than the upload's waits for the upload, and the workspaces' memory is
    not given to anyone else before the runs are done, also where the plan is dropped after a run.
    Runs of one plan share its workspaces: on several streams they have to be ordered by events.
    Captured runs are not ordered behind the upload (wait for it before the capture begins, as
    torch.cuda.graph does), and their graph needs the plan for as long as it is replayed."""

    def __init__(self, handle, kind, **info):
        self._h = ctypes.c_void_p(handle)
        self.kind = kind
        self.info = info
        self.layouts = {}  # of tensors that passed a run's checks
        self.int_ws = None
        self.float_ws = None
        self._uploaded = None    # event on the upload's stream
        self._streams = set()    # streams whose runs are ordered behind the upload

    def __del__(self):
        if getattr(self, "_h", None) and self._h.value and _lib is not None:
            _lib.bskv_plan_destroy(self._h)
            self._h = ctypes.c_void_p(None)

    @property
    def handle(self):
        return self._h

    def metadata(self):
        """The plan's int32 metadata words as a Python list."""
        lib = load_library()
        p = _I32P()
        n = ctypes.c_int64()
        _check("bskv_plan_metadata", lib.bskv_plan_metadata(self._h, ctypes.byref(p), ctypes.byref(n)))
        return [p[i] for i in range(n.value)]

    def workspace_sizes(self):
        lib = load_library()
        a, b = ctypes.c_size_t(), ctypes.c_size_t()
        _check("bskv_plan_workspace_sizes",
               lib.bskv_plan_workspace_sizes(self._h, ctypes.byref(a), ctypes.byref(b)))
        return a.value, b.value

    def upload(self, device="cuda", int_ws=None, float_ws=None):
        """Copy the metadata to the device (allocating the workspaces unless given)."""
        lib = load_library()
        ib, fb = self.workspace_sizes()
        if int_ws is None:
            int_ws = torch.empty(max(ib, 16), dtype=torch.uint8, device=device)
        if float_ws is None and fb > 0:
            float_ws = torch.empty(fb, dtype=torch.uint8, device=device)
        stream = torch.cuda.current_stream(int_ws.device)
        _check("bskv_plan_upload", lib.bskv_plan_upload(self._h, int_ws.data_ptr(), int_ws.numel(),
                                                        ctypes.c_void_p(stream.cuda_stream)))
        self.int_ws = int_ws
        self.float_ws = float_ws
        self._streams, self._uploaded = set(), None
        if not _capturing(int_ws.device):
            self._uploaded = torch.cuda.Event()
            self._uploaded.record(stream)
            self._streams.add(stream.cuda_stream)
        return self

    def on_stream(self, device):
        """Before a run on the current stream of the device: uploads at the first run, and lets a
        stream that is new to the plan wait for the upload."""
        if self.int_ws is None:
            self.upload(device)
        elif _raw_stream(device.index) not in self._streams:
            if self._uploaded is None or _capturing(device):
                return
            stream = torch.cuda.current_stream(device)
            stream.wait_event(self._uploaded)
            for ws in (self.int_ws, self.float_ws):
                if ws is not None:
                    ws.record_stream(stream)
            self._streams.add(stream.cuda_stream)


def bskv_plan_decode(kv_indptr, kv_indices, kv_last_page_len, num_pages, page_size,
                     num_qo_heads, num_kv_heads, head_dim, dtype=torch.bfloat16, num_sms=None,
                     max_workers=0):
    lib = load_library()
    ip, ipp = _i32_array(kv_indptr)
    ix, ixp = _i32_array(kv_indices)
    lp, lpp = _i32_array(kv_last_page_len)
    batch = ip.numel() - 1
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    _check("bskv_plan_decode", lib.bskv_plan_decode(
        ctypes.cast(ipp, _I32P), ctypes.cast(ixp, _I32P), ctypes.cast(lpp, _I32P), batch,
        int(num_pages), int(page_size), int(num_qo_heads), int(num_kv_heads), int(head_dim),
        _DT[dtype], int(ns), int(max_workers), ctypes.byref(h)))
    return Plan(h.value, "decode", batch=batch, num_qo_heads=num_qo_heads,
                num_kv_heads=num_kv_heads, head_dim=head_dim, dtype=dtype, page_size=page_size)


def bskv_run_decode(plan, q, kv_cache, out=None, lse=None, return_lse=False, sm_scale=None,
                    _entry="bskv_run_decode"):
    """Decode one query token per request; kv_cache [pages, 2, Hkv, page_size, D] (any
    strides with a contiguous last dim)."""
    lib = load_library()
    plan.on_stream(q.device)
    B, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((B, Hq), dtype=torch.float32, device=q.device)
    if sm_scale is None:
        sm_scale = 0.0  # the library applies 1/sqrt(head_dim)
    fw = plan.float_ws
    ks = kv_cache.stride()
    _check(_entry, getattr(lib, _entry)(
        plan.handle, q.data_ptr(), _strides(q.stride(0), q.stride(1)), kv_cache.data_ptr(),
        _strides(ks[0], ks[1], ks[2], ks[3]), out.data_ptr(), _strides(out.stride(0), out.stride(1)),
        _ptr(lse), float(sm_scale), _ptr(fw), 0 if fw is None else fw.numel(), _stream(q)))
    return (out, lse) if return_lse else out


def bskv_run_decode_partial(plan, q, kv_cache, out=None, lse=None, return_lse=False,
                            sm_scale=None):
    """Attention kernel of the decode only (see bskv_decode_merge)."""
    return bskv_run_decode(plan, q, kv_cache, out, lse, return_lse, sm_scale,
                           _entry="bskv_run_decode_partial")


def bskv_decode_merge(plan, out, lse=None):
    """Merge the split-KV partial states a bskv_run_decode_partial left in the plan's
    float workspace into out (and lse)."""
    lib = load_library()
    if plan.int_ws is not None:
        plan.on_stream(out.device)
    fw = plan.float_ws
    _check("bskv_decode_merge", lib.bskv_decode_merge(
        plan.handle, out.data_ptr(), _strides(out.stride(0), out.stride(1)), _ptr(lse), _ptr(fw),
        0 if fw is None else fw.numel(), _stream(out)))
    return out


def bskv_run_decode_noalloc(plan, q, kv_cache, out, lse=None, sm_scale=None):
    """Decode without any device allocation by the library or by this call: for callers
    that cannot allocate (see bskv.h). The caller passes the output (and optional lse);
    the plan is not uploaded, its metadata goes into a library-owned static array."""
    lib = load_library()
    B, Hq, D = q.shape
    if plan.kind != "decode" or (B, Hq, D) != (plan.info["batch"], plan.info["num_qo_heads"],
                                                plan.info["head_dim"]):
        raise ValueError("q %s does not match the decode plan" % (tuple(q.shape),))
    if tuple(out.shape) != (B, Hq, D) or out.dtype != plan.info["dtype"] or out.device != q.device:
        raise ValueError("out must be a %s tensor of shape %s on %s"
                         % (plan.info["dtype"], (B, Hq, D), q.device))
    if lse is not None and (tuple(lse.shape) != (B, Hq) or lse.dtype != torch.float32
                            or lse.device != q.device or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 tensor of shape %s on %s"
                         % ((B, Hq), q.device))
    if kv_cache.device != q.device:
        raise ValueError("kv_cache must be on %s" % q.device)
    if sm_scale is None:
        sm_scale = 0.0  # the library applies 1/sqrt(head_dim)
    ks = kv_cache.stride()
    _check("bskv_run_decode_noalloc", lib.bskv_run_decode_noalloc(
        plan.handle, q.data_ptr(), _strides(q.stride(0), q.stride(1)), kv_cache.data_ptr(),
        _strides(ks[0], ks[1], ks[2], ks[3]), out.data_ptr(), _strides(out.stride(0), out.stride(1)),
        _ptr(lse), float(sm_scale), _stream(q)))
    return out


def bskv_plan_bsr(indptr, indices, M, N, R, C, num_qo_heads, num_kv_heads, head_dim,
                  causal=False, dtype=torch.float16, num_sms=None):
    lib = load_library()
    ip, ipp = _i32_array(indptr)
    ix, ixp = _i32_array(indices)
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    _check("bskv_plan_bsr", lib.bskv_plan_bsr(
        ctypes.cast(ipp, _I32P), ctypes.cast(ixp, _I32P), int(M), int(N), int(R), int(C),
        int(num_qo_heads), int(num_kv_heads), int(head_dim), int(bool(causal)), _DT[dtype],
        int(ns), ctypes.byref(h)))
    return Plan(h.value, "bsr", M=M, N=N, R=R, C=C, num_qo_heads=num_qo_heads,
                num_kv_heads=num_kv_heads, head_dim=head_dim, dtype=dtype)


def bskv_run_bsr(plan, q, k, v, out=None, lse=None, return_lse=False, sm_scale=None):
    lib = load_library()
    plan.on_stream(q.device)
    M, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((M, Hq), dtype=torch.float32, device=q.device)
    if sm_scale is None:
        sm_scale = 0.0  # the library applies 1/sqrt(head_dim)
    fw = plan.float_ws
    _check("bskv_run_bsr", lib.bskv_run_bsr(
        plan.handle, q.data_ptr(), _strides(q.stride(0), q.stride(1)), k.data_ptr(),
        _strides(k.stride(0), k.stride(1)), v.data_ptr(), _strides(v.stride(0), v.stride(1)),
        out.data_ptr(), _strides(out.stride(0), out.stride(1)), _ptr(lse), float(sm_scale),
        _ptr(fw), 0 if fw is None else fw.numel(), _stream(q)))
    return (out, lse) if return_lse else out


def bskv_plan_bsr_masked(indptr, indices, M, N, R, C, num_qo_heads, num_kv_heads, head_dim,
                         dtype=torch.float16, num_sms=None):
    """BSR plan whose runs take a per-block token mask (packed bits, bskv_run_bsr_masked)."""
    lib = load_library()
    ip, ipp = _i32_array(indptr)
    ix, ixp = _i32_array(indices)
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    _check("bskv_plan_bsr_masked", lib.bskv_plan_bsr_masked(
        ctypes.cast(ipp, _I32P), ctypes.cast(ixp, _I32P), int(M), int(N), int(R), int(C),
        int(num_qo_heads), int(num_kv_heads), int(head_dim), _DT[dtype], int(ns),
        ctypes.byref(h)))
    return Plan(h.value, "bsr_masked", M=M, N=N, R=R, C=C, num_qo_heads=num_qo_heads,
                num_kv_heads=num_kv_heads, head_dim=head_dim, dtype=dtype)


def bskv_run_bsr_masked(plan, q, k, v, packed_mask, out=None, lse=None, return_lse=False,
                        sm_scale=None):
    """packed_mask: uint8 device tensor, the (nnz, R, C) mask packed little-endian per byte."""
    lib = load_library()
    plan.on_stream(q.device)
    M, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((M, Hq), dtype=torch.float32, device=q.device)
    if sm_scale is None:
        sm_scale = 0.0  # the library applies 1/sqrt(head_dim)
    _check("bskv_run_bsr_masked", lib.bskv_run_bsr_masked(
        plan.handle, q.data_ptr(), _strides(q.stride(0), q.stride(1)), k.data_ptr(),
        _strides(k.stride(0), k.stride(1)), v.data_ptr(), _strides(v.stride(0), v.stride(1)),
        packed_mask.data_ptr(), packed_mask.numel(), out.data_ptr(),
        _strides(out.stride(0), out.stride(1)), _ptr(lse), float(sm_scale), _stream(q)))
    return (out, lse) if return_lse else out


def bskv_plan_bsr_variable(block_mask_map, block_row_sz, block_col_sz, num_qo_heads,
                           num_kv_heads, head_dim, causal=False, dtype=torch.float16,
                           num_sms=None):
    """Variable-block plan: block_mask_map [Hkv, MB, NB] bool, block_row_sz [Hkv, MB],
    block_col_sz [Hkv, NB] int (host copies are made)."""
    lib = load_library()
    bm = torch.as_tensor(block_mask_map).to(torch.uint8).contiguous().cpu()
    rs, rsp = _i32_array(block_row_sz)
    cs, csp = _i32_array(block_col_sz)
    Hkv, MB, NB = bm.shape
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    _check("bskv_plan_bsr_variable", lib.bskv_plan_bsr_variable(
        ctypes.c_void_p(bm.data_ptr()), ctypes.cast(rsp, _I32P), ctypes.cast(csp, _I32P), int(MB),
        int(NB), int(num_qo_heads), int(num_kv_heads), int(head_dim), int(bool(causal)),
        _DT[dtype], int(ns), ctypes.byref(h)))
    return Plan(h.value, "bsr_variable", num_qo_heads=num_qo_heads, num_kv_heads=num_kv_heads,
                head_dim=head_dim, dtype=dtype, qo_len=int(rs.view(Hkv, MB)[0].sum()))


def bskv_run_bsr_variable(plan, q, k, v, out=None, lse=None, return_lse=False, sm_scale=None):
    """q [Hq, qo_len, D], k/v [Hkv, kv_len, D] -> out [Hq, qo_len, D] (and lse [Hq, qo_len])."""
    lib = load_library()
    plan.on_stream(q.device)
    Hq, L, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((Hq, L), dtype=torch.float32, device=q.device)
    if sm_scale is None:
        sm_scale = 0.0  # the library applies 1/sqrt(head_dim)
    _check("bskv_run_bsr_variable", lib.bskv_run_bsr_variable(
        plan.handle, q.data_ptr(), _strides(q.stride(1), q.stride(0)), k.data_ptr(),
        _strides(k.stride(1), k.stride(0)), v.data_ptr(), _strides(v.stride(1), v.stride(0)),
        out.data_ptr(), _strides(out.stride(1), out.stride(0)), _ptr(lse), float(sm_scale),
        _stream(q)))
    return (out, lse) if return_lse else out


def bskv_plan_prefill_paged(qo_indptr, kv_indptr, kv_indices, kv_last_page_len, num_pages,
                            page_size, num_qo_heads, num_kv_heads, head_dim, causal=True,
                            dtype=torch.bfloat16, num_sms=None):
    """Paged prefill plan from HOST ragged query and page-table arrays."""
    lib = load_library()
    qi, qip = _i32_array(qo_indptr)
    ip, ipp = _i32_array(kv_indptr)
    ix, ixp = _i32_array(kv_indices)
    lp, lpp = _i32_array(kv_last_page_len)
    batch = qi.numel() - 1
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    _check("bskv_plan_prefill_paged", lib.bskv_plan_prefill_paged(
        ctypes.cast(qip, _I32P), ctypes.cast(ipp, _I32P), ctypes.cast(ixp, _I32P),
        ctypes.cast(lpp, _I32P), int(batch), int(num_pages), int(page_size), int(num_qo_heads),
        int(num_kv_heads), int(head_dim), int(bool(causal)), _DT[dtype], int(ns),
        ctypes.byref(h)))
    return Plan(h.value, "prefill_paged", batch=batch, num_qo_heads=num_qo_heads,
                num_kv_heads=num_kv_heads, head_dim=head_dim, dtype=dtype)


def bskv_run_prefill_paged(plan, q, kv_cache, out=None, lse=None, return_lse=False,
                           sm_scale=None):
    """q [total_qo, Hq, D]; kv_cache [pages, 2, Hkv, page_size, D] (any strides)."""
    lib = load_library()
    plan.on_stream(q.device)
    T, Hq, D = q.shape
    if out is None:
        out = torch.empty_like(q)
    if lse is None and return_lse:
        lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device)
    if sm_scale is None:
        sm_scale = 0.0  # the library applies 1/sqrt(head_dim)
    _check("bskv_run_prefill_paged", lib.bskv_run_prefill_paged(
        plan.handle, q.data_ptr(), _strides(q.stride(0), q.stride(1)), kv_cache.data_ptr(),
        _strides(*kv_cache.stride()[:4]), out.data_ptr(), _strides(out.stride(0), out.stride(1)),
        _ptr(lse), float(sm_scale), _stream(q)))
    return (out, lse) if return_lse else out


def bskv_plan_mla_sparse(seq_lens, batch, q_len, num_heads, top_k, num_sms=None):
    lib = load_library()
    sl, slp = _i32_array(seq_lens)
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    _check("bskv_plan_mla_sparse", lib.bskv_plan_mla_sparse(
        ctypes.cast(slp, _I32P), int(batch), int(q_len), int(num_heads), int(top_k), int(ns),
        ctypes.byref(h)))
    return Plan(h.value, "mla", batch=batch, q_len=q_len, num_heads=num_heads, top_k=top_k)


def bskv_run_mla_sparse(plan, query, kv_rows, indices, bmm1_scale, bmm2_scale=1.0, out=None,
                        lse=None, return_lse=False):
    """query [B, T, H, 576] uint8/e4m3; kv_rows [rows, 576] (or [pages, page_size, 576])."""
    lib = load_library()
    plan.on_stream(query.device)
    B, T, H, _ = query.shape
    rows = kv_rows.numel() // 576
    if out is None:
        out = torch.empty((B, T, H, 512), dtype=torch.bfloat16, device=query.device)
    if lse is None and return_lse:
        lse = torch.empty((B, T, H), dtype=torch.float32, device=query.device)
    fw = plan.float_ws
    _check("bskv_run_mla_sparse", lib.bskv_run_mla_sparse(
        plan.handle, query.data_ptr(), kv_rows.data_ptr(), rows, indices.data_ptr(),
        float(bmm1_scale), float(bmm2_scale), out.data_ptr(), _ptr(lse), _ptr(fw),
        0 if fw is None else fw.numel(), _stream(query)))
    return (out, lse) if return_lse else out


def bskv_plan_mla_paged(kv_indptr, kv_indices, kv_last_page_len, batch, num_pages, page_size,
                        num_heads, num_sms=None):
    """Dense paged MLA decode plan from a HOST CSR page table (one query token per request)."""
    lib = load_library()
    ip, ipp = _i32_array(kv_indptr)
    ix, ixp = _i32_array(kv_indices)
    lp, lpp = _i32_array(kv_last_page_len)
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    _check("bskv_plan_mla_paged", lib.bskv_plan_mla_paged(
        ctypes.cast(ipp, _I32P), ctypes.cast(ixp, _I32P), ctypes.cast(lpp, _I32P), int(batch),
        int(num_pages), int(page_size), int(num_heads), int(ns), ctypes.byref(h)))
    return Plan(h.value, "mla_paged", batch=batch, num_heads=num_heads, num_pages=num_pages,
                page_size=page_size)


def bskv_run_mla_paged(plan, query, kv_pages, bmm1_scale, bmm2_scale=1.0, out=None, lse=None,
                       return_lse=False):
    """query [B, H, 576] uint8/e4m3; kv_pages [num_pages, page_size, 576] uint8/e4m3."""
    lib = load_library()
    plan.on_stream(query.device)
    B, H, _ = query.shape
    if out is None:
        out = torch.empty((B, H, 512), dtype=torch.bfloat16, device=query.device)
    if lse is None and return_lse:
        lse = torch.empty((B, H), dtype=torch.float32, device=query.device)
    fw = plan.float_ws
    _check("bskv_run_mla_paged", lib.bskv_run_mla_paged(
        plan.handle, query.data_ptr(), kv_pages.data_ptr(), float(bmm1_scale), float(bmm2_scale),
        out.data_ptr(), _ptr(lse), _ptr(fw), 0 if fw is None else fw.numel(), _stream(query)))
    return (out, lse) if return_lse else out


def bskv_rope_quantize_fp8(q_rope, k_rope, q_nope, k_nope, cos_sin_cache, pos_ids=None,
                           is_neox=True, quant_scale_q=1.0, quant_scale_kv=1.0,
                           q_rope_out=None, k_rope_out=None, q_nope_out=None, k_nope_out=None,
                           pos_ids_k=None):
    """RoPE + FP8 quantisation. pos_ids covers the query rows (and the key rows when
    pos_ids_k is None, the pages' single-nnz form). Outputs are uint8 E4M3 codes."""
    lib = load_library()
    dev = (q_rope if q_rope is not None else k_rope).device
    u8 = torch.uint8
    pos_q = pos_ids
    pos_k = pos_ids if pos_ids_k is None else pos_ids_k
    args = []
    if q_rope is not None:
        nq, H, _ = q_rope.shape
        if q_rope_out is None:
            q_rope_out = torch.empty((nq, H, 64), dtype=u8, device=dev)
        if q_nope_out is None:
            q_nope_out = torch.empty((nq, H, 512), dtype=u8, device=dev)
        args += [q_rope.data_ptr(), _strides(q_rope.stride(0), q_rope.stride(1)), q_nope.data_ptr(),
                 _strides(q_nope.stride(0), q_nope.stride(1)), pos_q.data_ptr(), nq, H,
                 q_rope_out.data_ptr(), _strides(q_rope_out.stride(0), q_rope_out.stride(1)),
                 q_nope_out.data_ptr(), _strides(q_nope_out.stride(0), q_nope_out.stride(1))]
    else:
        args += [None, None, None, None, None, 0, 0, None, None, None, None]
    if k_rope is not None:
        nk = k_rope.shape[0]
        if k_rope_out is None:
            k_rope_out = torch.empty((nk, 64), dtype=u8, device=dev)
        if k_nope_out is None:
            k_nope_out = torch.empty((nk, 512), dtype=u8, device=dev)
        args += [k_rope.data_ptr(), k_rope.stride(0), k_nope.data_ptr(), k_nope.stride(0),
                 pos_k.data_ptr(), nk, k_rope_out.data_ptr(), k_rope_out.stride(0),
                 k_nope_out.data_ptr(), k_nope_out.stride(0)]
    else:
        args += [None, 0, None, 0, None, 0, None, 0, None, 0]
    pos_any = pos_q if pos_q is not None else pos_k
    args += [_DT[pos_any.dtype], cos_sin_cache.data_ptr(), _DT[cos_sin_cache.dtype],
             cos_sin_cache.shape[0], int(bool(is_neox)), float(quant_scale_q),
             float(quant_scale_kv), _stream(cos_sin_cache)]
    _check("bskv_rope_quantize_fp8", lib.bskv_rope_quantize_fp8(*args))
    return q_rope_out, k_rope_out, q_nope_out, k_nope_out


def bskv_rope_quantize_fp8_append_paged(k_rope, k_nope, pos_k, cos_sin_cache, batch_indices,
                                        positions, kv_indptr, kv_indices, kv_pages,
                                        q_rope=None, q_nope=None, pos_q=None, is_neox=True,
                                        quant_scale_q=1.0, quant_scale_kv=1.0, q_rope_out=None,
                                        q_nope_out=None):
    """RoPE + FP8 with the key rows written into kv_pages [num_pages, page_size, 576] (uint8)
    through the device page table (int32 batch_indices, positions, kv_indptr, kv_indices).
    The optional query group is handled as by bskv_rope_quantize_fp8. Returns the query
    outputs (or None)."""
    lib = load_library()
    dev = k_rope.device
    u8 = torch.uint8
    args = []
    if q_rope is not None:
        nq, H, _ = q_rope.shape
        if q_rope_out is None:
            q_rope_out = torch.empty((nq, H, 64), dtype=u8, device=dev)
        if q_nope_out is None:
            q_nope_out = torch.empty((nq, H, 512), dtype=u8, device=dev)
        args += [q_rope.data_ptr(), _strides(q_rope.stride(0), q_rope.stride(1)), q_nope.data_ptr(),
                 _strides(q_nope.stride(0), q_nope.stride(1)), pos_q.data_ptr(), nq, H,
                 q_rope_out.data_ptr(), _strides(q_rope_out.stride(0), q_rope_out.stride(1)),
                 q_nope_out.data_ptr(), _strides(q_nope_out.stride(0), q_nope_out.stride(1))]
    else:
        args += [None, None, None, None, None, 0, 0, None, None, None, None]
    num_pages, page_size, _ = kv_pages.shape
    batch = kv_indptr.numel() - 1
    args += [k_rope.data_ptr(), k_rope.stride(0), k_nope.data_ptr(), k_nope.stride(0),
             pos_k.data_ptr(), k_rope.shape[0], batch_indices.data_ptr(), positions.data_ptr(),
             kv_indptr.data_ptr(), kv_indices.data_ptr(), int(batch), int(page_size),
             int(num_pages), kv_pages.data_ptr(),
             _DT[pos_k.dtype], cos_sin_cache.data_ptr(), _DT[cos_sin_cache.dtype],
             cos_sin_cache.shape[0], int(bool(is_neox)), float(quant_scale_q),
             float(quant_scale_kv), _stream(cos_sin_cache)]
    _check("bskv_rope_quantize_fp8_append_paged", lib.bskv_rope_quantize_fp8_append_paged(*args))
    return q_rope_out, q_nope_out


def _want(fn, name, t, shape, dtypes, device):
    """One argument check: a tensor of this shape (None: any size) and type on this device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: %s must be a tensor" % (fn, name))
    if t.shape != shape and (t.dim() != len(shape) or
                             any(n is not None and n != m for n, m in zip(shape, t.shape))):
        raise ValueError("%s: %s has shape %s, not %s"
                         % (fn, name, tuple(t.shape), tuple("*" if n is None else n for n in shape)))
    if t.dtype not in dtypes:
        raise ValueError("%s: %s is %s, not %s" % (fn, name, t.dtype, " or ".join(map(str, dtypes))))
    if t.device != device:
        raise ValueError("%s: %s is on %s; all tensors must be on one CUDA device"
                         % (fn, name, t.device))


def _cuda_of(fn, name, t):
    """The CUDA device of a call's first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s: %s must be a tensor" % (fn, name))
    dev = t.device
    if dev.type != "cuda":
        raise ValueError("%s: %s is on %s; all tensors must be on one CUDA device" % (fn, name, dev))
    return dev


def _rows_last(fn, name, t, written=False):
    """The last dimension contiguous; a tensor that is written has no expanded dimension."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1 and t.numel():
        raise ValueError("%s: the last dimension of %s must be contiguous" % (fn, name))
    if written and 0 in st and any(s == 0 and n > 1 for s, n in zip(st, t.shape)):
        raise ValueError("%s: %s is written and must not be an expanded view" % (fn, name))


def _dense(fn, *named):
    for name, t in named:
        if not t.is_contiguous():
            raise ValueError("%s: %s must be contiguous" % (fn, name))


_stride_arrays = {}


def _strides_of(t, n):
    """The first n strides as the C entry points take them; a dimension of size 1 counts as laid
    out densely behind the next."""
    st = t.stride()
    if 1 in t.shape:
        out, dense = [], 1
        for s, m in zip(reversed(st), reversed(t.shape)):
            out.append(dense if m == 1 else s)
            dense = max(dense, m * out[-1])
        st = tuple(out[::-1])
    st = st[:n]
    arr = _stride_arrays.get(st)
    if arr is None:
        if len(_stride_arrays) > 4096:
            _stride_arrays.clear()
        arr = _stride_arrays[st] = _strides(*st)
    return arr


def _call(fn, dev, *args):
    """The C entry point `fn` on the current stream of the tensors' device."""
    entry = getattr(_lib or load_library(), fn)
    if _current_device() == dev.index:
        code = entry(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            code = entry(*args, _raw_stream(dev.index))
    if code:
        _check(fn, code)


def _check_plan(fn, plan, kind):
    if not isinstance(plan, Plan) or plan.kind != kind:
        raise ValueError("%s: not a %s plan" % (fn, kind))


def _ready(fn, plan, device):
    """The plan's workspaces on this device, uploaded at the first run."""
    if plan.int_ws is None:
        if _capturing(device):
            raise RuntimeError("%s: upload the plan before the capture: a graph would copy its "
                               "host memory at every replay" % fn)
        with torch.cuda.device(device):
            plan.upload(device)
    elif plan.int_ws.device != device:
        raise ValueError("%s: the plan was uploaded to %s, the tensors are on %s"
                         % (fn, plan.int_ws.device, device))
    else:
        plan.on_stream(device)


_U8, _I32T, _F32T = (torch.uint8,), (torch.int32,), (torch.float32,)
_HALVES = (torch.bfloat16, torch.float16)


_call_layouts = {}


def _once(memo, check, fn, owner, *tensors):
    """check(fn, owner, *tensors), which depends on nothing but the memo's owner and the tensors'
    shapes, strides, types and devices: the answer is kept for calls with the same ones."""
    try:
        key = (fn,) + tuple([None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())
                             for t in tensors])
    except AttributeError:  # not tensors; the check says which
        return check(fn, owner, *tensors)
    found = memo.get(key)
    if found is None:
        found = check(fn, owner, *tensors)
        if len(memo) >= 1024:
            memo.clear()
        memo[key] = found
    return found


def _fp4_cache(fn, kv_codes, kv_scales, device, num_pages, page_size, num_kv_heads, head_dim,
               written=False):
    """Checks a 4-bit cache; its strides as the C entry points take them."""
    _want(fn, "kv_codes", kv_codes, (num_pages, 2, num_kv_heads, page_size, head_dim // 2), _U8, device)
    _want(fn, "kv_scales", kv_scales, (num_pages, 2, num_kv_heads, page_size, head_dim // 32), _U8,
          device)
    _rows_last(fn, "kv_codes", kv_codes, written)
    _rows_last(fn, "kv_scales", kv_scales, written)
    if page_size > 1 and kv_scales.stride(3) != head_dim // 32 and kv_scales.numel():
        raise ValueError("%s: the slots of kv_scales must be contiguous" % fn)
    return _strides_of(kv_codes, 4), _strides_of(kv_scales, 3)


def _fp4_rows(fn, k, v, dtypes, batch_indices, positions, kv_indptr, kv_indices, written=False):
    """Checks K / V rows and their device page table; (device, nnz, heads, head_dim, batch)."""
    dev = _cuda_of(fn, "k", k)
    if k.dim() != 3:
        raise ValueError("%s: k has shape %s, not (rows, heads, head_dim)" % (fn, tuple(k.shape)))
    shape = k.shape
    _want(fn, "k", k, shape, dtypes, dev)
    _want(fn, "v", v, shape, (k.dtype,), dev)
    _rows_last(fn, "k", k, written)
    _rows_last(fn, "v", v, written)
    for name, x in (("batch_indices", batch_indices), ("positions", positions)):
        _want(fn, name, x, (shape[0],), _I32T, dev)
    for name, x in (("kv_indptr", kv_indptr), ("kv_indices", kv_indices)):
        _want(fn, name, x, (None,), _I32T, dev)
    if kv_indptr.numel() < 1:
        raise ValueError("%s: kv_indptr is empty" % fn)
    _dense(fn, ("batch_indices", batch_indices), ("positions", positions), ("kv_indptr", kv_indptr),
           ("kv_indices", kv_indices))
    return dev, shape[0], shape[1], shape[2], kv_indptr.numel() - 1


def bskv_quantize_fp4_append_paged(k, v, batch_indices, positions, kv_indptr, kv_indices, kv_codes,
                                   kv_scales):
    """Quantise K / V rows [nnz, Hkv, D] (bf16 or fp16) to microscaled 4-bit values and write row
    i to token positions[i] of request batch_indices[i] of the paged cache kv_codes [pages, 2,
    Hkv, page_size, D / 2], kv_scales [pages, 2, Hkv, page_size, D / 32] (uint8), through the
    device page table (all int32)."""
    fn = "bskv_quantize_fp4_append_paged"
    dev, ks, vs, dtype, rows, cache, batch = _once(
        _call_layouts, _check_append, fn, None, k, v, batch_indices, positions, kv_indptr, kv_indices,
        kv_codes, kv_scales)
    _call(fn, dev, k.data_ptr(), ks, v.data_ptr(), vs, dtype, *rows, batch_indices.data_ptr(),
          positions.data_ptr(), kv_indptr.data_ptr(), kv_indices.data_ptr(), *batch,
          kv_codes.data_ptr(), cache[0], kv_scales.data_ptr(), cache[1])


def _check_append(fn, _, k, v, batch_indices, positions, kv_indptr, kv_indices, kv_codes,
                  kv_scales):
    dev, nnz, heads, dim, batch = _fp4_rows(fn, k, v, _HALVES, batch_indices, positions, kv_indptr,
                                            kv_indices)
    _want(fn, "kv_codes", kv_codes, (None, 2, heads, None, dim // 2), _U8, dev)
    pages, _, _, page_size, _ = kv_codes.shape
    cache = _fp4_cache(fn, kv_codes, kv_scales, dev, pages, page_size, heads, dim, written=True)
    return (dev, _strides_of(k, 2), _strides_of(v, 2), _DT[k.dtype], (nnz, heads, dim), cache,
            (batch, page_size, pages))


def bskv_dequantize_fp4_paged(kv_codes, kv_scales, batch_indices, positions, kv_indptr, kv_indices,
                              dtype=torch.bfloat16, k_out=None, v_out=None):
    """Rows of a 4-bit paged cache as values: (k, v) [nnz, Hkv, D] of `dtype` (bf16, fp16 or
    fp32; that of k_out and v_out where they are given), row i being token positions[i] of request batch_indices[i]. Rows whose token is out of
    range are left as they were (unspecified in outputs that are made here)."""
    fn = "bskv_dequantize_fp4_paged"
    if (k_out is None) != (v_out is None):
        raise ValueError("%s: give both outputs or neither" % fn)
    if dtype not in _read_layouts:
        raise ValueError("%s: dtype is %s, not %s" % (fn, dtype, " or ".join(map(str, _read_layouts))))
    dev, ks, vs, out_dtype, shape, cache, batch = _once(
        _read_layouts[dtype], _check_dequantize, fn, dtype, k_out, v_out, batch_indices, positions,
        kv_indptr, kv_indices, kv_codes, kv_scales)
    if k_out is None:
        k_out = torch.empty(shape, dtype=dtype, device=dev)
        v_out = torch.empty(shape, dtype=dtype, device=dev)
    _call(fn, dev, kv_codes.data_ptr(), cache[0], kv_scales.data_ptr(), cache[1],
          batch_indices.data_ptr(), positions.data_ptr(), kv_indptr.data_ptr(),
          kv_indices.data_ptr(), *batch, k_out.data_ptr(), ks, v_out.data_ptr(), vs, out_dtype, *shape)
    return k_out, v_out


_read_layouts = {torch.bfloat16: {}, torch.float16: {}, torch.float32: {}}


def _check_dequantize(fn, dtype, k, v, batch_indices, positions, kv_indptr, kv_indices, kv_codes,
                      kv_scales):
    dev = _cuda_of(fn, "kv_codes", kv_codes)
    if kv_codes.dim() != 5 or not isinstance(positions, torch.Tensor):
        raise ValueError("%s: kv_codes must be [pages, 2, Hkv, page_size, D / 2]" % fn)
    pages, _, heads, page_size, half = kv_codes.shape
    if k is None:  # what the caller gets
        k = v = torch.empty((positions.numel(), heads, 2 * half), dtype=dtype, device=dev)
    rows_dev, nnz, heads, dim, batch = _fp4_rows(fn, k, v, tuple(_read_layouts), batch_indices, positions,
                                                 kv_indptr, kv_indices, written=True)
    cache = _fp4_cache(fn, kv_codes, kv_scales, rows_dev, pages, page_size, heads, dim)
    return (dev, _strides_of(k, 2), _strides_of(v, 2), _DT[k.dtype], (nnz, heads, dim), cache,
            (batch, page_size, pages))


def bskv_plan_decode_fp4(kv_indptr, kv_indices, kv_last_page_len, num_pages, page_size,
                         num_qo_heads, num_kv_heads, head_dim, dtype=torch.bfloat16, num_sms=None,
                         max_workers=0):
    """Decode plan over a 4-bit paged cache, from a HOST page table (as bskv_plan_decode)."""
    lib = load_library()
    ip, ipp, ix, ixp, lp, lpp, batch = _page_table("bskv_plan_decode_fp4", kv_indptr, kv_indices,
                                                   kv_last_page_len)
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    _check("bskv_plan_decode_fp4", lib.bskv_plan_decode_fp4(
        ctypes.cast(ipp, _I32P), ctypes.cast(ixp, _I32P), ctypes.cast(lpp, _I32P), batch,
        int(num_pages), int(page_size), int(num_qo_heads), int(num_kv_heads), int(head_dim),
        _DT[dtype], int(ns), int(max_workers), ctypes.byref(h)))
    return Plan(h.value, "decode_fp4", batch=batch, num_pages=int(num_pages),
                page_size=int(page_size), num_qo_heads=int(num_qo_heads),
                num_kv_heads=int(num_kv_heads), head_dim=int(head_dim), dtype=dtype,
                q_shape=(batch, int(num_qo_heads), int(head_dim)))


def _page_table(fn, kv_indptr, kv_indices, kv_last_page_len):
    ip, ipp = _i32_array(kv_indptr)
    ix, ixp = _i32_array(kv_indices)
    lp, lpp = _i32_array(kv_last_page_len)
    batch = ip.numel() - 1
    if batch < 0 or lp.numel() < batch or (batch > 0 and ix.numel() < int(ip[-1])):
        raise ValueError("%s: page table arrays of %d, %d and %d entries do not fit together"
                         % (fn, ip.numel(), ix.numel(), lp.numel()))
    return ip, ipp, ix, ixp, lp, lpp, batch


def bskv_run_decode_fp4(plan, q, kv_codes, kv_scales, out=None, lse=None, return_lse=False,
                        sm_scale=None):
    """Decode one query token per request over a 4-bit paged cache: q [B, Hq, D]; kv_codes
    [pages, 2, Hkv, page_size, D / 2], kv_scales [pages, 2, Hkv, page_size, D / 32] uint8."""
    fn = "bskv_run_decode_fp4"
    _check_plan(fn, plan, "decode_fp4")
    dev, qs, cache, outs, shape = _once(plan.layouts, _check_decode_fp4, fn, plan, q, kv_codes,
                                        kv_scales, out, lse)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=dev)
    if lse is None and return_lse:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=dev)
    _ready(fn, plan, dev)
    fw = plan.float_ws
    _call(fn, dev, plan.handle, q.data_ptr(), qs, kv_codes.data_ptr(), cache[0], kv_scales.data_ptr(),
          cache[1], out.data_ptr(), outs, _ptr(lse), 0.0 if sm_scale is None else float(sm_scale),
          _ptr(fw), 0 if fw is None else fw.numel())
    return (out, lse) if return_lse else out


def _check_decode_fp4(fn, plan, q, kv_codes, kv_scales, out, lse):
    i = plan.info
    shape, dtypes = i["q_shape"], (i["dtype"],)
    dev = _cuda_of(fn, "q", q)
    _want(fn, "q", q, shape, dtypes, dev)
    _rows_last(fn, "q", q)
    cache = _fp4_pages(fn, plan, kv_codes, kv_scales, dev)
    if out is not None:
        _want(fn, "out", out, shape, dtypes, dev)
        _rows_last(fn, "out", out, written=True)
    if lse is not None:
        _want(fn, "lse", lse, shape[:2], _F32T, dev)
        _dense(fn, ("lse", lse))
    outs = _strides(shape[1] * shape[2], shape[2]) if out is None else _strides_of(out, 2)
    return dev, _strides_of(q, 2), cache, outs, shape


def bskv_plan_attn_weights(qo_indptr, kv_indptr, kv_indices, kv_last_page_len, num_pages, page_size,
                           num_qo_heads, num_kv_heads, head_dim, causal=True, dtype=torch.bfloat16,
                           num_sms=None):
    """Plan of the accumulated attention weights, from HOST arrays; qo_indptr None: one query per
    request (the decode step)."""
    fn = "bskv_plan_attn_weights"
    lib = load_library()
    ip, ipp, ix, ixp, lp, lpp, batch = _page_table(fn, kv_indptr, kv_indices, kv_last_page_len)
    qi, qip = (None, None) if qo_indptr is None else _i32_array(qo_indptr)
    if qi is not None and qi.numel() != batch + 1:
        raise ValueError("%s: qo_indptr has %d entries, kv_indptr %d" % (fn, qi.numel(), batch + 1))
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    _check(fn, lib.bskv_plan_attn_weights(
        None if qip is None else ctypes.cast(qip, _I32P), ctypes.cast(ipp, _I32P),
        ctypes.cast(ixp, _I32P), ctypes.cast(lpp, _I32P), batch, int(num_pages), int(page_size),
        int(num_qo_heads), int(num_kv_heads), int(head_dim), int(bool(causal)), _DT[dtype], int(ns),
        ctypes.byref(h)))
    total_qo = batch if qi is None else int(qi[-1])
    return Plan(h.value, "attn_weights", batch=batch, num_pages=int(num_pages), page_size=int(page_size),
                num_qo_heads=int(num_qo_heads), num_kv_heads=int(num_kv_heads),
                head_dim=int(head_dim), dtype=dtype,
                q_shape=(total_qo, int(num_qo_heads), int(head_dim)))


def _scores(fn, plan, scores, device):
    i = plan.info
    _want(fn, "scores", scores, (i["num_pages"], i["num_kv_heads"], i["page_size"]), _F32T, device)
    _rows_last(fn, "scores", scores, written=True)
    return _strides_of(scores, 2)


def _kv_pages(fn, plan, kv_cache, dtypes, device, written=False):
    i = plan.info
    _want(fn, "kv_cache", kv_cache, (i["num_pages"], 2, i["num_kv_heads"], i["page_size"],
                                     i["head_dim"]), dtypes, device)
    _rows_last(fn, "kv_cache", kv_cache, written)
    return (_strides_of(kv_cache, 4),)


def _fp4_pages(fn, plan, kv_codes, kv_scales, device, written=False):
    i = plan.info
    return _fp4_cache(fn, kv_codes, kv_scales, device, i["num_pages"], i["page_size"],
                      i["num_kv_heads"], i["head_dim"], written)


def _check_attn_weights(fn, plan, q, lse, scores, *cache):
    i = plan.info
    shape = i["q_shape"]
    dev = _cuda_of(fn, "q", q)
    _want(fn, "q", q, shape, (i["dtype"],), dev)
    _rows_last(fn, "q", q)
    _want(fn, "lse", lse, shape[:2], _F32T, dev)
    _dense(fn, ("lse", lse))
    strides = _fp4_pages(fn, plan, *cache, dev) if len(cache) == 2 else _kv_pages(
        fn, plan, *cache, (i["dtype"],), dev)
    return dev, _strides_of(q, 2), strides, _scores(fn, plan, scores, dev)


def bskv_run_attn_weights(plan, q, kv_cache, lse, scores, decay=1.0, sm_scale=None):
    """Add the queries' attention weights over the cached tokens, summed per kv head, to scores
    [pages, Hkv, page_size] float32 (in place): q [total_qo, Hq, D], kv_cache [pages, 2, Hkv,
    page_size, D], lse [total_qo, Hq] as the attention run returned it. Old scores are multiplied
    by decay first; those of the queries' own tokens (the last of each request), and all of them
    with decay 0, start anew."""
    fn = "bskv_run_attn_weights"
    _check_plan(fn, plan, "attn_weights")
    dev, qs, cache, where = _once(plan.layouts, _check_attn_weights, fn, plan, q, lse, scores, kv_cache)
    _ready(fn, plan, dev)
    _call(fn, dev, plan.handle, q.data_ptr(), qs, kv_cache.data_ptr(), cache[0], lse.data_ptr(),
          scores.data_ptr(), where, float(decay), 0.0 if sm_scale is None else float(sm_scale))
    return scores


def bskv_run_attn_weights_fp4(plan, q, kv_codes, kv_scales, lse, scores, decay=1.0, sm_scale=None):
    """bskv_run_attn_weights over a 4-bit paged cache."""
    fn = "bskv_run_attn_weights_fp4"
    _check_plan(fn, plan, "attn_weights")
    dev, qs, cache, where = _once(plan.layouts, _check_attn_weights, fn, plan, q, lse, scores, kv_codes,
                                  kv_scales)
    _ready(fn, plan, dev)
    _call(fn, dev, plan.handle, q.data_ptr(), qs, kv_codes.data_ptr(), cache[0], kv_scales.data_ptr(),
          cache[1], lse.data_ptr(), scores.data_ptr(), where, float(decay),
          0.0 if sm_scale is None else float(sm_scale))
    return scores


def bskv_plan_evict(kv_indptr, kv_indices, kv_last_page_len, keep_len, sink, recent, num_pages,
                    page_size, num_kv_heads, head_dim, dst_indptr=None, dst_indices=None,
                    num_sms=None):
    """Plan of an eviction to keep_len[b] tokens per request, from HOST arrays: into the pages
    dst_indptr / dst_indices, or in place without them. plan.info["kept_indptr"] delimits each
    request's entries in the runs' kept lists."""
    fn = "bskv_plan_evict"
    lib = load_library()
    ip, ipp, ix, ixp, lp, lpp, batch = _page_table(fn, kv_indptr, kv_indices, kv_last_page_len)
    kl, klp = _i32_array(keep_len)
    if kl.numel() != batch:
        raise ValueError("%s: keep_len has %d entries for %d requests" % (fn, kl.numel(), batch))
    dip = dxp = None
    if (dst_indptr is None) != (dst_indices is None):
        raise ValueError("%s: give dst_indptr and dst_indices, or neither" % fn)
    if dst_indptr is not None:
        di, dip = _i32_array(dst_indptr)
        dx, dxp = _i32_array(dst_indices)
        if di.numel() != batch + 1 or dx.numel() < int(di[-1]):
            raise ValueError("%s: dst_indptr has %d entries for %d requests, dst_indices %d"
                             % (fn, di.numel(), batch, dx.numel()))
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    _check(fn, lib.bskv_plan_evict(
        ctypes.cast(ipp, _I32P), ctypes.cast(ixp, _I32P), ctypes.cast(lpp, _I32P),
        ctypes.cast(klp, _I32P), int(sink), int(recent),
        None if dip is None else ctypes.cast(dip, _I32P),
        None if dxp is None else ctypes.cast(dxp, _I32P), batch, int(num_pages), int(page_size),
        int(num_kv_heads), int(head_dim), int(ns), ctypes.byref(h)))
    pages = ip[1:batch + 1] - ip[:batch]
    lens = torch.where(pages > 0, (pages - 1) * int(page_size) + lp[:batch], torch.zeros_like(pages))
    kept = [0]
    for n in torch.minimum(lens, kl).tolist():
        kept.append(kept[-1] + n)
    return Plan(h.value, "evict", batch=batch, num_pages=int(num_pages), page_size=int(page_size),
                num_kv_heads=int(num_kv_heads), head_dim=int(head_dim), kept_indptr=kept)


def _check_evict(fn, plan, scores, kept, *cache):
    dev = _cuda_of(fn, "scores", scores)
    shape = (plan.info["num_kv_heads"], plan.info["kept_indptr"][-1])
    if kept is not None:
        _want(fn, "kept", kept, shape, _I32T, dev)
        _dense(fn, ("kept", kept))
    strides = _fp4_pages(fn, plan, *cache, dev, written=True) if len(cache) == 2 else _kv_pages(
        fn, plan, *cache, _HALVES, dev, written=True)
    return dev, shape, strides, _scores(fn, plan, scores, dev)


def bskv_run_evict(plan, scores, kv_cache, kept=None, compact_scores=True):
    """Keep the plan's number of tokens per request, chosen per kv head by scores [pages, Hkv,
    page_size], and move their rows of kv_cache [pages, 2, Hkv, page_size, D] (16-bit), and with
    compact_scores their scores, to the front. Returns the old slots of the kept tokens [Hkv,
    kept_indptr[-1]] int32."""
    fn = "bskv_run_evict"
    _check_plan(fn, plan, "evict")
    dev, shape, cache, where = _once(plan.layouts, _check_evict, fn, plan, scores, kept, kv_cache)
    if kept is None:
        kept = torch.empty(shape, dtype=torch.int32, device=dev)
    _ready(fn, plan, dev)
    _call(fn, dev, plan.handle, scores.data_ptr(), where, int(bool(compact_scores)),
          kv_cache.data_ptr(), cache[0], kept.data_ptr())
    return kept


def bskv_run_evict_fp4(plan, scores, kv_codes, kv_scales, kept=None, compact_scores=True):
    """bskv_run_evict over a 4-bit paged cache."""
    fn = "bskv_run_evict_fp4"
    _check_plan(fn, plan, "evict")
    dev, shape, cache, where = _once(plan.layouts, _check_evict, fn, plan, scores, kept, kv_codes,
                                     kv_scales)
    if kept is None:
        kept = torch.empty(shape, dtype=torch.int32, device=dev)
    _ready(fn, plan, dev)
    _call(fn, dev, plan.handle, scores.data_ptr(), where, int(bool(compact_scores)),
          kv_codes.data_ptr(), cache[0], kv_scales.data_ptr(), cache[1], kept.data_ptr())
    return kept


class PageTable:
    """The index arrays of a batch as bskv_build_page_table writes them: kv_indptr and qo_indptr [B + 1],
    kv_indices, kv_last_page_len [B] and, per new token, batch_indices, positions (int32) and slots
    (int64, or None); free_left [1] where pages are handed out of a free list, else None. The tensors are
    checked here, once, and must not be resized."""

    __slots__ = ("kv_indptr", "kv_indices", "kv_last_page_len", "qo_indptr", "batch_indices", "positions",
                 "slots", "free_left", "_device", "_batch", "_entries", "_pointers")

    def __init__(self, kv_indptr, kv_indices, kv_last_page_len, qo_indptr, batch_indices, positions, slots=None,
                 free_left=None):
        fn = "PageTable"
        dev = _cuda_of(fn, "kv_indptr", kv_indptr)
        _list_of(fn, "kv_indptr", kv_indptr, None, dev)
        batch = kv_indptr.numel() - 1
        if batch < 0:
            raise ValueError("%s: kv_indptr is empty" % fn)
        _list_of(fn, "batch_indices", batch_indices, None, dev)
        rows = batch_indices.numel()
        for name, t, n in (("kv_indices", kv_indices, None), ("kv_last_page_len", kv_last_page_len, batch),
                           ("qo_indptr", qo_indptr, batch + 1), ("positions", positions, rows)):
            _list_of(fn, name, t, n, dev)
        if slots is not None:
            _list_of(fn, "slots", slots, rows, dev, _I64T)
        if free_left is not None:
            _list_of(fn, "free_left", free_left, 1, dev)
        self._device, self._batch, self._entries = dev, batch, kv_indices.numel()
        self._pointers = (_P(kv_indptr.data_ptr()), _P(kv_indices.data_ptr()), _I64(kv_indices.numel()),
                          _P(kv_last_page_len.data_ptr()), _P(qo_indptr.data_ptr()), _P(batch_indices.data_ptr()),
                          _P(positions.data_ptr()), _P(_ptr(slots)), _I64(rows))
        self.kv_indptr, self.kv_indices, self.kv_last_page_len = kv_indptr, kv_indices, kv_last_page_len
        self.qo_indptr, self.batch_indices, self.positions = qo_indptr, batch_indices, positions
        self.slots, self.free_left = slots, free_left

    def __setattr__(self, name, value):
        if hasattr(self, name):
            raise AttributeError("PageTable: %s cannot be replaced; make another PageTable" % name)
        object.__setattr__(self, name, value)


_I64T = (torch.int64,)


def _at(strides):
    """The address of an array of strides, which it keeps alive, as a call takes it without converting it again."""
    if strides is None:
        return None
    p = _P(ctypes.addressof(strides))
    p.strides = strides
    return p


def _list_of(fn, name, t, n, device, dtypes=_I32T):
    _want(fn, name, t, (n,), dtypes, device)
    _dense(fn, (name, t))


def _check_page_table(fn, _, seq_lens, block_table, new_lens, free_pages, free_count):
    dev = _cuda_of(fn, "seq_lens", seq_lens)
    _list_of(fn, "seq_lens", seq_lens, None, dev)
    batch = seq_lens.numel()
    _want(fn, "block_table", block_table, (batch, None), _I32T, dev)
    _rows_last(fn, "block_table", block_table, written=free_pages is not None)
    if new_lens is not None:
        _list_of(fn, "new_lens", new_lens, batch, dev)
    if (free_pages is None) != (free_count is None):
        raise ValueError("%s: give free_pages and free_count, or neither" % fn)
    if free_pages is not None:
        _list_of(fn, "free_pages", free_pages, None, dev)
        _list_of(fn, "free_count", free_count, 1, dev)
    most = block_table.shape[1]
    return (dev, batch, batch * most, _I32(batch), (_I64(_strides_of(block_table, 1)[0]), _I32(most)),
            _I32(0 if free_pages is None else free_pages.numel()))


def bskv_build_page_table(seq_lens, block_table, page_size, num_pages, new_lens=None, free_pages=None,
                          free_count=None, max_tokens=None, out=None):
    """Page table and token map of a batch from its requests' lengths, all int32 on the GPU: seq_lens [B] with
    the new tokens included, new_lens [B] (None: one each), block_table [B, max_pages]. With free_pages and
    free_count [1], pages that new tokens need come from the end of the free list and are written into
    block_table. The PageTable has room for max_tokens new tokens (None: B, and new_lens must be None);
    rows without one are -1. `out` is an earlier PageTable to write into (its room is what counts then)."""
    fn = "bskv_build_page_table"
    dev, batch, entries, requests, shape, most_free = _once(
        _call_layouts, _check_page_table, fn, None, seq_lens, block_table, new_lens, free_pages, free_count)
    o = out
    if o is None:
        if max_tokens is None:
            if new_lens is not None:
                raise ValueError("%s: new_lens need max_tokens (or out)" % fn)
            max_tokens = batch
        if int(max_tokens) < 0:
            raise ValueError("%s: max_tokens is %d" % (fn, max_tokens))

        def ints(n, dtype=torch.int32):
            return torch.empty(n, dtype=dtype, device=dev)

        o = PageTable(ints(batch + 1), ints(entries), ints(batch), ints(batch + 1), ints(int(max_tokens)),
                      ints(int(max_tokens)), ints(int(max_tokens), torch.int64),
                      None if free_pages is None else ints(1))
    elif not isinstance(o, PageTable):
        raise TypeError("%s: out must be a PageTable" % fn)
    elif o._device != dev or o._batch != batch or o._entries < entries:
        raise ValueError("%s: out is for %d requests and %d pages on %s; needed are %d, up to %d and %s"
                         % (fn, o._batch, o._entries, o._device, batch, entries, dev))
    elif free_pages is not None and o.free_left is None:
        raise ValueError("%s: free_pages need a PageTable with free_left" % fn)
    free = (None, most_free, None, None) if free_pages is None else (
        free_pages.data_ptr(), most_free, free_count.data_ptr(), o.free_left.data_ptr())
    _call(fn, dev, seq_lens.data_ptr(), _ptr(new_lens), requests, int(page_size), block_table.data_ptr(), *shape,
          int(num_pages), *free, *o._pointers)
    return o


def _check_norm_rope(fn, _, q, k, v, cos_sin_cache, batch_indices, positions, kv_indptr, kv_indices, kv_cache,
                     q_weight, k_weight, pos_ids, q_out):
    if q is None and k is None:
        raise ValueError("%s: give q, or k, v and kv_cache, or all" % fn)
    if (k is None) != (v is None) or (k is None) != (kv_cache is None):
        raise ValueError("%s: give k, v and kv_cache, or none of them" % fn)
    first = q if q is not None else k
    dev = _cuda_of(fn, "q" if q is not None else "k", first)
    if first.dim() != 3:
        raise ValueError("%s: %s has shape %s, not (rows, heads, head_dim)"
                         % (fn, "q" if q is not None else "k", tuple(first.shape)))
    nnz, _, dim = first.shape
    dtypes = (first.dtype,) if first.dtype in _HALVES else _HALVES
    qs = qos = ks = vs = cs = None
    hq = hkv = pages = 0
    page_size = 1
    if q is not None:
        _want(fn, "q", q, (nnz, None, dim), dtypes, dev)
        _rows_last(fn, "q", q)
        hq, qs = q.shape[1], _strides_of(q, 2)
        qos = _strides(hq * dim, dim)
        if q_out is not None:
            _want(fn, "q_out", q_out, q.shape, dtypes, dev)
            _rows_last(fn, "q_out", q_out, written=True)
            qos = _strides_of(q_out, 2)
    elif q_out is not None or q_weight is not None:
        raise ValueError("%s: q_out and q_weight need q" % fn)
    if k is not None:
        _want(fn, "k", k, (nnz, None, dim), dtypes, dev)
        hkv = k.shape[1]
        _want(fn, "v", v, (nnz, hkv, dim), dtypes, dev)
        _want(fn, "kv_cache", kv_cache, (None, 2, hkv, None, dim), dtypes, dev)
        _rows_last(fn, "k", k)
        _rows_last(fn, "v", v)
        _rows_last(fn, "kv_cache", kv_cache, written=True)
        ks, vs, cs = _strides_of(k, 2), _strides_of(v, 2), _strides_of(kv_cache, 4)
        pages, page_size = kv_cache.shape[0], kv_cache.shape[3]
    elif k_weight is not None:
        raise ValueError("%s: k_weight needs k" % fn)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _list_of(fn, name, w, dim, dev, dtypes)
    rot = limit = 0
    table = FP32
    if cos_sin_cache is not None:
        _want(fn, "cos_sin_cache", cos_sin_cache, (None, None), (torch.float32, torch.bfloat16), dev)
        _dense(fn, ("cos_sin_cache", cos_sin_cache))
        limit, rot = cos_sin_cache.shape
        table = _DT[cos_sin_cache.dtype]
    for name, x in (("batch_indices", batch_indices), ("positions", positions), ("pos_ids", pos_ids)):
        if x is not None or name != "pos_ids":
            _list_of(fn, name, x, nnz, dev)
    batch = 0
    if k is not None:
        _list_of(fn, "kv_indptr", kv_indptr, None, dev)
        _list_of(fn, "kv_indices", kv_indices, None, dev)
        batch = kv_indptr.numel() - 1
        if batch < 0:
            raise ValueError("%s: kv_indptr is empty" % fn)
    return (dev, _at(qs), _at(qos), _at(ks), _at(vs), _at(cs),
            (_I32(_DT[first.dtype]), _I64(nnz), _I32(hq), _I32(hkv), _I32(dim)), (_I32(table), _I64(limit), _I32(rot)),
            (_I32(batch), _I32(page_size), _I64(pages)))


def bskv_norm_rope_append_paged(q, k, v, cos_sin_cache, batch_indices, positions, kv_indptr, kv_indices,
                                kv_cache, q_weight=None, k_weight=None, eps=1e-6, is_neox=True, pos_ids=None,
                                q_out=None):
    """RMS norms per head (q_weight, k_weight [D]; None: none) and rotation by cos_sin_cache [max_seq_len,
    rotary_dim] (fp32 or bf16; None: none) at pos_ids (None: positions) of q [nnz, Hq, D] and k [nnz, Hkv, D];
    k and v are written to token positions[i] of request batch_indices[i] of kv_cache [pages, 2, Hkv, page_size, D]
    through the device page table (int32); rows with batch_indices -1 are passed over. q, or k, v and kv_cache, may be None.
    Returns q's result (q_out, which may be q; unspecified in rows that are passed over if it is made here), or None."""
    fn = "bskv_norm_rope_append_paged"
    dev, qs, qos, ks, vs, cs, shape, table, where = _once(
        _call_layouts, _check_norm_rope, fn, None, q, k, v, cos_sin_cache, batch_indices, positions, kv_indptr,
        kv_indices, kv_cache, q_weight, k_weight, pos_ids, q_out)
    if q is not None and q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    _call(fn, dev, _ptr(q), qs, _ptr(k), ks, _ptr(v), vs, *shape, _ptr(q_weight), _ptr(k_weight), float(eps),
          _ptr(cos_sin_cache), *table, int(bool(is_neox)), _ptr(pos_ids), batch_indices.data_ptr(),
          positions.data_ptr(), _ptr(kv_indptr), _ptr(kv_indices), *where, _ptr(q_out), qos, _ptr(kv_cache), cs)
    return q_out


def _bounds_strides(fn, bounds, shape, dtypes, device, written=False):
    _want(fn, "bounds", bounds, shape, dtypes, device)
    _rows_last(fn, "bounds", bounds, written)
    if bounds.stride(2) != shape[3] and bounds.numel():
        raise ValueError("%s: the last two dimensions of bounds must be contiguous" % fn)
    return _strides_of(bounds, 2)


def _check_block_bounds(fn, _, kv_cache, bounds, batch_indices, positions, kv_indptr, kv_indices, kv_last_page_len):
    dev = _cuda_of(fn, "kv_cache", kv_cache)
    _want(fn, "kv_cache", kv_cache, (None, 2, None, None, None), _HALVES, dev)
    _rows_last(fn, "kv_cache", kv_cache)
    pages, _, heads, page_size, dim = kv_cache.shape
    bs = _bounds_strides(fn, bounds, (pages, heads, 2, dim), (kv_cache.dtype,), dev, written=True)
    _list_of(fn, "batch_indices", batch_indices, None, dev)
    nnz = batch_indices.numel()
    _list_of(fn, "positions", positions, nnz, dev)
    _list_of(fn, "kv_indptr", kv_indptr, None, dev)
    _list_of(fn, "kv_indices", kv_indices, None, dev)
    batch = kv_indptr.numel() - 1
    if batch < 0:
        raise ValueError("%s: kv_indptr is empty" % fn)
    _list_of(fn, "kv_last_page_len", kv_last_page_len, batch, dev)
    return (dev, _at(_strides_of(kv_cache, 4)), _at(bs),
            (_I32(_DT[kv_cache.dtype]), _I32(heads), _I32(dim), _I32(page_size), _I64(pages)), _I64(nnz), _I32(batch))


def bskv_block_bounds_paged(kv_cache, bounds, batch_indices, positions, kv_indptr, kv_indices, kv_last_page_len):
    """Bring bounds [pages, Hkv, 2, D] (least and greatest key values per channel, in the cache's type) up to
    date for the pages of kv_cache [pages, 2, Hkv, page_size, D] that hold the rows (batch_indices,
    positions), through the device page table (all int32). Returns bounds."""
    fn = "bskv_block_bounds_paged"
    dev, cs, bs, shape, nnz, batch = _once(_call_layouts, _check_block_bounds, fn, None, kv_cache, bounds,
                                           batch_indices, positions, kv_indptr, kv_indices, kv_last_page_len)
    _call(fn, dev, kv_cache.data_ptr(), cs, *shape, batch_indices.data_ptr(), positions.data_ptr(), nnz,
          kv_indptr.data_ptr(), kv_indices.data_ptr(), kv_last_page_len.data_ptr(), batch, bounds.data_ptr(), bs)
    return bounds


def bskv_plan_decode_blocks(num_tokens, max_blocks, num_pages, page_size, num_qo_heads, num_kv_heads,
                            head_dim, top_k, sink=0, recent=1, dtype=torch.bfloat16, num_sms=None):
    """Plan of a block-sparse decode of num_tokens query rows over requests of up to max_blocks pages: each
    query and kv head attends to top_k pages, the first `sink` and the last `recent` among them."""
    fn = "bskv_plan_decode_blocks"
    lib = load_library()
    h = ctypes.c_void_p()
    ns = _num_sms() if num_sms is None else num_sms
    if dtype not in _DT:
        raise ValueError("%s: dtype is %s, not %s" % (fn, dtype, " or ".join(map(str, _HALVES))))
    _check(fn, lib.bskv_plan_decode_blocks(
        int(num_tokens), int(max_blocks), int(num_pages), int(page_size), int(num_qo_heads), int(num_kv_heads),
        int(head_dim), int(top_k), int(sink), int(recent), _DT[dtype], int(ns), ctypes.byref(h)))
    return Plan(h.value, "decode_blocks", num_pages=int(num_pages), page_size=int(page_size),
                num_qo_heads=int(num_qo_heads), num_kv_heads=int(num_kv_heads), head_dim=int(head_dim), dtype=dtype,
                max_blocks=int(max_blocks), blocks_shape=(int(num_tokens), int(num_kv_heads), int(top_k)),
                q_shape=(int(num_tokens), int(num_qo_heads), int(head_dim)))


def _check_blocks(fn, plan, q, blocks, batch_indices, positions, kv_indptr, kv_indices):
    i = plan.info
    dev = _cuda_of(fn, "q", q)
    _want(fn, "q", q, i["q_shape"], (i["dtype"],), dev)
    _rows_last(fn, "q", q)
    if blocks is not None:
        _want(fn, "blocks", blocks, i["blocks_shape"], _I32T, dev)
        _dense(fn, ("blocks", blocks))
    _list_of(fn, "batch_indices", batch_indices, i["q_shape"][0], dev)
    _list_of(fn, "positions", positions, i["q_shape"][0], dev)
    _list_of(fn, "kv_indptr", kv_indptr, None, dev)
    _list_of(fn, "kv_indices", kv_indices, None, dev)
    if kv_indptr.numel() < 1:
        raise ValueError("%s: kv_indptr is empty" % fn)
    return dev, _at(_strides_of(q, 2)), _I32(kv_indptr.numel() - 1)


def _check_select_blocks(fn, plan, q, bounds, *lists):
    i = plan.info
    dev, qs, batch = _check_blocks(fn, plan, q, *lists)
    bs = _bounds_strides(fn, bounds, (i["num_pages"], i["num_kv_heads"], 2, i["head_dim"]), (i["dtype"],), dev)
    return dev, qs, _at(bs), batch, i["blocks_shape"]


def bskv_run_select_blocks(plan, q, bounds, batch_indices, positions, kv_indptr, kv_indices, blocks=None):
    """The pages that each query row (token positions[t] of request batch_indices[t]) and kv head attends to, chosen
    by bounds [pages, Hkv, 2, D]: blocks [T, Hkv, top_k] int32, page numbers within the request, ascending, -1 where
    there are fewer; rows with batch_indices -1 are left as they were (unspecified in an output made here)."""
    fn = "bskv_run_select_blocks"
    _check_plan(fn, plan, "decode_blocks")
    dev, qs, bs, batch, shape = _once(plan.layouts, _check_select_blocks, fn, plan, q, bounds, blocks, batch_indices,
                                      positions, kv_indptr, kv_indices)
    if blocks is None:
        blocks = torch.empty(shape, dtype=torch.int32, device=dev)
    _ready(fn, plan, dev)
    fw = plan.float_ws
    _call(fn, dev, plan.handle, q.data_ptr(), qs, bounds.data_ptr(), bs, batch_indices.data_ptr(),
          positions.data_ptr(), kv_indptr.data_ptr(), kv_indices.data_ptr(), batch, blocks.data_ptr(), _ptr(fw),
          0 if fw is None else fw.numel())
    return blocks


def _check_decode_blocks(fn, plan, q, kv_cache, out, lse, *lists):
    i = plan.info
    if lists[0] is None:
        raise TypeError("%s: blocks must be a tensor" % fn)
    dev, qs, batch = _check_blocks(fn, plan, q, *lists)
    shape = i["q_shape"]
    cache = _kv_pages(fn, plan, kv_cache, (i["dtype"],), dev)
    if out is not None:
        _want(fn, "out", out, shape, (i["dtype"],), dev)
        _rows_last(fn, "out", out, written=True)
    if lse is not None:
        _want(fn, "lse", lse, shape[:2], _F32T, dev)
        _dense(fn, ("lse", lse))
    outs = _strides(shape[1] * shape[2], shape[2]) if out is None else _strides_of(out, 2)
    return dev, qs, _at(cache[0]), _at(outs), batch, shape


def bskv_run_decode_blocks(plan, q, kv_cache, blocks, batch_indices, positions, kv_indptr, kv_indices,
                           out=None, lse=None, return_lse=False, sm_scale=None):
    """Attention of query rows q [T, Hq, D] (token positions[t] of request batch_indices[t]) over the listed blocks
    [T, Hkv, top_k] of kv_cache [pages, 2, Hkv, page_size, D], each up to the query's own token. Rows with
    batch_indices -1 are left as they were (unspecified in outputs made here)."""
    fn = "bskv_run_decode_blocks"
    _check_plan(fn, plan, "decode_blocks")
    dev, qs, cs, outs, batch, shape = _once(plan.layouts, _check_decode_blocks, fn, plan, q, kv_cache, out, lse,
                                            blocks, batch_indices, positions, kv_indptr, kv_indices)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=dev)
    if lse is None and return_lse:
        lse = torch.empty(shape[:2], dtype=torch.float32, device=dev)
    _ready(fn, plan, dev)
    fw = plan.float_ws
    _call(fn, dev, plan.handle, q.data_ptr(), qs, kv_cache.data_ptr(), cs, blocks.data_ptr(),
          batch_indices.data_ptr(), positions.data_ptr(), kv_indptr.data_ptr(), kv_indices.data_ptr(), batch,
          out.data_ptr(), outs, _ptr(lse), 0.0 if sm_scale is None else float(sm_scale), _ptr(fw),
          0 if fw is None else fw.numel())
    return (out, lse) if return_lse else out


def bskv_merge_states(v, s, out_dtype=torch.float32, v_out=None, s_out=None):
    """v [seq, S, H, D] float32, s [seq, S, H] float32 -> (v_out [seq, H, D], s_out [seq, H])."""
    lib = load_library()
    seq, S, H, D = v.shape
    v = v.contiguous()
    s = s.contiguous()
    if v_out is None:
        v_out = torch.empty((seq, H, D), dtype=out_dtype, device=v.device)
    if s_out is None:
        s_out = torch.empty((seq, H), dtype=torch.float32, device=v.device)
    _check("bskv_merge_states", lib.bskv_merge_states(
        v.data_ptr(), s.data_ptr(), seq, S, H, D, v_out.data_ptr(), _DT[v_out.dtype],
        s_out.data_ptr(), _stream(v)))
    return v_out, s_out


def bskv_get_device_status(reset=True):
    lib = load_library()
    st = ctypes.c_int32()
    _check("bskv_get_device_status", lib.bskv_get_device_status(ctypes.byref(st), int(bool(reset))))
    return st.value


def bskv_set_debug_force_timeout(on):
    _check("bskv_set_debug_force_timeout", load_library().bskv_set_debug_force_timeout(int(bool(on))))
