"""Python binding of libar, the MI355X ring all-reduce library (ctypes over the in-tree ``libar.so``).

The binding only marshals arguments: torch tensors become device pointers, the current torch stream becomes
the hipStream_t, and a non-zero ar_status becomes an :class:`ArError`. Every step of the all-reduce runs in
the library's HIP kernels. There is no CPU fallback: if ``libar.so`` is missing or cannot be loaded, every
call raises.

Entry points (same names as ``include/ar.h``): ar_allreduce, ar_allreduce_ws, ar_allreduce_noalloc,
ar_allreduce_workspace_size,
ar_allreduce_buckets, ar_allreduce_tensors, ar_reduce_scatter, ar_all_gather, ar_bucket_plan, ar_bucket_pack,
ar_bucket_unpack, ar_fp8_quant, ar_fp8_dequant, ar_auto_algo, ar_chunk_bounds, ar_status_string, ar_last_call,
ar_version; next to the reduction in a transformer layer: ar_allreduce_rmsnorm, ar_allreduce_rmsnorm_bwd,
ar_allreduce_rmsnorm_bwd_workspace_size, ar_expert_rows, ar_expert_sort, ar_expert_sort_workspace_size,
ar_expert_dispatch, ar_expert_combine, ar_expert_combine_bwd, and between dispatch and combine ar_expert_gated,
ar_expert_gated_bwd, ar_expert_linear, ar_expert_linear_bwd; behind the gradients' all-reduce: ar_grad_plan,
ar_grad_norm, ar_grad_norm_workspace_size, ar_grad_clip. Helpers: chunk_bounds, make_copy_descs,
BucketedAllReduce.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import numpy as np

__all__ = [
    "AR_OK", "AR_ERR_INVALID", "AR_ERR_UNSUPPORTED", "AR_ERR_ALIAS", "AR_ERR_WORKSPACE", "AR_ERR_HIP",
    "AR_F32", "AR_BF16", "AR_F16", "AR_I32", "AR_SUM", "AR_AVG", "AR_MIN", "AR_MAX",
    "AR_ALGO_RING", "AR_ALGO_FUSED", "AR_ALGO_RHD", "AR_ALGO_RING_STEPWISE", "AR_ALGO_RHD_STEPWISE",
    "AR_ALGO_RING_FP8", "AR_ALGO_TREE", "AR_ALGO_TREE_STEPWISE", "AR_ALGO_AUTO", "AR_AUTO_STEP_NS",
    "AR_AUTO_LINK_GBPS", "AR_MAX_RANKS", "AR_FP8_BLOCK", "AR_NOALLOC_WS_BYTES", "ArError", "lib", "lib_path", "ar_auto_algo",
    "ar_allreduce", "ar_allreduce_ws", "ar_allreduce_noalloc", "ar_allreduce_workspace_size", "ar_allreduce_buckets",
    "ar_allreduce_tensors", "ar_reduce_scatter", "ar_all_gather", "ar_chunk_bounds", "chunk_bounds",
    "ar_bucket_plan",
    "ar_bucket_pack",
    "ar_bucket_unpack", "ar_fp8_quant", "ar_fp8_dequant", "ar_status_string", "ar_last_call", "ar_version",
    "make_copy_descs", "BucketedAllReduce", "dtype_code",
    "AR_NORM_MAX_HIDDEN", "AR_MAX_EXPERTS", "ar_allreduce_rmsnorm", "ar_allreduce_rmsnorm_bwd",
    "ar_allreduce_rmsnorm_bwd_workspace_size", "ar_expert_rows", "ar_expert_sort", "ar_expert_sort_workspace_size",
    "ar_expert_dispatch", "ar_expert_combine", "ar_expert_combine_bwd",
    "AR_PRODUCT_MAX_WIDTH", "AR_ACT_SILU", "AR_ACT_GELU", "AR_ACT_GELU_TANH", "ar_expert_gated", "ar_expert_gated_bwd",
    "ar_expert_linear", "ar_expert_linear_bwd",
    "AR_NORM_L2", "AR_NORM_MAX", "ar_grad_plan", "ar_grad_norm", "ar_grad_norm_workspace_size", "ar_grad_clip",
]

AR_OK, AR_ERR_INVALID, AR_ERR_UNSUPPORTED, AR_ERR_ALIAS, AR_ERR_WORKSPACE, AR_ERR_HIP = 0, 1, 2, 3, 4, 5
AR_F32, AR_BF16, AR_F16, AR_I32 = 0, 1, 2, 3
AR_SUM, AR_AVG, AR_MIN, AR_MAX = 0, 1, 2, 3
AR_ALGO_RING, AR_ALGO_FUSED, AR_ALGO_RHD, AR_ALGO_RING_STEPWISE, AR_ALGO_RHD_STEPWISE, AR_ALGO_RING_FP8 = range(6)
AR_ALGO_TREE, AR_ALGO_TREE_STEPWISE, AR_ALGO_AUTO = 6, 7, 8
AR_AUTO_STEP_NS, AR_AUTO_LINK_GBPS = 1900, 153
AR_MAX_RANKS = 64
AR_FP8_BLOCK = 128
AR_NORM_MAX_HIDDEN = 32768
AR_MAX_EXPERTS = 1024
AR_PRODUCT_MAX_WIDTH = 1 << 20
AR_ACT_SILU, AR_ACT_GELU, AR_ACT_GELU_TANH = 0, 1, 2
AR_NORM_L2, AR_NORM_MAX = 0, 1
AR_NOALLOC_WS_BYTES = 64 << 20

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libar.so")
_lib = None


class ArError(RuntimeError):
    def __init__(self, status: int, entry: str):
        self.status = status
        super().__init__(f"{entry}: {ar_status_string(status)}")


class _CallRecord(ctypes.Structure):
    _fields_ = [("seq", ctypes.c_uint64), ("entry", ctypes.c_char_p), ("nranks", ctypes.c_int),
                ("dtype", ctypes.c_int), ("op", ctypes.c_int), ("algo", ctypes.c_int), ("status", ctypes.c_int),
                ("count", ctypes.c_size_t)]


def lib_path() -> str:
    return _LIB_PATH


def lib():
    """Load libar.so (built in-tree by build.py). Raises if it is missing: there is no fallback path."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"libar.so not found at {_LIB_PATH}; build it first "
                               "(python -c 'import __graft_entry__ as g; g.build()')")
        L = ctypes.CDLL(_LIB_PATH)
        vp, sz, i32 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        L.ar_allreduce.argtypes = [vp, vp, i32, sz, i32, i32, i32, vp]
        L.ar_allreduce_ws.argtypes = [vp, vp, i32, sz, i32, i32, i32, vp, sz, vp]
        L.ar_allreduce_noalloc.argtypes = [vp, vp, i32, sz, i32, i32, i32, vp]
        L.ar_allreduce_workspace_size.argtypes = [i32, sz, i32, i32, i32, ctypes.POINTER(sz)]
        L.ar_allreduce_buckets.argtypes = [vp, vp, i32, vp, i32, i32, i32, i32, vp]
        L.ar_allreduce_tensors.argtypes = [vp, vp, vp, i32, i32, i32, i32, i32, vp]
        L.ar_reduce_scatter.argtypes = [vp, vp, i32, sz, i32, i32, vp]
        L.ar_all_gather.argtypes = [vp, vp, i32, sz, i32, vp]
        L.ar_bucket_plan.argtypes = [vp, i32, i32, i32, sz, vp, vp, vp, ctypes.POINTER(i32)]
        L.ar_bucket_pack.argtypes = [vp, i32, i32, vp]
        L.ar_bucket_unpack.argtypes = [vp, i32, i32, vp]
        L.ar_fp8_quant.argtypes = [vp, i32, sz, vp, vp, vp]
        L.ar_fp8_dequant.argtypes = [vp, vp, sz, vp, i32, vp]
        L.ar_auto_algo.argtypes = [i32, sz, i32]
        L.ar_chunk_bounds.argtypes = [i32, sz, vp]
        L.ar_epilogue.argtypes = [vp, vp, sz, i32, i32, i32, vp]
        f32 = ctypes.c_float
        L.ar_allreduce_rmsnorm.argtypes = [vp, i32, sz, sz, i32, vp, vp, i32, f32, vp, vp, vp, vp, vp, vp, vp]
        L.ar_allreduce_rmsnorm_bwd_workspace_size.argtypes = [sz, sz, ctypes.POINTER(sz)]
        L.ar_allreduce_rmsnorm_bwd.argtypes = [vp, i32, sz, sz, i32, vp, vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]
        L.ar_expert_rows.argtypes = [sz, i32, i32, i32, ctypes.POINTER(sz)]
        L.ar_expert_sort_workspace_size.argtypes = [sz, i32, i32, ctypes.POINTER(sz)]
        L.ar_expert_sort.argtypes = [vp, sz, i32, i32, i32, vp, vp, vp, vp, sz, vp, sz, vp]
        L.ar_expert_dispatch.argtypes = [vp, vp, vp, vp, vp, sz, i32, i32, sz, i32, vp, vp, sz, vp]
        L.ar_expert_combine.argtypes = [vp, vp, vp, vp, sz, i32, sz, i32, sz, vp, vp]
        L.ar_expert_combine_bwd.argtypes = [vp, vp, vp, vp, vp, vp, sz, i32, i32, sz, i32, sz, vp, vp, vp]
        L.ar_expert_gated.argtypes = [vp, vp, vp, sz, vp, vp, i32, sz, sz, sz, i32, i32, vp, vp, vp, vp]
        L.ar_expert_gated_bwd.argtypes = [vp, vp, vp, vp, vp, vp, sz, vp, vp, i32, sz, sz, sz, i32, i32, vp, vp, vp, vp,
                                          vp, sz, vp]
        L.ar_expert_linear.argtypes = [vp, vp, sz, vp, vp, i32, sz, sz, sz, i32, vp, vp]
        L.ar_expert_linear_bwd.argtypes = [vp, vp, vp, sz, vp, vp, i32, sz, sz, sz, i32, vp, vp, sz, vp]
        L.ar_grad_plan.argtypes = [vp, i32, vp, ctypes.POINTER(sz)]
        L.ar_grad_norm_workspace_size.argtypes = [sz, ctypes.POINTER(sz)]
        L.ar_grad_norm.argtypes = [vp, sz, i32, vp, vp, sz, vp]
        L.ar_grad_clip.argtypes = [vp, sz, i32, f32, f32, vp, vp, sz, vp]
        L.ar_status_string.argtypes = [i32]
        L.ar_status_string.restype = ctypes.c_char_p
        L.ar_last_call.argtypes = [ctypes.POINTER(_CallRecord)]
        for name in ("ar_allreduce", "ar_allreduce_ws", "ar_allreduce_noalloc", "ar_allreduce_workspace_size",
                     "ar_allreduce_buckets",
                     "ar_allreduce_tensors", "ar_reduce_scatter", "ar_all_gather", "ar_bucket_plan", "ar_bucket_pack",
                     "ar_bucket_unpack", "ar_fp8_quant", "ar_fp8_dequant", "ar_last_call", "ar_version",
                     "ar_auto_algo", "ar_chunk_bounds", "ar_epilogue", "ar_allreduce_rmsnorm",
                     "ar_allreduce_rmsnorm_bwd", "ar_allreduce_rmsnorm_bwd_workspace_size", "ar_expert_rows",
                     "ar_expert_sort", "ar_expert_sort_workspace_size", "ar_expert_dispatch", "ar_expert_combine",
                     "ar_expert_combine_bwd", "ar_expert_gated", "ar_expert_gated_bwd", "ar_expert_linear",
                     "ar_expert_linear_bwd", "ar_grad_plan", "ar_grad_norm_workspace_size", "ar_grad_norm",
                     "ar_grad_clip"):
            getattr(L, name).restype = i32
        _lib = L
    return _lib


# ------------------------------------------------------------------------------------------ marshalling
_DTYPE_CODES = {}


def dtype_code(t) -> int:
    if not _DTYPE_CODES:
        import torch
        _DTYPE_CODES.update({torch.float32: AR_F32, torch.bfloat16: AR_BF16, torch.float16: AR_F16,
                             torch.int32: AR_I32})
    if t not in _DTYPE_CODES:
        raise TypeError(f"unsupported dtype {t}; expected float32, bfloat16, float16 or int32")
    return _DTYPE_CODES[t]


def _stream(stream, device=None):
    """The HIP stream handle: `stream` (a torch stream or a raw handle), else the current stream of `device`."""
    import torch
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # the handle without a Stream object
        if raw is not None and device is not None and device.index is not None:
            return ctypes.c_void_p(raw(device.index))
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    if isinstance(stream, int):
        if not 0 <= stream < 2 ** 64 - 1:  # ctypes would cut it to 64 bits: to another stream, or the null stream
            raise ValueError("stream must be a torch stream or a raw handle")
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _on(device):
    """Make `device` current for a call (the library launches on the current device); no switch when it already
    is."""
    import torch
    if device.index is not None and device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def _gpu_tensor(t, what, dtype=None, device=None, min_numel=0):
    """Every tensor handed to the library: a contiguous GPU tensor (of `dtype`, on `device`, at least
    `min_numel` elements). A host tensor would give the kernels a host address."""
    if t.device.type != "cuda":
        raise ValueError(f"{what} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{what} must be on {device}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be {dtype}, not {t.dtype}")
    if t.numel() < min_numel:
        raise ValueError(f"{what} must hold at least {min_numel} elements")
    return t


def _check(rc: int, entry: str):
    if rc != AR_OK:
        raise ArError(rc, entry)


def _rank_arrays(ins, outs):
    """Check every rank tensor (all before any address is read), then the host arrays of their addresses. The
    checks are the per-tensor ones of _gpu_tensor plus equal dtype, element count and device, written with the
    cheapest accessors: this runs on every call, and for small messages it is most of the call's host time."""
    n = len(ins)
    if n != len(outs) or not n:
        raise ValueError("ins and outs must be non-empty lists of the same length (one tensor per rank)")
    t0 = ins[0]
    dt0, ne0, dev0 = t0.dtype, t0.numel(), t0.get_device()
    for t in (*ins, *outs):
        # every rank must call with the same count and dtype; one call enforces it
        if t.dtype is not dt0 or t.numel() != ne0 or t.get_device() != dev0:
            raise ValueError("all rank tensors must share dtype, element count and device")
        if not t.is_contiguous():
            raise ValueError("rank tensors must be contiguous")
    if dev0 < 0:  # get_device() is -1 for host tensors
        raise ValueError("rank tensors must be GPU tensors")
    arr_in = (ctypes.c_void_p * n)(*[t.data_ptr() for t in ins])
    arr_out = (ctypes.c_void_p * n)(*[t.data_ptr() for t in outs])
    return arr_in, arr_out, n, ne0, dtype_code(dt0)


def ar_allreduce(ins, outs, op=AR_SUM, algo=AR_ALGO_RING, stream=None):
    """All-reduce ins[r] -> outs[r] for every rank r (outs[r] may be ins[r])."""
    arr_in, arr_out, n, count, dt = _rank_arrays(ins, outs)
    dev = ins[0].device
    with _on(dev):
        _check(lib().ar_allreduce(arr_in, arr_out, n, count, dt, op, algo, _stream(stream, dev)), "ar_allreduce")


def ar_allreduce_workspace_size(nranks, count, dtype, op, algo) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ar_allreduce_workspace_size(nranks, count, dtype, op, algo, ctypes.byref(out)),
           "ar_allreduce_workspace_size")
    return out.value


def ar_allreduce_ws(ins, outs, op=AR_SUM, algo=AR_ALGO_RING, workspace=None, stream=None):
    """ar_allreduce with a caller workspace tensor (any dtype, contiguous, on the same GPU)."""
    if workspace is not None and ins:
        _gpu_tensor(workspace, "workspace", device=ins[0].device)
    arr_in, arr_out, n, count, dt = _rank_arrays(ins, outs)
    dev = ins[0].device
    wp = ctypes.c_void_p(workspace.data_ptr()) if workspace is not None else ctypes.c_void_p(0)
    wb = workspace.numel() * workspace.element_size() if workspace is not None else 0
    with _on(dev):
        _check(lib().ar_allreduce_ws(arr_in, arr_out, n, count, dt, op, algo, wp, wb, _stream(stream, dev)),
               "ar_allreduce_ws")


def ar_allreduce_noalloc(ins, outs, op=AR_SUM, algo=AR_ALGO_RING, stream=None):
    """ar_allreduce_ws with the library's fixed per-GPU scratch instead of a caller workspace (allocates nothing;
    calls that overlap on one GPU race on that scratch)."""
    arr_in, arr_out, n, count, dt = _rank_arrays(ins, outs)
    dev = ins[0].device
    with _on(dev):
        _check(lib().ar_allreduce_noalloc(arr_in, arr_out, n, count, dt, op, algo, _stream(stream, dev)),
               "ar_allreduce_noalloc")


def ar_allreduce_buckets(flat_ins, flat_outs, bucket_count, op=AR_SUM, algo=AR_ALGO_RING, stream=None):
    """All-reduce every bucket of the flat per-rank tensors in one launch (bucket_count: the plan's counts)."""
    arr_in, arr_out, n, total, dt = _rank_arrays(flat_ins, flat_outs)
    counts = np.ascontiguousarray(bucket_count, dtype=np.int64)
    if int(counts.sum()) > total:
        raise ValueError("the buckets do not fit in the flat tensors")
    dev = flat_ins[0].device
    with _on(dev):
        _check(lib().ar_allreduce_buckets(arr_in, arr_out, n, counts.ctypes.data, counts.size, dt, op, algo,
                                          _stream(stream, dev)), "ar_allreduce_buckets")


def ar_allreduce_tensors(descs, in_ptrs, out_ptrs, ntensors, nranks, dtype, op=AR_AVG, algo=AR_ALGO_RING,
                         stream=None):
    """descs: device int64 tensor [ntensors, 4] laid out as ar_tensor_desc; in_ptrs/out_ptrs: device int64
    tensors [ntensors * nranks] of device addresses (entry t * nranks + r)."""
    import torch
    dev = descs.device
    _gpu_tensor(descs, "descs", torch.int64, dev, 4 * ntensors)
    _gpu_tensor(in_ptrs, "in_ptrs", torch.int64, dev, ntensors * nranks)
    _gpu_tensor(out_ptrs, "out_ptrs", torch.int64, dev, ntensors * nranks)
    with _on(dev):
        _check(lib().ar_allreduce_tensors(ctypes.c_void_p(descs.data_ptr()), ctypes.c_void_p(in_ptrs.data_ptr()),
                                          ctypes.c_void_p(out_ptrs.data_ptr()), ntensors, nranks, dtype, op, algo,
                                          _stream(stream, dev)), "ar_allreduce_tensors")


def ar_chunk_bounds(nranks, count):
    """The library's balanced split (host only): chunk c = [lo[c], lo[c+1]), a list of nranks + 1 ints."""
    lo = (ctypes.c_int64 * (nranks + 1))() if 1 <= nranks <= AR_MAX_RANKS else None
    _check(lib().ar_chunk_bounds(nranks, count, lo), "ar_chunk_bounds")
    return list(lo)


def chunk_bounds(count, nranks):
    """ar_chunk_bounds with the arguments in (count, nranks) order."""
    return ar_chunk_bounds(nranks, count)


def _ptr(t):
    return t.data_ptr() if t is not None and t.numel() > 0 else 0


def _chunk_tensors(full, parts, what):
    """Check N full tensors and N chunk tensors (None allowed for an empty chunk) of one dtype and device."""
    n = len(full)
    if n == 0 or len(parts) != n:
        raise ValueError("one full tensor and one chunk tensor per rank")
    t0 = full[0]
    for t in full:
        if t.numel() != t0.numel():
            raise ValueError("all full tensors must have the same element count")
        _gpu_tensor(t, "full tensors", t0.dtype, t0.device)
    lo = chunk_bounds(t0.numel(), n)
    for c, p in enumerate(parts):
        want = lo[c + 1] - lo[c]
        if p is None:
            if want:
                raise ValueError(f"{what}[{c}] is None but chunk {c} has {want} elements")
            continue
        if p.numel() != want:
            raise ValueError(f"{what}[{c}] must hold exactly chunk {c} of the balanced split ({want} elements)")
        if want:
            _gpu_tensor(p, f"{what}[{c}]", t0.dtype, t0.device)
    return n, t0.numel(), t0.device


def ar_reduce_scatter(ins, outs, op=AR_SUM, stream=None):
    """ins: N full tensors; outs[c]: a tensor of chunk c's length (the balanced split) receiving chunk c."""
    n, count, dev = _chunk_tensors(ins, outs, "outs")
    arr_in = (ctypes.c_void_p * n)(*[t.data_ptr() for t in ins])
    arr_out = (ctypes.c_void_p * n)(*[_ptr(o) for o in outs])
    with _on(dev):
        _check(lib().ar_reduce_scatter(arr_in, arr_out, n, count, dtype_code(ins[0].dtype), op,
                                       _stream(stream, dev)), "ar_reduce_scatter")


def ar_all_gather(ins, outs, stream=None):
    """ins[r]: rank r's chunk (the balanced split of the outputs' length); outs: N full tensors."""
    n, count, dev = _chunk_tensors(outs, ins, "ins")
    arr_in = (ctypes.c_void_p * n)(*[_ptr(i) for i in ins])
    arr_out = (ctypes.c_void_p * n)(*[t.data_ptr() for t in outs])
    with _on(dev):
        _check(lib().ar_all_gather(arr_in, arr_out, n, count, dtype_code(outs[0].dtype), _stream(stream, dev)),
               "ar_all_gather")


def ar_bucket_plan(numels, dtype, nranks, cap_bytes=25 << 20):
    """Host-only plan; returns (bucket_of int32[T], offset_of int64[T], bucket_count int64[nbuckets])."""
    numels = np.ascontiguousarray(numels, dtype=np.int64)
    nt = numels.size
    bucket_of = np.zeros(max(nt, 1), np.int32)
    offset_of = np.zeros(max(nt, 1), np.int64)
    bcount = np.zeros(max(nt, 1), np.int64)
    nb = ctypes.c_int(0)
    _check(lib().ar_bucket_plan(numels.ctypes.data, nt, dtype, nranks, cap_bytes, bucket_of.ctypes.data,
                                offset_of.ctypes.data, bcount.ctypes.data, ctypes.byref(nb)), "ar_bucket_plan")
    return bucket_of[:nt], offset_of[:nt], bcount[: nb.value]


def make_copy_descs(tasks, device):
    """tasks: iterable of (src_ptr, dst_ptr, numel, zero_pad_after) -> device int64 tensor [ndescs, 4]
    laid out as ar_copy_desc (two pointers, two int64)."""
    import torch
    host = np.array(list(tasks), dtype=np.uint64).reshape(-1, 4).view(np.int64)
    return torch.from_numpy(host).to(device)


def _copy_descs(descs):
    import torch
    _gpu_tensor(descs, "descs", torch.int64)
    if descs.dim() != 2 or descs.shape[1] != 4:
        raise ValueError("descs must be an int64 tensor [ndescs, 4] (ar_copy_desc rows)")
    return descs.device


def ar_bucket_pack(descs, dtype, stream=None):
    dev = _copy_descs(descs)
    with _on(dev):
        _check(lib().ar_bucket_pack(ctypes.c_void_p(descs.data_ptr()), descs.shape[0], dtype, _stream(stream, dev)),
               "ar_bucket_pack")


def ar_bucket_unpack(descs, dtype, stream=None):
    dev = _copy_descs(descs)
    with _on(dev):
        _check(lib().ar_bucket_unpack(ctypes.c_void_p(descs.data_ptr()), descs.shape[0], dtype,
                                      _stream(stream, dev)), "ar_bucket_unpack")


def ar_fp8_quant(x, codes, scales, stream=None):
    """x: float32/bfloat16 GPU tensor; codes: uint8[numel]; scales: float32[ceil(numel/128)]."""
    import torch
    dev = _gpu_tensor(x, "x").device
    _gpu_tensor(codes, "codes", torch.uint8, dev, x.numel())
    _gpu_tensor(scales, "scales", torch.float32, dev, (x.numel() + AR_FP8_BLOCK - 1) // AR_FP8_BLOCK)
    with _on(dev):
        _check(lib().ar_fp8_quant(ctypes.c_void_p(x.data_ptr()), dtype_code(x.dtype), x.numel(),
                                  ctypes.c_void_p(codes.data_ptr()), ctypes.c_void_p(scales.data_ptr()),
                                  _stream(stream, dev)), "ar_fp8_quant")


def ar_fp8_dequant(codes, scales, out, stream=None):
    """codes: uint8[numel]; scales: float32[ceil(numel/128)]; out: float32/bfloat16 GPU tensor of numel."""
    import torch
    dev = _gpu_tensor(out, "out").device
    _gpu_tensor(codes, "codes", torch.uint8, dev, out.numel())
    _gpu_tensor(scales, "scales", torch.float32, dev, (out.numel() + AR_FP8_BLOCK - 1) // AR_FP8_BLOCK)
    with _on(dev):
        _check(lib().ar_fp8_dequant(ctypes.c_void_p(codes.data_ptr()), ctypes.c_void_p(scales.data_ptr()),
                                    out.numel(), ctypes.c_void_p(out.data_ptr()), dtype_code(out.dtype),
                                    _stream(stream, dev)), "ar_fp8_dequant")


def ar_epilogue(acc, out, op=AR_SUM, nranks=1, stream=None):
    """acc: float32 GPU tensor of partial results (int32 when `out` is int32); out: GPU tensor of as many elements,
    whose dtype is the output type (may be acc itself for float32/int32)."""
    import torch
    dev = _gpu_tensor(acc, "acc").device
    _gpu_tensor(out, "out", None, dev)
    _gpu_tensor(acc, "acc", torch.int32 if out.dtype == torch.int32 else torch.float32)
    if out.numel() != acc.numel():
        raise ValueError("acc and out must hold the same number of elements")
    with _on(dev):
        _check(lib().ar_epilogue(ctypes.c_void_p(acc.data_ptr()), ctypes.c_void_p(out.data_ptr()), acc.numel(),
                                 dtype_code(out.dtype), op, nranks, _stream(stream, dev)), "ar_epilogue")


def ar_auto_algo(nranks, count, dtype) -> int:
    """The algorithm AR_ALGO_AUTO runs for this shape (AR_ALGO_TREE or AR_ALGO_RING)."""
    a = lib().ar_auto_algo(nranks, count, dtype)
    if a < 0:
        raise ArError(-a, "ar_auto_algo")
    return a


def ar_status_string(status: int) -> str:
    return lib().ar_status_string(status).decode()


def ar_last_call():
    rec = _CallRecord()
    if lib().ar_last_call(ctypes.byref(rec)) != AR_OK:
        return None
    return {"seq": rec.seq, "entry": rec.entry.decode() if rec.entry else None, "nranks": rec.nranks,
            "count": rec.count, "dtype": rec.dtype, "op": rec.op, "algo": rec.algo, "status": rec.status}


def ar_version() -> int:
    return lib().ar_version()


# ------------------------------------------------------------------------------------------ block boundary
_native = None  # the compiled argument checks; False where they cannot be loaded


def _load_native():
    """Load and bind the compiled argument checks (_marshal.so). They do what the checks below do, for arguments that
    plainly fit, in a tenth of the time; without them every call goes through the ones below."""
    global _native
    L = lib()
    try:
        import torch
        from . import _marshal
        entries = (L.ar_allreduce_rmsnorm, L.ar_allreduce_rmsnorm_bwd, L.ar_expert_sort, L.ar_expert_dispatch,
                   L.ar_expert_combine, L.ar_expert_combine_bwd)
        products = (L.ar_expert_gated, L.ar_expert_gated_bwd, L.ar_expert_linear, L.ar_expert_linear_bwd, L.ar_grad_norm,
                    L.ar_grad_clip)
        _marshal.bind_products(*(ctypes.cast(f, ctypes.c_void_p).value for f in products))
        _marshal.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in entries), torch._C._cuda_getDevice,
                      torch._C._cuda_getCurrentRawStream)
        _native = _marshal
    except (ImportError, AttributeError) as e:
        import warnings
        warnings.warn(f"_marshal.so is missing or does not fit this torch ({e}): checking arguments in Python, slower")
        _native = False
    return _native


def _done(rc, entry):
    """Whether a compiled call went through (None: its arguments did not plainly fit); raises for an error status."""
    if rc is None:
        return False
    if rc != AR_OK:
        raise ArError(rc, entry)
    return True


def _addr(t, what, dtypes, shape, dev):
    """The address of a tensor that must be contiguous, of one of `dtypes`, of `shape`, on GPU `dev` (an index)."""
    if t.dtype not in dtypes:
        raise ValueError(f"{what} must be {' or '.join(map(str, dtypes))}, not {t.dtype}")
    if t.get_device() != dev or dev < 0:
        raise ValueError(f"{what} must be a GPU tensor on the device of the others")
    if t.shape != shape:
        raise ValueError(f"{what} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _opt(t, what, dtypes, shape, dev):
    return None if t is None else _addr(t, what, dtypes, shape, dev)


def _rank_addrs(ts, n, what, dtypes, shape, dev):
    if len(ts) != n:
        raise ValueError(f"{what} must hold one tensor per rank")
    return (ctypes.c_void_p * n)(*[_addr(t, what, dtypes, shape, dev) for t in ts])


_FLOATS = None


def _kinds():
    """(the dtypes of rows, of 8-bit rows, fp32 alone, int32 alone)"""
    global _FLOATS
    if _FLOATS is None:
        import torch
        _FLOATS = ((torch.float32, torch.bfloat16, torch.float16), (torch.uint8, torch.float8_e4m3fn),
                   (torch.float32,), (torch.int32,))
    return _FLOATS


def _matrix(t, what):
    rows_of = _kinds()[0]
    if t.dim() != 2:
        raise ValueError(f"{what} must be a matrix [rows, hidden]")
    if t.dtype not in rows_of:
        raise ValueError(f"{what} must be float32, bfloat16 or float16, not {t.dtype}")
    return t.shape, t.dtype, t.get_device()


def _sizes(**named):
    """Sizes as C takes them; ctypes would cut a larger number to its low bits, and a negative one to a huge one."""
    for what, v in named.items():
        if not 0 <= v < 2 ** 64:
            raise ValueError(f"{what} must be a size of 64 bits, not {v}")
    return tuple(named.values())


def _ints(**named):
    """Numbers that C takes as int."""
    for what, v in named.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{what} must be an int of 32 bits, not {v}")
    return tuple(named.values())


def _reals(**named):
    """Numbers that C takes as float. A tensor's value would have to be waited for, so only one on the host is a number."""
    import torch
    for what, v in named.items():
        if torch.is_tensor(v) and v.device.type != "cpu":
            raise ValueError(f"{what} must be a number, not a tensor on {v.device}: its value would be waited for")
        try:
            named[what] = float(v)
        except (TypeError, ValueError, OverflowError, RuntimeError) as e:
            raise ValueError(f"{what} must be a number: {e}") from None
    return tuple(named.values())


def _workspace_arg(ws, dev):
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous GPU tensor on the device of the others")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def ar_allreduce_rmsnorm(ins, gamma, outs, residual=None, residual_out=None, rstd=None, out_scales=None, saved=None,
                         saved_scales=None, eps=1e-5, stream=None):
    """Sum of the ranks' partial products ins[r] plus the residual, and its root-mean-square norm to every outs[r].

    ins: list of [rows, hidden] tensors, one per rank. gamma: [hidden] of their dtype or float32. outs: list of
    [rows, hidden] tensors of the same dtype (outs[r] may be ins[r]), or, with out_scales (a list of float32
    [rows, ceil(hidden/128)]), of uint8 / float8_e4m3fn codes. residual_out receives the new residual (it may be
    `residual`), rstd float32 [rows], saved and saved_scales the new residual in 8 bits."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.rmsnorm(ins, gamma, outs, residual, residual_out, rstd, out_scales, saved, saved_scales, eps,
                                      stream), "ar_allreduce_rmsnorm"):
        return
    kinds = _kinds()
    shape, dt, dev = _matrix(ins[0], "ins") if len(ins) else (None, None, -1)
    if shape is None:
        raise ValueError("ins must hold one tensor per rank")
    own, n = (dt,), len(ins)
    rows, hidden = shape
    nb = (rows, (hidden + AR_FP8_BLOCK - 1) // AR_FP8_BLOCK)
    arr_in = _rank_addrs(ins, n, "ins", own, shape, dev)
    arr_out = _rank_addrs(outs, n, "outs", own if out_scales is None else kinds[1], shape, dev)
    arr_sc = None if out_scales is None else _rank_addrs(out_scales, n, "out_scales", kinds[2], nb, dev)
    args = (_opt(residual, "residual", own, shape, dev),
            _addr(gamma, "gamma", (dt, kinds[2][0]), (hidden,), dev), dtype_code(gamma.dtype), eps, arr_out, arr_sc,
            _opt(residual_out, "residual_out", own, shape, dev), _opt(rstd, "rstd", kinds[2], (rows,), dev),
            _opt(saved, "saved", kinds[1], shape, dev), _opt(saved_scales, "saved_scales", kinds[2], nb, dev))
    device = ins[0].device
    with _on(device):
        _check(lib().ar_allreduce_rmsnorm(arr_in, n, rows, hidden, dtype_code(dt), *args, _stream(stream, device)),
               "ar_allreduce_rmsnorm")


def ar_allreduce_rmsnorm_bwd_workspace_size(rows, hidden) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ar_allreduce_rmsnorm_bwd_workspace_size(*_sizes(rows=rows, hidden=hidden), ctypes.byref(out)),
           "ar_allreduce_rmsnorm_bwd_workspace_size")
    return out.value


def ar_allreduce_rmsnorm_bwd(ins, saved, gamma, rstd, outs, dgamma, saved_scales=None, residual_grad=None,
                             workspace=None, stream=None):
    """The gradient of ar_allreduce_rmsnorm: ins are the ranks' partial gradients of y, saved the forward's
    residual_out (or its 8-bit `saved`, with saved_scales), rstd the forward's. outs[r] receives the gradient of
    every rank's partial product and of the residual, dgamma (float32 [hidden]) the weight's. workspace: a GPU tensor
    of ar_allreduce_rmsnorm_bwd_workspace_size(rows, hidden) bytes."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.rmsnorm_bwd(ins, saved, gamma, rstd, outs, dgamma, saved_scales, residual_grad, workspace,
                                          stream), "ar_allreduce_rmsnorm_bwd"):
        return
    kinds = _kinds()
    shape, dt, dev = _matrix(ins[0], "ins") if len(ins) else (None, None, -1)
    if shape is None:
        raise ValueError("ins must hold one tensor per rank")
    own, n = (dt,), len(ins)
    rows, hidden = shape
    nb = (rows, (hidden + AR_FP8_BLOCK - 1) // AR_FP8_BLOCK)
    arr_in = _rank_addrs(ins, n, "ins", own, shape, dev)
    arr_out = _rank_addrs(outs, n, "outs", own, shape, dev)
    args = (_addr(saved, "saved", own if saved_scales is None else kinds[1], shape, dev),
            _opt(saved_scales, "saved_scales", kinds[2], nb, dev),
            _addr(gamma, "gamma", (dt, kinds[2][0]), (hidden,), dev), dtype_code(gamma.dtype),
            _addr(rstd, "rstd", kinds[2], (rows,), dev), _opt(residual_grad, "residual_grad", own, shape, dev),
            arr_out, _addr(dgamma, "dgamma", kinds[2], (hidden,), dev), *_workspace_arg(workspace, dev))
    device = ins[0].device
    with _on(device):
        _check(lib().ar_allreduce_rmsnorm_bwd(arr_in, n, rows, hidden, dtype_code(dt), *args,
                                              _stream(stream, device)), "ar_allreduce_rmsnorm_bwd")


def ar_expert_rows(tokens, k, nexperts, align=1) -> int:
    """The most rows that tokens * k slots take when sorted (what src and the sorted rows must hold)."""
    out = ctypes.c_size_t(0)
    _check(lib().ar_expert_rows(*_sizes(tokens=tokens), *_ints(k=k, nexperts=nexperts, align=align), ctypes.byref(out)),
           "ar_expert_rows")
    return out.value


def ar_expert_sort_workspace_size(tokens, k, nexperts) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ar_expert_sort_workspace_size(*_sizes(tokens=tokens), *_ints(k=k, nexperts=nexperts), ctypes.byref(out)),
           "ar_expert_sort_workspace_size")
    return out.value


def ar_expert_sort(ids, offsets, counts, pos, src, align=1, workspace=None, stream=None):
    """Sort the slots ids[tokens, k] (int32; an id outside [0, experts) takes no row) by expert: offsets
    [experts + 1], counts [experts], pos [tokens, k] (a slot's row or -1) and src [rows] (a row's slot or -1), all
    int32. Segments start on multiples of `align`; rows >= ar_expert_rows(tokens, k, experts, align)."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.expert_sort(ids, offsets, counts, pos, src, align, workspace, stream), "ar_expert_sort"):
        return
    i32 = _kinds()[3]
    if ids.dim() != 2:
        raise ValueError("ids must be a matrix [tokens, k]")
    tokens, k = ids.shape
    dev = ids.get_device()
    experts, rows = counts.numel(), src.numel()
    args = (_addr(offsets, "offsets", i32, (experts + 1,), dev), _addr(counts, "counts", i32, (experts,), dev),
            _addr(pos, "pos", i32, ids.shape, dev), _addr(src, "src", i32, (rows,), dev))
    device = ids.device
    at = _addr(ids, "ids", i32, ids.shape, dev)
    numbers = _ints(k=k, experts=experts, align=align)
    with _on(device):
        _check(lib().ar_expert_sort(at, tokens, *numbers, *args, rows, *_workspace_arg(workspace, dev),
                                    _stream(stream, device)), "ar_expert_sort")


def _pads(offsets, counts, dev):
    """The addresses of offsets and counts (both or neither), and the number of experts."""
    if (offsets is None) != (counts is None):
        raise ValueError("offsets and counts go together")
    if counts is None:
        return None, None, 1
    i32, experts = _kinds()[3], counts.numel()
    return (_addr(offsets, "offsets", i32, (experts + 1,), dev), _addr(counts, "counts", i32, (experts,), dev), experts)


def ar_expert_dispatch(x, pos, offsets, counts, xs, x_scales=None, xs_scales=None, stream=None):
    """xs[pos[t, j]] = x[t] for the rows of x [tokens, hidden] (float32, bfloat16, float16, or uint8 /
    float8_e4m3fn with x_scales, whose rows go to xs_scales). The pad rows that offsets and counts describe are
    zeroed (both None: there are none)."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.expert_dispatch(x, pos, offsets, counts, xs, x_scales, xs_scales, stream), "ar_expert_dispatch"):
        return
    kinds = _kinds()
    if x.dim() != 2 or xs.dim() != 2 or pos.dim() != 2:
        raise ValueError("x, xs and pos must be matrices")
    dt, dev = x.dtype, x.get_device()
    if dt not in (kinds[1] if x_scales is not None else kinds[0]):
        raise ValueError(f"x must be 8-bit rows with x_scales, or float32, bfloat16 or float16 without, not {dt}")
    if (x_scales is None) != (xs_scales is None):
        raise ValueError("x_scales and xs_scales go together")
    tokens, hidden = x.shape
    rows, k, nb = xs.shape[0], pos.shape[1], (hidden + AR_FP8_BLOCK - 1) // AR_FP8_BLOCK
    at = (_addr(x, "x", (dt,), x.shape, dev), _opt(x_scales, "x_scales", kinds[2], (tokens, nb), dev),
          _addr(pos, "pos", kinds[3], (tokens, k), dev))
    off, cnt, experts = _pads(offsets, counts, dev)
    to = (_addr(xs, "xs", (dt,), (rows, hidden), dev), _opt(xs_scales, "xs_scales", kinds[2], (rows, nb), dev))
    numbers = _ints(k=k, experts=experts)
    device = x.device
    with _on(device):
        _check(lib().ar_expert_dispatch(*at, off, cnt, tokens, *numbers, hidden, x.element_size(), *to, rows,
                                        _stream(stream, device)), "ar_expert_dispatch")


def ar_expert_combine(ys, pos, out, weights=None, addend=None, stream=None):
    """out[t] = sum_j weights[t, j] ys[pos[t, j]] + addend[t]; weights float32 [tokens, k] (None: 1, the gradient of
    ar_expert_dispatch), addend [tokens, hidden] (may be `out`)."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.expert_combine(ys, pos, out, weights, addend, stream), "ar_expert_combine"):
        return
    kinds = _kinds()
    shape, dt, dev = _matrix(out, "out")
    if ys.dim() != 2 or pos.dim() != 2:
        raise ValueError("ys and pos must be matrices")
    (tokens, hidden), rows, k = shape, ys.shape[0], pos.shape[1]
    at = (_addr(ys, "ys", (dt,), (rows, hidden), dev), _addr(pos, "pos", kinds[3], (tokens, k), dev),
          _opt(weights, "weights", kinds[2], (tokens, k), dev), _opt(addend, "addend", (dt,), shape, dev))
    device = out.device
    to = _addr(out, "out", (dt,), shape, dev)
    with _on(device):
        _check(lib().ar_expert_combine(*at, tokens, *_ints(k=k), hidden, dtype_code(dt), rows, to, _stream(stream, device)),
               "ar_expert_combine")


def ar_expert_combine_bwd(dout, ys, pos, weights, offsets, counts, dys, dweights, stream=None):
    """The gradient of ar_expert_combine: dys[pos[t, j]] = weights[t, j] dout[t] (pad rows zeroed as in
    ar_expert_dispatch; dys may be ys) and dweights[t, j] = <dout[t], ys[pos[t, j]]> (float32 [tokens, k])."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.expert_combine_bwd(dout, ys, pos, weights, offsets, counts, dys, dweights, stream), "ar_expert_combine_bwd"):
        return
    kinds = _kinds()
    shape, dt, dev = _matrix(dout, "dout")
    if ys.dim() != 2 or pos.dim() != 2:
        raise ValueError("ys and pos must be matrices")
    (tokens, hidden), rows, k = shape, ys.shape[0], pos.shape[1]
    at = (_addr(dout, "dout", (dt,), shape, dev), _addr(ys, "ys", (dt,), (rows, hidden), dev),
          _addr(pos, "pos", kinds[3], (tokens, k), dev), _addr(weights, "weights", kinds[2], (tokens, k), dev))
    off, cnt, experts = _pads(offsets, counts, dev)
    to = (_addr(dys, "dys", (dt,), (rows, hidden), dev), _addr(dweights, "dweights", kinds[2], (tokens, k), dev))
    device = dout.device
    with _on(device):
        _check(lib().ar_expert_combine_bwd(*at, off, cnt, tokens, *_ints(k=k, experts=experts), hidden, dtype_code(dt), rows, *to,
                                           _stream(stream, device)), "ar_expert_combine_bwd")


# ------------------------------------------------------------------------------------------ experts' products
def _segments(offsets, counts, dev):
    """The addresses of offsets and counts (counts alone may be None; both: one segment of all rows), and the number
    of experts (None without offsets)."""
    if offsets is None:
        if counts is not None:
            raise ValueError("counts need offsets")
        return None, None, None
    i32, experts = _kinds()[3], offsets.numel() - 1
    if experts < 1:
        raise ValueError("offsets must hold one entry per expert and the end")
    return (_addr(offsets, "offsets", i32, (experts + 1,), dev), _opt(counts, "counts", i32, (experts,), dev), experts)


def _weights(w, what, dt, experts, out, inside, dev):
    """The address of a weight [experts, out, inside] (without segments also [out, inside]) whose matrices are dense but
    may lie apart, and the elements between them."""
    if w is None:
        return None, out * inside
    shape = (1 if experts is None else experts, out, inside)
    if w.dim() == 2 and experts is None:
        w = w.unsqueeze(0)
    if w.dtype is not dt or tuple(w.shape) != shape:
        raise ValueError(f"{what} must be {dt} of the shape {shape}, not {w.dtype} {tuple(w.shape)}")
    if w.get_device() != dev or dev < 0:
        raise ValueError(f"{what} must be a GPU tensor on the device of the others")
    if not w[0].is_contiguous():
        raise ValueError(f"{what} must hold dense matrices")
    return w.data_ptr(), w.stride(0) if shape[0] > 1 else out * inside


def _pair(first, second, what):
    """Two weights of one call lie alike: the elements between their matrices."""
    if first[1] != second[1]:
        raise ValueError(f"{what} must have the same distance between their matrices")
    return first[0], second[0], first[1]


def ar_expert_gated(xs, w_gate, w_up, out, offsets=None, counts=None, gate=None, up=None, act=AR_ACT_SILU, stream=None):
    """out = act(xs w_gate[e]^T) * (xs w_up[e]^T) for the rows of every expert's segment (offsets, counts as
    ar_expert_sort wrote them; both None: one matrix for all rows). xs [rows, hidden], out [rows, inner]; w_gate and w_up
    [experts, inner, hidden] (without segments also [inner, hidden]) may be parts of one tensor, such as w[:, :inner] and
    w[:, inner:]. gate, up [rows, inner] receive the two products for ar_expert_gated_bwd. Rows outside the segments are
    neither read nor written."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.expert_gated(xs, w_gate, w_up, out, offsets, counts, gate, up, act, stream), "ar_expert_gated"):
        return
    shape, dt, dev = _matrix(xs, "xs")
    if out.dim() != 2:
        raise ValueError("out must be a matrix [rows, inner]")
    (rows, hidden), own = shape, (dt,)
    wide = (rows, out.shape[1])
    off, cnt, experts = _segments(offsets, counts, dev)
    at = _addr(xs, "xs", own, shape, dev)
    w = _pair(_weights(w_gate, "w_gate", dt, experts, wide[1], hidden, dev),
              _weights(w_up, "w_up", dt, experts, wide[1], hidden, dev), "w_gate and w_up")
    to = (_addr(out, "out", own, wide, dev), _opt(gate, "gate", own, wide, dev), _opt(up, "up", own, wide, dev))
    numbers = _ints(experts=1 if experts is None else experts)
    device = xs.device
    with _on(device):
        _check(lib().ar_expert_gated(at, *w, off, cnt, *numbers, rows, hidden, wide[1], dtype_code(dt), *_ints(act=act), *to,
                                     _stream(stream, device)), "ar_expert_gated")


def ar_expert_gated_bwd(dout, gate, up, xs, w_gate, w_up, dgate, dup, dxs=None, dw_gate=None, dw_up=None, offsets=None,
                        counts=None, act=AR_ACT_SILU, stream=None):
    """The gradient of ar_expert_gated: dout, gate and up [rows, inner] (gate and up as the forward wrote them) give dgate
    and dup [rows, inner] (either may be dout, gate or up), and of these dxs [rows, hidden] (None: not wanted; w_gate and
    w_up may then be None) and the weights' gradients dw_gate, dw_up [experts, inner, hidden] (None: not wanted; xs may
    then be None), which may be parts of one tensor as the weights may."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.expert_gated_bwd(dout, gate, up, xs, w_gate, w_up, dgate, dup, dxs, dw_gate, dw_up, offsets, counts,
                                               act, stream), "ar_expert_gated_bwd"):
        return
    wide, dt, dev = _matrix(dout, "dout")
    rows, inner = wide
    known = [t for t in (xs, dxs) if t is not None]
    if known and known[0].dim() != 2:
        raise ValueError("xs and dxs must be matrices [rows, hidden]")
    if not known:  # the gradients of the two products alone
        if any(t is not None for t in (dw_gate, dw_up)):
            raise ValueError("dw_gate and dw_up need xs")
        w_gate = w_up = None
    if (dw_gate is None) != (dw_up is None):
        raise ValueError("dw_gate and dw_up go together")
    if dw_gate is not None and xs is None:
        raise ValueError("dw_gate and dw_up need xs")
    if dxs is not None and (w_gate is None or w_up is None):
        raise ValueError("dxs needs w_gate and w_up")
    hidden = known[0].shape[1] if known else 1
    own, narrow = (dt,), (rows, hidden)
    off, cnt, experts = _segments(offsets, counts, dev)
    at = (_addr(dout, "dout", own, wide, dev), _addr(gate, "gate", own, wide, dev), _addr(up, "up", own, wide, dev),
          _opt(xs, "xs", own, narrow, dev))
    both = lambda g, u, what: _pair(_weights(g, "w_gate", dt, experts, inner, hidden, dev),
                                    _weights(u, "w_up", dt, experts, inner, hidden, dev), what)
    w = both(w_gate, w_up, "w_gate and w_up") if dxs is not None else (None, None, inner * hidden)
    to = (_addr(dgate, "dgate", own, wide, dev), _addr(dup, "dup", own, wide, dev), _opt(dxs, "dxs", own, narrow, dev),
          *both(dw_gate, dw_up, "dw_gate and dw_up"))
    numbers = _ints(experts=1 if experts is None else experts)
    device = dout.device
    with _on(device):
        _check(lib().ar_expert_gated_bwd(*at, *w, off, cnt, *numbers, rows, hidden, inner, dtype_code(dt), *_ints(act=act),
                                         *to, _stream(stream, device)), "ar_expert_gated_bwd")


def ar_expert_linear(xs, w, out, offsets=None, counts=None, stream=None):
    """out = xs w[e]^T for the rows of every expert's segment: xs [rows, in], w [experts, out, in] (without segments also
    [out, in]), out [rows, out]. Segments and weights as in ar_expert_gated."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.expert_linear(xs, w, out, offsets, counts, stream), "ar_expert_linear"):
        return
    shape, dt, dev = _matrix(xs, "xs")
    if out.dim() != 2:
        raise ValueError("out must be a matrix [rows, out]")
    rows, inside = shape
    off, cnt, experts = _segments(offsets, counts, dev)
    at = _addr(xs, "xs", (dt,), shape, dev)
    if w is None:
        raise ValueError("w must be a tensor")
    weight = _weights(w, "w", dt, experts, out.shape[1], inside, dev)
    to = _addr(out, "out", (dt,), (rows, out.shape[1]), dev)
    numbers = _ints(experts=1 if experts is None else experts)
    device = xs.device
    with _on(device):
        _check(lib().ar_expert_linear(at, *weight, off, cnt, *numbers, rows, inside, out.shape[1], dtype_code(dt), to,
                                      _stream(stream, device)), "ar_expert_linear")


def ar_expert_linear_bwd(dout, xs, w, dxs=None, dw=None, offsets=None, counts=None, stream=None):
    """The gradient of ar_expert_linear: dxs = dout w[e] [rows, in] (None: not wanted; w may then be None) and
    dw[e] = dout^T xs [experts, out, in] over the expert's rows (None: not wanted; xs may then be None)."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.expert_linear_bwd(dout, xs, w, dxs, dw, offsets, counts, stream), "ar_expert_linear_bwd"):
        return
    wide, dt, dev = _matrix(dout, "dout")
    rows, out = wide
    if dxs is not None and w is None:
        raise ValueError("dxs needs w")
    if dw is not None and xs is None:
        raise ValueError("dw needs xs")
    known = dxs if dxs is not None else xs
    if known is None or known.dim() != 2:
        raise ValueError("dxs or dw must be wanted, and xs and dxs must be matrices [rows, in]")
    narrow = (rows, known.shape[1])
    off, cnt, experts = _segments(offsets, counts, dev)
    at = (_addr(dout, "dout", (dt,), wide, dev), _opt(xs, "xs", (dt,), narrow, dev))
    weight = _weights(w if dxs is not None else None, "w", dt, experts, out, narrow[1], dev)
    to = (_opt(dxs, "dxs", (dt,), narrow, dev), *_weights(dw, "dw", dt, experts, out, narrow[1], dev))
    numbers = _ints(experts=1 if experts is None else experts)
    device = dout.device
    with _on(device):
        _check(lib().ar_expert_linear_bwd(*at, *weight, off, cnt, *numbers, rows, narrow[1], out, dtype_code(dt), *to,
                                          _stream(stream, device)), "ar_expert_linear_bwd")


# ------------------------------------------------------------------------------------------ gradients' norm
_PIECE = np.dtype([("in", np.uint64), ("out", np.uint64), ("numel", np.int64), ("dtype", np.int32), ("reserved", np.int32)])


def ar_grad_plan(tensors, outs=None):
    """The table that ar_grad_norm and ar_grad_clip work through, for the gradients `tensors` (contiguous GPU tensors of
    float32, bfloat16 and float16, any shapes), int64 [pieces, 4] on their device. outs: where clipping writes, one tensor
    of the same type and size each (None: in place). The table holds addresses: it is built once, and the tensors are to
    stay as long as it is used."""
    import torch
    tensors = list(tensors)
    outs = tensors if outs is None else list(outs)
    if not tensors or len(outs) != len(tensors):
        raise ValueError("tensors must hold at least one tensor, and outs one for each")
    device, kinds = tensors[0].device, _kinds()[0]
    table = np.zeros(len(tensors), _PIECE)
    for i, (t, o) in enumerate(zip(tensors, outs)):
        if t.dtype not in kinds:
            raise ValueError(f"tensors must be float32, bfloat16 or float16, not {t.dtype}")
        _gpu_tensor(t, "a gradient", device=device)
        _gpu_tensor(o, "an output", dtype=t.dtype, device=device)
        if o.numel() != t.numel():
            raise ValueError("an output must have its gradient's size")
        table[i] = (t.data_ptr(), 0 if o is t else o.data_ptr(), t.numel(), dtype_code(t.dtype), 0)
    n = ctypes.c_size_t(0)
    _check(lib().ar_grad_plan(table.ctypes.data, *_ints(ntensors=len(table)), None, ctypes.byref(n)), "ar_grad_plan")
    pieces = np.zeros(n.value, _PIECE)
    if n.value:
        _check(lib().ar_grad_plan(table.ctypes.data, len(table), pieces.ctypes.data, ctypes.byref(n)), "ar_grad_plan")
    return torch.from_numpy(pieces.view(np.int64).reshape(-1, 4)).to(device)


def ar_grad_norm_workspace_size(npieces) -> int:
    out = ctypes.c_size_t(0)
    _check(lib().ar_grad_norm_workspace_size(*_sizes(npieces=npieces), ctypes.byref(out)), "ar_grad_norm_workspace_size")
    return out.value


def _plan_args(plan, norm, workspace):
    import torch
    if plan.dim() != 2 or plan.shape[1] != 4:
        raise ValueError("plan must be a table of ar_grad_plan")
    dev = plan.get_device()
    at = _addr(plan, "plan", (torch.int64,), plan.shape, dev)
    if norm.numel() != 1:
        raise ValueError("norm must hold one element")
    return at, plan.shape[0], _addr(norm, "norm", _kinds()[2], norm.shape, dev), _workspace_arg(workspace, dev)


def ar_grad_norm(plan, norm, kind=AR_NORM_L2, workspace=None, stream=None):
    """norm (float32, one element) = the norm over all gradients of a plan: the square root of the sum of squares
    (AR_NORM_L2) or the largest magnitude (AR_NORM_MAX). workspace: a GPU tensor of
    ar_grad_norm_workspace_size(plan.shape[0]) bytes."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.grad_norm(plan, norm, kind, workspace, stream), "ar_grad_norm"):
        return
    at, n, to, ws = _plan_args(plan, norm, workspace)
    with _on(plan.device):
        _check(lib().ar_grad_norm(at, n, *_ints(kind=kind), to, *ws, _stream(stream, plan.device)), "ar_grad_norm")


def ar_grad_clip(plan, max_norm, norm, kind=AR_NORM_L2, eps=1e-6, workspace=None, stream=None):
    """ar_grad_norm, and all gradients times min(1, max_norm / (norm + eps)) into the plan's outputs. max_norm and eps are
    numbers on the host: a GPU tensor is refused, not waited for."""
    native = _native if _native is not None else _load_native()
    if native and _done(native.grad_clip(plan, max_norm, norm, kind, eps, workspace, stream), "ar_grad_clip"):
        return
    at, n, to, ws = _plan_args(plan, norm, workspace)
    with _on(plan.device):
        _check(lib().ar_grad_clip(at, n, *_ints(kind=kind), *_reals(max_norm=max_norm, eps=eps), to, *ws,
                                  _stream(stream, plan.device)), "ar_grad_clip")


# ------------------------------------------------------------------------------------------ bucketing
class BucketedAllReduce:
    """DDP-style bucketed all-reduce of per-rank tensor lists: pack every rank's tensors into its bucket
    buffer (one launch), all-reduce each bucket with the ring kernel, unpack to per-tensor outputs (one
    launch). The plan and descriptor tables are built once; bucket buffers are torch allocations."""

    def __init__(self, ins, outs, op=AR_AVG, algo=AR_ALGO_RING, cap_bytes=25 << 20):
        import torch
        self.n = len(ins)
        self.nt = len(ins[0])
        if any(len(x) != self.nt for x in list(ins) + list(outs)):
            raise ValueError("every rank needs the same number of tensors")
        for t in range(self.nt):
            _rank_arrays([ins[r][t] for r in range(self.n)], [outs[r][t] for r in range(self.n)])
        t00 = ins[0][0]
        self.dtype = dtype_code(t00.dtype)
        self.op, self.algo = op, algo
        numels = [ins[0][t].numel() for t in range(self.nt)]
        self.bucket_of, self.offset_of, self.bucket_count = ar_bucket_plan(numels, self.dtype, self.n, cap_bytes)
        self.bucket_start = np.concatenate([[0], np.cumsum(self.bucket_count)]).astype(np.int64)
        total = int(self.bucket_start[-1])
        self.buffers = [torch.empty(total, dtype=t00.dtype, device=t00.device) for _ in range(self.n)]
        es = t00.element_size()
        g = 16 // es
        pack, unpack = [], []
        for r in range(self.n):
            base = self.buffers[r].data_ptr()
            for t in range(self.nt):
                b = int(self.bucket_of[t])
                off = int(self.bucket_start[b] + self.offset_of[t])
                numel = numels[t]
                # zero pad up to the next tensor's start (or the bucket's end)
                nxt = t + 1
                end = (int(self.bucket_start[b] + self.offset_of[nxt])
                       if nxt < self.nt and int(self.bucket_of[nxt]) == b else int(self.bucket_start[b + 1]))
                pad = end - off - numel
                assert pad >= 0 and pad < max(g * self.n, g) + g * self.n
                pack.append((ins[r][t].data_ptr(), base + off * es, numel, pad))
                unpack.append((base + off * es, outs[r][t].data_ptr(), numel, 0))
        self.pack_descs = make_copy_descs(pack, t00.device)
        self.unpack_descs = make_copy_descs(unpack, t00.device)
        # the fused path: one descriptor per tensor (numel, offset in its bucket, bucket count / N) and the
        # [tensor, rank] pointer tables
        import torch as _t
        tdesc = np.zeros((self.nt, 4), np.int64)
        for t in range(self.nt):
            b = int(self.bucket_of[t])
            tdesc[t] = (numels[t], int(self.offset_of[t]), int(self.bucket_count[b]) // self.n, 0)
        self.tensor_descs = _t.from_numpy(tdesc).to(t00.device)
        iptr = np.array([[ins[r][t].data_ptr() for r in range(self.n)] for t in range(self.nt)], np.uint64)
        optr = np.array([[outs[r][t].data_ptr() for r in range(self.n)] for t in range(self.nt)], np.uint64)
        self.in_ptrs = _t.from_numpy(iptr.reshape(-1).view(np.int64)).to(t00.device)
        self.out_ptrs = _t.from_numpy(optr.reshape(-1).view(np.int64)).to(t00.device)
        self.views = [[self.buffers[r][int(self.bucket_start[b]):int(self.bucket_start[b + 1])]
                       for r in range(self.n)] for b in range(len(self.bucket_count))]

    @property
    def nbuckets(self):
        return len(self.bucket_count)

    def pack(self, stream=None):
        ar_bucket_pack(self.pack_descs, self.dtype, stream)

    def reduce(self, stream=None):
        """Every bucket in one launch (per-bucket rings, bit-identical to one ar_allreduce per bucket)."""
        ar_allreduce_buckets(self.buffers, self.buffers, self.bucket_count, self.op, self.algo, stream)

    def reduce_per_bucket(self, stream=None):
        """One ar_allreduce launch per bucket."""
        for v in self.views:
            ar_allreduce(v, v, self.op, self.algo, stream)

    def unpack(self, stream=None):
        ar_bucket_unpack(self.unpack_descs, self.dtype, stream)

    def fused(self, stream=None):
        """The whole bucketed all-reduce in one launch, reading and writing the tensors in place of the buckets
        (same bits as pack + reduce + unpack)."""
        ar_allreduce_tensors(self.tensor_descs, self.in_ptrs, self.out_ptrs, self.nt, self.n, self.dtype, self.op,
                             self.algo, stream)

    def __call__(self, stream=None):
        self.pack(stream)
        self.reduce(stream)
        self.unpack(stream)
