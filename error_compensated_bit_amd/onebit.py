"""Python binding of libonebit (include/onebit.h): same names, argument marshalling only.

Device buffers are torch CUDA tensors (PyTorch supplies device memory and the
stream); every computation runs in the library's HIP kernels.  A missing library
raises immediately: there is no fallback path.
"""
from __future__ import annotations

import atexit
import ctypes as C
import os
import re
import sys
import weakref

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libonebit.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "onebit.h")

ONEBIT_OK, ONEBIT_ERR_INVALID, ONEBIT_ERR_ALIGN, ONEBIT_ERR_HIP, ONEBIT_ERR_NOMEM, ONEBIT_ERR_UNSUPPORTED = range(6)
ONEBIT_F32, ONEBIT_BF16, ONEBIT_F16 = 0, 1, 2

_P, _I64, _I, _D, _U64, _SZ = C.c_void_p, C.c_int64, C.c_int, C.c_double, C.c_uint64, C.c_size_t

_SIGS = {
    "onebit_status_string": (C.c_char_p, [_I]),
    "onebit_set_spin_limit": (None, [C.c_uint32]),
    "onebit_set_grid_cap": (None, [C.c_int32]),
    "onebit_plan_create": (_I, [_P, _I64, _P, _P, _I64, C.POINTER(_P)]),
    "onebit_plan_destroy": (None, [_P]),
    "onebit_plan_host_tables": (_I, [_P, _I64, _P, _P, _I64, _P, _P, _P, _P, _P]),
    "onebit_plan_elements": (_I64, [_P]),
    "onebit_plan_chunks": (_I64, [_P]),
    "onebit_plan_words": (_I64, [_P]),
    "onebit_plan_workspace_bytes": (_SZ, [_P]),
    "onebit_workspace_init": (_I, [_P, _SZ, _P]),
    "onebit_workspace_status": (_I, [_P, C.POINTER(_U64), _P]),
    "onebit_device_resident_capacity": (C.c_int32, []),
    "onebit_plan_stats": (None, [_P, _P]),
    "onebit_onepass_max_elements": (_I64, []),
    "onebit_profile_begin": (None, []),
    "onebit_profile_begin_classes": (None, [C.c_uint32]),
    "onebit_profile_end": (_I, [_P, _P]),
    "onebit_adam_warmup_step": (_I, [_P, _P, _P, _P, _I, _I64, _D, _D, _D, _D, _D, _I, _I64, _P]),
    "onebit_compress_update": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _D, _D, _D, _D, _P, _P]),
    "onebit_compress_update_packed": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P, _D, _D, _D, _D, _P, _P]),
    "onebit_compress_update_static": (_I, [_P, _P, _I, _P, _P, _P, _P, _P, _P, _P, _D, _D, _D, _D, _P, _P]),
    "onebit_momentum_update_packed": (_I, [_P, _P, _P, _P, _P, _P, _P, _D, _D, _D, _P]),
    "onebit_server_reduce": (_I, [_P, _I, _P, _P, _P, _P, _P, _P, _P, _P]),
    "onebit_stream_probe": (_I, [_P, _I, _P, _I, _I64, _I, _I, _I, _P]),
    "onebit_philox_probe": (_I, [_U64, _I64, _P, _I, _I, _P]),
    "onebit_momentum_update": (_I, [_P, _P, _P, _P, _P, _I64, _D, _D, _D, _P]),
    "onebit_decompress": (_I, [_P, _P, _P, _P, _P, _P]),
    "onebit_average_rows": (_I, [_P, _I, _I, _I64, _I64, _P, _P]),
    "qsgd_quantize": (_I, [_P, _I, _I64, _I, _I, _U64, _P, _P, _P]),
    "qsgd_reduce": (_I, [_I, _P, _I64, _P, _I64, _I64, _I, _I, _P, _P, _P]),
    "loco_quantize": (_I, [_P, _I, _P, _I64, _I, _I, _D, _U64, _P, _P, _P]),
    "qsdp_quantize": (_I, [_P, _I64, _I, _I, _U64, _P, _P, _P, _P]),
    "qsdp_dequantize": (_I, [_P, _P, _P, _I64, _I, _I, _P, _P, _P]),
    "qsdp_error_stats": (_I, [_P, _P, _I64, _P, _P, _P, _P]),
    "qsdp_mean_abs_error": (_I, [_P, _P, _I64, _I, _P, _P, _P]),
    "kvq_quantize": (_I, [_P, _P, _I, _I64, _I64, _I64, _I64, _I64, _P, _P, _P]),
    "qsdp_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "qsdp_linear": (_I, [_P, _I, _I64, _I64, _P, _P, _I64, _P, _SZ, _P]),
    "qsdp_linear_grad": (_I, [_P, _I, _I64, _I64, _P, _P, _I64, _P, _SZ, _P]),
    "kvq_append": (_I, [_P, _P, _P, _I, _I64, _I, _I64, _I64, _I64, _I64, _I64, _I64, _P, _P, _I64, _I, _I, _P, _P, _P,
                        _I64, _I64, _P]),
    "kvq_dequantize": (_I, [_P, _P, _I64, _P, _P, _I, _P]),
    "kvq_attention_workspace_bytes": (_SZ, [_I64, _I64, _I, _I, _I]),
    "kvq_attention": (_I, [_P, _I, _I64, _I, _I64, _I64, _P, _P, _I64, _P, _I64, _I64, _P, _D, _D, _I, _P, _P, _P, _SZ,
                           _P]),
}

QSDP_STATS_PARTIALS = 1024
QSDP_LINEAR_EXACT_TOKENS = 32

_lib = None


class OnebitError(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__(f"{what}: {onebit_status_string(status)} (status {status})")


def load():
    """Load libonebit.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                              "(hipcc --offload-arch=gfx950); there is no fallback implementation")
        # torch ships its own HIP runtime; loading it first makes the library bind to
        # that same runtime (loaded the other way round, the process would hold two
        # runtimes and the library's first HIP call would fail)
        import torch  # noqa: F401
        lib = C.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            f = getattr(lib, name)
            f.restype = res
            f.argtypes = args
        _lib = lib
    return _lib


def header_functions():
    """Names of the functions include/onebit.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text)) - {"defined"})


def _check(status, what):
    if status != ONEBIT_OK:
        raise OnebitError(status, what)


def _ptr(t):
    """Device address of a tensor whose innermost dimension is dense.  Host tensors
    are refused here: the kernels would fault on a host address."""
    if t is None:
        return None
    if not t.is_cuda:
        raise TypeError(f"expected a device (GPU) tensor, got one on {t.device}")
    if t.numel() > 1 and t.stride(-1) != 1:
        raise ValueError("the innermost dimension of a tensor argument must be contiguous")
    if t.dim() == 1 and t.numel() > 1 and not t.is_contiguous():
        raise ValueError("one-dimensional tensor arguments must be contiguous")
    return t.data_ptr()


def _rows(t, row_len, what):
    """A [rows, row_len] tensor laid out row-major with no padding between rows."""
    if t.dim() != 2 or t.shape[1] < row_len or (t.shape[0] > 1 and t.stride(0) != row_len):
        raise ValueError(f"{what} must be a [W, {row_len}] row-major tensor with rows of exactly {row_len} entries")


def _stream(stream):
    if stream is not None:
        return stream if isinstance(stream, int) else stream.cuda_stream
    import torch
    return torch.cuda.current_stream().cuda_stream


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return ONEBIT_F32
    if t.dtype in (torch.bfloat16, torch.int16):
        return ONEBIT_BF16
    if t.dtype == torch.float16:
        return ONEBIT_F16
    raise TypeError(f"gradient dtype {t.dtype} is not float32, bfloat16 or float16")


# ---------------------------------------------------------------- API

def onebit_status_string(status: int) -> str:
    return load().onebit_status_string(int(status)).decode()


_live_plans = weakref.WeakSet()


class Plan:
    """Owning handle of an onebit_plan_t (destroyed with the object, or at interpreter
    exit while the HIP runtime is still up; never from a finalizing interpreter)."""

    def __init__(self, handle):
        self.handle = handle
        _live_plans.add(self)

    def close(self):
        if getattr(self, "handle", None) and _lib is not None:
            _lib.onebit_plan_destroy(self.handle)
        self.handle = None

    def __del__(self):
        if not sys.is_finalizing():
            self.close()


@atexit.register
def _release_plans():
    for p in list(_live_plans):
        p.close()

    @property
    def _as_parameter_(self):
        return self.handle


def onebit_plan_create(chunk_offsets, tensor_offsets=None, tensor_keep=None) -> Plan:
    lib = load()
    co = np.ascontiguousarray(chunk_offsets, dtype=np.int64)
    to = None if tensor_offsets is None else np.ascontiguousarray(tensor_offsets, dtype=np.int64)
    tk = None if tensor_keep is None else np.ascontiguousarray(tensor_keep, dtype=np.uint8)
    out = _P()
    n_tensors = 0 if to is None else to.size - 1
    _check(lib.onebit_plan_create(co.ctypes.data, co.size - 1, None if to is None else to.ctypes.data,
                                  None if tk is None else tk.ctypes.data, n_tensors, C.byref(out)),
           "onebit_plan_create")
    return Plan(out.value)


def onebit_plan_host_tables(chunk_offsets, tensor_offsets=None, tensor_keep=None):
    """Host-only plan tables: (tiles int64[n_tiles, 6], words, masked intervals int64[k, 2])."""
    lib = load()
    co = np.ascontiguousarray(chunk_offsets, dtype=np.int64)
    to = None if tensor_offsets is None else np.ascontiguousarray(tensor_offsets, dtype=np.int64)
    tk = None if tensor_keep is None else np.ascontiguousarray(tensor_keep, dtype=np.uint8)
    n_t = 0 if to is None else to.size - 1
    nt, nw, ni = C.c_int64(), C.c_int64(), C.c_int64()
    args = (co.ctypes.data, co.size - 1, None if to is None else to.ctypes.data,
            None if tk is None else tk.ctypes.data, n_t)
    _check(lib.onebit_plan_host_tables(*args, C.byref(nt), C.byref(nw), None, C.byref(ni), None),
           "onebit_plan_host_tables")
    tiles = np.zeros((nt.value, 6), dtype=np.int64)
    iv = np.zeros((ni.value, 2), dtype=np.int64)
    _check(lib.onebit_plan_host_tables(*args, None, None, tiles.ctypes.data, None, iv.ctypes.data),
           "onebit_plan_host_tables")
    return tiles, int(nw.value), iv


def onebit_plan_destroy(plan: Plan):
    load()
    plan.close()


def onebit_plan_elements(plan) -> int:
    return int(load().onebit_plan_elements(plan.handle))


def onebit_plan_chunks(plan) -> int:
    return int(load().onebit_plan_chunks(plan.handle))


def onebit_plan_words(plan) -> int:
    return int(load().onebit_plan_words(plan.handle))


def onebit_plan_workspace_bytes(plan) -> int:
    return int(load().onebit_plan_workspace_bytes(plan.handle))


def onebit_plan_stats(plan) -> dict:
    out = np.zeros(6, dtype=np.int64)
    load().onebit_plan_stats(plan.handle, out.ctypes.data)
    return dict(zip(("tiles", "onepass_tiles", "twopass_tiles", "resident_capacity", "max_chunk_tiles", "aligned"),
                    out.tolist()))


def onebit_device_resident_capacity() -> int:
    return int(load().onebit_device_resident_capacity())


def onebit_onepass_max_elements() -> int:
    return int(load().onebit_onepass_max_elements())


PROFILE_CLASSES = ("warmup", "compress_pass1", "compress_onepass", "compress_pass2", "qsdp_quantize",
                   "qsdp_dequantize", "server_pass1", "server_onepass", "server_pass2", "finalize",
                   "momentum_update", "qsgd_quantize", "qsgd_reduce", "loco_quantize")


def onebit_profile_begin(classes=None):
    """classes: names from PROFILE_CLASSES to bracket with events (None: all; an
    empty list: none)."""
    if classes is None:
        load().onebit_profile_begin()
        return
    mask = 0
    for name in classes:
        mask |= 1 << PROFILE_CLASSES.index(name)
    load().onebit_profile_begin_classes(mask)


def onebit_profile_end() -> dict:
    """{class: (total_ms, launches)} for the launches since onebit_profile_begin."""
    ms = np.zeros(len(PROFILE_CLASSES), dtype=np.float64)
    cnt = np.zeros(len(PROFILE_CLASSES), dtype=np.int64)
    _check(load().onebit_profile_end(ms.ctypes.data, cnt.ctypes.data), "onebit_profile_end")
    return {k: (float(ms[i]), int(cnt[i])) for i, k in enumerate(PROFILE_CLASSES)}


def onebit_workspace_init(workspace, stream=None):
    _check(load().onebit_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream(stream)), "onebit_workspace_init")


def onebit_workspace_status(workspace, stream=None) -> int:
    out = _U64()
    _check(load().onebit_workspace_status(_ptr(workspace), C.byref(out), _stream(stream)), "onebit_workspace_status")
    return int(out.value)


def onebit_adam_warmup_step(x, m, v, g, *, lr, beta1, beta2, eps, weight_decay, bias_correction, step,
                            stream=None):
    _check(load().onebit_adam_warmup_step(_ptr(x), _ptr(m), _ptr(v), _ptr(g), _dtype_code(g), x.numel(), lr, beta1,
                                          beta2, eps, weight_decay, int(bias_correction), int(step),
                                          _stream(stream)), "onebit_adam_warmup_step")


def onebit_compress_update(plan, g, m, e, v, x, x_bf16, bits, scales, *, lr, beta1, eps, weight_decay,
                           workspace, stream=None):
    _check(load().onebit_compress_update(plan.handle, _ptr(g), _dtype_code(g), _ptr(m), _ptr(e), _ptr(v), _ptr(x),
                                         _ptr(x_bf16), _ptr(bits), _ptr(scales), lr, beta1, eps, weight_decay,
                                         _ptr(workspace), _stream(stream)), "onebit_compress_update")


def onebit_compress_update_static(plan, g, m, e, v, x, x_bf16, bits, scales, *, lr, beta1, eps, weight_decay,
                                  wait_status=None, stream=None):
    """onebit_compress_update without a workspace (the library's scratch instead);
    wait_status: optional int64 device tensor of one element."""
    _check(load().onebit_compress_update_static(plan.handle, _ptr(g), _dtype_code(g), _ptr(m), _ptr(e), _ptr(v),
                                                _ptr(x), _ptr(x_bf16), _ptr(bits), _ptr(scales), lr, beta1, eps,
                                                weight_decay, _ptr(wait_status), _stream(stream)),
           "onebit_compress_update_static")


def onebit_compress_update_packed(plan, g, m_bits, m_scales, e, v, x, x_bf16, bits, scales, *, lr, beta1, eps,
                                  weight_decay, workspace, m_mask=None, stream=None):
    _check(load().onebit_compress_update_packed(plan.handle, _ptr(g), _dtype_code(g), _ptr(m_bits), _ptr(m_scales),
                                                _ptr(m_mask), _ptr(e), _ptr(v), _ptr(x), _ptr(x_bf16), _ptr(bits),
                                                _ptr(scales), lr, beta1, eps, weight_decay, _ptr(workspace),
                                                _stream(stream)),
           "onebit_compress_update_packed")


def onebit_momentum_update_packed(plan, m_bits, m_scales, mask, v, x, x_bf16, *, lr, eps, weight_decay, stream=None):
    _check(load().onebit_momentum_update_packed(plan.handle, _ptr(m_bits), _ptr(m_scales), _ptr(mask), _ptr(v), _ptr(x),
                                                _ptr(x_bf16), lr, eps, weight_decay, _stream(stream)),
           "onebit_momentum_update_packed")


def onebit_server_reduce(plan, worker_bits, worker_scales, server_error, server_bits, server_scales, m_out,
                         workspace, stream=None):
    W = int(worker_scales.shape[0])
    _rows(worker_bits, onebit_plan_words(plan), "worker_bits")
    _rows(worker_scales, onebit_plan_chunks(plan), "worker_scales")
    _check(load().onebit_server_reduce(plan.handle, W, _ptr(worker_bits), _ptr(worker_scales), _ptr(server_error),
                                       _ptr(server_bits), _ptr(server_scales), _ptr(m_out), _ptr(workspace),
                                       _stream(stream)), "onebit_server_reduce")


def onebit_stream_probe(inputs, outputs, grid, block=256, policy=1, stream=None):
    """inputs / outputs: lists of equally long fp32 device tensors (one of the mixes
    the library supports); block: threads per workgroup (256, 512 or 1024); policy:
    0 default cache policy, 1 (or True) nontemporal, 2 nontemporal loads staged in
    LDS by the load unit (256-thread workgroups, at least one input)."""
    import torch
    dev = (inputs or outputs)[0].device
    n = (inputs or outputs)[0].numel()
    pin = torch.tensor([t.data_ptr() for t in inputs] or [0], dtype=torch.int64, device=dev)
    pout = torch.tensor([t.data_ptr() for t in outputs] or [0], dtype=torch.int64, device=dev)
    _check(load().onebit_stream_probe(_ptr(pin), len(inputs), _ptr(pout), len(outputs), n, int(grid),
                                      int(block), int(policy), _stream(stream)), "onebit_stream_probe")
    return pin, pout           # keep the pointer arrays alive until the launch has run


def onebit_philox_probe(seed, n_blocks, out, grid, block=256, stream=None):
    """out: int32/uint32 device tensor of grid * block words (one XOR-folded word per thread)."""
    if out.numel() != grid * block:
        raise ValueError("out must hold grid * block words")
    _check(load().onebit_philox_probe(int(seed), int(n_blocks), _ptr(out), int(grid), int(block), _stream(stream)),
           "onebit_philox_probe")


def onebit_set_spin_limit(limit: int) -> None:
    load().onebit_set_spin_limit(int(limit))


def onebit_set_grid_cap(cap: int) -> None:
    load().onebit_set_grid_cap(int(cap))


def onebit_momentum_update(m, mask, v, x, x_bf16, *, lr, eps, weight_decay, stream=None):
    """mask: uint8 (or bool) tensor of n elements, or None."""
    _check(load().onebit_momentum_update(_ptr(m), _ptr(mask), _ptr(v), _ptr(x), _ptr(x_bf16), x.numel(), lr, eps,
                                         weight_decay, _stream(stream)), "onebit_momentum_update")


def onebit_decompress(plan, bits, scales, mask, out, stream=None):
    _check(load().onebit_decompress(plan.handle, _ptr(bits), _ptr(scales), _ptr(mask), _ptr(out), _stream(stream)),
           "onebit_decompress")


def onebit_average_rows(g, out, stream=None):
    """g: [W, n] (or 1-D for one row) fp32, bf16 or fp16 tensor with contiguous rows; out: fp32 [n]."""
    W = g.shape[0] if g.dim() == 2 else 1
    n = g.shape[-1]
    stride = g.stride(0) if g.dim() == 2 else n
    _check(load().onebit_average_rows(_ptr(g), _dtype_code(g), W, stride, n, _ptr(out), _stream(stream)),
           "onebit_average_rows")


def qsgd_quantize(g, bucket, bits, seed, codes, norms, stream=None):
    _check(load().qsgd_quantize(_ptr(g), _dtype_code(g), g.numel(), int(bucket), int(bits), int(seed) & (2 ** 64 - 1),
                                _ptr(codes), _ptr(norms), _stream(stream)), "qsgd_quantize")


def loco_quantize(g, err_avg, bucket, bits, beta, seed, codes, norms, stream=None):
    _check(load().loco_quantize(_ptr(g), _dtype_code(g), _ptr(err_avg), g.numel(), int(bucket), int(bits), float(beta),
                                int(seed) & (2 ** 64 - 1), _ptr(codes), _ptr(norms), _stream(stream)), "loco_quantize")


def qsgd_reduce(codes, norms, n, bucket, bits, out_f32=None, out_bf16=None, stream=None):
    """codes: uint8 [W, stride] (or 1-D for one worker); norms: float32 [W, stride] (or 1-D)."""
    W = codes.shape[0] if codes.dim() == 2 else 1
    cs = codes.stride(0) if codes.dim() == 2 else 0
    ns = norms.stride(0) if norms.dim() == 2 else 0
    _check(load().qsgd_reduce(W, _ptr(codes), cs, _ptr(norms), ns, int(n), int(bucket), int(bits), _ptr(out_f32),
                              _ptr(out_bf16), _stream(stream)), "qsgd_reduce")


def qsdp_quantize(x_bf16, bucket, bits, seed, codes, bucket_min, bucket_max, stream=None):
    _check(load().qsdp_quantize(_ptr(x_bf16), x_bf16.numel(), int(bucket), int(bits), int(seed) & (2 ** 64 - 1),
                                _ptr(codes), _ptr(bucket_min), _ptr(bucket_max), _stream(stream)), "qsdp_quantize")


def qsdp_dequantize(codes, bucket_min, bucket_max, n, bucket, bits, out_bf16=None, out_f32=None, stream=None):
    _check(load().qsdp_dequantize(_ptr(codes), _ptr(bucket_min), _ptr(bucket_max), int(n), int(bucket), int(bits),
                                  _ptr(out_bf16), _ptr(out_f32), _stream(stream)), "qsdp_dequantize")


def qsdp_error_stats(x_bf16, y, ysum, sums, partials, stream=None):
    _check(load().qsdp_error_stats(_ptr(x_bf16), _ptr(y), y.numel(), _ptr(ysum), _ptr(sums), _ptr(partials),
                                   _stream(stream)), "qsdp_error_stats")


def qsdp_mean_abs_error(x_bf16, ysum, seeds, out, partials, stream=None):
    _check(load().qsdp_mean_abs_error(_ptr(x_bf16), _ptr(ysum), ysum.numel(), int(seeds), _ptr(out), _ptr(partials),
                                      _stream(stream)), "qsdp_mean_abs_error")


# ------------------------------------------------ products with coded weights

class QsdpMatrix(C.Structure):
    """qsdp_matrix_t."""
    _fields_ = [("codes", _P), ("bucket_min", _P), ("bucket_max", _P), ("rows", _I64), ("cols", _I64), ("bucket", _I),
                ("bits", _I)]


def _same_device(first, *tensors) -> int:
    """Index of the one device all the given tensors (None skipped) are on."""
    index = first.get_device()                 # -1 for a host tensor
    for t in (first, *tensors):
        if t is not None and (t.get_device() != index or index < 0):
            if not t.is_cuda:
                raise TypeError(f"expected a device (GPU) tensor, got one on {t.device}")
            raise ValueError(f"all tensors of a call must be on one device, got {first.device} and {t.device}")
    return index


def _dense(t, dtype, what):
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _call(name, index, stream, *args):
    """Run the call with the tensors' device as the current one, on `stream` (default: that
    device's current stream)."""
    import torch
    if stream is None:
        # the stream's number itself: building a Stream object takes longer than a small call's kernel
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        if stream.device.index != index:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on cuda:{index}")
        stream = stream.cuda_stream
    call = getattr(_lib or load(), name)
    if torch.cuda.current_device() == index:
        status = call(*args, stream)
    else:
        with torch.cuda.device(index):
            status = call(*args, stream)
    _check(status, name)


def _matrix_rows(t, what):
    """Stride of a [tokens, length] tensor whose rows are dense."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 2:
        raise ValueError(f"{what} must have two dimensions, got {list(shape)}")
    if strides[1] != 1 and shape[1] > 1:
        raise ValueError(f"the rows of {what} must be contiguous")
    # (the stride of a dimension of one entry is never used and may be anything)
    return strides[0] if shape[0] > 1 else shape[1] + -shape[1] % 8


def _linear(name, x, y, rows, cols, codes, bucket_min, bucket_max, bucket, bits, workspace, stream):
    import torch
    device = _same_device(x, y, codes, bucket_min, bucket_max, workspace)
    if x.dtype != y.dtype or x.shape[0] != y.shape[0]:
        raise ValueError("input and output must have one type and as many rows")
    if bits not in (4, 8):
        raise ValueError(f"bits must be 4 or 8, got {bits}")
    if not 1 <= bucket <= 65536:
        raise ValueError(f"bucket must be from 1 to 65536, got {bucket}")
    n = rows * cols
    buckets = -(-n // bucket)
    if codes.numel() != (n * bits + 7) // 8 or bucket_min.numel() != buckets or bucket_max.numel() != buckets:
        raise ValueError(f"{rows} x {cols} weights in buckets of {bucket} need {(n * bits + 7) // 8} bytes of codes and "
                         f"{buckets} minima and maxima, got {codes.numel()}, {bucket_min.numel()} and {bucket_max.numel()}")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    w = QsdpMatrix(_dense(codes, torch.uint8, "codes"), _dense(bucket_min, torch.float32, "bucket_min"),
                   _dense(bucket_max, torch.float32, "bucket_max"), rows, cols, bucket, bits)
    _call(name, device, stream, x.data_ptr(), _dtype_code(x), x.shape[0], _matrix_rows(x, "the input"), C.byref(w),
          y.data_ptr(), _matrix_rows(y, "the output"), workspace.data_ptr(),
          workspace.numel() * workspace.element_size())


def qsdp_linear_workspace_bytes(tokens, rows, cols) -> int:
    """Bytes for qsdp_linear or qsdp_linear_grad, also with fewer tokens; 0 for sizes that they refuse.  The
    first alone takes 16 bytes with up to QSDP_LINEAR_EXACT_TOKENS tokens and those of cols = 32 with
    more, the second alone those of rows = 1."""
    return int(load().qsdp_linear_workspace_bytes(int(tokens), int(rows), int(cols)))


def qsdp_linear(x, codes, bucket_min, bucket_max, out, *, bucket, bits, workspace, stream=None):
    """out = x w^T.  x: [tokens, cols], out: [tokens, rows], bf16 or fp16 (any row stride); codes, bucket_min,
    bucket_max: a [rows, cols] matrix as qsdp_quantize codes it."""
    _linear("qsdp_linear", x, out, out.shape[-1], x.shape[-1], codes, bucket_min, bucket_max, bucket, bits, workspace, stream)


def qsdp_linear_grad(dy, codes, bucket_min, bucket_max, dx, *, bucket, bits, workspace, stream=None):
    """dx = dy w.  dy: [tokens, rows], dx: [tokens, cols]; the rest as in qsdp_linear."""
    _linear("qsdp_linear_grad", dy, dx, dy.shape[-1], dx.shape[-1], codes, bucket_min, bucket_max, bucket, bits, workspace,
            stream)


# ------------------------------------------------ coded key/value cache

class KvqCache(C.Structure):
    """kvq_cache_t."""
    _fields_ = [("k_codes", _P), ("k_scales", _P), ("v_codes", _P), ("v_scales", _P), ("n_pages", _I64),
                ("page", _I), ("kv_heads", _I), ("head_dim", _I), ("bits", _I)]


def _kvq_cache(k_codes, k_scales, v_codes, v_scales, bits):
    """kvq_cache_t of codes [n_pages, kv_heads, page, head_dim * bits / 8] and scales
    [n_pages, kv_heads, page]."""
    import torch
    if bits not in (4, 8):
        raise ValueError(f"bits must be 4 or 8, got {bits}")
    shape = k_codes.shape
    if len(shape) != 4 or shape != v_codes.shape:
        raise ValueError("k_codes and v_codes must both be [n_pages, kv_heads, page, head_dim * bits / 8]")
    if k_scales.shape != shape[:3] or v_scales.shape != shape[:3]:
        raise ValueError("k_scales and v_scales must both be [n_pages, kv_heads, page]")
    codes, scales = torch.uint8, torch.float32
    n_pages, heads, page, row = shape
    return KvqCache(_dense(k_codes, codes, "k_codes"), _dense(k_scales, scales, "k_scales"),
                    _dense(v_codes, codes, "v_codes"), _dense(v_scales, scales, "v_scales"),
                    n_pages, page, heads, row * 8 // bits, bits)


def _kvq_rows(t, heads, dim, what):
    """(token stride, head stride) of [tokens, heads, head_dim] rows whose innermost dimension is dense."""
    shape, strides = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{what} must be [tokens, {heads}, {dim}], got {list(shape)}")
    if strides[2] != 1:
        raise ValueError(f"the innermost dimension of {what} must be contiguous")
    # the stride of a dimension of one entry is never used and may be anything
    return (strides[0] if shape[0] > 1 else heads * dim), (strides[1] if heads > 1 else dim)


def _kvq_slots(slots, tokens):
    import torch
    if slots.dim() != 1 or slots.shape[0] != tokens:
        raise ValueError(f"slots must be [{tokens}], got {list(slots.shape)}")
    return _dense(slots, torch.int64, "slots")


def kvq_quantize(k, v, slots, k_codes, k_scales, v_codes, v_scales, *, bits, stream=None):
    """k, v: [tokens, kv_heads, head_dim] (any token and head strides); slots: int64 [tokens]."""
    device = _same_device(k, v, slots, k_codes, k_scales, v_codes, v_scales)
    cache = _kvq_cache(k_codes, k_scales, v_codes, v_scales, bits)
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have one shape and type")
    kt, kh = _kvq_rows(k, cache.kv_heads, cache.head_dim, "k")
    vt, vh = _kvq_rows(v, cache.kv_heads, cache.head_dim, "v")
    _call("kvq_quantize", device, stream, k.data_ptr(), v.data_ptr(), _dtype_code(k), k.shape[0], kt, kh, vt, vh,
          _kvq_slots(slots, k.shape[0]), C.byref(cache))


def kvq_append(q, k, v, positions, rotary, slots, k_codes, k_scales, v_codes, v_scales, q_out, *, bits, interleaved=False,
               stream=None):
    """q, q_out: [tokens, q_heads, head_dim] (q_out may be q; both None: keys and values only); k, v: [tokens,
    kv_heads, head_dim]; any token and head strides, one type; positions, slots: int64 [tokens]; rotary: float32
    [max_position, rot_dim], cosines and then sines."""
    import torch
    device = _same_device(k, v, q, q_out, positions, rotary, slots, k_codes, k_scales, v_codes, v_scales)
    cache = _kvq_cache(k_codes, k_scales, v_codes, v_scales, bits)
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must have one shape and type")
    kt, kh = _kvq_rows(k, cache.kv_heads, cache.head_dim, "k")
    vt, vh = _kvq_rows(v, cache.kv_heads, cache.head_dim, "v")
    tokens, heads = k.shape[0], 0
    qt = qh = ot = oh = 0
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out are given both or not at all")
    if q is not None:
        if q.dtype != k.dtype or q_out.dtype != k.dtype:
            raise ValueError("q, q_out and k must have one type")
        if q.dim() != 3 or q.shape[0] != tokens or q_out.shape != q.shape:
            raise ValueError(f"q and q_out must both be [{tokens}, q_heads, head_dim]")
        heads = q.shape[1]
        qt, qh = _kvq_rows(q, heads, cache.head_dim, "q")
        ot, oh = _kvq_rows(q_out, heads, cache.head_dim, "q_out")
    if positions.dim() != 1 or positions.shape[0] != tokens:
        raise ValueError(f"positions must be [{tokens}], got {list(positions.shape)}")
    if rotary.dim() != 2:
        raise ValueError(f"rotary must be [max_position, rot_dim], got {list(rotary.shape)}")
    _call("kvq_append", device, stream, None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(), _dtype_code(k),
          tokens, heads, qt, qh, kt, kh, vt, vh, _dense(positions, torch.int64, "positions"),
          _dense(rotary, torch.float32, "rotary"), rotary.shape[0], rotary.shape[1], int(interleaved),
          _kvq_slots(slots, tokens), C.byref(cache), None if q is None else q_out.data_ptr(), ot, oh)


def kvq_dequantize(k_codes, k_scales, v_codes, v_scales, slots, k_out, v_out, *, bits, stream=None):
    """slots: int64 [tokens]; k_out, v_out: contiguous [tokens, kv_heads, head_dim] of one type."""
    device = _same_device(k_out, v_out, slots, k_codes, k_scales, v_codes, v_scales)
    cache = _kvq_cache(k_codes, k_scales, v_codes, v_scales, bits)
    if k_out.dtype != v_out.dtype or k_out.shape != v_out.shape:
        raise ValueError("k_out and v_out must have one shape and type")
    _kvq_rows(k_out, cache.kv_heads, cache.head_dim, "k_out")
    _call("kvq_dequantize", device, stream, C.byref(cache), _kvq_slots(slots, k_out.shape[0]), k_out.shape[0],
          _dense(k_out, k_out.dtype, "k_out"), _dense(v_out, v_out.dtype, "v_out"), _dtype_code(k_out))


def kvq_attention_workspace_bytes(batch, total_q, q_heads, kv_heads, head_dim) -> int:
    """Bytes for the current device; 0 for sizes that kvq_attention refuses."""
    return int(load().kvq_attention_workspace_bytes(int(batch), int(total_q), int(q_heads), int(kv_heads),
                                                    int(head_dim)))


def kvq_attention(q, k_codes, k_scales, v_codes, v_scales, block_table, kv_lens, out, *, bits, workspace, scale=None,
                  q_offsets=None, softcap=0.0, window=0, lse=None, stream=None):
    """q: [total_q, q_heads, head_dim] (any token and head strides), bf16 or fp16; block_table: int32
    [batch, max_pages]; kv_lens: int32 [batch]; out: contiguous, of q's shape and type; q_offsets: int32
    [batch + 1] (None: total_q / batch rows for every sequence); lse: float32 [total_q, q_heads]; scale:
    default 1 / sqrt(head_dim)."""
    import torch
    device = _same_device(q, k_codes, k_scales, v_codes, v_scales, block_table, kv_lens, out, workspace, q_offsets, lse)
    cache = _kvq_cache(k_codes, k_scales, v_codes, v_scales, bits)
    if q.dim() != 3:
        raise ValueError(f"q must be [total_q, q_heads, head_dim], got {list(q.shape)}")
    total, q_heads = q.shape[0], q.shape[1]
    qt, qh = _kvq_rows(q, q_heads, cache.head_dim, "q")
    if out.dtype != q.dtype or out.shape != q.shape:
        raise ValueError("out must have q's shape and type")
    if kv_lens.dim() != 1 or block_table.dim() != 2 or block_table.shape[0] != kv_lens.shape[0]:
        raise ValueError("kv_lens must be [batch] and block_table [batch, max_pages]")
    batch, max_pages = block_table.shape
    if block_table.dtype != torch.int32 or (max_pages > 1 and block_table.stride(1) != 1):
        raise TypeError("block_table must be int32 with contiguous rows")
    if q_offsets is not None and list(q_offsets.shape) != [batch + 1]:
        raise ValueError(f"q_offsets must be [{batch + 1}]")
    if lse is not None and list(lse.shape) != [total, q_heads]:
        raise ValueError(f"lse must be [{total}, {q_heads}]")
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    if abs(window) >= 2 ** 31:                 # (would be cut to 32 bits on its way)
        raise ValueError(f"window must be from 0 to 2^31 - 1, got {window}")
    _call("kvq_attention", device, stream, q.data_ptr(), _dtype_code(q), total, q_heads, qt, qh,
          None if q_offsets is None else _dense(q_offsets, torch.int32, "q_offsets"),
          _dense(kv_lens, torch.int32, "kv_lens"), batch, block_table.data_ptr(), max_pages,
          block_table.stride(0) if batch > 1 else max_pages, C.byref(cache),
          cache.head_dim ** -0.5 if scale is None else float(scale), float(softcap), int(window),
          _dense(out, q.dtype, "out"), None if lse is None else _dense(lse, torch.float32, "lse"),
          _ptr(workspace), workspace.numel() * workspace.element_size())
