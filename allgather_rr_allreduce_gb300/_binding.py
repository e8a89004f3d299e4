"""ctypes binding of librr.so (include/rr.h).  Argument marshalling only.

Every function has the C name and the C argument order.  Device buffers may
be given as integers (device addresses) or as CUDA tensors (their data
pointer is used); dtypes as rr_dtype codes, "bf16"/"fp16"/"fp32"/"int32" or
torch dtypes; streams as integers, torch.cuda.Stream objects, or None for
torch's current stream.  A non-zero rr_status raises RRError.  Nothing here
computes: if librr.so is missing, every call raises.
"""
import array
import ctypes
import os
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "librr.so")

RR_BF16, RR_FP16, RR_FP32, RR_INT32 = 0, 1, 2, 3
RR_OK = 0
STATUS_NAMES = {
    0: "RR_OK", 1: "RR_ERR_INVALID_ARG", 2: "RR_ERR_UNSUPPORTED_DTYPE", 3: "RR_ERR_ALIGNMENT",
    4: "RR_ERR_ALIAS", 5: "RR_ERR_TOO_MANY_BLOCKS", 6: "RR_ERR_CUDA", 7: "RR_ERR_TIMEOUT",
    8: "RR_ERR_WRONG_DEVICE",
}
RR_ERR_INVALID_ARG, RR_ERR_UNSUPPORTED_DTYPE, RR_ERR_ALIGNMENT, RR_ERR_ALIAS = 1, 2, 3, 4
RR_ERR_TOO_MANY_BLOCKS, RR_ERR_CUDA, RR_ERR_TIMEOUT, RR_ERR_WRONG_DEVICE = 5, 6, 7, 8
RR_BARRIER_ARRIVE, RR_BARRIER_STAGE, RR_BARRIER_MID, RR_BARRIER_END = 0, 1, 2, 3
RR_MAX_WORLD, RR_MAX_SPLITS = 16, 256

OPTIONS = {
    "timeout_ns": 0, "blocks_per_rank": 1, "gather_engine": 2, "inject_skip": 3, "round_bytes": 4,
    "reduce_engine": 5, "twoshot_mode": 6, "device_generation": 7, "debug_iterations": 8,
    "debug_skew_ns": 9,
    "generation": 16, "last_grid": 17, "last_blocks_per_rank": 18, "last_engine": 19,
    "world_size": 20, "max_blocks_per_rank": 21,
}
_DTYPE_NAMES = {"bf16": RR_BF16, "fp16": RR_FP16, "fp32": RR_FP32, "int32": RR_INT32}


RR_ADAMW8_BLOCK = 256


class rr_adamw_hyper(ctypes.Structure):
    """rr_adamw_hyper(lr, beta1, beta2, eps, weight_decay, step)."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("step", ctypes.c_int64)]


class RRError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {message}")


_lib = None
_tensor_class = None  # torch.Tensor, once torch has been imported by the caller
_device = None                # torch's current device, from then on
_raw_stream = None            # torch's current stream, once CUDA has been started
_vp = ctypes.c_void_p
_PP = ctypes.POINTER(ctypes.c_void_p)


def lib():
    """Load librr.so (raises if it has not been built)."""
    global _lib, _tensor_class, _device
    if _tensor_class is None and "torch" in sys.modules:
        torch = sys.modules["torch"]
        _tensor_class = getattr(torch, "Tensor", None)
        if _tensor_class is not None:
            _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with allgather_rr_allreduce_gb300.build.build()")
        l = ctypes.CDLL(LIB_PATH)
        i32, i64, u64 = ctypes.c_int, ctypes.c_int64, ctypes.c_uint64
        sig = {
            "rr_signal_pad_create": [i32, i32, u64, ctypes.POINTER(_vp)],
            "rr_signal_pad_destroy": [_vp],
            "rr_signal_pad_status": [_vp, _vp],
            "rr_signal_pad_timeout_info": [_vp, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                           ctypes.POINTER(i32), ctypes.POINTER(ctypes.c_uint32)],
            "rr_signal_pad_set_option": [_vp, i32, i64],
            "rr_signal_pad_get_option": [_vp, i32, ctypes.POINTER(i64)],
            "rr_allreduce_oneshot": [_PP, _PP, _PP, i32, i64, i32, i32, _vp, _vp],
            "rr_allreduce_twoshot": [_PP, _PP, _PP, i32, i64, i32, i32, _vp, _vp],
            "rr_allgather": [_PP, _PP, i32, i64, i32, _vp, _vp],
            "rr_allgather_param_contiguous": [_PP, _PP, i32, ctypes.POINTER(i64), i32, i32, _vp, _vp],
            "rr_allgather_list": [_PP, _PP, i32, i64, i32, _vp, _vp],
            "rr_allreduce_oneshot_noalloc": [_PP, _PP, _PP, i32, i64, i32, i32, _vp],
            "rr_allreduce_oneshot_noalloc_status": [_vp],
            "rr_layer_norm": [_vp] * 6 + [i64] * 4 + [ctypes.c_float, i32, i32, _vp],
            "rr_layer_norm_backward": [_vp] * 8 + [i64] * 5 + [i32, i32, _vp, ctypes.c_size_t, _vp],
            "rr_layer_norm_backward_workspace": [i64, i64, ctypes.POINTER(ctypes.c_size_t)],
            "rr_grad_norm": [_vp, _vp, i32, i32, ctypes.c_float, ctypes.c_float, _vp, _vp, _vp, ctypes.c_size_t, _vp],
            "rr_grad_norm_workspace": [i32, ctypes.POINTER(ctypes.c_size_t)],
            "rr_adamw": [_vp] * 6 + [i32, i32, i32, ctypes.POINTER(rr_adamw_hyper), _vp, _vp],
            "rr_adamw8": [_vp] * 8 + [i32, i32, i32, ctypes.POINTER(rr_adamw_hyper), ctypes.c_uint32, _vp, _vp],
        }
        for name, args in sig.items():
            f = getattr(l, name)
            f.argtypes = args
            f.restype = ctypes.c_int
        l.rr_status_string.argtypes = [ctypes.c_int]
        l.rr_status_string.restype = ctypes.c_char_p
        l.rr_last_error.argtypes = []
        l.rr_last_error.restype = ctypes.c_char_p
        _lib = l
    return _lib


def _check(status):
    if status != RR_OK:
        raise RRError(status, lib().rr_last_error().decode(errors="replace"))


def _addr(x):
    if x is None:
        return 0
    if x.__class__ is _tensor_class and x.is_cuda:
        return x.data_ptr()
    if isinstance(x, int):
        return x
    if hasattr(x, "data_ptr"):
        if getattr(x, "is_cuda", True) is False:
            raise ValueError("device buffers must be CUDA tensors or device addresses")
        return x.data_ptr()
    raise TypeError(f"cannot take a device address from {type(x)!r}")


def pointer_array(items):
    """Host array of device addresses (NULL for None)."""
    arr = (ctypes.c_void_p * len(items))()
    for i, x in enumerate(items):
        arr[i] = _addr(x) or None
    return arr


def dtype_code(dtype):
    if isinstance(dtype, str):
        return _DTYPE_NAMES[dtype]
    if isinstance(dtype, int):
        return dtype
    import torch
    return {torch.bfloat16: RR_BF16, torch.float16: RR_FP16, torch.float32: RR_FP32,
            torch.int32: RR_INT32}[dtype]


def stream_handle(stream, device=None):
    """A stream as the C entries take it; `device`: the current one, where the caller knows it."""
    if stream is None:
        if _raw_stream is not None:  # the current stream without a Stream object
            return _raw_stream(_device() if device is None else device)
        import torch
        current = torch.cuda.current_stream().cuda_stream  # starts CUDA
        if _device is not None:
            globals().update(_raw_stream=getattr(torch._C, "_cuda_getCurrentRawStream", None))
        return current
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


class SignalPad:
    """Owner of an rr_signal_pad*.  close() (or garbage collection) destroys it."""

    def __init__(self, handle, world_size):
        self.handle = handle
        self.world_size = world_size

    @property
    def _as_parameter_(self):
        return ctypes.c_void_p(self.handle)

    def close(self):
        if self.handle:
            h, self.handle = self.handle, None
            _check(lib().rr_signal_pad_destroy(h))

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def status(self, stream=None):
        """rr_signal_pad_status: synchronise the stream, raise RRError on a recorded timeout."""
        _check(lib().rr_signal_pad_status(self.handle, stream_handle(stream)))

    def timeout_info(self):
        b, r, k = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        g = ctypes.c_uint32()
        _check(lib().rr_signal_pad_timeout_info(self.handle, ctypes.byref(b), ctypes.byref(r),
                                                ctypes.byref(k), ctypes.byref(g)))
        return {"barrier": b.value, "rank": r.value, "block": k.value, "generation": g.value}

    def set_option(self, name, value):
        _check(lib().rr_signal_pad_set_option(self.handle, OPTIONS[name], int(value)))

    def get_option(self, name):
        v = ctypes.c_int64()
        _check(lib().rr_signal_pad_get_option(self.handle, OPTIONS[name], ctypes.byref(v)))
        return v.value


def rr_signal_pad_create(world_size, max_blocks_per_rank=0, timeout_ns=0):
    h = ctypes.c_void_p()
    _check(lib().rr_signal_pad_create(world_size, max_blocks_per_rank, timeout_ns, ctypes.byref(h)))
    return SignalPad(h.value, world_size)


def rr_signal_pad_destroy(pad):
    pad.close()


def rr_signal_pad_status(pad, stream=None):
    pad.status(stream)


def _pad_handle(pad):
    return pad.handle if isinstance(pad, SignalPad) else pad


def rr_allreduce_oneshot(inputs, rank_bufs, outputs, world_size, numel, dtype, copy_mode, pad,
                         stream=None):
    ins = pointer_array(inputs) if inputs is not None else None
    _check(lib().rr_allreduce_oneshot(ins, pointer_array(rank_bufs), pointer_array(outputs),
                                      world_size, numel, dtype_code(dtype), int(bool(copy_mode)),
                                      _pad_handle(pad), stream_handle(stream)))


def rr_allreduce_twoshot(inputs, rank_bufs, outputs, world_size, numel, dtype, copy_mode, pad,
                         stream=None):
    ins = pointer_array(inputs) if inputs is not None else None
    _check(lib().rr_allreduce_twoshot(ins, pointer_array(rank_bufs), pointer_array(outputs),
                                      world_size, numel, dtype_code(dtype), int(bool(copy_mode)),
                                      _pad_handle(pad), stream_handle(stream)))


def rr_allreduce_oneshot_noalloc(inputs, rank_bufs, outputs, world_size, numel, dtype, copy_mode,
                                 stream=None):
    """The one-shot allreduce without a pad (the library's static signal array)."""
    ins = pointer_array(inputs) if inputs is not None else None
    _check(lib().rr_allreduce_oneshot_noalloc(ins, pointer_array(rank_bufs), pointer_array(outputs),
                                              world_size, numel, dtype_code(dtype),
                                              int(bool(copy_mode)), stream_handle(stream)))


def rr_allreduce_oneshot_noalloc_status(stream=None):
    """Synchronise the stream; raise RRError if the last allocation-free call timed out."""
    _check(lib().rr_allreduce_oneshot_noalloc_status(stream_handle(stream)))


def rr_allgather(rank_bufs, outputs, world_size, numel_per_rank, dtype, pad, stream=None):
    _check(lib().rr_allgather(pointer_array(rank_bufs), pointer_array(outputs), world_size,
                              numel_per_rank, dtype_code(dtype), _pad_handle(pad),
                              stream_handle(stream)))


def rr_allgather_param_contiguous(rank_bufs, outputs, world_size, split_sizes, dtype, pad,
                                  stream=None):
    n = len(split_sizes)
    sp = (ctypes.c_int64 * max(1, n))(*[int(s) for s in split_sizes])
    _check(lib().rr_allgather_param_contiguous(pointer_array(rank_bufs), pointer_array(outputs),
                                               world_size, sp, n, dtype_code(dtype),
                                               _pad_handle(pad), stream_handle(stream)))


def rr_allgather_list(rank_bufs, output_lists, world_size, numel_per_rank, dtype, pad, stream=None):
    """output_lists: W entries, each a list of W device buffers (rank q's
    all_gather tensor_list) or None (not materialised)."""
    flat = []
    for row in output_lists:
        flat.extend([None] * world_size if row is None else list(row))
    _check(lib().rr_allgather_list(pointer_array(rank_bufs), pointer_array(flat), world_size,
                                   numel_per_rank, dtype_code(dtype), _pad_handle(pad),
                                   stream_handle(stream)))


# ---------------------------------------------------------------- training step
# Kernels run on the current device, so tensors have to be there.  _here() is that
# device, None until a CUDA tensor has been seen (then CUDA has been started).
_current = None


def _here():
    return None if _current is None else _current()


def _near(x, here):
    """_addr of a buffer on the current device."""
    if x is None:
        return 0
    if x.__class__ is _tensor_class and x.get_device() == here:
        return x.data_ptr()
    return _look(x)


def _look(x):
    """_near of what is not known to be a tensor of the current device."""
    global _current
    if _device is not None and hasattr(x, "get_device"):
        device = x.get_device()
        if device < 0:
            raise ValueError("device buffers must be CUDA tensors or device addresses")
        _current, here = _device, _device()
        if device != here:
            raise RRError(RR_ERR_WRONG_DEVICE, f"a tensor is on device {device}, the current device is {here}")
    return _addr(x)


def _pointers(items, here, count, name):
    """A buffer of `count` device addresses for a list of tensors or addresses;
    None for None.  A pointer_array made before passes through, so that a loop
    over the same tensors need not marshal them again."""
    if items is None:
        return None
    if len(items) != count:
        raise ValueError(f"{name} has {len(items)} entries, sizes has {count}")
    if isinstance(items, ctypes.Array):
        return items
    try:  # tensors of the current device throughout, without a Python-level step for each
        if {here}.issuperset(map(_tensor_class.get_device, items)):
            return array.array("Q", map(_tensor_class.data_ptr, items))
    except (AttributeError, TypeError):
        pass
    return array.array("Q", map(_look, items))


def _at(buffer):
    """Where a buffer's first element lies."""
    if buffer is None:
        return 0
    return buffer.buffer_info()[0] if buffer.__class__ is array.array else ctypes.addressof(buffer)


def rr_layer_norm(x, weight, bias, y, mean, rstd, rows, cols, x_stride, y_stride, eps, dtype, weight_dtype,
                  stream=None):
    """y = layer norm of each row of x; weight, bias, mean and rstd may be None."""
    l, here = lib(), _here()
    _check(l.rr_layer_norm(_near(x, here), _near(weight, here), _near(bias, here), _near(y, here), _near(mean, here),
                           _near(rstd, here), rows, cols, x_stride, y_stride, eps, dtype_code(dtype),
                           dtype_code(weight_dtype), stream_handle(stream, here)))


def rr_layer_norm_backward(dy, x, weight, mean, rstd, dx, dweight, dbias, rows, cols, dy_stride, x_stride, dx_stride,
                           dtype, weight_dtype, workspace, workspace_bytes, stream=None):
    """Gradients of rr_layer_norm; weight and any of dx, dweight, dbias may be None."""
    l, here = lib(), _here()
    _check(l.rr_layer_norm_backward(_near(dy, here), _near(x, here), _near(weight, here), _near(mean, here),
                                    _near(rstd, here), _near(dx, here), _near(dweight, here), _near(dbias, here), rows,
                                    cols, dy_stride, x_stride, dx_stride, dtype_code(dtype), dtype_code(weight_dtype),
                                    _near(workspace, here), workspace_bytes, stream_handle(stream, here)))


def rr_layer_norm_backward_workspace(rows, cols):
    """Bytes of workspace for rr_layer_norm_backward."""
    n = ctypes.c_size_t()
    _check(lib().rr_layer_norm_backward_workspace(rows, cols, ctypes.byref(n)))
    return n.value


def rr_grad_norm(grads, sizes, dtype, inv_scale, max_norm, norm, scale, workspace, workspace_bytes, stream=None):
    """Norm over a list of gradient tensors and the factor that clips it; norm or scale may be None."""
    l, n, here = lib(), len(sizes), _here()
    s, g = array.array("q", sizes), _pointers(grads, here, n, "grads")
    _check(l.rr_grad_norm(_at(g), _at(s), n, dtype_code(dtype), inv_scale, max_norm, _near(norm, here),
                          _near(scale, here), _near(workspace, here), workspace_bytes, stream_handle(stream, here)))


def rr_grad_norm_workspace(num_tensors):
    """Bytes of workspace for rr_grad_norm."""
    n = ctypes.c_size_t()
    _check(lib().rr_grad_norm_workspace(num_tensors, ctypes.byref(n)))
    return n.value


def rr_adamw(params, grads, exp_avg, exp_avg_sq, master, sizes, param_dtype, grad_dtype, hyper, grad_scale=None,
             stream=None):
    """One AdamW step over a list of tensors, states in binary32; master may be None."""
    l, n, here = lib(), len(sizes), _here()
    s, p, g = array.array("q", sizes), _pointers(params, here, n, "params"), _pointers(grads, here, n, "grads")
    m, v = _pointers(exp_avg, here, n, "exp_avg"), _pointers(exp_avg_sq, here, n, "exp_avg_sq")
    w = _pointers(master, here, n, "master")
    _check(l.rr_adamw(_at(p), _at(g), _at(m), _at(v), _at(w), _at(s), n, dtype_code(param_dtype),
                      dtype_code(grad_dtype), hyper, _near(grad_scale, here), stream_handle(stream, here)))


def rr_adamw8(params, grads, exp_avg, exp_avg_scale, exp_avg_sq, exp_avg_sq_scale, master, sizes, param_dtype,
              grad_dtype, hyper, seed, grad_scale=None, stream=None):
    """One AdamW step over a list of tensors, states in 8 bits; master may be None."""
    l, n, here = lib(), len(sizes), _here()
    s, p, g = array.array("q", sizes), _pointers(params, here, n, "params"), _pointers(grads, here, n, "grads")
    m, ms = _pointers(exp_avg, here, n, "exp_avg"), _pointers(exp_avg_scale, here, n, "exp_avg_scale")
    v, vs = _pointers(exp_avg_sq, here, n, "exp_avg_sq"), _pointers(exp_avg_sq_scale, here, n, "exp_avg_sq_scale")
    w = _pointers(master, here, n, "master")
    _check(l.rr_adamw8(_at(p), _at(g), _at(m), _at(ms), _at(v), _at(vs), _at(w), _at(s), n, dtype_code(param_dtype),
                       dtype_code(grad_dtype), hyper, seed & 0xFFFFFFFF, _near(grad_scale, here),
                       stream_handle(stream, here)))


def bound_call(name, *args):
    """Marshal the arguments of one C entry point once and return a
    zero-argument callable that re-issues the call (for back-to-back issue
    where per-call Python marshalling would dominate).  Arguments are given
    in the C order, already in C form except for pointer lists, dtypes,
    pads and streams, which are converted here."""
    fn = getattr(lib(), name)
    conv = []
    for a in args:
        if isinstance(a, (list, tuple)):
            conv.append(pointer_array(a))
        elif isinstance(a, SignalPad):
            conv.append(a.handle)
        else:
            conv.append(a)
    l = lib()

    def call():
        st = fn(*conv)
        if st != RR_OK:
            raise RRError(st, l.rr_last_error().decode(errors="replace"))
    return call
