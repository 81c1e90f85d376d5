"""Python binding of libmpt: the loss-scaled FP32-master optimizer step on B200.

Argument marshalling only (ctypes over the C ABI in ``include/mpt.h``): every
step of the path runs in the library's CUDA kernels.  PyTorch supplies the
device workspace and the stream.  There is no CPU fallback: if ``libmpt.so``
cannot be loaded (or built with nvcc), importing the library fails loudly.

    opt = MPT(sizes, Config(growth_interval=4))
    for i, w in enumerate(initial_weights):
        opt.master(i).copy_(w)
    opt.refresh_half()
    opt.set_scaler_state(2.0 ** 16)
    res = opt.step(grads, scale=opt.scale, lr=0.01, momentum=0.9,
                   weight_decay=1e-4, clip=1.0)
"""
import collections
import contextlib
import ctypes
import os

from . import build as _build

__all__ = ["MPT", "Config", "MptError", "GradList", "xent_loss", "xent_grad", "lib", "grad_pointers", "check_flat_noalloc",
           "MPT_FLAG_CHECKED", "MPT_FLAG_COUNT_STALE", "MPT_FLAG_GRAD_STATS",
           "MPT_SCALER_DYNAMIC", "MPT_SCALER_DIRECT", "MPT_OPT_MOMENTUM", "MPT_OPT_NESTEROV",
           "MPT_OPT_ADAGRAD"]

MPT_FLAG_CHECKED = 0x1
MPT_FLAG_COUNT_STALE = 0x2
MPT_FLAG_GRAD_STATS = 0x4
MPT_SCALER_DYNAMIC = 0
MPT_SCALER_DIRECT = 1
MPT_OPT_MOMENTUM = 0
MPT_OPT_NESTEROV = 1
MPT_OPT_ADAGRAD = 2

MPT_OK = 0
MPT_ERR_INVALID_ARG = -1
MPT_ERR_WORKSPACE = -2
MPT_ERR_CUDA = -3
MPT_ERR_DEVICE_CHECK = -4
MPT_ERR_BROKEN = -5
MPT_ERR_TOO_LARGE = -6
MPT_NOALLOC_MAX_ELEMS = 1 << 30
MPT_PARTIAL_BYTES = 32
MPT_F16, MPT_BF16, MPT_F32 = 0, 1, 2
MPT_LIST_TENSOR_NORMS = 0x1
MPT_LIST_UNSCALE = 0x2
MPT_XENT_MEAN, MPT_XENT_SUM = 0, 1


class MptError(RuntimeError):
    def __init__(self, code, what):
        self.code = code
        super().__init__(f"{what}: {lib().mpt_error_string(code).decode()} ({code})")


class Config(ctypes.Structure):
    _fields_ = [("backoff", ctypes.c_float), ("growth", ctypes.c_float),
                ("growth_interval", ctypes.c_int32), ("min_scale", ctypes.c_float),
                ("max_scale", ctypes.c_float), ("flags", ctypes.c_uint32),
                ("check_chunk_elems", ctypes.c_int32), ("scaler_mode", ctypes.c_int32),
                ("direct_margin", ctypes.c_float), ("optimizer", ctypes.c_int32),
                ("eps", ctypes.c_float), ("update_chunk_elems", ctypes.c_int32)]

    def __init__(self, **kw):
        super().__init__()
        lib().mpt_config_init(ctypes.byref(self))
        for k, v in kw.items():
            if k not in dict(self._fields_):
                raise TypeError(f"unknown config field {k}")
            setattr(self, k, v)


class StepResult(ctypes.Structure):
    _fields_ = [("found_inf", ctypes.c_int32), ("clipped", ctypes.c_int32),
                ("new_scale", ctypes.c_float), ("clean_run", ctypes.c_int32),
                ("grad_norm", ctypes.c_double), ("clip_coef", ctypes.c_float),
                ("max_abs_grad", ctypes.c_float), ("n_zero", ctypes.c_uint64),
                ("n_subnormal", ctypes.c_uint64), ("n_nonfinite", ctypes.c_uint64),
                ("n_fp16_stale", ctypes.c_uint64)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_}


class CheckResult(ctypes.Structure):
    """``mpt_check_result``: what mpt_check_flat_noalloc writes to device memory."""
    _fields_ = [("found_inf", ctypes.c_int32), ("clipped", ctypes.c_int32),
                ("grad_norm", ctypes.c_double), ("clip_coef", ctypes.c_float),
                ("reserved", ctypes.c_int32), ("n_nonfinite", ctypes.c_uint64)]

    def as_dict(self):
        return {k: getattr(self, k) for k, _ in self._fields_ if k != "reserved"}


class XentArgs(ctypes.Structure):
    """``mpt_xent_args``."""
    _fields_ = [("type", ctypes.c_int32), ("target_bytes", ctypes.c_int32),
                ("n", ctypes.c_int64), ("v", ctypes.c_int64), ("d", ctypes.c_int64),
                ("hidden", ctypes.c_void_p), ("ld_hidden", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("ld_weight", ctypes.c_int64),
                ("targets", ctypes.c_void_p), ("ignore_index", ctypes.c_int64),
                ("reduction", ctypes.c_int32), ("scale", ctypes.c_float),
                ("d_scale", ctypes.c_void_p), ("loss", ctypes.c_void_p),
                ("token_loss", ctypes.c_void_p), ("lse", ctypes.c_void_p),
                ("n_valid", ctypes.c_void_p), ("grad_hidden", ctypes.c_void_p),
                ("ld_grad_hidden", ctypes.c_int64), ("grad_weight", ctypes.c_void_p),
                ("ld_grad_weight", ctypes.c_int64)]


class Stats(ctypes.Structure):
    _fields_ = [("steps", ctypes.c_uint64), ("skipped", ctypes.c_uint64),
                ("scale", ctypes.c_float), ("clean_run", ctypes.c_int32),
                ("last", StepResult), ("n_fp16_stale_total", ctypes.c_uint64),
                ("timed_steps", ctypes.c_uint64), ("check_ms_total", ctypes.c_double),
                ("update_ms_total", ctypes.c_double)]

    def as_dict(self):
        d = {k: getattr(self, k) for k, _ in self._fields_}
        d["last"] = self.last.as_dict()
        return d


_LIB = None


def lib():
    """Load (building with nvcc if needed) ``libmpt.so``; raises if impossible."""
    global _LIB
    if _LIB is None:
        path = _build.LIB
        if not os.path.exists(path) or os.environ.get("MPT_REBUILD"):
            path = _build.build()
        L = ctypes.CDLL(path)
        vp, i32, f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float
        sig = {
            "mpt_config_init": [ctypes.POINTER(Config)],
            "mpt_workspace_bytes": [vp, i32, ctypes.POINTER(Config), ctypes.POINTER(ctypes.c_size_t)],
            "mpt_create": [vp, i32, ctypes.POINTER(Config), vp, ctypes.c_size_t, ctypes.POINTER(vp)],
            "mpt_tensor_views": [vp, i32, ctypes.POINTER(vp), ctypes.POINTER(vp), ctypes.POINTER(vp)],
            "mpt_refresh_half": [vp, vp],
            "mpt_step": [vp, vp, f32, f32, f32, f32, f32, vp, ctypes.POINTER(StepResult)],
            "mpt_stats": [vp, ctypes.POINTER(Stats)],
            "mpt_get_scaler_state": [vp, ctypes.POINTER(f32), ctypes.POINTER(i32)],
            "mpt_set_scaler_state": [vp, f32, i32],
            "mpt_set_timing": [vp, i32],
            "mpt_destroy": [vp],
            "mpt_check_flat_noalloc": [vp, ctypes.c_int64, f32, f32, vp, vp],
            "mpt_step_async": [vp, vp, f32, f32, f32, f32, vp],
            "mpt_wait": [vp, vp, ctypes.POINTER(StepResult)],
            "mpt_device_scale": [vp, ctypes.POINTER(vp)],
            "mpt_grad_histogram": [vp, ctypes.POINTER(ctypes.c_uint64 * 32)],
            "mpt_shard_len": [ctypes.c_int64, i32, ctypes.POINTER(ctypes.c_int64)],
            "mpt_step_partial": [vp, vp, vp, ctypes.POINTER(vp)],
            "mpt_step_finish": [vp, vp, i32, f32, f32, f32, f32, vp],
            "mpt_debug_fail_next_step": [vp],
            "mpt_list_workspace_bytes": [vp, vp, vp, i32, ctypes.POINTER(ctypes.c_size_t)],
            "mpt_list_create": [vp, vp, vp, i32, vp, ctypes.c_size_t, ctypes.POINTER(vp)],
            "mpt_list_norm": [vp, vp, f32, vp, f32, ctypes.c_uint32, vp],
            "mpt_list_clip": [vp, vp, vp, f32, vp, f32, ctypes.c_uint32, vp],
            "mpt_list_views": [vp, ctypes.POINTER(vp), ctypes.POINTER(vp)],
            "mpt_list_wait": [vp, vp, ctypes.POINTER(CheckResult)],
            "mpt_list_destroy": [vp],
            "mpt_xent_args_init": [ctypes.POINTER(XentArgs)],
            "mpt_xent_workspace_bytes": [ctypes.POINTER(XentArgs), ctypes.POINTER(ctypes.c_size_t)],
            "mpt_xent": [ctypes.POINTER(XentArgs), vp, ctypes.c_size_t, vp],
            "mpt_debug_xent_give_up": [i32],
        }
        for name, args in sig.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        L.mpt_error_string.argtypes = [ctypes.c_int]
        L.mpt_error_string.restype = ctypes.c_char_p
        _LIB = L
    return _LIB


def _check(code, what):
    if code != MPT_OK:
        raise MptError(code, what)


def grad_pointers(tensors):
    """Host array of device pointers (build once, reuse across steps)."""
    return (ctypes.c_void_p * len(tensors))(*[t.data_ptr() for t in tensors])


def check_flat_noalloc(grads, scale, clip, out, stream=None):
    """Queue ``mpt_check_flat_noalloc`` on one contiguous FP16 CUDA tensor;
    ``out`` is a CUDA tensor of at least ``ctypes.sizeof(CheckResult)`` bytes
    that receives the result.  Returns without waiting."""
    if not grads.is_contiguous() or grads.element_size() != 2:
        raise ValueError("grads must be one contiguous 2-byte tensor")
    if out.numel() * out.element_size() < ctypes.sizeof(CheckResult):
        raise ValueError("out is too small for mpt_check_result")
    _check(lib().mpt_check_flat_noalloc(ctypes.c_void_p(grads.data_ptr()), grads.numel(),
                                        scale, clip, ctypes.c_void_p(out.data_ptr()),
                                        _stream_ptr(stream, grads.device)),
           "mpt_check_flat_noalloc")


def shard_len(total, world):
    """Elements per rank of the sharded step (``mpt_shard_len``)."""
    n = ctypes.c_int64()
    _check(lib().mpt_shard_len(int(total), int(world), ctypes.byref(n)), "mpt_shard_len")
    return n.value


def _stream_ptr(stream, device):
    import torch
    if stream is None:  # the raw handle: current_stream() builds a Stream object
        return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(device.index))
    return ctypes.c_void_p(stream.cuda_stream)


def _check_stream(stream, device):
    """A stream of another device would run the work there, on this one's
    addresses."""
    import torch
    if stream is not None and torch.device(stream.device) != device:
        raise ValueError(f"the stream belongs to {stream.device}, the tensors to {device}")


def _on(device, stream):
    """A context in which ``device`` (and ``stream``, if given) are current."""
    import torch
    if stream is not None:
        return torch.cuda.stream(stream)
    if torch._C._cuda_getDevice() == device.index:
        return contextlib.nullcontext()
    return torch.cuda.device(device)


class MPT:
    """One optimizer over a fixed list of tensor sizes (one CUDA device)."""

    def __init__(self, sizes, config=None, device=None):
        import torch
        self.sizes = [int(s) for s in sizes]
        self.n = len(self.sizes)
        self.config = config if config is not None else Config()
        self.device = torch.device(device if device is not None else "cuda", )
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._sizes_c = (ctypes.c_int64 * self.n)(*self.sizes)
        nbytes = ctypes.c_size_t()
        _check(lib().mpt_workspace_bytes(self._sizes_c, self.n, ctypes.byref(self.config),
                                         ctypes.byref(nbytes)), "mpt_workspace_bytes")
        self.workspace_bytes = nbytes.value
        self.workspace = torch.empty(self.workspace_bytes, dtype=torch.uint8, device=self.device)
        h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(lib().mpt_create(self._sizes_c, self.n, ctypes.byref(self.config),
                                    ctypes.c_void_p(self.workspace.data_ptr()),
                                    self.workspace_bytes, ctypes.byref(h)), "mpt_create")
        self._h = h
        self._views = [self._make_views(i) for i in range(self.n)]
        self._ptr_cache = None

    # -- state views ---------------------------------------------------------
    def _make_views(self, i):
        import torch
        m, v, w = ctypes.c_void_p(), ctypes.c_void_p(), ctypes.c_void_p()
        _check(lib().mpt_tensor_views(self._h, i, ctypes.byref(m), ctypes.byref(v),
                                      ctypes.byref(w)), "mpt_tensor_views")
        base = self.workspace.data_ptr()
        n = self.sizes[i]
        ws = self.workspace
        return (ws[m.value - base: m.value - base + 4 * n].view(torch.float32),
                ws[v.value - base: v.value - base + 4 * n].view(torch.float32),
                ws[w.value - base: w.value - base + 2 * n].view(torch.float16))

    def master(self, i):
        return self._views[i][0]

    def momentum(self, i):
        return self._views[i][1]

    def w16(self, i):
        return self._views[i][2]

    # -- calls ---------------------------------------------------------------
    def refresh_half(self, stream=None):
        _check(lib().mpt_refresh_half(self._h, _stream_ptr(stream, self.device)),
               "mpt_refresh_half")

    def step(self, grads, scale, lr, momentum, weight_decay, clip=0.0, stream=None):
        """``grads``: list of FP16 (or int16 bit-pattern) CUDA tensors, or an
        array from :func:`grad_pointers`.  Returns the step result as a dict."""
        ptrs = self._ptrs(grads)
        r = StepResult()
        _check(lib().mpt_step(self._h, ptrs, scale, lr, momentum, weight_decay, clip,
                              _stream_ptr(stream, self.device), ctypes.byref(r)), "mpt_step")
        return r.as_dict()

    def _ptrs(self, grads):
        if isinstance(grads, ctypes.Array):
            return grads
        if len(grads) != self.n:
            raise ValueError(f"expected {self.n} gradient tensors, got {len(grads)}")
        for g, n in zip(grads, self.sizes):
            if g.numel() != n or g.element_size() != 2 or g.device != self.device:
                raise ValueError("gradient tensor does not match its size/dtype/device")
            if not g.is_contiguous():
                raise ValueError("gradient tensors must be contiguous")
        return grad_pointers(grads)

    def step_async(self, grads, lr, momentum, weight_decay, clip=0.0, stream=None):
        """Queue one step without waiting; S is the device scale state
        (:meth:`device_scale`).  Call :meth:`wait` for the result."""
        _check(lib().mpt_step_async(self._h, self._ptrs(grads), lr, momentum, weight_decay, clip,
                                    _stream_ptr(stream, self.device)), "mpt_step_async")

    def wait(self, stream=None):
        """Wait for the queued steps; returns the last step's result."""
        r = StepResult()
        _check(lib().mpt_wait(self._h, _stream_ptr(stream, self.device), ctypes.byref(r)),
               "mpt_wait")
        return r.as_dict()

    def device_scale(self):
        """A 1-element float32 CUDA tensor aliasing the device scale state."""
        p = ctypes.c_void_p()
        _check(lib().mpt_device_scale(self._h, ctypes.byref(p)), "mpt_device_scale")
        off = p.value - self.workspace.data_ptr()
        import torch
        return self.workspace[off:off + 4].view(torch.float32)

    def head_grad(self, i, hidden, targets, grad_weight=True, ignore_index=-100, reduction="mean",
                  grad_hidden=True, stream=None):
        """Loss and gradients of a linear head whose weight is tensor ``i``
        (classes x width, row-major): :func:`xent_grad` with the FP16 working
        copy and the device loss scale, as a step's first half.

            r = opt.head_grad(0, hidden, targets, grad_weight=grads[0].view(v, d))
            ...                       # r.grad_hidden goes back through the model
            opt.step_async(grads, lr, momentum, weight_decay)
        """
        if hidden.dim() != 2 or hidden.shape[1] == 0 or self.sizes[i] % hidden.shape[1]:
            raise ValueError(f"tensor {i} has no rows of the width of hidden")
        weight = self.w16(i).view(-1, hidden.shape[1])
        return xent_grad(hidden, weight, targets, scale=self.device_scale(), ignore_index=ignore_index,
                         reduction=reduction, grad_hidden=grad_hidden, grad_weight=grad_weight, stream=stream)

    def step_partial(self, grads, stream=None):
        """Sharded step, phase 2: queue the check pass; returns a 32-byte
        uint8 CUDA tensor aliasing this rank's record."""
        import torch
        p = ctypes.c_void_p()
        _check(lib().mpt_step_partial(self._h, self._ptrs(grads), _stream_ptr(stream, self.device),
                                      ctypes.byref(p)), "mpt_step_partial")
        off = p.value - self.workspace.data_ptr()
        return self.workspace[off:off + MPT_PARTIAL_BYTES]

    def step_finish(self, partials, world, lr, momentum, weight_decay, clip=0.0, stream=None):
        """Sharded step, phase 4: ``partials`` is a CUDA tensor holding the
        ``world`` records in rank order."""
        _check(lib().mpt_step_finish(self._h, ctypes.c_void_p(partials.data_ptr()), world, lr,
                                     momentum, weight_decay, clip,
                                     _stream_ptr(stream, self.device)), "mpt_step_finish")

    def grad_histogram(self):
        """Gradients of the last step per binary16 exponent field (32 bins)."""
        h = (ctypes.c_uint64 * 32)()
        _check(lib().mpt_grad_histogram(self._h, ctypes.byref(h)), "mpt_grad_histogram")
        return list(h)

    def stats(self):
        s = Stats()
        _check(lib().mpt_stats(self._h, ctypes.byref(s)), "mpt_stats")
        return s.as_dict()

    @property
    def scale(self):
        return self.scaler_state()[0]

    def scaler_state(self):
        s, c = ctypes.c_float(), ctypes.c_int32()
        _check(lib().mpt_get_scaler_state(self._h, ctypes.byref(s), ctypes.byref(c)),
               "mpt_get_scaler_state")
        return s.value, c.value

    def set_scaler_state(self, scale, clean_run=0):
        _check(lib().mpt_set_scaler_state(self._h, scale, clean_run), "mpt_set_scaler_state")

    def set_timing(self, every=1):
        """Time the two kernels of every ``every``-th following step (0 or
        False: off; True or 1: every step)."""
        _check(lib().mpt_set_timing(self._h, int(every)), "mpt_set_timing")

    def debug_fail_next_step(self):
        """Test hook: the next step fails like a failed kernel launch and the
        handle becomes unusable (``mpt_debug_fail_next_step``)."""
        _check(lib().mpt_debug_fail_next_step(self._h), "mpt_debug_fail_next_step")

    def close(self):
        if getattr(self, "_h", None):
            lib().mpt_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _type_code(dtype):
    code = {"torch.float16": MPT_F16, "torch.bfloat16": MPT_BF16, "torch.float32": MPT_F32}.get(str(dtype))
    if code is None:
        raise ValueError(f"{dtype} is not float16, bfloat16 or float32")
    return code


def _scale_args(scale, device):
    """(host S, device pointer of S) of a number or a 1-element CUDA tensor."""
    import torch
    if isinstance(scale, torch.Tensor):
        if scale.dtype != torch.float32 or scale.numel() != 1 or scale.device != device:
            raise ValueError("a scale on the device is one float32 on the same device")
        return 1.0, ctypes.c_void_p(scale.data_ptr())
    return float(scale), None


def _used_on(stream, *tensors):
    """Tell the allocator that ``stream`` reads or writes these tensors."""
    import torch
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)


class GradList:
    """Global gradient norm over a fixed list of tensors, and clipping
    (``mpt_list_*``): FP16, BF16 or FP32 tensors, one type for all or one each.

        clipper = GradList(sizes, torch.bfloat16)
        clipper.clip(grads, 1.0)            # in place, queued
        norm = clipper.wait()["grad_norm"]

    ``scale`` is the loss scale S that the gradients carry: a number, or a
    1-element float32 CUDA tensor such as :meth:`MPT.device_scale`.  The calls
    return views of the list's own result buffers, which the next call
    overwrites: ``norm`` (float64), ``coef`` (float32), ``found_inf`` (int32),
    ``n_nonfinite`` (int64), and ``tensor_norms`` (float64) if asked.  A list may
    be dropped while its calls run, but not while a graph that captured one lives.
    """

    def __init__(self, sizes, dtypes, out_dtypes=None, device=None):
        import torch
        self.sizes = [int(s) for s in sizes]
        self.n = len(self.sizes)
        self.dtypes = self._types(dtypes)
        self.out_dtypes = self.dtypes if out_dtypes is None else self._types(out_dtypes)
        self.device = torch.device(device if device is not None else "cuda")
        if self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        i32n = ctypes.c_int32 * self.n
        args = ((ctypes.c_int64 * self.n)(*self.sizes), i32n(*map(_type_code, self.dtypes)),
                i32n(*map(_type_code, self.out_dtypes)), self.n)
        nbytes = ctypes.c_size_t()
        _check(lib().mpt_list_workspace_bytes(*args, ctypes.byref(nbytes)), "mpt_list_workspace_bytes")
        self.workspace = torch.empty(nbytes.value, dtype=torch.uint8, device=self.device)
        self._streams = {_stream_ptr(None, self.device).value}  # that the allocator knows to use it
        self._h = ctypes.c_void_p()
        with torch.cuda.device(self.device):
            _check(lib().mpt_list_create(*args, ctypes.c_void_p(self.workspace.data_ptr()), nbytes.value,
                                         ctypes.byref(self._h)), "mpt_list_create")
        rec, norms = ctypes.c_void_p(), ctypes.c_void_p()
        _check(lib().mpt_list_views(self._h, ctypes.byref(rec), ctypes.byref(norms)), "mpt_list_views")

        def view(address, nbytes, dtype):
            off = address - self.workspace.data_ptr()
            return self.workspace[off:off + nbytes].view(dtype)
        field = CheckResult
        self._result = {"norm": view(rec.value + field.grad_norm.offset, 8, torch.float64),
                        "coef": view(rec.value + field.clip_coef.offset, 4, torch.float32),
                        "found_inf": view(rec.value + field.found_inf.offset, 4, torch.int32),
                        "n_nonfinite": view(rec.value + field.n_nonfinite.offset, 8, torch.int64)}
        self._tensor_norms = view(norms.value, 8 * self.n, torch.float64)

    def _types(self, dtypes):
        import torch
        if isinstance(dtypes, torch.dtype):
            return [dtypes] * self.n
        dtypes = list(dtypes)
        if len(dtypes) != self.n:
            raise ValueError(f"expected {self.n} types, got {len(dtypes)}")
        return dtypes

    def _ptrs(self, tensors, dtypes, what):
        if isinstance(tensors, ctypes.Array):
            if len(tensors) != self.n:
                raise ValueError(f"expected {self.n} {what} pointers, got {len(tensors)}")
            return tensors
        if len(tensors) != self.n:
            raise ValueError(f"expected {self.n} {what} tensors, got {len(tensors)}")
        for t, n, dt in zip(tensors, self.sizes, dtypes):
            if t.numel() != n or t.dtype != dt or t.device != self.device or not t.is_contiguous():
                raise ValueError(f"{what} tensor does not match its size/dtype/device or is not contiguous")
        return grad_pointers(tensors)

    def _queue_on(self, stream):
        """The raw stream of a call.  The list may be dropped while the call
        runs, so the allocator hears of any stream but the one that was current
        at creation."""
        import torch
        raw = _stream_ptr(stream, self.device)
        if raw.value not in self._streams:
            _used_on(stream if stream is not None else torch.cuda.current_stream(self.device), self.workspace)
            self._streams.add(raw.value)
        return raw

    def _views(self, tensor_norms):
        return self._result | {"tensor_norms": self._tensor_norms} if tensor_norms else dict(self._result)

    def norm(self, grads, scale=1.0, clip=0.0, tensor_norms=False, stream=None):
        """Queue the norm of ``grads`` (CUDA tensors, or an array from
        :func:`grad_pointers`); ``clip`` only sets the ``coef`` reported."""
        _check_stream(stream, self.device)
        host, dev = _scale_args(scale, self.device)
        g = self._ptrs(grads, self.dtypes, "gradient")
        if stream is not None:
            _used_on(stream, scale, *(() if g is grads else grads))
        with _on(self.device, stream):
            _check(lib().mpt_list_norm(self._h, g, host, dev, clip,
                                       MPT_LIST_TENSOR_NORMS if tensor_norms else 0,
                                       self._queue_on(stream)), "mpt_list_norm")
        return self._views(tensor_norms)

    def clip(self, grads, clip, out=None, scale=1.0, unscale=False, tensor_norms=False, stream=None):
        """Queue the norm and the scaling of ``grads`` to a norm of at most
        ``clip``, into ``out`` (default: in place)."""
        _check_stream(stream, self.device)
        host, dev = _scale_args(scale, self.device)
        g = self._ptrs(grads, self.dtypes, "gradient")
        if out is None and self.out_dtypes != self.dtypes:
            raise ValueError("outputs of another type need tensors of their own")
        o = g if out is None else self._ptrs(out, self.out_dtypes, "output")
        if stream is not None:
            _used_on(stream, scale, *(() if g is grads else grads), *(() if out is None or o is out else out))
        flags = (MPT_LIST_TENSOR_NORMS if tensor_norms else 0) | (MPT_LIST_UNSCALE if unscale else 0)
        with _on(self.device, stream):
            _check(lib().mpt_list_clip(self._h, g, o, host, dev, clip, flags, self._queue_on(stream)), "mpt_list_clip")
        return self._views(tensor_norms)

    def wait(self, stream=None):
        """Wait for the queued work; the last result as a dict of numbers."""
        _check_stream(stream, self.device)
        r = CheckResult()
        with _on(self.device, stream):
            _check(lib().mpt_list_wait(self._h, _stream_ptr(stream, self.device), ctypes.byref(r)),
                   "mpt_list_wait")
        return r.as_dict()

    def close(self):
        if getattr(self, "_h", None):
            lib().mpt_list_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


XentLoss = collections.namedtuple("XentLoss", "loss token_loss lse n_valid")
XentGrad = collections.namedtuple("XentGrad", "loss token_loss lse n_valid grad_hidden grad_weight")


def _rows(t, what, dtype, device, shape=None):
    """The row distance of a 2-D CUDA tensor whose rows are contiguous."""
    if t.dim() != 2 or t.dtype != dtype or t.device != device or (shape is not None and t.shape != shape):
        raise ValueError(f"{what} must be a 2-D tensor of the type, device and width of hidden"
                         + (f" and the shape {tuple(shape)}" if shape is not None else ""))
    (n, d), (ld, step) = t.shape, t.stride()
    if step != 1 and d > 1:
        raise ValueError(f"{what} must have contiguous rows")
    return ld if n > 1 else (d + 7) // 8 * 8  # one row has no next


def _xent(hidden, weight, targets, scale, ignore_index, reduction, grad_hidden, grad_weight, stream):
    import torch
    L = lib()
    dev, dtype = hidden.device, hidden.dtype
    if dev.type != "cuda" or dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("hidden must be a float16 or bfloat16 CUDA tensor")
    ld_h = _rows(hidden, "hidden", dtype, dev)
    n, d = hidden.shape
    ld_w = _rows(weight, "weight", dtype, dev)
    v, width = weight.shape
    if width != d:
        raise ValueError("hidden and weight must have rows of one width")
    if targets.shape != (n,) or targets.device != dev or not targets.is_contiguous() or \
            targets.dtype not in (torch.int64, torch.int32):
        raise ValueError("targets must be one int32 or int64 per row of hidden, contiguous, on its device")
    if reduction not in ("mean", "sum"):
        raise ValueError("reduction is 'mean' or 'sum'")
    _check_stream(stream, dev)
    host_scale, dev_scale = _scale_args(scale, dev)
    if stream is not None:
        _used_on(stream, hidden, weight, targets, scale, grad_hidden, grad_weight)
    # what the call allocates belongs to the stream that it runs on
    with _on(dev, stream):
        # one allocation for the small results
        n_valid, loss, _, token_loss, lse = torch.unsafe_split_with_sizes(
            hidden.new_empty(4 + 2 * n, dtype=torch.float32), (2, 1, 1, n, n))
        n_valid = n_valid.view(torch.int64)
        gh = gw = None
        ld_gh = ld_gw = 0
        if grad_hidden is not None and grad_hidden is not False:
            gh = hidden.new_empty((n, d)) if grad_hidden is True else grad_hidden
            ld_gh = _rows(gh, "grad_hidden", dtype, dev, hidden.shape)
        if grad_weight is not None and grad_weight is not False:
            gw = hidden.new_empty((v, d)) if grad_weight is True else grad_weight
            ld_gw = _rows(gw, "grad_weight", dtype, dev, weight.shape)
        a = XentArgs(_type_code(dtype), targets.element_size(), n, v, d, hidden.data_ptr(), ld_h,
                     weight.data_ptr(), ld_w, targets.data_ptr(), ignore_index,
                     MPT_XENT_SUM if reduction == "sum" else MPT_XENT_MEAN, host_scale, dev_scale,
                     loss.data_ptr(), token_loss.data_ptr(), lse.data_ptr(), n_valid.data_ptr(),
                     None if gh is None else gh.data_ptr(), ld_gh, None if gw is None else gw.data_ptr(), ld_gw)
        nbytes = ctypes.c_size_t()
        _check(L.mpt_xent_workspace_bytes(ctypes.byref(a), ctypes.byref(nbytes)), "mpt_xent_workspace_bytes")
        ws = hidden.new_empty(nbytes.value, dtype=torch.uint8)
        _check(L.mpt_xent(ctypes.byref(a), ws.data_ptr(), nbytes.value, _stream_ptr(stream, dev)), "mpt_xent")
    return loss, token_loss, lse, n_valid, gh, gw


def xent_loss(hidden, weight, targets, ignore_index=-100, reduction="mean", stream=None):
    """Softmax cross entropy of ``hidden @ weight.T`` against ``targets``
    (``mpt_xent`` without gradients), queued; the logits are not stored.

    Returns ``XentLoss``: ``loss`` (float32, 1 value), ``token_loss`` and
    ``lse`` (float32, one per row), ``n_valid`` (int64, 1 value)."""
    return XentLoss(*_xent(hidden, weight, targets, 1.0, ignore_index, reduction, None, None, stream)[:4])


def xent_grad(hidden, weight, targets, scale=1.0, ignore_index=-100, reduction="mean", grad_hidden=True,
              grad_weight=True, stream=None):
    """The same with the gradients of ``scale * loss`` (``mpt_xent``).  At most
    256 MB of the logits' gradient are held at a time, and up to 256 MB of logits.

    ``scale`` is S: a number, or a 1-element float32 CUDA tensor such as
    :meth:`MPT.device_scale`.  ``grad_hidden`` and ``grad_weight`` are tensors
    to write, True for new ones, or None for none.  Returns ``XentGrad``."""
    return XentGrad(*_xent(hidden, weight, targets, scale, ignore_index, reduction, grad_hidden, grad_weight, stream))
