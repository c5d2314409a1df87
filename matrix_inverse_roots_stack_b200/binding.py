"""ctypes binding of libdash_b200.so (argument marshalling only).

Every function named ``shampoo_*`` here forwards to the C entry point of the
same name declared in ``include/dash_b200.h``.  The torch helpers at the end
only allocate device buffers with PyTorch and pass their pointers; all of the
step's arithmetic runs in the library's CUDA kernels.  There is no fallback:
if the shared library is missing the import of this module's users fails.
"""

import ctypes
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libdash_b200.so")

SHAMPOO_OK = 0
SHAMPOO_EINVAL = -1
SHAMPOO_EUNSUPPORTED = -2
SHAMPOO_EWORKSPACE = -3
SHAMPOO_ECUDA = -4
SHAMPOO_ENONFINITE = -5
SHAMPOO_ETIMEOUT = -6
SOLVER_NEWTON_DB = 0
SOLVER_CHEBYSHEV = 1
SOLVER_COUPLED_NEWTON = 2
SCALING_SPECTRAL = 0
SCALING_FROBENIUS = 1
PI_STARTS = 32
DTYPE_F32 = 0
DTYPE_BF16 = 1
DTYPE_F16 = 2
QBLOCK = 256  # elements that share a scale in 8-bit moments
MAX_STEP = 0x7fffffff  # step numbers are C ints, which ctypes cuts to their low 32 bits


class ShampooError(RuntimeError):
    def __init__(self, code, where):
        super().__init__(f"{where}: {strerror(code)} ({code})")
        self.code = code


class ShampooParam(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("param", ctypes.c_void_p),
                ("grad", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p)]


class ShampooHParams(ctypes.Structure):
    _fields_ = [("block_size", ctypes.c_int), ("beta", ctypes.c_float), ("eps", ctypes.c_float),
                ("init_scale", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("adam_eps", ctypes.c_float), ("lr", ctypes.c_float), ("solver", ctypes.c_int),
                ("ndb_iters1", ctypes.c_int), ("ndb_iters2", ctypes.c_int), ("cheb_degree", ctypes.c_int),
                ("cheb_delta", ctypes.c_float), ("pi_starts", ctypes.c_int), ("pi_iters", ctypes.c_int),
                ("root_every", ctypes.c_int), ("scaling", ctypes.c_int), ("cn_iters", ctypes.c_int),
                ("cn_fp16", ctypes.c_int)]


class ShampooGrad(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("grad", ctypes.c_void_p), ("dtype", ctypes.c_int)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("copy", ctypes.c_void_p), ("m", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("m_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p), ("param_dtype", ctypes.c_int),
                ("grad_dtype", ctypes.c_int), ("copy_dtype", ctypes.c_int), ("state_bits", ctypes.c_int),
                ("lr_scale", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class AdamwHParams(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_float), ("beta2", ctypes.c_float), ("adam_eps", ctypes.c_float),
                ("seed", ctypes.c_uint64)]


def make_hparams(block_size=1024, beta=0.95, eps=1e-6, init_scale=1e-6, beta1=0.9, beta2=0.999,
                 adam_eps=1e-8, lr=1e-3, solver=SOLVER_NEWTON_DB, ndb_iters1=14, ndb_iters2=14,
                 cheb_degree=16, cheb_delta=1e-3, pi_starts=PI_STARTS, pi_iters=10, root_every=1,
                 scaling=SCALING_SPECTRAL, cn_iters=16, cn_fp16=0):
    return ShampooHParams(block_size, beta, eps, init_scale, beta1, beta2, adam_eps, lr, solver,
                          ndb_iters1, ndb_iters2, cheb_degree, cheb_delta, pi_starts, pi_iters, root_every,
                          scaling, cn_iters, cn_fp16)


def make_adamw_hparams(beta1=0.9, beta2=0.999, adam_eps=1e-8, seed=0):
    return AdamwHParams(beta1, beta2, adam_eps, seed)


_lib = None

_VP, _SZ, _I, _F = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
_PROTOS = {
    "shampoo_init_blocks": (_I, [ctypes.POINTER(_VP), ctypes.POINTER(ShampooParam), _I,
                                 ctypes.POINTER(ShampooHParams), ctypes.POINTER(_SZ)]),
    "shampoo_ctx_info": (_I, [_VP, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "shampoo_block_table": (_I, [_VP, ctypes.POINTER(ctypes.c_int64)]),
    "shampoo_init_factors": (_I, [_VP, _VP, _VP]),
    "shampoo_accumulate": (_I, [_VP, _VP, _VP, _SZ, _VP]),
    "shampoo_precondition_step": (_I, [_VP, _VP, _VP, _I, _VP, _VP, _VP, _SZ, _VP]),
    "shampoo_inv_root_newton_db": (_I, [_VP, _VP, _I, _I, _I, _I, _F, _VP, _I, _VP, _VP, _SZ, _VP]),
    "shampoo_inv_root_chebyshev": (_I, [_VP, _VP, _I, _I, _I, _F, _F, _VP, _I, _VP, _VP, _SZ, _VP]),
    "shampoo_inv_root_coupled_newton": (_I, [_VP, _VP, _I, _I, _I, _I, _F, _VP, _I, _VP, _VP, _SZ, _VP]),
    "shampoo_inv_root_workspace_bytes": (_SZ, [_I, _I, _I]),
    "shampoo_read_status": (_I, [_VP, _VP, ctypes.POINTER(ctypes.c_uint)]),
    "shampoo_read_static_status": (_I, [_VP, ctypes.POINTER(ctypes.c_uint)]),
    "shampoo_get_status": (_I, [_VP, ctypes.POINTER(ctypes.c_int)]),
    "shampoo_strerror": (ctypes.c_char_p, [_I]),
    "shampoo_destroy": (None, [_VP]),
    "shampoo_inv_root_newton_db_static": (_I, [_VP, _VP, _I, _I, _I, _I, _F, _VP, _I, _VP, _VP]),
    "shampoo_grads_init": (_I, [ctypes.POINTER(_VP), ctypes.POINTER(ShampooGrad), _I, ctypes.POINTER(_SZ)]),
    "shampoo_grads_bind": (_I, [_VP, _VP, _SZ, _VP]),
    "shampoo_grad_norm": (_I, [_VP, _F, _F, _VP, _VP, _SZ, _VP]),
    "shampoo_grad_clip": (_I, [_VP, _F, _F, _VP, _VP, _SZ, _VP]),
    "shampoo_grads_destroy": (None, [_VP]),
    "shampoo_adamw_init": (_I, [ctypes.POINTER(_VP), ctypes.POINTER(AdamwTensor), _I, ctypes.POINTER(AdamwHParams),
                                ctypes.POINTER(_SZ), ctypes.POINTER(ctypes.c_int64)]),
    "shampoo_adamw_bind": (_I, [_VP, _I, _VP, _SZ, _VP]),
    "shampoo_adamw_step": (_I, [_VP, _I, _F, _VP, _VP, _VP, _SZ, _VP]),
    "shampoo_adamw_load_moments": (_I, [_VP, _VP, _VP, _VP, _SZ, _VP]),
    "shampoo_adamw_read_moments": (_I, [_VP, _VP, _VP, _I, _VP, _SZ, _VP]),
    "shampoo_adamw_steps_taken": (_I, [_VP, _VP, _SZ, _VP, ctypes.POINTER(_I)]),
    "shampoo_adamw_destroy": (None, [_VP]),
    "shampoo_debug_inject_timeout": (_I, []),
    "shampoo_profile_enable": (_I, [_I]),
    "shampoo_profile_reset": (_I, []),
    "shampoo_profile_read": (_I, [ctypes.POINTER(ctypes.c_double), _I]),
}


def load():
    """Load the shared library (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing; build it with "
                              "`python -m matrix_inverse_roots_stack_b200.build`")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _PROTOS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def exported_names():
    return sorted(_PROTOS)


def strerror(code):
    return load().shampoo_strerror(int(code)).decode()


def _check(code, where):
    if code != SHAMPOO_OK:
        raise ShampooError(code, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# --------------------------------------------------------------------------
# torch helpers (device memory and streams only)
# --------------------------------------------------------------------------

def _workspace(nbytes, device):
    import torch
    # torch's caching allocator returns 512-byte aligned blocks
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def _outputs(stream, device, given, make):
    """`given`, and in the places of None what `make` allocates there: on
    `stream`, where it is written.  (What was freed on the current stream may
    be in its queued work's use still.)  The current stream, which uses them
    next, holds them too."""
    if all(t is not None for t in given):
        return given
    import torch
    with torch.cuda.stream(stream):
        out = [f() if t is None else t for t, f in zip(given, make)]
    if stream is not None:
        for t, g in zip(out, given):
            if g is None:
                t.record_stream(torch.cuda.current_stream(device))
    return out


def inv_root_workspace_bytes(n, B, solver=SOLVER_NEWTON_DB):
    return int(load().shampoo_inv_root_workspace_bytes(n, B, solver))


def inv_root_newton_db(A, v0, iters1=14, iters2=14, eps=0.0, pi_iters=10, X=None, lam=None, ws=None,
                       stream=None):
    """X = (A + eps I)^(-1/4) for a (n, B, B) fp32 CUDA stack via the library's
    Newton-DB path.  Returns (X, lambda, ws)."""
    import torch
    n, B = A.shape[0], A.shape[1]
    need = inv_root_workspace_bytes(n, B, SOLVER_NEWTON_DB)
    X, lam, ws = _outputs(stream, A.device, (X, lam, ws), (
        lambda: torch.empty_like(A), lambda: torch.empty(n, dtype=torch.float32, device=A.device),
        lambda: _workspace(need, A.device)))
    rc = load().shampoo_inv_root_newton_db(_ptr(A), _ptr(X), n, B, iters1, iters2, eps, _ptr(v0), pi_iters,
                                           _ptr(lam), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "shampoo_inv_root_newton_db")
    return X, lam, ws


def inv_root_chebyshev(A, v0, degree=16, delta=1e-3, eps=0.0, pi_iters=10, X=None, lam=None, ws=None,
                       stream=None):
    """Chebyshev/Clenshaw variant of :func:`inv_root_newton_db`."""
    import torch
    n, B = A.shape[0], A.shape[1]
    need = inv_root_workspace_bytes(n, B, SOLVER_CHEBYSHEV)
    X, lam, ws = _outputs(stream, A.device, (X, lam, ws), (
        lambda: torch.empty_like(A), lambda: torch.empty(n, dtype=torch.float32, device=A.device),
        lambda: _workspace(need, A.device)))
    rc = load().shampoo_inv_root_chebyshev(_ptr(A), _ptr(X), n, B, degree, delta, eps, _ptr(v0), pi_iters,
                                           _ptr(lam), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "shampoo_inv_root_chebyshev")
    return X, lam, ws


STATIC_SCRATCH_BYTES = 64 << 20


def inv_root_coupled_newton(A, v0, iters=16, fp16=False, eps=0.0, pi_iters=10, X=None, lam=None, ws=None,
                            stream=None):
    """Coupled-Newton variant of :func:`inv_root_newton_db` (fp16: single-pass
    fp16 products)."""
    import torch
    n, B = A.shape[0], A.shape[1]
    need = inv_root_workspace_bytes(n, B, SOLVER_COUPLED_NEWTON)
    X, lam, ws = _outputs(stream, A.device, (X, lam, ws), (
        lambda: torch.empty_like(A), lambda: torch.empty(n, dtype=torch.float32, device=A.device),
        lambda: _workspace(need, A.device)))
    rc = load().shampoo_inv_root_coupled_newton(_ptr(A), _ptr(X), n, B, iters, 1 if fp16 else 0, eps, _ptr(v0),
                                                pi_iters, _ptr(lam), _ptr(ws), ws.numel(), _stream(stream))
    _check(rc, "shampoo_inv_root_coupled_newton")
    return X, lam, ws


def inv_root_newton_db_static(A, v0, iters1=14, iters2=14, eps=0.0, pi_iters=10, X=None, lam=None, stream=None):
    """:func:`inv_root_newton_db` through the entry point that uses the
    library's fixed scratch instead of a workspace (nothing is allocated by
    the library; X and lambda are allocated here only if not given)."""
    import torch
    n, B = A.shape[0], A.shape[1]
    X, lam = _outputs(stream, A.device, (X, lam), (
        lambda: torch.empty_like(A), lambda: torch.empty(n, dtype=torch.float32, device=A.device)))
    rc = load().shampoo_inv_root_newton_db_static(_ptr(A), _ptr(X), n, B, iters1, iters2, eps, _ptr(v0), pi_iters,
                                                  _ptr(lam), _stream(stream))
    _check(rc, "shampoo_inv_root_newton_db_static")
    return X, lam


def read_status(ws, stream=None):
    """Synchronise and return (code, flags) of a workspace's status word."""
    flags = ctypes.c_uint(0)
    rc = load().shampoo_read_status(_ptr(ws), _stream(stream), ctypes.byref(flags))
    return rc, flags.value


def read_static_status(stream=None):
    """(code, flags) of the static scratch's status word (after
    :func:`inv_root_newton_db_static`)."""
    flags = ctypes.c_uint(0)
    rc = load().shampoo_read_static_status(_stream(stream), ctypes.byref(flags))
    return rc, flags.value


PROFILE_STAGES = ("gemm", "accumulate", "power_iteration", "solver", "precondition", "adam_update", "gemm_wide",
                  "ndb_fused")


def profile_enable(on=True):
    _check(load().shampoo_profile_enable(1 if on else 0), "shampoo_profile_enable")


def profile_reset():
    _check(load().shampoo_profile_reset(), "shampoo_profile_reset")


def profile_read():
    """Return {stage: (ms, count, flops)}, plus "launches" and "dropped"."""
    n = 3 * len(PROFILE_STAGES) + 3
    buf = (ctypes.c_double * n)()
    _check(load().shampoo_profile_read(buf, n), "shampoo_profile_read")
    out = {s: (buf[3 * i], int(buf[3 * i + 1]), buf[3 * i + 2]) for i, s in enumerate(PROFILE_STAGES)}
    out["launches"] = int(buf[n - 3])
    out["dropped"] = int(buf[n - 2])
    out["wide_regs"] = int(buf[n - 1])
    return out


class Shampoo:
    """Batched block-Shampoo optimizer state over a list of CUDA fp32
    parameter/gradient tensors.  The factor stack, Adam moments and
    workspace are torch allocations; every step runs in the library."""

    def __init__(self, params, grads, hp=None, v0=None, m=None, v=None):
        import torch
        self.hp = hp if hp is not None else make_hparams()
        self.params, self.grads = list(params), list(grads)
        dev = self.params[0].device
        self.m = m if m is not None else [torch.zeros_like(p) for p in self.params]
        self.v = v if v is not None else [torch.zeros_like(p) for p in self.params]
        for t in self.params + self.grads + self.m + self.v:
            if t.dtype != torch.float32 or not t.is_contiguous() or t.dim() != 2 or not t.is_cuda:
                raise ValueError("parameters, gradients and moments must be contiguous 2-D fp32 CUDA tensors")
        arr = (ShampooParam * len(self.params))()
        for i, (p, g, m_, v_) in enumerate(zip(self.params, self.grads, self.m, self.v)):
            arr[i] = ShampooParam(p.shape[0], p.shape[1], p.data_ptr(), g.data_ptr(), m_.data_ptr(),
                                  v_.data_ptr())
        ctx = ctypes.c_void_p()
        nbytes = ctypes.c_size_t(0)
        _check(load().shampoo_init_blocks(ctypes.byref(ctx), arr, len(self.params), ctypes.byref(self.hp),
                                          ctypes.byref(nbytes)), "shampoo_init_blocks")
        self._ctx = ctx
        nb, nf, B = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
        load().shampoo_ctx_info(ctx, ctypes.byref(nb), ctypes.byref(nf), ctypes.byref(B))
        self.n_blocks, self.n_factors, self.B = nb.value, nf.value, B.value
        self.ws = _workspace(nbytes.value, dev)
        self.factors = torch.empty((self.n_factors, self.B, self.B), dtype=torch.float32, device=dev)
        if v0 is None:
            from .workloads import pi_start_vectors
            v0 = torch.from_numpy(pi_start_vectors(self.B, PI_STARTS, seed=0)).to(dev)
        self.v0 = v0
        self.lam = torch.empty(self.n_factors, dtype=torch.float32, device=dev)
        self.t = 0
        _check(load().shampoo_init_factors(ctx, _ptr(self.factors), _stream(None)), "shampoo_init_factors")

    def block_table(self):
        import numpy as np
        out = np.zeros((self.n_blocks, 7), dtype=np.int64)
        _check(load().shampoo_block_table(self._ctx, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))),
               "shampoo_block_table")
        return out

    def accumulate(self, stream=None):
        _check(load().shampoo_accumulate(self._ctx, _ptr(self.factors), _ptr(self.ws), self.ws.numel(),
                                         _stream(stream)), "shampoo_accumulate")

    def precondition_step(self, roots_out=None, stream=None, device_step=False):
        """device_step: take the step number from the counter on the device
        (for steps captured into a CUDA graph; needs an earlier eager step)."""
        self.t += 1
        _check(load().shampoo_precondition_step(self._ctx, _ptr(self.factors), _ptr(self.v0),
                                                0 if device_step else self.t,
                                                _ptr(self.lam), _ptr(roots_out), _ptr(self.ws),
                                                self.ws.numel(), _stream(stream)),
               "shampoo_precondition_step")

    def step(self, roots_out=None, stream=None, device_step=False):
        """One full step: factor EMA, roots, precondition, Adam graft, update."""
        self.accumulate(stream)
        self.precondition_step(roots_out, stream, device_step)

    def status(self, stream=None):
        return read_status(self.ws, stream)

    def get_status(self):
        """(code, flags) of the last step call's workspace, on the stream it
        was given (the library remembers both)."""
        flags = ctypes.c_int(0)
        rc = load().shampoo_get_status(self._ctx, ctypes.byref(flags))
        return rc, flags.value

    def __del__(self):
        ctx = getattr(self, "_ctx", None)
        if ctx is not None and _lib is not None:
            _lib.shampoo_destroy(ctx)
            self._ctx = None


# --------------------------------------------------------------------------
# operators over a list of tensors: gradient norm and clipping, AdamW
# --------------------------------------------------------------------------

def _dtype_code(t):
    import torch
    return {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16, torch.float16: DTYPE_F16}.get(t.dtype)


def _check_list(tensors, what, dtypes, device, like=None):
    """Contiguous CUDA tensors (or None entries) of one device and of the given
    types; `like`: tensors whose shapes they have."""
    index = device.index
    for i, t in enumerate(tensors):
        if t is None:
            continue
        if t.dtype not in dtypes or t.get_device() != index or not t.is_contiguous():
            raise ValueError(f"{what}[{i}] must be a contiguous tensor on {device} of type "
                             f"{' or '.join(str(d) for d in dtypes)}")
        if like is not None and t.shape != like[i].shape:
            raise ValueError(f"{what}[{i}] has shape {tuple(t.shape)}, not {tuple(like[i].shape)}")


class _TensorList:
    """What the operators over a list of tensors share: the library's list,
    its workspace, and the streams it is used on.  A step is one launch of a
    few microseconds, so what a call needs is looked up here once."""

    _destroy = None

    def _adopt(self, ctx, ws_bytes, held):
        """held: every tensor that the list's calls work on.  Those that the
        caller made are, as with torch's own operations, taken to be the
        current stream's."""
        import torch
        self._ctx = ctx
        self._cuda, self._device = torch.cuda, torch.cuda.current_device
        self._index = self.device.index
        self.ws = _workspace(ws_bytes, self.device)
        self._ws_at, self._ws_bytes = self.ws.data_ptr(), self.ws.numel()
        self._held = [self.ws] + held
        self._streams = {torch.cuda.current_stream(self.device).cuda_stream}
        # the current stream's handle, without an object around it where torch offers that
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        self._current = raw if raw is not None else lambda index: torch.cuda.current_stream(index).cuda_stream

    def _on(self, stream, *passed):
        """The handle of `stream` (default: the current stream of the list's
        device).  passed: the caller's tensors that the call works on."""
        if stream is None:
            raw = self._current(self._index)
        elif stream.device != self.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors are on {self.device}")
        else:
            raw = stream.cuda_stream
            for t in passed:
                if t is not None:
                    t.record_stream(stream)
        if raw not in self._streams:
            # the list's memory is not handed out again before this stream is done with it
            for t in self._held:
                t.record_stream(self._cuda.current_stream(self.device) if stream is None else stream)
            self._streams.add(raw)
        return raw

    def _run(self, fn, *args):
        """A library call, on the list's device."""
        if self._device() == self._index:
            rc = fn(*args)
        else:
            with self._cuda.device(self.device):
                rc = fn(*args)
        if rc:
            raise ShampooError(rc, fn.__name__)

    def status(self, stream=None):
        """Synchronise and return (code, flags) of the last call."""
        return read_status(self.ws, self._cuda.current_stream(self.device) if stream is None else stream)

    def __del__(self):
        ctx = getattr(self, "_ctx", None)
        if ctx is not None and _lib is not None:
            getattr(_lib, self._destroy)(ctx)
            self._ctx = None


class GradClip(_TensorList):
    """Global norm and clipping of a list of CUDA gradients (fp32, bf16 or
    fp16, any shapes).  The gradients' addresses are fixed here, their values
    are read at every call.  Results stay on the device, in :attr:`out`:
    [norm, coef], with coef = inv_scale min(1, max_norm / norm), NaN where a
    gradient is not finite.  (The norm of finite gradients that lies beyond
    fp32 is infinite there, and coef finite all the same.)"""

    _destroy = "shampoo_grads_destroy"

    def __init__(self, grads):
        import torch
        self.grads = list(grads)
        if not self.grads:
            raise ValueError("no gradients")
        self.device = self.grads[0].device
        _check_list(self.grads, "grads", (torch.float32, torch.bfloat16, torch.float16), self.device)
        arr = (ShampooGrad * len(self.grads))()
        for i, g in enumerate(self.grads):
            arr[i] = ShampooGrad(g.numel(), g.data_ptr(), _dtype_code(g))
        ctx, nbytes = ctypes.c_void_p(), ctypes.c_size_t(0)
        _check(load().shampoo_grads_init(ctypes.byref(ctx), arr, len(self.grads), ctypes.byref(nbytes)),
               "shampoo_grads_init")
        self.out = torch.zeros(2, dtype=torch.float32, device=self.device)
        self._out_at = self.out.data_ptr()
        self._adopt(ctx, nbytes.value, self.grads + [self.out])
        self._norm, self._clip = _lib.shampoo_grad_norm, _lib.shampoo_grad_clip
        self._run(_lib.shampoo_grads_bind, ctx, self._ws_at, self._ws_bytes, self._on(None))
        torch.cuda.current_stream(self.device).synchronize()  # ready for any stream

    def norm(self, max_norm=float("inf"), inv_scale=1.0, stream=None):
        """Fill and return :attr:`out`; the gradients are only read."""
        self._run(self._norm, self._ctx, max_norm, inv_scale, self._out_at, self._ws_at, self._ws_bytes,
                  self._on(stream))
        return self.out

    def clip(self, max_norm, inv_scale=1.0, stream=None):
        """:meth:`norm`, then every gradient times coef, in place (zero where
        coef is NaN)."""
        self._run(self._clip, self._ctx, max_norm, inv_scale, self._out_at, self._ws_at, self._ws_bytes,
                  self._on(stream))
        return self.out


class AdamW(_TensorList):
    """AdamW (decoupled weight decay) over a list of CUDA parameters of any
    shapes, one kernel launch a step.

    params: fp32 or bf16 (bf16 is rounded stochastically); grads: fp32, bf16
    or fp16.  copies: for fp32 parameters, 16-bit tensors (or None entries)
    that receive the new values too.  state_bits: 32 or 8, for all or for each
    parameter; moments that are not given are allocated as zeros: fp32, or
    8-bit codes with a scale for each 256 elements.  lr_scale and weight_decay:
    for all or for each parameter.  Addresses are fixed here; the contents may
    change between steps.
    """

    _destroy = "shampoo_adamw_destroy"

    def __init__(self, params, grads, hp=None, copies=None, state_bits=32, m=None, v=None, m_scale=None,
                 v_scale=None, lr_scale=1.0, weight_decay=0.0, steps_taken=0):
        import torch
        f32, bf16, f16 = torch.float32, torch.bfloat16, torch.float16
        self.hp = hp if hp is not None else make_adamw_hparams()
        self.params, self.grads = list(params), list(grads)
        n = len(self.params)
        if not n:
            raise ValueError("no parameters")
        self.device = dev = self.params[0].device

        def each(x, what):
            x = list(x) if isinstance(x, (list, tuple)) else [x] * n
            if len(x) != n:
                raise ValueError(f"{len(x)} {what} for {n} parameters")
            return x

        self.state_bits = each(state_bits, "state_bits")
        lr_scale, weight_decay = each(lr_scale, "lr_scale"), each(weight_decay, "weight_decay")
        self.copies = each(copies, "copies")
        if any(b not in (8, 32) for b in self.state_bits):
            raise ValueError("state_bits must be 8 or 32")
        if not -MAX_STEP <= steps_taken <= MAX_STEP:  # the library refuses negative ones
            raise ValueError(f"steps_taken {steps_taken} is not a 32-bit number")
        if len(self.grads) != n:
            raise ValueError(f"{len(self.grads)} gradients for {n} parameters")
        _check_list(self.params, "params", (f32, bf16), dev)
        _check_list(self.grads, "grads", (f32, bf16, f16), dev, self.params)
        sizes = [p.numel() for p in self.params]
        eight = [b == 8 for b in self.state_bits]

        def state(given, what, types, numels):
            """The given moments or scales, checked, or zeros; None where a
            parameter has none."""
            out = each(given, what)
            for i, (t, dtype, numel) in enumerate(zip(out, types, numels)):
                if t is None:
                    if numel is not None:
                        out[i] = torch.zeros(numel, dtype=dtype, device=dev)
                elif numel is None:
                    raise ValueError(f"{what}[{i}] is for 8-bit moments only")
                elif t.numel() != numel:
                    raise ValueError(f"{what}[{i}] has {t.numel()} elements, not {numel}")
                elif t.dtype != dtype:
                    raise ValueError(f"{what}[{i}] must be of type {dtype}")
            _check_list(out, what, (f32, torch.uint8), dev)
            return out

        codes = [torch.uint8 if e else f32 for e in eight]
        bytes_ = [torch.uint8] * n
        blocks = [-(-k // QBLOCK) if e else None for k, e in zip(sizes, eight)]
        self.m, self.v = state(m, "m", codes, sizes), state(v, "v", codes, sizes)
        self.m_scale = state(m_scale, "m_scale", bytes_, blocks)
        self.v_scale = state(v_scale, "v_scale", bytes_, blocks)
        if any(c is not None and p.dtype != f32 for p, c in zip(self.params, self.copies)):
            raise ValueError("copies are for fp32 parameters only")
        _check_list(self.copies, "copies", (bf16, f16), dev, self.params)
        code = {f32: DTYPE_F32, bf16: DTYPE_BF16, f16: DTYPE_F16}
        at = lambda t: None if t is None else t.data_ptr()
        arr = (AdamwTensor * n)(*[
            (k, p.data_ptr(), g.data_ptr(), at(c), m_.data_ptr(), v_.data_ptr(), at(ms), at(vs), code[p.dtype],
             code[g.dtype], DTYPE_F32 if c is None else code[c.dtype], b, ls, wd)
            for k, p, g, c, m_, v_, ms, vs, b, ls, wd in zip(sizes, self.params, self.grads, self.copies, self.m, self.v,
                                                             self.m_scale, self.v_scale, self.state_bits, lr_scale,
                                                             weight_decay)])
        ctx, nbytes, elems = ctypes.c_void_p(), ctypes.c_size_t(0), ctypes.c_int64(0)
        _check(load().shampoo_adamw_init(ctypes.byref(ctx), arr, n, ctypes.byref(self.hp), ctypes.byref(nbytes),
                                         ctypes.byref(elems)), "shampoo_adamw_init")
        self.moment_elems = elems.value
        held = self.params + self.grads + self.copies + self.m + self.v + self.m_scale + self.v_scale
        self._adopt(ctx, nbytes.value, [t for t in held if t is not None])
        self._dtypes = {f32: DTYPE_F32, bf16: DTYPE_BF16}
        self._step = _lib.shampoo_adamw_step
        self._read, self._load = _lib.shampoo_adamw_read_moments, _lib.shampoo_adamw_load_moments
        self._run(_lib.shampoo_adamw_bind, ctx, steps_taken, self._ws_at, self._ws_bytes, self._on(None))
        torch.cuda.current_stream(dev).synchronize()  # ready for any stream

    def step(self, lr=1e-3, coef=None, step=0, stream=None):
        """One step.  lr: a number, or one fp32 value on the device (read when
        the step runs, also from a replayed graph).  coef: one fp32 value on
        the device that multiplies the gradients (``GradClip.out[1:]``); where
        it is not finite the step is not taken.  step: this step's number, or
        0 to continue the counter on the device."""
        held = lr_at = coef_at = None
        if type(lr) is not float:
            if hasattr(lr, "data_ptr"):
                lr, lr_at, held = 0.0, self._scalar(lr, "lr"), lr
            else:
                lr = float(lr)
        if coef is not None:
            coef_at = self._scalar(coef, "coef")
        if not -MAX_STEP <= step <= MAX_STEP:  # the library refuses negative ones
            raise ValueError(f"step {step} is not a 32-bit number")
        self._run(self._step, self._ctx, step, lr, lr_at, coef_at, self._ws_at, self._ws_bytes,
                  self._on(stream, held, coef))

    def steps_taken(self, stream=None):
        """Synchronise and read the step counter."""
        t = ctypes.c_int(0)
        self._run(_lib.shampoo_adamw_steps_taken, self._ctx, self._ws_at, self._ws_bytes, self._on(stream),
                  ctypes.byref(t))
        return t.value

    def _scalar(self, t, what):
        if self._dtypes.get(t.dtype) != DTYPE_F32 or t.numel() != 1 or t.get_device() != self._index:
            raise ValueError(f"{what} must be one fp32 value on {self.device}")
        return t.data_ptr()

    def _flat(self, t, what):
        if t.dtype not in self._dtypes or t.numel() != self.moment_elems or not t.is_contiguous() or \
                t.get_device() != self._index:
            raise ValueError(f"{what} must be {self.moment_elems} contiguous fp32 or bf16 values on {self.device}")
        return t.data_ptr()

    def views(self, flat):
        """Each parameter's part of a flat tensor of moments, in its shape."""
        out, at = [], 0
        for p in self.params:
            out.append(flat[at:at + p.numel()].view(p.shape))
            at += -(-p.numel() // QBLOCK) * QBLOCK
        return out

    def read_moments(self, dtype=None, m=None, v=None, stream=None):
        """Both moments as flat tensors (see :meth:`views`) of fp32 or bf16
        (default: the type of the one that is given, or fp32), into m and v
        where given.  Those that are not given are made
        on `stream`: other streams wait for it before they use them."""
        if m is None or v is None:
            import torch
            given = m if v is None else v
            of = dtype or (torch.float32 if given is None else given.dtype)
            m, v = _outputs(stream, self.device, (m, v),
                            (lambda: torch.empty(self.moment_elems, dtype=of, device=self.device),) * 2)
        m_at, v_at = self._flat(m, "m"), self._flat(v, "v")
        if v.dtype != m.dtype or (dtype is not None and m.dtype != dtype):
            raise ValueError("m and v must be of the one type asked for")
        self._run(self._read, self._ctx, m_at, v_at, self._dtypes[m.dtype], self._ws_at,
                  self._ws_bytes, self._on(stream, m, v))
        return m, v

    def load_moments(self, m, v, stream=None):
        """Set both moments from flat fp32 tensors (see :meth:`views`)."""
        m_at, v_at = self._flat(m, "m"), self._flat(v, "v")
        if self._dtypes[m.dtype] != DTYPE_F32 or self._dtypes[v.dtype] != DTYPE_F32:
            raise ValueError("moments are set from fp32 values")
        self._run(self._load, self._ctx, m_at, v_at, self._ws_at, self._ws_bytes,
                  self._on(stream, m, v))
