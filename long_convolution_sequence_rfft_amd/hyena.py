"""ctypes binding to ``libhyena_mi355x.so`` (the C ABI of include/hyena.h).

The functions below carry the C names and only marshal arguments: every step
of the computation runs in the library's HIP kernels.  ``Plan`` is a small
convenience wrapper that takes torch tensors (torch provides device memory
and the current HIP stream) and calls the same entry points.

There is no fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import struct
import threading

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhyena_mi355x.so")

HYENA_OK = 0
HYENA_ERR_INVALID_ARGUMENT = 1
HYENA_ERR_UNSUPPORTED = 2
HYENA_ERR_WORKSPACE = 3
HYENA_ERR_DEVICE = 4

HYENA_F32 = 0
HYENA_BF16 = 1
HYENA_F16 = 2

HYENA_PATH_AUTO = 0
HYENA_PATH_LDS1D = 1
HYENA_PATH_FOURSTEP1D = 2
HYENA_PATH_ROWCOL2D = 3
HYENA_PATH_ROWCOL3D = 4

EXPORTED_SYMBOLS = (
    "hyena_plan_create", "hyena_plan_query", "hyena_workspace_init", "hyena_filter_spectrum",
    "hyena_forward", "hyena_spectrum_export", "hyena_plan_destroy", "hyena_status_string",
    "hyena_last_error", "hyena_timing_begin", "hyena_timing_end", "hyena_timing_kernel",
    "hyena_timing_release", "hyena_implicit_scratch_bytes", "hyena_filter_spectrum_implicit",
    "hyena_plan_create_ex", "hyena_nd_mixer_forward", "hyena_workspace_release",
    "hyena_plan_path",
    "hyena_forward_noalloc",
    "hyena_recurrence_create", "hyena_recurrence_query", "hyena_recurrence_forward",
    "hyena_recurrence_backward", "hyena_recurrence_step", "hyena_recurrence_destroy",
    "hyena_qk_norm_forward", "hyena_qk_norm_scratch_bytes", "hyena_qk_norm_backward",
)

HYENA_NOALLOC_SCRATCH_BYTES = 128 << 20


class NdMixer(ctypes.Structure):
    """hyena_nd_mixer: q, k, v and the short-convolution taps (device pointers)."""
    _fields_ = [("q", ctypes.c_void_p), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("short_w", ctypes.c_void_p), ("short_b", ctypes.c_void_p)]

HYENA_FLAG_CIRCULAR = 1


class ImplicitFilter(ctypes.Structure):
    """hyena_implicit_filter: weights of the sine MLP that generates the taps
    (device pointers as ints; see include/hyena.h)."""
    _fields_ = [("n_freqs", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("omega", ctypes.c_float), ("W1", ctypes.c_void_p), ("b1", ctypes.c_void_p),
                ("W2", ctypes.c_void_p), ("b2", ctypes.c_void_p), ("W3", ctypes.c_void_p),
                ("b3", ctypes.c_void_p), ("alpha", ctypes.c_void_p)]


HYENA_NORM_NONE = 0
HYENA_NORM_RMS = 1
HYENA_NORM_L2 = 2
HYENA_ROTARY_HALF = 0
HYENA_ROTARY_INTERLEAVED = 1


class View(ctypes.Structure):
    """hyena_view: a [B, N, heads, width] tensor seen through element strides."""
    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_int64), ("token", ctypes.c_int64),
                ("head", ctypes.c_int64)]


class RecurrenceInputs(ctypes.Structure):
    """hyena_recurrence_inputs (device pointers as ints; see include/hyena.h)."""
    _fields_ = [("q", View), ("k", View), ("v", View), ("g", View), ("state", ctypes.c_void_p),
                ("lengths", ctypes.c_void_p), ("scale", ctypes.c_float)]


class RecurrenceGrads(ctypes.Structure):
    """hyena_recurrence_grads."""
    _fields_ = [("dq", ctypes.c_void_p), ("dk", ctypes.c_void_p), ("dv", ctypes.c_void_p),
                ("dg", ctypes.c_void_p), ("d_state", ctypes.c_void_p)]


class QkNorm(ctypes.Structure):
    """hyena_qk_norm: norms of queries and keys with the position rotation."""
    _fields_ = [("B", ctypes.c_int64), ("N", ctypes.c_int64), ("q_heads", ctypes.c_int64),
                ("k_heads", ctypes.c_int64), ("D", ctypes.c_int64), ("io_dtype", ctypes.c_int32),
                ("norm", ctypes.c_int32), ("layout", ctypes.c_int32), ("rotary_dim", ctypes.c_int64),
                ("eps", ctypes.c_float), ("rotary_scale", ctypes.c_float),
                ("freqs", ctypes.c_void_p), ("q_weight", ctypes.c_void_p),
                ("k_weight", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("position_offset", ctypes.c_int64), ("q", View), ("k", View)]

_lock = threading.Lock()
_lib = None


class HyenaError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {status_name(status)}: {detail}")
        self.status = status


def load():
    """Load the HIP library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with "
                    "long_convolution_sequence_rfft_amd.build.build()")
            lib = ctypes.CDLL(LIB_PATH)
            i64, i32, p, sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
            lib.hyena_plan_create.argtypes = [ctypes.POINTER(p), i64, i64, i64, i32,
                                              ctypes.POINTER(i64), i32, i32, i32]
            lib.hyena_plan_create_ex.argtypes = [ctypes.POINTER(p), i64, i64, i64, i32,
                                                 ctypes.POINTER(i64), i32, i32, i32, i32, i32]
            lib.hyena_plan_query.argtypes = [p, ctypes.POINTER(sz), ctypes.POINTER(sz)]
            lib.hyena_plan_path.argtypes = [p, ctypes.POINTER(i32)]
            lib.hyena_workspace_init.argtypes = [p, p, p]
            lib.hyena_workspace_release.argtypes = [p, p]
            lib.hyena_filter_spectrum.argtypes = [p, p, p, p, p]
            lib.hyena_forward.argtypes = [p, p, ctypes.POINTER(p), p, p, p, p, p]
            lib.hyena_forward_noalloc.argtypes = [p, p, ctypes.POINTER(p), p, p, p, p]
            lib.hyena_spectrum_export.argtypes = [p, p, p, p]
            lib.hyena_plan_destroy.argtypes = [p]
            lib.hyena_status_string.argtypes = [ctypes.c_int]
            lib.hyena_status_string.restype = ctypes.c_char_p
            lib.hyena_last_error.argtypes = []
            lib.hyena_last_error.restype = ctypes.c_char_p
            lib.hyena_timing_begin.argtypes = [i32]
            lib.hyena_timing_end.argtypes = [ctypes.POINTER(i32), ctypes.POINTER(i64)]
            lib.hyena_timing_kernel.argtypes = [i32, ctypes.POINTER(ctypes.c_char_p),
                                                ctypes.POINTER(i64)] + \
                [ctypes.POINTER(ctypes.c_double)] * 3
            lib.hyena_timing_release.argtypes = []
            lib.hyena_implicit_scratch_bytes.argtypes = [p, i32, ctypes.POINTER(sz)]
            lib.hyena_nd_mixer_forward.argtypes = [p, ctypes.POINTER(NdMixer), p, p, p, p, p]
            lib.hyena_filter_spectrum_implicit.argtypes = [p, ctypes.POINTER(ImplicitFilter), p, p,
                                                           p, p]
            lib.hyena_recurrence_create.argtypes = [ctypes.POINTER(p), i64, i64, i64, i64, i64, i32]
            lib.hyena_recurrence_query.argtypes = [p, ctypes.POINTER(sz), ctypes.POINTER(sz)]
            lib.hyena_recurrence_forward.argtypes = [p, p, p, p, p, p]
            lib.hyena_recurrence_backward.argtypes = [p, p, p, p, p, p, p]
            lib.hyena_recurrence_step.argtypes = [p, p, p, i64, p, p, p]
            lib.hyena_recurrence_destroy.argtypes = [p]
            lib.hyena_qk_norm_forward.argtypes = [p, p, p, p]
            lib.hyena_qk_norm_scratch_bytes.argtypes = [p, ctypes.POINTER(sz)]
            lib.hyena_qk_norm_backward.argtypes = [p] * 9
            for name in ("hyena_plan_create", "hyena_plan_create_ex", "hyena_plan_query",
                         "hyena_plan_path",
                         "hyena_workspace_init", "hyena_workspace_release",
                         "hyena_filter_spectrum", "hyena_forward", "hyena_forward_noalloc",
                         "hyena_spectrum_export",
                         "hyena_plan_destroy", "hyena_timing_begin", "hyena_timing_end",
                         "hyena_timing_kernel", "hyena_timing_release",
                         "hyena_implicit_scratch_bytes", "hyena_filter_spectrum_implicit",
                         "hyena_nd_mixer_forward", "hyena_recurrence_create",
                         "hyena_recurrence_query", "hyena_recurrence_forward",
                         "hyena_recurrence_backward", "hyena_recurrence_step",
                         "hyena_recurrence_destroy", "hyena_qk_norm_forward",
                         "hyena_qk_norm_scratch_bytes", "hyena_qk_norm_backward"):
                getattr(lib, name).restype = ctypes.c_int
            _lib = lib
    return _lib


def status_name(status: int) -> str:
    return load().hyena_status_string(int(status)).decode()


def hyena_last_error() -> str:
    return load().hyena_last_error().decode()


def hyena_status_string(status: int) -> str:
    return status_name(status)


def _check(status: int, where: str):
    if status != HYENA_OK:
        raise HyenaError(status, where, hyena_last_error())


# --------------------------------------------------------------------------
# C entry points (raw pointers as Python ints)
# --------------------------------------------------------------------------

def hyena_plan_create(B, N, d, order, dims, io_dtype=HYENA_F32, spectrum_dtype=None,
                      path=HYENA_PATH_AUTO, check=True, flags=0):
    """Returns (status, plan handle or None); a path other than AUTO, or flags,
    go through hyena_plan_create_ex."""
    lib = load()
    if spectrum_dtype is None:
        spectrum_dtype = HYENA_F32 if io_dtype == HYENA_F16 else io_dtype
    dims_arr = (ctypes.c_int64 * max(1, len(dims)))(*[int(x) for x in dims])
    h = ctypes.c_void_p()
    if flags or path != HYENA_PATH_AUTO:
        st = lib.hyena_plan_create_ex(ctypes.byref(h), int(B), int(N), int(d), int(order),
                                      dims_arr, len(dims), int(io_dtype), int(spectrum_dtype),
                                      int(path), int(flags))
    else:
        st = lib.hyena_plan_create(ctypes.byref(h), int(B), int(N), int(d), int(order), dims_arr,
                                   len(dims), int(io_dtype), int(spectrum_dtype))
    if check:
        _check(st, "hyena_plan_create")
    return st, (h.value if st == HYENA_OK else None)


def hyena_plan_query(plan):
    spec = ctypes.c_size_t()
    ws = ctypes.c_size_t()
    path = ctypes.c_int32()
    _check(load().hyena_plan_query(plan, ctypes.byref(spec), ctypes.byref(ws)), "hyena_plan_query")
    _check(load().hyena_plan_path(plan, ctypes.byref(path)), "hyena_plan_path")
    return spec.value, ws.value, path.value


def hyena_workspace_init(plan, workspace, stream=0):
    return load().hyena_workspace_init(plan, workspace, stream)


def hyena_workspace_release(plan, workspace):
    return load().hyena_workspace_release(plan, workspace)


def hyena_filter_spectrum(plan, h, H, workspace, stream=0):
    return load().hyena_filter_spectrum(plan, h, H, workspace, stream)


def hyena_forward(plan, u, gates, H, D, y, workspace, stream=0):
    arr = (ctypes.c_void_p * max(1, len(gates)))(*gates)
    return load().hyena_forward(plan, u, arr, H, D, y, workspace, stream)


def hyena_forward_noalloc(plan, u, gates, H, D, y, stream=0):
    arr = (ctypes.c_void_p * max(1, len(gates)))(*gates)
    return load().hyena_forward_noalloc(plan, u, arr, H, D, y, stream)


def hyena_implicit_scratch_bytes(plan, hidden):
    """Returns (status, bytes)."""
    n = ctypes.c_size_t()
    st = load().hyena_implicit_scratch_bytes(plan, int(hidden), ctypes.byref(n))
    return st, n.value


def hyena_filter_spectrum_implicit(plan, f, H, workspace, scratch, stream=0):
    return load().hyena_filter_spectrum_implicit(plan, ctypes.byref(f) if f is not None else None,
                                                 H, workspace, scratch, stream)


def hyena_nd_mixer_forward(plan, mixer, H, D, y, workspace, stream=0):
    return load().hyena_nd_mixer_forward(plan, ctypes.byref(mixer) if mixer is not None else None,
                                         H, D, y, workspace, stream)


def hyena_spectrum_export(plan, H, natural, stream=0):
    return load().hyena_spectrum_export(plan, H, natural, stream)


def hyena_plan_destroy(plan):
    return load().hyena_plan_destroy(plan)


def hyena_timing_begin(max_launches):
    _check(load().hyena_timing_begin(int(max_launches)), "hyena_timing_begin")


def hyena_timing_end():
    """Stop recording; returns ({kernel name: {launches, total_ms, min_ms,
    max_ms}}, dropped launches)."""
    lib = load()
    n = ctypes.c_int32()
    dropped = ctypes.c_int64()
    _check(lib.hyena_timing_end(ctypes.byref(n), ctypes.byref(dropped)), "hyena_timing_end")
    out = {}
    for i in range(n.value):
        name = ctypes.c_char_p()
        launches = ctypes.c_int64()
        tot, mn, mx = ctypes.c_double(), ctypes.c_double(), ctypes.c_double()
        _check(lib.hyena_timing_kernel(i, ctypes.byref(name), ctypes.byref(launches),
                                       ctypes.byref(tot), ctypes.byref(mn), ctypes.byref(mx)),
               "hyena_timing_kernel")
        out[name.value.decode()] = {"launches": launches.value, "total_ms": tot.value,
                                    "min_ms": mn.value, "max_ms": mx.value}
    return out, dropped.value


def hyena_timing_release():
    _check(load().hyena_timing_release(), "hyena_timing_release")


def _ref(x):
    """Address of a structure; the wrapper's packed bytes stand for themselves."""
    return ctypes.byref(x) if isinstance(x, ctypes.Structure) else x


def hyena_recurrence_create(B, N, heads, dk, dv, io_dtype=HYENA_F32, check=True):
    """Returns (status, plan handle or None)."""
    h = ctypes.c_void_p()
    st = load().hyena_recurrence_create(ctypes.byref(h), int(B), int(N), int(heads), int(dk), int(dv),
                                        int(io_dtype))
    if check:
        _check(st, "hyena_recurrence_create")
    return st, (h.value if st == HYENA_OK else None)


def hyena_recurrence_query(plan):
    """Returns (forward, backward) workspace bytes."""
    fwd, bwd = ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().hyena_recurrence_query(plan, ctypes.byref(fwd), ctypes.byref(bwd)),
           "hyena_recurrence_query")
    return fwd.value, bwd.value


def hyena_recurrence_forward(plan, inputs, o, final_state, workspace, stream=0):
    return load().hyena_recurrence_forward(plan, _ref(inputs), o, final_state, workspace, stream)


def hyena_recurrence_backward(plan, inputs, d_o, d_final, grads, workspace, stream=0):
    return load().hyena_recurrence_backward(plan, _ref(inputs), _ref(d_o), d_final, _ref(grads),
                                            workspace, stream)


def hyena_recurrence_step(plan, inputs, slots, n_slots, states, o, stream=0):
    return load().hyena_recurrence_step(plan, _ref(inputs), slots, int(n_slots), states, o, stream)


def hyena_recurrence_destroy(plan):
    return load().hyena_recurrence_destroy(plan)


def hyena_qk_norm_forward(op, q_out, k_out, stream=0):
    return load().hyena_qk_norm_forward(_ref(op), q_out, k_out, stream)


def hyena_qk_norm_scratch_bytes(op):
    """Returns (status, bytes)."""
    n = ctypes.c_size_t()
    st = load().hyena_qk_norm_scratch_bytes(_ref(op), ctypes.byref(n))
    return st, n.value


def hyena_qk_norm_backward(op, dq_out, dk_out, dq, dk, dq_weight, dk_weight, scratch, stream=0):
    return load().hyena_qk_norm_backward(_ref(op), _ref(dq_out), _ref(dk_out), dq, dk, dq_weight,
                                         dk_weight, scratch, stream)


# --------------------------------------------------------------------------
# torch convenience wrapper (device memory and stream plumbing only)
# --------------------------------------------------------------------------

class Plan:
    """One plan plus its workspace on a torch device.

    ``dims`` is ``(N,)`` for sequences, ``(X, Y)`` or ``(X, Y, Z)`` for grids.  Tensors are
    float32 or bfloat16 (io), channels last; see include/hyena.h for layouts.
    """

    def __init__(self, B, d, order, dims, io_dtype=HYENA_F32, spectrum_dtype=None,
                 path=HYENA_PATH_AUTO, device="cuda", circular=False):
        import torch
        self.torch = torch
        N = 1
        for v in dims:
            N *= int(v)
        self.B, self.N, self.d, self.order, self.dims = int(B), N, int(d), int(order), tuple(dims)
        self.io_dtype = io_dtype
        if spectrum_dtype is None:  # binary16 io takes a float32 spectrum
            spectrum_dtype = HYENA_F32 if io_dtype == HYENA_F16 else io_dtype
        self.spectrum_dtype = spectrum_dtype
        self.circular = bool(circular)
        _, self.handle = hyena_plan_create(B, N, d, order, dims, io_dtype, self.spectrum_dtype,
                                           path, flags=HYENA_FLAG_CIRCULAR if circular else 0)
        self.spectrum_bytes, self.workspace_bytes, self.path = hyena_plan_query(self.handle)
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self.workspace = torch.empty(max(self.workspace_bytes, 256), dtype=torch.uint8,
                                     device=self.device)
        _check(hyena_workspace_init(self.handle, self.workspace.data_ptr(), self.stream()),
               "hyena_workspace_init")

    def stream(self):
        return self.torch.cuda.current_stream(self.device).cuda_stream

    @property
    def torch_io_dtype(self):
        return {HYENA_F32: self.torch.float32, HYENA_BF16: self.torch.bfloat16,
                HYENA_F16: self.torch.float16}[self.io_dtype]

    # ------------------------------------------------------------------
    # argument checks: every tensor is checked (dtype, contiguity, device,
    # shape or byte count) before anything is enqueued, so an undersized or
    # misplaced buffer raises ValueError instead of reaching a kernel
    # ------------------------------------------------------------------
    @property
    def act_shape(self):
        """Shape of u, the gates and y: [B, *dims, d]."""
        return (self.B,) + self.dims + (self.d,)

    @property
    def filter_shape(self):
        """Shape of the taps h: [order, d, N] or [order, d, 2X-1, 2Y-1(, 2Z-1)]."""
        if len(self.dims) == 1:
            return (self.order, self.d, self.N)
        return (self.order, self.d) + tuple(2 * int(s) - 1 for s in self.dims)

    def _tensor(self, t, name, dtype, shape=None, min_bytes=None):
        torch = self.torch
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{name} must be a torch tensor")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}, got {t.device}")
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
        if min_bytes is not None and t.numel() * t.element_size() < min_bytes:
            raise ValueError(f"{name} must hold at least {min_bytes} bytes, got "
                             f"{t.numel() * t.element_size()}")
        return t

    def _io(self, t, name, shape=None):
        return self._tensor(t, name, self.torch_io_dtype,
                            self.act_shape if shape is None else shape)

    def _spec(self, H, name="H"):
        return self._tensor(H, name, self.torch.uint8, min_bytes=self.spectrum_bytes)

    def _f32(self, t, name, shape):
        return self._tensor(t, name, self.torch.float32, shape)

    def _feedthrough(self, D):
        """D: float32 [order, d] ([d] is accepted for order 1)."""
        shape = (self.order, self.d)
        if self.order == 1 and isinstance(D, self.torch.Tensor) and D.dim() == 1:
            shape = (self.d,)
        return self._f32(D, "D", shape)

    def spectrum(self, h, H=None):
        h = self._io(h, "h", self.filter_shape)
        if H is None:
            H = self.torch.empty(self.spectrum_bytes, dtype=self.torch.uint8, device=self.device)
        self._spec(H)
        _check(hyena_filter_spectrum(self.handle, h.data_ptr(), H.data_ptr(),
                                     self.workspace.data_ptr(), self.stream()),
               "hyena_filter_spectrum")
        return H

    def spectrum_implicit(self, W1, b1, W2, b2, W3, b3, alpha, omega, H=None):
        """Spectrum from an implicit filter; weights are float32 device tensors
        W1 [hidden, 2K+1], b1 [hidden], W2 [hidden, hidden], b2 [hidden],
        W3 [order*d, hidden], b3 [order*d], alpha [order, d]."""
        ws = [W1, b1, W2, b2, W3, b3, alpha]
        if not isinstance(W1, self.torch.Tensor) or W1.dim() != 2:
            raise ValueError("W1 must be a 2-D tensor [hidden, 2K+1]")
        hidden, m = (int(x) for x in W1.shape)
        if m % 2 != 1:
            raise ValueError(f"W1 must have an odd width 2K+1, got {m}")
        nd = self.order * self.d
        for t, name, shape in ((W1, "W1", (hidden, m)), (b1, "b1", (hidden,)),
                               (W2, "W2", (hidden, hidden)), (b2, "b2", (hidden,)),
                               (W3, "W3", (nd, hidden)), (b3, "b3", (nd,)),
                               (alpha, "alpha", (self.order, self.d))):
            self._f32(t, name, shape)
        f = ImplicitFilter((m - 1) // 2, hidden, float(omega), *[t.data_ptr() for t in ws])
        st, nbytes = hyena_implicit_scratch_bytes(self.handle, hidden)
        _check(st, "hyena_implicit_scratch_bytes")
        # kept with the plan and reused, like the workspace (calls of one plan
        # must not run concurrently on different streams)
        scratch = getattr(self, "_implicit_scratch", None)
        if scratch is None or scratch.numel() < nbytes:
            scratch = self._implicit_scratch = None
            scratch = self.torch.empty(max(nbytes, 256), dtype=self.torch.uint8, device=self.device)
        if H is None:
            H = self.torch.empty(self.spectrum_bytes, dtype=self.torch.uint8, device=self.device)
        self._spec(H)
        _check(hyena_filter_spectrum_implicit(self.handle, f, H.data_ptr(),
                                              self.workspace.data_ptr(), scratch.data_ptr(),
                                              self.stream()),
               "hyena_filter_spectrum_implicit")
        self._implicit_scratch = scratch
        return H

    def forward(self, u, gates, H, D, y=None):
        u = self._io(u, "u")
        gates = list(gates)
        if len(gates) != self.order:
            raise ValueError(f"need one gate per filter ({self.order}), got {len(gates)}")
        gates = [self._io(g, f"gate {n}") for n, g in enumerate(gates)]
        self._spec(H)
        self._feedthrough(D)
        if y is None:
            y = self.torch.empty_like(u)
        self._io(y, "y")
        _check(hyena_forward(self.handle, u.data_ptr(), [g.data_ptr() for g in gates],
                             H.data_ptr(), D.data_ptr(), y.data_ptr(), self.workspace.data_ptr(),
                             self.stream()),
               "hyena_forward")
        return y

    def nd_mixer(self, q, k, v, short_w, short_b, H, D, y=None):
        """HyenaND mixer (ndims = 2 or 3, order 1): y = SiLU(sc(v)) . (K * z + D z),
        z = sc(q) . SiLU(sc(k)); short_w float32 [3, d, 3, 3] (2D) or [3, d, 3, 3, 3]
        (3D), short_b [3, d] or None."""
        q, k, v = self._io(q, "q"), self._io(k, "k"), self._io(v, "v")
        taps = (3,) * len(self.dims)
        self._f32(short_w, "short_w", (3, self.d) + taps)
        if short_b is not None:
            self._f32(short_b, "short_b", (3, self.d))
        self._feedthrough(D)
        self._spec(H)
        if y is None:
            y = self.torch.empty_like(q)
        self._io(y, "y")
        m = NdMixer(q.data_ptr(), k.data_ptr(), v.data_ptr(), short_w.data_ptr(),
                    short_b.data_ptr() if short_b is not None else None)
        _check(hyena_nd_mixer_forward(self.handle, m, H.data_ptr(), D.data_ptr(), y.data_ptr(),
                                      self.workspace.data_ptr(), self.stream()),
               "hyena_nd_mixer_forward")
        return y

    def export_spectrum(self, H):
        self._spec(H)
        if len(self.dims) == 1:
            M = 1
            while M < (self.N if self.circular else 2 * self.N):
                M *= 2
            shape = (self.order, self.d, M // 2 + 1, 2)
        elif len(self.dims) == 2:
            X, Y = self.dims
            shape = (self.order, self.d, 2 * X, Y + 1, 2)
        else:
            X, Y, Z = self.dims
            shape = (self.order, self.d, 2 * X, 2 * Y, Z + 1, 2)
        out = self.torch.zeros(shape, dtype=self.torch.float32, device=self.device)
        _check(hyena_spectrum_export(self.handle, H.data_ptr(), out.data_ptr(), self.stream()),
               "hyena_spectrum_export")
        return out

    def __del__(self):
        try:
            if getattr(self, "handle", None):
                hyena_plan_destroy(self.handle)
                self.handle = None
        except Exception:
            pass


class _Mixer:
    """Checks and stream plumbing shared by the operators on q, k and v.

    A call's structures are packed in one go (their layouts are those of View,
    RecurrenceInputs and QkNorm): a decoded token's kernel takes a few
    microseconds, and so may not its arguments."""

    def _place(self, io_dtype, device):
        import torch
        self.torch = torch
        dtypes = {HYENA_F32: torch.float32, HYENA_BF16: torch.bfloat16, HYENA_F16: torch.float16}
        if io_dtype not in dtypes:
            raise ValueError(f"unknown io dtype {io_dtype}")
        self.io_dtype, self.dtype = io_dtype, dtypes[io_dtype]
        dev = torch.device(device)
        if dev.type != "cuda":
            raise ValueError(f"the device must be a GPU, got {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device, self.index = dev, dev.index
        self._lib = load()
        self._raw_stream, self._current = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        self._first_stream = self._stream()

    def _stream(self):
        return self._raw_stream(self.index)

    def _call(self, where, fn, *args):
        # launches go to the current device; a plan of another one makes its own current
        if self._current() == self.index:
            st = fn(*args)
        else:
            with self.torch.cuda.device(self.device):
                st = fn(*args)
        if st != HYENA_OK:
            _check(st, where)

    def _keep(self, buffer, stream):
        """Address of a buffer the plan owns.  It may be used on a stream other
        than the one it was allocated on: its memory is not given out again
        before that stream's work is done."""
        if buffer is None:
            return None
        if stream != self._first_stream:
            buffer.record_stream(self.torch.cuda.current_stream(self.device))
        return buffer.data_ptr()

    def _fits(self, t, shape, dtype):
        return isinstance(t, self.torch.Tensor) and t.dtype == dtype and t.device == self.device and t.shape == shape

    def _check_tensor(self, t, name, shape, dtype):
        if not isinstance(t, self.torch.Tensor):
            raise ValueError(f"{name} must be a torch tensor")
        if t.dtype != dtype:
            raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
        if t.device != self.device:
            raise ValueError(f"{name} must be on {self.device}, got {t.device}")
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")

    def _dense(self, t, name, shape, dtype):
        """Address of a contiguous tensor, 0 for None."""
        if t is None:
            return 0
        if not self._fits(t, shape, dtype):
            self._check_tensor(t, name, shape, dtype)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def _view(self, t, name, shape, dtype):
        """Address and strides (batch, token, head) of a [B, N, heads, width] or [B, N, heads]
        tensor."""
        if not self._fits(t, shape, dtype):
            self._check_tensor(t, name, shape, dtype)
        st = t.stride()
        if len(shape) == 4 and st[3] != 1 and shape[3] > 1:
            raise ValueError(f"the last axis of {name} must be contiguous")
        # torch gives axes of one element any stride
        return (t.data_ptr(), st[0] if shape[0] > 1 else 0, st[1] if shape[1] > 1 else 0,
                st[2] if shape[2] > 1 else 0)

    def _token_view(self, t, name, shape, dtype):
        """The same of one token per row: [B, heads, width] or [B, heads]."""
        if not self._fits(t, shape, dtype):
            self._check_tensor(t, name, shape, dtype)
        st = t.stride()
        if len(shape) == 3 and st[2] != 1 and shape[2] > 1:
            raise ValueError(f"the last axis of {name} must be contiguous")
        return (t.data_ptr(), st[0] if shape[0] > 1 else 0, 0, st[1] if shape[1] > 1 else 0)

    def _out(self, out, name, shape, dtype, like=None):
        """An output: the caller's, checked, or a new one (like a checked input of its shape and type,
        which is made sooner)."""
        if out is None:
            if like is not None:
                return self.torch.empty_like(like, memory_format=self.torch.contiguous_format)
            return self.torch.empty(shape, dtype=dtype, device=self.device)
        self._dense(out, name, shape, dtype)
        return out


_PACK_VIEW = struct.Struct("P3q").pack
_PACK_RECURRENCE = struct.Struct("P3q" * 4 + "PPf4x").pack
_PACK_GRADS = struct.Struct("5P").pack
_PACK_QK_NORM = struct.Struct("5q3i4xq2f4Pq" + "P3q" * 2).pack


class Recurrence(_Mixer):
    """Gated linear recurrence S_t = exp(g_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t
    for rows of N tokens (see include/hyena.h for shapes, masks and precision).

    q, k: [B, N, heads, dk], v: [B, N, heads, dv] in the io dtype, g: float32
    [B, N, heads] (log decays, at most 0); views are taken as they are as long as the last
    axis of q, k and v is contiguous.  States are float32 [B, heads, dk, dv].
    ``training`` allocates the backward pass's workspace.  Calls of one plan
    share its workspace and must not run concurrently on different streams.
    Outputs carry no autograd history: ``backward`` is called by the caller.
    """

    def __init__(self, B, N, heads, dk, dv, io_dtype=HYENA_F32, training=False, device="cuda"):
        self._place(io_dtype, device)
        self.B, self.N, self.heads, self.dk, self.dv = (int(x) for x in (B, N, heads, dk, dv))
        _, self.handle = hyena_recurrence_create(B, N, heads, dk, dv, io_dtype)
        self.forward_bytes, self.backward_bytes = hyena_recurrence_query(self.handle)
        self.training = bool(training)
        n = max(self.forward_bytes, self.backward_bytes if training else 0)
        self.workspace = self.torch.empty(n, dtype=self.torch.uint8, device=self.device) if n else None

    @property
    def state_shape(self):
        return (self.B, self.heads, self.dk, self.dv)

    def _inputs(self, q, k, v, g, scale, state=None, lengths=None):
        torch = self.torch
        B, N, H = self.B, self.N, self.heads
        return _PACK_RECURRENCE(
            *self._view(q, "q", (B, N, H, self.dk), self.dtype), *self._view(k, "k", (B, N, H, self.dk), self.dtype),
            *self._view(v, "v", (B, N, H, self.dv), self.dtype), *self._view(g, "g", (B, N, H), torch.float32),
            self._dense(state, "state", self.state_shape, torch.float32),
            self._dense(lengths, "lengths", (B,), torch.int32), self.dk ** -0.5 if scale is None else scale)

    def forward(self, q, k, v, g, scale=None, state=None, lengths=None, return_state=False, o=None,
                final_state=None):
        """(o, final state or None).  scale: 1 / sqrt(dk) by default.  state: the state before
        token 0.  lengths: int32 [B], tokens per row (the others' o is 0)."""
        x = self._inputs(q, k, v, g, scale, state, lengths)
        o = self._out(o, "o", (self.B, self.N, self.heads, self.dv), self.dtype, v)
        if return_state or final_state is not None:
            final_state = self._out(final_state, "final_state", self.state_shape, self.torch.float32)
        stream = self._stream()
        self._call("hyena_recurrence_forward", self._lib.hyena_recurrence_forward, self.handle, x, o.data_ptr(),
                   final_state.data_ptr() if final_state is not None else None,
                   self._keep(self.workspace, stream), stream)
        return o, final_state

    def backward(self, d_o, q, k, v, g, scale=None, state=None, lengths=None, d_final=None):
        """(dq, dk, dv, dg, d_state) from the gradients of o and (or None) of the final state;
        d_state is None without a state."""
        torch = self.torch
        if not self.training:
            raise ValueError("backward needs a plan made with training=True")
        x = self._inputs(q, k, v, g, scale, state, lengths)
        rows = (self.B, self.N, self.heads)
        d = _PACK_VIEW(*self._view(d_o, "d_o", rows + (self.dv,), self.dtype))
        df = self._dense(d_final, "d_final", self.state_shape, torch.float32)
        new = lambda shape, dt=self.dtype: torch.empty(shape, dtype=dt, device=self.device)  # noqa: E731
        dq, dk, dv = new(rows + (self.dk,)), new(rows + (self.dk,)), new(rows + (self.dv,))
        dg = new(rows, torch.float32)
        ds = new(self.state_shape, torch.float32) if state is not None else None
        grads = _PACK_GRADS(dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(),
                            ds.data_ptr() if ds is not None else 0)
        stream = self._stream()
        self._call("hyena_recurrence_backward", self._lib.hyena_recurrence_backward, self.handle, x, d, df, grads,
                   self._keep(self.workspace, stream), stream)
        return dq, dk, dv, dg, ds

    def step(self, q, k, v, g, states, scale=None, slots=None, o=None):
        """One token per row: q, k [B, heads, dk], v [B, heads, dv], g [B, heads].  Updates
        states[slots] (float32 [n, heads, dk, dv], slots int32 [B], row b by default) in place and
        returns o [B, heads, dv].  Rows with a slot outside the table take no part (o = 0); the
        other slots have to differ."""
        torch = self.torch
        B, H = self.B, self.heads
        x = _PACK_RECURRENCE(
            *self._token_view(q, "q", (B, H, self.dk), self.dtype), *self._token_view(k, "k", (B, H, self.dk), self.dtype),
            *self._token_view(v, "v", (B, H, self.dv), self.dtype), *self._token_view(g, "g", (B, H), torch.float32),
            0, 0, self.dk ** -0.5 if scale is None else scale)
        n = states.shape[0] if isinstance(states, self.torch.Tensor) and states.dim() == 4 else 0
        table = self._dense(states, "states", (n, H, self.dk, self.dv), torch.float32)
        if not table:
            raise ValueError("states must be a torch tensor of at least one state")
        at = self._dense(slots, "slots", (B,), torch.int32)
        o = self._out(o, "o", (B, H, self.dv), self.dtype, v)
        self._call("hyena_recurrence_step", self._lib.hyena_recurrence_step, self.handle, x, at, n, table, o.data_ptr(),
                   self._stream())
        return o

    def __del__(self):
        try:
            if getattr(self, "handle", None):
                hyena_recurrence_destroy(self.handle)
                self.handle = None
        except Exception:
            pass


def rotary_frequencies(rotary_dim, base=10000.0, stretch=1.0, device="cuda"):
    """float64 [rotary_dim / 2]: base^(-2 i / rotary_dim) / stretch.  stretch > 1 spreads the
    positions of a longer context over the trained range; any other scaling is a table of the
    caller's own."""
    import torch
    # made on the host: the copy is done before this returns, so any stream may read it
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    return (base ** (-i / max(rotary_dim, 1)) / stretch).to(device)


class QKNorm(_Mixer):
    """Norms of queries and keys per head with the position rotation in the same pass.

    q: [B, N, q_heads, D], k: [B, N, k_heads, D] in the io dtype (views; the last axis
    contiguous); norm "rms", "l2" or "none"; weights float32 [D] or None.  The first
    ``rotary_dim`` channels are rotated (D by default, 0: none), pairs (i, i + rotary_dim / 2)
    in the "half" layout and (2i, 2i + 1) in the "interleaved" one, by position * freqs[i]
    (float64, by default ``rotary_frequencies(rotary_dim)``); sines and cosines are multiplied
    by ``rotary_scale``.  Outputs carry no autograd history: ``backward`` is called by the caller.
    """

    _NORMS = {"none": HYENA_NORM_NONE, "rms": HYENA_NORM_RMS, "l2": HYENA_NORM_L2}
    _LAYOUTS = {"half": HYENA_ROTARY_HALF, "interleaved": HYENA_ROTARY_INTERLEAVED}

    def __init__(self, B, N, q_heads, k_heads, D, io_dtype=HYENA_F32, norm="rms", rotary_dim=None,
                 layout="half", eps=1e-6, freqs=None, rotary_scale=1.0, device="cuda"):
        self._place(io_dtype, device)
        if norm not in self._NORMS:
            raise ValueError(f"norm must be one of {sorted(self._NORMS)}, got {norm!r}")
        if layout not in self._LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(self._LAYOUTS)}, got {layout!r}")
        self.B, self.N, self.q_heads, self.k_heads, self.D = (int(x) for x in (B, N, q_heads, k_heads, D))
        self.rotary_dim = int(D if rotary_dim is None else rotary_dim)
        if self.rotary_dim % 2 or not 0 <= self.rotary_dim <= self.D:
            raise ValueError(f"rotary_dim must be even and in 0..{self.D}, got {self.rotary_dim}")
        if freqs is None:
            freqs = rotary_frequencies(self.rotary_dim, device=self.device)
        self._dense(freqs, "freqs", (self.rotary_dim // 2,), self.torch.float64)
        self.norm, self.layout, self.eps, self.freqs = norm, layout, float(eps), freqs
        self.rotary_scale = float(rotary_scale)
        st, n = hyena_qk_norm_scratch_bytes(self._op((0, 0, 0, 0), (0, 0, 0, 0)))
        _check(st, "hyena_qk_norm_scratch_bytes")
        self.scratch_bytes = n

    def _op(self, q, k, q_weight=0, k_weight=0, positions=0, offset=0):
        return _PACK_QK_NORM(self.B, self.N, self.q_heads, self.k_heads, self.D, self.io_dtype,
                             self._NORMS[self.norm], self._LAYOUTS[self.layout], self.rotary_dim, self.eps,
                             self.rotary_scale, self.freqs.data_ptr() if self.rotary_dim else 0,
                             q_weight, k_weight, positions, offset, *q, *k)

    def _describe(self, q, k, q_weight, k_weight, positions, offset):
        torch = self.torch
        return self._op(self._view(q, "q", (self.B, self.N, self.q_heads, self.D), self.dtype),
                        self._view(k, "k", (self.B, self.N, self.k_heads, self.D), self.dtype),
                        self._dense(q_weight, "q_weight", (self.D,), torch.float32),
                        self._dense(k_weight, "k_weight", (self.D,), torch.float32),
                        self._dense(positions, "positions", (self.B, self.N), torch.int32), offset)

    def forward(self, q, k, q_weight=None, k_weight=None, positions=None, offset=0, q_out=None,
                k_out=None):
        """(normed and rotated q, k), dense.  positions: int32 [B, N], or token n is at
        offset + n."""
        op = self._describe(q, k, q_weight, k_weight, positions, offset)
        q_out = self._out(q_out, "q_out", (self.B, self.N, self.q_heads, self.D), self.dtype, q)
        k_out = self._out(k_out, "k_out", (self.B, self.N, self.k_heads, self.D), self.dtype, k)
        stream = self._stream()
        self._keep(self.freqs, stream)
        self._call("hyena_qk_norm_forward", self._lib.hyena_qk_norm_forward, op, q_out.data_ptr(), k_out.data_ptr(), stream)
        return q_out, k_out

    def backward(self, dq_out, dk_out, q, k, q_weight=None, k_weight=None, positions=None, offset=0):
        """(dq, dk, dq_weight, dk_weight) from the gradients of forward's outputs; a weight that is
        None has no gradient."""
        torch = self.torch
        op = self._describe(q, k, q_weight, k_weight, positions, offset)
        qs, ks = (self.B, self.N, self.q_heads, self.D), (self.B, self.N, self.k_heads, self.D)
        dqo = _PACK_VIEW(*self._view(dq_out, "dq_out", qs, self.dtype))
        dko = _PACK_VIEW(*self._view(dk_out, "dk_out", ks, self.dtype))
        new = lambda shape, dt=self.dtype: torch.empty(shape, dtype=dt, device=self.device)  # noqa: E731
        dq, dk = new(qs), new(ks)
        has = [w is not None and self.norm != "none" for w in (q_weight, k_weight)]
        dqw, dkw = (new((self.D,), torch.float32) if h else None for h in has)
        scratch = new((self.scratch_bytes,), torch.uint8) if any(has) else None
        stream = self._stream()
        self._keep(self.freqs, stream)
        ptr = lambda t: t.data_ptr() if t is not None else None  # noqa: E731
        self._call("hyena_qk_norm_backward", self._lib.hyena_qk_norm_backward, op, dqo, dko, dq.data_ptr(), dk.data_ptr(),
                   ptr(dqw), ptr(dkw), ptr(scratch), stream)
        return dq, dk, dqw, dkw
