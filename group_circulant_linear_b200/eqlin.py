"""Thin Python binding of the C ABI in ``include/eqlin.h`` (ctypes).

The functions carry the ABI's names (``eqlin_create`` -> ``create`` and so on)
and do argument marshalling only: they check that tensors are contiguous CUDA
tensors of the handle's dtype and shape, then pass raw device pointers and the
current CUDA stream.  Every step of the layer runs in ``libeqlin.so``.  There
is no fallback: if the library is missing or the call fails, this module
raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libeqlin.so")

F32, F16, BF16 = 0, 1, 2
CYCLIC, DIHEDRAL = 0, 1
_GROUPS = {"cyclic": CYCLIC, "dihedral": DIHEDRAL}
_DT = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
_TORCH_DT = {v: k for k, v in _DT.items()}
_NAMES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}

STATUS = {0: "EQLIN_OK", -1: "EQLIN_ERR_INVALID_ARG", -2: "EQLIN_ERR_UNSUPPORTED",
          -3: "EQLIN_ERR_MISALIGNED", -4: "EQLIN_ERR_CUDA", -5: "EQLIN_ERR_NO_WEIGHTS",
          -6: "EQLIN_ERR_TIMEOUT", -7: "EQLIN_ERR_OOM"}

# Every entry point include/eqlin.h declares, with its ctypes signature.
_vp, _i64, _int, _u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint32
_f32 = ctypes.c_float


class AttentionDesc(ctypes.Structure):
    """eqlin_attention_t."""
    _fields_ = [("tokens", _i64), ("heads", _i64), ("kv_heads", _i64), ("head_dim", _i64),
                ("q_stride", _i64), ("k_stride", _i64), ("v_stride", _i64), ("o_stride", _i64),
                ("docs", _i64), ("offsets", _vp), ("max_len", _i64), ("pos", _vp), ("slopes", _vp),
                ("axes", _int), ("scale", _f32), ("cap", _f32), ("err", _vp), ("wait_limit", _u32)]


SIGNATURES = {
    "eqlin_create": ([_int, _i64, _i64, _int, ctypes.POINTER(_vp)], _int),
    "eqlin_create_group": ([_int, _int, _i64, _i64, _int, ctypes.POINTER(_vp)], _int),
    "eqlin_set_weights": ([_vp, _vp, _vp, _vp], _int),
    "eqlin_forward": ([_vp, _vp, _vp, _i64, _vp], _int),
    "eqlin_forward_gauss": ([_vp, _vp, _vp, _i64, _vp], _int),
    "eqlin_backward_dx": ([_vp, _vp, _vp, _i64, _vp], _int),
    "eqlin_backward_dw": ([_vp, _vp, _vp, _vp, _vp, _i64, _vp], _int),
    "eqlin_get_error": ([_vp], _int),
    "eqlin_error_detail": ([_vp, ctypes.POINTER(ctypes.c_uint32)], _int),
    "eqlin_set_wait_limit": ([_vp, _u32], _int),
    "eqlin_set_tail_split": ([_vp, _int], _int),
    "eqlin_backend_name": ([_vp], ctypes.c_char_p),
    "eqlin_status_string": ([_int], ctypes.c_char_p),
    "eqlin_launch_count": ([], ctypes.c_uint64),
    "eqlin_backward_dw_noalloc": ([_int, _i64, _i64, _int, _vp, _vp, _vp, _vp, _i64, _vp], _int),
    "eqlin_spectra_ld": ([_i64], _i64),
    "eqlin_forward_stash": ([_vp, _vp, _vp, _vp, _i64, _vp], _int),
    "eqlin_backward_dx_stash": ([_vp, _vp, _vp, _vp, _i64, _vp], _int),
    "eqlin_backward_dw_spectra": ([_vp, _vp, _vp, _vp, _vp, _i64, _vp], _int),
    "eqlin_backward": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp], _int),
    "eqlin_destroy": ([_vp], None),
    "eqlin_norm_forward": ([_int, _i64, _int, _vp, _vp, _vp, _vp, _f32, _vp, _vp, _vp, _vp, _i64, _vp], _int),
    "eqlin_norm_workspace_bytes": ([_int, _i64, _i64], _i64),
    "eqlin_norm_backward": ([_int, _i64, _int, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _vp],
                            _int),
    "eqlin_rope_create": ([_int, _i64, _int, ctypes.POINTER(_i64), ctypes.POINTER(ctypes.c_double),
                           ctypes.POINTER(_vp)], _int),
    "eqlin_rope_destroy": ([_vp], None),
    "eqlin_rope_apply": ([_vp, _int, _vp, _vp, _i64, _vp, _i64, _i64, _int, _i64, _vp], _int),
    "eqlin_attention_forward": ([ctypes.POINTER(AttentionDesc), _int, _vp, _vp, _vp, _vp, _vp, _vp], _int),
    "eqlin_attention_backward": ([ctypes.POINTER(AttentionDesc), _int, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                  _vp, _i64, _vp, _i64, _vp, _vp], _int),
}

_lib = None


class EqlinError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib().eqlin_status_string(status).decode() if _lib else str(status)
        super().__init__(f"{where}: {STATUS.get(status, status)} ({msg})")


def lib():
    """Load libeqlin.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing; build it with "
                               "`python -m group_circulant_linear_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def _check(status: int, where: str):
    if status != 0:
        raise EqlinError(status, where)


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _dev_ptr(t: torch.Tensor, dtype, shape, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return ctypes.c_void_p(t.data_ptr())


class Handle:
    """An eqlin_t plus the layer shape it was created for.

    ``T`` is the group order (the length of the group axis).  For
    ``group="dihedral"`` pass ``m`` (D_m, order 2m) and T = 2m, or T = None."""

    def __init__(self, T, Cp: int, Dp: int, dtype, group="cyclic", m: int | None = None):
        if isinstance(dtype, str):
            dtype = _NAMES[dtype]
        self.group = _GROUPS[group] if isinstance(group, str) else int(group)
        if self.group == DIHEDRAL:
            if m is None:
                m = int(T) // 2
            self.m = int(m)
            T = 2 * self.m
        else:
            self.m = int(T)
        self.T, self.Cp, self.Dp, self.dtype = int(T), int(Cp), int(Dp), dtype
        out = ctypes.c_void_p()
        _check(lib().eqlin_create_group(self.group, self.m, self.Cp, self.Dp, _DT[dtype], ctypes.byref(out)),
               "eqlin_create_group")
        self._h = out

    @property
    def ptr(self):
        return self._h

    def close(self):
        if self._h:
            lib().eqlin_destroy(self._h)
            self._h = ctypes.c_void_p()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def backend(self) -> str:
        return lib().eqlin_backend_name(self._h).decode()

    def __copy__(self):
        raise TypeError("a Handle owns device buffers; use copy.deepcopy for a new handle of the same shape")

    def __deepcopy__(self, memo):
        # a new handle of the same shape; it holds no weights until set_weights
        return Handle(self.T, self.Cp, self.Dp, self.dtype, group=self.group, m=self.m)


# ------------------------------------------------------------------ the ABI

def create(T: int, Cp: int, Dp: int, dtype) -> Handle:
    return Handle(T, Cp, Dp, dtype)


def create_group(group, m: int, Cp: int, Dp: int, dtype) -> Handle:
    """A layer over the cyclic group Z_m or the dihedral group D_m (order 2m)."""
    g = _GROUPS[group] if isinstance(group, str) else int(group)
    return Handle(m if g == CYCLIC else 2 * m, Cp, Dp, dtype, group=g, m=m)


def set_weights(h: Handle, W: torch.Tensor, b: torch.Tensor | None = None, stream=None):
    pw = _dev_ptr(W, h.dtype, (h.Dp, h.Cp, h.T), "W")
    pb = None if b is None else _dev_ptr(b, h.dtype, (h.Dp,), "b")
    _check(lib().eqlin_set_weights(h.ptr, pw, pb, _stream(stream)), "eqlin_set_weights")


def forward(h: Handle, x: torch.Tensor, y: torch.Tensor, stream=None):
    N = x.shape[0]
    px = _dev_ptr(x, h.dtype, (N, h.Cp * h.T), "x")
    py = _dev_ptr(y, h.dtype, (N, h.Dp * h.T), "y")
    _check(lib().eqlin_forward(h.ptr, px, py, N, _stream(stream)), "eqlin_forward")


def forward_gauss(h: Handle, x: torch.Tensor, y: torch.Tensor, stream=None):
    """eqlin_forward with the complex products as three real GEMMs (p4 only)."""
    N = x.shape[0]
    px = _dev_ptr(x, h.dtype, (N, h.Cp * h.T), "x")
    py = _dev_ptr(y, h.dtype, (N, h.Dp * h.T), "y")
    _check(lib().eqlin_forward_gauss(h.ptr, px, py, N, _stream(stream)), "eqlin_forward_gauss")


def backward_dx(h: Handle, gy: torch.Tensor, dx: torch.Tensor, stream=None):
    N = gy.shape[0]
    pg = _dev_ptr(gy, h.dtype, (N, h.Dp * h.T), "gy")
    pd = _dev_ptr(dx, h.dtype, (N, h.Cp * h.T), "dx")
    _check(lib().eqlin_backward_dx(h.ptr, pg, pd, N, _stream(stream)), "eqlin_backward_dx")


def backward_dw(h: Handle, x: torch.Tensor, gy: torch.Tensor, dW: torch.Tensor,
                db: torch.Tensor | None = None, stream=None):
    N = x.shape[0]
    px = _dev_ptr(x, h.dtype, (N, h.Cp * h.T), "x")
    pg = _dev_ptr(gy, h.dtype, (N, h.Dp * h.T), "gy")
    pw = _dev_ptr(dW, torch.float32, (h.Dp, h.Cp, h.T), "dW")
    pb = None if db is None else _dev_ptr(db, torch.float32, (h.Dp,), "db")
    _check(lib().eqlin_backward_dw(h.ptr, px, pg, pw, pb, N, _stream(stream)), "eqlin_backward_dw")


def spectra_ld(N: int) -> int:
    """Row pitch (tokens) of a spectra buffer for N tokens."""
    return int(lib().eqlin_spectra_ld(int(N)))


def spectra_shape(h: Handle, which: str, N: int) -> tuple:
    """Shape of the spectra buffer of the input ("x": [T, C', ld]) or of the
    output gradient ("gy": [T, D', ld]) for N tokens."""
    ch = {"x": h.Cp, "gy": h.Dp}[which]
    return (h.T, ch, spectra_ld(N))


def empty_spectra(h: Handle, which: str, N: int, device=None) -> torch.Tensor:
    return torch.empty(spectra_shape(h, which, N), dtype=h.dtype, device=device or "cuda")


def forward_stash(h: Handle, x: torch.Tensor, y: torch.Tensor, xs: torch.Tensor, stream=None):
    """Forward that also writes X = DFT(x) into xs [T, C', ld]."""
    N = x.shape[0]
    px = _dev_ptr(x, h.dtype, (N, h.Cp * h.T), "x")
    py = _dev_ptr(y, h.dtype, (N, h.Dp * h.T), "y")
    ps = _dev_ptr(xs, h.dtype, spectra_shape(h, "x", N), "xs")
    _check(lib().eqlin_forward_stash(h.ptr, px, py, ps, N, _stream(stream)), "eqlin_forward_stash")


def backward_dx_stash(h: Handle, gy: torch.Tensor, dx: torch.Tensor, gs: torch.Tensor, stream=None):
    """Input gradient that also writes G = DFT(gy) into gs [T, D', ld]."""
    N = gy.shape[0]
    pg = _dev_ptr(gy, h.dtype, (N, h.Dp * h.T), "gy")
    pd = _dev_ptr(dx, h.dtype, (N, h.Cp * h.T), "dx")
    ps = _dev_ptr(gs, h.dtype, spectra_shape(h, "gy", N), "gs")
    _check(lib().eqlin_backward_dx_stash(h.ptr, pg, pd, ps, N, _stream(stream)), "eqlin_backward_dx_stash")


def backward_dw_spectra(h: Handle, xs: torch.Tensor, gs: torch.Tensor, N: int, dW: torch.Tensor,
                        db: torch.Tensor | None = None, stream=None):
    """dW, db from the spectra of the same N tokens."""
    pxs = _dev_ptr(xs, h.dtype, spectra_shape(h, "x", N), "xs")
    pgs = _dev_ptr(gs, h.dtype, spectra_shape(h, "gy", N), "gs")
    pw = _dev_ptr(dW, torch.float32, (h.Dp, h.Cp, h.T), "dW")
    pb = None if db is None else _dev_ptr(db, torch.float32, (h.Dp,), "db")
    _check(lib().eqlin_backward_dw_spectra(h.ptr, pxs, pgs, pw, pb, int(N), _stream(stream)),
           "eqlin_backward_dw_spectra")


def backward(h: Handle, gy: torch.Tensor, xs: torch.Tensor, dx: torch.Tensor, gs: torch.Tensor,
             dW: torch.Tensor, db: torch.Tensor | None = None, stream=None):
    """The whole backward (dx, dW, db) given the forward's stash xs; writes gs."""
    N = gy.shape[0]
    pg = _dev_ptr(gy, h.dtype, (N, h.Dp * h.T), "gy")
    pxs = _dev_ptr(xs, h.dtype, spectra_shape(h, "x", N), "xs")
    pd = _dev_ptr(dx, h.dtype, (N, h.Cp * h.T), "dx")
    pgs = _dev_ptr(gs, h.dtype, spectra_shape(h, "gy", N), "gs")
    pw = _dev_ptr(dW, torch.float32, (h.Dp, h.Cp, h.T), "dW")
    pb = None if db is None else _dev_ptr(db, torch.float32, (h.Dp,), "db")
    _check(lib().eqlin_backward(h.ptr, pg, pxs, pd, pgs, pw, pb, N, _stream(stream)), "eqlin_backward")


def backward_dw_noalloc(T: int, x: torch.Tensor, gy: torch.Tensor, dW: torch.Tensor,
                        db: torch.Tensor | None = None, stream=None):
    """dW/db with no handle and no device allocation (see eqlin_backward_dw_noalloc)."""
    Dp, Cp = dW.shape[0], dW.shape[1]
    N = x.shape[0]
    px = _dev_ptr(x, x.dtype, (N, Cp * T), "x")
    pg = _dev_ptr(gy, x.dtype, (N, Dp * T), "gy")
    pw = _dev_ptr(dW, torch.float32, (Dp, Cp, T), "dW")
    pb = None if db is None else _dev_ptr(db, torch.float32, (Dp,), "db")
    _check(lib().eqlin_backward_dw_noalloc(T, Cp, Dp, _DT[x.dtype], px, pg, pw, pb, N, _stream(stream)),
           "eqlin_backward_dw_noalloc")


def get_error(h: Handle) -> int:
    """Device-side status (0, or -6 for a wait that timed out); clears it."""
    return int(lib().eqlin_get_error(h.ptr))


def error_detail(h: Handle) -> dict:
    """Where the last non-OK eqlin_get_error came from (see eqlin_error_detail)."""
    d = (ctypes.c_uint32 * 4)()
    _check(lib().eqlin_error_detail(h.ptr, d), "eqlin_error_detail")
    return {"status": d[0], "kernel": d[1] >> 8, "role": (d[1] >> 4) & 15, "barrier": d[1] & 15,
            "cta": d[2] & 0xFFF, "iteration": d[2] >> 12, "polls": d[3] & 0xFFFFF, "ms": d[3] >> 20}


def set_tail_split(h: Handle, enable: bool):
    """Split the last wave's tiles of the f16/bf16 forward and dx over two SMs
    each (off by default): shorter lone calls, at the price of extra work."""
    _check(lib().eqlin_set_tail_split(h.ptr, 1 if enable else 0), "eqlin_set_tail_split")


def set_wait_limit(h: Handle, iterations: int):
    _check(lib().eqlin_set_wait_limit(h.ptr, int(iterations)), "eqlin_set_wait_limit")


def launch_count() -> int:
    """Kernels the library has enqueued in this process (all handles)."""
    return int(lib().eqlin_launch_count())


def status_string(status: int) -> str:
    return lib().eqlin_status_string(int(status)).decode()


def destroy(h: Handle):
    h.close()


# ------------------------------------------ norm, rotary positions, attention
#
# These calls belong to no handle.  They run on the tensors' device (all on one)
# and, unless told otherwise, on its current stream.

NO_POLLS = 0xFFFFFFFF             # wait_limit: a wait that is not over when it begins runs out


class _On:
    """Make the tensors' device current for a call and find the stream."""

    def __init__(self, t: torch.Tensor, stream):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError("expected a CUDA tensor")
        self.index, self.stream = t.get_device(), stream

    def __enter__(self):
        cur = torch.cuda.current_device()
        self.prev = cur if cur != self.index else None
        if self.prev is not None:
            torch.cuda.set_device(self.index)
        if self.stream is None:
            # torch.cuda.current_stream().cuda_stream, without the 3 us of building a Stream
            return torch._C._cuda_getCurrentRawStream(self.index)
        return self.stream.cuda_stream if hasattr(self.stream, "cuda_stream") else int(self.stream)

    def __exit__(self, *exc):
        if self.prev is not None:
            torch.cuda.set_device(self.prev)
        return False


def _ptr(t, dtype, shape, name, index):
    """The address of a contiguous tensor on device `index`; small calls are bound by
    their checks, so what is right is found out in four steps."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.is_contiguous() \
            and (shape is None or t.shape == shape):
        return t.data_ptr()
    _dev_ptr(t, dtype, shape, name)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _opt(t, dtype, shape, name, index):
    return None if t is None else _ptr(t, dtype, shape, name, index)


def _shape2(x, name):
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{name} must be a CUDA tensor")
    if x.dim() != 2:
        raise ValueError(f"{name} must be [N, C'*T], got {tuple(x.shape)}")
    if x.dtype not in _DT:
        raise TypeError(f"{name} must be float32, float16 or bfloat16, got {x.dtype}")
    return x.shape


def norm_forward(x: torch.Tensor, w: torch.Tensor, b: torch.Tensor, y: torch.Tensor, mean: torch.Tensor,
                 rstd: torch.Tensor, T: int, eps: float = 1e-6, res: torch.Tensor | None = None,
                 xsum: torch.Tensor | None = None, stream=None):
    """Group layer norm of x (or of x + res, which xsum receives); see eqlin_norm_forward."""
    N, F = _shape2(x, "x")
    dt, dev, Cp = x.dtype, x.get_device(), w.shape[0]
    if Cp * T != F:
        raise ValueError(f"x has {F} features, w {Cp} channels of {T}")
    with _On(x, stream) as st:
        _check(lib().eqlin_norm_forward(
            T, Cp, _DT[dt], _ptr(x, dt, None, "x", dev), _opt(res, dt, (N, F), "res", dev),
            _ptr(w, dt, (Cp,), "w", dev), _ptr(b, dt, (Cp,), "b", dev), eps, _opt(xsum, dt, (N, F), "xsum", dev),
            _ptr(y, dt, (N, F), "y", dev), _ptr(mean, torch.float32, (N,), "mean", dev),
            _ptr(rstd, torch.float32, (N,), "rstd", dev), N, st), "eqlin_norm_forward")


def norm_workspace(T: int, Cp: int, N: int, device=None) -> torch.Tensor:
    """A workspace for norm_backward on N rows."""
    n = int(lib().eqlin_norm_workspace_bytes(int(T), int(Cp), int(N)))
    if n < 0:
        raise ValueError(f"no norm of {Cp} channels of {T} on {N} rows")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def norm_backward(gy: torch.Tensor, x: torch.Tensor, w: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                  dx: torch.Tensor, dw: torch.Tensor, db: torch.Tensor, T: int, gsum: torch.Tensor | None = None,
                  res: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients of the norm of x (or of x + res), both as the forward had them: not
    xsum, whose rounding would go into dw.  See eqlin_norm_backward."""
    N, F = _shape2(gy, "gy")
    dt, dev, Cp = gy.dtype, gy.get_device(), w.shape[0]
    if Cp * T != F:
        raise ValueError(f"gy has {F} features, w {Cp} channels of {T}")
    with _On(gy, stream) as st:
        if workspace is None:
            if stream is not None:
                raise ValueError("pass a workspace along with a stream")
            workspace = norm_workspace(T, Cp, N, gy.device)
        need = lib().eqlin_norm_workspace_bytes(T, Cp, N)
        if workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} bytes, needs {need}")
        _check(lib().eqlin_norm_backward(
            T, Cp, _DT[dt], _ptr(gy, dt, None, "gy", dev), _opt(gsum, dt, (N, F), "gsum", dev),
            _ptr(x, dt, (N, F), "x", dev), _opt(res, dt, (N, F), "res", dev), _ptr(w, dt, (Cp,), "w", dev),
            _ptr(mean, torch.float32, (N,), "mean", dev),
            _ptr(rstd, torch.float32, (N,), "rstd", dev), _ptr(dx, dt, (N, F), "dx", dev),
            _ptr(dw, torch.float32, (Cp,), "dw", dev), _ptr(db, torch.float32, (Cp,), "db", dev),
            _ptr(workspace, workspace.dtype, None, "workspace", dev), N, st), "eqlin_norm_backward")


class Rope:
    """A plan of rotary positions for heads of [Ch, T] features.

    ``sections[a]`` channel pairs follow axis a of the positions; pair k of a
    section of n turns by ``base ** (-k / n)`` radians per unit of position,
    unless ``freqs`` gives one frequency for each pair of all sections."""

    def __init__(self, T: int, Ch: int, sections, base: float = 100.0, freqs=None):
        self.T, self.Ch, self.sections = int(T), int(Ch), tuple(int(n) for n in sections)
        if not self.sections or min(self.sections) < 0:
            raise ValueError("sections holds a number of channel pairs for each axis")
        if freqs is None:
            freqs = [float(base) ** (-k / n) for n in self.sections for k in range(n)]
        self.freqs = tuple(float(f) for f in freqs)
        if len(self.freqs) != sum(self.sections):
            raise ValueError(f"{len(self.freqs)} frequencies for {sum(self.sections)} channel pairs")
        out = ctypes.c_void_p()
        self._r = None
        _check(lib().eqlin_rope_create(self.T, self.Ch, self.axes, (_i64 * self.axes)(*self.sections),
                                       (ctypes.c_double * max(1, len(self.freqs)))(*self.freqs), ctypes.byref(out)),
               "eqlin_rope_create")
        self._r = out

    @property
    def axes(self) -> int:
        return len(self.sections)

    @property
    def ptr(self):
        return self._r

    def __del__(self):
        try:
            if self._r:
                lib().eqlin_rope_destroy(self._r)
                self._r = None
        except Exception:
            pass

    def __copy__(self):
        return self

    def __deepcopy__(self, memo):
        return self                # immutable, in host memory

    def __reduce__(self):
        return Rope, (self.T, self.Ch, self.sections, 1.0, self.freqs)


def _heads(t, dtype, shape, name, index):
    """A [N, heads, D] tensor whose heads lie one after the other: address and token stride."""
    N, H, D = shape
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.shape == shape:
        s = t.stride()
        if (s[2] == 1 or D == 1) and (s[1] == D or H == 1) or t.numel() == 0:
            # a single token has no next one: its stride says nothing
            return t.data_ptr(), (s[0] if N > 1 else H * D)
        raise ValueError(f"{name}: the heads of a token must lie one after the other")
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def rope(r: Rope, pos: torch.Tensor, src: torch.Tensor, dst: torch.Tensor, inverse: bool = False, stream=None):
    """Turn the heads src [N, heads, Ch*T] by their positions pos [N, axes] into
    dst (which may be src); ``inverse`` turns back.  See eqlin_rope_apply."""
    if not isinstance(src, torch.Tensor) or src.dim() != 3:
        raise ValueError("src must be [N, heads, Ch*T]")
    N, H, D = src.shape
    if D != r.Ch * r.T:
        raise ValueError(f"src has heads of {D} features, the plan {r.Ch} channels of {r.T}")
    if src.dtype not in _DT:
        raise TypeError(f"src must be float32, float16 or bfloat16, got {src.dtype}")
    with _On(src, stream) as st:
        dev = src.get_device()
        ps, ss = _heads(src, src.dtype, (N, H, D), "src", dev)
        pd, ds = _heads(dst, src.dtype, (N, H, D), "dst", dev)
        _check(lib().eqlin_rope_apply(r.ptr, _DT[src.dtype], _ptr(pos, torch.float32, (N, r.axes), "pos", dev),
                                      ps, ss, pd, ds, H, 1 if inverse else 0, N, st), "eqlin_rope_apply")


def _attention_desc(q, k, v, o, lse, docs, offsets, max_len, pos, slopes, scale, cap, err, wait_limit):
    if not isinstance(q, torch.Tensor) or q.dim() != 3 or not isinstance(k, torch.Tensor) or k.dim() != 3:
        raise ValueError("q, k and v must be [N, heads, D]")
    if q.dtype not in _DT:
        raise TypeError(f"q must be float32, float16 or bfloat16, got {q.dtype}")
    N, H, D = q.shape
    K = k.shape[1]
    dev = q.get_device()
    if offsets is not None:
        if offsets.dim() != 1 or offsets.numel() < 1:
            raise ValueError("offsets must be [docs + 1]")
        docs = offsets.numel() - 1
    axes = 0
    if (pos is None) != (slopes is None):
        raise ValueError("pos and slopes go together")
    if pos is not None:
        if pos.dim() != 2 or pos.shape[1] < 1:
            raise ValueError("pos must be [N, axes]")
        axes = pos.shape[1]
    pq, sq = _heads(q, q.dtype, (N, H, D), "q", dev)
    pk, sk = _heads(k, q.dtype, (N, K, D), "k", dev)
    pv, sv = _heads(v, q.dtype, (N, K, D), "v", dev)
    po, so = _heads(o, q.dtype, (N, H, D), "o", dev)
    desc = AttentionDesc(                  # in the structure's order
        N, H, K, D, sq, sk, sv, so, int(docs), _opt(offsets, torch.int32, None, "offsets", dev), int(max_len or 0),
        _opt(pos, torch.float32, (N, axes), "pos", dev), _opt(slopes, torch.float32, (H,), "slopes", dev), axes,
        D ** -0.5 if scale is None else float(scale), float(cap), _opt(err, torch.int32, (4,), "err", dev),
        int(wait_limit))
    return desc, (pq, pk, pv, po), _ptr(lse, torch.float32, (H, N), "lse", dev)


def attention_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor, *,
                      docs: int = 1, offsets: torch.Tensor | None = None, max_len: int | None = None,
                      pos: torch.Tensor | None = None, slopes: torch.Tensor | None = None, scale: float | None = None,
                      cap: float = 0.0, err: torch.Tensor | None = None, wait_limit: int = 0, stream=None):
    """Attention within documents: q, o [N, heads, D], k, v [N, kv_heads, D],
    lse [heads, N] float32.  ``docs`` documents of equal length, or ``offsets``
    (int32 [docs + 1]) for packed ones; see eqlin_attention_forward."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a CUDA tensor")
    with _On(q, stream) as st:
        desc, (pq, pk, pv, po), pl = _attention_desc(q, k, v, o, lse, docs, offsets, max_len, pos, slopes, scale, cap,
                                                     err, wait_limit)
        _check(lib().eqlin_attention_forward(ctypes.byref(desc), _DT[q.dtype], pq, pk, pv, po, pl, st),
               "eqlin_attention_forward")


def attention_backward(go: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                       lse: torch.Tensor, dq: torch.Tensor, dk: torch.Tensor, dv: torch.Tensor, delta: torch.Tensor,
                       *, docs: int = 1, offsets: torch.Tensor | None = None, max_len: int | None = None,
                       pos: torch.Tensor | None = None, slopes: torch.Tensor | None = None,
                       scale: float | None = None, cap: float = 0.0, err: torch.Tensor | None = None,
                       wait_limit: int = 0, stream=None):
    """Gradients of attention_forward into dq, dk and dv; delta [heads, N]
    float32 is a workspace.  See eqlin_attention_backward."""
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a CUDA tensor")
    with _On(q, stream) as st:
        desc, (pq, pk, pv, po), pl = _attention_desc(q, k, v, o, lse, docs, offsets, max_len, pos, slopes, scale, cap,
                                                     err, wait_limit)
        dev, dt = q.get_device(), q.dtype
        pg, sg = _heads(go, dt, q.shape, "go", dev)
        pdq, sdq = _heads(dq, dt, q.shape, "dq", dev)
        pdk, sdk = _heads(dk, dt, k.shape, "dk", dev)
        pdv, sdv = _heads(dv, dt, k.shape, "dv", dev)
        _check(lib().eqlin_attention_backward(
            ctypes.byref(desc), _DT[dt], pg, sg, pq, pk, pv, po, pl, pdq, sdq, pdk, sdk, pdv, sdv,
            _ptr(delta, torch.float32, (q.shape[1], q.shape[0]), "delta", dev), st), "eqlin_attention_backward")


def attention_error(err: torch.Tensor) -> int:
    """What the attention calls that were given ``err`` recorded: 0, or -6 for a
    wait that timed out; clears it.  Waits for the current stream: synchronise
    others that the calls ran on before."""
    if not isinstance(err, torch.Tensor) or err.dtype != torch.int32 or tuple(err.shape) != (4,):
        raise TypeError("err must be an int32 tensor of 4")
    if err.tolist()[0] == 0:
        return 0
    err.zero_()
    return -6


# ------------------------------------------------------- allocating helpers

class EQLinear:
    """Convenience wrapper: owns a handle and allocates outputs with torch."""

    def __init__(self, W: torch.Tensor, b: torch.Tensor | None = None, group="cyclic"):
        Dp, Cp, T = W.shape
        if group == "dihedral":
            self.h = create_group("dihedral", T // 2, Cp, Dp, W.dtype)
        else:
            self.h = create(T, Cp, Dp, W.dtype)
        self.set_weights(W, b)

    def set_weights(self, W, b=None, stream=None):
        set_weights(self.h, W.contiguous(), None if b is None else b.contiguous(), stream)

    def forward(self, x, stream=None):
        y = torch.empty((x.shape[0], self.h.Dp * self.h.T), dtype=self.h.dtype, device=x.device)
        forward(self.h, x, y, stream)
        return y

    def backward_dx(self, gy, stream=None):
        dx = torch.empty((gy.shape[0], self.h.Cp * self.h.T), dtype=self.h.dtype, device=gy.device)
        backward_dx(self.h, gy, dx, stream)
        return dx

    def backward_dw(self, x, gy, stream=None):
        dW = torch.empty((self.h.Dp, self.h.Cp, self.h.T), dtype=torch.float32, device=x.device)
        db = torch.empty((self.h.Dp,), dtype=torch.float32, device=x.device)
        backward_dw(self.h, x, gy, dW, db, stream)
        return dW, db
