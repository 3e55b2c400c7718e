"""Python binding of the C ABI, one function per entry point of include/instant.h.

Each function takes torch CUDA tensors, checks their shapes against each other,
and passes raw device pointers, extents and the current CUDA stream to the
library.  No arithmetic of the method happens here.
"""

from __future__ import annotations

import array
import ctypes
import dataclasses
import operator

import torch

from ._lib import (ACTIVATIONS, GRAD_X_STATIC_SCRATCH_BYTES, INSTANT_BF16, INSTANT_F32, TOP_MAX, AccumulateItem,
                   CalibParams, CalibProblem, GradItem, check, lib)

__all__ = [
    "compress_act",
    "forward",
    "forward_workspace",
    "project_grad",
    "grad_w",
    "grad_x",
    "grad_x_workspace_bytes",
    "grad_w_x",
    "backward",
    "backward_workspace",
    "backward_workspace_bytes",
    "grad_x_core",
    "expand",
    "grad_x_static",
    "launch_count",
    "calib_accumulate",
    "calib_accumulate_batch",
    "calib_solve",
    "calib_solve_batch",
    "CalibBatch",
    "calib_workspace_bytes",
    "calib_batch_workspace_bytes",
    "ckpt_buffers",
    "ckpt_pack",
    "ckpt_unpack",
    "rms_norm",
    "rms_norm_backward",
    "rms_norm_backward_workspace",
    "linear_act",
    "linear_act_grad",
    "ckpt_grad_w",
    "ckpt_grad_w_workspace",
    "embed",
    "embed_grad",
    "embed_grad_workspace",
    "token_logprobs",
    "token_logprobs_grad",
    "GradClip",
    "grad_clip",
    "device_status",
    "reconstruction_error",
    "CalibResult",
    "dtype_code",
]


def dtype_code(t: torch.dtype) -> int:
    if t == torch.bfloat16:
        return INSTANT_BF16
    if t == torch.float32:
        return INSTANT_F32
    raise TypeError(f"unsupported dtype {t}: use torch.bfloat16 or torch.float32")


def _dev(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must live on a CUDA device")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


# the current stream's handle without building a torch.cuda.Stream around it
# (0.1 us against 3 us)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _on_stream(stream):
    """Context in which torch allocates for the stream that a call runs on."""
    if stream is None or isinstance(stream, torch.cuda.Stream):
        return torch.cuda.stream(stream)
    return torch.cuda.stream(torch.cuda.ExternalStream(int(stream)))


def _same_dtype(dt, *pairs):
    for name, t in pairs:
        if t.dtype != dt:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dt}")


def compress_act(x: torch.Tensor, P: torch.Tensor, xhat: torch.Tensor, stream=None) -> torch.Tensor:
    """``xhat[b] = P @ x[b]``: x ``[B, L, Cx]``, P ``[Rx, L]``, xhat ``[B, Rx, Cx]``."""
    B, L, Cx = x.shape
    Rx = P.shape[0]
    if P.shape != (Rx, L) or xhat.shape != (B, Rx, Cx):
        raise ValueError("compress_act: inconsistent shapes")
    _same_dtype(x.dtype, ("P", P), ("xhat", xhat))
    check(lib().instant_compress_act(_dev(x, "x"), _dev(P, "P"), _dev(xhat, "xhat"), B, L, Cx, Rx,
                                     dtype_code(x.dtype), _stream(stream)), "instant_compress_act")
    return xhat


def forward_workspace(B: int, L: int, Cx: int, Rx: int, dtype: torch.dtype, device) -> torch.Tensor:
    """A zeroed workspace for :func:`forward` (it must start at zero; every call
    leaves it zero)."""
    n = int(lib().instant_forward_workspace_bytes(B, L, Cx, Rx, dtype_code(dtype)))
    return torch.zeros(max(n, 16), dtype=torch.uint8, device=device)


def forward(x: torch.Tensor, w: torch.Tensor, y: torch.Tensor, P: torch.Tensor | None = None,
            xhat: torch.Tensor | None = None, ws: torch.Tensor | None = None, stream=None):
    """``y[b] = x[b] w^T`` and, with ``P``, ``xhat[b] = P x[b]`` in the same pass:
    x ``[B, L, Cx]``, w ``[Cy, Cx]``, y ``[B, L, Cy]``, P ``[Rx, L]``,
    xhat ``[B, Rx, Cx]``; ws from :func:`forward_workspace`."""
    B, L, Cx = x.shape
    Cy = w.shape[0]
    if w.shape != (Cy, Cx) or y.shape != (B, L, Cy):
        raise ValueError("forward: inconsistent shapes")
    Rx = 0
    if P is not None:
        Rx = P.shape[0]
        if P.shape != (Rx, L) or xhat is None or xhat.shape != (B, Rx, Cx) or ws is None:
            raise ValueError("forward: P needs xhat [B, Rx, Cx] and a workspace")
        _same_dtype(x.dtype, ("P", P), ("xhat", xhat))
    _same_dtype(x.dtype, ("w", w), ("y", y))
    check(lib().instant_forward(_dev(x, "x"), _dev(w, "w"), _dev(P, "P") if P is not None else None,
                                _dev(y, "y"), _dev(xhat, "xhat") if P is not None else None,
                                _dev(ws, "ws") if ws is not None else None,
                                ws.numel() * ws.element_size() if ws is not None else 0, B, L, Cx,
                                Cy, Rx, dtype_code(x.dtype), _stream(stream)), "instant_forward")
    return y, xhat


def project_grad(g_y: torch.Tensor, PQ: torch.Tensor, Sx: torch.Tensor, Sq: torch.Tensor,
                 Rx: int, Ry: int, stream=None):
    """``Sx[b] = P g_y[b]``, ``Sq[b] = Q g_y[b]`` with ``PQ = [P; Q]``.

    g_y ``[B, L, Cy]``, PQ ``[Rx+Ry, L]``, Sx ``[B*Rx, Cy]``, Sq ``[B*Ry, Cy]``."""
    B, L, Cy = g_y.shape
    if PQ.shape != (Rx + Ry, L) or Sx.shape != (B * Rx, Cy) or Sq.shape != (B * Ry, Cy):
        raise ValueError("project_grad: inconsistent shapes")
    _same_dtype(g_y.dtype, ("PQ", PQ), ("Sx", Sx), ("Sq", Sq))
    check(lib().instant_project_grad(_dev(g_y, "g_y"), _dev(PQ, "PQ"), _dev(Sx, "Sx"), _dev(Sq, "Sq"),
                                     B, L, Cy, Rx, Ry, dtype_code(g_y.dtype), _stream(stream)),
          "instant_project_grad")
    return Sx, Sq


def grad_w(Sx: torch.Tensor, xhat: torch.Tensor, gw: torch.Tensor, B: int, accumulate: bool = False,
           stream=None) -> torch.Tensor:
    """``gw (+)= Sx^T xhat``: Sx ``[B*Rx, Cy]``, xhat ``[B*Rx, Cx]`` (or ``[B, Rx, Cx]``),
    gw ``[Cy, Cx]`` fp32."""
    K, Cy = Sx.shape
    xh = xhat.reshape(K, -1) if xhat.dim() == 3 else xhat
    Cx = xh.shape[1]
    if K % B != 0 or xh.shape[0] != K or gw.shape != (Cy, Cx) or gw.dtype != torch.float32:
        raise ValueError("grad_w: inconsistent shapes")
    _same_dtype(Sx.dtype, ("xhat", xhat))
    check(lib().instant_grad_w(_dev(Sx, "Sx"), _dev(xhat, "xhat"), _dev(gw, "gw"), int(bool(accumulate)),
                               B, K // B, Cx, Cy, dtype_code(Sx.dtype), _stream(stream)),
          "instant_grad_w")
    return gw


def grad_x_workspace_bytes(B: int, L: int, Cx: int, Cy: int, Ry: int, dtype: torch.dtype) -> int:
    return int(lib().instant_grad_x_workspace_bytes(B, L, Cx, Cy, Ry, dtype_code(dtype)))


def grad_x(Sq: torch.Tensor, w: torch.Tensor, Q: torch.Tensor, gx: torch.Tensor,
           ws: torch.Tensor, stream=None) -> torch.Tensor:
    """``gx[b] = Q^T (Sq[b] w)``: Sq ``[B*Ry, Cy]``, w ``[Cy, Cx]``, Q ``[Ry, L]``,
    gx ``[B, L, Cx]``; ws is scratch of ``grad_x_workspace_bytes`` bytes."""
    B, L, Cx = gx.shape
    Ry = Q.shape[0]
    Cy = w.shape[0]
    if Q.shape != (Ry, L) or w.shape != (Cy, Cx) or Sq.shape != (B * Ry, Cy):
        raise ValueError("grad_x: inconsistent shapes")
    _same_dtype(Sq.dtype, ("w", w), ("Q", Q), ("gx", gx))
    check(lib().instant_grad_x(_dev(Sq, "Sq"), _dev(w, "w"), _dev(Q, "Q"), _dev(gx, "gx"),
                               _dev(ws, "ws"), ws.numel() * ws.element_size(), B, L, Cx, Cy, Ry,
                               dtype_code(Sq.dtype), _stream(stream)), "instant_grad_x")
    return gx


def grad_w_x(Sx: torch.Tensor, xhat: torch.Tensor, gw: torch.Tensor, Sq: torch.Tensor,
             w: torch.Tensor, Q: torch.Tensor, gx: torch.Tensor, ws: torch.Tensor, B: int, *,
             accumulate: bool = False, stream=None):
    """:func:`grad_w` and :func:`grad_x` in one call (one launch where the
    single-kernel input gradient applies).  Returns ``(gw, gx)``."""
    Bg, L, Cx = gx.shape
    Ry = Q.shape[0]
    Cy = w.shape[0]
    Rx = Sx.shape[0] // B
    if (Bg != B or Q.shape != (Ry, L) or w.shape != (Cy, Cx) or Sq.shape != (B * Ry, Cy)
            or Sx.shape != (B * Rx, Cy) or xhat.numel() != B * Rx * Cx or gw.shape != (Cy, Cx)):
        raise ValueError("grad_w_x: inconsistent shapes")
    if gw.dtype != torch.float32:
        raise TypeError("grad_w_x: gw must be float32")
    _same_dtype(Sq.dtype, ("Sx", Sx), ("xhat", xhat), ("w", w), ("Q", Q), ("gx", gx))
    check(lib().instant_grad_w_x(_dev(Sx, "Sx"), _dev(xhat, "xhat"), _dev(gw, "gw"), int(bool(accumulate)),
                                 _dev(Sq, "Sq"), _dev(w, "w"), _dev(Q, "Q"), _dev(gx, "gx"),
                                 _dev(ws, "ws"), ws.numel() * ws.element_size(), B, L, Cx, Cy, Rx,
                                 Ry, dtype_code(Sq.dtype), _stream(stream)), "instant_grad_w_x")
    return gw, gx


def backward_workspace_bytes(B: int, L: int, Cx: int, Cy: int, Ry: int, dtype: torch.dtype) -> int:
    return int(lib().instant_backward_workspace_bytes(B, L, Cx, Cy, Ry, dtype_code(dtype)))


def backward_workspace(B: int, L: int, Cx: int, Cy: int, Ry: int, dtype: torch.dtype,
                       device) -> torch.Tensor:
    """A zeroed workspace for :func:`backward` (its counters must start at zero)."""
    return torch.zeros(backward_workspace_bytes(B, L, Cx, Cy, Ry, dtype), dtype=torch.uint8,
                       device=device)


def backward(g_y: torch.Tensor, PQ: torch.Tensor, xhat: torch.Tensor, w: torch.Tensor,
             Sx: torch.Tensor, Sq: torch.Tensor, gw: torch.Tensor, gx: torch.Tensor,
             ws: torch.Tensor, Rx: int, *, accumulate: bool = False, stream=None):
    """:func:`project_grad` then :func:`grad_w_x` in one call (one launch where
    the single-kernel input gradient applies).  ``ws`` comes from
    :func:`backward_workspace`.  Returns ``(gw, gx)``."""
    B, L, Cy = g_y.shape
    Ry = PQ.shape[0] - Rx
    Cx = w.shape[1]
    if (PQ.shape[1] != L or Ry < 1 or w.shape != (Cy, Cx) or xhat.numel() != B * Rx * Cx
            or Sx.shape != (B * Rx, Cy) or Sq.shape != (B * Ry, Cy) or gw.shape != (Cy, Cx)
            or gx.shape != (B, L, Cx)):
        raise ValueError("backward: inconsistent shapes")
    if gw.dtype != torch.float32:
        raise TypeError("backward: gw must be float32")
    _same_dtype(g_y.dtype, ("PQ", PQ), ("xhat", xhat), ("w", w), ("Sx", Sx), ("Sq", Sq), ("gx", gx))
    check(lib().instant_backward(_dev(g_y, "g_y"), _dev(PQ, "PQ"), _dev(xhat, "xhat"), _dev(w, "w"),
                                 _dev(Sx, "Sx"), _dev(Sq, "Sq"), _dev(gw, "gw"),
                                 int(bool(accumulate)), _dev(gx, "gx"), _dev(ws, "ws"),
                                 ws.numel() * ws.element_size(), B, L, Cx, Cy, Rx, Ry,
                                 dtype_code(g_y.dtype), _stream(stream)), "instant_backward")
    return gw, gx


def grad_x_core(Sq: torch.Tensor, w: torch.Tensor, ws: torch.Tensor, B: int, stream=None):
    """First half of :func:`grad_x`: ``g_hat_x = Sq w`` into the workspace."""
    Cy, Cx = w.shape
    Ry = Sq.shape[0] // B
    if Sq.shape != (B * Ry, Cy):
        raise ValueError("grad_x_core: inconsistent shapes")
    _same_dtype(Sq.dtype, ("w", w))
    check(lib().instant_grad_x_core(_dev(Sq, "Sq"), _dev(w, "w"), _dev(ws, "ws"),
                                    ws.numel() * ws.element_size(), B, Cx, Cy, Ry,
                                    dtype_code(Sq.dtype), _stream(stream)), "instant_grad_x_core")
    return ws


def grad_x_static(Sq: torch.Tensor, w: torch.Tensor, Q: torch.Tensor, gx: torch.Tensor,
                  stream=None) -> torch.Tensor:
    """:func:`grad_x` for callers that cannot allocate device memory: no
    workspace argument; ``g_hat_x`` lives in a fixed array of the library
    (``GRAD_X_STATIC_SCRATCH_BYTES`` per device) that every call on a device
    shares, so calls must not overlap in time.  The first call on a device
    looks the array up and should come before any stream capture."""
    B, L, Cx = gx.shape
    Ry = Q.shape[0]
    Cy = w.shape[0]
    if Q.shape != (Ry, L) or w.shape != (Cy, Cx) or Sq.shape != (B * Ry, Cy):
        raise ValueError("grad_x_static: inconsistent shapes")
    _same_dtype(Sq.dtype, ("w", w), ("Q", Q), ("gx", gx))
    status = lib().instant_grad_x_static(_dev(Sq, "Sq"), _dev(w, "w"), _dev(Q, "Q"), _dev(gx, "gx"),
                                         B, L, Cx, Cy, Ry, dtype_code(Sq.dtype), _stream(stream))
    if status == 5:
        need = grad_x_workspace_bytes(B, L, Cx, Cy, Ry, Sq.dtype)
        raise ValueError(f"grad_x_static: g_hat_x needs {need} bytes, more than the "
                         f"{GRAD_X_STATIC_SCRATCH_BYTES}-byte fixed array; use grad_x with a workspace")
    check(status, "instant_grad_x_static")
    return gx


def expand(Q: torch.Tensor, gx: torch.Tensor, ws: torch.Tensor, Cy: int, stream=None):
    """Second half of :func:`grad_x`: ``gx[b] = Q^T g_hat_x[b]`` from the workspace."""
    B, L, Cx = gx.shape
    Ry = Q.shape[0]
    if Q.shape != (Ry, L):
        raise ValueError("expand: inconsistent shapes")
    _same_dtype(Q.dtype, ("gx", gx))
    check(lib().instant_expand(_dev(Q, "Q"), _dev(gx, "gx"), _dev(ws, "ws"),
                               ws.numel() * ws.element_size(), B, L, Cx, Cy, Ry,
                               dtype_code(Q.dtype), _stream(stream)), "instant_expand")
    return gx


def launch_count() -> int:
    """Kernels launched by the library so far in this process."""
    return int(lib().instant_launch_count())


def calib_accumulate(t: torch.Tensor, C: torch.Tensor, stream=None) -> torch.Tensor:
    """``C += sum_b t[b] t[b]^T``: t ``[B, L, C]``, C ``[L, L]`` fp32."""
    B, L, Cd = t.shape
    if C.shape != (L, L) or C.dtype != torch.float32:
        raise ValueError("calib_accumulate: C must be [L, L] float32")
    check(lib().instant_calib_accumulate(_dev(t, "t"), _dev(C, "C"), B, L, Cd, dtype_code(t.dtype),
                                         _stream(stream)), "instant_calib_accumulate")
    return C


def calib_accumulate_batch(pairs, stream=None) -> None:
    """``C += sum_b t[b] t[b]^T`` for every ``(t, C)`` in ``pairs`` (one token
    length L; t ``[B, L, Cdim]`` of one dtype, C ``[L, L]`` fp32), up to four
    statistics per launch."""
    pairs = list(pairs)
    if not pairs:
        raise ValueError("calib_accumulate_batch: nothing to accumulate")
    L = pairs[0][0].shape[1]
    dt = pairs[0][0].dtype
    arr = (AccumulateItem * len(pairs))()
    for i, (t, C) in enumerate(pairs):
        B, Lt, Cd = t.shape
        if Lt != L or t.dtype != dt or C.shape != (L, L) or C.dtype != torch.float32:
            raise ValueError("calib_accumulate_batch: inconsistent shapes or dtypes")
        arr[i] = AccumulateItem(_dev(t, "t"), _dev(C, "C"), B, Cd)
    check(lib().instant_calib_accumulate_batch(arr, len(pairs), L, dtype_code(dt), _stream(stream)),
          "instant_calib_accumulate_batch")


def calib_workspace_bytes(L: int, r_cap: int) -> int:
    return int(lib().instant_calib_workspace_bytes(L, r_cap))


@dataclasses.dataclass
class CalibResult:
    k: int
    R: int
    scale: float
    energy: float
    eigenvalues: list


def calib_solve(C: torch.Tensor, n_samples: int, rows_out: torch.Tensor, *, eps: float = 0.95,
                p: int = 0, r_override: int = 0, scale_on: bool = True, max_iter: int = 0,
                tol: float = 0.0, ws: torch.Tensor | None = None, stream=None,
                raise_on_error: bool = True, warm_start: bool = False):
    """Projector rows from an accumulated statistic; synchronises the stream.

    With ``warm_start`` the rows already in ``rows_out`` (a previous projector
    of the same statistic) seed the eigensolver.

    Returns a :class:`CalibResult` (and the raw status when ``raise_on_error``
    is False)."""
    L = C.shape[0]
    r_cap = rows_out.shape[0]
    if C.shape != (L, L) or C.dtype != torch.float32 or rows_out.shape[1] != L:
        raise ValueError("calib_solve: inconsistent shapes")
    if ws is None:
        ws = torch.empty(calib_workspace_bytes(L, r_cap), dtype=torch.uint8, device=C.device)
    prm = CalibParams(eps, p, r_override, int(bool(scale_on)), max_iter, tol, int(bool(warm_start)))
    k = ctypes.c_int(0)
    R = ctypes.c_int(0)
    s = ctypes.c_float(0)
    E = ctypes.c_double(0)
    eig = (ctypes.c_double * r_cap)()
    st = lib().instant_calib_solve(_dev(C, "C"), int(n_samples), L, ctypes.byref(prm),
                                   _dev(rows_out, "rows_out"), r_cap, dtype_code(rows_out.dtype),
                                   ctypes.byref(k), ctypes.byref(R), ctypes.byref(s),
                                   ctypes.byref(E), eig, _dev(ws, "ws"),
                                   ws.numel() * ws.element_size(), _stream(stream))
    res = CalibResult(k.value, R.value, s.value, E.value, list(eig))
    if raise_on_error:
        check(st, "instant_calib_solve")
        return res
    return res, st


def calib_batch_workspace_bytes(L: int, count: int) -> int:
    return int(lib().instant_calib_batch_workspace_bytes(L, count))


def calib_solve_batch(problems, *, ws: torch.Tensor | None = None, stream=None,
                      raise_on_error: bool = True):
    """Several statistics of one token length in one call; synchronises the stream.

    ``problems`` is a sequence of dicts with the keys ``C`` (``[L, L]`` fp32),
    ``n_samples`` and ``rows_out`` (``[r_cap, L]``, one dtype for all), and
    optionally the keyword parameters of :func:`calib_solve` (``eps``, ``p``,
    ``r_override``, ``scale_on``, ``max_iter``, ``tol``, ``warm_start``).
    Returns a list of :class:`CalibResult` (and the list of per-problem
    statuses when ``raise_on_error`` is False)."""
    n = len(problems)
    if n < 1:
        raise ValueError("calib_solve_batch: no problems")
    L = problems[0]["C"].shape[0]
    dt = problems[0]["rows_out"].dtype
    arr = (CalibProblem * n)()
    eigs = []
    for i, q in enumerate(problems):
        C, rows = q["C"], q["rows_out"]
        if C.shape != (L, L) or C.dtype != torch.float32 or rows.shape[1] != L or rows.dtype != dt:
            raise ValueError("calib_solve_batch: inconsistent shapes or dtypes")
        r_cap = rows.shape[0]
        eig = (ctypes.c_double * r_cap)()
        eigs.append(eig)
        prm = CalibParams(q.get("eps", 0.95), q.get("p", 0), q.get("r_override", 0),
                          int(bool(q.get("scale_on", True))), q.get("max_iter", 0), q.get("tol", 0.0),
                          int(bool(q.get("warm_start", False))))
        arr[i] = CalibProblem(_dev(C, "C"), int(q["n_samples"]), prm, _dev(rows, "rows_out"), r_cap,
                              ctypes.cast(eig, ctypes.POINTER(ctypes.c_double)), 0, 0, 0.0, 0.0, 0)
    if ws is None:
        ws = torch.empty(calib_batch_workspace_bytes(L, n), dtype=torch.uint8,
                         device=problems[0]["C"].device)
    st = lib().instant_calib_solve_batch(arr, n, L, dtype_code(dt), _dev(ws, "ws"),
                                         ws.numel() * ws.element_size(), _stream(stream))
    res = [CalibResult(arr[i].k, arr[i].R, arr[i].scale, arr[i].energy, list(eigs[i]))
           for i in range(n)]
    if raise_on_error:
        check(st, "instant_calib_solve_batch")
        return res
    return res, [arr[i].status for i in range(n)]


class CalibBatch:
    """The same statistics solved together again and again (a layer's C_X into
    P and C_G into Q, every N_t steps): the argument block of
    ``instant_calib_solve_batch`` is built once; :meth:`solve` updates the
    sample counts and the warm-start flag and passes it.  The tensors given
    here must stay alive and in place."""

    def __init__(self, problems, ws: torch.Tensor):
        self.n = len(problems)
        if self.n < 1:
            raise ValueError("CalibBatch: no problems")
        self.L = problems[0]["C"].shape[0]
        self.dt = problems[0]["rows_out"].dtype
        self.arr = (CalibProblem * self.n)()
        self.eigs = []
        for i, q in enumerate(problems):
            C, rows = q["C"], q["rows_out"]
            if (C.shape != (self.L, self.L) or C.dtype != torch.float32 or rows.shape[1] != self.L
                    or rows.dtype != self.dt):
                raise ValueError("CalibBatch: inconsistent shapes or dtypes")
            eig = (ctypes.c_double * rows.shape[0])()
            self.eigs.append(eig)
            prm = CalibParams(q.get("eps", 0.95), q.get("p", 0), q.get("r_override", 0),
                              int(bool(q.get("scale_on", True))), q.get("max_iter", 0),
                              q.get("tol", 0.0), 0)
            self.arr[i] = CalibProblem(_dev(C, "C"), 1, prm, _dev(rows, "rows_out"), rows.shape[0],
                                       ctypes.cast(eig, ctypes.POINTER(ctypes.c_double)), 0, 0, 0.0,
                                       0.0, 0)
        need = calib_batch_workspace_bytes(self.L, self.n)
        if ws.numel() * ws.element_size() < need:
            raise ValueError("CalibBatch: workspace too small")
        self.ws_ptr = _dev(ws, "ws")
        self.ws_bytes = ws.numel() * ws.element_size()
        self.dcode = dtype_code(self.dt)

    def solve(self, n_samples, warm_start: bool = False, r_override=None, stream=None):
        """Solves every problem (``n_samples[i]`` samples in statistic i);
        ``r_override``: optional per-problem overrides.  Returns the list of
        :class:`CalibResult`; raises on the first failing problem."""
        for i in range(self.n):
            q = self.arr[i]
            q.n_samples = int(n_samples[i])
            q.prm.warm_start = int(bool(warm_start))
            if r_override is not None:
                q.prm.r_override = int(r_override[i])
        st = lib().instant_calib_solve_batch(self.arr, self.n, self.L, self.dcode, self.ws_ptr,
                                             self.ws_bytes, _stream(stream))
        check(st, "instant_calib_solve_batch")
        return [CalibResult(self.arr[i].k, self.arr[i].R, self.arr[i].scale, self.arr[i].energy,
                            list(self.eigs[i])) for i in range(self.n)]


def reconstruction_error(t: torch.Tensor, Q: torch.Tensor, S: torch.Tensor, ws: torch.Tensor,
                         stream=None) -> tuple[float, float]:
    """``(sum_b ||t_b - Q^T S_b||^2, sum_b ||t_b||^2)`` for ``S = Q t`` per sample
    (t ``[B, L, C]``, Q ``[R, L]``, S ``[B*R, C]``); synchronises the stream.
    ``ws`` is at least 16 bytes of device scratch."""
    B, L, C = t.shape
    R = Q.shape[0]
    if Q.shape != (R, L) or S.shape != (B * R, C):
        raise ValueError("reconstruction_error: inconsistent shapes")
    _same_dtype(t.dtype, ("Q", Q), ("S", S))
    e2 = ctypes.c_double(0)
    n2 = ctypes.c_double(0)
    check(lib().instant_reconstruction_error(_dev(t, "t"), _dev(Q, "Q"), _dev(S, "S"), B, L, C, R,
                                             dtype_code(t.dtype), ctypes.byref(e2),
                                             ctypes.byref(n2), _dev(ws, "ws"),
                                             ws.numel() * ws.element_size(), _stream(stream)),
          "instant_reconstruction_error")
    return e2.value, n2.value


# --------------------------------------------------------------------------
# operators of an MLP block: norm, products with epilogues, 8-bit checkpoints
# --------------------------------------------------------------------------
def _ptr(t, shape, dt):
    """Device pointer of a contiguous CUDA tensor of this shape and dtype, None
    for None, -1 for anything else (the caller then finds out what is wrong; one
    token's call takes less time on the GPU than a full report's checks)."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.shape == shape and t.dtype is dt and t.is_cuda and t.is_contiguous():
        return t.data_ptr()
    return -1


def _matrix(where: str, name: str, t):
    """Shape of a matrix; anything else is refused."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 2:
        raise ValueError(f"{where}: {name} must be a matrix [rows, channels], got {list(t.shape)}")
    return t.shape


def _refuse(where: str, *wanted, ckpts=()):
    """Raises for the first of ``(name, tensor, shape, dtype)`` that is not what
    it should be: shapes and dtypes first, then device and layout."""
    for name, t, shape, dt in wanted:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.shape != shape:
            raise ValueError(f"{where}: {name} must be {list(shape)}, got {list(t.shape)}")
        _same_dtype(dt, (name, t))
    for q, s, rows, C, names in ckpts:
        _ckpt_refuse(where, rows, C, q, s, names)
    for name, t, _, _ in wanted:
        if t is not None:
            _dev(t, name)
    for q, s, _, _, names in ckpts:
        if q is not None:
            _dev(q, names[0])
            _dev(s, names[1])


def _ckpt_refuse(where: str, rows: int, C: int, q, s, names):
    if (q is None) != (s is None):
        raise ValueError(f"{where}: {names[0]} and {names[1]} come together")
    if q is None:
        return
    if q.shape != (rows, -(-C // 16) * 16) or s.shape != (-(-C // 128), rows):
        raise ValueError(f"{where}: a checkpoint of [{rows}, {C}] has {names[0]} "
                         f"[{rows}, {-(-C // 16) * 16}] and {names[1]} [{-(-C // 128)}, {rows}]")
    if q.dtype != torch.int8 or s.dtype != torch.uint8:
        raise TypeError(f"{where}: {names[0]} must be int8 and {names[1]} uint8")


def _ckpt_ptrs(rows: int, C: int, q, s):
    """Pointers of a checkpoint of ``[rows, C]``: both, (None, None), or a -1."""
    if q is None and s is None:
        return None, None
    if q is None or s is None:
        return -1, -1
    return _ptr(q, (rows, -(-C // 16) * 16), torch.int8), _ptr(s, (-(-C // 128), rows), torch.uint8)


def _act(act: str) -> int:
    if act not in ACTIVATIONS:
        raise ValueError(f"unknown activation {act!r}: use one of {sorted(ACTIVATIONS)}")
    return ACTIVATIONS[act]


def ckpt_buffers(rows: int, C: int, device):
    """Empty code and scale arrays of an 8-bit checkpoint of ``[rows, C]``:
    ``q`` int8 ``[rows, C rounded up to 16]``, ``s`` uint8 ``[ceil(C / 128), rows]``."""
    return (torch.empty(rows, -(-C // 16) * 16, dtype=torch.int8, device=device),
            torch.empty(-(-C // 128), rows, dtype=torch.uint8, device=device))


def ckpt_pack(x: torch.Tensor, q: torch.Tensor, s: torch.Tensor, stream=None):
    """The 8-bit checkpoint of x ``[rows, C]``; q, s from :func:`ckpt_buffers`."""
    rows, C = shape = _matrix("ckpt_pack", "x", x)
    px = _ptr(x, shape, x.dtype)
    pq, ps = _ckpt_ptrs(rows, C, q, s)
    if -1 in (px, pq, ps):
        _refuse("ckpt_pack", ("x", x, shape, x.dtype), ckpts=[(q, s, rows, C, ("q", "s"))])
    check(lib().instant_ckpt_pack(px, pq, ps, rows, C, dtype_code(x.dtype), _stream(stream)),
          "instant_ckpt_pack")
    return q, s


def ckpt_unpack(q: torch.Tensor, s: torch.Tensor, x: torch.Tensor, stream=None) -> torch.Tensor:
    """The values a checkpoint stands for, into x ``[rows, C]`` (exact in bf16)."""
    rows, C = shape = _matrix("ckpt_unpack", "x", x)
    px = _ptr(x, shape, x.dtype)
    pq, ps = _ckpt_ptrs(rows, C, q, s)
    if -1 in (px, pq, ps):
        _refuse("ckpt_unpack", ("x", x, shape, x.dtype), ckpts=[(q, s, rows, C, ("q", "s"))])
    check(lib().instant_ckpt_unpack(pq, ps, px, rows, C, dtype_code(x.dtype), _stream(stream)),
          "instant_ckpt_unpack")
    return x


def rms_norm(x: torch.Tensor, gamma: torch.Tensor, y: torch.Tensor | None, *,
             residual: torch.Tensor | None = None, h: torch.Tensor | None = None,
             q: torch.Tensor | None = None, s: torch.Tensor | None = None,
             r: torch.Tensor | None = None, eps: float = 1e-5, stream=None):
    """``h = x + residual``, ``r = rsqrt(mean(h^2) + eps)``, ``u = h r``,
    ``y = u gamma``; q, s take the 8-bit checkpoint of u and r ``[rows]`` fp32
    the factor (both for :func:`rms_norm_backward`).  Returns y."""
    rows, C = shape = _matrix("rms_norm", "x", x)
    dt = x.dtype
    p = (_ptr(x, shape, dt), _ptr(residual, shape, dt), _ptr(gamma, (C,), dt), _ptr(h, shape, dt),
         _ptr(y, shape, dt), *_ckpt_ptrs(rows, C, q, s), _ptr(r, (rows,), torch.float32))
    if -1 in p:
        _refuse("rms_norm", ("x", x, shape, dt), ("residual", residual, shape, dt), ("h", h, shape, dt),
                ("y", y, shape, dt), ("gamma", gamma, (C,), dt), ("r", r, (rows,), torch.float32),
                ckpts=[(q, s, rows, C, ("q", "s"))])
    check(lib().instant_rms_norm(*p, rows, C, eps, dtype_code(dt), _stream(stream)), "instant_rms_norm")
    return y


def rms_norm_backward_workspace(rows: int, C: int, device) -> torch.Tensor:
    n = lib().instant_rms_norm_backward_workspace_bytes(rows, C)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def rms_norm_backward(g_y: torch.Tensor, q: torch.Tensor, s: torch.Tensor, r: torch.Tensor,
                      gamma: torch.Tensor, gx: torch.Tensor, ggamma: torch.Tensor,
                      ws: torch.Tensor, *, residual: torch.Tensor | None = None,
                      accumulate: bool = False, stream=None):
    """Gradient of :func:`rms_norm` from the checkpoint of u: ``gx`` (with the
    gradient ``residual`` that bypassed the norm added) and ``ggamma`` ``[C]``
    fp32 (added to with ``accumulate``).  Returns ``(gx, ggamma)``."""
    rows, C = shape = _matrix("rms_norm_backward", "g_y", g_y)
    dt, f32 = g_y.dtype, torch.float32
    p = (_ptr(g_y, shape, dt), *_ckpt_ptrs(rows, C, q, s), _ptr(r, (rows,), f32), _ptr(gamma, (C,), dt),
         _ptr(residual, shape, dt), _ptr(gx, shape, dt), _ptr(ggamma, (C,), f32))
    if -1 in p:
        _refuse("rms_norm_backward", ("g_y", g_y, shape, dt), ("gx", gx, shape, dt),
                ("residual", residual, shape, dt), ("gamma", gamma, (C,), dt), ("r", r, (rows,), f32),
                ("ggamma", ggamma, (C,), f32), ckpts=[(q, s, rows, C, ("q", "s"))])
    check(lib().instant_rms_norm_backward(*p, int(accumulate), _dev(ws, "ws"),
                                          ws.numel() * ws.element_size(), rows, C, dtype_code(dt),
                                          _stream(stream)), "instant_rms_norm_backward")
    return gx, ggamma


def linear_act(x: torch.Tensor, w: torch.Tensor, y: torch.Tensor | None, *,
               bias: torch.Tensor | None = None, act: str = "none",
               residual: torch.Tensor | None = None, zq: torch.Tensor | None = None,
               zs: torch.Tensor | None = None, yq: torch.Tensor | None = None,
               ys: torch.Tensor | None = None, stream=None):
    """``z = x w^T + bias``, ``y = act(z) + residual``: x ``[rows, Cx]``, w ``[Cy, Cx]``,
    y ``[rows, Cy]``; zq, zs take the 8-bit checkpoint of z, yq, ys that of y.
    act: "none", "relu", "gelu" (erf form) or "silu".  Returns y."""
    rows, Cx = shape = _matrix("linear_act", "x", x)
    Cy = _matrix("linear_act", "w", w)[0]
    dt = x.dtype
    out = (rows, Cy)
    p = (_ptr(x, shape, dt), _ptr(w, (Cy, Cx), dt), _ptr(bias, (Cy,), dt), _ptr(residual, out, dt),
         _ptr(y, out, dt), *_ckpt_ptrs(rows, Cy, zq, zs), *_ckpt_ptrs(rows, Cy, yq, ys))
    if -1 in p:
        _refuse("linear_act", ("x", x, shape, dt), ("w", w, (Cy, Cx), dt), ("y", y, out, dt),
                ("residual", residual, out, dt), ("bias", bias, (Cy,), dt),
                ckpts=[(zq, zs, rows, Cy, ("zq", "zs")), (yq, ys, rows, Cy, ("yq", "ys"))])
    check(lib().instant_linear_act(*p, rows, Cx, Cy, _act(act), dtype_code(dt), _stream(stream)),
          "instant_linear_act")
    return y


def linear_act_grad(g_y: torch.Tensor, w: torch.Tensor, gx: torch.Tensor, *, act: str = "none",
                    zq: torch.Tensor | None = None, zs: torch.Tensor | None = None,
                    residual: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``gx = (g_y w) act'(z) + residual``: g_y ``[rows, Cy]``, w ``[Cy, Cx]``, gx
    ``[rows, Cx]``; zq, zs is the checkpoint of the activation's input z."""
    rows, Cy = shape = _matrix("linear_act_grad", "g_y", g_y)
    Cx = _matrix("linear_act_grad", "w", w)[1]
    dt = g_y.dtype
    out = (rows, Cx)
    p = (_ptr(g_y, shape, dt), _ptr(w, (Cy, Cx), dt), *_ckpt_ptrs(rows, Cx, zq, zs),
         _ptr(residual, out, dt), _ptr(gx, out, dt))
    if -1 in p:
        _refuse("linear_act_grad", ("g_y", g_y, shape, dt), ("w", w, (Cy, Cx), dt), ("gx", gx, out, dt),
                ("residual", residual, out, dt), ckpts=[(zq, zs, rows, Cx, ("zq", "zs"))])
    check(lib().instant_linear_act_grad(*p, rows, Cx, Cy, _act(act), dtype_code(dt), _stream(stream)),
          "instant_linear_act_grad")
    return gx


def ckpt_grad_w_workspace(rows: int, Cx: int, Cy: int, device) -> torch.Tensor:
    n = lib().instant_ckpt_grad_w_workspace_bytes(rows, Cx, Cy)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def ckpt_grad_w(g_y: torch.Tensor, q: torch.Tensor, s: torch.Tensor, gw: torch.Tensor,
                ws: torch.Tensor | None = None, *, gb: torch.Tensor | None = None,
                col_scale: torch.Tensor | None = None, accumulate: bool = False, stream=None):
    """``gw (+)= (g_y^T v) diag(col_scale)`` and ``gb (+)= sum over rows of g_y``, v the
    values of the checkpoint q, s of the layer's input: g_y ``[rows, Cy]``, gw
    ``[Cy, Cx]`` fp32, gb ``[Cy]`` fp32 (needs ws).  ws from
    :func:`ckpt_grad_w_workspace`; without gb it may be left out, and bf16 calls
    then allocate it.  Returns ``(gw, gb)``."""
    rows, Cy = shape = _matrix("ckpt_grad_w", "g_y", g_y)
    Cx = _matrix("ckpt_grad_w", "gw", gw)[1]
    dt, f32 = g_y.dtype, torch.float32
    if gb is not None and ws is None:
        raise ValueError("ckpt_grad_w: gb needs a workspace")
    p = (_ptr(g_y, shape, dt), *_ckpt_ptrs(rows, Cx, q, s), _ptr(col_scale, (Cx,), dt),
         _ptr(gw, (Cy, Cx), f32), _ptr(gb, (Cy,), f32))
    if -1 in p:
        _refuse("ckpt_grad_w", ("gw", gw, (Cy, Cx), f32), ("g_y", g_y, shape, dt),
                ("col_scale", col_scale, (Cx,), dt), ("gb", gb, (Cy,), f32),
                ckpts=[(q, s, rows, Cx, ("q", "s"))])
    if ws is None and dt == torch.bfloat16:
        # from the pool of the stream that uses it: a block freed on another stream may
        # still be in use there
        with _on_stream(stream):
            ws = ckpt_grad_w_workspace(rows, Cx, Cy, g_y.device)
    check(lib().instant_ckpt_grad_w(*p, int(accumulate), None if ws is None else _dev(ws, "ws"),
                                    0 if ws is None else ws.numel() * ws.element_size(), rows, Cx, Cy,
                                    dtype_code(dt), _stream(stream)), "instant_ckpt_grad_w")
    return gw, gb


# --------------------------------------------------------------------------
# the ends of a language model: embedding, token log probabilities, gradient norm
# --------------------------------------------------------------------------
_TOKEN_BYTES = {torch.int64: 8, torch.int32: 4}


def _vector(where: str, name: str, t):
    """Length of a vector; anything else is refused."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 1:
        raise ValueError(f"{where}: {name} must be a vector [rows], got {list(t.shape)}")
    return t.shape[0]


def _token_bytes(where: str, tokens) -> int:
    n = _TOKEN_BYTES.get(tokens.dtype)
    if n is None:
        raise TypeError(f"{where}: tokens must be int32 or int64, got {tokens.dtype}")
    return n


_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_DTYPE = {torch.float32: INSTANT_F32, torch.bfloat16: INSTANT_BF16}
_F32, _I64 = torch.float32, torch.int64


def _at(t, shape, dt, dev):
    """Device pointer of a contiguous tensor of this shape and dtype on device dev, None
    for None, -1 for anything else: small calls take longer here than on the GPU, so what
    is wrong is found out later, by :func:`_refuse_at`."""
    if t is None:
        return None
    try:
        if t.shape == shape and t.dtype is dt and t.get_device() == dev and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    return -1


def _refuse_at(where: str, dev: int, *wanted):
    """Raises for the first of ``(name, tensor, shape, dtype)`` that :func:`_at` answered -1 for."""
    _refuse(where, *wanted)
    for name, t, _, _ in wanted:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{where}: {name} is on {t.device}, others on device {dev}")


def _launch_on(where: str, stream, dev: int) -> int:
    """The handle of the stream on the tensors' device, which has to be the current one."""
    if dev != _device():
        raise ValueError(f"{where}: tensors on device {dev}, but the current device is {_device()}")
    return _raw_stream(dev) if stream is None and _raw_stream is not None else _stream(stream)


def embed(tokens: torch.Tensor, table: torch.Tensor, y: torch.Tensor, *, scale: float = 1.0,
          stream=None) -> torch.Tensor:
    """``y[i] = scale * table[tokens[i]]``, zeros for a negative token: tokens ``[rows]``
    int32 or int64, table ``[V, C]``, y ``[rows, C]``."""
    try:
        (rows,), (V, C), dt, dev = tokens.shape, table.shape, table.dtype, table.get_device()
        n, dc = _TOKEN_BYTES[tokens.dtype], _DTYPE[dt]
    except (AttributeError, KeyError, ValueError):
        _vector("embed", "tokens", tokens)
        _matrix("embed", "table", table)
        _token_bytes("embed", tokens)
        dtype_code(table.dtype)
        raise
    pt, pe, py = (_at(tokens, (rows,), tokens.dtype, dev), _at(table, (V, C), dt, dev), _at(y, (rows, C), dt, dev))
    if dev < 0 or -1 in (pt, pe, py) or y is None:
        _refuse_at("embed", dev, ("table", table, (V, C), dt), ("y", y, (rows, C), dt),
                   ("tokens", tokens, (rows,), tokens.dtype))
        raise TypeError("y must be a torch.Tensor")
    check(lib().instant_embed(pt, n, pe, py, rows, V, C, scale, dc, _launch_on("embed", stream, dev)),
          "instant_embed")
    return y


def embed_grad_workspace(rows: int, V: int, C: int, device) -> torch.Tensor:
    n = lib().instant_embed_grad_workspace_bytes(rows, V, C)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def embed_grad(g_y: torch.Tensor, tokens: torch.Tensor, gtable: torch.Tensor, ws: torch.Tensor, *,
               scale: float = 1.0, accumulate: bool = False, stream=None) -> torch.Tensor:
    """``gtable[v] (+)= scale * sum of g_y[i]`` over the i with ``tokens[i] = v``: g_y
    ``[rows, C]``, gtable ``[V, C]`` fp32; ws from :func:`embed_grad_workspace`."""
    try:
        (rows, C), (V, _), dt, dev = g_y.shape, gtable.shape, g_y.dtype, g_y.get_device()
        n, dc = _TOKEN_BYTES[tokens.dtype], _DTYPE[dt]
    except (AttributeError, KeyError, ValueError):
        _matrix("embed_grad", "g_y", g_y)
        _matrix("embed_grad", "gtable", gtable)
        _vector("embed_grad", "tokens", tokens)
        _token_bytes("embed_grad", tokens)
        dtype_code(g_y.dtype)
        raise
    pg, pt, po = (_at(g_y, (rows, C), dt, dev), _at(tokens, (rows,), tokens.dtype, dev), _at(gtable, (V, C), _F32, dev))
    if dev < 0 or -1 in (pg, pt, po):
        _vector("embed_grad", "tokens", tokens)
        _refuse_at("embed_grad", dev, ("tokens", tokens, (rows,), tokens.dtype), ("gtable", gtable, (V, C), _F32),
                   ("g_y", g_y, (rows, C), dt))
    pw = _dev(ws, "ws")
    if ws.get_device() != dev:
        raise ValueError(f"embed_grad: ws is on {ws.device}, others on device {dev}")
    check(lib().instant_embed_grad(pg, pt, n, po, int(accumulate), pw, ws.numel() * ws.element_size(), rows, V, C,
                                   scale, dc, _launch_on("embed_grad", stream, dev)), "instant_embed_grad")
    return gtable


def _vocab(where: str, ld: int, vocab) -> int:
    if vocab is None:
        return ld
    if not 1 <= vocab <= ld:
        raise ValueError(f"{where}: a vocabulary of {vocab} in rows of {ld} logits")
    return vocab


def _alternatives(where: str, name: str, t, V: int, other: int) -> int:
    k = _matrix(where, name, t)[1]
    if not 1 <= k <= min(TOP_MAX, V) or other not in (0, k):
        raise ValueError(f"{where}: {name} [rows, k] takes 1 to {min(TOP_MAX, V)} alternatives, as many as the "
                         f"other one, got {k}")
    return k


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor | None, logp: torch.Tensor | None, *,
                   vocab: int | None = None, scale: float = 1.0, stats: torch.Tensor | None = None,
                   entropy: torch.Tensor | None = None, top_ids: torch.Tensor | None = None,
                   top_logp: torch.Tensor | None = None, stream=None):
    """Log probabilities of the rows' tokens under ``softmax(scale * logits[:, :vocab])``:
    logits ``[rows, ld]``, tokens ``[rows]`` int32 or int64 (negative: none, its logp is
    0), logp ``[rows]`` fp32; scale within 2^-120 .. 2^120.  Optional outputs: stats ``[rows, 2]`` (for
    :func:`token_logprobs_grad`) and entropy ``[rows]`` fp32, top_ids ``[rows, k]`` int64
    and top_logp ``[rows, k]`` fp32 of the k <= 32 likeliest tokens, ties by lower index.
    Returns logp."""
    where = "token_logprobs"
    try:
        rows, ld = shape = logits.shape
        dt, dev = logits.dtype, logits.get_device()
        n, dc = 8 if tokens is None else _TOKEN_BYTES[tokens.dtype], _DTYPE[dt]
    except (AttributeError, KeyError, ValueError):
        _matrix(where, "logits", logits)
        if tokens is not None:
            _vector(where, "tokens", tokens)
            _token_bytes(where, tokens)
        dtype_code(logits.dtype)
        raise
    V = _vocab(where, ld, vocab)
    if tokens is None and logp is not None:
        raise ValueError(f"{where}: logp needs tokens")
    top, one = 0, (rows,)
    if top_ids is not None:
        top = _alternatives(where, "top_ids", top_ids, V, top)
    if top_logp is not None:
        top = _alternatives(where, "top_logp", top_logp, V, top)
    p = (_at(logits, shape, dt, dev), None if tokens is None else _at(tokens, one, tokens.dtype, dev),
         _at(logp, one, _F32, dev), _at(stats, (rows, 2), _F32, dev), _at(entropy, one, _F32, dev),
         _at(top_ids, (rows, top), _I64, dev), _at(top_logp, (rows, top), _F32, dev))
    if dev < 0 or -1 in p:
        if tokens is not None:
            _vector(where, "tokens", tokens)
        _refuse_at(where, dev, ("logp", logp, one, _F32), ("stats", stats, (rows, 2), _F32),
                   ("entropy", entropy, one, _F32), ("top_ids", top_ids, (rows, top), _I64),
                   ("top_logp", top_logp, (rows, top), _F32), ("logits", logits, shape, dt),
                   *(() if tokens is None else (("tokens", tokens, one, tokens.dtype),)))
    check(lib().instant_token_logprobs(p[0], p[1], n, p[2], p[3], p[4], p[5], p[6], rows, V, ld, top, scale, dc,
                                       _launch_on(where, stream, dev)), "instant_token_logprobs")
    return logp


def token_logprobs_grad(logits: torch.Tensor, tokens: torch.Tensor | None, stats: torch.Tensor,
                        g_logits: torch.Tensor, *, vocab: int | None = None, scale: float = 1.0,
                        g_logp: torch.Tensor | None = None, g_entropy: torch.Tensor | None = None,
                        entropy: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Gradient of :func:`token_logprobs`'s logp (times g_logp ``[rows]`` fp32) and entropy
    (times g_entropy ``[rows]``, with the forward's entropy) into g_logits ``[rows, ld]``,
    which may be logits; zero past ``vocab``."""
    where = "token_logprobs_grad"
    try:
        rows, ld = shape = logits.shape
        dt, dev = logits.dtype, logits.get_device()
        n, dc = 8 if tokens is None else _TOKEN_BYTES[tokens.dtype], _DTYPE[dt]
    except (AttributeError, KeyError, ValueError):
        _matrix(where, "logits", logits)
        if tokens is not None:
            _vector(where, "tokens", tokens)
            _token_bytes(where, tokens)
        dtype_code(logits.dtype)
        raise
    V = _vocab(where, ld, vocab)
    if (g_entropy is None) != (entropy is None):
        raise ValueError(f"{where}: g_entropy and entropy come together")
    if g_logp is None and g_entropy is None or g_logp is not None and tokens is None:
        raise ValueError(f"{where}: give g_logp with tokens, or g_entropy with entropy, or all")
    one = (rows,)
    p = (_at(logits, shape, dt, dev), None if tokens is None else _at(tokens, one, tokens.dtype, dev),
         _at(stats, (rows, 2), _F32, dev), _at(g_logp, one, _F32, dev), _at(g_entropy, one, _F32, dev),
         _at(entropy, one, _F32, dev), _at(g_logits, shape, dt, dev))
    if dev < 0 or -1 in p or stats is None or g_logits is None:
        if tokens is not None:
            _vector(where, "tokens", tokens)
        _refuse_at(where, dev, ("stats", stats, (rows, 2), _F32), ("g_logits", g_logits, shape, dt),
                   ("g_logp", g_logp, one, _F32), ("g_entropy", g_entropy, one, _F32),
                   ("entropy", entropy, one, _F32), ("logits", logits, shape, dt),
                   *(() if tokens is None else (("tokens", tokens, one, tokens.dtype),)))
        raise TypeError("stats and g_logits must be torch.Tensor")
    check(lib().instant_token_logprobs_grad(p[0], p[1], n, p[2], p[3], p[4], p[5], p[6], rows, V, ld, scale, dc,
                                            _launch_on(where, stream, dev)), "instant_token_logprobs_grad")
    return g_logits


def _ptrs(tensors):
    return list(map(torch.Tensor.data_ptr, tensors))


def _clip_ptrs(grads, outs):
    """The pointers of both lists if all tensors are right for :class:`GradClip` and none shares
    memory with another, else None: seen list by list (a GradClip of 400 gradients is made in 240 us
    in place and 470 with other outputs, with a look at one tensor after the other in some 850)."""
    try:
        dev, dts, nbytes = grads[0].get_device(), [g.dtype for g in grads], [g.nbytes for g in grads]
        at = to = all_at = _ptrs(grads)
        lists = (grads,)
        if outs is not grads:
            if [o.dtype for o in outs] != dts or [o.shape for o in outs] != [g.shape for g in grads]:
                return None
            to = _ptrs(outs)
            all_at, nbytes, lists = at + to, nbytes * 2, (grads, outs)
        for tensors in lists:
            if set(map(torch.Tensor.get_device, tensors)) != {dev} \
                    or not all(map(torch.Tensor.is_contiguous, tensors)):
                return None
    except (AttributeError, TypeError):
        return None
    # disjoint if no tensor starts, in the order of addresses, before as many as lie below have ended
    starts, ends = sorted(all_at), sorted(map(operator.add, all_at, nbytes))
    if dev < 0 or not set(dts) <= _DTYPE.keys() or any(map(operator.lt, starts[1:], ends)):
        return None
    return at, to


def _refuse_clip(grads, outs):
    """Raises for the first tensor that :class:`GradClip` can't take, or for two that share
    memory one of them is written in; returns where nothing is wrong."""
    if not isinstance(grads[0], torch.Tensor):
        raise TypeError("grads[0] must be a torch.Tensor")
    dev, spans = grads[0].device, []
    for i, (g, o) in enumerate(zip(grads, outs)):
        a, n, dt = _dev(g, f"grads[{i}]"), g.numel(), g.dtype
        b = a if o is g else _dev(o, f"outs[{i}]")
        if o.shape != g.shape or o.dtype != dt:
            raise ValueError(f"GradClip: outs[{i}] must be {list(g.shape)} of {dt}")
        if g.device != dev or o.device != dev:
            raise ValueError(f"GradClip: grads[{i}] or outs[{i}] is not on {dev}, as the others are")
        dtype_code(dt)
        # an output is alone in its memory; gradients that are only read may overlap
        if n:
            n *= g.element_size()
            spans.append((a, a + n, a == b, i))
            if a != b:
                spans.append((b, b + n, True, i))
    spans.sort()
    end, written, at = 0, False, 0
    for a, b, w, i in spans:
        if a >= end:
            end, written, at = b, w, i
        elif w or written:
            raise ValueError(f"GradClip: tensors {at} and {i} share memory that is written")
        elif b > end:
            end, at = b, i


class GradClip:
    """The gradients of a model as one list: a call takes their common norm and clips
    them by it, in place or into ``outs`` (of the same shapes and dtypes).  The argument
    block and the workspace are made once (of 400 gradients in 240 us, with other outputs
    in 470), so the tensors given here must stay alive and in place; a call belongs to one
    stream at a time."""

    def __init__(self, grads, outs=None):
        grads = list(grads)
        outs = grads if outs is None else list(outs)
        if not grads or len(outs) != len(grads):
            raise ValueError("GradClip: a list of gradients, and as many outs")
        ptrs = _clip_ptrs(grads, outs)
        if ptrs is None:
            _refuse_clip(grads, outs)
            ptrs = _ptrs(grads), _ptrs(outs)
        words = array.array("q", bytes(32 * len(grads)))  # four words an item, see GradItem
        for i, column in enumerate((*ptrs, map(torch.Tensor.numel, grads), [_DTYPE[g.dtype] for g in grads])):
            words[i::4] = array.array("q", column)
        self.words = (ctypes.c_longlong * len(words)).from_buffer(words)
        self.arr = ctypes.cast(self.words, ctypes.POINTER(GradItem))
        self.count = len(grads)
        self.device = grads[0].device
        self.grads, self.outs = grads, outs
        n = lib().instant_grad_clip_workspace_bytes(len(grads))
        self.ws = torch.empty(n, dtype=torch.uint8, device=self.device)
        self.ws_ptr, self.ws_bytes = self.ws.data_ptr(), n

    def __call__(self, max_norm: float, norm: torch.Tensor, *, scale: float = 1.0, stream=None) -> torch.Tensor:
        """``norm`` ``[2]`` fp32 gets ``scale * (sum of g^2)^(1/2)`` and the factor
        ``min(1, max_norm / norm)`` (1 where the norm is not finite); the outputs are
        ``g * scale * factor``.  Returns norm."""
        dev = self.device.index
        p = _at(norm, (2,), _F32, dev)
        if p is None or p == -1:
            _refuse_at("GradClip", dev, ("norm", norm, (2,), _F32))
            raise TypeError("norm must be a torch.Tensor")
        check(lib().instant_grad_clip(self.arr, self.count, max_norm, scale, p, self.ws_ptr, self.ws_bytes,
                                      _launch_on("GradClip", stream, dev)), "instant_grad_clip")
        return norm


def grad_clip(grads, max_norm: float, norm: torch.Tensor, *, outs=None, scale: float = 1.0,
              stream=None) -> torch.Tensor:
    """One call of a :class:`GradClip` that is not kept; a program whose gradients stay in place
    keeps one, as making it takes longer than the call."""
    with _on_stream(stream):  # the workspace comes from the pool of the stream that uses it
        clip = GradClip(grads, outs)
    return clip(max_norm, norm, scale=scale, stream=stream)


def device_status(clear: bool = True, stream=None) -> int:
    """Sticky device-side status (0 when no bounded wait ran out and no token lay past
    its table)."""
    return int(lib().instant_device_status(int(clear), _stream(stream)))
