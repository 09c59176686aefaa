"""ParaGRU / ParaLSTM parallel-in-time Newton solve for B200 (sm_100a).

Thin ctypes binding over ``libpararnn.so`` (C ABI: ``include/pararnn.h``).
The functions named ``pararnn_*`` mirror the C entry points one to one and
only marshal arguments: torch tensors are passed as device pointers, the
current torch CUDA stream is used unless one is given, and a negative return
code raises :class:`PararnnError`.  Every step of the solve runs in the CUDA
kernels; there is no CPU fallback.  If the shared library has not been built
(``python -m nonlinear_rnn_paragru_b200.build``) the first call raises.

Convenience wrappers (:func:`gru_solve`, :func:`lstm_solve`, :func:`adjoint`)
allocate outputs, stats and workspace with torch and call the same entry
points.  Beside the nonlinear solves stand the gated linear recurrence
(:func:`linrec_solve`, :func:`linrec_adjoint`, :func:`linrec_step`) and the
norms around a block (:func:`block_norm`, :func:`block_norm_adjoint`).
"""
import contextlib
import ctypes
import os

import torch

__all__ = [
    "PARARNN_F32", "PARARNN_BF16", "PARARNN_GRU", "PARARNN_LSTM",
    "PararnnOpts", "PararnnError", "library_path", "load_library",
    "pararnn_workspace_size", "pararnn_workspace_init", "pararnn_gru_solve",
    "pararnn_lstm_solve", "pararnn_adjoint", "pararnn_adjoint_ex", "pararnn_adjoint_noalloc",
    "pararnn_seq_baseline", "pararnn_gru_step", "pararnn_lstm_step",
    "pararnn_unfused_workspace_size", "pararnn_solve_unfused", "solve_unfused",
    "pararnn_dense_workspace_size", "pararnn_dense_gru_solve", "dense_gru_solve",
    "pararnn_dense_matmul",
    "pararnn_shard_workspace_size", "pararnn_shard_eval", "pararnn_shard_combine",
    "pararnn_shard_apply",
    "pararnn_strerror", "gru_solve", "lstm_solve", "adjoint", "seq_baseline",
    "gru_step", "lstm_step",
    "PARARNN_LIN_GRU", "PARARNN_LIN_DECAY", "PARARNN_ACT_SILU", "PARARNN_ACT_SIGMOID",
    "pararnn_linrec_solve", "pararnn_linrec_workspace_size", "pararnn_linrec_adjoint",
    "pararnn_linrec_solve_ex", "pararnn_linrec_adjoint_ex", "pararnn_linrec_step", "linrec_solve",
    "linrec_adjoint", "linrec_step",
    "pararnn_block_norm", "pararnn_block_norm_workspace_size", "pararnn_block_norm_adjoint",
    "pararnn_block_norm_adjoint_ex", "block_norm", "block_norm_adjoint",
    "Workspace", "read_stats",
]

PARARNN_F32, PARARNN_BF16 = 0, 1
PARARNN_GRU, PARARNN_LSTM = 0, 1
PARARNN_LIN_GRU, PARARNN_LIN_DECAY = 2, 3
PARARNN_ACT_SILU, PARARNN_ACT_SIGMOID = 0, 1
PARARNN_FLAG_INJECT_WITHHOLD = 1
PARARNN_FLAG_FORCE_CHUNKED = 2
PARARNN_FLAG_FORCE_ROW = 4
PARARNN_FLAG_DENSE_SIMT = 8
PARARNN_FLAG_EXACT_STEPS = 16
STATUS_NAMES = {0: "converged", 1: "not_converged", 2: "nonfinite", 3: "timeout"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


class PararnnError(RuntimeError):
    def __init__(self, code, what):
        super().__init__(f"{what}: pararnn error {code} "
                         f"({pararnn_strerror(code) if _LIB else '?'})")
        self.code = code


class PararnnOpts(ctypes.Structure):
    _fields_ = [("tol", ctypes.c_float), ("max_iters", ctypes.c_int),
                ("flags", ctypes.c_uint), ("inject_chunk", ctypes.c_int),
                ("timeout_us", ctypes.c_uint), ("max_cluster", ctypes.c_int),
                ("chan_iters", ctypes.c_void_p)]


def library_path() -> str:
    return os.path.join(_HERE, "libpararnn.so")


def load_library():
    """Load the CUDA library (raises if it is missing: no fallback)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise ImportError(
            f"{path} is missing; build it with "
            "`python -m nonlinear_rnn_paragru_b200.build` (nvcc, sm_100a)")
    lib = ctypes.CDLL(path)
    vp, fp, ip = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
    i, sz = ctypes.c_int, ctypes.c_size_t
    ll, fl = ctypes.c_longlong, ctypes.c_float
    op = ctypes.POINTER(PararnnOpts)
    sigs = {
        "pararnn_workspace_size": (sz, [i, i, i, i, i, i]),
        "pararnn_workspace_init": (i, [vp, sz, vp]),
        "pararnn_gru_solve": (i, [vp, i, fp, fp, fp, fp, i, i, i, op, vp, ip,
                                  vp, sz, vp]),
        "pararnn_lstm_solve": (i, [vp, i, fp, fp, fp, fp, fp, fp, i, i, i, op,
                                   vp, ip, vp, sz, vp]),
        "pararnn_adjoint": (i, [i, vp, i, fp, fp, fp, fp, fp, fp, fp, fp, fp,
                                fp, fp, fp, i, i, i, ip, vp, sz, vp]),
        "pararnn_seq_baseline": (i, [i, vp, i, fp, fp, fp, fp, fp, fp, i, i,
                                     i, vp]),
        "pararnn_adjoint_ex": (i, [i, vp, i, fp, fp, fp, fp, fp, fp, fp, fp, fp,
                                   fp, fp, fp, i, i, i, ip, vp, sz, op, vp]),
        "pararnn_adjoint_noalloc": (i, [i, vp, i, fp, fp, fp, fp, fp, fp, fp,
                                        fp, fp, fp, fp, fp, i, i, i, ip, vp]),
        "pararnn_unfused_workspace_size": (sz, [i, i, i, i]),
        "pararnn_solve_unfused": (i, [i, vp, i, fp, fp, fp, fp, fp, fp, i, i, i,
                                      op, vp, vp, sz, vp]),
        "pararnn_dense_workspace_size": (sz, [i, i, i]),
        "pararnn_dense_matmul": (i, [fp, fp, fp, i, i, i, i, i, ip, vp]),
        "pararnn_dense_gru_solve": (i, [vp, i, fp, fp, fp, fp, i, i, i, op, vp, vp,
                                        sz, vp]),
        "pararnn_shard_workspace_size": (sz, [i, i, i, i]),
        "pararnn_shard_eval": (i, [i, vp, i, fp, fp, fp, fp, fp, fp, i, i, i, fp, fp, fp,
                                   vp, sz, vp]),
        "pararnn_shard_combine": (i, [i, fp, fp, i, i, i, i, fp, fp, vp]),
        "pararnn_shard_apply": (i, [i, fp, fp, fp, i, i, i, vp, sz, vp]),
        "pararnn_gru_step": (i, [vp, i, fp, fp, fp, fp, i, i, vp]),
        "pararnn_lstm_step": (i, [vp, i, fp, fp, fp, fp, fp, fp, i, i, vp]),
        "pararnn_linrec_solve": (i, [i, vp, i, ll, ll, ll, fp, fp, fp, vp, fp, i, i, i, fl, vp]),
        "pararnn_linrec_solve_ex": (i, [i, vp, i, ll, ll, ll, fp, fp, fp, vp, fp, i, i, i, fl, ip, op,
                                        vp]),
        "pararnn_linrec_workspace_size": (sz, [i, i, i, i]),
        "pararnn_linrec_adjoint": (i, [i, vp, i, ll, ll, ll, fp, fp, fp, vp, fp, fp, vp, i, fp, fp,
                                       fp, i, i, i, fl, vp, sz, vp]),
        "pararnn_linrec_adjoint_ex": (i, [i, vp, i, ll, ll, ll, fp, fp, fp, vp, fp, fp, vp, i, fp, fp,
                                          fp, i, i, i, fl, ip, vp, sz, op, vp]),
        "pararnn_linrec_step": (i, [i, vp, i, ll, ll, fp, fp, fp, fp, i, i, fl, vp]),
        "pararnn_block_norm": (i, [vp, i, ll, vp, i, ll, i, fp, vp, i, ll, fp, fp, vp, i, vp, i, fl,
                                   ll, i, vp]),
        "pararnn_block_norm_workspace_size": (sz, [ll, i]),
        "pararnn_block_norm_adjoint": (i, [vp, i, ll, vp, i, ll, i, fp, vp, i, ll, fp, fp, vp, i, ll,
                                           vp, i, ll, vp, vp, vp, fp, fp, fp, fl, ll, i, vp, sz, vp]),
        "pararnn_block_norm_adjoint_ex": (i, [vp, i, ll, vp, i, ll, i, fp, vp, i, ll, fp, fp, vp, i, ll,
                                              vp, i, ll, vp, vp, vp, fp, fp, fp, fl, ll, i, ip, vp, sz,
                                              op, vp]),
        "pararnn_strerror": (ctypes.c_char_p, [i]),
    }
    for name, (res, args) in sigs.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = lib
    return lib


# ------------------------------------------------------------ marshalling --
def _ptr(t, dtype=torch.float32):
    """Device pointer of a contiguous CUDA tensor of `dtype` (None -> NULL)."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("pararnn expects contiguous CUDA tensors")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"pararnn expects {dtype}, got {t.dtype}")
    return t.data_ptr()


def _uptr(u):
    return _ptr(u, None)


def _iptr(t):
    return _ptr(t, torch.int32)


def _wptr(t):
    return _ptr(t, None)


def _mptr(t):
    """Device pointer of a mask of bytes: elements of any other size would be
    read as several."""
    if t is not None and not isinstance(t, int) and t.dtype not in (torch.bool, torch.uint8):
        raise TypeError(f"pararnn expects a mask of torch.bool or torch.uint8, got {t.dtype}")
    return _ptr(t, None)


def _stream(stream):
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(u):
    if u.dtype == torch.bfloat16:
        return PARARNN_BF16
    if u.dtype == torch.float32:
        return PARARNN_F32
    return -1  # let the library reject it


def _check(rc, what):
    if rc != 0:
        raise PararnnError(rc, what)


def _opts(tol=1e-6, max_iters=0, flags=0, inject_chunk=-1, timeout_us=0,
          max_cluster=0, chan_iters=None):
    return PararnnOpts(float(tol), int(max_iters), int(flags), int(inject_chunk),
                       int(timeout_us), int(max_cluster), _iptr(chan_iters))


# ------------------------------------------------------------ C entry points --
def pararnn_workspace_size(cell, B, T, D, max_iters=0, adjoint=0) -> int:
    return int(load_library().pararnn_workspace_size(cell, B, T, D, max_iters,
                                                     adjoint))


def pararnn_workspace_init(workspace, stream=None):
    _check(load_library().pararnn_workspace_init(
        _wptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), "pararnn_workspace_init")


def pararnn_gru_solve(u, a, bias, h0, h, opts, stats, iter_hist, workspace,
                      stream=None):
    _check(load_library().pararnn_gru_solve(
        _uptr(u), _dtype_code(u), _ptr(a), _ptr(bias), _ptr(h0), _ptr(h),
        u.shape[0], u.shape[1], u.shape[3], ctypes.byref(opts), _iptr(stats),
        _iptr(iter_hist), _wptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "pararnn_gru_solve")


def pararnn_lstm_solve(u, a, bias, c0, h0, c, h, opts, stats, iter_hist,
                       workspace, stream=None):
    _check(load_library().pararnn_lstm_solve(
        _uptr(u), _dtype_code(u), _ptr(a), _ptr(bias), _ptr(c0), _ptr(h0),
        _ptr(c), _ptr(h), u.shape[0], u.shape[1], u.shape[3],
        ctypes.byref(opts), _iptr(stats), _iptr(iter_hist), _wptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "pararnn_lstm_solve")


def pararnn_adjoint(cell, u, a, bias, c0, h0, c, h, dLdh, du, da, dbias, dc0,
                    dh0, status, workspace, stream=None):
    _check(load_library().pararnn_adjoint(
        cell, _uptr(u), _dtype_code(u), _ptr(a), _ptr(bias), _ptr(c0),
        _ptr(h0), _ptr(c), _ptr(h), _ptr(dLdh), _ptr(du), _ptr(da),
        _ptr(dbias), _ptr(dc0), _ptr(dh0), u.shape[0], u.shape[1], u.shape[3],
        _iptr(status), _wptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "pararnn_adjoint")


def pararnn_adjoint_ex(cell, u, a, bias, c0, h0, c, h, dLdh, du, da, dbias, dc0,
                       dh0, status, workspace, opts, stream=None):
    _check(load_library().pararnn_adjoint_ex(
        cell, _uptr(u), _dtype_code(u), _ptr(a), _ptr(bias), _ptr(c0),
        _ptr(h0), _ptr(c), _ptr(h), _ptr(dLdh), _ptr(du), _ptr(da),
        _ptr(dbias), _ptr(dc0), _ptr(dh0), u.shape[0], u.shape[1], u.shape[3],
        _iptr(status), _wptr(workspace),
        workspace.numel() * workspace.element_size(),
        ctypes.byref(opts) if opts is not None else None, _stream(stream)),
        "pararnn_adjoint_ex")


def pararnn_adjoint_noalloc(cell, u, a, bias, c0, h0, c, h, dLdh, du, da, dbias,
                            dc0, dh0, status, stream=None):
    """pararnn_adjoint with the library's built-in scratch instead of a
    workspace: for callers that cannot provide device scratch memory."""
    _check(load_library().pararnn_adjoint_noalloc(
        cell, _uptr(u), _dtype_code(u), _ptr(a), _ptr(bias), _ptr(c0),
        _ptr(h0), _ptr(c), _ptr(h), _ptr(dLdh), _ptr(du), _ptr(da),
        _ptr(dbias), _ptr(dc0), _ptr(dh0), u.shape[0], u.shape[1], u.shape[3],
        _iptr(status), _stream(stream)), "pararnn_adjoint_noalloc")


def pararnn_seq_baseline(cell, u, a, bias, c0, h0, c, h, stream=None):
    _check(load_library().pararnn_seq_baseline(
        cell, _uptr(u), _dtype_code(u), _ptr(a), _ptr(bias), _ptr(c0),
        _ptr(h0), _ptr(c), _ptr(h), u.shape[0], u.shape[1], u.shape[3],
        _stream(stream)), "pararnn_seq_baseline")


def pararnn_unfused_workspace_size(cell, B, T, D) -> int:
    return int(load_library().pararnn_unfused_workspace_size(cell, B, T, D))


def pararnn_solve_unfused(cell, u, a, bias, c0, h0, c, h, opts, stats, workspace,
                          stream=None):
    _check(load_library().pararnn_solve_unfused(
        cell, _uptr(u), _dtype_code(u), _ptr(a), _ptr(bias), _ptr(c0), _ptr(h0),
        _ptr(c), _ptr(h), u.shape[0], u.shape[1], u.shape[3], ctypes.byref(opts),
        _iptr(stats), _wptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "pararnn_solve_unfused")


def pararnn_dense_matmul(A, Bm, C, store_mode, err, stream=None):
    """C[z] = A[z] @ Bm[z].T on the tensor cores (tf32 products, fp32 sums):
    A [Z, M, K], Bm [Z, N, K], C [Z, M, N] (or [Z, N, M] transposed per
    store_mode), err int32 [1]."""
    Z, M, K = A.shape
    N = Bm.shape[1]
    _check(load_library().pararnn_dense_matmul(
        _ptr(A), _ptr(Bm), _ptr(C), M, N, K, Z, int(store_mode), _iptr(err), _stream(stream)),
        "pararnn_dense_matmul")


def pararnn_dense_workspace_size(B, T, D) -> int:
    return int(load_library().pararnn_dense_workspace_size(B, T, D))


def pararnn_dense_gru_solve(u, W, bias, h0, h, opts, stats, workspace, stream=None):
    _check(load_library().pararnn_dense_gru_solve(
        _uptr(u), _dtype_code(u), _ptr(W), _ptr(bias), _ptr(h0), _ptr(h), u.shape[0],
        u.shape[1], u.shape[3], ctypes.byref(opts), _iptr(stats), _wptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "pararnn_dense_gru_solve")


def pararnn_shard_workspace_size(cell, B, Ts, D) -> int:
    return int(load_library().pararnn_shard_workspace_size(cell, B, Ts, D))


def pararnn_shard_eval(cell, u, a, bias, c_bound, h_bound, c, h, agg, last, rmax, workspace,
                       stream=None):
    _check(load_library().pararnn_shard_eval(
        cell, _uptr(u), _dtype_code(u), _ptr(a), _ptr(bias), _ptr(c_bound), _ptr(h_bound),
        _ptr(c), _ptr(h), u.shape[0], u.shape[1], u.shape[3], _ptr(agg), _ptr(last),
        _ptr(rmax), _wptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)), "pararnn_shard_eval")


def pararnn_shard_combine(cell, aggs, lasts, r, din, bound, stream=None):
    W, _, B, D = aggs.shape
    _check(load_library().pararnn_shard_combine(
        cell, _ptr(aggs), _ptr(lasts), W, r, B, D, _ptr(din), _ptr(bound), _stream(stream)),
        "pararnn_shard_combine")


def pararnn_shard_apply(cell, din, c, h, workspace, stream=None):
    B, Ts, D = h.shape
    _check(load_library().pararnn_shard_apply(
        cell, _ptr(din), _ptr(c), _ptr(h), B, Ts, D, _wptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)), "pararnn_shard_apply")


def pararnn_gru_step(u_t, a, bias, h_prev, h_next, stream=None):
    _check(load_library().pararnn_gru_step(
        _uptr(u_t), _dtype_code(u_t), _ptr(a), _ptr(bias), _ptr(h_prev),
        _ptr(h_next), u_t.shape[0], u_t.shape[2], _stream(stream)),
        "pararnn_gru_step")


def pararnn_lstm_step(u_t, a, bias, c_prev, h_prev, c_next, h_next, stream=None):
    _check(load_library().pararnn_lstm_step(
        _uptr(u_t), _dtype_code(u_t), _ptr(a), _ptr(bias), _ptr(c_prev),
        _ptr(h_prev), _ptr(c_next), _ptr(h_next), u_t.shape[0], u_t.shape[2],
        _stream(stream)), "pararnn_lstm_step")


def pararnn_strerror(code) -> str:
    return load_library().pararnn_strerror(int(code)).decode()


# --------------------------------------------------------------- wrappers --
class Workspace:
    """A zero-initialised device workspace that grows on demand."""

    def __init__(self, device="cuda"):
        self.device = device
        self.buf = None

    def get(self, nbytes, stream=None):
        nbytes = max(int(nbytes), 256)
        if self.buf is None or self.buf.numel() < nbytes:
            self.buf = torch.empty(nbytes, dtype=torch.uint8, device=self.device)
            pararnn_workspace_init(self.buf, stream)
        return self.buf


def read_stats(stats) -> dict:
    s = stats.cpu()
    return {"iters": int(s[0]), "max_residual": float(s[1:2].view(torch.float32)[0]),
            "status": STATUS_NAMES.get(int(s[2]), int(s[2])), "evals": int(s[3])}


def _new_stats(device):
    return torch.zeros(4, dtype=torch.int32, device=device)


def gru_solve(u, a, bias=None, h0=None, *, tol=1e-6, max_iters=64, hist=False,
              workspace=None, h=None, stats=None, stream=None, opts=None,
              max_cluster=0, flags=0, chan_iters=None):
    """ParaGRU solve -> (h, stats, iter_hist or None).  `chan_iters`: an
    int32 [B, D] CUDA tensor that receives each channel's iteration index."""
    B, T, G, D = u.shape
    dev = u.device
    h = torch.empty((B, T, D), dtype=torch.float32, device=dev) if h is None else h
    stats = _new_stats(dev) if stats is None else stats
    ih = torch.empty(max_iters + 2, dtype=torch.int32, device=dev) if hist else None
    ws = workspace if workspace is not None else Workspace(dev)
    buf = ws.get(pararnn_workspace_size(PARARNN_GRU, B, T, D, max_iters, 0), stream)
    o = opts if opts is not None else _opts(tol, max_iters, flags=flags,
                                            max_cluster=max_cluster,
                                            chan_iters=chan_iters)
    pararnn_gru_solve(u, a, bias, h0, h, o, stats, ih, buf, stream)
    return h, stats, ih


def lstm_solve(u, a, bias=None, c0=None, h0=None, *, tol=1e-6, max_iters=64,
               hist=False, workspace=None, c=None, h=None, stats=None,
               stream=None, opts=None, max_cluster=0, flags=0, chan_iters=None):
    """ParaLSTM solve -> (c, h, stats, iter_hist or None); `chan_iters` as
    for gru_solve."""
    B, T, G, D = u.shape
    dev = u.device
    c = torch.empty((B, T, D), dtype=torch.float32, device=dev) if c is None else c
    h = torch.empty((B, T, D), dtype=torch.float32, device=dev) if h is None else h
    stats = _new_stats(dev) if stats is None else stats
    ih = torch.empty(max_iters + 2, dtype=torch.int32, device=dev) if hist else None
    ws = workspace if workspace is not None else Workspace(dev)
    buf = ws.get(pararnn_workspace_size(PARARNN_LSTM, B, T, D, max_iters, 0), stream)
    o = opts if opts is not None else _opts(tol, max_iters, flags=flags,
                                            max_cluster=max_cluster,
                                            chan_iters=chan_iters)
    pararnn_lstm_solve(u, a, bias, c0, h0, c, h, o, stats, ih, buf, stream)
    return c, h, stats, ih


def adjoint(cell, u, a, bias, h0, h, dLdh, c0=None, c=None, *, workspace=None,
            want_dbias=True, want_dh0=True, stream=None, out=None, opts=None):
    B, T, G, D = u.shape
    dev = u.device
    o = out or {}
    du = o.get("du") if o.get("du") is not None else torch.empty((B, T, G, D), dtype=torch.float32, device=dev)
    da = o.get("da") if o.get("da") is not None else torch.empty((G, D), dtype=torch.float32, device=dev)
    db = (o.get("dbias") if o.get("dbias") is not None else torch.empty((G, D), dtype=torch.float32, device=dev)) if want_dbias else None
    dh0 = (o.get("dh0") if o.get("dh0") is not None else torch.empty((B, D), dtype=torch.float32, device=dev)) if want_dh0 else None
    dc0 = None
    if cell == PARARNN_LSTM and want_dh0:
        dc0 = o.get("dc0") if o.get("dc0") is not None else torch.empty((B, D), dtype=torch.float32, device=dev)
    status = o.get("status") if o.get("status") is not None else torch.zeros(1, dtype=torch.int32, device=dev)
    ws = workspace if workspace is not None else Workspace(dev)
    buf = ws.get(pararnn_workspace_size(cell, B, T, D, 0, 1), stream)
    if opts is None:
        pararnn_adjoint(cell, u, a, bias, c0, h0, c, h, dLdh, du, da, db, dc0, dh0,
                        status, buf, stream)
    else:
        pararnn_adjoint_ex(cell, u, a, bias, c0, h0, c, h, dLdh, du, da, db, dc0, dh0,
                           status, buf, opts, stream)
    return {"du": du, "da": da, "dbias": db, "dh0": dh0, "dc0": dc0,
            "status": status}


def solve_unfused(cell, u, a, bias=None, c0=None, h0=None, *, tol=1e-6, max_iters=64,
                  workspace=None, stream=None):
    """The unfused tier: returns (c, h, stats) with c None for ParaGRU.
    Synchronises the stream (the host checks the residual each iteration)."""
    B, T, G, D = u.shape
    dev = u.device
    h = torch.empty((B, T, D), dtype=torch.float32, device=dev)
    c = torch.empty((B, T, D), dtype=torch.float32, device=dev) if cell == PARARNN_LSTM else None
    stats = _new_stats(dev)
    ws = workspace if workspace is not None else Workspace(dev)
    buf = ws.get(pararnn_unfused_workspace_size(cell, B, T, D), stream)
    pararnn_solve_unfused(cell, u, a, bias, c0, h0, c, h, _opts(tol, max_iters), stats,
                          buf, stream)
    return c, h, stats


def dense_gru_solve(u, W, bias=None, h0=None, *, tol=1e-6, max_iters=64, workspace=None,
                    stream=None, flags=0):
    """Newton solve of the GRU with full recurrent matrices W [3, D, D]:
    returns (h, stats).  Synchronises the stream."""
    B, T, G, D = u.shape
    h = torch.empty((B, T, D), dtype=torch.float32, device=u.device)
    stats = _new_stats(u.device)
    ws = workspace if workspace is not None else Workspace(u.device)
    nbytes = pararnn_dense_workspace_size(B, T, D)
    if nbytes == 0:
        raise PararnnError(-1, "pararnn_dense_workspace_size (unsupported shape)")
    buf = ws.get(nbytes, stream)
    pararnn_dense_gru_solve(u, W, bias, h0, h, _opts(tol, max_iters, flags=flags), stats, buf,
                            stream)
    return h, stats


def gru_step(u_t, a, bias=None, h_prev=None, *, out=None, stream=None):
    """One ParaGRU decode step: u_t [B, 3, D] -> the next state [B, D].
    `out` may be `h_prev` (in-place update)."""
    B, G, D = u_t.shape
    h = torch.empty((B, D), dtype=torch.float32, device=u_t.device) if out is None else out
    pararnn_gru_step(u_t, a, bias, h_prev, h, stream)
    return h


def lstm_step(u_t, a, bias=None, c_prev=None, h_prev=None, *, out=None, stream=None):
    """One ParaLSTM decode step: u_t [B, 4, D] -> (c, h) [B, D] each.
    `out` = (c, h) may be (c_prev, h_prev) (in-place update)."""
    B, G, D = u_t.shape
    if out is None:
        out = (torch.empty((B, D), dtype=torch.float32, device=u_t.device),
               torch.empty((B, D), dtype=torch.float32, device=u_t.device))
    pararnn_lstm_step(u_t, a, bias, c_prev, h_prev, out[0], out[1], stream)
    return out


def seq_baseline(cell, u, a, bias=None, c0=None, h0=None, stream=None):
    B, T, G, D = u.shape
    h = torch.empty((B, T, D), dtype=torch.float32, device=u.device)
    c = torch.empty((B, T, D), dtype=torch.float32, device=u.device) if cell == PARARNN_LSTM else None
    pararnn_seq_baseline(cell, u, a, bias, c0, h0, c, h, stream)
    return c, h


# ------------------------------------- gated linear recurrence, block norm --
# The wrappers (linrec_*, block_norm*) check every shape, type and device, since
# the library sees pointers only; they run on the device of their tensors,
# whatever the current one is, and allocate what they return (and their scratch)
# on the stream they launch on, so both live as long as the work in flight, in a
# captured graph too.  Inputs made on another stream are the caller's to order,
# as with every CUDA call.  A decode step takes the GPU 2 us, so the checks are
# written to cost little.  The bindings of the C names take tensors of the
# current device, and their sizes on trust.
_F32, _BF16 = torch.float32, torch.bfloat16
_DTYPES = {_F32: PARARNN_F32, _BF16: PARARNN_BF16}
_FLOATS = (_F32, _BF16)
_MASKS = (torch.bool, torch.uint8)
_LIN_CELLS = {PARARNN_LIN_GRU: 2, PARARNN_LIN_DECAY: 3}
_ACTS = {"silu": PARARNN_ACT_SILU, "sigmoid": PARARNN_ACT_SIGMOID}
# the current stream's handle, without building a Stream object
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _code(t):
    """The library's code of a tensor's type (-1 lets the library reject it)."""
    return 0 if t is None else _DTYPES.get(t.dtype, -1)


def _need(t, name, shape, device, dtypes=(_F32,)):
    """Pointer of a contiguous tensor of this shape, one of these types, on
    this device (None -> NULL)."""
    if t is None:
        return None
    if t.shape == shape and t.dtype in dtypes and t.device == device and t.is_contiguous():
        return t.data_ptr()
    if t.device != device:
        raise ValueError(f"{name}: expected a tensor on {device}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: expected {' or '.join(map(str, dtypes))}, got {t.dtype}")
    raise ValueError(f"{name}: expected a contiguous tensor")


def _like(t, shape, dtype, base):
    """A new contiguous tensor: like `t` where that has its shape and type (the
    cheaper call), else of `base`'s device."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return torch.empty_like(t)
    return base.new_empty(shape, dtype=dtype)


def _first(t, name):
    """The device of the leading tensor of a call."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name}: pararnn expects a CUDA tensor")
    return t.device


@contextlib.contextmanager
def _moved(device, stream):
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device=device)
    if stream is not None and stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


_HERE_NOW = contextlib.nullcontext()


def _on(device, stream):
    """The context a call launches and allocates in."""
    if stream is None and device.index == torch.cuda.current_device():
        return _HERE_NOW
    return _moved(device, stream)


def _lin_u(cell, u, ndim):
    G = _LIN_CELLS.get(cell)
    if G is None:
        raise PararnnError(-1, f"linear recurrence: unknown cell {cell}")
    dev = _first(u, "u")
    shape = u.shape
    if len(shape) != ndim or shape[-2] != G:
        raise ValueError(f"u: expected {'[B, T, G, D]' if ndim == 4 else '[B, G, D]'} with G = {G},"
                         f" got {tuple(shape)}")
    st = u.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError("u: channels must be contiguous")
    # an axis of one has no stride
    return dev, G, [0 if n == 1 else k for n, k in zip(shape[:-1], st)]


def _lin_params(cell, dev, B, G, D, lam, bias, h0, h0_name="h0"):
    if (lam is None) != (cell == PARARNN_LIN_GRU):
        raise ValueError("lam: given exactly for PARARNN_LIN_DECAY")
    return (_need(lam, "lam", (D,), dev), _need(bias, "bias", (G, D), dev),
            _need(h0, h0_name, (B, D), dev))


def _here(*tensors):
    """The bindings launch on the current device, whose memory they need."""
    dev = torch.cuda.current_device()
    for t in tensors:
        if t is not None and not isinstance(t, int) and t.device.index != dev:
            raise ValueError(f"expected a tensor on cuda:{dev}, got {t.device}")


def pararnn_linrec_solve(cell, u, lam, bias, h0, reset, h, kappa=8.0, stream=None):
    _here(u, lam, bias, h0, reset, h)
    B, T, G, D = u.shape
    _check(load_library().pararnn_linrec_solve(
        cell, u.data_ptr(), _code(u), *_lin_u(cell, u, 4)[2], _ptr(lam), _ptr(bias), _ptr(h0),
        _mptr(reset), _ptr(h), B, T, D, kappa, _stream(stream)), "pararnn_linrec_solve")


def pararnn_linrec_solve_ex(cell, u, lam, bias, h0, reset, h, status, opts, kappa=8.0, stream=None):
    _here(u, lam, bias, h0, reset, h, status)
    B, T, G, D = u.shape
    _check(load_library().pararnn_linrec_solve_ex(
        cell, u.data_ptr(), _code(u), *_lin_u(cell, u, 4)[2], _ptr(lam), _ptr(bias), _ptr(h0),
        _mptr(reset), _ptr(h), B, T, D, kappa, _iptr(status),
        ctypes.byref(opts) if opts is not None else None, _stream(stream)),
        "pararnn_linrec_solve_ex")


def pararnn_linrec_workspace_size(cell, B, T, D) -> int:
    return int(load_library().pararnn_linrec_workspace_size(cell, B, T, D))


def pararnn_linrec_adjoint(cell, u, lam, bias, h0, reset, h, dLdh, du, dlam, dbias, dh0,
                           workspace, kappa=8.0, stream=None):
    _here(u, lam, bias, h0, reset, h, dLdh, du, dlam, dbias, dh0, workspace)
    B, T, G, D = u.shape
    _check(load_library().pararnn_linrec_adjoint(
        cell, u.data_ptr(), _code(u), *_lin_u(cell, u, 4)[2], _ptr(lam), _ptr(bias), _ptr(h0),
        _mptr(reset), _ptr(h), _ptr(dLdh), _ptr(du, None), _code(du), _ptr(dlam),
        _ptr(dbias), _ptr(dh0), B, T, D, kappa, _wptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "pararnn_linrec_adjoint")


def pararnn_linrec_adjoint_ex(cell, u, lam, bias, h0, reset, h, dLdh, du, dlam, dbias, dh0, status,
                              workspace, opts, kappa=8.0, stream=None):
    _here(u, lam, bias, h0, reset, h, dLdh, du, dlam, dbias, dh0, status, workspace)
    B, T, G, D = u.shape
    _check(load_library().pararnn_linrec_adjoint_ex(
        cell, u.data_ptr(), _code(u), *_lin_u(cell, u, 4)[2], _ptr(lam), _ptr(bias), _ptr(h0),
        _mptr(reset), _ptr(h), _ptr(dLdh), _ptr(du, None), _code(du), _ptr(dlam),
        _ptr(dbias), _ptr(dh0), B, T, D, kappa, _iptr(status), _wptr(workspace),
        workspace.numel() * workspace.element_size(),
        ctypes.byref(opts) if opts is not None else None, _stream(stream)),
        "pararnn_linrec_adjoint_ex")


def pararnn_linrec_step(cell, u_t, lam, bias, h_prev, h_next, kappa=8.0, stream=None):
    _here(u_t, lam, bias, h_prev, h_next)
    B, G, D = u_t.shape
    _check(load_library().pararnn_linrec_step(
        cell, u_t.data_ptr(), _code(u_t), *_lin_u(cell, u_t, 3)[2], _ptr(lam), _ptr(bias),
        _ptr(h_prev), _ptr(h_next), B, D, kappa, _stream(stream)), "pararnn_linrec_step")


def _wait_args(status, opts, dev):
    """Pointers of a call's status word (int32 [1]) and its options."""
    return (_need(status, "status", (1,), dev, (torch.int32,)),
            None if opts is None else ctypes.byref(opts))


def linrec_solve(cell, u, lam=None, bias=None, h0=None, *, reset=None, kappa=8.0, out=None,
                 status=None, opts=None, stream=None):
    """Gated linear recurrence: u [B, T, G, D] (bf16 or fp32) -> states h
    [B, T, D] fp32.  cell PARARNN_LIN_GRU (G = 2: z, c) or PARARNN_LIN_DECAY
    (G = 3: r, i, x, with lam [D]).  u may be a view into a larger projection
    (channels contiguous, strides multiples of 8 elements, 16-byte aligned).
    reset [B, T] (bool or uint8): the state that enters a marked step is zero.
    `out`: the tensor to write h to.  `status`: an int32 [1] CUDA tensor that
    receives 0, or the TIMEOUT status where a wait inside the kernel ran out
    (what depends on it is NaN); `opts` bounds those waits (timeout_us)."""
    dev, G, st = _lin_u(cell, u, 4)
    B, T, _, D = u.shape
    lp, bp, hp = _lin_params(cell, dev, B, G, D, lam, bias, h0)
    rp = _need(reset, "reset", (B, T), dev, _MASKS)
    wait = _wait_args(status, opts, dev)
    op = _need(out, "out", (B, T, D), dev)
    with _on(dev, stream):
        if out is None:
            out = u.new_empty((B, T, D), dtype=_F32)
            op = out.data_ptr()
        _check(load_library().pararnn_linrec_solve_ex(
            cell, u.data_ptr(), _code(u), *st, lp, bp, hp, rp, op, B, T, D, kappa, *wait,
            _raw_stream(dev.index)), "pararnn_linrec_solve")
    return out


def linrec_adjoint(cell, u, lam, bias, h0, h, dLdh, *, reset=None, kappa=8.0, want_params=True,
                   want_dh0=True, du_dtype=None, out=None, status=None, opts=None, stream=None):
    """Adjoint of :func:`linrec_solve` along its states h: a dict of du
    [B, T, G, D] (u's type, or `du_dtype` = torch.float32), dlam [D], dbias
    [G, D] and dh0 [B, D] (None where not wanted or absent).  `out`: a dict of
    tensors to write to instead of new ones.  `status`, `opts`: as for
    linrec_solve."""
    dev, G, st = _lin_u(cell, u, 4)
    B, T, _, D = u.shape
    lp, bp, hp = _lin_params(cell, dev, B, G, D, lam, bias, h0)
    rp = _need(reset, "reset", (B, T), dev, _MASKS)
    if h is None or dLdh is None:
        raise ValueError("h and dLdh are needed")
    sp, gp = _need(h, "h", (B, T, D), dev), _need(dLdh, "dLdh", (B, T, D), dev)
    du = dlam = dbias = dh0 = None
    if out:
        du, dlam, dbias, dh0 = (out.get(k) for k in ("du", "dlam", "dbias", "dh0"))
        _need(du, "du", (B, T, G, D), dev, _FLOATS)
        _need(dlam, "dlam", (D,), dev)
        _need(dbias, "dbias", (G, D), dev)
        _need(dh0, "dh0", (B, D), dev)
    sw, ow = _wait_args(status, opts, dev)
    lib = load_library()
    with _on(dev, stream):
        if du is None:
            du = _like(u, u.shape, du_dtype or u.dtype, u)
        if not want_params:
            dlam = dbias = None
        else:
            if lam is None:
                dlam = None
            elif dlam is None:
                dlam = torch.empty_like(lam)
            if dbias is None:
                dbias = _like(bias, (G, D), _F32, u)
        if not want_dh0:
            dh0 = None
        elif dh0 is None:
            dh0 = _like(h0, (B, D), _F32, u)
        nbytes = max(256, lib.pararnn_linrec_workspace_size(cell, B, T, D))
        ws = u.new_empty(nbytes, dtype=torch.uint8)
        _check(lib.pararnn_linrec_adjoint_ex(
            cell, u.data_ptr(), _code(u), *st, lp, bp, hp, rp, sp, gp, du.data_ptr(), _code(du),
            _any_ptr(dlam), _any_ptr(dbias), _any_ptr(dh0), B, T, D, kappa, sw, ws.data_ptr(),
            nbytes, ow, _raw_stream(dev.index)), "pararnn_linrec_adjoint")
    return {"du": du, "dlam": dlam, "dbias": dbias, "dh0": dh0}


def linrec_step(cell, u_t, lam=None, bias=None, h_prev=None, *, kappa=8.0, out=None, stream=None):
    """One decode step of the gated linear recurrence: u_t [B, G, D] -> the
    next state [B, D].  `out` may be `h_prev` (in-place update)."""
    dev, G, st = _lin_u(cell, u_t, 3)
    B, _, D = u_t.shape
    lp, bp, hp = _lin_params(cell, dev, B, G, D, lam, bias, h_prev, "h_prev")
    op = _need(out, "out", (B, D), dev)
    with _on(dev, stream):
        if out is None:
            out = u_t.new_empty((B, D), dtype=_F32) if h_prev is None else torch.empty_like(h_prev)
            op = out.data_ptr()
        _check(load_library().pararnn_linrec_step(
            cell, u_t.data_ptr(), _code(u_t), *st, lp, bp, hp, op, B, D, kappa,
            _raw_stream(dev.index)), "pararnn_linrec_step")
    return out


def _any_ptr(t):
    return None if t is None else t.data_ptr()


def _rptr(t):
    """Device pointer of rows that may lie apart (None -> NULL)."""
    if t is None:
        return None
    if not t.is_cuda or (t.stride(-1) != 1 and t.shape[-1] > 1):
        raise ValueError("pararnn expects CUDA tensors with contiguous channels")
    return t.data_ptr()


def pararnn_block_norm(h, h_stride, gate, gate_stride, act, w_post, res, res_stride, scale, w_pre, s,
                       x, eps, N, D, stream=None):
    _here(h, gate, w_post, res, scale, w_pre, s, x)
    _check(load_library().pararnn_block_norm(
        _rptr(h), _code(h), h_stride, _rptr(gate), _code(gate), gate_stride, act, _ptr(w_post),
        _rptr(res), _code(res), res_stride, _ptr(scale), _ptr(w_pre), _ptr(s, None), _code(s),
        _ptr(x, None), _code(x), eps, N, D, _stream(stream)), "pararnn_block_norm")


def pararnn_block_norm_workspace_size(N, D) -> int:
    return int(load_library().pararnn_block_norm_workspace_size(N, D))


def pararnn_block_norm_adjoint(h, h_stride, gate, gate_stride, act, w_post, res, res_stride, scale,
                               w_pre, ds, ds_stride, dx, dx_stride, dh, dgate, dres, dw_post, dscale,
                               dw_pre, eps, N, D, workspace, stream=None):
    _here(h, gate, w_post, res, scale, w_pre, ds, dx, dh, dgate, dres, dw_post, dscale,
          dw_pre, workspace)
    _check(load_library().pararnn_block_norm_adjoint(
        _rptr(h), _code(h), h_stride, _rptr(gate), _code(gate), gate_stride, act, _ptr(w_post),
        _rptr(res), _code(res), res_stride, _ptr(scale), _ptr(w_pre), _rptr(ds), _code(ds),
        ds_stride, _rptr(dx), _code(dx), dx_stride, _ptr(dh, None), _ptr(dgate, None),
        _ptr(dres, None), _ptr(dw_post), _ptr(dscale), _ptr(dw_pre), eps, N, D, _wptr(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)),
        "pararnn_block_norm_adjoint")


def pararnn_block_norm_adjoint_ex(h, h_stride, gate, gate_stride, act, w_post, res, res_stride, scale,
                                  w_pre, ds, ds_stride, dx, dx_stride, dh, dgate, dres, dw_post, dscale,
                                  dw_pre, eps, N, D, status, workspace, opts, stream=None):
    _here(h, gate, w_post, res, scale, w_pre, ds, dx, dh, dgate, dres, dw_post, dscale,
          dw_pre, status, workspace)
    _check(load_library().pararnn_block_norm_adjoint_ex(
        _rptr(h), _code(h), h_stride, _rptr(gate), _code(gate), gate_stride, act, _ptr(w_post),
        _rptr(res), _code(res), res_stride, _ptr(scale), _ptr(w_pre), _rptr(ds), _code(ds),
        ds_stride, _rptr(dx), _code(dx), dx_stride, _ptr(dh, None), _ptr(dgate, None),
        _ptr(dres, None), _ptr(dw_post), _ptr(dscale), _ptr(dw_pre), eps, N, D, _iptr(status),
        _wptr(workspace), workspace.numel() * workspace.element_size(),
        ctypes.byref(opts) if opts is not None else None, _stream(stream)),
        "pararnn_block_norm_adjoint_ex")


def _rows(t, name, shape, dev):
    """(pointer, type code, row stride in elements) of a [..., D] tensor whose
    leading axes make up one axis of rows (None -> NULL)."""
    if t is None:
        return None, 0, 0
    if t.device != dev or t.shape != shape:
        raise ValueError(f"{name}: expected {tuple(shape)} on {dev}, got {tuple(t.shape)} on {t.device}")
    if t.is_contiguous():
        return t.data_ptr(), _code(t), shape[-1]
    st = t.stride()
    if st[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"{name}: channels must be contiguous")
    ld, rows = None, 1          # rows below the axis at hand, and their common stride
    for n, s in zip(reversed(shape[:-1]), reversed(st[:-1])):
        if n == 1:
            continue
        if ld is None:
            ld = s
        elif s != ld * rows:
            raise ValueError(f"{name}: rows must lie at one stride")
        rows *= n
    return t.data_ptr(), _code(t), shape[-1] if ld is None else ld


def _norm_parts(h, gate, act, w_post, res, scale, w_pre):
    """(device, shape, rows, channels, the library's arguments from h to w_pre)"""
    dev = _first(h, "h")
    shape = h.shape
    if not shape or h.numel() == 0:
        raise PararnnError(-1, f"block norm of shape {tuple(shape)}")
    kind = _ACTS.get(act)
    if kind is None:
        raise ValueError(f"act: expected one of {sorted(_ACTS)}, got {act!r}")
    D = shape[-1]
    w = (D,)
    return (dev, shape, h.numel() // D, D,
            (*_rows(h, "h", shape, dev), *_rows(gate, "gate", shape, dev), kind,
             _need(w_post, "w_post", w, dev), *_rows(res, "res", shape, dev),
             _need(scale, "scale", w, dev), _need(w_pre, "w_pre", w, dev)))


def block_norm(h, *, gate=None, act="silu", w_post=None, res=None, scale=None, w_pre=None, eps=1e-6,
               s_dtype=None, x_dtype=torch.bfloat16, want_s=True, out=None, stream=None):
    """The norms around a block with its gate and residual scale, on the rows
    of h [..., D] (fp32 states or a bf16 projection), each part optional:

        s = res + scale * (rms_norm(h) * w_post) * act(gate)
        x = rms_norm(s) * w_pre

    Returns (s, x); x is None without w_pre, s is None with want_s=False.
    s_dtype: res's type by default, bf16 without res.  gate, res: h's shape,
    bf16 or fp32; they and h may be views whose rows lie at one stride (a
    multiple of 8 elements).  `out` = (s, x), either None for a new tensor; s
    may be res (in-place update)."""
    dev, shape, N, D, parts = _norm_parts(h, gate, act, w_post, res, scale, w_pre)
    s, x = out or (None, None)
    sp, xp = _need(s, "s", shape, dev, _FLOATS), _need(x, "x", shape, dev, _FLOATS)
    with _on(dev, stream):
        if s is None and (want_s or w_pre is None):
            s = _like(res if res is not None else h, shape,
                      s_dtype or (_BF16 if res is None else res.dtype), h)
            sp = s.data_ptr()
        if x is None and w_pre is not None:
            x = _like(h, shape, x_dtype, h)
            xp = x.data_ptr()
        _check(load_library().pararnn_block_norm(*parts, sp, _code(s), xp, _code(x), eps, N, D,
                                                 _raw_stream(dev.index)), "pararnn_block_norm")
    return s, x


def block_norm_adjoint(h, ds, dx, *, gate=None, act="silu", w_post=None, res=None, scale=None,
                       w_pre=None, eps=1e-6, status=None, opts=None, stream=None):
    """Adjoint of :func:`block_norm` from ds = dL/ds (or None) and dx = dL/dx
    (given exactly when w_pre is): a dict of dh, dgate, dres (contiguous, in
    the types of h, gate, res) and dw_post, dscale, dw_pre [D] fp32, None
    where the part is absent.  h, gate and res hold what the forward call
    read.  `status`, `opts`: as for linrec_solve."""
    dev, shape, N, D, parts = _norm_parts(h, gate, act, w_post, res, scale, w_pre)
    if (dx is None) != (w_pre is None):
        raise ValueError("dx: given exactly when w_pre is")
    given = (*_rows(ds, "ds", shape, dev), *_rows(dx, "dx", shape, dev))
    sw, ow = _wait_args(status, opts, dev)
    with _on(dev, stream):
        def like(t):
            return None if t is None else _like(t, shape, t.dtype, t)
        outs = [like(h), like(gate), like(res)]
        outs += [None if t is None else torch.empty_like(t) for t in (w_post, scale, w_pre)]
        lib = load_library()
        nbytes = max(256, lib.pararnn_block_norm_workspace_size(N, D))
        ws = h.new_empty(nbytes, dtype=torch.uint8)
        _check(lib.pararnn_block_norm_adjoint_ex(*parts, *given, *map(_any_ptr, outs), eps, N, D, sw,
                                                 ws.data_ptr(), nbytes, ow, _raw_stream(dev.index)),
               "pararnn_block_norm_adjoint")
    return dict(zip(("dh", "dgate", "dres", "dw_post", "dscale", "dw_pre"), outs))
