"""ctypes binding of libgmm (include/gmm.h).

Argument marshalling only: every step of the EM iteration runs in the HIP
kernels of libgmm.so.  PyTorch provides device memory and the stream.  If
the library is missing the import fails; there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgmm.so")

GMM_OK, GMM_E_ARG, GMM_E_UNSUPPORTED, GMM_E_WORKSPACE, GMM_E_HIP, GMM_E_NOT_PD, GMM_E_NONFINITE = range(7)
COV = {"diag": 0, "iso": 1, "full": 2}
DTYPE = {"f32": 0, "bf16": 1, "f16": 2}
TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


class GmmError(RuntimeError):
    def __init__(self, status: int, call: str):
        self.status = status
        super().__init__(f"{call}: {status_str(status)} (status {status})")


class Desc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("d", ctypes.c_int64), ("k", ctypes.c_int64),
                ("ldx", ctypes.c_int64), ("cov", ctypes.c_int32), ("x_dtype", ctypes.c_int32),
                ("var_floor", ctypes.c_float), ("ridge_rel", ctypes.c_float)]


class FitOpts(ctypes.Structure):
    _fields_ = [("max_iter", ctypes.c_int32), ("init", ctypes.c_int32), ("seed", ctypes.c_uint64),
                ("tol", ctypes.c_double), ("batch", ctypes.c_int32), ("use_graph", ctypes.c_int32)]


INIT = {"given": 0, "random_points": 1}


class Diag(ctypes.Structure):
    _fields_ = [("bad_params", ctypes.c_int32), ("not_pd", ctypes.c_int32),
                ("ridge_retries", ctypes.c_int32), ("empty", ctypes.c_int32),
                ("nonfinite", ctypes.c_int32), ("x_range", ctypes.c_int32), ("ill_cond", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("ll", ctypes.c_double)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python -m soft_clustering_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, S, D = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(Desc)
    sig = {
        "gmm_workspace_bytes": [D, ctypes.POINTER(ctypes.c_size_t)],
        "gmm_prepare": [D, P, S, P, P, P, P],
        "gmm_em_step": [D, P, S, P, P, P],
        "gmm_finalize": [D, P, S, P, P, P, P],
        "gmm_loglik": [D, P, S, P, P, P, P, P],
        "gmm_get_stats": [D, P, S, P, P, P, P],
        "gmm_diagnostics": [D, P, S, ctypes.POINTER(Diag), P],
        "gmm_assign": [D, P, S, P, ctypes.c_int32, P, P, P, P],
        "gmm_fit": [D, P, S, P, ctypes.POINTER(FitOpts), P, P, P, P, ctypes.POINTER(ctypes.c_int32), P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.gmm_em_iteration_noalloc.argtypes = [D, P, P, P, P, P, P, P, P, P]
    lib.gmm_em_iteration_noalloc.restype = ctypes.c_int
    lib.gmm_noalloc_max_workspace.argtypes = []
    lib.gmm_noalloc_max_workspace.restype = ctypes.c_size_t
    lib.gmm_status_str.argtypes = [ctypes.c_int]
    lib.gmm_status_str.restype = ctypes.c_char_p
    lib.gmm_version.argtypes = []
    lib.gmm_version.restype = ctypes.c_char_p
    # calibration kernels (include/gmm_calib.h)
    lib.gmm_calib_sink_bytes.argtypes = [ctypes.c_int]
    lib.gmm_calib_sink_bytes.restype = ctypes.c_size_t
    lib.gmm_calib_read.argtypes = [P, S, ctypes.c_int, P, P]
    lib.gmm_calib_read.restype = ctypes.c_int
    lib.gmm_calib_mfma.argtypes = [ctypes.c_int64, ctypes.c_int, P, P]
    lib.gmm_calib_mfma.restype = ctypes.c_int
    lib.gmm_calib_mfma_flops.argtypes = [ctypes.c_int64, ctypes.c_int]
    lib.gmm_calib_mfma_flops.restype = ctypes.c_double
    return lib


_lib = _load()

EXPORTED = ("gmm_workspace_bytes", "gmm_prepare", "gmm_em_step", "gmm_finalize", "gmm_loglik",
            "gmm_assign", "gmm_fit", "gmm_get_stats", "gmm_diagnostics", "gmm_status_str", "gmm_version",
            "gmm_calib_sink_bytes", "gmm_calib_read", "gmm_calib_mfma", "gmm_calib_mfma_flops",
            "gmm_em_iteration_noalloc", "gmm_noalloc_max_workspace",
            # the lists and the components' models (bound in experts.py)
            "gmm_route_workspace_bytes", "gmm_route", "gmm_dispatch", "gmm_dispatch_backward", "gmm_combine",
            "gmm_combine_backward", "gmm_linear", "gmm_linear_backward_workspace_bytes", "gmm_linear_backward",
            "gmm_quantize4", "gmm_linear4")


def status_str(status: int) -> str:
    return _lib.gmm_status_str(status).decode()


def version() -> str:
    return _lib.gmm_version().decode()


def _check(status: int, call: str):
    if status != GMM_OK:
        raise GmmError(status, call)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_desc(n, d, k, cov="diag", x_dtype="f32", ldx=None, var_floor=1e-6, ridge_rel=1e-3) -> Desc:
    return Desc(int(n), int(d), int(k), int(d if ldx is None else ldx), COV[cov], DTYPE[x_dtype],
                float(var_floor), float(ridge_rel))


def workspace_bytes(desc: Desc) -> int:
    out = ctypes.c_size_t(0)
    _check(_lib.gmm_workspace_bytes(ctypes.byref(desc), ctypes.byref(out)), "gmm_workspace_bytes")
    return int(out.value)


@dataclass
class Stats:
    s0: torch.Tensor
    s1: torch.Tensor
    s2: torch.Tensor


class Gmm:
    """One descriptor plus its workspace (a torch uint8 device buffer)."""

    def __init__(self, n, d, k, cov="diag", x_dtype="f32", ldx=None, var_floor=1e-6,
                 ridge_rel=1e-3, device="cuda"):
        self.desc = make_desc(n, d, k, cov, x_dtype, ldx, var_floor, ridge_rel)
        self.n, self.d, self.k, self.cov, self.x_dtype = int(n), int(d), int(k), cov, x_dtype
        self.device = torch.device(device)
        self.ws_bytes = workspace_bytes(self.desc)
        self.ws = torch.empty(self.ws_bytes + 256, dtype=torch.uint8, device=self.device)
        off = (-self.ws.data_ptr()) % 256          # the library wants 256-byte alignment
        self.ws_view = self.ws[off:off + self.ws_bytes]

    # --- shapes -----------------------------------------------------------
    @property
    def cov_shape(self):
        return {"diag": (self.k, self.d), "iso": (self.k,), "full": (self.k, self.d, self.d)}[self.cov]

    def _ws(self):
        return ctypes.c_void_p(self.ws_view.data_ptr()), ctypes.c_size_t(self.ws_bytes)

    def _check_x(self, x):
        if x.device.type != "cuda" or x.dtype != TORCH_DTYPE[self.x_dtype]:
            raise ValueError("x must be a device tensor of the descriptor's storage dtype")
        if x.dim() != 2 or x.shape[0] != self.n or x.shape[1] != self.d or x.stride(1) != 1 \
                or (self.n > 1 and x.stride(0) != self.desc.ldx):
            raise ValueError("x must be [n, d] with unit column stride and row stride ldx")

    # --- calls ------------------------------------------------------------
    def prepare(self, pi, mu, cov, stream=None):
        for t in (pi, mu, cov):
            if t.dtype != torch.float32 or not t.is_contiguous() or t.device.type != "cuda":
                raise ValueError("parameters must be contiguous fp32 device tensors")
        ws, nb = self._ws()
        _check(_lib.gmm_prepare(ctypes.byref(self.desc), ws, nb, _ptr(pi), _ptr(mu), _ptr(cov),
                                _stream(stream)), "gmm_prepare")

    def em_step(self, x, ll_out=None, stream=None):
        self._check_x(x)
        ws, nb = self._ws()
        _check(_lib.gmm_em_step(ctypes.byref(self.desc), ws, nb, _ptr(x), _ptr(ll_out),
                                _stream(stream)), "gmm_em_step")

    def finalize(self, pi_out=None, mu_out=None, cov_out=None, stream=None):
        ws, nb = self._ws()
        _check(_lib.gmm_finalize(ctypes.byref(self.desc), ws, nb, _ptr(pi_out), _ptr(mu_out),
                                 _ptr(cov_out), _stream(stream)), "gmm_finalize")

    def loglik(self, x, ll_out=None, point_lse=None, point_argmax=None, stream=None):
        if self.n > 0:
            self._check_x(x)
        ws, nb = self._ws()
        _check(_lib.gmm_loglik(ctypes.byref(self.desc), ws, nb, _ptr(x) if self.n > 0 else None,
                               _ptr(ll_out), _ptr(point_lse), _ptr(point_argmax), _stream(stream)),
               "gmm_loglik")

    def assign(self, x, m, out_idx=None, out_gamma=None, ll_out=None, stream=None):
        """Top-m soft assignment: (idx int32 [n, m], gamma fp32 [n, m])."""
        if self.n > 0:
            self._check_x(x)
        if out_idx is None:
            out_idx = torch.empty((self.n, m), dtype=torch.int32, device=self.device)
        if out_gamma is None:
            out_gamma = torch.empty((self.n, m), dtype=torch.float32, device=self.device)
        ws, nb = self._ws()
        _check(_lib.gmm_assign(ctypes.byref(self.desc), ws, nb, _ptr(x) if self.n > 0 else None,
                               int(m), _ptr(out_idx), _ptr(out_gamma), _ptr(ll_out), _stream(stream)),
               "gmm_assign")
        return out_idx, out_gamma

    def fit(self, x, pi, mu, cov, max_iter=100, tol=1e-6, init="given", seed=0, batch=8,
            use_graph=True, ll_hist=None, stream=None):
        """EM to convergence; pi / mu / cov (device fp32) are the start (init
        "given") and receive the final parameters.  Returns (iterations, LL per
        iteration as a device fp64 tensor [max_iter])."""
        self._check_x(x)
        for t in (pi, mu, cov):
            if t.dtype != torch.float32 or not t.is_contiguous() or t.device.type != "cuda":
                raise ValueError("parameters must be contiguous fp32 device tensors")
        if ll_hist is None:
            ll_hist = torch.full((max_iter,), float("nan"), dtype=torch.float64, device=self.device)
        opts = FitOpts(int(max_iter), INIT[init], int(seed) & ((1 << 64) - 1), float(tol), int(batch),
                       1 if use_graph else 0)
        nit = ctypes.c_int32(0)
        if stream is None and use_graph:
            stream = torch.cuda.current_stream()
        ws, nb = self._ws()
        _check(_lib.gmm_fit(ctypes.byref(self.desc), ws, nb, _ptr(x), ctypes.byref(opts), _ptr(pi), _ptr(mu),
                            _ptr(cov), _ptr(ll_hist), ctypes.byref(nit), _stream(stream)), "gmm_fit")
        return int(nit.value), ll_hist

    def get_stats(self, stream=None) -> Stats:
        f64 = dict(dtype=torch.float64, device=self.device)
        s0 = torch.empty(self.k, **f64)
        s1 = torch.empty(self.k, self.d, **f64)
        s2 = torch.empty({"diag": (self.k, self.d), "iso": (self.k,),
                          "full": (self.k, self.d, self.d)}[self.cov], **f64)
        ws, nb = self._ws()
        _check(_lib.gmm_get_stats(ctypes.byref(self.desc), ws, nb, _ptr(s0), _ptr(s1), _ptr(s2),
                                  _stream(stream)), "gmm_get_stats")
        return Stats(s0, s1, s2)

    def diagnostics(self, stream=None) -> Diag:
        out = Diag()
        ws, nb = self._ws()
        _check(_lib.gmm_diagnostics(ctypes.byref(self.desc), ws, nb, ctypes.byref(out),
                                    _stream(stream)), "gmm_diagnostics")
        return out

    # --- convenience: one full iteration ---------------------------------
    def iterate(self, x, pi_out, mu_out, cov_out, ll_out=None, stream=None):
        """gmm_em_step then gmm_finalize (the finalize also prepares the next step)."""
        self.em_step(x, ll_out, stream)
        self.finalize(pi_out, mu_out, cov_out, stream)


# --- calibration kernels (measured ceilings; include/gmm_calib.h) -----------
def calib_sink(grid, device="cuda"):
    return torch.empty(int(_lib.gmm_calib_sink_bytes(int(grid))), dtype=torch.uint8, device=device)


def calib_read(buf, grid, sink, stream=None):
    """Streaming read of every byte of the device tensor `buf` (launch only)."""
    nbytes = buf.numel() * buf.element_size()
    _check(_lib.gmm_calib_read(_ptr(buf), nbytes, int(grid), _ptr(sink), _stream(stream)),
           "gmm_calib_read")
    return nbytes // 16 * 16


def calib_mfma(iters, grid, sink, stream=None):
    """Register-resident fp16 MFMA chains (launch only); returns their flops."""
    _check(_lib.gmm_calib_mfma(int(iters), int(grid), _ptr(sink), _stream(stream)), "gmm_calib_mfma")
    return float(_lib.gmm_calib_mfma_flops(int(iters), int(grid)))
