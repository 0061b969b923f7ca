"""Python binding of libcr.so (the GB300 conditional-simulation library).

Argument marshalling only: every computation runs in the library's CUDA kernels.  PyTorch
supplies device memory and streams.  Matrices are column-major like the C ABI: a column-major
n x m matrix is a torch tensor whose transpose is contiguous (stride (1, ld)); the helpers
``colmajor_empty`` / ``as_colmajor`` build such tensors.

The functions mirror include/cr.h:
  TileMat(n, nb)                         cr_tilemat_create / destroy
  cov_build(V, xy, ...)                  cr_cov_build
  tile_stats(V)                          cr_tile_stats
  tile_stats_records(V)                  cr_tile_stats_records
  precision_map(V, amp, fixedacc, auto)  cr_precision_map
  potrf_adaptive(V)                      cr_potrf_adaptive
  tilemat_to_dense(V, what)              cr_tilemat_to_dense
  rnorm(n, M, seed, offset)              cr_rnorm
  trmm_sim(V, Z, M, ...)                 cr_trmm_sim
  krige(V, Xo, Xp, yo)                   cr_krige
  krige_correct(W, yo, Y, n_p, n_o)      cr_krige_correct
  correct_calibrate(W, yo, Y, ...)       cr_correct_calibrate (correction fused with calibration)
  Weights(W)                             cr_weights_prepare / cr_weights_release
  krige_correct_prepared(Wp, yo, Y)      cr_krige_correct_prepared
  correct_calibrate_prepared(Wp, ...)    cr_correct_calibrate_prepared
  calibrate(S, zhat, v, u, level)        cr_calibrate (negative=True: cr_calibrate_negative)
  morton_order(xy)                       cr_morton_order (host only)
  affine(W, X, bias, act, residual)      cr_affine
  affine_backward(W, X, dY, Z, act)      cr_affine_backward
  rmsnorm(X, gamma, residual)            cr_rmsnorm (rmsnorm_e4m3: the 8-bit output)
  rmsnorm_backward(H, gamma, dY, dH)     cr_rmsnorm_backward
  gated_scan(G, X, gate, offsets, h0)    cr_gated_scan
  gated_scan_backward(G, X, dH, ...)     cr_gated_scan_backward
  gated_step(G, X, h, gate)              cr_gated_step
The library is never replaced by a fallback: if libcr.so is missing or fails to load, every
call raises.
"""
from __future__ import annotations

import ctypes
import os
import re

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_lib", "libcr.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "cr.h")

CR_PREC_FP64, CR_PREC_FP32, CR_PREC_FP16 = 0, 1, 2
CR_COV_MATERN, CR_COV_POWEXP = 0, 1
CR_TRMM_FP16_DEST, CR_TRMM_GENERATE, CR_TRMM_SPLIT_L, CR_TRMM_FP16_PER_GEMM = 1, 2, 4, 8
CR_OPT_WAIT_LIMIT_US, CR_OPT_DIAG_ARITH, CR_OPT_FP64_GEMM = 1, 2, 4
CR_DIAG_AUTO, CR_DIAG_FP64, CR_DIAG_DF = 0, 1, 2
CR_GEMM_DF, CR_GEMM_OZAKI = 0, 1
CR_TYPE_F32, CR_TYPE_F16, CR_TYPE_BF16, CR_TYPE_E4M3 = 0, 1, 2, 3
CR_ACT_NONE, CR_ACT_RELU, CR_ACT_SILU, CR_ACT_GELU = 0, 1, 2, 3
CR_GATE_COEFF, CR_GATE_CONVEX, CR_GATE_VARIANCE = 0, 1, 2
CR_PEAK_DFMA, CR_PEAK_FFMA, CR_PEAK_DF_MAC, CR_PEAK_DMMA = 1, 2, 3, 4
STATUS = {0: "CR_OK", 1: "CR_ERR_ARG", 2: "CR_ERR_CUDA", 3: "CR_ERR_NOMEM", 4: "CR_ERR_NOT_SPD",
          5: "CR_ERR_EMPTY_SAMPLE", 6: "CR_ERR_NONPOS_MSPE", 7: "CR_ERR_TIMEOUT", 8: "CR_ERR_STATE",
          9: "CR_ERR_NOT_IMPLEMENTED", 10: "CR_ERR_RANGE"}


class CrError(RuntimeError):
    def __init__(self, code: int, detail: str):
        self.code = code
        self.name = STATUS.get(code, f"CR_ERR_{code}")
        self.detail = detail
        super().__init__(f"{self.name}: {detail}")


class CovParams(ctypes.Structure):
    _fields_ = [("family", ctypes.c_int), ("sigma2", ctypes.c_double), ("range", ctypes.c_double),
                ("nu", ctypes.c_double), ("nugget", ctypes.c_double), ("n_pred", ctypes.c_int),
                ("tau2", ctypes.c_double)]


class PmapInfo(ctypes.Structure):
    _fields_ = [("fixedacc", ctypes.c_double), ("iters", ctypes.c_int), ("n_fp64", ctypes.c_int),
                ("n_fp32", ctypes.c_int), ("n_fp16", ctypes.c_int), ("R_hp", ctypes.c_double),
                ("rho1", ctypes.c_double), ("rho2", ctypes.c_double), ("check1", ctypes.c_int),
                ("check2", ctypes.c_int), ("ell", ctypes.c_double), ("u_s", ctypes.c_double),
                ("s", ctypes.c_double), ("range_ok", ctypes.c_int)]


class CalibInfo(ctypes.Structure):
    _fields_ = [("q_in", ctypes.c_double), ("q_out", ctypes.c_double), ("n_psi", ctypes.c_int),
                ("n_phi", ctypes.c_int)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_D = ctypes.c_double
_U64 = ctypes.c_uint64

_SIGNATURES = {
    "cr_status_str": (ctypes.c_char_p, [_I]),
    "cr_last_error_detail": (ctypes.c_char_p, []),
    "cr_version": (_I, [ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "cr_kernel_launches": (_I, [ctypes.POINTER(_U64)]),
    "cr_workspace_trim": (_I, []),
    "cr_set_option": (_I, [_I, ctypes.c_longlong]),
    "cr_peak_probe": (_I, [_I, _I, ctypes.POINTER(_D), _P]),
    "cr_get_option": (_I, [_I, ctypes.POINTER(ctypes.c_longlong)]),
    "cr_timing_enable": (_I, [_I]),
    "cr_timing_read": (_I, [ctypes.c_char_p, ctypes.POINTER(ctypes.c_double), ctypes.POINTER(_U64)]),
    "cr_timing_reset": (_I, []),
    "cr_tilemat_create": (_I, [_I, _I, ctypes.POINTER(_P)]),
    "cr_tilemat_destroy": (_I, [_P]),
    "cr_tilemat_info": (_I, [_P, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "cr_cov_build": (_I, [_P, _P, ctypes.POINTER(CovParams), _P]),
    "cr_tile_stats": (_I, [_P, _P, _P, _P]),
    "cr_tile_stats_records": (_I, [_P, _P, _P, _P, _P]),
    "cr_precision_map": (_I, [_P, _I, _D, _I, _P, ctypes.POINTER(PmapInfo)]),
    "cr_potrf_adaptive": (_I, [_P, _P, ctypes.POINTER(_I)]),
    "cr_tilemat_to_dense": (_I, [_P, _I, _P, _I, _P]),
    "cr_rnorm": (_I, [_P, _I, _I, _I, _U64, _U64, _P]),
    "cr_trmm_sim": (_I, [_P, _P, _I, _I, _U64, _U64, _P, _I, _I, ctypes.POINTER(_D), _P]),
    "cr_krige": (_I, [_P, _P, _P, _P, _P, _I, _P, _P, _P, ctypes.POINTER(_I)]),
    "cr_krige_correct": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _P, _I, _P]),
    "cr_morton_order": (_I, [_P, _I, _P]),
    "cr_calibrate": (_I, [_P, _I, _I, _I, _P, _P, _D, _D, _P, _P, _P, _P, _P, ctypes.POINTER(CalibInfo), _P]),
    "cr_correct_calibrate": (_I, [_P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _D, _D, _I, _P, _P, _P, _P, _P,
                                  ctypes.POINTER(CalibInfo), _P]),
    "cr_calibrate_negative": (_I, [_P, _I, _I, _I, _P, _P, _D, _D, _P, _P, _P, _P, _P, ctypes.POINTER(CalibInfo),
                                   _P]),
    "cr_calibrate_noalloc": (_I, [_P, _I, _I, _I, _P, _P, _D, _D, _P, _P, _P, _P, _P, ctypes.POINTER(CalibInfo),
                                  _P]),
    "cr_weights_prepare": (_I, [_P, _I, _I, _I, _P, ctypes.POINTER(_P)]),
    "cr_weights_release": (_I, [_P]),
    "cr_krige_correct_prepared": (_I, [_P, _P, _P, _I, _I, _P, _I, _P]),
    "cr_correct_calibrate_prepared": (_I, [_P, _P, _P, _I, _I, _P, _P, _D, _D, _I, _P, _P, _P, _P, _P,
                                           ctypes.POINTER(CalibInfo), _P]),
    "cr_affine": (_I, [_I, _P, _I, _P, _I, _I, _I, _I, _P, _P, _P, _I, _I, _P, _I, _P, _I, _P, _I, _P]),
    "cr_affine_backward": (_I, [_I, _P, _I, _P, _I, _P, _I, _P, _I, _I, _I, _I, _I, _P, _I, _I, _P, _I, _P, _P]),
    "cr_rmsnorm": (_I, [_I, _P, _I, _P, _I, _P, _I, _I, _D, _P, _I, _I, _P, _I, _P, _P]),
    "cr_rmsnorm_backward": (_I, [_I, _P, _I, _P, _P, _I, _P, _I, _I, _I, _D, _P, _I, _P, _P]),
    "cr_gated_scan_saved": (_I, [_I, _I, ctypes.POINTER(ctypes.c_size_t)]),
    "cr_gated_scan": (_I, [_I, _I, _P, _I, _P, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _I, _P, _P]),
    "cr_gated_scan_backward": (_I, [_I, _I, _P, _I, _P, _I, _P, _I, _I, _I, _P, _I, _P, _I, _P, _I, _P, _P, _I, _P, _I,
                                    _P, _I, _P]),
    "cr_gated_step": (_I, [_I, _I, _P, _I, _P, _I, _P, _I, _I, _I, _P, _I, _P, _I, _P]),
}


def header_functions() -> list[str]:
    """Names of the entry points declared in include/cr.h."""
    src = open(HEADER).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(cr_[a-z0-9_]+)\s*\(", src)))


def load(path: str | None = None):
    """Loads libcr.so (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it first (python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(p)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(code: int):
    if code != 0:
        raise CrError(code, (_lib.cr_last_error_detail() or b"").decode())


def _ptr(t) -> int | None:
    if t is None:
        return None
    return t.data_ptr()


def _stream(stream) -> int | None:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


def colmajor_empty(n: int, m: int, dtype, device="cuda"):
    """Uninitialised n x m column-major tensor (leading dimension n)."""
    import torch
    return torch.empty((m, n), dtype=dtype, device=device).T


def as_colmajor(t):
    """t as a column-major tensor (copies if needed); returns (tensor, ld)."""
    if t.dim() == 1:
        return t.contiguous(), t.shape[0]
    if t.stride(0) != 1:
        t = t.T.contiguous().T
    return t, max(1, t.stride(1))


def kernel_launches() -> int:
    """cr_kernel_launches: kernels launched by the library in this process so far."""
    load()
    c = _U64(0)
    _check(_lib.cr_kernel_launches(ctypes.byref(c)))
    return c.value


def workspace_trim() -> None:
    """cr_workspace_trim: return the library's pooled scratch memory to the driver."""
    load()
    _check(_lib.cr_workspace_trim())


def set_option(option: int, value: int) -> None:
    """cr_set_option: CR_OPT_WAIT_LIMIT_US (microseconds), CR_OPT_DIAG_ARITH (CR_DIAG_*) or
    CR_OPT_FP64_GEMM (CR_GEMM_*)."""
    load()
    _check(_lib.cr_set_option(option, int(value)))


def peak_probe(kind: int, iters: int = 4096, stream=None) -> float:
    """cr_peak_probe: measured TFLOP/s of one arithmetic unit (CR_PEAK_*)."""
    load()
    v = _D(0.0)
    _check(_lib.cr_peak_probe(kind, iters, ctypes.byref(v), _stream(stream)))
    return v.value


def get_option(option: int) -> int:
    load()
    v = ctypes.c_longlong(0)
    _check(_lib.cr_get_option(option, ctypes.byref(v)))
    return v.value


def timing_enable(on: bool) -> None:
    """cr_timing_enable: bracket launches of the timed kernels with CUDA events."""
    load()
    _check(_lib.cr_timing_enable(1 if on else 0))


def timing_read(kernel: str) -> tuple[float, int]:
    """cr_timing_read: (total milliseconds, launches) of a timed kernel; synchronises."""
    load()
    ms = ctypes.c_double(0.0)
    n = _U64(0)
    _check(_lib.cr_timing_read(kernel.encode(), ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


def timing_reset() -> None:
    """cr_timing_reset: clear the accumulated kernel times."""
    load()
    _check(_lib.cr_timing_reset())


class TileMat:
    """Opaque lower-tile storage of a symmetric n x n matrix (cr_tilemat)."""

    def __init__(self, n: int, nb: int):
        load()
        h = _P()
        _check(_lib.cr_tilemat_create(n, nb, ctypes.byref(h)))
        self._h = h
        self.n, self.nb = n, nb
        self.nt = (n + nb - 1) // nb

    @property
    def handle(self):
        return self._h

    def close(self):
        if getattr(self, "_h", None):
            _lib.cr_tilemat_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def morton_order(xy) -> np.ndarray:
    """cr_morton_order: the stable Z-order permutation of the (n, 2) FP64 host array xy."""
    load()
    xy = np.ascontiguousarray(xy, dtype=np.float64)
    assert xy.ndim == 2 and xy.shape[1] == 2
    n = xy.shape[0]
    perm = np.empty(n, dtype=np.int32)
    _check(_lib.cr_morton_order(xy.ctypes.data if n else None, n, perm.ctypes.data if n else None))
    return perm


def cov_build(V: TileMat, xy, family: str = "matern", sigma2: float = 1.0, range: float = 0.1, nu: float = 0.5,
              nugget: float = 0.0, n_pred: int | None = None, tau2: float = 0.0, stream=None):
    """cr_cov_build: xy is an (n, 2) float64 CUDA tensor (row-major pairs)."""
    assert xy.is_cuda and xy.dtype.is_floating_point and xy.shape == (V.n, 2) and xy.is_contiguous()
    p = CovParams(CR_COV_MATERN if family == "matern" else CR_COV_POWEXP, sigma2, range, nu, nugget,
                  V.n if n_pred is None else n_pred, tau2)
    _check(_lib.cr_cov_build(V.handle, _ptr(xy), ctypes.byref(p), _stream(stream)))


def tile_stats(V: TileMat):
    nt = V.nt
    f, a, b = (np.zeros((nt, nt)) for _ in range(3))
    _check(_lib.cr_tile_stats(V.handle, f.ctypes.data, a.ctypes.data, b.ctypes.data))
    return f, a, b


def tile_stats_records(V: TileMat):
    """cr_tile_stats_records: (frob, vmin, vmax, err) as NT x NT arrays, nothing recomputed."""
    nt = V.nt
    f, a, b, e = (np.zeros((nt, nt)) for _ in range(4))
    _check(_lib.cr_tile_stats_records(V.handle, f.ctypes.data, a.ctypes.data, b.ctypes.data, e.ctypes.data))
    return f, a, b, e


def precision_map(V: TileMat, amp: bool = True, fixedacc: float = 1e-4, auto: bool = False):
    m = np.zeros((V.nt, V.nt), dtype=np.int8)
    info = PmapInfo()
    _check(_lib.cr_precision_map(V.handle, 1 if amp else 0, fixedacc, 1 if auto else 0, m.ctypes.data,
                                 ctypes.byref(info)))
    d = {k: getattr(info, k) for k, _ in PmapInfo._fields_}
    return m, d


def potrf_adaptive(V: TileMat, stream=None) -> int:
    info = _I(0)
    code = _lib.cr_potrf_adaptive(V.handle, _stream(stream), ctypes.byref(info))
    if code == 4:   # CR_ERR_NOT_SPD: report through info like LAPACK
        return info.value
    _check(code)
    return info.value


def tilemat_to_dense(V: TileMat, what: int = 1, stream=None):
    import torch
    out = colmajor_empty(V.n, V.n, torch.float64)
    _check(_lib.cr_tilemat_to_dense(V.handle, what, _ptr(out), V.n, _stream(stream)))
    return out


def rnorm(n: int, M: int, seed: int, offset: int = 0, out=None, stream=None):
    import torch
    load()
    if out is None:
        out = colmajor_empty(n, M, torch.float64)
    out, ld = as_colmajor(out)
    _check(_lib.cr_rnorm(_ptr(out), ld, n, M, seed, offset, _stream(stream)))
    return out


def trmm_sim(V: TileMat, Z, M: int, seed: int = 0, offset: int = 0, out=None, flags: int = 0,
             want_bnorm: bool = False, stream=None):
    """cr_trmm_sim: Z is n x M column-major FP64 (or None with CR_TRMM_GENERATE)."""
    import torch
    if out is None:
        out = colmajor_empty(V.n, M, torch.float64)
    out, ldy = as_colmajor(out)
    zp, ldz = (None, V.n)
    if Z is not None:
        Z, ldz = as_colmajor(Z)
        zp = _ptr(Z)
    bn = _D(0.0)
    _check(_lib.cr_trmm_sim(V.handle, zp, ldz, M, seed, offset, _ptr(out), ldy, flags,
                            ctypes.byref(bn) if want_bnorm else None, _stream(stream)))
    return (out, bn.value) if want_bnorm else out


def krige(V: TileMat, Xo, Xp, yo, stream=None):
    import torch
    n_o, n_p = Xo.shape[0], Xp.shape[0]
    Xo, _ = as_colmajor(Xo)
    Xp, _ = as_colmajor(Xp)
    W = colmajor_empty(n_o, n_p, torch.float64)
    zhat = torch.empty(n_p, dtype=torch.float64, device="cuda")
    v = torch.empty(n_p, dtype=torch.float64, device="cuda")
    info = _I(0)
    _check(_lib.cr_krige(V.handle, _ptr(Xo), _ptr(Xp), _ptr(yo.contiguous()), _ptr(W), n_o, _ptr(zhat), _ptr(v),
                         _stream(stream), ctypes.byref(info)))
    return W, zhat, v


def krige_correct(W, yo, Y, n_p: int, n_o: int, out=None, stream=None):
    import torch
    W, ldw = as_colmajor(W)
    Y, ldy = as_colmajor(Y)
    M = Y.shape[1]
    if out is None:
        out = colmajor_empty(n_p, M, torch.float64)
    out, lds = as_colmajor(out)
    _check(_lib.cr_krige_correct(_ptr(W), ldw, _ptr(yo.contiguous()), _ptr(Y), ldy, n_p, n_o, M, _ptr(out), lds,
                                 _stream(stream)))
    return out


def _calib_outputs(n_p: int, M: int, counts: bool, extrema: bool):
    import torch
    cin = torch.empty(n_p, dtype=torch.uint8, device="cuda")
    cout = torch.empty(n_p, dtype=torch.uint8, device="cuda")
    cnt = torch.empty(n_p, dtype=torch.int32, device="cuda") if counts else None
    psi = torch.empty(M, dtype=torch.float64, device="cuda") if extrema else None
    phi = torch.empty(M, dtype=torch.float64, device="cuda") if extrema else None
    return cin, cout, cnt, psi, phi, CalibInfo()


def _calib_dict(cin, cout, cnt, psi, phi, info, counts: bool, extrema: bool):
    out = {"q_in": info.q_in, "q_out": info.q_out, "n_psi": info.n_psi, "n_phi": info.n_phi, "c_in": cin,
           "c_out": cout}
    if counts:
        out["count"] = cnt
    if extrema:
        out["psi"], out["phi"] = psi, phi
    return out


def correct_calibrate(W, yo, Y, n_p: int, n_o: int, zhat, v, u: float, level: float, counts: bool = True,
                      extrema: bool = False, negative: bool = False, stream=None):
    """cr_correct_calibrate: the correction S = M_p + W^T (y_o 1^T - M_o) fused with the
    calibration (S is never formed); returns the dict of calibrate()."""
    W, ldw = as_colmajor(W)
    Y, ldy = as_colmajor(Y)
    M = Y.shape[1]
    cin, cout, cnt, psi, phi, info = _calib_outputs(n_p, M, counts, extrema)
    _check(_lib.cr_correct_calibrate(_ptr(W), ldw, _ptr(yo.contiguous()), _ptr(Y), ldy, n_p, n_o, M,
                                     _ptr(zhat.contiguous()), _ptr(v.contiguous()), u, level, 1 if negative else 0,
                                     _ptr(cin), _ptr(cout), _ptr(cnt), _ptr(psi), _ptr(phi), ctypes.byref(info),
                                     _stream(stream)))
    return _calib_dict(cin, cout, cnt, psi, phi, info, counts, extrema)


class Weights:
    """cr_weights: kriging weights W (n_o x n_p) prepared for repeated Ozaki corrections."""

    def __init__(self, W, stream=None):
        load()
        W, ldw = as_colmajor(W)
        self.n_o, self.n_p = W.shape
        h = _P()
        _check(_lib.cr_weights_prepare(_ptr(W), ldw, self.n_o, self.n_p, _stream(stream), ctypes.byref(h)))
        self.handle = h

    def close(self):
        if self.handle:
            _check(_lib.cr_weights_release(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def krige_correct_prepared(Wp: Weights, yo, Y, out=None, stream=None):
    """cr_krige_correct_prepared: the Ozaki correction with prepared weights; returns S."""
    import torch
    Y, ldy = as_colmajor(Y)
    M = Y.shape[1]
    if out is None:
        out = colmajor_empty(Wp.n_p, M, torch.float64)
    out, lds = as_colmajor(out)
    _check(_lib.cr_krige_correct_prepared(Wp.handle, _ptr(yo.contiguous()), _ptr(Y), ldy, M, _ptr(out), lds,
                                          _stream(stream)))
    return out


def correct_calibrate_prepared(Wp: Weights, yo, Y, zhat, v, u: float, level: float, counts: bool = True,
                               extrema: bool = False, negative: bool = False, stream=None):
    """cr_correct_calibrate_prepared: the Ozaki correction with prepared weights, then the
    calibration; returns the dict of calibrate()."""
    Y, ldy = as_colmajor(Y)
    M = Y.shape[1]
    cin, cout, cnt, psi, phi, info = _calib_outputs(Wp.n_p, M, counts, extrema)
    _check(_lib.cr_correct_calibrate_prepared(Wp.handle, _ptr(yo.contiguous()), _ptr(Y), ldy, M,
                                              _ptr(zhat.contiguous()), _ptr(v.contiguous()), u, level,
                                              1 if negative else 0, _ptr(cin), _ptr(cout), _ptr(cnt), _ptr(psi),
                                              _ptr(phi), ctypes.byref(info), _stream(stream)))
    return _calib_dict(cin, cout, cnt, psi, phi, info, counts, extrema)


def calibrate(S, zhat, v, u: float, level: float, counts: bool = True, extrema: bool = False, negative: bool = False,
              stream=None):
    """cr_calibrate (cr_calibrate_negative with negative=True: the negative excursion set);
    returns a dict with q_in, q_out, n_psi, n_phi, c_in, c_out and optionally count, psi, phi
    (CUDA tensors)."""
    import torch
    S, lds = as_colmajor(S)
    n_p, M = S.shape
    cin = torch.empty(n_p, dtype=torch.uint8, device="cuda")
    cout = torch.empty(n_p, dtype=torch.uint8, device="cuda")
    cnt = torch.empty(n_p, dtype=torch.int32, device="cuda") if counts else None
    psi = torch.empty(M, dtype=torch.float64, device="cuda") if extrema else None
    phi = torch.empty(M, dtype=torch.float64, device="cuda") if extrema else None
    info = CalibInfo()
    fn = _lib.cr_calibrate_negative if negative else _lib.cr_calibrate
    _check(fn(_ptr(S), lds, n_p, M, _ptr(zhat.contiguous()), _ptr(v.contiguous()), u, level,
                             _ptr(cin), _ptr(cout), _ptr(cnt), _ptr(psi), _ptr(phi), ctypes.byref(info),
                             _stream(stream)))
    out = {"q_in": info.q_in, "q_out": info.q_out, "n_psi": info.n_psi, "n_phi": info.n_phi, "c_in": cin,
           "c_out": cout}
    if counts:
        out["count"] = cnt
    if extrema:
        out["psi"], out["phi"] = psi, phi
    return out


# ---------------------------------------------------------------- trend network
# Plain functions of memory, without autograd: results of tensors that require gradients carry none.
# The *_backward functions are the gradients, to be called by the user or from a torch.autograd.Function.

_ACTS = {"none": CR_ACT_NONE, "relu": CR_ACT_RELU, "silu": CR_ACT_SILU, "gelu": CR_ACT_GELU}
_GATES = {"coeff": CR_GATE_COEFF, "convex": CR_GATE_CONVEX, "variance": CR_GATE_VARIANCE}
_INT_MAX = 2 ** 31 - 1   # the C entries' sizes: ctypes would cut larger ones to 32 bits
_types = None
_torch = None


def _ready() -> None:
    """Loads the library, and torch once for this section: a call is a few microseconds, in
    which import statements would show."""
    global _torch, _types
    if _torch is None:
        load()
        import torch
        _types = {torch.float32: CR_TYPE_F32, torch.float16: CR_TYPE_F16, torch.bfloat16: CR_TYPE_BF16,
                  torch.float8_e4m3fn: CR_TYPE_E4M3}
        _torch = torch


def _type_of(t, what: str) -> int:
    """CR_TYPE_* of a CUDA tensor."""
    k = _types.get(t.dtype)
    if k is None or not t.is_cuda:
        raise CrError(1, f"{what}: a CUDA tensor of FP32, FP16, BF16 or e4m3 is needed, not {t.dtype} on {t.device}")
    return k


def _matrix(t, n: int, m: int, dtype, what: str):
    """(tensor, address, leading dimension) of a column-major n x m matrix argument, copied if it
    is not column-major or its leading dimension passes the C int; (None, None, n) for None."""
    if t is None:
        return None, None, n
    if t.dtype is not dtype or not t.is_cuda or t.shape != (n, m):
        raise CrError(1, f"{what}: a CUDA matrix of shape {(n, m)} and {dtype} is needed, not "
                         f"{tuple(t.shape)} and {t.dtype} on {t.device}")
    s0, s1 = t.stride()
    if m == 1:
        s1 = n
    if (s0 != 1 and n > 1) or not n <= s1 <= _INT_MAX:
        t = t.T.contiguous().T
        s1 = n
    return t, t.data_ptr(), s1


def _vector(t, n: int, what: str):
    """(tensor, address) of an FP32 vector argument, copied if it is strided."""
    if t is None:
        return None, None
    if t.dtype is not _torch.float32 or not t.is_cuda or t.shape != (n,):
        raise CrError(1, f"{what}: an FP32 CUDA vector of {n} is needed, not {tuple(t.shape)} and {t.dtype} on {t.device}")
    if not t.is_contiguous():
        t = t.contiguous()
    return t, t.data_ptr()


def _empty(n: int, m: int, dtype, device):
    return _torch.empty_strided((n, m), (1, n), dtype=dtype, device=device)


def _on(stream, fn, *args, **kw):
    """fn with `stream` as the current stream, so that its outputs and copies belong to it; the
    memory of its arguments is kept until the stream has passed the call."""
    _ready()
    with _torch.cuda.stream(stream):
        for t in (*args, *kw.values()):
            if isinstance(t, _torch.Tensor) and t.is_cuda:
                t.record_stream(stream)
        return fn(*args, **kw)


def _raw_stream(device) -> int:
    return _torch._C._cuda_getCurrentRawStream(device.index)


def _code(table, name, what: str) -> int:
    k = table.get(name)
    if k is None:
        raise CrError(1, f"{what} is one of {sorted(table)}, not {name!r}")
    return k


def _shape(t, what: str):
    if t.dim() != 2:
        raise CrError(1, f"{what}: a matrix is needed, not {t.dim()} dimensions")
    n, m = t.shape
    if n > _INT_MAX or m > _INT_MAX:
        raise CrError(1, f"{what}: {n} x {m} is beyond the library's sizes, which end at 2^31 - 2^16")
    return n, m


def affine(W, X, bias=None, act: str = "none", residual=None, w_scale=None, x_scale=None, out_dtype=None,
           save: bool = False, out=None, stream=None):
    """cr_affine: Y = act(W^T X + bias) + residual for W (K, N) and X (K, M); e4m3 operands take
    w_scale (N) and x_scale (M).  out_dtype: FP32, FP16 or BF16 (default: X's, BF16 for e4m3).
    save=True returns (Y, Z) with Z the pre-activation that affine_backward reads."""
    if stream is not None:
        return _on(stream, affine, W, X, bias, act, residual, w_scale, x_scale, out_dtype, save, out)
    if _torch is None:
        _ready()
    kind = _type_of(X, "affine X")
    dtype, device = X.dtype, X.device
    K, M = _shape(X, "affine X")
    N = _shape(W, "affine W")[1]
    X, px, ldx = _matrix(X, K, M, dtype, "affine X")
    W, pw, ldw = _matrix(W, K, N, dtype, "affine W")
    if out is None:
        out_dtype = out_dtype or (_torch.bfloat16 if kind == CR_TYPE_E4M3 else dtype)
        out = _empty(N, M, out_dtype, device)
        py, ldy = out.data_ptr(), N
    else:
        out_dtype = out_dtype or out.dtype
        y, py, ldy = _matrix(out, N, M, out_dtype, "affine out")
        if y is not out:
            raise CrError(1, "affine out: a column-major matrix is needed")
    residual, pr, ldr = _matrix(residual, N, M, out_dtype, "affine residual")
    Z = _empty(N, M, out_dtype, device) if save else None
    bias, pb = _vector(bias, N, "affine bias")
    w_scale, pws = _vector(w_scale, N, "affine w_scale")
    x_scale, pxs = _vector(x_scale, M, "affine x_scale")
    _check(_lib.cr_affine(kind, pw, ldw, px, ldx, K, N, M, pws, pxs, pb, _code(_ACTS, act, "affine act"),
                          _type_of(out, "affine out"), pr, ldr, Z.data_ptr() if save else None, N, py, ldy,
                          _raw_stream(device)))
    return (out, Z) if save else out


def affine_backward(W, X, dY, Z=None, act: str = "none", need=(True, True, True), dw_dtype=None, stream=None):
    """cr_affine_backward: (dX, dW, dbias) of affine at the saved Z; need says which of the three
    are wanted (None for the others).  dw_dtype: X's type (default) or FP32."""
    if stream is not None:
        return _on(stream, affine_backward, W, X, dY, Z, act, need, dw_dtype)
    _ready()
    kind = _type_of(X, "affine_backward X")
    dtype, device = X.dtype, X.device
    K, M = _shape(X, "affine_backward X")
    N = _shape(W, "affine_backward W")[1]
    X, px, ldx = _matrix(X, K, M, dtype, "affine_backward X")
    W, pw, ldw = _matrix(W, K, N, dtype, "affine_backward W")
    dY, pdy, lddy = _matrix(dY, N, M, dtype, "affine_backward dY")
    Z, pz, ldz = _matrix(Z, N, M, dtype, "affine_backward Z")
    dX = _empty(K, M, dtype, device) if need[0] else None
    dW = _empty(K, N, dw_dtype or dtype, device) if need[1] else None
    db = _torch.empty(N, dtype=_torch.float32, device=device) if need[2] else None
    _check(_lib.cr_affine_backward(kind, pw, ldw, px, ldx, pdy, lddy, pz, ldz, K, N, M,
                                   _code(_ACTS, act, "affine_backward act"), _ptr(dX), K,
                                   _type_of(dW, "affine_backward dw_dtype") if need[1] else kind, _ptr(dW), K, _ptr(db),
                                   _raw_stream(device)))
    return dX, dW, db


def _rmsnorm(X, gamma, residual, eps, e4m3: bool):
    if _torch is None:
        _ready()
    kind = _type_of(X, "rmsnorm X")
    dtype, device = X.dtype, X.device
    D, T = _shape(X, "rmsnorm X")
    X, px, ldx = _matrix(X, D, T, dtype, "rmsnorm X")
    residual, pr, ldr = _matrix(residual, D, T, dtype, "rmsnorm residual")
    gamma, pg = _vector(gamma, D, "rmsnorm gamma")
    H = ph = scale = ps = None
    if residual is not None:
        H = _empty(D, T, dtype, device)
        ph = H.data_ptr()
    if e4m3:
        Y, out = _empty(D, T, _torch.float8_e4m3fn, device), CR_TYPE_E4M3
        scale = _torch.empty(T, dtype=_torch.float32, device=device)
        ps = scale.data_ptr()
    else:
        Y, out = _empty(D, T, dtype, device), kind
    _check(_lib.cr_rmsnorm(kind, px, ldx, pr, ldr, pg, D, T, eps, ph, D, out, Y.data_ptr(), D, ps, _raw_stream(device)))
    return Y, scale, H


def rmsnorm(X, gamma, residual=None, eps: float = 1e-6, stream=None):
    """cr_rmsnorm: (Y, H) with H = X + residual (None without one) and Y its normalised columns."""
    if stream is not None:
        return _on(stream, rmsnorm, X, gamma, residual, eps)
    Y, _, H = _rmsnorm(X, gamma, residual, eps, False)
    return Y, H


def rmsnorm_e4m3(X, gamma, residual=None, eps: float = 1e-6, stream=None):
    """cr_rmsnorm with the 8-bit output: (Y in e4m3, scale per column, H)."""
    if stream is not None:
        return _on(stream, rmsnorm_e4m3, X, gamma, residual, eps)
    return _rmsnorm(X, gamma, residual, eps, True)


def rmsnorm_backward(H, gamma, dY, dH=None, eps: float = 1e-6, stream=None):
    """cr_rmsnorm_backward: (dX, dgamma) at the sum H that rmsnorm returned (or its X)."""
    if stream is not None:
        return _on(stream, rmsnorm_backward, H, gamma, dY, dH, eps)
    _ready()
    kind = _type_of(H, "rmsnorm_backward H")
    dtype, device = H.dtype, H.device
    D, T = _shape(H, "rmsnorm_backward H")
    H, ph, ldh = _matrix(H, D, T, dtype, "rmsnorm_backward H")
    dY, pdy, lddy = _matrix(dY, D, T, dtype, "rmsnorm_backward dY")
    dH, pdh, lddh = _matrix(dH, D, T, dtype, "rmsnorm_backward dH")
    gamma, pg = _vector(gamma, D, "rmsnorm_backward gamma")
    dX = _empty(D, T, dtype, device)
    dgamma = _torch.empty(D, dtype=_torch.float32, device=device)
    _check(_lib.cr_rmsnorm_backward(kind, ph, ldh, pg, pdy, lddy, pdh, lddh, D, T, eps, dX.data_ptr(), D,
                                    dgamma.data_ptr(), _raw_stream(device)))
    return dX, dgamma


def _series(offsets, what: str):
    """(tensor, address, number of series) of the offsets."""
    if offsets is None:
        return None, None, 1
    if offsets.dtype is not _torch.int32 or offsets.dim() != 1 or offsets.shape[0] < 1 or not offsets.is_cuda:
        raise CrError(1, f"{what}: int32 CUDA offsets (series + 1) are needed")
    if offsets.shape[0] > _INT_MAX:
        raise CrError(1, f"{what}: {offsets.shape[0]} is beyond the library's sizes, which end at 2^31 - 2^16")
    offsets = offsets.contiguous()
    return offsets, offsets.data_ptr(), offsets.shape[0] - 1


def _saved_count(D: int, T: int) -> int:
    count = ctypes.c_size_t(0)
    _check(_lib.cr_gated_scan_saved(D, T, ctypes.byref(count)))
    return count.value


def gated_scan(G, X, gate: str = "convex", offsets=None, h0=None, save: bool = False, stream=None):
    """cr_gated_scan: (H, hT) for G and X (D, T) with packed series in the T columns; save=True
    returns (H, hT, saved), saved being what gated_scan_backward restarts from."""
    if stream is not None:
        return _on(stream, gated_scan, G, X, gate, offsets, h0, save)
    _ready()
    kind = _type_of(X, "gated_scan X")
    dtype, device, f32 = X.dtype, X.device, _torch.float32
    D, T = _shape(X, "gated_scan X")
    X, px, ldx = _matrix(X, D, T, dtype, "gated_scan X")
    G, pg, ldg = _matrix(G, D, T, dtype, "gated_scan G")
    offsets, po, n = _series(offsets, "gated_scan offsets")
    h0, p0, ld0 = _matrix(h0, D, n, f32, "gated_scan h0")
    H, hT = _empty(D, T, dtype, device), _empty(D, n, f32, device)
    saved = _torch.empty(_saved_count(D, T), dtype=f32, device=device) if save else None
    _check(_lib.cr_gated_scan(kind, _code(_GATES, gate, "gated_scan gate"), pg, ldg, px, ldx, D, T, po, n, p0, ld0,
                              H.data_ptr(), D, hT.data_ptr(), D, _ptr(saved), _raw_stream(device)))
    return (H, hT, saved) if save else (H, hT)


def gated_scan_backward(G, X, dH, gate: str = "convex", offsets=None, h0=None, dhT=None, saved=None, stream=None):
    """cr_gated_scan_backward: (dG, dX, dh0); saved is gated_scan's (None: recomputed)."""
    if stream is not None:
        return _on(stream, gated_scan_backward, G, X, dH, gate, offsets, h0, dhT, saved)
    _ready()
    kind = _type_of(X, "gated_scan_backward X")
    dtype, device, f32 = X.dtype, X.device, _torch.float32
    D, T = _shape(X, "gated_scan_backward X")
    X, px, ldx = _matrix(X, D, T, dtype, "gated_scan_backward X")
    G, pg, ldg = _matrix(G, D, T, dtype, "gated_scan_backward G")
    dH, pd, ldd = _matrix(dH, D, T, dtype, "gated_scan_backward dH")
    offsets, po, n = _series(offsets, "gated_scan_backward offsets")
    h0, p0, ld0 = _matrix(h0, D, n, f32, "gated_scan_backward h0")
    dhT, pt, ldt = _matrix(dhT, D, n, f32, "gated_scan_backward dhT")
    saved, ps = _vector(saved, _saved_count(D, T), "gated_scan_backward saved")
    dG, dX = _empty(D, T, dtype, device), _empty(D, T, dtype, device)
    dh0 = _empty(D, n, f32, device)
    _check(_lib.cr_gated_scan_backward(kind, _code(_GATES, gate, "gated_scan_backward gate"), pg, ldg, px, ldx, pd, ldd,
                                       D, T, po, n, p0, ld0, pt, ldt, ps, dG.data_ptr(), D, dX.data_ptr(), D,
                                       dh0.data_ptr(), D, _raw_stream(device)))
    return dG, dX, dh0


def gated_step(G, X, h, gate: str = "convex", out=None, stream=None):
    """cr_gated_step: (H, hnext) for one step of B series; out receives hnext and may be h."""
    if stream is not None:
        return _on(stream, gated_step, G, X, h, gate, out)
    if _torch is None:
        _ready()
    kind = _type_of(X, "gated_step X")
    dtype, device, f32 = X.dtype, X.device, _torch.float32
    D, B = _shape(X, "gated_step X")
    X, px, ldx = _matrix(X, D, B, dtype, "gated_step X")
    G, pg, ldg = _matrix(G, D, B, dtype, "gated_step G")
    h, ph, ldh = _matrix(h, D, B, f32, "gated_step h")
    if out is None:
        out = _empty(D, B, f32, device)
        pn, ldn = out.data_ptr(), D
    else:
        n, pn, ldn = _matrix(out, D, B, f32, "gated_step out")
        if n is not out:
            raise CrError(1, "gated_step out: a column-major matrix is needed")
    H = _empty(D, B, dtype, device)
    _check(_lib.cr_gated_step(kind, _code(_GATES, gate, "gated_step gate"), pg, ldg, px, ldx, ph, ldh, D, B,
                              H.data_ptr(), D, pn, ldn, _raw_stream(device)))
    return H, out
