"""Python binding of libkq (the MI355X HIP library for the online 4-bit activation path).

Argument marshalling only: every step of the path runs in the library's HIP kernels.
Tensors are torch tensors on the ROCm device (PyTorch provides device memory and the
stream); outputs are allocated here when not given.  The binding fails loudly if the
library is missing: there is no fallback.

    xf = kq.Xform.kron(A, B, K)                     # or Xform.rpbh(perm, sign), Xform.none(K)
    codes, scales, mu = kq.transform_quantize(X, xf, fmt="mxfp4", center=False)
    wcodes, wscales, wbar = kq.fold_inverse_into_weights(W, xf, fmt="mxfp4")     # W [K][N]
    Y = kq.w4a4_linear(codes, scales, wcodes, wscales, X=X, L1=L1, L2=L2, mu=mu, wbar=wbar)
    # or, with the down-projection done separately (or fused into the transform):
    T = kq.lowrank_down(X, L1)
    Y = kq.w4a4_linear_t(codes, scales, wcodes, wscales, T=T, L2=L2, mu=mu, wbar=wbar)

    # the 8-bit path: a gated feed-forward block behind its norm
    wc, ws = kq.quantize_fp8(W)                                 # offline, W [N][K]
    codes, scales, h = kq.rmsnorm_quantize_fp8(X, gamma, residual=h)
    codes, scales = kq.fp8_gated_linear(codes, scales, gate_up_codes, gate_up_scales, act="silu")
    X = kq.fp8_linear(codes, scales, down_codes, down_scales, dtype=X.dtype)

With ``stream`` a call runs with that stream as torch's current one: outputs and workspaces that
the binding allocates itself are then that stream's memory, so no work still pending on another
stream writes into them.  Outputs are also marked as used on the stream that was current before
the call (``record_stream``), where their user may drop them while its own work on them is pending.
Given tensors are the caller's to order.
"""

import ctypes
import os

__all__ = ["mfma_fp4_probe", "load", "lib_path", "abi_version", "status_str", "lloyd_max_levels", "Xform",
           "transform_quantize", "fold_inverse_into_weights", "fold_inverse_into_weights_nk",
           "w4a4_linear", "w4a4_linear_t", "w4a4_linear_workspace_bytes",
           "lowrank_down", "lowrank_down_workspace_bytes", "transform_quantize_lowrank",
           "svd_lowrank", "svd_lowrank_workspace_bytes", "fp8_scale_cols", "quantize_fp8", "rmsnorm_quantize_fp8",
           "fp8_linear", "fp8_gated_linear", "fp8_gated_linear_workspace_bytes",
           "KQError"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

KQ_OK = 0
XFORM_NONE, XFORM_KRON, XFORM_RPBH, XFORM_DENSE, XFORM_KRON_BLOCKS = 0, 1, 2, 3, 4
FMT_MXFP4, FMT_LM4, FMT_LM2 = 0, 1, 2
DT_F16, DT_BF16 = 0, 1
_PRECISE = 0x100
_ACT = {"silu": 0, "gelu": 1, "gelu_tanh": 2}
_FMT = {"mxfp4": FMT_MXFP4, "lm4": FMT_LM4, "lm2": FMT_LM2}


class KQError(RuntimeError):
    def __init__(self, status, what):
        super().__init__(f"{what}: {status_str(status)}")
        self.status = status


class _XformC(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("reserved", ctypes.c_int32), ("K", ctypes.c_int64),
                ("A", ctypes.c_float * 16), ("B", ctypes.c_float * 64),
                ("perm", ctypes.c_void_p), ("sign", ctypes.c_void_p), ("P", ctypes.c_void_p),
                ("AB", ctypes.c_void_p), ("pts", ctypes.c_void_p)]


def lib_path():
    return os.path.join(_HERE, "libkq.so")


def load():
    """Load libkq.so (built in-tree by build.py); raise if it is missing."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built; run `python -m w4a4_post_quantization_amd.build`")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.kq_abi_version.restype = i32
    lib.kq_abi_version.argtypes = []
    lib.kq_status_str.restype = ctypes.c_char_p
    lib.kq_status_str.argtypes = [i32]
    lib.kq_clock_probe.restype = i32
    lib.kq_clock_probe.argtypes = [i32, vp, vp]
    lib.kq_mfma_fp4_probe.restype = i32
    lib.kq_mfma_fp4_probe.argtypes = [i32, i32, vp, vp, vp]
    lib.kq_lloyd_max_levels.restype = i32
    lib.kq_lloyd_max_levels.argtypes = [i32, ctypes.POINTER(ctypes.c_double)]
    lib.kq_transform_quantize.restype = i32
    lib.kq_transform_quantize.argtypes = [ctypes.POINTER(_XformC), i32, i32, vp, i64, i64, vp, vp, vp, vp]
    lib.kq_fold_inverse_into_weights.restype = i32
    lib.kq_fold_inverse_into_weights.argtypes = [ctypes.POINTER(_XformC), i32, vp, i64, i64, vp, vp, vp, vp]
    lib.kq_fold_inverse_into_weights_nk.restype = i32
    lib.kq_fold_inverse_into_weights_nk.argtypes = [ctypes.POINTER(_XformC), i32, vp, i64, i64, vp, vp, vp, vp]
    lib.kq_lowrank_down.restype = i32
    lib.kq_lowrank_down.argtypes = [vp, vp, i64, i64, i32, vp, vp, ctypes.c_size_t, vp]
    lib.kq_lowrank_down_workspace_bytes.restype = ctypes.c_size_t
    lib.kq_lowrank_down_workspace_bytes.argtypes = [i64, i64, i32]
    lib.kq_transform_quantize_lowrank.restype = i32
    lib.kq_transform_quantize_lowrank.argtypes = [ctypes.POINTER(_XformC), i32, vp, i64, i64, vp, vp, vp, vp, i32,
                                                  vp, vp, ctypes.c_size_t, vp]
    lib.kq_svd_lowrank_workspace_bytes.restype = ctypes.c_size_t
    lib.kq_svd_lowrank_workspace_bytes.argtypes = [i64, i64, i32, i32]
    lib.kq_svd_lowrank.restype = i32
    lib.kq_svd_lowrank.argtypes = [vp, i64, i64, i32, vp, i32, i32, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.kq_w4a4_linear_workspace_bytes.restype = ctypes.c_size_t
    lib.kq_w4a4_linear_workspace_bytes.argtypes = [i64, i32]
    lib.kq_w4a4_linear.restype = i32
    lib.kq_w4a4_linear.argtypes = [i32, vp, vp, i64, i64, vp, vp, i64, vp, vp, vp, i32, vp, vp, vp, vp,
                                   ctypes.c_size_t, vp]
    lib.kq_w4a4_linear_noalloc.restype = i32
    lib.kq_w4a4_linear_noalloc.argtypes = [i32, vp, vp, i64, i64, vp, vp, i64, vp, vp, vp, i32, vp, vp, vp, vp]
    lib.kq_w4a4_linear_t.restype = i32
    lib.kq_w4a4_linear_t.argtypes = [i32, vp, vp, i64, i64, vp, vp, i64, vp, vp, i32, vp, vp, vp, vp]
    lib.kq_fp8_scale_cols.restype = i64
    lib.kq_fp8_scale_cols.argtypes = [i64]
    lib.kq_quantize_fp8.restype = i32
    lib.kq_quantize_fp8.argtypes = [i32, vp, i64, i64, vp, vp, vp]
    lib.kq_rmsnorm_quantize_fp8.restype = i32
    lib.kq_rmsnorm_quantize_fp8.argtypes = [i32, vp, vp, vp, ctypes.c_float, i64, i64, vp, vp, vp, vp]
    lib.kq_fp8_linear.restype = i32
    lib.kq_fp8_linear.argtypes = [i32, vp, vp, i64, i64, vp, vp, i64, vp, vp, vp]
    lib.kq_fp8_gated_linear_workspace_bytes.restype = sz
    lib.kq_fp8_gated_linear_workspace_bytes.argtypes = [i64, i64, i64]
    lib.kq_fp8_gated_linear.restype = i32
    lib.kq_fp8_gated_linear.argtypes = [i32, vp, vp, i64, i64, vp, vp, i64, vp, vp, vp, sz, vp]
    _LIB = lib
    return lib


def abi_version():
    return int(load().kq_abi_version())


def status_str(s):
    return load().kq_status_str(int(s)).decode()


def clock_probe(spin_us, out=None, stream=None):
    """Launch the shader-clock probe on `stream` (see kq_clock_probe): returns the device
    uint64 [2] tensor that will hold (shader cycles, 100 MHz reference ticks)."""
    if stream is not None:
        return _on(stream, clock_probe, spin_us, out)
    torch = _torch()
    if out is None:
        out = torch.empty((2,), dtype=torch.int64, device="cuda")      # no fill kernel to race with
    _check(out, "out", torch.int64, (2,))
    s = load().kq_clock_probe(int(spin_us), _ptr(out), _stream())
    if s != KQ_OK:
        raise KQError(s, "kq_clock_probe")
    return out


def mfma_fp4_probe(iters, workgroups, codes, out=None, stream=None):
    """Launch the FP4 matrix-core rate probe on `stream` (see kq_mfma_fp4_probe): `codes` is a
    device uint8 tensor of at least 2048 bytes (its first 2048 are the operands); returns the
    float32 [4 * workgroups] tensor of per-wavefront sums.  The caller times the launch; the
    work is 64 * iters * workgroups products of 2 * 32 * 32 * 64 flops."""
    if stream is not None:
        return _on(stream, mfma_fp4_probe, iters, workgroups, codes, out)
    torch = _torch()
    if codes.dtype != torch.uint8 or not codes.is_cuda or not codes.is_contiguous() or codes.numel() < 2048:
        raise ValueError("codes must be a contiguous device uint8 tensor of at least 2048 bytes")
    if out is None:
        out = torch.empty((4 * int(workgroups),), dtype=torch.float32, device=codes.device)
    _check(out, "out", torch.float32, (4 * int(workgroups),))
    s = load().kq_mfma_fp4_probe(int(iters), int(workgroups), _ptr(codes), _ptr(out), _stream())
    if s != KQ_OK:
        raise KQError(s, "kq_mfma_fp4_probe")
    return out


def lloyd_max_levels(n):
    """Positive levels of the library's n-level (4 or 16) Lloyd-Max codebook (host call)."""
    out = (ctypes.c_double * (n // 2))()
    s = load().kq_lloyd_max_levels(n, out)
    if s != KQ_OK:
        raise KQError(s, "kq_lloyd_max_levels")
    return [float(v) for v in out]


# ------------------------------------------------------------------ marshalling helpers

_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(_torch().cuda.current_stream().cuda_stream)


def _on(stream, f, *args, **kw):
    """f(*args, **kw) with `stream` as the current stream.  Memory of the allocator belongs to the
    stream it was allocated for: taken for another one, its last owner's kernels may still be
    writing to it.  Outputs made here are recorded on the caller's stream as well."""
    torch = _torch()
    here = torch.cuda.current_stream(stream.device)
    device = torch.cuda.current_device()
    if stream == here and stream.device.index == device:
        return f(*args, **kw)
    torch.cuda.set_stream(stream)                            # and its device; 5 us less than the context manager
    try:
        out = f(*args, **kw)
    finally:
        torch.cuda.set_stream(here)
        if stream.device.index != device:
            torch.cuda.set_device(device)
    given = [id(t) for t in (*args, *kw.values())]
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None and id(t) not in given:
            t.record_stream(here)
    return out


def _check(t, name, dtype, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on the GPU (got {t.device})")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)} (got {tuple(t.shape)})")
    return t


class Xform:
    """One layer's block transform descriptor (KRON_4X8, RPBH_32, DENSE_32 or NONE)."""

    def __init__(self, kind, K, A=None, B=None, perm=None, sign=None, P=None, AB=None, pts=None):
        self.kind, self.K = kind, int(K)
        self._c = _XformC()
        self._c.kind, self._c.reserved, self._c.K = kind, 0, self.K
        if kind == XFORM_KRON:
            a = [float(v) for v in _flat(A)]
            b = [float(v) for v in _flat(B)]
            if len(a) != 16 or len(b) != 64:
                raise ValueError("A must be 4x4 and B 8x8")
            self._c.A[:] = a
            self._c.B[:] = b
        self.perm, self.sign = perm, sign      # keep the device arrays alive
        if kind == XFORM_RPBH:
            torch = _torch()
            _check(perm, "perm", torch.int32, (self.K,))
            _check(sign, "sign", torch.int8, (self.K,))
            self._c.perm, self._c.sign = perm.data_ptr(), sign.data_ptr()
        self.P = P
        if kind == XFORM_DENSE:
            torch = _torch()
            _check(P, "P", torch.float32, (32, 32))
            self._c.P = P.data_ptr()
        self.AB = AB
        if kind == XFORM_KRON_BLOCKS:
            _check(AB, "AB", _torch().float32, (self.K // 32, 80))
            self._c.AB = AB.data_ptr()
        self.pts = pts
        if pts is not None:
            _check(pts, "pts", _torch().int8, (self.K,))
            self._c.pts = pts.data_ptr()

    def with_pts(self, pts):
        """The same transform preceded by power-of-two channel scaling: pts is an int8 [K]
        device tensor of exponents (0..15); x_k -> fp16(x_k 2^-pts[k]), weights x 2^pts[k]."""
        return Xform(self.kind, self.K, A=list(self._c.A), B=list(self._c.B), perm=self.perm, sign=self.sign,
                     P=self.P, AB=self.AB, pts=pts)

    @classmethod
    def kron(cls, A, B, K):
        return cls(XFORM_KRON, K, A=A, B=B)

    @classmethod
    def kron_blocks(cls, AB, K):
        """AB: float32 [K/32][80] device tensor, row b = A_b (4x4) then B_b (8x8), row-major;
        block b of every token becomes x_b . (A_b (x) B_b)."""
        return cls(XFORM_KRON_BLOCKS, K, AB=AB)

    @staticmethod
    def pack_block_factors(A, B):
        """Host helper: A [nb][4][4], B [nb][8][8] -> the float32 [nb][80] table (numpy)."""
        import numpy as np
        A = np.asarray(A, dtype=np.float32)
        B = np.asarray(B, dtype=np.float32)
        return np.ascontiguousarray(np.concatenate([A.reshape(len(A), 16), B.reshape(len(B), 64)], axis=1))

    @classmethod
    def dense(cls, P, K):
        """P: float32 [32][32] device tensor, y_b = x_b . P for every block."""
        return cls(XFORM_DENSE, K, P=P)

    @classmethod
    def rpbh(cls, perm, sign):
        return cls(XFORM_RPBH, perm.shape[0], perm=perm, sign=sign)

    @classmethod
    def none(cls, K):
        return cls(XFORM_NONE, K)

    def c(self):
        return ctypes.byref(self._c)


def _flat(a):
    try:
        import numpy as np
        return np.asarray(a, dtype=np.float32).reshape(-1).tolist()
    except Exception:
        return list(a)


def transform_quantize(X, xform, fmt="mxfp4", center=False, codes=None, scales=None, mu=None, stream=None):
    """[centre] -> block transform -> 4-bit quantize + pack.  Returns (codes, scales, mu)."""
    if stream is not None:
        return _on(stream, transform_quantize, X, xform, fmt, center, codes, scales, mu)
    torch = _torch()
    _check(X, "X", torch.float16)
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M, K]")
    M, K = X.shape
    f = _FMT[fmt]
    if f not in (FMT_MXFP4, FMT_LM4):
        raise ValueError("fmt must be 'mxfp4' or 'lm4'")
    dev = X.device
    if codes is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    _check(codes, "codes", torch.uint8, (M, K // 2))
    if scales is None:
        scales = torch.empty((M, K // 32) if f == FMT_MXFP4 else (M,),
                             dtype=torch.uint8 if f == FMT_MXFP4 else torch.float32, device=dev)
    if f == FMT_MXFP4:
        _check(scales, "scales", torch.uint8, (M, K // 32))
    else:
        _check(scales, "scales", torch.float32, (M,))
    if center:
        if mu is None:
            mu = torch.empty((M,), dtype=torch.float16, device=dev)
        _check(mu, "mu", torch.float16, (M,))
    else:
        mu = None
    s = load().kq_transform_quantize(xform.c(), f, int(bool(center)), _ptr(X), M, K, _ptr(codes), _ptr(scales),
                                     _ptr(mu), _stream())
    if s != KQ_OK:
        raise KQError(s, "kq_transform_quantize")
    return codes, scales, mu


def _fold(name, W, N, K, xform, fmt, with_wbar):
    torch = _torch()
    f = _FMT[fmt]
    dev = W.device
    if f == FMT_MXFP4:
        wcodes = torch.empty((N, K // 2), dtype=torch.uint8, device=dev)
        wscales = torch.empty((N, K // 32), dtype=torch.uint8, device=dev)
    elif f == FMT_LM2:
        wcodes = torch.empty((N, K // 4), dtype=torch.uint8, device=dev)
        wscales = torch.empty((N, K // 32), dtype=torch.float16, device=dev)
    else:
        raise ValueError("fmt must be 'mxfp4' or 'lm2'")
    wbar = torch.empty((N,), dtype=torch.float16, device=dev) if with_wbar else None
    fn = getattr(load(), name)
    if name == "kq_fold_inverse_into_weights":
        s = fn(xform.c(), f, _ptr(W), K, N, _ptr(wcodes), _ptr(wscales), _ptr(wbar), _stream())
    else:
        s = fn(xform.c(), f, _ptr(W), N, K, _ptr(wcodes), _ptr(wscales), _ptr(wbar), _stream())
    if s != KQ_OK:
        raise KQError(s, name)
    return wcodes, wscales, wbar


def fold_inverse_into_weights(W, xform, fmt="mxfp4", with_wbar=True, stream=None):
    """Offline: W' = P^-1 W, quantized along K.  W is fp16 [K][N] (Y = X W).
    Returns (wcodes [N][K/2], wscales [N][K/32], wbar [N] or None)."""
    if stream is not None:
        return _on(stream, fold_inverse_into_weights, W, xform, fmt, with_wbar)
    torch = _torch()
    _check(W, "W", torch.float16)
    if W.dim() != 2:
        raise ValueError("W must be 2-D [K, N]")
    K, N = W.shape
    return _fold("kq_fold_inverse_into_weights", W, N, K, xform, fmt, with_wbar)


def fold_inverse_into_weights_nk(Wt, xform, fmt="mxfp4", with_wbar=True, stream=None):
    """The same fold for weights in the [out][in] layout: Wt is fp16 [N][K]."""
    if stream is not None:
        return _on(stream, fold_inverse_into_weights_nk, Wt, xform, fmt, with_wbar)
    torch = _torch()
    _check(Wt, "Wt", torch.float16)
    if Wt.dim() != 2:
        raise ValueError("Wt must be 2-D [N, K]")
    N, K = Wt.shape
    return _fold("kq_fold_inverse_into_weights_nk", Wt, N, K, xform, fmt, with_wbar)


def lowrank_down_workspace_bytes(M, K, r):
    """Workspace bytes that let kq_lowrank_down split K over workgroups (0: no split)."""
    return int(load().kq_lowrank_down_workspace_bytes(M, K, r))


def lowrank_down(X, L1, T=None, workspace=None, stream=None):
    """T = fp16(X L1^T): the low-rank branch's down-projection (fp16 [M][r]).  workspace:
    a uint8 device tensor for the split-K partials; by default one of the size
    lowrank_down_workspace_bytes is taken from torch's allocator."""
    if stream is not None:
        return _on(stream, lowrank_down, X, L1, T, workspace)
    torch = _torch()
    _check(X, "X", torch.float16)
    M, K = X.shape
    r = L1.shape[0]
    _check(L1, "L1", torch.float16, (r, K))
    if T is None:
        T = torch.empty((M, r), dtype=torch.float16, device=X.device)
    _check(T, "T", torch.float16, (M, r))
    if workspace is None:
        nb = lowrank_down_workspace_bytes(M, K, r)
        workspace = torch.empty((nb,), dtype=torch.uint8, device=X.device) if nb else None
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8)
    wp, wn = (_ptr(workspace), workspace.numel()) if workspace is not None else (None, 0)
    s = load().kq_lowrank_down(_ptr(X), _ptr(L1), M, K, r, _ptr(T), wp, wn, _stream())
    if s != KQ_OK:
        raise KQError(s, "kq_lowrank_down")
    return T


def transform_quantize_lowrank(X, xform, L1, center=False, codes=None, scales=None, mu=None, T=None, workspace=None,
                               stream=None):
    """One pass over X: MXFP4 codes and scales of the (optionally centred, RPBH only)
    block-transformed X and the low-rank down-projection T = fp16(X L1^T).
    Returns (codes, scales, mu or None, T)."""
    if stream is not None:
        return _on(stream, transform_quantize_lowrank, X, xform, L1, center, codes, scales, mu, T, workspace)
    torch = _torch()
    _check(X, "X", torch.float16)
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M, K]")
    M, K = X.shape
    r = L1.shape[0]
    _check(L1, "L1", torch.float16, (r, K))
    dev = X.device
    if codes is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    _check(codes, "codes", torch.uint8, (M, K // 2))
    if scales is None:
        scales = torch.empty((M, K // 32), dtype=torch.uint8, device=dev)
    _check(scales, "scales", torch.uint8, (M, K // 32))
    if center:
        if mu is None:
            mu = torch.empty((M,), dtype=torch.float16, device=dev)
        _check(mu, "mu", torch.float16, (M,))
    else:
        mu = None
    if T is None:
        T = torch.empty((M, r), dtype=torch.float16, device=dev)
    _check(T, "T", torch.float16, (M, r))
    if workspace is None:
        nb = lowrank_down_workspace_bytes(M, K, r)
        workspace = torch.empty((nb,), dtype=torch.uint8, device=dev) if nb else None
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8)
    wp, wn = (_ptr(workspace), workspace.numel()) if workspace is not None else (None, 0)
    s = load().kq_transform_quantize_lowrank(xform.c(), int(bool(center)), _ptr(X), M, K, _ptr(codes), _ptr(scales),
                                             _ptr(mu), _ptr(L1), r, _ptr(T), wp, wn, _stream())
    if s != KQ_OK:
        raise KQError(s, "kq_transform_quantize_lowrank")
    return codes, scales, mu, T


def svd_lowrank_workspace_bytes(N, K, r, l):
    return int(load().kq_svd_lowrank_workspace_bytes(N, K, r, l))


def svd_lowrank(W, r, omega, iters=4, L1=None, L2=None, R=None, sigma=None, workspace=None, stream=None):
    """Offline rank-r extraction: W (fp16 [N][K]) ~ L2 L1 + R.  omega: float32 [K][l]
    device starting block (l > r).  Returns (L1 [r][K], L2 [N][r], R [N][K], sigma [r])."""
    if stream is not None:
        return _on(stream, svd_lowrank, W, r, omega, iters, L1, L2, R, sigma, workspace)
    torch = _torch()
    _check(W, "W", torch.float16)
    N, K = W.shape
    _check(omega, "omega", torch.float32)
    if omega.dim() != 2 or omega.shape[0] != K:
        raise ValueError("omega must be [K, l]")
    l = omega.shape[1]
    dev = W.device

    def _new(shape, dtype):
        return torch.empty(shape, dtype=dtype, device=dev)
    L1 = _new((r, K), torch.float16) if L1 is None else L1
    L2 = _new((N, r), torch.float16) if L2 is None else L2
    R = _new((N, K), torch.float16) if R is None else R
    sigma = _new((r,), torch.float32) if sigma is None else sigma
    _check(L1, "L1", torch.float16, (r, K))
    _check(L2, "L2", torch.float16, (N, r))
    _check(R, "R", torch.float16, (N, K))
    _check(sigma, "sigma", torch.float32, (r,))
    nb = svd_lowrank_workspace_bytes(N, K, r, l)
    if workspace is None:
        workspace = _new((max(nb, 256),), torch.uint8)
    _check(workspace, "workspace", torch.uint8)
    s = load().kq_svd_lowrank(_ptr(W), N, K, r, _ptr(omega), l, int(iters), _ptr(L1), _ptr(L2), _ptr(R),
                              _ptr(sigma), _ptr(workspace), workspace.numel(), _stream())
    if s != KQ_OK:
        raise KQError(s, "kq_svd_lowrank")
    return L1, L2, R, sigma


def _linear_operands(xcodes, xscales, wcodes, wscales, fmt):
    torch = _torch()
    f = _FMT[fmt]
    _check(xcodes, "xcodes", torch.uint8)
    M = xcodes.shape[0]
    K = xcodes.shape[1] * 2
    N = wcodes.shape[0]
    _check(wcodes, "wcodes", torch.uint8, (N, K // 2) if f == FMT_MXFP4 else (N, K // 4))
    if f == FMT_MXFP4:
        _check(xscales, "xscales", torch.uint8, (M, K // 32))
        _check(wscales, "wscales", torch.uint8, (N, K // 32))
    else:
        _check(xscales, "xscales", torch.float32, (M,))
        _check(wscales, "wscales", torch.float16, (N, K // 32))
    return f, M, K, N


def _linear_tail(M, N, mu, wbar, Y, dev):
    torch = _torch()
    if mu is not None:
        _check(mu, "mu", torch.float16, (M,))
        _check(wbar, "wbar", torch.float16, (N,))
    Y = torch.empty((M, N), dtype=torch.float16, device=dev) if Y is None else Y
    return _check(Y, "Y", torch.float16, (M, N))


def w4a4_linear_workspace_bytes(M, r):
    """Workspace bytes kq_w4a4_linear needs for M tokens and rank r (0 when r == 0)."""
    return int(load().kq_w4a4_linear_workspace_bytes(M, r))


def w4a4_linear(xcodes, xscales, wcodes, wscales, X=None, L1=None, L2=None, mu=None, wbar=None,
                fmt="mxfp4", Y=None, workspace=None, stream=None):
    """Y = Xq Wq^T + (X L1^T) L2^T + mu wbar^T (fp16 [M][N]): the down-projection of the
    low-rank branch runs inside the call (its result held in the workspace).  X fp16
    [M][K], L1 fp16 [r][K], L2 fp16 [N][r].  workspace: a uint8 device tensor of at least
    w4a4_linear_workspace_bytes(M, r) bytes (256-byte aligned); by default one is taken
    from torch's allocator.  fmt 'mxfp4' (W4A4) or 'lm2' (W2A4, no branches)."""
    if stream is not None:
        return _on(stream, w4a4_linear, xcodes, xscales, wcodes, wscales, X, L1, L2, mu, wbar, fmt, Y, workspace)
    torch = _torch()
    f, M, K, N = _linear_operands(xcodes, xscales, wcodes, wscales, fmt)
    r = 0
    if L1 is not None:
        r = L1.shape[0]
        _check(X, "X", torch.float16, (M, K))
        _check(L1, "L1", torch.float16, (r, K))
        _check(L2, "L2", torch.float16, (N, r))
    Y = _linear_tail(M, N, mu, wbar, Y, xcodes.device)
    if r and workspace is None:
        workspace = torch.empty((w4a4_linear_workspace_bytes(M, r),), dtype=torch.uint8, device=xcodes.device)
    if workspace is not None:
        _check(workspace, "workspace", torch.uint8)
    wp, wn = (_ptr(workspace), workspace.numel()) if workspace is not None else (None, 0)
    s = load().kq_w4a4_linear(f, _ptr(xcodes), _ptr(xscales), M, K, _ptr(wcodes), _ptr(wscales), N,
                              _ptr(X if r else None), _ptr(L1 if r else None), _ptr(L2 if r else None), r,
                              _ptr(mu), _ptr(wbar), _ptr(Y), wp, wn, _stream())
    if s != KQ_OK:
        raise KQError(s, "kq_w4a4_linear")
    return Y


def w4a4_linear_t(xcodes, xscales, wcodes, wscales, T=None, L2=None, mu=None, wbar=None,
                  fmt="mxfp4", Y=None, stream=None):
    """Y = Xq Wq^T + T L2^T + mu wbar^T (fp16 [M][N]) with the down-projection T (fp16
    [M][r]) already computed.  fmt 'mxfp4' (W4A4) or 'lm2' (W2A4)."""
    if stream is not None:
        return _on(stream, w4a4_linear_t, xcodes, xscales, wcodes, wscales, T, L2, mu, wbar, fmt, Y)
    torch = _torch()
    f, M, K, N = _linear_operands(xcodes, xscales, wcodes, wscales, fmt)
    r = 0
    if T is not None:
        r = T.shape[1]
        _check(T, "T", torch.float16, (M, r))
        _check(L2, "L2", torch.float16, (N, r))
    Y = _linear_tail(M, N, mu, wbar, Y, xcodes.device)
    s = load().kq_w4a4_linear_t(f, _ptr(xcodes), _ptr(xscales), M, K, _ptr(wcodes), _ptr(wscales), N,
                                _ptr(T), _ptr(L2 if r else None), r, _ptr(mu), _ptr(wbar), _ptr(Y),
                                _stream())
    if s != KQ_OK:
        raise KQError(s, "kq_w4a4_linear_t")
    return Y


# ------------------------------------------------------------------------- the 8-bit path
# One-token calls take 2 to 14 us on the GPU, so the host side is kept short: one combined test
# per given tensor (the named refusal is worked out only when it fails), none for those made
# here, and one library call.

def _matrix(t, name):
    if not isinstance(t, _torch().Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D torch.Tensor")
    return t.shape


def _dtype16(torch, dtype, name):
    if dtype is torch.bfloat16:
        return DT_BF16
    if dtype is torch.float16:
        return DT_F16
    raise ValueError(f"{name} must be torch.float16 or torch.bfloat16 (got {dtype})")


def _same(t, name, dtype, shape, index):
    """t: a contiguous tensor of the dtype and shape on GPU `index`; its address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0 and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    _check(t, name, dtype, shape)
    raise ValueError(f"{name} is on {t.device}, the first tensor on GPU {index}")


def _call(torch, name, index, args):
    """One library call on the current stream of the tensors' GPU, which is made the current device
    for the call if it is not."""
    raw = torch._C._cuda_getCurrentRawStream(index)
    fn = getattr(_LIB or load(), name)
    if torch._C._cuda_getDevice() == index:
        s = fn(*args, raw)
    else:
        with torch.cuda.device(index):
            s = fn(*args, raw)
    if s != KQ_OK:
        raise KQError(s, name)


def _on_fp8(stream, first, f, *args, **kw):
    """_on for a call whose first tensor is `first`: its GPU must be the stream's."""
    if isinstance(first, _torch().Tensor) and first.is_cuda and stream.device.index != first.get_device():
        raise ValueError(f"{f.__name__}: the stream is on {stream.device}, the tensors on GPU {first.get_device()}")
    return _on(stream, f, first, *args, **kw)


def fp8_scale_cols(K):
    """Scale bytes of a row of K values: one per 128, padded to a multiple of four."""
    return (K + 511) // 512 * 4


def _fp8_out(torch, rows, K, codes, scales, index, like=None):
    """codes and scales (made here where not given) and their addresses; like: a checked tensor of
    codes' shape.  torch makes a tensor in 1.2 us like another, 1.3 from shape and strides, 1.7 from
    a shape alone."""
    if codes is None:
        if like is None:
            codes = torch.empty_strided((rows, K), (K, 1), dtype=torch.float8_e4m3fn, device=index)
        else:
            codes = torch.empty_like(like, dtype=torch.float8_e4m3fn)
        c = codes.data_ptr()
    else:
        c = _same(codes, "codes", torch.float8_e4m3fn, (rows, K), index)
    cols = (K + 511) // 512 * 4
    if scales is None:
        scales = torch.empty_strided((rows, cols), (cols, 1), dtype=torch.uint8, device=index)
        return codes, scales, c, scales.data_ptr()
    return codes, scales, c, _same(scales, "scales", torch.uint8, (rows, cols), index)


def quantize_fp8(X, codes=None, scales=None, stream=None):
    """E4M3 codes (float8_e4m3fn [M][K]) and E8M0 scale bytes (uint8 [M][fp8_scale_cols(K)],
    one per 128 values) of X (fp16 or bf16 [M][K], K a multiple of 16).  Also for weights
    [N][K], offline."""
    if stream is not None:
        return _on_fp8(stream, X, quantize_fp8, codes, scales)
    torch = _torch()
    shape = M, K = _matrix(X, "X")
    dtype, index = X.dtype, X.get_device()
    dt = _dtype16(torch, dtype, "X")
    x = _same(X, "X", dtype, shape, index)
    codes, scales, c, s = _fp8_out(torch, M, K, codes, scales, index, X)
    _call(torch, "kq_quantize_fp8", index, (dt, x, M, K, c, s))
    return codes, scales


def rmsnorm_quantize_fp8(X, gamma, eps=1e-6, residual=None, codes=None, scales=None, residual_out=None, stream=None):
    """h = X + residual; codes and scales (as quantize_fp8) of h / sqrt(mean h^2 + eps) * gamma.
    X, residual fp16 or bf16 [M][K], gamma [K] of the same dtype, K <= 16384.  Returns (codes,
    scales, h rounded to the dtype); the last is None without a residual, and residual_out (where h
    is to go) is then refused.  residual_out may be residual itself (updated in place)."""
    if residual is None and residual_out is not None:
        raise ValueError("residual_out is given without a residual: h is X itself")
    if stream is not None:
        return _on_fp8(stream, X, rmsnorm_quantize_fp8, gamma, eps, residual, codes, scales, residual_out)
    torch = _torch()
    shape = M, K = _matrix(X, "X")
    dtype, index = X.dtype, X.get_device()
    dt = _dtype16(torch, dtype, "X")
    x = _same(X, "X", dtype, shape, index)
    g = _same(gamma, "gamma", dtype, (K,), index)
    r = o = None
    if residual is not None:
        r = _same(residual, "residual", dtype, shape, index)
        if residual_out is None:
            residual_out = torch.empty_like(X)
            o = residual_out.data_ptr()
        else:
            o = _same(residual_out, "residual_out", dtype, shape, index)
    codes, scales, c, s = _fp8_out(torch, M, K, codes, scales, index, X)
    _call(torch, "kq_rmsnorm_quantize_fp8", index, (dt, x, r, g, eps, M, K, c, s, o))
    return codes, scales, residual_out


def _fp8_operands(torch, xcodes, xscales, wcodes, wscales):
    """M, N, K, the GPU and the addresses of both operands."""
    f8, u8 = torch.float8_e4m3fn, torch.uint8
    shape = M, K = _matrix(xcodes, "xcodes")
    N = _matrix(wcodes, "wcodes")[0]
    index, cols = xcodes.get_device(), (K + 511) // 512 * 4
    return (M, N, K, index, _same(xcodes, "xcodes", f8, shape, index), _same(xscales, "xscales", u8, (M, cols), index),
            _same(wcodes, "wcodes", f8, (N, K), index), _same(wscales, "wscales", u8, (N, cols), index))


def fp8_linear(xcodes, xscales, wcodes, wscales, bias=None, dtype=None, Y=None, stream=None, precise=False):
    """Y = Xq Wq^T (+ bias), fp16 or bf16 [M][N], float32 accumulation.  xcodes [M][K] and
    wcodes [N][K] float8_e4m3fn with their scale bytes (quantize_fp8); N a multiple of 16; bias
    [N] of Y's dtype.  dtype: Y's (default: Y's own, the bias's, or float16, where sums past 65504
    turn infinite).  precise: every
    product exact and added in float32, as up to 16 tokens always; else calls of more tokens take
    the 8-bit matrix instructions, which cut products off at 2^-13 of the largest of each eight and
    are up to twice as fast (KQ_FP8_PRECISE in kq.h)."""
    if stream is not None:
        return _on_fp8(stream, xcodes, fp8_linear, xscales, wcodes, wscales, bias, dtype, Y, precise=precise)
    torch = _torch()
    M, N, K, index, x, xs, w, ws = _fp8_operands(torch, xcodes, xscales, wcodes, wscales)
    if dtype is None:
        like = Y if Y is not None else bias
        dtype = torch.float16 if like is None else getattr(like, "dtype", type(like))
    dt = _dtype16(torch, dtype, "dtype")
    b = None if bias is None else _same(bias, "bias", dtype, (N,), index)
    if Y is None:
        Y = torch.empty_strided((M, N), (N, 1), dtype=dtype, device=index)
        y = Y.data_ptr()
    else:
        y = _same(Y, "Y", dtype, (M, N), index)
    _call(torch, "kq_fp8_linear", index, (dt | _PRECISE if precise else dt, x, xs, M, K, w, ws, N, b, y))
    return Y


def fp8_gated_linear_workspace_bytes(M, F, K):
    """Workspace bytes kq_fp8_gated_linear needs (0: none)."""
    return load().kq_fp8_gated_linear_workspace_bytes(M, F, K)


def fp8_gated_linear(xcodes, xscales, wcodes, wscales, act="silu", codes=None, scales=None, workspace=None,
                     stream=None, precise=False):
    """codes and scales (as quantize_fp8, [M][F]) of act(Xq Wg^T) * (Xq Wu^T).  wcodes [2 F][K]
    holds the F rows of Wg, then the F rows of Wu; F a multiple of 16.  act: 'silu', 'gelu' or
    'gelu_tanh'.  The result feeds fp8_linear with the down-projection's weights.  workspace: a
    uint8 device tensor of fp8_gated_linear_workspace_bytes(M, F, K) bytes (256-byte aligned); by
    default one is taken from torch's allocator.  precise: as in fp8_linear."""
    if stream is not None:
        return _on_fp8(stream, xcodes, fp8_gated_linear, xscales, wcodes, wscales, act, codes, scales, workspace,
                       precise=precise)
    torch = _torch()
    if act not in _ACT:
        raise ValueError(f"act must be one of {sorted(_ACT)} (got {act!r})")
    M, N, K, index, x, xs, w, ws = _fp8_operands(torch, xcodes, xscales, wcodes, wscales)
    if N % 2:
        raise ValueError("wcodes must hold as many gate rows as up rows")
    F = N // 2
    codes, scales, c, s = _fp8_out(torch, M, F, codes, scales, index)
    wk = nb = 0
    if workspace is not None:
        wk = _same(workspace, "workspace", torch.uint8, getattr(workspace, "shape", None), index)
        nb = workspace.numel()
    else:
        nb = fp8_gated_linear_workspace_bytes(M, F, K)
        if nb:
            workspace = torch.empty((nb,), dtype=torch.uint8, device=index)
            wk = workspace.data_ptr()
    _call(torch, "kq_fp8_gated_linear", index, (_ACT[act] | _PRECISE if precise else _ACT[act], x, xs, M, K, w, ws, F, c, s, wk or None, nb))
    return codes, scales
