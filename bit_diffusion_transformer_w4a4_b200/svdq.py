"""Python binding of libsvdq (include/svdq.h) -- argument marshalling only.

Every step of the layer runs in the library's CUDA kernels; this module only
converts numpy / torch buffers into pointers, passes the current CUDA stream
and raises on non-OK status codes.  There is no CPU fallback: if the shared
library is missing or the device is not an sm_100 GPU, calls raise.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os

import numpy as np

from . import build as _build

INT4 = 0
NVFP4 = 1
EPI_GELU = 1
GEMM_SINGLE_SM = 2
INT4_F16 = 4
EPI_QKV_NORM_ROPE = 8

STATUS = {
    0: "SVDQ_OK", 1: "SVDQ_ERR_INVALID_ARG", 2: "SVDQ_ERR_SHAPE", 3: "SVDQ_ERR_ALIGNMENT",
    4: "SVDQ_ERR_UNSUPPORTED_DEVICE", 5: "SVDQ_ERR_OOM", 6: "SVDQ_ERR_CUDA",
    7: "SVDQ_ERR_DEVICE_TIMEOUT", 8: "SVDQ_ERR_RANGE",
}

EXPORTED = [
    "svdq_weights_load", "svdq_weights_free", "svdq_act_scales_bytes",
    "svdq_quantize_act_lowrank_down", "svdq_w4a4_gemm_lowrank_up", "svdq_linear_forward",
    "svdq_linear_forward_host", "svdq_device_status", "svdq_debug_set_fault",
    "svdq_selftest_division", "svdq_status_string", "svdq_version",
    "svdq_quantize_act_lowrank_down_static",
    "svdq_awq_load", "svdq_awq_free", "svdq_awq_w4a16_forward",
    "svdq_prep_calibrate", "svdq_prep_lowrank", "svdq_prep_residual_quantize",
    "svdq_w4a4_gemm_lowrank_up_qkv", "svdq_linear_forward_qkv",
    "svdq_w4a4_gemm_lowrank_up_chain", "svdq_linear_forward_chain", "svdq_device_error_site",
    "svdq_set_deterministic",
    "svdq_dense_forward", "svdq_rms_quantize8",
    "svdq_rope_load", "svdq_rope_free", "svdq_rope_apply", "svdq_rope_table", "svdq_ops_device_error_site",
    "svdq_ops_debug_set_fault", "svdq_ops_debug_dense_variant",
]


class SvdqError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {STATUS.get(code, code)}")


class WeightDesc(ctypes.Structure):
    _fields_ = [
        ("variant", ctypes.c_int),
        ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("r", ctypes.c_int64),
        ("max_M", ctypes.c_int64),
        ("flags", ctypes.c_uint32),
        ("lam", ctypes.c_void_p), ("L1", ctypes.c_void_p), ("L2", ctypes.c_void_p),
        ("w_codes", ctypes.c_void_p), ("w_scales", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("w_scale_exp", ctypes.c_int32),
        ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p), ("norm_eps", ctypes.c_float),
    ]


class AWQDesc(ctypes.Structure):
    _fields_ = [
        ("K", ctypes.c_int64), ("N", ctypes.c_int64), ("max_M", ctypes.c_int64),
        ("a", ctypes.c_void_p), ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
        ("zeros", ctypes.c_void_p), ("bias", ctypes.c_void_p),
    ]


_LIB = None


def lib(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libsvdq.so (building it first when absent or stale)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = _build.LIB
    if build_if_missing and _build.stale():
        _build.build()
    if not os.path.exists(path):
        raise OSError(f"libsvdq.so not found at {path}; run python -m "
                      "bit_diffusion_transformer_w4a4_b200.build")
    L = ctypes.CDLL(path)
    vp, i64, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    L.svdq_weights_load.argtypes = [ctypes.POINTER(WeightDesc), ctypes.POINTER(vp), vp]
    L.svdq_weights_free.argtypes = [vp]
    L.svdq_act_scales_bytes.argtypes = [vp, i64, ctypes.POINTER(ctypes.c_size_t)]
    L.svdq_quantize_act_lowrank_down.argtypes = [vp, vp, i64, vp, vp, vp, vp]
    L.svdq_w4a4_gemm_lowrank_up.argtypes = [vp, vp, vp, vp, i64, vp, vp]
    L.svdq_linear_forward.argtypes = [vp, vp, vp, i64, vp]
    L.svdq_linear_forward_host.argtypes = [vp, vp, vp, i64, vp]
    L.svdq_device_status.argtypes = [vp, vp]
    L.svdq_debug_set_fault.argtypes = [vp, ctypes.c_uint32, ctypes.c_uint32]
    L.svdq_selftest_division.argtypes = [ctypes.c_int, ctypes.c_void_p]
    L.svdq_w4a4_gemm_lowrank_up_qkv.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp]
    L.svdq_w4a4_gemm_lowrank_up_chain.argtypes = [vp, vp, vp, vp, i64, vp, vp, vp, vp, vp, vp]
    L.svdq_linear_forward_chain.argtypes = [vp, vp, vp, vp, i64, vp]
    L.svdq_device_error_site.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int)]
    L.svdq_set_deterministic.argtypes = [vp, ctypes.c_int]
    L.svdq_linear_forward_qkv.argtypes = [vp, vp, vp, vp, i64, vp]
    L.svdq_awq_load.argtypes = [ctypes.POINTER(AWQDesc), ctypes.POINTER(vp), vp]
    L.svdq_awq_free.argtypes = [vp]
    L.svdq_awq_w4a16_forward.argtypes = [vp, vp, vp, i64, vp]
    L.svdq_prep_calibrate.argtypes = [vp, i64, vp, i64, i64, ctypes.c_float, vp, vp]
    L.svdq_prep_lowrank.argtypes = [vp, vp, i64, i64, i64, vp, i64, ctypes.c_int, vp, vp, vp]
    L.svdq_prep_residual_quantize.argtypes = [st, vp, vp, vp, vp, i64, i64, i64, ctypes.c_int, vp, vp,
                                              ctypes.POINTER(ctypes.c_int32), vp]
    L.svdq_quantize_act_lowrank_down_static.argtypes = [st, i64, i64, vp, vp, vp, i64, vp, vp, vp, vp, vp]
    L.svdq_dense_forward.argtypes = [vp, vp]
    L.svdq_rms_quantize8.argtypes = [vp, vp]
    L.svdq_ops_device_error_site.argtypes = [vp, ctypes.POINTER(ctypes.c_int)]
    L.svdq_ops_debug_dense_variant.argtypes = [i64, i64, i64, st, ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    L.svdq_ops_debug_set_fault.argtypes = [ctypes.c_uint32, ctypes.c_uint32]
    L.svdq_rope_load.argtypes = [vp, ctypes.POINTER(vp)]
    L.svdq_rope_free.argtypes = [vp]
    L.svdq_rope_apply.argtypes = [vp, st, i64, i64, vp, vp, vp, st, vp]
    L.svdq_rope_table.argtypes = [vp, i64, i64, vp, vp, vp]
    L.svdq_status_string.argtypes = [st]
    L.svdq_status_string.restype = ctypes.c_char_p
    L.svdq_version.restype = ctypes.c_char_p
    for name in EXPORTED:
        f = getattr(L, name)
        if f.restype is None or f.restype is ctypes.c_int:
            f.restype = st
    _LIB = L
    return L


def _check(code: int, where: str) -> None:
    if code != 0:
        raise SvdqError(code, where)


def _ptr(a) -> int:
    """Device or host address of a torch tensor / numpy array (None -> 0)."""
    if a is None:
        return 0
    if isinstance(a, np.ndarray):
        return a.ctypes.data
    return a.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        import torch
        if not torch.cuda.is_available():
            return 0            # the library itself reports the missing device
        return torch.cuda.current_stream().cuda_stream
    return int(stream)


def selftest_division(variant: int) -> tuple[int, int]:
    """(code mismatches, normal-range quotient mismatches) -- both 0 expected."""
    n = (ctypes.c_ulonglong * 2)()
    _check(lib().svdq_selftest_division(variant, n), "svdq_selftest_division")
    return int(n[0]), int(n[1])


class SVDQWeights:
    """A loaded layer: owns a library handle (``svdq_weights_t``)."""

    def __init__(self, pw, max_M: int, stream=None, single_sm: bool = False,
                 int4_f16: bool = False, qkv_norm=None):
        """``pw`` has fields variant, K, N, r, lam, L1, L2, codes, scales, bias, gelu
        (host numpy arrays in the formats of ``svdq_weight_desc``).  ``single_sm``
        sets SVDQ_GEMM_SINGLE_SM (NVFP4 GEMM on single SMs; by default it runs on
        pairs of SMs when M > 128).  ``int4_f16`` sets SVDQ_INT4_F16 (INT4 GEMM as
        one fp16 GEMM of the exactly dequantised operands).  ``qkv_norm`` =
        (q_norm bf16 [128], k_norm bf16 [128], eps) sets SVDQ_EPI_QKV_NORM_ROPE."""
        self._keep = [np.ascontiguousarray(pw.lam, dtype=np.float32),
                      np.ascontiguousarray(pw.L1, dtype=np.uint16),
                      np.ascontiguousarray(pw.L2, dtype=np.uint16),
                      np.ascontiguousarray(pw.codes, dtype=np.uint8),
                      np.ascontiguousarray(pw.scales),
                      None if pw.bias is None else np.ascontiguousarray(pw.bias, dtype=np.uint16)]
        lam, L1, L2, codes, scales, bias = self._keep
        qn = kn = None
        eps = 0.0
        if qkv_norm is not None:
            qn = np.ascontiguousarray(qkv_norm[0], dtype=np.uint16)
            kn = np.ascontiguousarray(qkv_norm[1], dtype=np.uint16)
            eps = float(qkv_norm[2])
            self._keep += [qn, kn]
        self.qkv = qkv_norm is not None
        self.variant, self.K, self.N, self.r = int(pw.variant), int(pw.K), int(pw.N), int(pw.r)
        self.max_M = int(max_M)
        self.gelu = bool(pw.gelu)
        d = WeightDesc(self.variant, self.K, self.N, self.r, self.max_M,
                       (EPI_GELU if self.gelu else 0) | (GEMM_SINGLE_SM if single_sm else 0)
                       | (INT4_F16 if int4_f16 else 0) | (EPI_QKV_NORM_ROPE if self.qkv else 0),
                       _ptr(lam), _ptr(L1) if self.r else 0, _ptr(L2) if self.r else 0,
                       _ptr(codes), _ptr(scales), _ptr(bias), int(getattr(pw, "w_scale_exp", 0)),
                       _ptr(qn), _ptr(kn), eps)
        h = ctypes.c_void_p(0)
        self._lib = lib()
        _check(self._lib.svdq_weights_load(ctypes.byref(d), ctypes.byref(h), _stream(stream)),
               "svdq_weights_load")
        self.handle = h

    @property
    def G(self) -> int:
        return 64 if self.variant == INT4 else 16

    def act_scales_bytes(self, M: int) -> int:
        n = ctypes.c_size_t(0)
        _check(self._lib.svdq_act_scales_bytes(self.handle, M, ctypes.byref(n)), "svdq_act_scales_bytes")
        return int(n.value)

    # --------------------------------------------------------------- the calls
    def quantize_act_lowrank_down(self, x, M, act_codes, act_scales, t, stream=None):
        _check(self._lib.svdq_quantize_act_lowrank_down(
            self.handle, _ptr(x), int(M), _ptr(act_codes), _ptr(act_scales), _ptr(t),
            _stream(stream)), "svdq_quantize_act_lowrank_down")

    def w4a4_gemm_lowrank_up(self, act_codes, act_scales, t, M, y, stream=None):
        _check(self._lib.svdq_w4a4_gemm_lowrank_up(
            self.handle, _ptr(act_codes), _ptr(act_scales), _ptr(t), int(M), _ptr(y),
            _stream(stream)), "svdq_w4a4_gemm_lowrank_up")

    def w4a4_gemm_lowrank_up_qkv(self, act_codes, act_scales, t, M, rope, y, stream=None):
        _check(self._lib.svdq_w4a4_gemm_lowrank_up_qkv(
            self.handle, _ptr(act_codes), _ptr(act_scales), _ptr(t), int(M), _ptr(rope), _ptr(y),
            _stream(stream)), "svdq_w4a4_gemm_lowrank_up_qkv")

    def linear_forward_qkv(self, x, rope, y, M, stream=None):
        _check(self._lib.svdq_linear_forward_qkv(self.handle, _ptr(x), _ptr(rope), _ptr(y), int(M),
                                                 _stream(stream)), "svdq_linear_forward_qkv")

    def linear_forward(self, x, y, M, stream=None):
        _check(self._lib.svdq_linear_forward(self.handle, _ptr(x), _ptr(y), int(M), _stream(stream)),
               "svdq_linear_forward")

    def linear_forward_host(self, x_host, y_host, M, stream=None):
        _check(self._lib.svdq_linear_forward_host(self.handle, _ptr(x_host), _ptr(y_host), int(M),
                                                  _stream(stream)), "svdq_linear_forward_host")

    def device_status(self, stream=None) -> int:
        return int(self._lib.svdq_device_status(self.handle, _stream(stream)))

    def device_error_site(self, stream=None) -> int:
        """Wait-site code of the first expired bounded wait (0 if none)."""
        v = ctypes.c_int(0)
        _check(self._lib.svdq_device_error_site(self.handle, _stream(stream), ctypes.byref(v)),
               "svdq_device_error_site")
        return int(v.value)

    def set_deterministic(self, on: bool = True) -> None:
        """Sum kernel 1's split partial T tiles in a fixed order (bit-reproducible
        T and Y) instead of with fp32 reductions."""
        _check(self._lib.svdq_set_deterministic(self.handle, 1 if on else 0), "svdq_set_deterministic")

    def debug_set_fault(self, mask: int, timeout_us: int) -> None:
        _check(self._lib.svdq_debug_set_fault(self.handle, mask, timeout_us), "svdq_debug_set_fault")

    # ------------------------------------------------------- torch conveniences
    def alloc_act(self, M: int, device="cuda"):
        """Allocate (codes, scales, t) device buffers for M tokens."""
        import torch
        codes = torch.empty((M, self.K // 2), dtype=torch.uint8, device=device)
        scales = torch.empty(self.act_scales_bytes(M), dtype=torch.uint8, device=device)
        t = torch.empty((M, max(self.r, 1)), dtype=torch.float32, device=device)
        return codes, scales, t

    def close(self) -> None:
        if getattr(self, "handle", None) is not None and self.handle.value:
            self._lib.svdq_weights_free(self.handle)
            self.handle = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class AWQWeights:
    """A loaded AWQ W4A16 layer: owns a library handle (``svdq_awq_t``)."""

    def __init__(self, p, max_M: int, stream=None):
        """``p`` has fields K, N, a, codes, scales, zeros, bias (host numpy
        arrays in the formats of ``svdq_awq_desc``)."""
        self._keep = [np.ascontiguousarray(p.a, dtype=np.float32),
                      np.ascontiguousarray(p.codes, dtype=np.uint8),
                      np.ascontiguousarray(p.scales, dtype=np.uint16),
                      np.ascontiguousarray(p.zeros, dtype=np.uint8),
                      None if p.bias is None else np.ascontiguousarray(p.bias, dtype=np.uint16)]
        a, codes, scales, zeros, bias = self._keep
        self.K, self.N, self.max_M = int(p.K), int(p.N), int(max_M)
        d = AWQDesc(self.K, self.N, self.max_M, _ptr(a), _ptr(codes), _ptr(scales), _ptr(zeros),
                    _ptr(bias))
        h = ctypes.c_void_p(0)
        self._lib = lib()
        _check(self._lib.svdq_awq_load(ctypes.byref(d), ctypes.byref(h), _stream(stream)), "svdq_awq_load")
        self.handle = h

    def forward(self, x, y, M, stream=None):
        _check(self._lib.svdq_awq_w4a16_forward(self.handle, _ptr(x), _ptr(y), int(M), _stream(stream)),
               "svdq_awq_w4a16_forward")

    def close(self) -> None:
        if getattr(self, "handle", None) is not None and self.handle.value:
            self._lib.svdq_awq_free(self.handle)
            self.handle = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ------------------------------------------------------------- weight prep
def prep_calibrate(x, M, w, K, N, lam, alpha=0.5, stream=None):
    """lambda (fp32 [K], written) from calibration activations x (bf16
    [M x K]) and the weight w (bf16 [K x N]), all device tensors."""
    _check(lib().svdq_prep_calibrate(_ptr(x), int(M), _ptr(w), int(K), int(N), float(alpha), _ptr(lam),
                                     _stream(stream)), "svdq_prep_calibrate")


def prep_lowrank(w, lam, K, N, r, omega, l, power_iters, L1, L2, stream=None):
    """Rank-r bf16 factors L1 [K x r], L2 [r x N] (written) of diag(lam) w by
    a randomized SVD with the caller's Gaussian test matrix omega (fp32
    [N x l])."""
    _check(lib().svdq_prep_lowrank(_ptr(w), _ptr(lam), int(K), int(N), int(r), _ptr(omega), int(l),
                                   int(power_iters), _ptr(L1), _ptr(L2), _stream(stream)), "svdq_prep_lowrank")


def prep_residual_quantize(variant, w, lam, L1, L2, K, N, r, codes, scales, tensor_scale=False,
                           stream=None) -> int:
    """Codes [N x K/2] and scales [N x K/G] (written) of the residual
    diag(lam) w - L1 L2; returns the per-tensor scale exponent (0 without
    tensor_scale)."""
    e = ctypes.c_int32(0)
    _check(lib().svdq_prep_residual_quantize(int(variant), _ptr(w), _ptr(lam), _ptr(L1), _ptr(L2), int(K),
                                             int(N), int(r), int(bool(tensor_scale)), _ptr(codes),
                                             _ptr(scales), ctypes.byref(e), _stream(stream)),
           "svdq_prep_residual_quantize")
    return int(e.value)


def gemm_lowrank_up_chain(h1, act_codes, act_scales, t, M, y1, h2, codes2, scales2, t2, stream=None):
    """h1's kernel 2 with h2's activation side in its epilogue (see
    svdq_w4a4_gemm_lowrank_up_chain); y1 may be None."""
    _check(lib().svdq_w4a4_gemm_lowrank_up_chain(
        h1.handle, _ptr(act_codes), _ptr(act_scales), _ptr(t), int(M), _ptr(y1), h2.handle, _ptr(codes2),
        _ptr(scales2), _ptr(t2), _stream(stream)), "svdq_w4a4_gemm_lowrank_up_chain")


def linear_forward_chain(h1, h2, x, y2, M, stream=None):
    """y2 = fc2(fc1(x)) with fc2's activation side fused into fc1's GEMM."""
    _check(lib().svdq_linear_forward_chain(h1.handle, h2.handle, _ptr(x), _ptr(y2), int(M), _stream(stream)),
           "svdq_linear_forward_chain")


def untile_nvfp4_scales(buf: np.ndarray, M: int, K: int) -> np.ndarray:
    """Tensor-core tiled E4M3 activation scales -> canonical [M x K/16]."""
    buf = np.asarray(buf, dtype=np.uint8)
    m = np.arange(M)[:, None]
    b = np.arange(K // 16)[None, :]
    off = ((m // 128) * (K // 64) + b // 4) * 512 + (m % 32) * 16 + ((m // 32) % 4) * 4 + b % 4
    return buf[off]


# ------------------------------------- operators around the 4-bit layers
# These take torch tensors whose shapes and strides say what the C structs
# spell out (2-D tensors with contiguous rows, any row distance).  They run on
# the tensors' own device, on `stream` or that device's current stream.  Shapes,
# dtypes and devices are checked in _bind (csrc/bind.cpp), which raises
# TypeError or ValueError, everything else by the library (SvdqError).
BF16, FP16, FP32, E4M3, INT8 = range(5)
ACTS = {None: 0, "none": 0, "gelu": 1, "silu": 2}
_BIND = None


def _bind():
    """The marshalling module (built first when absent or stale)."""
    global _BIND
    if _BIND is None:
        import torch  # noqa: F401  (its libraries have to be loaded)
        L = lib()
        spec = importlib.util.spec_from_file_location(f"{__package__}._bind", _build.build_bind())
        module = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(module)
        module.init(*(ctypes.cast(f, ctypes.c_void_p).value
                      for f in (L.svdq_dense_forward, L.svdq_rms_quantize8, L.svdq_rope_apply)))
        _BIND = module
    return _BIND


class RopeDesc(ctypes.Structure):
    _fields_ = [
        ("head_dim", ctypes.c_int64), ("axes", ctypes.c_int), ("axis_dim", ctypes.c_int64 * 4),
        ("theta", ctypes.c_double * 4), ("interleaved", ctypes.c_int), ("shared", ctypes.c_int),
    ]


class RopePositions(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("type", ctypes.c_int), ("batch_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64), ("axis_stride", ctypes.c_int64)]


def dense_forward(a, w, y, a_scale=None, w_scale=None, bias=None, act=None, gate=None, gate_rows=0,
                  residual=None, device_error=None, stream=None):
    """y = residual + gate * act(a_scale w_scale (a @ w.T) + bias), written to
    and returned as ``y`` (svdq_dense_forward).

    a [M, K] and w [N, K] are bf16, fp16, float8_e4m3fn or int8; y [M, N],
    bias [N], gate and residual [M, N] are bf16 or fp16 (the operands' type
    where that is one of them).  a_scale [M] and w_scale [N] are fp32 and for
    8-bit operands only.  act: None, "gelu" (tanh form) or "silu".  gate is [N]
    or [ceil(M / gate_rows), N].  residual may be y."""
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act: {act!r}, expected one of {list(ACTS)}")
    code = (_BIND or _bind()).dense(a, w, y, a_scale, w_scale, bias, code, gate, gate_rows, residual, device_error, stream)
    if code:
        raise SvdqError(code, "svdq_dense_forward")
    return y


def rms_quantize8(x, codes, scales, residual=None, h=None, weight=None, weight_rows=0, eps=1e-6, norm=True,
                  stream=None):
    """h = x + residual; codes, scales = the RMS norm of h times weight in 8
    bits (svdq_rms_quantize8), or of h times weight itself with ``norm=False``.

    x, residual and h [M, K] are bf16, fp16 or fp32, codes [M, K] is
    float8_e4m3fn or int8, scales [M] fp32.  weight is [K] or
    [ceil(M / weight_rows), K].  residual, h and weight may be None; h may be x
    or residual.  Returns (codes, scales)."""
    code = (_BIND or _bind()).rms8(x, codes, scales, residual, h, weight, weight_rows, eps, norm, stream)
    if code:
        raise SvdqError(code, "svdq_rms_quantize8")
    return codes, scales


def ops_error_site(stream=None) -> int:
    """Wait-site code of the first bounded wait that expired on the current
    device since the last ask (0 if none), in rms_quantize8 or in dense_forward
    without device_error; clears it.  Synchronises the stream."""
    v = ctypes.c_int(0)
    _check(lib().svdq_ops_device_error_site(_stream(stream), ctypes.byref(v)), "svdq_ops_device_error_site")
    return int(v.value)


def ops_debug_dense_variant(M: int, N: int, K: int, in_: int, sms: int) -> tuple:
    """(pair of SMs, tokens per tile, K split) of dense_forward on this shape."""
    v = (ctypes.c_int * 3)()
    _check(lib().svdq_ops_debug_dense_variant(M, N, K, in_, sms, v), "svdq_ops_debug_dense_variant")
    return tuple(v)


def ops_debug_set_fault(mask: int, timeout_us: int) -> None:
    _check(lib().svdq_ops_debug_set_fault(mask, timeout_us), "svdq_ops_debug_set_fault")


class RopeAxes:
    """Rotary positions with several axes: owns a library handle
    (``svdq_rope_t``; host memory only, usable on every device)."""

    def __init__(self, head_dim, axis_dims, theta=10000.0, interleaved=True, shared=False):
        """``axis_dims``: rotated elements per axis (even, at most four axes,
        together at most head_dim).  ``theta``: one base, or one per axis.
        ``interleaved``: pairs (2p, 2p + 1), else (p, p + R/2).  ``shared``: the
        axes are sections of one line of frequencies."""
        dims = [int(v) for v in axis_dims]
        thetas = [float(v) for v in theta] if isinstance(theta, (list, tuple)) else [float(theta)] * max(1, len(dims))
        self.head_dim, self.axis_dims, self.axes, self.handle = int(head_dim), dims, len(dims), None
        if len(dims) > 4 or len(thetas) != max(1, len(dims)):
            raise SvdqError(2, "svdq_rope_load")
        d = RopeDesc(self.head_dim, len(dims), (ctypes.c_int64 * 4)(*dims), (ctypes.c_double * 4)(*thetas),
                     1 if interleaved else 0, 1 if shared else 0)
        h = ctypes.c_void_p(0)
        self._lib = lib()
        _check(self._lib.svdq_rope_load(ctypes.byref(d), ctypes.byref(h)), "svdq_rope_load")
        self.handle = h

    def apply(self, q, pos, k=None, q_out=None, k_out=None, inverse=False, stream=None):
        """Rotate q and k ([S, H, D] or [B, S, H, D], any strides between heads,
        tokens and sequences; bf16, fp16 or fp32) into q_out and k_out (None: in
        place); ``inverse`` turns back, which is the gradient.  pos is int32,
        int64 or fp32: [S, axes] (shared), [B * S, axes] or [B, S, axes].
        Returns q's output, or both."""
        code = (_BIND or _bind()).rope(self.handle.value, self.head_dim, self.axes, q, pos, k, q_out, k_out, inverse, stream)
        if code:
            raise SvdqError(code, "svdq_rope_apply")
        q_out = q if q_out is None else q_out
        return q_out if k is None else (q_out, k if k_out is None else k_out)

    def table(self, pos, table, stream=None):
        """(cos, sin) of every token and pair into ``table`` (contiguous fp32 of
        tokens x R elements), the ``rope`` argument of ``linear_forward_qkv``
        when R = 128.  pos is [tokens, axes]."""
        import torch
        types = {torch.int32: 0, torch.int64: 1, torch.float32: 2}
        if pos.dtype not in types:
            raise TypeError(f"pos: dtype {pos.dtype} is not supported here")
        if pos.dim() != 2 or pos.shape[1] != self.axes:
            raise ValueError(f"pos: shape {tuple(pos.shape)}, expected [tokens, {self.axes}]")
        S = pos.shape[0]
        if table.dtype != torch.float32 or not table.is_contiguous() or table.numel() != S * sum(self.axis_dims):
            raise ValueError(f"table: expected {S * sum(self.axis_dims)} contiguous fp32 elements")
        if table.device != pos.device:
            raise ValueError(f"table is on {table.device}, expected {pos.device}")
        p = RopePositions(pos.data_ptr(), types[pos.dtype], 0, *pos.stride())

        def call(s):
            return self._lib.svdq_rope_table(self.handle, 1, S, ctypes.byref(p), table.data_ptr(), s)

        if pos.is_cuda:
            with torch.cuda.device(pos.device):
                code = call(_stream(stream))
        elif torch.cuda.is_available():
            raise ValueError(f"the tensors are on {pos.device}, expected a CUDA device")
        else:
            code = call(_stream(stream))     # the library reports the missing device
        _check(code, "svdq_rope_table")
        return table

    def close(self) -> None:
        if getattr(self, "handle", None) is not None and self.handle.value:
            self._lib.svdq_rope_free(self.handle)
            self.handle = ctypes.c_void_p(0)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
