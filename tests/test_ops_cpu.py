"""Argument checks of the operators around the 4-bit layers, which run on the
host before any device work: on a machine without a GPU a valid call ends with
SVDQ_ERR_UNSUPPORTED_DEVICE, every refusal before that."""
import ctypes

import pytest
import torch

from bit_diffusion_transformer_w4a4_b200 import svdq

class DenseDesc(ctypes.Structure):
    _fields_ = [
        ("in_", ctypes.c_int), ("out", ctypes.c_int), ("act", ctypes.c_int),
        ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("a", ctypes.c_void_p), ("lda", ctypes.c_int64),
        ("w", ctypes.c_void_p), ("ldw", ctypes.c_int64),
        ("a_scale", ctypes.c_void_p), ("w_scale", ctypes.c_void_p), ("bias", ctypes.c_void_p),
        ("gate", ctypes.c_void_p), ("ldg", ctypes.c_int64), ("gate_rows", ctypes.c_int64),
        ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
        ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64),
        ("device_error", ctypes.c_void_p),
    ]


class Rms8Desc(ctypes.Structure):
    _fields_ = [
        ("in_", ctypes.c_int), ("out", ctypes.c_int), ("M", ctypes.c_int64), ("K", ctypes.c_int64),
        ("x", ctypes.c_void_p), ("ldx", ctypes.c_int64),
        ("residual", ctypes.c_void_p), ("ldr", ctypes.c_int64),
        ("h", ctypes.c_void_p), ("ldh", ctypes.c_int64),
        ("weight", ctypes.c_void_p), ("ldw", ctypes.c_int64), ("weight_rows", ctypes.c_int64),
        ("norm", ctypes.c_int), ("eps", ctypes.c_float),
        ("codes", ctypes.c_void_p), ("ldc", ctypes.c_int64), ("scales", ctypes.c_void_p),
    ]


class RopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("stride", ctypes.c_int64 * 3), ("out_stride", ctypes.c_int64 * 3)]


OK, ARG, SHAPE, ALIGN, DEVICE = 0, 1, 2, 3, 4
NO_GPU = not torch.cuda.is_available()
pytestmark = pytest.mark.skipif(not NO_GPU, reason="valid calls on made-up addresses would run on a GPU")

A, W, Y, R, G, B, SA, SW = (0x10000000 * (i + 1) for i in range(8))   # made-up addresses, far apart


def _dense(**kw):
    f = dict(in_=svdq.BF16, out=svdq.BF16, act=0, M=100, N=200, K=64, a=A, lda=64, w=W, ldw=64, a_scale=0, w_scale=0,
             bias=0, gate=0, ldg=200, gate_rows=100, residual=0, ldr=200, y=Y, ldy=200, device_error=0)
    f.update(kw)
    return svdq.lib().svdq_dense_forward(ctypes.byref(DenseDesc(**f)), None)


@pytest.mark.parametrize("kw,code", [
    ({}, DEVICE), (dict(M=0, a=0, y=0), OK), (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(K=0), SHAPE),
    (dict(K=65537, lda=65600, ldw=65600), SHAPE), (dict(M=(1 << 24) + 1), SHAPE), (dict(M=1 << 24, N=1 << 24, ldy=1 << 24), SHAPE),
    (dict(in_=svdq.FP32), ARG), (dict(in_=9), ARG), (dict(out=svdq.FP32), ARG), (dict(out=svdq.FP16), ARG),
    (dict(act=3), ARG), (dict(a=0), ARG), (dict(w=0), ARG), (dict(y=0), ARG),
    (dict(a_scale=SA), ARG), (dict(in_=svdq.E4M3, a_scale=SA, w_scale=SW), DEVICE),
    (dict(in_=svdq.INT8, out=svdq.FP16, a_scale=SA + 2), ALIGN),
    (dict(a=A + 8), ALIGN), (dict(w=W + 2), ALIGN), (dict(lda=68), ALIGN), (dict(ldw=68), ALIGN), (dict(lda=63), SHAPE),
    (dict(ldw=56), SHAPE), (dict(ldy=199), SHAPE), (dict(M=1, lda=3, ldy=7), DEVICE), (dict(N=1, ldw=5), DEVICE),
    (dict(y=Y + 1), ALIGN), (dict(bias=B + 1), ALIGN), (dict(gate=G + 1), ALIGN), (dict(residual=R + 1), ALIGN),
    (dict(device_error=B + 2), ALIGN), (dict(bias=B, gate=G, residual=R, y=Y + 2), DEVICE),
    (dict(gate=G, gate_rows=0), SHAPE), (dict(gate=G, gate_rows=1 << 40), DEVICE), (dict(gate=G, ldg=-1), SHAPE),
    (dict(residual=R, ldr=0), DEVICE), (dict(residual=R, ldr=-1), SHAPE),
    (dict(residual=Y), DEVICE), (dict(residual=Y, ldr=208), ARG), (dict(residual=Y + 2), ARG), (dict(residual=Y, ldr=0), ARG),
    (dict(ldy=400, residual=Y + 400, ldr=400), DEVICE), (dict(ldy=400, residual=Y + 398, ldr=400), ARG),
    (dict(ldy=400, residual=Y + 402, ldr=400), ARG),
    (dict(y=A), ARG), (dict(y=W + 64), ARG), (dict(bias=Y + 10), ARG), (dict(gate=Y), ARG),
    (dict(lda=264, ldy=264, y=A + 128), DEVICE), (dict(lda=264, ldy=264, y=A + 126), ARG),
    (dict(in_=svdq.E4M3, a_scale=Y, w_scale=SW), ARG), (dict(in_=svdq.E4M3, a_scale=SA, w_scale=Y + 4), ARG),
])
def test_dense_arguments(kw, code):
    assert _dense(**kw) == code


X, RES, H, WT, C, S = (0x20000000 * (i + 1) for i in range(6))


def _rms(**kw):
    f = dict(in_=svdq.BF16, out=svdq.E4M3, M=50, K=256, x=X, ldx=256, residual=0, ldr=256, h=0, ldh=256, weight=0, ldw=256,
             weight_rows=50, norm=1, eps=1e-6, codes=C, ldc=256, scales=S)
    f.update(kw)
    return svdq.lib().svdq_rms_quantize8(ctypes.byref(Rms8Desc(**f)), None)


@pytest.mark.parametrize("kw,code", [
    ({}, DEVICE), (dict(M=0, x=0, codes=0, scales=0), OK), (dict(M=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=32769), SHAPE),
    (dict(M=1 << 31), SHAPE), (dict(in_=svdq.INT8), ARG), (dict(out=svdq.BF16), ARG), (dict(norm=2), ARG),
    (dict(eps=0.0), ARG), (dict(eps=1.0), ARG), (dict(eps=float("nan")), ARG), (dict(eps=0.0, norm=0), DEVICE),
    (dict(x=0), ARG), (dict(codes=0), ARG), (dict(scales=0), ARG), (dict(x=X + 1), ALIGN), (dict(scales=S + 2), ALIGN),
    (dict(in_=svdq.FP32, x=X + 2), ALIGN), (dict(residual=RES, h=H, weight=WT), DEVICE), (dict(residual=RES + 1), ALIGN),
    (dict(ldc=255), SHAPE), (dict(h=H, ldh=255), SHAPE), (dict(ldx=0), DEVICE), (dict(ldx=-1), SHAPE), (dict(M=1, ldc=0), DEVICE),
    (dict(weight=WT, weight_rows=0), SHAPE), (dict(weight=WT, ldw=-1), SHAPE), (dict(ldx=(1 << 28) + 1), SHAPE),
    (dict(h=X), DEVICE), (dict(residual=RES, h=RES), DEVICE), (dict(h=X, ldh=264), ARG), (dict(h=X + 2), ARG),
    (dict(h=X, ldx=0), ARG), (dict(codes=X), ARG), (dict(scales=C + 4), ARG), (dict(h=H, codes=H + 16), ARG),
    (dict(weight=WT, h=WT), ARG), (dict(scales=X), ARG),
])
def test_rms8_arguments(kw, code):
    assert _rms(**kw) == code


def _rope_desc(**kw):
    f = dict(head_dim=64, axes=2, axis_dim=(32, 32, 0, 0), theta=(1e4, 1e4, 0, 0), interleaved=1, shared=0)
    f.update(kw)
    return svdq.RopeDesc(**f)


def _rope_load(**kw):
    h = ctypes.c_void_p(0)
    code = svdq.lib().svdq_rope_load(ctypes.byref(_rope_desc(**kw)), ctypes.byref(h))
    assert bool(h.value) == (code == 0)
    assert svdq.lib().svdq_rope_free(h) == 0
    return code


@pytest.mark.parametrize("kw,code", [
    ({}, OK), (dict(head_dim=1), SHAPE), (dict(head_dim=258), SHAPE), (dict(axes=0), SHAPE), (dict(axes=5), SHAPE),
    (dict(axis_dim=(31, 32, 0, 0)), SHAPE), (dict(axis_dim=(0, 32, 0, 0)), SHAPE), (dict(axis_dim=(34, 32, 0, 0)), SHAPE),
    (dict(axis_dim=(-32, 32, 0, 0)), SHAPE), (dict(theta=(1e4, 0.5, 0, 0)), ARG), (dict(theta=(1e4, 0, 0, 0), shared=1), OK),
    (dict(theta=(float("nan"), 1e4, 0, 0)), ARG), (dict(theta=(1e31, 1e4, 0, 0)), ARG), (dict(interleaved=2), ARG), (dict(shared=-1), ARG),
])
def test_rope_load_arguments(kw, code):
    assert _rope_load(**kw) == code


def _rope_apply(B=2, S=10, q=None, k=None, pos=None, dtype=svdq.BF16, inverse=0):
    L = svdq.lib()
    h = ctypes.c_void_p(0)
    assert L.svdq_rope_load(ctypes.byref(_rope_desc()), ctypes.byref(h)) == 0
    tensor = lambda d, at: RopeTensor(**{**dict(x=at, out=at + 0x8000000, heads=3, stride=(1920, 192, 64),  # noqa: E731
                                                     out_stride=(1920, 192, 64)), **d})
    p = svdq.RopePositions(**{**dict(p=S_POS, type=0, batch_stride=20, token_stride=2, axis_stride=1), **(pos or {})})
    tq = tensor(q or {}, X)
    code = L.svdq_rope_apply(h, dtype, B, S, ctypes.byref(p), ctypes.byref(tq),
                             ctypes.byref(tensor(k, RES)) if k is not None else None, inverse, None)
    L.svdq_rope_free(h)
    return code


S_POS = 0x7000000


@pytest.mark.parametrize("kw,code", [
    ({}, DEVICE), (dict(k={}), DEVICE), (dict(S=0), OK), (dict(B=0), OK), (dict(q=dict(heads=0)), OK), (dict(B=-1), SHAPE),
    (dict(B=1 << 20, S=1 << 20), SHAPE), (dict(dtype=svdq.E4M3), ARG), (dict(inverse=2), ARG),
    (dict(q=dict(heads=-1)), SHAPE), (dict(q=dict(x=0)), ARG), (dict(q=dict(x=X + 1)), ALIGN), (dict(q=dict(out=0)), ARG),
    (dict(pos=dict(p=0)), ARG), (dict(pos=dict(type=3)), ARG), (dict(pos=dict(p=S_POS + 2)), ALIGN),
    (dict(pos=dict(type=1, p=S_POS + 4)), ALIGN), (dict(pos=dict(token_stride=-1)), SHAPE),
    (dict(q=dict(out=X)), DEVICE), (dict(q=dict(out=X, out_stride=(3840, 384, 128))), ARG), (dict(q=dict(out=X + 64)), ARG),
    (dict(q=dict(stride=(0, 0, 64))), DEVICE), (dict(q=dict(out_stride=(0, 192, 64))), SHAPE),
    (dict(q=dict(out_stride=(1920, 192, 63))), SHAPE), (dict(q=dict(out_stride=(1920, 128, 64))), SHAPE),
    (dict(q=dict(stride=(1 << 50, 192, 64))), SHAPE),
    # [B, H, S, D]
    (dict(q=dict(stride=(1920, 64, 640), out_stride=(1920, 64, 640))), DEVICE),
    # slices of one packed buffer: q and k side by side, then k one element too early
    (dict(q=dict(x=X, out=X, stride=(3840, 384, 64), out_stride=(3840, 384, 64)),
          k=dict(x=X + 384, out=X + 384, stride=(3840, 384, 64), out_stride=(3840, 384, 64))), DEVICE),
    (dict(q=dict(x=X, out=X, stride=(3840, 384, 64), out_stride=(3840, 384, 64)),
          k=dict(x=X + 382, out=X + 382, stride=(3840, 384, 64), out_stride=(3840, 384, 64))), ARG),
    (dict(k=dict(out=X)), ARG), (dict(k=dict(out=X + 0x8000000)), ARG),
])
def test_rope_apply_arguments(kw, code):
    assert _rope_apply(**kw) == code


def test_null_arguments():
    L = svdq.lib()
    h = ctypes.c_void_p(0)
    assert L.svdq_dense_forward(None, None) == ARG
    assert L.svdq_rms_quantize8(None, None) == ARG
    assert L.svdq_rope_load(None, ctypes.byref(h)) == ARG
    assert L.svdq_rope_load(ctypes.byref(_rope_desc()), None) == ARG
    assert L.svdq_rope_apply(None, 0, 1, 1, None, None, None, 0, None) == ARG
    assert L.svdq_rope_table(None, 1, 1, None, None, None) == ARG
    assert L.svdq_rope_free(None) == OK


BF = torch.bfloat16


@pytest.mark.parametrize("change,error", [
    (dict(a=torch.zeros(4, 64)), TypeError), (dict(w=torch.zeros(8, 64, dtype=torch.float16)), TypeError),
    (dict(w=torch.zeros(8, 32, dtype=BF)), ValueError), (dict(y=torch.zeros(4, 9, dtype=BF)), ValueError),
    (dict(y=torch.zeros(8, 4, dtype=BF).t()), ValueError), (dict(bias=torch.zeros(7, dtype=BF)), ValueError),
    (dict(bias=torch.zeros(8)), TypeError), (dict(act="relu"), ValueError), (dict(gate=torch.zeros(3, 8, dtype=BF), gate_rows=2), ValueError),
    (dict(gate_rows=-2, gate=torch.zeros(2, 8, dtype=BF)), ValueError), (dict(residual=torch.zeros(4, 8)), TypeError),
    (dict(a_scale=torch.zeros(4, dtype=BF)), TypeError), (dict(a=torch.zeros(4, 1, 64, dtype=BF)), ValueError),
    (dict(device_error=torch.zeros(1)), TypeError),
    ({}, svdq.SvdqError), (dict(a_scale=torch.zeros(4)), svdq.SvdqError),
])
def test_dense_python_checks(change, error):
    a = dict(a=torch.zeros(4, 64, dtype=BF), w=torch.zeros(8, 64, dtype=BF), y=torch.zeros(4, 8, dtype=BF))
    a.update(change)
    with pytest.raises(error):
        svdq.dense_forward(**a)


@pytest.mark.parametrize("change,error", [
    (dict(codes=torch.zeros(4, 64)), TypeError), (dict(codes=torch.zeros(4, 65, dtype=torch.int8)), ValueError),
    (dict(scales=torch.zeros(3)), ValueError), (dict(h=torch.zeros(4, 64)), TypeError),
    (dict(weight=torch.zeros(2, 64, dtype=BF), weight_rows=3, x=torch.zeros(7, 64, dtype=BF)), ValueError),
    (dict(weight=torch.zeros(63, dtype=BF)), ValueError), ({}, svdq.SvdqError),
])
def test_rms8_python_checks(change, error):
    a = dict(x=torch.zeros(4, 64, dtype=BF), codes=torch.zeros(4, 64, dtype=torch.int8), scales=torch.zeros(4))
    a.update(change)
    with pytest.raises(error):
        svdq.rms_quantize8(**a)


@pytest.mark.parametrize("change,error", [
    (dict(q=torch.zeros(6, 2, 62, dtype=BF)), ValueError), (dict(q=torch.zeros(6, 64, dtype=BF)), ValueError),
    (dict(pos=torch.zeros(6, 3, dtype=torch.int32)), ValueError), (dict(pos=torch.zeros(6, 2, dtype=torch.int16)), TypeError),
    (dict(k=torch.zeros(5, 2, 64, dtype=BF)), ValueError), (dict(k=torch.zeros(6, 2, 64)), TypeError),
    (dict(q_out=torch.zeros(6, 3, 64, dtype=BF)), ValueError), (dict(q_out=torch.zeros(6, 2, 64)), TypeError),
    (dict(q=torch.zeros(6, 2, 64, dtype=BF).transpose(1, 2).contiguous().transpose(1, 2)), ValueError), ({}, svdq.SvdqError),
])
def test_rope_python_checks(change, error):
    a = dict(q=torch.zeros(6, 2, 64, dtype=BF), pos=torch.zeros(6, 2, dtype=torch.int32))
    a.update(change)
    with pytest.raises(error):
        svdq.RopeAxes(64, [32, 32]).apply(**a)


def test_rope_python_load_and_table_checks():
    with pytest.raises(svdq.SvdqError):
        svdq.RopeAxes(64, [32, 34])
    with pytest.raises(svdq.SvdqError):
        svdq.RopeAxes(64, [])
    with pytest.raises(svdq.SvdqError):
        svdq.RopeAxes(64, [2] * 5)
    with pytest.raises(svdq.SvdqError):
        svdq.RopeAxes(64, [32, 32], theta=[1e4])
    r = svdq.RopeAxes(64, [32, 32])
    with pytest.raises(ValueError):
        r.table(torch.zeros(6, 2, dtype=torch.int32), torch.zeros(6, 32))
    r.close()
    r.close()



def test_not_tensors_and_bad_numbers():
    a, w, y = torch.zeros(4, 64, dtype=BF), torch.zeros(8, 64, dtype=BF), torch.zeros(4, 8, dtype=BF)
    for bad in (dict(a=1), dict(w=None), dict(bias=[1.0]), dict(stream="s"), dict(gate=torch.zeros(1, 8, dtype=BF), gate_rows=1.5)):
        with pytest.raises(TypeError):
            svdq.dense_forward(**{**dict(a=a, w=w, y=y), **bad})
    with pytest.raises(TypeError):
        svdq.rms_quantize8(a, torch.zeros(4, 64, dtype=torch.int8), None)
    with pytest.raises(TypeError):
        svdq.rms_quantize8(a, torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4), eps="x")
    r = svdq.RopeAxes(64, [32, 32])
    r.close()
    with pytest.raises(TypeError):
        r.apply(torch.zeros(6, 2, 64, dtype=BF), torch.zeros(6, 2, dtype=torch.int32))


def test_same_tensor_for_q_and_k_refused():
    q = torch.zeros(6, 2, 64, dtype=BF)
    with pytest.raises(svdq.SvdqError) as e:
        svdq.RopeAxes(64, [32, 32]).apply(q, torch.zeros(6, 2, dtype=torch.int32), k=q)
    assert e.value.code == ARG
