"""Calls that the operators' documentation allows or refuses at its edges, by
the checks that run before any device work: on a machine without a GPU a valid
call ends with SVDQ_ERR_UNSUPPORTED_DEVICE."""
import pytest
import torch

from bit_diffusion_transformer_w4a4_b200 import svdq
from test_ops_cpu import ARG, DEVICE, OK, SHAPE, A, B, BF, C, G, H, R, S, SA, SW, WT, X, Y, W, RES, _dense, _rms

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls on made-up addresses would run on a GPU")
FAR = 1 << 40                    # beyond every limit of a row distance


@pytest.mark.parametrize("kw,code", [
    (dict(M=1, lda=FAR), DEVICE), (dict(M=1, ldy=FAR), DEVICE), (dict(N=1, ldw=FAR, ldy=1), DEVICE),
    (dict(M=1, residual=R, ldr=FAR), DEVICE), (dict(gate=G, ldg=FAR), DEVICE), (dict(gate=G, ldg=FAR, gate_rows=50), SHAPE),
    (dict(lda=FAR), SHAPE), (dict(M=1, ldy=FAR, residual=Y, ldr=3), DEVICE),
])
def test_dense_distance_of_a_single_row(kw, code):
    assert _dense(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(M=1, ldx=FAR), DEVICE), (dict(M=1, residual=RES, ldr=FAR), DEVICE), (dict(M=1, h=H, ldh=FAR), DEVICE),
    (dict(M=1, ldc=FAR), DEVICE), (dict(weight=WT, ldw=FAR), DEVICE), (dict(weight=WT, ldw=FAR, weight_rows=49), SHAPE),
    (dict(ldx=FAR), SHAPE), (dict(M=1, h=X, ldh=FAR, ldx=5), DEVICE),
])
def test_norm_distance_of_a_single_row(kw, code):
    assert _rms(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(device_error=Y), ARG), (dict(device_error=Y + 2 * 200 * 99 + 396), ARG), (dict(device_error=A + 16), ARG),
    (dict(device_error=W), ARG), (dict(device_error=B, bias=B), ARG), (dict(device_error=G + 4, gate=G), ARG),
    (dict(device_error=R, residual=R), ARG), (dict(device_error=SA, in_=svdq.E4M3, a_scale=SA, w_scale=SW), ARG),
    (dict(device_error=SW + 4, in_=svdq.E4M3, a_scale=SA, w_scale=SW), ARG),
    (dict(device_error=Y + 2 * 200 * 100), DEVICE), (dict(device_error=Y + 400, ldy=202), DEVICE),
])
def test_dense_error_word_is_an_output(kw, code):
    assert _dense(**kw) == code


def _positions(at, B=2, S=10, **pos):
    """svdq_rope_apply of X in place with its positions at `at`."""
    from test_ops_cpu import _rope_apply
    return _rope_apply(B=B, S=S, q=dict(out=X), pos={**dict(p=at), **pos})


@pytest.mark.parametrize("at,pos,code", [
    (X, {}, ARG), (X + 2 * 3840 - 4, {}, ARG), (X + 2 * 3840, {}, DEVICE), (X - 40 * 4, {}, DEVICE), (X - 40 * 4 + 4, {}, ARG),
    (X - 40 * 8 + 8, dict(type=1), ARG), (X - 40 * 8, dict(type=1), DEVICE), (X - 8, dict(batch_stride=0, token_stride=0), DEVICE),
    (X - 4, dict(batch_stride=0, token_stride=0), ARG), (0x7000000, dict(token_stride=1 << 60), SHAPE),
])
def test_positions_are_not_in_an_output(at, pos, code):
    assert _positions(at, **pos) == code


def test_table_is_not_in_the_positions():
    import ctypes
    L = svdq.lib()
    h = ctypes.c_void_p(0)
    desc = svdq.RopeDesc(64, 2, (32, 32, 0, 0), (1e4, 1e4, 0, 0), 1, 0)
    assert L.svdq_rope_load(ctypes.byref(desc), ctypes.byref(h)) == 0
    p = svdq.RopePositions(X, 0, 0, 2, 1)
    for at, code in ((X, ARG), (X + 72, ARG), (X + 80, DEVICE), (X - 8 * 32 * 10, DEVICE), (X - 8 * 32 * 10 + 8, ARG)):
        assert L.svdq_rope_table(h, 1, 10, ctypes.byref(p), at, None) == code, hex(at)
    L.svdq_rope_free(h)


MOST = (1 << 63) - 1


@pytest.mark.parametrize("rows", [100, MOST - 50, MOST])
def test_rows_each_at_its_largest(rows):
    """ceil(M / rows) must not overflow: the one row's overlap is still seen."""
    assert _dense(gate=G, gate_rows=rows) == DEVICE
    assert _dense(gate=Y, gate_rows=rows) == ARG
    assert _rms(weight=WT, weight_rows=rows) == DEVICE
    assert _rms(weight=C, weight_rows=rows) == ARG


def test_rows_each_at_its_largest_in_python():
    a, w, y = torch.zeros(4, 64, dtype=BF), torch.zeros(8, 64, dtype=BF), torch.zeros(4, 8, dtype=BF)
    for rows in (4, MOST - 1, MOST):
        with pytest.raises(svdq.SvdqError):
            svdq.dense_forward(a, w, y, gate=torch.zeros(1, 8, dtype=BF), gate_rows=rows)
        with pytest.raises(ValueError):
            svdq.dense_forward(a, w, y, gate=torch.zeros(2, 8, dtype=BF), gate_rows=rows)


class NoTruth:
    def __bool__(self):
        raise KeyError("no truth value")


def test_flag_without_a_truth_value():
    """The object's own exception, not a SystemError."""
    x, codes, scales = torch.zeros(4, 64, dtype=BF), torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    with pytest.raises(KeyError):
        svdq.rms_quantize8(x, codes, scales, norm=NoTruth())
    with pytest.raises(KeyError):
        svdq.RopeAxes(64, [32, 32]).apply(torch.zeros(6, 2, 64, dtype=BF), torch.zeros(6, 2, dtype=torch.int32), inverse=NoTruth())


@pytest.mark.parametrize("rows", [0, 1, 50])
def test_no_tokens_with_the_gates_and_weights_of_some_images(rows):
    """A call for no rows does nothing, whatever rows its gate or weight has."""
    w, y = torch.zeros(8, 64, dtype=BF), torch.zeros(0, 8, dtype=BF)
    for n in (0, 1, 2):
        assert svdq.dense_forward(torch.zeros(0, 64, dtype=BF), w, y, gate=torch.zeros(n, 8, dtype=BF), gate_rows=rows) is y
        svdq.rms_quantize8(torch.zeros(0, 64, dtype=BF), torch.zeros(0, 64, dtype=torch.int8), torch.zeros(0),
                           weight=torch.zeros(n, 64, dtype=BF), weight_rows=rows)
    with pytest.raises(ValueError):
        svdq.dense_forward(torch.zeros(0, 64, dtype=BF), w, y, gate=torch.zeros(2, 9, dtype=BF), gate_rows=rows)
