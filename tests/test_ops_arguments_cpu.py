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
