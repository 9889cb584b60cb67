"""Which layouts of Q, K and their outputs svdq_rope_apply takes: buffers that
share memory without two heads meeting are taken, heads that meet are refused.
On a machine without a GPU a call that passes the checks ends with
SVDQ_ERR_UNSUPPORTED_DEVICE."""
import ctypes
import itertools
import random

import pytest
import torch

from bit_diffusion_transformer_w4a4_b200 import svdq

pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="valid calls on made-up addresses would run on a GPU")
ARG, SHAPE, DEVICE = 1, 2, 4
BF = torch.bfloat16


class RopeTensor(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("heads", ctypes.c_int64),
                ("stride", ctypes.c_int64 * 3), ("out_stride", ctypes.c_int64 * 3)]


def _apply(*args, **kw):
    with pytest.raises(svdq.SvdqError) as e:
        svdq.RopeAxes(64, [32, 32]).apply(*args, **kw)
    return e.value.code


@pytest.mark.parametrize("B", [1, 2, 3])
def test_joint_sequence_in_place(B):
    """The image part of text + image tokens, Q, K and V side by side."""
    T, S, H = 5, 9, 3
    buf = torch.zeros(B, T + S, 3, H, 64, dtype=BF)
    pos = torch.zeros(S, 2, dtype=torch.int32)
    assert _apply(buf[:, T:, 0], pos, k=buf[:, T:, 1]) == DEVICE
    assert _apply(buf[:, T:, 0], pos, k=buf[:, :S, 0]) == ARG       # tokens T .. S - 1 are in both
    assert _apply(buf[:, T:, 0], pos, k=buf[:, T:, 0]) == ARG


@pytest.mark.parametrize("B", [1, 2, 3])
def test_heads_packed_with_q_k_v(B):
    S, H = 7, 4
    buf = torch.zeros(B, S, H, 3, 64, dtype=BF)
    pos = torch.zeros(S, 2, dtype=torch.int32)
    assert _apply(buf[:, :, :, 0], pos, k=buf[:, :, :, 1]) == DEVICE
    assert _apply(buf[:, :, :, 0], pos, k=buf[:, :, :, 2], q_out=buf[:, :, :, 1]) == DEVICE
    assert _apply(buf[:, :, :, 0], pos, k=buf[:, :, :, 1], q_out=buf[:, :, :, 1]) == ARG


@pytest.mark.parametrize("B", [1, 2])
def test_grouped_and_single_k_heads(B):
    S, H = 6, 4
    pos = torch.zeros(S, 2, dtype=torch.int32)
    for HK in (1, 2):
        tokens = torch.zeros(B, S + 3, H + 2 * HK, 64, dtype=BF)[:, 3:]
        assert _apply(tokens[:, :, :H], pos, k=tokens[:, :, H:H + HK]) == DEVICE
        assert _apply(tokens[:, :, :H], pos, k=tokens[:, :, H - 1:H + HK - 1]) == ARG
        planes = torch.zeros(B, H + 2 * HK, S + 3, 64, dtype=BF)[:, :, 3:].transpose(1, 2)
        assert _apply(planes[:, :, :H], pos, k=planes[:, :, H:H + HK]) == DEVICE
        assert _apply(planes[:, :, :H], pos, k=planes[:, :, H - 1:H + HK - 1]) == ARG


def _heads(base, stride, n, D):
    """First elements of all heads."""
    return [base + sum(i * s for i, s in zip(at, stride)) for at in itertools.product(*map(range, n))]


def _meet(a, b, D):
    """Whether a head of one set shares an element with a head of the other."""
    taken = {h + i for h in a for i in range(D)}
    return any(h + i in taken for h in b for i in range(D))


def test_random_strides():
    """Against the sets of elements themselves: heads that meet are always
    refused; with equal strides nothing else is."""
    rng = random.Random(0)
    L, D = svdq.lib(), 4
    handle = ctypes.c_void_p(0)
    desc = svdq.RopeDesc(D, 1, (4, 0, 0, 0), (1e4, 0, 0, 0), 1, 0)
    assert L.svdq_rope_load(ctypes.byref(desc), ctypes.byref(handle)) == 0
    pos = svdq.RopePositions(0x7000000, 0, 0, 1, 1)
    base, seen = 0x10000000, {DEVICE: 0, ARG: 0}
    for _ in range(6000):
        B, S, H = (rng.randint(1, 3) for _ in range(3))
        # a nested box whose dimensions leave room for others inside
        order, stride, unit = rng.sample(range(3), 3), [0, 0, 0], D * rng.randint(1, 3)
        for d in order:
            stride[d] = unit
            unit = unit * (B, S, H)[d] + D * rng.randint(0, 2)
        HK = rng.randint(1, H)
        off = rng.randint(-unit, 2 * unit)
        other = list(stride)
        same = rng.random() < 0.8
        if not same:
            other[rng.randrange(3)] += rng.randint(1, 8)
        q = RopeTensor(base, base, H, (ctypes.c_int64 * 3)(*stride), (ctypes.c_int64 * 3)(*stride))
        at = base + 2 * off
        k = RopeTensor(at, at, HK, (ctypes.c_int64 * 3)(*other), (ctypes.c_int64 * 3)(*other))
        code = L.svdq_rope_apply(handle, svdq.BF16, B, S, ctypes.byref(pos), ctypes.byref(q), ctypes.byref(k), 0, None)
        if code == SHAPE:            # the changed strides made K's own heads meet
            assert not same
            continue
        meet = _meet(_heads(0, stride, (B, S, H), D), _heads(off, other, (B, S, HK), D), D)
        assert code in (ARG, DEVICE)
        if meet or same:
            assert code == (ARG if meet else DEVICE), (B, S, H, HK, stride, other, off)
        seen[code] += 1
    L.svdq_rope_free(handle)
    assert min(seen.values()) > 500
