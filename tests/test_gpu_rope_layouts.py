"""Rotary positions in place on parts of larger buffers, several sequences at
once, in every type and pairing.

Tolerance: as derived in test_gpu_rope_axes, plus half a subnormal step of the
type.  That file's half step, eps / 2 times the result, holds for normal
results only: below 2^-14 fp16 values are 2^-24 apart whatever their size, so
rounding alone is off by up to 2^-25 (bf16: below 2^-126, 2^-134; fp32:
2^-150)."""
import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq
from test_gpu_rope_axes import T, _pos, _reference

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


SUB = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25, "fp32": 2.0 ** -150}   # half a subnormal step


def _check(o, x, pos, dims, theta, inter, shared, inverse):
    want, tol = _reference(x, pos, dims, theta, inter, shared, inverse)
    kind = next(k for k, t in T.items() if t == x.dtype)
    off = (o.double() - want).abs() - tol - SUB[kind]
    assert off.max().item() <= 0, f"{off.max().item():.3e} beyond the tolerance"


def _randn(*shape, kind):
    g = torch.Generator(device="cuda")
    g.manual_seed(sum(shape))
    return torch.randn(*shape, generator=g, device="cuda").to(T[kind])


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("B,D,dims", [(2, 64, [16, 24, 24]), (3, 80, [32, 32]), (2, 50, [10, 6, 14])])
def test_parts_of_a_buffer_in_place(B, D, dims, kind, inter):
    T0, S, H = 5, 23, 3
    r = svdq.RopeAxes(D, dims, interleaved=inter)
    pos = _pos(B, S, len(dims), 700, torch.int32)
    # the image part of a joint sequence: Q and K of B x (T0 + S) x 3 x H heads
    buf = _randn(B, T0 + S, 3, H, D, kind=kind)
    was = buf.clone()
    r.apply(buf[:, T0:, 0], pos, k=buf[:, T0:, 1])
    for i in (0, 1):
        _check(buf[:, T0:, i], was[:, T0:, i], pos, dims, 10000.0, inter, False, False)
    assert torch.equal(buf[:, :T0], was[:, :T0]) and torch.equal(buf[:, :, 2], was[:, :, 2])
    # Q, K and V packed head by head, the rotated Q in V's place
    buf = _randn(B, S, H, 3, D, kind=kind)
    was = buf.clone()
    r.apply(buf[:, :, :, 0], pos, k=buf[:, :, :, 1], q_out=buf[:, :, :, 2], inverse=True)
    _check(buf[:, :, :, 2], was[:, :, :, 0], pos, dims, 10000.0, inter, False, True)
    _check(buf[:, :, :, 1], was[:, :, :, 1], pos, dims, 10000.0, inter, False, True)
    assert torch.equal(buf[:, :, :, 0], was[:, :, :, 0])
    # one K head behind the Q heads, [B, heads, tokens, D]
    buf = _randn(B, H + 2, T0 + S, D, kind=kind)
    was = buf.clone()
    heads, old = buf[:, :, T0:].transpose(1, 2), was[:, :, T0:].transpose(1, 2)
    r.apply(heads[:, :, :H], pos, k=heads[:, :, H:H + 1])
    _check(heads[:, :, :H + 1], old[:, :, :H + 1], pos, dims, 10000.0, inter, False, False)
    assert torch.equal(buf[:, :, :T0], was[:, :, :T0]) and torch.equal(buf[:, H + 1], was[:, H + 1])
    # unaligned heads
    buf = _randn(B, S, H, D + 3, kind=kind)
    was = buf.clone()
    r.apply(buf[..., 1:D + 1], pos)
    _check(buf[..., 1:D + 1], was[..., 1:D + 1], pos, dims, 10000.0, inter, False, False)
    assert torch.equal(buf[..., :1], was[..., :1]) and torch.equal(buf[..., D + 1:], was[..., D + 1:])
