"""GPU parity of rotary positions with several axes (svdq_rope_*) against the
formula in fp64.

Tolerance per element of a rotated pair (a, b): half a step of the type times
the result, plus 2^-20 (|a| + |b|): the reduced angle in half turns is rounded
to fp32 (2^-25 absolute, times pi), sincospi is off by under 2 units (2^-22),
and the products and the sum round three times (2^-24 each)."""

import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _angles(pos, dims, theta, shared):
    """[..., pairs] in fp64 from pos [..., axes]."""
    out, p, R = [], 0, sum(dims)
    for a, d in enumerate(dims):
        for i in range(d // 2):
            th = theta[a] if isinstance(theta, (list, tuple)) and not shared else (
                theta[0] if isinstance(theta, (list, tuple)) else theta)
            out.append(pos[..., a].double() * th ** (-2.0 * (p if shared else i) / (R if shared else d)))
            p += 1
    return torch.stack(out, dim=-1)


def _reference(x, pos, dims, theta, inter, shared, inverse):
    """(out, tolerance); x [B, S, H, D], pos [B, S, axes]."""
    ang = _angles(pos, dims, theta, shared)[:, :, None, :]
    R = sum(dims)
    v = x.double()
    a, b = (v[..., 0:R:2], v[..., 1:R:2]) if inter else (v[..., :R // 2], v[..., R // 2:R])
    c, s = torch.cos(ang), torch.sin(ang) * (-1 if inverse else 1)
    o, tol = v.clone(), torch.zeros_like(v)
    for k, val in ((0, a * c - b * s), (1, a * s + b * c)):
        sl = slice(k, R, 2) if inter else slice(k * R // 2, (k + 1) * R // 2)
        o[..., sl] = val
        tol[..., sl] = val.abs() * (torch.finfo(x.dtype).eps / 2) + 2.0 ** -20 * (a.abs() + b.abs())
    return o, tol


def _pos(B, S, n, far, dtype, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + B + S)
    p = torch.floor(torch.rand(B, S, n, generator=g, device="cuda", dtype=torch.float64) * far)
    if dtype == torch.float32:
        p = p + 0.25
    return p.to(dtype)


def _check(o, x, pos, dims, theta, inter, shared, inverse):
    want, tol = _reference(x, pos, dims, theta, inter, shared, inverse)
    off = (o.double() - want).abs() - tol
    assert off.max().item() <= 0, f"{off.max().item():.3e} beyond the tolerance"


CASES = [  # D, axis dims
    (128, [16, 56, 56]), (64, [64]), (80, [32, 32]), (128, [44, 42, 42]), (2, [2]), (256, [64, 64, 64, 64]),
    (50, [10, 6, 14]), (96, [16, 32]), (254, [254]),
]


@pytest.mark.parametrize("inter", [True, False])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("D,dims", CASES)
def test_rope(D, dims, kind, inter):
    B, S, H, HK = 2, 37, 5, 2
    g = torch.Generator(device="cuda")
    g.manual_seed(D)
    q = torch.randn(B, S, H, D, generator=g, device="cuda").to(T[kind])
    k = torch.randn(B, S, HK, D, generator=g, device="cuda").to(T[kind])
    for shared, inverse, theta in ((False, False, 10000.0), (True, True, 500.0)):
        r = svdq.RopeAxes(D, dims, theta, interleaved=inter, shared=shared)
        pos = _pos(B, S, len(dims), 5000, torch.int32)
        qo, ko = torch.full_like(q, 7), torch.full_like(k, 7)
        r.apply(q, pos, k=k, q_out=qo, k_out=ko, inverse=inverse)
        _check(qo, q, pos, dims, theta, inter, shared, inverse)
        _check(ko, k, pos, dims, theta, inter, shared, inverse)
        q2, k2 = q.clone(), k.clone()
        r.apply(q2, pos, k=k2, inverse=inverse)
        assert torch.equal(q2, qo) and torch.equal(k2, ko)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64, torch.float32])
@pytest.mark.parametrize("far", [2 ** 20, 2 ** 24])
def test_rope_far_positions(dtype, far):
    """Angles of a million radians and more keep fp32 accuracy."""
    x = torch.randn(1, 500, 2, 64, device="cuda")
    pos = _pos(1, 500, 2, far, dtype) + (far // 2 if dtype != torch.float32 else 0)
    o = torch.empty_like(x)
    svdq.RopeAxes(64, [32, 32]).apply(x, pos, q_out=o)
    _check(o, x, pos, [32, 32], 10000.0, True, False, False)


def test_rope_theta_per_axis_and_shared_positions():
    x = torch.randn(3, 40, 4, 64, device="cuda").to(torch.bfloat16)
    pos = _pos(1, 40, 2, 300, torch.int64)[0]
    o = torch.empty_like(x)
    svdq.RopeAxes(64, [24, 40], theta=[100.0, 1e6], interleaved=False).apply(x, pos, q_out=o)
    _check(o, x, pos.expand(3, 40, 2), [24, 40], [100.0, 1e6], False, False, False)


@pytest.mark.parametrize("inter", [True, False])
def test_rope_layouts(inter):
    """[B, H, S, D] views, slices of a packed [B, S, (H + 2 HK) D] buffer in
    place (V untouched), unaligned heads, position planes [axes, B, S]."""
    B, S, H, HK, D, dims = 2, 19, 4, 2, 64, [16, 24, 24]
    r = svdq.RopeAxes(D, dims, interleaved=inter)
    pos = _pos(B, S, 3, 900, torch.int32)
    planes = pos.permute(2, 0, 1).contiguous().permute(1, 2, 0)
    ref = torch.randn(B, S, H, D, device="cuda").to(torch.bfloat16)
    a = ref.transpose(1, 2).contiguous()
    r.apply(a.transpose(1, 2), planes)
    _check(a.transpose(1, 2), ref, pos, dims, 10000.0, inter, False, False)
    packed = torch.randn(B, S, (H + 2 * HK) * D, device="cuda").to(torch.bfloat16)
    before = packed.clone()
    heads = packed.view(B, S, H + 2 * HK, D)
    r.apply(heads[:, :, :H], pos, k=heads[:, :, H:H + HK])
    was = before.view(B, S, H + 2 * HK, D)
    _check(heads[:, :, :H + HK], was[:, :, :H + HK], pos, dims, 10000.0, inter, False, False)
    assert torch.equal(heads[:, :, H + HK:], was[:, :, H + HK:])
    odd = torch.randn(B * S, H, D + 3, device="cuda").to(torch.bfloat16)
    was, view = odd.clone(), odd[:, :, 1:D + 1]
    r.apply(view, pos.reshape(B * S, 3))
    _check(view.reshape(B, S, H, D), was[:, :, 1:D + 1].reshape(B, S, H, D), pos, dims, 10000.0, inter, False, False)
    assert torch.equal(odd[:, :, :1], was[:, :, :1]) and torch.equal(odd[:, :, D + 1:], was[:, :, D + 1:])


@pytest.mark.parametrize("S,H", [(1, 1), (1, 64), (3, 7), (257, 3), (1030, 24)])
def test_rope_lengths(S, H):
    x = torch.randn(S, H, 128, device="cuda").to(torch.bfloat16)
    pos = _pos(1, S, 3, 4096, torch.int32)[0]
    o = torch.empty_like(x)
    svdq.RopeAxes(128, [16, 56, 56]).apply(x, pos, q_out=o)
    _check(o[None], x[None], pos[None], [16, 56, 56], 10000.0, True, False, False)


def test_rope_inverse_is_the_gradient():
    """Against autograd of the formula, and against differences."""
    S, H, D, dims = 6, 2, 16, [4, 8]
    pos = _pos(1, S, 2, 50, torch.int32)
    x = torch.randn(1, S, H, D, device="cuda", dtype=torch.float64, requires_grad=True)
    gy = torch.randn(1, S, H, D, device="cuda")
    y, _ = _reference_f64(x, pos, dims)
    (gx,) = torch.autograd.grad(y, x, gy.double())
    r = svdq.RopeAxes(D, dims)
    got = torch.empty_like(gy)
    r.apply(gy, pos, q_out=got, inverse=True)
    assert (got.double() - gx).abs().max() <= 2.0 ** -20 * 2 * gy.abs().max()
    e = torch.randn_like(gy)
    xf = x.detach().float()
    hi, lo = torch.empty_like(xf), torch.empty_like(xf)
    r.apply(xf + e, pos, q_out=hi)
    r.apply(xf - e, pos, q_out=lo)
    num = ((hi.double() - lo.double()) / 2 * gy.double()).sum()     # linear: no truncation error
    assert abs(num - (got.double() * e.double()).sum()) <= 2.0 ** -17 * (e.abs() * gy.abs()).sum()


def _reference_f64(x, pos, dims):
    ang = _angles(pos, dims, 10000.0, False)[:, :, None, :]
    R = sum(dims)
    a, b = x[..., 0:R:2], x[..., 1:R:2]
    y = torch.stack([a * torch.cos(ang) - b * torch.sin(ang), a * torch.sin(ang) + b * torch.cos(ang)], dim=-1)
    return torch.cat([y.flatten(-2), x[..., R:]], dim=-1), None


def test_rope_no_tokens_no_heads_and_capture():
    r = svdq.RopeAxes(64, [32, 32])
    x = torch.randn(8, 4, 64, device="cuda").to(torch.bfloat16)
    pos = _pos(1, 8, 2, 64, torch.int32)[0]
    r.apply(x[:0], pos[:0])
    o = torch.empty_like(x)
    r.apply(x, pos, k=x[:, :0], q_out=o)
    want = o.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        r.apply(x, pos, q_out=o)
    o.zero_()
    g.replay()
    assert torch.equal(o, want)


@pytest.mark.parametrize("dtype", [torch.int32, torch.float32])
def test_rope_table(dtype):
    dims = [16, 56, 56]
    pos = _pos(1, 1000, 3, 4096, dtype)[0]
    t = torch.empty(1000, 128, device="cuda")
    svdq.RopeAxes(128, dims).table(pos, t)
    ang = _angles(pos, dims, 10000.0, False)
    want = torch.stack([torch.cos(ang), torch.sin(ang)], dim=-1).reshape(1000, 128)
    assert (t.double() - want).abs().max() <= 2.0 ** -21
