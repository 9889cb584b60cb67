"""GPU parity of svdq_rms_quantize8 on many rows: every CTA of the persistent
form takes several rows, so that its ring is refilled and its weight row
changes on the way; rows whose squares overflow, rows with a NaN or an infinity
and zero rows stand among ordinary ones at early and late places; the residual
stream in place; packed rows of odd length with a weight row per image.

Codes, scales and tolerances as in test_gpu_rms8 (codes bit for bit by the
documented fp32 steps, scales within 2^-18 of fp64), on the GPU."""
import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
Q = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}


def _check(h, w, out, codes, scales, norm, lost):
    """h [M, K] as stored, w [M, K] or None (a row for every row of h)."""
    t = h.float() * w.float() if w is not None else h.float()
    top = t.abs().amax(dim=1)
    fine = torch.ones(len(h), dtype=torch.bool, device="cuda")
    fine[lost] = False
    assert torch.isnan(scales[~fine]).all()
    live = fine & (top >= 2.0 ** -118)
    inv = torch.where(live, torch.full_like(top, TOP[out]) / top, torch.zeros_like(top))
    q = t * inv[:, None]
    q = q.round().to(torch.int8) if out == "int8" else q.to(torch.float8_e4m3fn)
    assert torch.equal(codes[fine].float(), q[fine].float())
    s = top.double()
    if norm:
        s = s / torch.sqrt(torch.cat([v.double().square().mean(dim=1) for v in h.split(4096)]) + 1e-6)
    s = torch.where(live, s / TOP[out], torch.zeros_like(s))
    assert ((scales.double() - s).abs() <= 2.0 ** -18 * s)[fine].all()


# rows, length, rows of a weight row (0: one weight): three rows a CTA and more
MANY = [(4000, 3072, 0), (4000, 3072, 1000), (5001, 12288, 777), (20000, 256, 333), (16000, 8, 7), (20000, 64, 0),
        (3000, 4096, 1), (1500, 8192, 400)]


@pytest.mark.parametrize("out", ["e4m3", "int8"])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K,each", MANY)
def test_many_rows(M, K, each, kind, out):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(T[kind])  # noqa: E731
    x, res = r(M, K), r(M, K)
    rows = -(-M // each) if each else 1
    w = (1 + 0.3 * torch.randn(rows, K, generator=g, device="cuda")).to(T[kind])
    lost = [11, M // 2, M - 3]                       # NaN, infinity, NaN
    x[lost[0], K // 2] = float("nan")
    x[lost[1], K - 1] = float("-inf")
    x[lost[2], 0] = float("nan")
    for m in (5, M // 2 + 1, M - 1):
        x[m], res[m] = 0, 0
    if kind != "fp16":                               # sums of squares that overflow fp32
        for m in (7, M // 2 + 2, M - 2, M - 4):
            x[m] = (x[m].float() * 1e30).to(T[kind])
    h = (x.float() + res.float()).to(T[kind])
    each = each or M
    wide = w.repeat_interleave(each, 0)[:M]
    got_h, codes, scales = torch.empty_like(x), torch.empty(M, K, dtype=Q[out], device="cuda"), torch.full((M,), -1.0, device="cuda")
    svdq.rms_quantize8(x, codes, scales, residual=res, h=got_h, weight=w, weight_rows=each)
    same = (got_h == h) | (torch.isnan(got_h) & torch.isnan(h))
    assert same.all()
    _check(h, wide, out, codes, scales, True, lost)
    first = codes.view(torch.uint8).clone(), scales.clone()
    for i in range(2):                               # the stream in place of x, and of the residual
        place = (x, res)[i].clone()
        svdq.rms_quantize8(place if i == 0 else x, codes, scales, residual=place if i else res, h=place, weight=w, weight_rows=each)
        assert torch.equal(place.view(torch.uint8), got_h.view(torch.uint8))
        assert torch.equal(codes.view(torch.uint8), first[0])
        assert torch.equal(scales.view(torch.int32), first[1].view(torch.int32))
    svdq.rms_quantize8(h, codes, scales)             # neither residual nor weight
    _check(h, None, out, codes, scales, True, lost)
    svdq.rms_quantize8(h, codes, scales, norm=False, weight=w, weight_rows=each)
    _check(h, wide, out, codes, scales, False, lost)


@pytest.mark.parametrize("out", ["e4m3", "int8"])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K,each", [(3001, 257, 100), (700, 1001, 7), (517, 2047, 259), (40, 4099, 20), (900, 901, 300), (11, 9001, 1)])
def test_odd_rows_with_a_weight_row_per_image(M, K, each, kind, out):
    g = torch.Generator(device="cuda")
    g.manual_seed(M + K)
    x, res = (torch.randn(M, K, generator=g, device="cuda").to(T[kind]) for _ in range(2))
    rows, V = -(-M // each), 4 if kind == "fp32" else 8
    buf = (1 + 0.3 * torch.randn(rows, -(-K // V) * V, generator=g, device="cuda")).to(T[kind])
    x[M - 2, K - 1] = float("nan")
    h = (x.float() + res.float()).to(T[kind])
    wide = buf[:, :K].repeat_interleave(each, 0)[:M]
    codes, scales = torch.empty(M, K, dtype=Q[out], device="cuda"), torch.empty(M, device="cuda")
    for w in (buf[:, :K], buf[:, :K].contiguous()):  # aligned weight rows, and packed ones
        svdq.rms_quantize8(x, codes, scales, residual=res, weight=w, weight_rows=each)
        _check(h, wide, out, codes, scales, True, [M - 2])
