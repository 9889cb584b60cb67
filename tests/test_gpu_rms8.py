"""GPU parity of svdq_rms_quantize8 (residual's addition, RMS norm, 8-bit codes
with one scale per row).

Codes: computed in fp32 from t = h w and the row's maximum alone, each step
one IEEE rounding, so they equal the same steps on the CPU bit for bit; and
they lie within half a step (plus the fp32 steps' 2^-21 relative) of the fp64
quotient.  Scales: the sum of K squares (at most 32 terms a thread, then 10
levels), the square root and two divisions: under 50 roundings of 2^-24, so
2^-18 relative covers them."""
import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
Q = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}
TOP = {"e4m3": 448.0, "int8": 127.0}


def _inputs(M, K, kind, residual, weight, pad=0, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + M * 31 + K)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x = (r(M, K + pad) * (1 + 20 * (r(K + pad) > 2))).to(T[kind])[:, :K]
    return (x, (3 * r(M, K + pad)).to(T[kind])[:, :K] if residual else None, (1 + 0.3 * r(K)).to(T[kind]) if weight else None)


def _run(x, res, w, out, norm=True, pad=0, weight_rows=0, eps=1e-6):
    M, K = x.shape
    codes = torch.full((M + 1, K + pad), 3.0, device="cuda").to(Q[out])
    scales = torch.full((M + 1,), -1.0, device="cuda")
    h = torch.full((M + 1, K + pad), 9.0, device="cuda", dtype=x.dtype) if res is not None else None
    svdq.rms_quantize8(x, codes[:M, :K], scales[:M], residual=res, h=None if h is None else h[:M, :K], weight=w,
                       weight_rows=weight_rows, norm=norm, eps=eps)
    torch.cuda.synchronize()
    assert (codes[M].float() == 3).all() and (codes[:, K:].float() == 3).all() and scales[M] == -1
    if h is not None:
        assert (h[M] == 9).all() and (h[:, K:] == 9).all()
    return codes[:M, :K].cpu(), scales[:M].cpu(), None if h is None else h[:M, :K].cpu()


def _expected_h(x, res):
    x = x.cpu()
    return x if res is None else (x.float() + res.cpu().float()).to(x.dtype)


def _check(x, res, w, out, got, norm=True, eps=1e-6):
    codes, scales, h = got
    want_h = _expected_h(x, res)
    if h is not None:
        assert torch.equal(h, want_h)
    wt = torch.ones(1, x.shape[1]) if w is None else w.cpu().reshape(-1, x.shape[1]).float()
    t = want_h.float() * wt
    top = t.abs().amax(dim=1)
    live = top >= 2.0 ** -118
    inv = torch.where(live, torch.full_like(top, TOP[out]) / top, torch.zeros_like(top))
    q = t * inv[:, None]
    q = q.round().to(torch.int8) if out == "int8" else q.to(torch.float8_e4m3fn)
    assert torch.equal(codes.float(), q.float())
    # in fp64
    hd = want_h.double()
    v = hd * wt.double()
    if norm:
        v = v / torch.sqrt((hd * hd).mean(dim=1, keepdim=True) + eps)
    s = v.abs().amax(dim=1) / TOP[out]
    s = torch.where(live, s, torch.zeros_like(s))
    assert ((scales.double() - s).abs() <= 2.0 ** -18 * s).all()
    z = v / torch.where(s > 0, s, torch.ones_like(s))[:, None]
    z = torch.where(live[:, None], z, torch.zeros_like(z))
    step = torch.full_like(z, 0.5) if out == "int8" else torch.clamp(z.abs() * 2.0 ** -4, min=2.0 ** -10)
    assert ((codes.double() - z).abs() <= step + 2.0 ** -20 * z.abs()).all()


@pytest.mark.parametrize("out", ["e4m3", "int8"])
@pytest.mark.parametrize("kind", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M,K", [(1, 1), (1, 4096), (3, 8), (5, 31), (7, 256), (300, 1000), (517, 2047), (9, 8192),
                                 (400, 4096), (2, 32768), (2, 32767), (400, 12288), (700, 520)])
def test_rms8(M, K, kind, out):
    x, res, w = _inputs(M, K, kind, True, True)
    _check(x, res, w, out, _run(x, res, w, out))


@pytest.mark.parametrize("out", ["e4m3", "int8"])
@pytest.mark.parametrize("residual,weight,norm", [(0, 0, 0), (0, 0, 1), (1, 0, 1), (0, 1, 1), (1, 1, 0)])
@pytest.mark.parametrize("M,K,pad", [(10, 512, 0), (10, 512, 3), (310, 768, 8), (310, 333, 1)])
def test_rms8_terms_and_row_distances(M, K, pad, residual, weight, norm, out):
    x, res, w = _inputs(M, K, "bf16", residual, weight, pad)
    _check(x, res, w, out, _run(x, res, w, out, bool(norm), pad), bool(norm))


def test_rms8_weight_rows():
    x, res, _ = _inputs(10, 256, "bf16", True, False)
    w = (1 + 0.2 * torch.randn(4, 256, device="cuda")).to(torch.bfloat16)
    got = _run(x, res, w, "e4m3", weight_rows=3)
    _check(x, res, w.repeat_interleave(3, 0)[:10], "e4m3", got)


@pytest.mark.parametrize("which", ["x", "residual"])
@pytest.mark.parametrize("K", [512, 333])
def test_rms8_stream_in_place(which, K):
    x, res, w = _inputs(50, K, "bf16", True, True)
    want = _run(x, res, w, "e4m3")
    codes = torch.empty(50, K, dtype=torch.float8_e4m3fn, device="cuda")
    scales = torch.empty(50, device="cuda")
    h = x if which == "x" else res
    svdq.rms_quantize8(x, codes, scales, residual=res, h=h, weight=w)
    assert torch.equal(h.cpu(), want[2]) and torch.equal(codes.cpu().float(), want[0].float())
    assert torch.equal(scales.cpu(), want[1])


@pytest.mark.parametrize("out", ["e4m3", "int8"])
@pytest.mark.parametrize("K", [64, 65])
def test_rms8_extreme_rows(K, out):
    """Zero rows, subnormal rows, rows whose squares overflow fp32, rows with
    a NaN or an infinity between ordinary ones."""
    x, _, _ = _inputs(8, K, "bf16", False, False)
    x[1] = 0
    x[2] = x[2] * 1e-39
    x[3] = x[3] * 1e-36                     # squares underflow: eps decides
    x[4] = x[4] / x[4].abs().max() * 3e38   # squares overflow
    x[5, 3] = float("nan")
    x[6, K - 1] = float("-inf")
    codes, scales, _ = _run(x, None, None, out)
    assert torch.isnan(scales[5]) and torch.isnan(scales[6])
    ok = [0, 1, 2, 3, 4, 7]
    assert torch.isfinite(scales[ok]).all() and scales[1] == 0 and (codes[1].float() == 0).all()
    assert scales[2] == 0 and (codes[2].float() == 0).all()
    _check(x[ok], None, None, out, (codes[ok], scales[ok], None))


def test_rms8_overflowing_sum_in_place():
    """The second look at a row's squares reads the row from registers, not
    from an input that the call has already overwritten."""
    x = torch.full((2, 300), 2e38, device="cuda").to(torch.bfloat16)
    r = torch.full((2, 300), 1e38, device="cuda").to(torch.bfloat16)
    want = _run(x, r, None, "int8")
    codes = torch.empty(2, 300, dtype=torch.int8, device="cuda")
    scales = torch.empty(2, device="cuda")
    svdq.rms_quantize8(x, codes, scales, residual=r, h=x)
    assert (codes == 127).all() and torch.equal(scales.cpu(), want[1])
    assert torch.allclose(scales.cpu().double(), torch.full((2,), 1 / 127.0, dtype=torch.float64), rtol=2.0 ** -18)


def test_rms8_no_rows_and_capture():
    x, res, w = _inputs(30, 640, "fp16", True, True)
    want = _run(x, res, w, "int8")
    codes = torch.empty(30, 640, dtype=torch.int8, device="cuda")
    scales = torch.empty(30, device="cuda")
    svdq.rms_quantize8(x[:0], codes[:0], scales[:0])
    h = torch.empty_like(x)
    svdq.rms_quantize8(x, codes, scales, residual=res, h=h, weight=w)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svdq.rms_quantize8(x, codes, scales, residual=res, h=h, weight=w)
    codes.zero_(), scales.zero_()
    g.replay()
    assert torch.equal(codes.cpu(), want[0]) and torch.equal(scales.cpu(), want[1])
