"""GPU parity of the dense linear with a fused epilogue (svdq_dense_forward)
against the formula in fp64: every operand and output type, token counts from
one to several tiles, odd widths, K tails, row distances, unaligned outputs,
every epilogue term, in-place residuals and captured graphs.

Tolerance per element, from the arithmetic: half a step of the output type
times |y| (and of its subnormals), plus what the fp32 steps can add:
  - the sum: each of the ceil(K / 16) tensor-core additions is off by at most
    2 units in the last place of the partial sums, 2^-22 sum|a w| (int8: exact)
  - activation slopes are at most 1.2, and the fp32 epilogue rounds a few
    times, each 2^-24 of its terms (2^-20 of them covers the approximate
    exponential and reciprocal, 2^-22 relative each)
"""
import math

import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

T = {"bf16": torch.bfloat16, "fp16": torch.float16, "e4m3": torch.float8_e4m3fn, "int8": torch.int8}
SUB = {"bf16": 2.0 ** -134, "fp16": 2.0 ** -25}     # half a subnormal step


def _operand(g, rows, cols, kind, pad):
    """[rows, cols] inside a wider buffer whose spare columns hold NaN (or 77)."""
    es = 1 if kind in ("e4m3", "int8") else 2
    step = 16 // es
    ld = -(-cols // step) * step + pad * step
    x = torch.randn(rows, cols, generator=g, device="cuda")
    buf = torch.full((rows, ld), 77.0 if kind == "int8" else float("nan"), device="cuda")
    scale = None
    if es == 1:
        scale = x.abs().amax(dim=1) / (127.0 if kind == "int8" else 448.0)
        x = x / scale[:, None]
        if kind == "int8":
            x = x.round()
    buf[:, :cols] = x
    return buf.to(T[kind])[:, :cols], scale


def _problem(M, N, K, kind, out, act, bias, gate_rows, residual, seed=0, pad=0, ypad=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed + 7 * M + 11 * N + 13 * K)
    a, sa = _operand(g, M, K, kind, pad)
    w, sw = _operand(g, N, K, kind, pad)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(T[out])  # noqa: E731
    y = torch.full((M + 2, N + ypad), 5.0, device="cuda", dtype=T[out])
    return dict(a=a, w=w, y=y[1:M + 1, :N], a_scale=sa, w_scale=sw, bias=r(N) if bias else None, act=act,
                gate=r(-(-M // gate_rows), N) if gate_rows else None, gate_rows=gate_rows,
                residual=r(M, N + ypad)[:, :N] if residual else None), y


def _reference(p, K, kind, out):
    """(y, tolerance) in fp64."""
    d = lambda t: t.double()  # noqa: E731
    a, w = d(p["a"]), d(p["w"])
    acc, mag = a @ w.t(), a.abs() @ w.abs().t()
    err = mag * 0 if kind == "int8" else mag * (math.ceil(K / 16) * 2.0 ** -22)
    if p["a_scale"] is not None:
        s = d(p["a_scale"])[:, None] * d(p["w_scale"])[None, :]
        acc, err = acc * s, err * s
    if p["bias"] is not None:
        acc = acc + d(p["bias"])
    small = acc.abs() * 2.0 ** -20
    if p["bias"] is not None:
        small = small + d(p["bias"]).abs() * 2.0 ** -20 * 2
    v = acc
    if p["act"] == "gelu":
        v = 0.5 * acc * (1 + torch.tanh(math.sqrt(2 / math.pi) * (acc + 0.044715 * acc ** 3)))
    elif p["act"] == "silu":
        v = acc * torch.sigmoid(acc)
    err = 1.2 * err + 1.2 * small
    if p["gate"] is not None:
        gt = d(p["gate"]).repeat_interleave(p["gate_rows"], 0)[:v.shape[0]]
        v, err = v * gt, err * gt.abs()
    if p["residual"] is not None:
        v = v + d(p["residual"])
        err = err + d(p["residual"]).abs() * 2.0 ** -23
    return v, v.abs() * (torch.finfo(T[out]).eps / 2) + err * 1.01 + SUB[out]


def _check(p, buf, K, kind, out, ref=None):
    v, tol = ref if ref is not None else _reference(p, K, kind, out)
    y = p["y"]
    off = (y.double() - v).abs() - tol
    assert torch.isfinite(y).all()
    assert off.max().item() <= 0, f"{off.max().item():.3e} beyond the tolerance at {off.argmax().item()}"
    # rows around and columns beyond the output are as they were
    assert (buf[0] == 5).all() and (buf[-1] == 5).all() and (buf[:, y.shape[1]:] == 5).all()


KINDS = [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "bf16"), ("e4m3", "fp16"), ("int8", "bf16"), ("int8", "fp16")]


@pytest.mark.parametrize("kind,out", KINDS)
@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (1, 1, 16), (2, 130, 1000), (16, 257, 64), (17, 96, 528),
                                   (33, 1501, 1000), (100, 640, 2048), (129, 255, 400)])
def test_dense_small(M, N, K, kind, out):
    p, buf = _problem(M, N, K, kind, out, "none", True, 0, False, ypad=1)
    svdq.dense_forward(**p)
    _check(p, buf, K, kind, out)


@pytest.mark.parametrize("kind,out", KINDS)
@pytest.mark.parametrize("M,N,K,act,gate_rows,residual", [
    (300, 1111, 600, "gelu", 150, True), (513, 2048, 512, "silu", 513, False), (1000, 3000, 272, "none", 7, True),
    (2100, 1030, 336, "gelu", 0, True), (4100, 2600, 144, "none", 1025, False)])
def test_dense_large(M, N, K, kind, out, act, gate_rows, residual):
    p, buf = _problem(M, N, K, kind, out, act, True, gate_rows, residual, pad=1, ypad=3)
    svdq.dense_forward(**p)
    _check(p, buf, K, kind, out)


# (M, N, 128-byte blocks of K): one or more shapes for each tile size and K split
VARIANTS = [
    (3, 200, 2), (1, 9000, 24), (9, 300, 9), (5, 130, 17), (1000, 1000, 1), (17, 9000, 40), (1000, 100, 16), (257, 200, 16),
    (4100, 130, 1), (33, 9000, 40), (2100, 120, 16), (700, 104, 16), (500, 4096, 1), (200, 9000, 16), (4100, 120, 24),
    (1000, 120, 96), (1000, 4096, 1), (4100, 2600, 3), (300, 18000, 5), (500, 3001, 40), (510, 3000, 41), (130, 3001, 96),
    (250, 3000, 97),
]


@pytest.mark.parametrize("ypad", [0, 1, 2, 7])
@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("e4m3", "fp16"), ("int8", "bf16")])
@pytest.mark.parametrize("M,N,blocks", VARIANTS)
def test_dense_variants(M, N, blocks, kind, out, ypad):
    """Every tile size and K split, with every form of the stores: Y's rows on
    16-byte, 4-byte and 2-byte boundaries; all epilogue terms; a gate whose
    rows change inside a tile."""
    K = blocks * (64 if kind == "bf16" else 128) - (8 if kind == "bf16" else 48)
    p, buf = _problem(M, N, K, kind, out, "gelu" if ypad % 2 else None, True, -(-M // 3) if M > 2 else 1, True, ypad=ypad)
    svdq.dense_forward(**p)
    _check(p, buf, K, kind, out)


@pytest.mark.parametrize("M,N,blocks,ypad", [(4100, 2600, 3, 0), (510, 3000, 41, 0), (250, 3000, 97, 1), (300, 18001, 5, 7), (2000, 3000, 20, 0)])
def test_dense_variants_in_place_twice(M, N, blocks, ypad):
    """y = residual on the large variants, and equal bits from equal calls."""
    K = 64 * blocks
    p, buf = _problem(M, N, K, "bf16", "bf16", "silu", True, 100, True, ypad=ypad)
    ref = _reference(p, K, "bf16", "bf16")
    svdq.dense_forward(**p)
    first = p["y"].clone()
    p["y"].copy_(p["residual"])
    p["residual"] = p["y"]
    svdq.dense_forward(**p)
    _check(p, buf, K, "bf16", "bf16", ref)
    assert torch.equal(first, p["y"])


@pytest.mark.parametrize("K", [1, 7, 63, 64, 65, 127, 128, 129, 1023])
@pytest.mark.parametrize("kind", ["bf16", "int8"])
def test_dense_k_tails(K, kind):
    """K is free; what lies between K and the row distance (NaN here) is not read."""
    p, buf = _problem(40, 200, K, kind, "bf16", None, False, 0, False, pad=1)
    svdq.dense_forward(**p)
    _check(p, buf, K, kind, "bf16")


@pytest.mark.parametrize("M", [1, 5, 40, 700])
@pytest.mark.parametrize("act", [None, "gelu", "silu"])
@pytest.mark.parametrize("terms", range(8))
def test_dense_epilogue_terms(M, act, terms):
    p, buf = _problem(M, 333, 256, "e4m3", "bf16", act, terms & 1, 3 if terms & 2 else 0, terms & 4, ypad=2)
    svdq.dense_forward(**p)
    _check(p, buf, 256, "e4m3", "bf16")


@pytest.mark.parametrize("M,N,K", [(3, 300, 2048), (33, 1000, 4096), (700, 3000, 512)])
def test_dense_residual_in_place(M, N, K):
    """y = residual, also where several CTAs share a tile's K range."""
    p, buf = _problem(M, N, K, "bf16", "bf16", None, True, M, True, ypad=1)
    p["y"].copy_(p["residual"])
    ref = _reference(p, K, "bf16", "bf16")
    p["residual"] = p["y"]
    svdq.dense_forward(**p)
    _check(p, buf, K, "bf16", "bf16", ref)


def test_dense_broadcast_residual_and_gate_per_token():
    p, buf = _problem(90, 500, 128, "fp16", "fp16", "silu", False, 1, True)
    p["residual"] = p["residual"][:1].expand(90, 500)
    svdq.dense_forward(**p)
    _check(p, buf, 128, "fp16", "fp16")


def test_dense_scales_one_sided():
    p, buf = _problem(20, 140, 256, "int8", "fp16", None, False, 0, False)
    ones = torch.ones(20, device="cuda")
    p["a_scale"] = None
    q = dict(p, a_scale=ones)
    svdq.dense_forward(**p)
    got = p["y"].clone()
    svdq.dense_forward(**q)
    assert torch.equal(got, q["y"])
    _check(q, buf, 256, "int8", "fp16")


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int8"])
@pytest.mark.parametrize("M,N,K", [(1, 640, 4096), (50, 640, 4096), (600, 2560, 512)])
def test_dense_same_bits_twice_and_captured(kind, M, N, K):
    p, buf = _problem(M, N, K, kind, "bf16", "gelu", True, M, True)
    svdq.dense_forward(**p)
    first = p["y"].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        svdq.dense_forward(**p)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(first, p["y"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        svdq.dense_forward(**p)
        svdq.dense_forward(**p)
    p["y"].zero_()
    g.replay()
    g.replay()
    assert torch.equal(first, p["y"])


def test_dense_nan_and_inf_stay_in_their_rows():
    p, buf = _problem(40, 300, 512, "bf16", "bf16", None, True, 0, False)
    p["a"][3, 5] = float("nan")
    p["a"][9, 7] = float("inf")
    svdq.dense_forward(**p)
    y = p["y"]
    rows = [m for m in range(40) if m not in (3, 9)]
    assert torch.isnan(y[3]).all() and not torch.isfinite(y[9]).any()
    v, tol = _reference(dict(p, a=p["a"][rows]), 512, "bf16", "bf16")
    assert ((y[rows].double() - v).abs() <= tol).all()


def test_dense_no_error_recorded():
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    p, buf = _problem(300, 900, 512, "bf16", "bf16", None, False, 0, False)
    svdq.dense_forward(device_error=err, **p)
    assert err.item() == 0


def test_dense_no_tokens():
    p, buf = _problem(3, 64, 64, "bf16", "bf16", None, False, 0, False)
    svdq.dense_forward(p["a"][:0], p["w"], p["y"][:0])
    assert (p["y"] == 5).all()


def test_dense_int8_largest_sums():
    """-128 * -128 over the longest K: the int32 sum is exact."""
    K = 65536
    a = torch.full((2, K), -128, dtype=torch.int8, device="cuda")
    w = torch.full((130, K), -128, dtype=torch.int8, device="cuda")
    y = torch.empty(2, 130, dtype=torch.bfloat16, device="cuda")
    svdq.dense_forward(a, w, y)
    assert (y.double() == 2.0 ** 30).all()


def test_dense_cpu_tensors_refused():
    a = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        svdq.dense_forward(a, a, torch.zeros(2, 2, dtype=torch.bfloat16))
