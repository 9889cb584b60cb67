"""Bounded waits of the norm that expire: the test hook leaves a row's copies out
and shortens the limit; the kernel ends, the rows that it gave up are marked,
and all others are right."""
import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF = torch.bfloat16


@pytest.fixture
def hook():
    yield svdq.ops_debug_set_fault
    svdq.ops_debug_set_fault(0, 0)


@pytest.mark.parametrize("kind,K,residual,weight", [(BF, 3072, True, True), (BF, 64, False, False),
                                                    (torch.float32, 1024, False, True), (torch.float16, 12288, True, False)])
def test_norm_row_given_up_as_one(hook, kind, K, residual, weight):
    """The row whose copies never arrive and the later rows of its CTA (a fixed
    distance apart) get the scale NaN; all others are as they are without it."""
    M = 6001 if K > 64 else 20001           # more than two rows a CTA
    g = torch.Generator(device="cuda")
    g.manual_seed(K)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(kind)  # noqa: E731
    x, res, w = r(M, K), r(M, K) if residual else None, r(K) if weight else None
    h = torch.empty_like(x) if residual else None
    out = [(torch.empty(M, K, dtype=torch.int8, device="cuda"), torch.full((M,), -1.0, device="cuda")) for _ in range(3)]
    svdq.rms_quantize8(x, *out[0], residual=res, h=h, weight=w)
    hook(2, 20000)
    svdq.rms_quantize8(x, *out[1], residual=res, weight=w)
    hook(0, 0)
    svdq.rms_quantize8(x, *out[2], residual=res, weight=w)
    torch.cuda.synchronize()
    lost = torch.isnan(out[1][1]).nonzero().flatten().tolist()
    assert lost[0] == M // 3 and len(lost) >= 2
    step = lost[1] - lost[0]
    assert lost == list(range(M // 3, M, step))
    kept = torch.ones(M, dtype=torch.bool, device="cuda")
    kept[lost] = False
    for i in (0, 1):
        assert torch.equal(out[0][i][kept], out[1][i][kept]) and torch.equal(out[0][i], out[2][i])
