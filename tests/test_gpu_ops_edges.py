"""Calls at the edges of what the operators document, against the same call
without the edge."""
import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF = torch.bfloat16


def _row(t, distance=(1 << 40) + 3):
    """The same single row with a row distance that no buffer has."""
    return torch.as_strided(t, t.shape, (distance, 1))


def test_distance_of_a_single_row():
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    a, w, b, gate, res = r(1, 512), r(640, 512), r(640), r(1, 640), r(1, 640)
    y = [torch.empty(1, 640, dtype=BF, device="cuda") for _ in range(2)]
    svdq.dense_forward(a, w, y[0], bias=b, gate=gate, gate_rows=1, residual=res)
    svdq.dense_forward(_row(a), w, _row(y[1]), bias=b, gate=_row(gate), gate_rows=1, residual=_row(res))
    assert torch.equal(*y)
    x, res, wt = r(1, 512), r(1, 512), r(1, 512)
    out = [(torch.empty(1, 512, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda"), torch.empty(1, 512, dtype=BF, device="cuda"))
           for _ in range(2)]
    svdq.rms_quantize8(x, out[0][0], out[0][1], residual=res, h=out[0][2], weight=wt, weight_rows=1)
    svdq.rms_quantize8(_row(x), _row(out[1][0]), out[1][1], residual=_row(res), h=_row(out[1][2]), weight=_row(wt), weight_rows=1)
    assert all(torch.equal(*v) for v in zip(*out))
