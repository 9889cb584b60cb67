"""An expired wait is seen by the host also where the call takes no error word."""
import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
BF = torch.bfloat16


@pytest.fixture
def hook():
    svdq.ops_error_site()
    yield svdq.ops_debug_set_fault
    svdq.ops_debug_set_fault(0, 0)
    svdq.ops_error_site()


def test_dense_without_error_word(hook):
    a, w, y = torch.ones(40, 512, dtype=BF, device="cuda"), torch.ones(300, 512, dtype=BF, device="cuda"), torch.zeros(40, 300, dtype=BF, device="cuda")
    hook(1, 20000)
    svdq.dense_forward(a, w, y)
    hook(0, 0)
    site = svdq.ops_error_site()
    assert 0x300 < site < 0x320 and svdq.ops_error_site() == 0      # reported once
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    hook(1, 20000)
    svdq.dense_forward(a, w, y, device_error=err)                   # a word of its own instead
    hook(0, 0)
    assert svdq.ops_error_site() == 0 and err.item() != 0
    svdq.dense_forward(a, w, y)
    assert svdq.ops_error_site() == 0 and (y == 512).all()


def test_norm(hook):
    x = torch.randn(4000, 512, device="cuda").to(BF)
    codes, scales = torch.empty(4000, 512, dtype=torch.int8, device="cuda"), torch.empty(4000, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    hook(2, 20000)
    svdq.rms_quantize8(x, codes, scales, stream=s.cuda_stream)
    hook(0, 0)
    assert svdq.ops_error_site(s.cuda_stream) == 0x321
    assert torch.isnan(scales).any()
    svdq.rms_quantize8(x, codes, scales)
    assert svdq.ops_error_site() == 0 and torch.isfinite(scales).all()


def test_not_during_a_capture(hook):
    g = torch.cuda.CUDAGraph()
    x, codes, scales = torch.ones(8, 64, device="cuda"), torch.empty(8, 64, dtype=torch.int8, device="cuda"), torch.empty(8, device="cuda")
    with torch.cuda.graph(g):
        svdq.rms_quantize8(x, codes, scales)
        with pytest.raises(svdq.SvdqError):
            svdq.ops_error_site()
    g.replay()
    assert svdq.ops_error_site() == 0 and (codes == 127).all()
