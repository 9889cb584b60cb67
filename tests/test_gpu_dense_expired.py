"""Dense calls with a bounded wait that expires (the test hook makes a stage of
the first tile wait in vain): the call ends, reports the wait, writes nothing
that lacks a part of its sum, and leaves the next call alone."""
import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq
from test_gpu_dense import _problem

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.fixture
def hook():
    yield svdq.ops_debug_set_fault
    svdq.ops_debug_set_fault(0, 0)


# (M, N, 128-byte blocks of K, row padding of Y); single SMs whole and split in two to eight,
# pairs split, pairs whole with tiled and with plain stores
@pytest.mark.parametrize("kind", ["bf16", "int8"])
@pytest.mark.parametrize("M,N,blocks,ypad", [
    (1000, 1000, 1, 0), (3, 200, 2, 0), (17, 9000, 40, 1), (5, 130, 17, 0), (1000, 100, 16, 0), (1, 640, 96, 0),
    (500, 3001, 40, 1), (510, 3000, 41, 0), (250, 3000, 97, 0), (4100, 2600, 3, 0), (4100, 2600, 3, 1)])
def test_expired_wait(hook, M, N, blocks, ypad, kind):
    K = blocks * (64 if kind == "bf16" else 128)
    p, _ = _problem(M, N, K, kind, "bf16", "gelu", True, M, True, ypad=ypad)
    mark = 12352.0                                   # no result comes near it
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    svdq.dense_forward(device_error=err, **p)
    good = p["y"].clone()
    assert err.item() == 0 and good.abs().max() < mark
    p["y"].fill_(mark)
    hook(1, 20000)
    svdq.dense_forward(device_error=err, **p)
    hook(0, 0)
    torch.cuda.synchronize()
    assert 0x300 < err.item() < 0x320
    lost = p["y"] == mark
    assert lost[0, 0]
    assert torch.equal(p["y"][~lost], good[~lost])
    if (M, N) != (4100, 2600):                       # the persistent pair loses its later tiles too
        assert not lost[256:].any() and not lost[:, 256:].any()
    assert (~lost).any()
    err.zero_()
    svdq.dense_forward(device_error=err, **p)
    assert torch.equal(p["y"], good) and err.item() == 0
