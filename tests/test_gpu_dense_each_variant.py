"""Every variant of the dense linear by name: each shape is checked to take the
variant that it stands for, then compared with the formula in fp64 (tolerances
as derived in test_gpu_dense), with every form of the stores and with terms
that change inside a tile; and the longest call that the library's workloads
make, 16896 tokens."""
import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq
from test_dense_variants_cpu import SHAPES
from test_gpu_dense import _check, _problem

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
CASES = [(v, *s) for v, shapes in SHAPES.items() for s in shapes]


def _sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("kind,out", [("bf16", "bf16"), ("fp16", "fp16"), ("e4m3", "fp16"), ("int8", "bf16")])
@pytest.mark.parametrize("variant,M,N,blocks", CASES)
def test_variant(variant, M, N, blocks, kind, out):
    es = 2 if kind in ("bf16", "fp16") else 1
    K = 128 * blocks // es - 16 // es
    if _sms() == 148:
        code = {"bf16": svdq.BF16, "fp16": svdq.FP16, "e4m3": svdq.E4M3, "int8": svdq.INT8}[kind]
        assert svdq.ops_debug_dense_variant(M, N, K, code, 148) == variant
    for ypad in (0, 1, 2, 7):
        p, buf = _problem(M, N, K, kind, out, "silu" if ypad % 2 else "gelu", True, max(1, M // 3), True, ypad=ypad)
        svdq.dense_forward(**p)
        _check(p, buf, K, kind, out)


@pytest.mark.parametrize("kind,K,N,act,residual", [("bf16", 3072, 3072, None, True), ("int8", 12288, 3072, None, True),
                                                   ("e4m3", 3072, 12288, "gelu", False)])
def test_longest_call(kind, K, N, act, residual):
    """2048-px images."""
    M = 16896
    p, buf = _problem(M, N, K, kind, "bf16", act, True, M // 2, residual)
    svdq.dense_forward(**p)
    _check(p, buf, K, kind, "bf16")
