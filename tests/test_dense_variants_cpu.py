"""The rule that picks a dense kernel: every variant is some call's, and there
are shapes with remainders in M, N and K for each, which the GPU tests run."""
import ctypes

import pytest

from bit_diffusion_transformer_w4a4_b200 import svdq

SMS = 148
# variant (pair of SMs, tokens per tile, K split): shapes (M, N, 128-byte blocks of K) that take it on 148 SMs
SHAPES = {
    (0, 16, 1): [(1, 17, 1), (2, 9001, 6)],
    (0, 16, 2): [(78, 2285, 19)],
    (0, 16, 4): [(1, 17, 8), (7, 4001, 24)],
    (0, 16, 8): [(2, 17, 16), (5, 641, 96)],
    (0, 32, 1): [(854, 514, 1), (498, 898, 1)],
    (0, 32, 2): [(1204, 262, 18)],
    (0, 32, 4): [(564, 21, 10)],
    (0, 32, 8): [(244, 20, 16)],
    (0, 64, 1): [(1334, 644, 1)],
    (0, 64, 2): [(691, 662, 19)],
    (0, 64, 4): [(579, 131, 13)],
    (0, 64, 8): [(275, 138, 16)],
    (0, 128, 1): [(1590, 1158, 1)],
    (0, 128, 2): [(3191, 519, 10)],
    (0, 128, 4): [(967, 412, 17)],
    (0, 128, 8): [(563, 142, 43)],
    (1, 256, 1): [(2396, 1550, 1), (4100, 2600, 3)],
    (1, 256, 2): [(7913, 225, 13), (510, 3000, 41)],
    (1, 256, 4): [(1237, 684, 43), (250, 3000, 97)],
}


@pytest.mark.parametrize("variant", SHAPES)
def test_shapes_of_a_variant(variant):
    for M, N, blocks in SHAPES[variant]:
        for kind, size in ((svdq.BF16, 2), (svdq.INT8, 1)):
            K = 128 * blocks // size
            assert svdq.ops_debug_dense_variant(M, N, K, kind, SMS) == variant
            assert svdq.ops_debug_dense_variant(M, N, K - 16 // size, kind, SMS) == variant


def test_all_variants_are_there():
    """Three pair kernels and four tile sizes with four K splits each."""
    assert set(SHAPES) == {(1, 256, s) for s in (1, 2, 4)} | {(0, n, s) for n in (16, 32, 64, 128) for s in (1, 2, 4, 8)}


def test_arguments():
    v = (ctypes.c_int * 3)()
    call = svdq.lib().svdq_ops_debug_dense_variant
    assert call(1, 1, 1, svdq.BF16, SMS, v) == 0
    assert call(1, 1, 1, svdq.FP32, SMS, v) == 1 and call(1, 1, 1, svdq.BF16, 0, v) == 1 and call(1, 1, 1, svdq.BF16, SMS, None) == 1
    for shape in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1 << 25, 1, 1), (1, 1, 65537)):
        assert call(*shape, svdq.BF16, SMS, v) == 2
