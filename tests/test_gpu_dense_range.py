"""Products of block-scaled E4M3 matrices at the ends of their scales: a bf16 y takes
scales of 2^-126 to 2^127 whatever the values are; a float32 y takes values from
2^-126 up to below 2^128, a value beyond counting as infinite.  One product a sum,
so that y is that product rounded once."""
import math

import pytest
import torch

import sketched_parameter_sharing_amd as ss1

pytestmark = pytest.mark.gpu
F, H = torch.float32, torch.bfloat16


def single(rows, code, scale, K=384, at=300):
    """Rows of zeros but for ``code`` with the scale byte ``scale`` in one place."""
    b = ss1.Fp8Blocks.empty(rows, K)
    b.codes.view(torch.uint8).zero_()
    b.codes[:, at] = code
    b.scale.fill_(127)
    b.scale[:, at // 128] = scale
    return b


ENDS = [(1.0, 254, 1.0, 1), (1.875, 254, 1.0, 20), (-1.875, 254, 0.5, 127), (448.0, 246, 1.0, 3), (1.0, 1, 448.0, 246),
        (448.0, 1, 448.0, 127), (2.0 ** -9, 10, 1.0, 254), (1.75, 1, 1.75, 127)]
BEYOND = [(2.0, 254, 1.0, 20), (448.0, 247, 1.0, 20), (448.0, 254, 448.0, 2), (-448.0, 254, 1.0, 1)]
TINY = [(2.0 ** -9, 1, 1.0, 254), (2.0 ** -9, 1, 448.0, 246), (2.0 ** -6, 1, 448.0, 254)]


@pytest.mark.parametrize("M,N", [(3, 5), (16, 70), (40, 70), (300, 200)])
@pytest.mark.parametrize("dtype", [H, F])
def test_ends_of_the_scales(M, N, dtype):
    for ca, sa, cb, sb in ENDS + (BEYOND + TINY if dtype == H else []):
        want = torch.tensor(math.ldexp(ca * cb, sa + sb - 254), dtype=torch.float64).to(F).to(dtype).item()
        for y in (ss1.matmul_fp8_blocks(single(M, ca, sa), single(N, cb, sb), dtype=dtype),
                  ss1.matmul_fp8_blocks(single(M, cb, sb), single(N, ca, sa), dtype=dtype)):
            assert y.unique().tolist() == [want], (ca, sa, cb, sb)


@pytest.mark.parametrize("M,N", [(3, 5), (16, 70), (40, 70), (300, 200)])
def test_values_beyond_float32_count_as_infinite(M, N):
    for ca, sa, cb, sb in BEYOND:
        y = ss1.matmul_fp8_blocks(single(M, ca, sa), single(N, cb, sb), dtype=F)
        assert y.isinf().all() and ((y > 0) == (ca * cb > 0)).all(), (ca, sa, cb, sb)


def test_a_float32_layer_at_the_ends_of_float32():
    """|x| up to 1.9375 * 2^127 keeps a value that float32 holds; the largest number rounds to 2^128."""
    w = single(70, 1.0, 127, 128, 5)
    for v, want in ((1.875 * 2.0 ** 127, 1.875 * 2.0 ** 127), (-2.0 ** -126, -2.0 ** -126), (3.4028234e38, math.inf)):
        for M in (2, 40):
            x = torch.zeros((M, 128), device="cuda")
            x[:, 5] = v
            assert ss1.dense_forward_fp8(x, w)[0].unique().tolist() == [want]
