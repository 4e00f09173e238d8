"""A dense layer's results are the bits of the calls that define them (quantisation,
then the product of the codes), whichever of its results are asked for together:
on both sides of every rule by which the gradients share a launch."""
import pytest
import torch

import sketched_parameter_sharing_amd as ss1

pytestmark = pytest.mark.gpu
F, H = torch.float32, torch.bfloat16

# [M][K] and [M][N]: up to 16 tokens against reductions of one run and of several for each of the four waves,
# few rows on either side or on both, more tokens, and layers too large for one launch
SIZES = [(1, 768, 768), (1, 300, 520), (2, 500, 2048), (3, 1000, 1283), (4, 130, 2049), (7, 256, 1920), (8, 64, 8192),
         (15, 1000, 1000), (16, 768, 2048), (16, 64, 16384), (16, 12, 600), (9, 600, 12), (16, 1024, 1088), (16, 1500, 1500),
         (17, 768, 2048), (40, 500, 1500), (333, 500, 768), (700, 1000, 1003)]


def matrix(rows, cols, dtype, seed, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device="cuda") * std
    return torch.where(torch.rand((1, cols), generator=g, device="cuda") < 0.01, x * 20, x).to(dtype)


@pytest.mark.parametrize("M,K,N", SIZES)
@pytest.mark.parametrize("dtype", [H, F])
@pytest.mark.parametrize("dW_dtype", [H, F])
def test_gradients_together_and_alone(M, K, N, dtype, dW_dtype):
    x, dy = matrix(M, K, dtype, 3), matrix(M, N, dtype, 5, 0.01)
    w, wt = ss1.quantize_fp8_blocks(matrix(N, K, F, 6, 0.02), tile=True, qt=True)
    xq, xt = ss1.quantize_fp8_blocks(x, qt=True)
    dq, dqt = ss1.quantize_fp8_blocks(dy, qt=True)
    assert torch.equal(ss1.dense_forward_fp8(x, w)[0], ss1.matmul_fp8_blocks(xq, w, dtype=dtype))
    dx, dW = ss1.dense_backward_fp8(dy, xt, wt, dW_dtype=dW_dtype)
    assert torch.equal(dx, ss1.dense_backward_fp8(dy, None, wt, dW=None)[0])
    assert torch.equal(dW, ss1.dense_backward_fp8(dy, xt, None, dx=None, dW_dtype=dW_dtype)[1])
    assert torch.equal(dx, ss1.matmul_fp8_blocks(dq, wt, dtype=dtype))
    assert torch.equal(dW, ss1.matmul_fp8_blocks(dqt, xt, dtype=dW_dtype))
