"""Sizes at which a launch's grid reaches its limit of 2^32 threads: quantisation
of 2^23 tiles and more, a product of few rows with 2^28 and more; and gradients of
millions of tokens."""
import pytest
import torch

import sketched_parameter_sharing_amd as ss1

pytestmark = pytest.mark.gpu
H = torch.bfloat16


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("along", ["q", "qt"])
def test_quantising_more_tiles_than_one_launch_takes(along):
    """A row, or a column, of 2^23 tiles and a bit: every part's codes are those of that part alone, to the last one."""
    n = (1 << 30) + 300
    x = torch.empty(n, dtype=H, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(7)
    for i in range(0, n, 1 << 26):
        part = x[i:i + (1 << 26)]
        part.copy_(torch.randn(part.numel(), generator=g, device="cuda") * 2.0 ** (i >> 26))

    def quantized(v):
        if along == "q":
            return ss1.quantize_fp8_blocks(v[None])[0]
        return ss1.quantize_fp8_blocks(v[:, None], q=None, qt=True)[1]

    b = quantized(x)
    width = -(-n // 128) * 128
    assert b.codes.shape == (1, width) and b.scale.shape == (1, -(-n // 512) * 4)
    codes, scale = b.codes.view(torch.uint8).view(-1), b.scale.view(-1)
    for i in range(0, n, 1 << 26):
        end = min(n, i + (1 << 26))
        part = quantized(x[i:end])
        wide = part.codes.shape[1]
        assert same(codes[i:i + wide], part.codes.view(-1)), i
        assert same(scale[i // 128:i // 128 + part.scale.shape[1]], part.scale.view(-1)), i


def test_few_rows_against_more_than_one_launch_takes():
    """Sums that float32 holds exactly: codes of multiples of 2^-9 below 1/2, times 0, 1 or 2."""
    M, N, K = 2, (1 << 28) + 77, 128
    b = ss1.Fp8Blocks.empty(N, K, 128)
    b.codes.view(torch.uint8).random_(0, 0x30, generator=torch.Generator(device="cuda").manual_seed(5))
    b.scale.fill_(127)
    a = ss1.Fp8Blocks.empty(M, K)
    v = torch.randint(0, 3, (M, K), device="cuda", generator=torch.Generator(device="cuda").manual_seed(6)).float()
    a.codes.copy_(v.to(torch.float8_e4m3fn))
    a.scale.fill_(127)
    y = ss1.matmul_fp8_blocks(a, b, dtype=torch.float32)
    h = ss1.matmul_fp8_blocks(a, b)
    for i in range(0, N, 1 << 22):
        want = v @ b.codes[i:i + (1 << 22)].float().t()
        assert torch.equal(y[:, i:i + (1 << 22)], want), i
        assert torch.equal(h[:, i:i + (1 << 22)], want.to(H)), i


@pytest.mark.parametrize("M,V", [(20_000_003, 3000), (3_000_001, 300_000)], ids=["dealt", "not dealt"])
@pytest.mark.parametrize("kind", ["some", "same"])
def test_gradients_of_millions_of_tokens(M, V, kind):
    """Whole numbers: every partial sum is one that float32 holds."""
    g = torch.Generator(device="cuda").manual_seed(9)
    dy = torch.randint(-1, 2, (M, 4), generator=g, device="cuda").to(H)
    ids = torch.randint(-1, V, (M,), generator=g, device="cuda", dtype=torch.int32)
    if kind == "same":
        ids[ids % 8 > 0] = 7
    dE = ss1.embedding_backward(dy, ids, V, dtype=torch.float32)
    real = (ids >= 0).cpu()
    want = torch.zeros((V, 4), dtype=torch.float64)
    want.index_add_(0, ids.cpu()[real].long(), dy.double().cpu()[real])
    assert torch.equal(dE.double().cpu(), want)
    more = ss1.embedding_backward(dy, ids, V, dE=dE.clone(), accumulate=True)
    assert torch.equal(more, dE * 2)
