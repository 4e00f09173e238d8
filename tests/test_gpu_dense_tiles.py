"""Products of block-scaled E4M3 matrices in every tile, type of y and number of
splits, with reductions that fill, start and end its ring of LDS buffers in every
way, at sizes that leave a part of a tile on both sides.  Definitions and
tolerances are those of the dense layer's tests."""
import pytest
import torch

import sketched_parameter_sharing_amd as ss1
from test_gpu_dense_fp8 import F, H, blocks, close, value, whole_numbers

pytestmark = pytest.mark.gpu

# ((rows, columns of a tile), splits): type of y -> (M, N, blocks of 128 of the reduction)
# (no product of one or two blocks deep with up to 300 x 300 tiles goes in the others)
TILES = {
    ((64, 64), 1): {H: [(61, 61, s) for s in range(1, 10)] + [(700, 900, 6)],
                    F: [(61, 61, s) for s in range(1, 10)] + [(700, 900, 6)]},
    ((64, 64), 2): {H: [(500, 700, 35), (500, 700, 36), (500, 641, 37), (500, 641, 38)],
                    F: [(333, 641, 21), (333, 641, 22), (500, 641, 23), (641, 641, 28)]},
    ((64, 64), 4): {H: [(61, 61, s) for s in range(16, 21)], F: [(61, 61, s) for s in range(16, 21)]},
    ((64, 64), 8): {H: [(61, 61, s) for s in range(32, 38)], F: [(61, 61, s) for s in range(32, 38)]},
    ((64, 128), 1): {H: [(129, 12001, s) for s in range(1, 8)], F: [(129, 12001, s) for s in range(3, 10)]},
    ((128, 128), 1): {H: [(641, 6007, s) for s in range(2, 6)],
                      F: [(641, 9001, s) for s in range(1, 5)] + [(641, 6007, 11)]},
    ((192, 256), 1): {H: [(641, 12001, s) for s in range(3, 7)],
                      F: [(2049, 5000, 1), (2049, 5000, 2)] + [(641, 12001, s) for s in range(3, 7)]},
    ((256, 256), 1): {H: [(9001, 1283, 3), (9001, 1283, 4), (8100, 1283, 7), (8100, 1283, 8)]},
}
PRODUCTS = [(tile, splits, dtype, size) for (tile, splits), types in TILES.items() for dtype, sizes in types.items()
            for size in sizes]


def name(p):
    (bm, bn), splits, dtype, (M, N, stages) = p
    return f"{bm}x{bn}x{splits}-{'bf16' if dtype == H else 'f32'}-{M}-{N}-{stages}"


@pytest.mark.parametrize("product", PRODUCTS, ids=name)
def test_products_of_every_tile(product):
    _, _, dtype, (M, N, stages) = product
    K = stages * 128 - 37
    a, b = blocks(M, K, seed=stages), blocks(N, K, True, seed=stages + 40)
    home = torch.full((M * N + 64,), 7.0, device="cuda", dtype=dtype)
    y = home[16:16 + M * N].view(M, N)
    ss1.matmul_fp8_blocks(a, b, y=y)
    close(y, value(a), value(b))
    assert (home[:16] == 7).all() and (home[16 + M * N:] == 7).all()
    assert torch.equal(ss1.matmul_fp8_blocks(a, b, dtype=dtype), y)
    # every row, column, scale and block of the reduction in its place
    for of_a, of_b in ((1, 128), (128, 1), (1, 1), (128, 128)):
        a, b = whole_numbers(M, K, of_a, 7 + stages), whole_numbers(N, K, of_b, 8 + stages)
        y = ss1.matmul_fp8_blocks(a, b, dtype=dtype)
        assert torch.equal(y.double(), (value(a) @ value(b).t()).to(dtype).double()), (of_a, of_b)
