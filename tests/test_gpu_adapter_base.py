"""Adapters beside a base that is large against their share: the result carries one
rounding at base's size, not one for every product.

Tolerances as for the other batches: the sum's own error goes by the sizes of its
products, base enters with one addition (2 units of 2^-24 of it)."""
import pytest

import sketched_parameter_sharing_amd as ss1
from test_gpu_adapter import BF, F, Case

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ss1.load()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("size", [1.0, 1000.0])
@pytest.mark.parametrize("segs,ranks,K,N", [
    ([(1, 0), (9, 1), (3, 0)], [16, 31], 64, 264),            # one launch
    ([(7, i % 2) for i in range(50)], [128, 47], 8, 520),     # short segments
    ([(300, 0), (130, 1)], [128, 64], 1288, 8),               # long ones
    ([(184, 0), (182, 1)], [127, 16], 16, 1224),
])
def test_one_rounding_at_the_size_of_base(segs, ranks, K, N, size, dtype):
    c = Case(segs, ranks, K, N, dtype, seed=K + N)
    c.base, c.dxb = size * c.base, size * c.dxb
    y, v = c.forward(base=c.base, save_v=True)
    ry, _, ty, _ = c.forward64()
    assert ((y.double() - ry).abs() <= ty).all()
    dx, _, _ = c.backward(v, dx_base=c.dxb)
    (rx, _, _), (tx, _, _) = c.backward64(v)
    assert ((dx.double() - rx).abs() <= tx).all()
