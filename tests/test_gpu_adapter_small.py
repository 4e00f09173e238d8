"""Adapters of small batches on the GPU, at the sizes where the library changes
from one launch for both products to two: tokens, ranks, bytes of a factor and
their total.  Definitions and tolerances as for the other batches."""
import copy

import pytest
import torch

import sketched_parameter_sharing_amd as ss1
from test_gpu_adapter import BF, F, Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ss1.load()


def singles(n, adapters, none_every=0):
    return [(1, -1 if none_every and i % none_every == 0 else i % adapters) for i in range(n)]


EDGES = [
    # (segments, ranks, K, N): tokens 256 | 257, in one segment, several, or one each
    ([(256, 0)], [16], 256, 512), ([(257, 0)], [16], 256, 512),
    ([(100, 0), (56, 1), (100, 2)], [8, 16, 32], 128, 1032), ([(100, 0), (57, 1), (100, 2)], [8, 16, 32], 128, 1032),
    (singles(256, 5, 7), [16, 8, 1, 12, 4], 256, 264), (singles(257, 5, 7), [16, 8, 1, 12, 4], 256, 264),
    # largest rank 16 | 17, 32 | 33
    (singles(9, 2), [16, 3], 512, 520), (singles(9, 2), [17, 3], 512, 520),
    ([(9, 0), (8, 1), (1, 0)], [32, 31], 512, 520), ([(9, 0), (8, 1), (1, 0)], [33, 31], 512, 520),
    # A of 64 KB (float32) and 128 KB (bf16) and a little more, in either direction
    (singles(4, 4), [16] * 4, 1024, 1024), (singles(4, 4), [16] * 4, 1032, 1032),
    (singles(4, 4), [16] * 4, 4096, 1024), (singles(4, 4), [16] * 4, 1024, 4096),
    (singles(4, 4), [16] * 4, 4104, 1032),
    # many pieces: the total of the reads under and over its bound
    (singles(40, 40), [16] * 40, 2048, 2048), (singles(256, 64), [32] * 64, 1024, 4096),
    # eight tokens and nine of one adapter
    ([(8, 0)], [16], 1024, 256), ([(9, 0)], [16], 1024, 256),
]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("edge", range(len(EDGES)))
def test_edges(edge, dtype):
    segs, ranks, K, N = EDGES[edge]
    check(Case(segs, ranks, K, N, dtype, seed=300 + edge))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_one_and_two_launches_agree_within_the_tolerance(dtype):
    # the same tokens alone (one launch) and with others behind them (two)
    c = Case([(3, 0), (200, 1), (90, 0)], [16, 24], 264, 520, dtype, seed=41)
    y, _ = c.forward(base=c.base)
    _, _, ty, _ = c.forward64()
    seg = torch.tensor([0, 3, 203], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    few, _ = ss1.adapter_forward(c.x[:203].contiguous(), c.set, seg, ids, base=c.base[:203].contiguous())
    assert ((few.double() - y[:203].double()).abs() <= 2 * ty[:203]).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_in_place_and_each_gradient_alone(dtype):
    c = Case([(5, 0), (4, -1), (30, 1)], [7, 30], 136, 1544, dtype, seed=42)
    y, v = c.forward(base=c.base, save_v=True)
    own = c.base.clone()
    assert torch.equal(c.forward(base=own, y=own)[0], y)
    dx, dA, dB = c.backward(v, dx_base=c.dxb)
    own = c.dxb.clone()
    assert torch.equal(c.backward(v, dx_base=own, dx=own)[0], dx)
    assert torch.equal(c.backward(v, dx_base=c.dxb, dA=None)[0], dx)
    assert torch.equal(c.backward(v, dx_base=c.dxb, dA=None)[2], dB)
    assert torch.equal(c.backward(v, dx_base=c.dxb, dB=None)[1], dA)


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_infinities_and_nan_stay_with_their_request(dtype):
    segs = [(3, 0), (1, 1), (4, 0), (1, 2)]
    c = Case(segs, [16, 9, 4], 128, 264, dtype, seed=43)
    y0, v = c.forward(base=c.base, save_v=True)
    dx0, _, _ = c.backward(v, dx_base=c.dxb)
    c.x[3, 5] = float("nan")
    c.dy[3, 7] = float("inf")
    c.A[16:25] = float("inf")
    c.B[16:25] = float("nan")
    y, _ = c.forward(base=c.base)
    dx, dA, dB = c.backward(v, dx_base=c.dxb)
    keep = torch.arange(9, device="cuda") != 3
    assert torch.equal(y[keep], y0[keep]) and torch.equal(dx[keep], dx0[keep])
    rows = torch.ones(29, dtype=torch.bool, device="cuda")
    rows[16:25] = False
    assert torch.isfinite(dA[rows]).all() and torch.isfinite(dB[rows]).all()


def test_a_used_set_is_copied_and_changed():
    c = Case([(3, 0), (2, 1)], [8, 4], 64, 72, F, seed=44)
    y, _ = c.forward(base=c.base)
    twin = copy.deepcopy(c.set)
    assert torch.equal(ss1.adapter_forward(c.x, twin, c.seg, c.ids, base=c.base)[0], y)
    again = copy.copy(c.set)
    assert torch.equal(ss1.adapter_forward(c.x, again, c.seg, c.ids, base=c.base)[0], y)
    # other factors, by the attribute and by the tensor's memory
    twin.B = torch.zeros_like(twin.B)
    assert torch.equal(ss1.adapter_forward(c.x, twin, c.seg, c.ids, base=c.base)[0], c.base)
    c.set.B.data = torch.zeros_like(c.set.B)
    assert torch.equal(c.forward(base=c.base)[0], c.base)
