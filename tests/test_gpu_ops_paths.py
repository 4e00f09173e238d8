"""Forms of the operators' calls that the tests by size do not reach: a gradient of A
without one of x over several slices, results in place of base for long segments and
long rows, and workspaces of the caller's with exactly the queried bytes."""
import ctypes

import pytest

import sketched_parameter_sharing_amd as ss1
from sketched_parameter_sharing_amd import _lib, _ops

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_adapter import BF, F, Case  # noqa: E402
from test_gpu_layernorm import make as make_norm  # noqa: E402

BOTH = pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ss1.load()


# (segments, ranks, K, N): N of several slices of 1024 bytes and more
LONG_N = [([(100, 0), (60, 1)], [16, 40], 72, 2056), ([(1, i % 3) for i in range(20)], [64, 3, 33], 136, 4096),
          ([(40, 0), (0, 1), (25, -1), (9, 1)], [50, 7], 64, 1544), ([(700, 0), (300, 1)], [24, 64], 264, 5120)]


@BOTH
@pytest.mark.parametrize("case", range(len(LONG_N)))
def test_the_gradient_of_a_alone(case, dtype):
    segs, ranks, K, N = LONG_N[case]
    c = Case(segs, ranks, K, N, dtype, seed=70 + case)
    _, v = c.forward(save_v=True)
    (_, want, _), (_, tol, _) = c.backward64(v)
    dx, dA, dB = c.backward(None, dx=None, dB=None)
    assert dx is None and dB is None
    assert ((dA.double() - want).abs() <= tol).all()
    # the slices are joined in the same order as beside dx
    assert torch.equal(dA, c.backward(v, dx_base=c.dxb)[1])
    both = c.backward(v, dx=None)
    assert torch.equal(both[1], dA) and torch.equal(both[2], c.backward(v, dx_base=c.dxb)[2])


@BOTH
@pytest.mark.parametrize("segs,ranks,K,N", [([(300, 0), (130, 1)], [16, 64], 1288, 2056), ([(70, 1), (65, -1)], [8, 100], 4096, 520),
                                            ([(1000, 0), (3, 1), (64, 0)], [32, 16], 520, 5120)])
def test_in_place_of_base_in_long_segments(segs, ranks, K, N, dtype):
    c = Case(segs, ranks, K, N, dtype, seed=K)
    y, v = c.forward(base=c.base, save_v=True)
    own = c.base.clone()
    got, gv = c.forward(base=own, y=own, save_v=True)
    assert got is own and torch.equal(own, y) and torch.equal(gv, v)
    dx, dA, dB = c.backward(v, dx_base=c.dxb)
    own = c.dxb.clone()
    got = c.backward(v, dx_base=own, dx=own)
    assert got[0] is own and torch.equal(own, dx) and torch.equal(got[1], dA) and torch.equal(got[2], dB)


@BOTH
@pytest.mark.parametrize("M,K", [(3, 40000), (2, 16385), (5, 12296), (300, 8192)])
def test_in_place_in_long_rows(M, K, dtype):
    x, gamma, beta, dy = make_norm(M, K, dtype, F, seed=K)
    y, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
    own = x.clone()
    assert ss1.layernorm_forward(own, gamma, beta, y=own)[0] is own and torch.equal(own, y)
    dx, dg, db = ss1.layernorm_backward(dy, x, gamma, mean, rstd)
    own = dy.clone()
    got = ss1.layernorm_backward(own, x, gamma, mean, rstd, dx=own)
    assert got[0] is own and torch.equal(own, dx) and torch.equal(got[1], dg) and torch.equal(got[2], db)


def guarded(nbytes):
    """A workspace of nbytes whose contents are NaN in every format, between guards."""
    buf = torch.full((nbytes + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    return buf, buf[256:256 + nbytes]


def untouched(buf):
    return bool((buf[:256] == 0xFF).all()) and bool((buf[-256:] == 0xFF).all())


def asked(query, *args):
    n = ctypes.c_size_t(0)
    assert query(*args, ctypes.byref(n)) == _lib.OK
    return n.value


@BOTH
@pytest.mark.parametrize("case", range(len(LONG_N) + 2))
def test_an_adapters_workspace_of_the_callers(case, dtype):
    segs, ranks, K, N = (LONG_N + [([(1, 0)], [16], 4096, 264), ([(2500, 0), (300, 1), (2700, 0)], [17, 24], 520, 264)])[case]
    c = Case(segs, ranks, K, N, dtype, seed=90 + case)
    y, v = c.forward(base=c.base, save_v=True)
    want = c.backward(v, dx_base=c.dxb)
    ad = ctypes.byref(c.set._struct(0))
    need = asked(_lib.load().ss1_adapter_forward_query, c.M, ad)
    buf, ws = guarded(need)
    got = c.forward(base=c.base, save_v=True, workspace=ws)
    assert torch.equal(got[0], y) and torch.equal(got[1], v) and untouched(buf)
    need_back = asked(_lib.load().ss1_adapter_backward_query, c.M, ad)
    buf, ws = guarded(need_back)
    for a, b in zip(c.backward(v, dx_base=c.dxb, workspace=ws), want):
        assert torch.equal(a, b)
    assert untouched(buf)
    # used again as it was left
    for a, b in zip(c.backward(v, dx_base=c.dxb, workspace=ws), want):
        assert torch.equal(a, b)
    with pytest.raises(_lib.SS1Error):
        c.forward(base=c.base, workspace=ws[:need - 16])
    with pytest.raises(_lib.SS1Error):
        c.backward(v, workspace=ws[:need_back - 16])


@BOTH
@pytest.mark.parametrize("M,K", [(37, 1280), (1500, 1000), (3, 40000), (1281, 72), (9000, 4096)])
def test_a_layer_norms_workspace_of_the_callers(M, K, dtype):
    x, gamma, beta, dy = make_norm(M, K, dtype, F, seed=M)
    _, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
    want = ss1.layernorm_backward(dy, x, gamma, mean, rstd)
    need = asked(_lib.load().ss1_layernorm_backward_query, ctypes.byref(_ops._matrix(x, 0)))
    buf, ws = guarded(need)
    for _ in range(2):
        for a, b in zip(ss1.layernorm_backward(dy, x, gamma, mean, rstd, workspace=ws), want):
            assert torch.equal(a, b)
        assert untouched(buf)
    with pytest.raises(_lib.SS1Error):
        ss1.layernorm_backward(dy, x, gamma, mean, rstd, workspace=ws[:need - 16])
