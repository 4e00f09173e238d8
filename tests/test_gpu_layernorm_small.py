"""Layer norm's gradients at the sizes where the library changes from one launch
to two, and in the cases that keep small inputs from the single launch.
Definitions and tolerances as for the other sizes."""
import pytest
import torch

import sketched_parameter_sharing_amd as ss1
from test_gpu_layernorm import IDS, TYPES, make, test_backward as check_backward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ss1.load()


@pytest.mark.parametrize("dtype,affine", TYPES, ids=IDS)
@pytest.mark.parametrize("M,K", [(1280, 72), (1281, 72), (1024, 4096), (1025, 4096), (1280, 3276), (127, 15), (128, 17),
                                 (129, 513), (300, 1025), (7, 2056), (511, 4095)])
def test_edges(M, K, dtype, affine):
    check_backward(M, K, dtype, affine)


@pytest.mark.parametrize("dtype,affine", TYPES, ids=IDS)
@pytest.mark.parametrize("M,K", [(37, 1280), (200, 65), (1, 4096)])
def test_skipped_and_in_place(M, K, dtype, affine):
    x, gamma, beta, dy = make(M, K, dtype, affine, seed=M + K)
    _, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
    dx, dg, db = ss1.layernorm_backward(dy, x, gamma, mean, rstd)
    assert torch.equal(ss1.layernorm_backward(dy, x, gamma, mean, rstd, dgamma=None, dbeta=None)[0], dx)
    assert torch.equal(ss1.layernorm_backward(dy, x, gamma, mean, rstd, dx=None, dbeta=None)[1], dg)
    assert torch.equal(ss1.layernorm_backward(dy, x, gamma, mean, rstd, dgamma=None)[2], db)
    for which in ("dy", "x"):  # dx on dy, and on x
        t = {"dy": dy.clone(), "x": x.clone()}
        out, g, b = ss1.layernorm_backward(t["dy"], t["x"], gamma, mean, rstd, dx=t[which])
        assert out is t[which] and torch.equal(out, dx)
        # the column sums run in another order there
        size = (dy.double().abs() * (1 + ((x.double() - mean.double()[:, None]) * rstd.double()[:, None]).abs())).sum(0)
        tol = (8 * M ** 0.5 + 64) * 2.0 ** -23 * size + (2.0 ** -7 if affine == torch.bfloat16 else 2.0 ** -22) * \
            torch.maximum(g.double().abs(), b.double().abs())
        assert ((g.double() - dg.double()).abs() <= tol).all() and ((b.double() - db.double()).abs() <= tol).all()


def test_special_values_reach_their_columns_sums_and_row_alone():
    x, gamma, beta, dy = make(40, 200, torch.float32, torch.float32, seed=12)
    _, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
    dx, dg, db = ss1.layernorm_backward(dy, x, gamma, mean, rstd)
    bad = dy.clone()
    bad[3, 17] = float("nan")
    dx2, dg2, db2 = ss1.layernorm_backward(bad, x, gamma, mean, rstd)
    rows, cols = torch.arange(40, device="cuda") != 3, torch.arange(200, device="cuda") != 17
    assert torch.equal(dx2[rows], dx[rows]) and torch.isnan(dx2[3]).all()
    assert torch.equal(dg2[cols], dg[cols]) and torch.equal(db2[cols], db[cols])
    assert torch.isnan(dg2[17]) and torch.isnan(db2[17])
