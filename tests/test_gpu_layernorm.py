"""Layer norm on the GPU against its formula in 64 bits, and its gradient
against central differences of the forward.

Tolerances: a float32 sum of n terms in any order has a relative error to the
sum of the terms' sizes of at most about 8 sqrt(n) + 64 units of 2^-24 (eight
standard deviations of random roundings, and a floor for short sums); each
output adds its own rounding, 2^-8 of its value in bf16 and 2^-23 in float32.
"""
import math

import pytest

import sketched_parameter_sharing_amd as ss1

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ss1.load()


def n_eff(n):
    return 8 * math.sqrt(n) + 64


def out_ulp(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -23


def make(M, K, dtype, affine, seed=0, offset=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    x = (r(M, K) + offset * r(M, 1)).to(dtype)
    return x, (1 + 0.2 * r(K)).to(affine), (0.2 * r(K)).to(affine), r(M, K).to(dtype)


def forward64(x, gamma, beta, eps):
    x = x.double()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1)
    rstd = (var + eps).rsqrt()
    xh = (x - mean[:, None]) * rstd[:, None]
    y = xh * gamma.double()
    return (y if beta is None else y + beta.double()), mean, rstd, xh


def forward_tolerances(x, gamma, beta, eps, dtype):
    """Bounds of (y, mean, rstd) by the errors of the two sums."""
    y, mean, rstd, xh = forward64(x, gamma, beta, eps)
    K = x.shape[1]
    e = n_eff(K) * U
    dmean = e * x.double().abs().mean(1) + 1e-30
    # rstd: the relative error of the variance, half of it, plus the differences' own rounding
    drel = e + 4 * U + dmean.square() * rstd.square() + 4 * U * mean.abs() * rstd
    dy = ((dmean * rstd)[:, None] + xh.abs() * drel[:, None] + 4 * U * (mean.abs() * rstd)[:, None]) \
        * gamma.double().abs() + 4 * U * (y.abs() + (0 if beta is None else beta.double().abs()))
    return (y, mean, rstd, xh), (dy + out_ulp(dtype) * y.abs() + 1e-30, dmean, drel * rstd)


SHAPES = [(1, 1), (3, 1), (1, 2), (5, 7), (2, 63), (4, 64), (3, 65), (17, 257), (1, 1024), (9, 1280), (33, 768),
          (6, 2047), (2, 2049), (130, 4096), (3, 5121), (2, 8192), (2, 12296), (1, 16384), (2, 16385), (1, 40000),
          (700, 72), (2500, 33)]
TYPES = [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.bfloat16, torch.bfloat16)]
IDS = ["f32", "bf16", "bf16-affine-bf16"]


@pytest.mark.parametrize("dtype,affine", TYPES, ids=IDS)
@pytest.mark.parametrize("M,K", SHAPES)
def test_forward(M, K, dtype, affine):
    x, gamma, beta, _ = make(M, K, dtype, affine, seed=M * 100003 + K)
    for b in (beta, None):
        y, mean, rstd = ss1.layernorm_forward(x, gamma, b, eps=1e-5)
        (ry, rm, rr, _), (ty, tm, tr) = forward_tolerances(x, gamma, b, 1e-5, dtype)
        assert y.dtype == dtype and y.shape == x.shape
        assert ((mean.double() - rm).abs() <= tm).all()
        assert ((rstd.double() - rr).abs() <= tr).all()
        assert ((y.double() - ry).abs() <= ty).all()


@pytest.mark.parametrize("dtype,affine", TYPES, ids=IDS)
@pytest.mark.parametrize("M,K", SHAPES)
def test_backward(M, K, dtype, affine):
    x, gamma, beta, dy = make(M, K, dtype, affine, seed=M * 100003 + K)
    _, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
    dx, dgamma, dbeta = ss1.layernorm_backward(dy, x, gamma, mean, rstd)
    # the formula from the same mean and rstd, so that only this pass's errors count
    mu, rs, d = mean.double()[:, None], rstd.double()[:, None], dy.double()
    xh = (x.double() - mu) * rs
    g = d * gamma.double()
    ref = rs * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    exh = 4 * U * (x.double().abs() + mu.abs()) * rs           # error of one xh
    e = n_eff(K) * U
    dm1 = e * g.abs().mean(1, keepdim=True)
    dm2 = (e * (g * xh).abs() + g.abs() * exh).mean(1, keepdim=True)
    m2 = (g * xh).mean(1, keepdim=True).abs()
    tol = rs * (dm1 + xh.abs() * dm2 + exh * m2
                + 4 * U * (g.abs() + g.mean(1, keepdim=True).abs() + xh.abs() * m2)) + out_ulp(dtype) * ref.abs()
    assert ((dx.double() - ref).abs() <= tol + 1e-30).all()
    em = n_eff(M) * U
    rg, rb = (d * xh).sum(0), d.sum(0)
    tg = em * (d * xh).abs().sum(0) + (d.abs() * exh).sum(0) + out_ulp(affine) * rg.abs()
    tb = em * d.abs().sum(0) + out_ulp(affine) * rb.abs()
    assert dgamma.dtype == affine and dgamma.shape == (K,)
    assert ((dgamma.double() - rg).abs() <= tg + 1e-30).all()
    assert ((dbeta.double() - rb).abs() <= tb + 1e-30).all()


@pytest.mark.parametrize("M,K", [(3, 40), (5, 129), (2, 4096)])
def test_gradient_against_differences(M, K):
    # L = sum(w y): central differences along random directions of x, gamma and beta.  With steps h the
    # third derivative leaves O(h^2) and the float32 outputs an error of about 2^-23 |w||y| sqrt(MK) / h:
    # h = 2^-6 balances the two at under 1 % of the directional derivatives' size
    x, gamma, beta, w = make(M, K, torch.float32, torch.float32, seed=5, offset=0.5)
    _, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
    dx, dgamma, dbeta = ss1.layernorm_backward(w, x, gamma, mean, rstd)
    h = 2.0 ** -6
    loss = lambda a, b, c: (ss1.layernorm_forward(a, b, c)[0].double() * w.double()).sum()  # noqa: E731
    for i, (t, grad) in enumerate([(x, dx), (gamma, dgamma), (beta, dbeta)]):
        d = torch.randn(t.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(i))
        args = [x, gamma, beta]
        up, down = list(args), list(args)
        up[i], down[i] = t + h * d, t - h * d
        num = (loss(*up) - loss(*down)) / (2 * h)
        ana = (grad.double() * d.double()).sum()
        size = grad.double().norm() * 1.0 + 1e-12
        assert abs(num - ana) <= 1e-2 * size, (i, float(num), float(ana))


def test_no_rows_and_empty_gradients():
    x = torch.empty((0, 96), device="cuda")
    gamma = torch.ones(96, device="cuda")
    y, mean, rstd = ss1.layernorm_forward(x, gamma)
    assert y.shape == (0, 96) and mean.shape == (0,)
    dx, dgamma, dbeta = ss1.layernorm_backward(x, x, gamma, mean, rstd)
    assert dx.shape == (0, 96) and (dgamma == 0).all() and (dbeta == 0).all()


def test_skipped_outputs_and_in_place():
    x, gamma, beta, dy = make(37, 1280, torch.bfloat16, torch.float32, seed=3)
    y, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
    dx, dg, db = ss1.layernorm_backward(dy, x, gamma, mean, rstd)
    only = ss1.layernorm_backward(dy, x, gamma, mean, rstd, dgamma=None, dbeta=None)
    assert only[1] is None and torch.equal(only[0], dx)
    only = ss1.layernorm_backward(dy, x, gamma, mean, rstd, dx=None, dbeta=None)
    assert only[0] is None and only[2] is None and torch.equal(only[1], dg)
    only = ss1.layernorm_backward(dy, x, gamma, mean, rstd, dx=None, dgamma=None)
    assert torch.equal(only[2], db)
    xc, dyc = x.clone(), dy.clone()
    ss1.layernorm_forward(xc, gamma, beta, y=xc)                      # y is x
    assert torch.equal(xc, y)
    ss1.layernorm_backward(dyc, x, gamma, mean, rstd, dx=dyc)         # dx is dy
    assert torch.equal(dyc, dx)


@pytest.mark.parametrize("K", [72, 4096, 40000])
def test_special_values_stay_in_their_row(K):
    x, gamma, beta, dy = make(6, K, torch.float32, torch.float32, seed=11)
    want, wm, wr = ss1.layernorm_forward(x, gamma, beta)
    bad = x.clone()
    bad[1, K // 2], bad[4, 0] = float("inf"), float("nan")
    y, mean, rstd = ss1.layernorm_forward(bad, gamma, beta)
    ok = [0, 2, 3, 5]
    assert torch.equal(y[ok], want[ok])
    assert torch.isnan(y[4]).all() and torch.isnan(y[1]).all()
    dx, _, _ = ss1.layernorm_backward(dy, bad, gamma, mean, rstd)
    full, _, _ = ss1.layernorm_backward(dy, x, gamma, wm, wr)
    assert torch.equal(dx[ok], full[ok])


def test_constant_and_large_rows():
    # a constant row has variance 0: rstd = 1/sqrt(eps), y = beta; a mean of 1000 sigma loses no more than
    # the differences' rounding
    gamma, beta = torch.ones(640, device="cuda"), torch.full((640,), 0.25, device="cuda")
    x = torch.full((2, 640), 3.0, device="cuda")
    y, mean, rstd = ss1.layernorm_forward(x, gamma, beta, eps=1e-4)
    assert (y == 0.25).all() and (mean == 3).all() and torch.allclose(rstd, torch.full_like(rstd, 100.0), rtol=1e-6)
    x, gamma, beta, _ = make(8, 1283, torch.float32, torch.float32, seed=1, offset=1000.0)
    y, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
    (ry, rm, rr, _), (ty, tm, tr) = forward_tolerances(x, gamma, beta, 1e-5, torch.float32)
    assert ((y.double() - ry).abs() <= ty).all() and ((rstd.double() - rr).abs() <= tr).all()


def test_offsets_past_32_bits():
    # 4.6 GB of x; the last rows, against the same rows in a tensor of their own
    M, K = 140001, 16384
    x = torch.randn((M, K), device="cuda", dtype=torch.bfloat16)
    gamma = torch.rand(K, device="cuda") + 0.5
    y, mean, rstd = ss1.layernorm_forward(x, gamma)
    dx, _, _ = ss1.layernorm_backward(x, x, gamma, mean, rstd)
    for rows in (slice(0, 5), slice(M - 5, M)):
        yt, mt, rt = ss1.layernorm_forward(x[rows].clone(), gamma)
        assert torch.equal(y[rows], yt) and torch.equal(mean[rows], mt) and torch.equal(rstd[rows], rt)
        xt = x[rows].clone()
        assert torch.equal(dx[rows], ss1.layernorm_backward(xt, xt, gamma, mt, rt)[0])


def test_equal_calls_give_equal_bits_and_other_streams():
    x, gamma, beta, dy = make(1500, 1000, torch.bfloat16, torch.bfloat16, seed=8)
    y, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
    a = ss1.layernorm_backward(dy, x, gamma, mean, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, m2, r2 = ss1.layernorm_forward(x, gamma, beta)
        b = ss1.layernorm_backward(dy, x, gamma, m2, r2)
    s.synchronize()
    assert torch.equal(y, y2)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


def test_graph_replays():
    x, gamma, beta, dy = make(300, 1280, torch.bfloat16, torch.float32, seed=2)
    outs = {}

    def call():
        outs["y"], outs["m"], outs["r"] = ss1.layernorm_forward(x, gamma, beta)
        outs["dx"], outs["dg"], outs["db"] = ss1.layernorm_backward(dy, x, gamma, outs["m"], outs["r"])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    held = dict(outs)
    x0 = x.clone()
    for r in range(3):
        x.copy_(x0 * (1 + 0.5 * r))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in held.items()}
        call()
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], outs[k]), (r, k)
