"""The global gradient norm and clipping against their definition in 64 bits.

Tolerances: squares and sums are float64 (a rounding each: about 1e-15 here), so
norm and coefficient are within the half step of their one rounding to float32,
2^-24 relative (and 1e-12 for the float64 part).  Clipped gradients are compared
bit for bit with round(g * coef) in IEEE float32 on the host."""
import copy
import io
import math

import pytest
import torch

import sketched_parameter_sharing_amd as ss1

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -24 + 1e-12
SIZES = [[1], [7, 0, 4096, 3], [4095, 4097, 16384, 1, 2049, 40_000], [0, 0], [], [2_000_003, 5, 123_457],
         [300 + 37 * i for i in range(700)], [20_000_000],
         [5000 + i % 3 for i in range(1024)], [4096 * 2049]]


def make(sizes, kinds=(torch.float32, torch.bfloat16), seed=1, std=0.01):
    """Tensors inside larger ones whose other elements must not be touched."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    homes = [(torch.randn(n + 16, device="cuda", generator=g) * std * (1 + i % 5)).to(kinds[i % len(kinds)])
             for i, n in enumerate(sizes)]
    return homes, [h[8:8 + n] for h, n in zip(homes, sizes)]


def norm64(grads):
    return math.sqrt(sum(t.double().square().sum().item() for t in grads))


@pytest.mark.parametrize("sizes", SIZES, ids=[str(i) for i in range(len(SIZES))])
@pytest.mark.parametrize("kinds", [(torch.float32,), (torch.bfloat16,), (torch.float32, torch.bfloat16)],
                         ids=["f32", "bf16", "mixed"])
def test_norm_and_clip(sizes, kinds):
    homes, grads = make(sizes, kinds)
    plan = ss1.GradNormPlan.make(grads)
    want = norm64(grads)
    before = [h.clone() for h in homes]
    for bound in (float("inf"), want * 2, want * 0.3, 0.0):
        norm, coef = plan.norm(bound)
        assert abs(norm.item() - want) <= HALF * want
        c = bound / want if want > bound else 1.0
        assert abs(coef.item() - c) <= HALF * c
        assert all(torch.equal(h, b) for h, b in zip(homes, before))
        again = plan.norm(bound)
        assert torch.equal(norm, again[0]) and torch.equal(coef, again[1])
    norm2, coef2 = plan.clip(want * 2 + 1)
    assert torch.equal(norm2, norm) and coef2.item() == 1.0
    assert all(torch.equal(h, b) for h, b in zip(homes, before))
    norm3, coef3 = plan.clip(want * 0.3)
    assert torch.equal(norm3, norm) and (want == 0 or coef3.item() < 1.0)
    for h, b, n in zip(homes, before, sizes):
        expect = b.cpu()
        expect[8:8 + n] = (expect[8:8 + n].float() * coef3.cpu()).to(b.dtype)
        assert torch.equal(h.cpu(), expect)


def test_gradients_of_every_size_of_number():
    """Squares that float32 cannot hold, and sums of very unequal ones."""
    for scale in (1e-30, 1e-42, 1e30, 3e38):
        g = torch.full((5000,), scale, device="cuda")
        norm, coef = ss1.GradNormPlan.make([g]).norm(scale)
        want = g[0].item() * math.sqrt(5000)
        if want < 3.4e38:
            assert abs(norm.item() - want) <= HALF * want + 2.0 ** -150
        else:
            assert math.isinf(norm.item())  # beyond float32; the coefficient is the float64 norm's
        c = scale / want
        assert abs(coef.item() - c) <= HALF * c
    g = torch.zeros(100_000, device="cuda")
    g[0], g[1:] = 1e4, 1e-4
    norm, _ = ss1.GradNormPlan.make([g]).norm()
    want = norm64([g])
    assert abs(norm.item() - want) <= HALF * want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_infinity_and_nan(dtype):
    for special, norm_is, coef_is in ((float("inf"), math.isinf, lambda c: c == 0.0),
                                      (float("-inf"), math.isinf, lambda c: c == 0.0),
                                      (float("nan"), math.isnan, math.isnan)):
        a, b = torch.ones(5000, device="cuda", dtype=dtype), torch.ones(100, device="cuda", dtype=dtype)
        a[4999] = special
        plan = ss1.GradNormPlan.make([a, b])
        norm, coef = plan.clip(1.0)
        assert norm_is(norm.item()) and coef_is(coef.item())
        # what a product with the coefficient gives: 0 and NaN, or NaN everywhere
        assert math.isnan(a[4999].item())
        assert (b == 0).all() if not math.isnan(coef.item()) else b.isnan().all()
    a = torch.ones(3, device="cuda", dtype=dtype)
    a[1] = float("inf")
    norm, coef = ss1.GradNormPlan.make([a]).norm(float("inf"))
    assert math.isinf(norm.item()) and coef.item() == 1.0


def test_offsets_past_32_bits():
    g = torch.zeros(2 ** 31 + 4103, dtype=torch.bfloat16, device="cuda")
    g[-1], g[2 ** 31], g[5] = 3.0, 4.0, 12.0
    plan = ss1.GradNormPlan.make([g])
    norm, coef = plan.clip(6.5)
    assert norm.item() == 13.0 and coef.item() == 0.5
    assert (g[-1].item(), g[2 ** 31].item(), g[5].item()) == (1.5, 2.0, 6.0)


def test_given_outputs_workspace_and_stream():
    _, grads = make([5000, 70_001])
    plan = ss1.GradNormPlan.make(grads)
    want = plan.norm(0.1)
    norm, coef = (torch.full((1,), 7.0, device="cuda") for _ in range(2))
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = plan.norm(0.1, norm=norm, coef=coef, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got[0] is norm and got[1] is coef
    assert torch.equal(norm, want[0]) and torch.equal(coef, want[1])
    with pytest.raises(ss1.SS1Error):
        plan.norm(0.1, workspace=ws[:16])
    with pytest.raises(ss1.SS1Error):
        plan.norm(-0.1)
    with pytest.raises(ValueError):
        plan.norm(0.1, norm=torch.zeros(2, device="cuda"))


def test_copies_and_saved_plans_have_gradients_of_their_own():
    _, grads = make([5000, 301])
    plan = ss1.GradNormPlan.make(grads)
    file = io.BytesIO()
    torch.save(plan, file)
    file.seek(0)
    for other in (copy.deepcopy(plan), torch.load(file, weights_only=False)):
        other.grads[0].zero_()
        want = norm64(other.grads)
        assert abs(other.norm()[0].item() - want) <= HALF * want
    want = norm64(grads)
    assert abs(plan.norm()[0].item() - want) <= HALF * want


def test_captured_calls_replay_on_new_gradients():
    """Two graphs that share the plan and a workspace, replayed in turn between eager work."""
    _, grads = make([5000, 70_001, 3])
    plan = ss1.GradNormPlan.make(grads)
    ws = torch.empty(1 << 16, dtype=torch.uint8, device="cuda")
    plan.norm(0.1, workspace=ws)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for call in (plan.norm, plan.clip):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(0.25, workspace=ws))
        graphs.append(graph)
    for k in range(4):
        fresh = make([5000, 70_001, 3], seed=10 + k, std=0.01 * 4 ** k)[1]
        for t, f in zip(grads, fresh):
            t.copy_(f)
        graphs[0].replay()
        want = norm64(fresh)
        assert abs(outs[0][0].item() - want) <= HALF * want
        graphs[1].replay()
        torch.cuda.synchronize()
        c = min(1.0, 0.25 / want)
        assert abs(outs[1][1].item() - c) <= HALF * c
        for t, f in zip(grads, fresh):
            assert torch.equal(t.cpu(), (f.cpu().float() * outs[1][1].cpu()).to(t.dtype))


def test_coefficient_feeds_the_optimizer():
    """A step with the coefficient of the norm equals one over gradients that were clipped by it in float32."""
    _, grads = make([5000, 301], (torch.float32,))
    params = [torch.ones_like(g) for g in grads]
    others = [p.clone() for p in params]
    plan = ss1.GradNormPlan.make(grads)
    _, coef = plan.norm(0.05)
    ss1.AdamWPlan.make(params, grads).step(step=1, lr=1e-2, grad_scale=coef)
    plan.clip(0.05)
    ss1.AdamWPlan.make(others, grads).step(step=1, lr=1e-2)
    assert all(torch.equal(a, b) for a, b in zip(params, others))
