"""AdamW steps without a seed draw other random bits each step."""
import pytest

import sketched_parameter_sharing_amd as ss1

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def test_steps_without_a_seed_move_every_element():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    # a constant gradient moves p by lr a step, an eighth of p's bf16 quantum of 2^-7: with bits that differ from step
    # to step an element stays for all 48 with probability (7/8)^48 = 0.0016, with the same bits each time with 7/8
    n, steps, quantum = 4096, 48, 2.0 ** -7
    p = torch.full((n,), 1.5, device="cuda", dtype=torch.bfloat16)
    plan = ss1.AdamWPlan.make([p], [torch.ones(n, device="cuda")])
    for t in range(1, steps + 1):
        plan.step(step=t, lr=quantum / 8, eps=0.0)
    moved = 1.5 - p.double()
    assert (moved == 0).sum() <= 40  # 6.7 on average, six standard deviations of 2.6 above: 22
    # the mean: steps of quantum / 8, within six of its standard deviations
    off = abs(float(moved.mean()) - steps * quantum / 8)
    assert off <= 6 * quantum * (steps * 7 / 64) ** 0.5 / n ** 0.5


def test_the_default_seed_is_the_step():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    out = []
    for kw in ({}, {"seed": 7}, {"seed": 8}):
        g = torch.Generator(device="cuda").manual_seed(2)
        p = torch.randn(5000, generator=g, device="cuda").bfloat16()
        plan = ss1.AdamWPlan.make([p], [torch.randn(5000, generator=g, device="cuda")], state="fp8")
        plan.step(step=7, lr=1e-3, **kw)
        out.append([p, plan.m[0].view(torch.uint8), plan.v[0].view(torch.uint8)])
    for a, b, c in zip(*out):
        assert torch.equal(a, b) and not torch.equal(a, c)
