"""Infinities and NaN in the gradients of 8-bit AdamW states: they stay with their
elements, in the codes and over the steps that follow.

The other elements are compared bit for bit with a twin whose gradient and states
are zero at those places, so that they count in no maximum there either.
"""
import pytest

import sketched_parameter_sharing_amd as ss1
from test_gpu_adamw import BF, F, HYPER, make

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

N = 777  # three blocks of 256 and a part of one
PLACES = {"one": [300], "first of a block": [256], "last": [N - 1], "several": [3, 4, 255, 290, 511],
          "a thread's eight": list(range(264, 272)), "a block": list(range(256, 512)), "all": list(range(N))}
VALUES = {"nan": float("nan"), "inf": float("inf"), "-inf": -float("inf"),
          "square past the range": 3e38}  # g^2 is infinite, m is not


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ss1.load()


def codes(d, key):
    return d[key][0].view(torch.uint8)


@pytest.mark.parametrize("param,master,grad", [(F, False, F), (BF, True, BF), (BF, False, BF)],
                         ids=["f32", "master", "bf16"])
@pytest.mark.parametrize("value", VALUES)
@pytest.mark.parametrize("where", PLACES)
def test_special_values_stay_with_their_elements(where, value, param, master, grad):
    at = torch.tensor(PLACES[where], device="cuda")
    d, plan = make([N], param, master, grad, "fp8", seed=3)
    e, twin = make([N], param, master, grad, "fp8", seed=3)
    # a large finite m sets its block's scale, as it should: only r is looked at then
    scale_m = value != "square past the range"
    for t in (e["grads"][0], codes(e, "m"), codes(e, "v")):
        t[at] = 0
    d["grads"][0][at] = VALUES[value]
    keep = torch.ones(N, dtype=torch.bool, device="cuda")
    keep[at] = False
    for step in (5, 6, 7):
        plan.step(step=step, seed=step, **HYPER)
        twin.step(step=step, seed=step, **HYPER)
        for k in ("m", "v") if scale_m else ("v",):
            assert torch.equal(d[k + "_scales"][0], e[k + "_scales"][0]), (step, k)
            assert torch.equal(codes(d, k)[keep], codes(e, k)[keep]), (step, k)
            assert torch.isnan(d[k][0].float()[at]).all(), (step, k)
        if scale_m or step == 5:
            for k in ("params", "masters") if master else ("params",):
                assert torch.equal(d[k][0][keep], e[k][0][keep]), (step, k)
        if scale_m:
            assert torch.isnan(d["params"][0][at]).all(), step
        else:  # the update of an infinite second moment is zero, that of the NaN it is held as is not
            assert torch.isfinite(d["params"][0]).all() if step == 5 else torch.isnan(d["params"][0][at]).all()
        # the gradients that follow are ordinary
        d["grads"][0].copy_(e["grads"][0])


def test_all_gradients_nan_leaves_no_finite_state():
    d, plan = make([1000], F, False, F, "fp8", seed=1)
    d["grads"][0].fill_(float("nan"))
    plan.step(step=2, seed=1, **HYPER)
    for k in ("m", "v"):
        assert torch.isnan(d[k][0].float()).all() and (d[k + "_scales"][0] == 1).all()
