"""An AdamW plan over memory that two of its entries would write is refused (no GPU:
the tensors only say that they lie on one)."""
import pytest

import sketched_parameter_sharing_amd as ss1
from test_ops_devices import On

torch = pytest.importorskip("torch")


def on(t):
    return On(t, 0)


def lists(sizes=(300, 7, 0, 1000), param=torch.bfloat16, state=torch.float32):
    make = lambda dtype: [on(torch.zeros(n).to(dtype)) for n in sizes]  # noqa: E731
    d = dict(params=make(param), grads=make(torch.float32), m=make(state), v=make(state))
    if param == torch.bfloat16:
        d["masters"] = make(torch.float32)
    if state != torch.float32:
        for k in ("m_scales", "v_scales"):
            d[k] = [on(torch.ones(-(-n // 256))) for n in sizes]
    return d


@pytest.mark.parametrize("param", [torch.float32, torch.bfloat16], ids=["f32", "bf16"])
@pytest.mark.parametrize("state", [torch.float32, torch.float8_e4m3fn], ids=["f32", "fp8"])
def test_separate_tensors_and_views_side_by_side(param, state):
    assert ss1.AdamWPlan.make(**lists(param=param, state=state)).count == 4
    # views of one buffer that meet without overlapping, and one tensor of gradients for two params
    d = lists(sizes=(256, 256), param=param, state=state)
    for k in ("params", "m", "v"):
        flat = torch.zeros(512).to(d[k][0].dtype)
        d[k] = [on(flat[:256]), on(flat[256:])]
    d["grads"] = [d["grads"][0]] * 2
    assert ss1.AdamWPlan.make(**d).count == 2


@pytest.mark.parametrize("what", ["params", "m", "v", "masters", "m_scales", "v_scales"])
def test_the_same_tensor_twice(what):
    d = lists(sizes=(300, 300), state=torch.float8_e4m3fn)
    d[what][1] = d[what][0]
    with pytest.raises(ValueError, match="share memory"):
        ss1.AdamWPlan.make(**d)


def test_overlaps_across_lists_and_by_a_part():
    d = lists()
    d["v"] = d["m"]
    with pytest.raises(ValueError, match="share memory"):
        ss1.AdamWPlan.make(**d)
    flat = torch.zeros(1000)
    d = lists(sizes=(260, 300), param=torch.float32)
    d["params"] = [on(flat[:260]), on(flat[256:556])]
    with pytest.raises(ValueError, match="share memory"):
        ss1.AdamWPlan.make(**d)
    # a float32 tensor's bytes, not its elements
    d = lists(sizes=(64, 64), param=torch.float32)
    raw = torch.zeros(128)
    d["params"], d["m"] = [on(raw[:64]), d["params"][1]], [on(raw[32:96]), d["m"][1]]
    with pytest.raises(ValueError, match="share memory"):
        ss1.AdamWPlan.make(**d)


def test_empty_tensors_share_nothing():
    assert ss1.AdamWPlan.make(**lists(sizes=(0, 0, 5))).count == 3
