"""Copies and pickles of an AdamW plan: its table holds device addresses, so a copy
makes its own from its own tensors."""
import copy
import io
import pickle

import pytest

import sketched_parameter_sharing_amd as ss1

torch = pytest.importorskip("torch")


def host_plan(n=300):
    """A plan's fields over host tensors; the table stands for addresses that must not travel."""
    t = lambda value: [torch.full((n,), float(value)), torch.full((7,), float(value))]  # noqa: E731
    p, g, m, v, masters = t(1), t(2), t(3), t(4), [None, None]
    return ss1.AdamWPlan(torch.full((88,), 0xAB, dtype=torch.uint8), torch.zeros((1, 2), dtype=torch.int32), 2, 1,
                         (p, g, m, v, masters, None, None), m, v, None, None, masters, [0.1, 0.0])


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_a_copy_makes_a_table_of_its_own_tensors(how, monkeypatch):
    plan, asked = host_plan(), []
    monkeypatch.setattr(ss1.AdamWPlan, "make", classmethod(lambda cls, *a: asked.append(a) or "made"))
    again = {"copy": copy.copy, "deepcopy": copy.deepcopy, "pickle": lambda p: pickle.loads(pickle.dumps(p))}[how](plan)
    assert again == "made" and len(asked) == 1
    *lists, m_scales, v_scales, decay = asked[0]
    assert m_scales is None and v_scales is None and decay == [0.1, 0.0] and lists[4] == [None, None]
    for old, new in zip(plan.tensors[:4], lists[:4]):
        for a, b in zip(old, new):
            assert torch.equal(a, b) and (a.data_ptr() == b.data_ptr()) == (how == "copy")
    assert b"\xab" * 88 not in pickle.dumps(plan)


def step(plan, at):
    plan.step(step=at, lr=1e-2, seed=at)


def values(plan):
    return [t.float().clone() for part in plan.tensors if part is not None for t in part if t is not None]


def saved_and_loaded(plan):
    file = io.BytesIO()
    torch.save(plan, file)
    file.seek(0)
    return torch.load(file, weights_only=False)  # written two lines above


@pytest.mark.gpu
@pytest.mark.parametrize("state", ["f32", "fp8"])
@pytest.mark.parametrize("how", ["deepcopy", "save"])
def test_a_stepped_copy_moves_and_the_original_stays(how, state):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    g = torch.Generator(device="cuda").manual_seed(1)
    full = [torch.randn(n, generator=g, device="cuda") for n in (1000, 3, 257)]
    plan = ss1.AdamWPlan.make([t.bfloat16() for t in full], [t.clone() for t in full], masters=full,
                              weight_decay=[0.1, 0.0, 0.2], state=state)
    step(plan, 1)
    before = values(plan)
    twin = copy.deepcopy(plan) if how == "deepcopy" else saved_and_loaded(plan)
    step(twin, 2)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(values(plan), before))
    moved = values(twin)
    assert not torch.equal(moved[0], before[0])
    # the original's own second step gives the copy's values
    step(plan, 2)
    assert all(torch.equal(a, b) for a, b in zip(values(plan), moved))


@pytest.mark.gpu
def test_a_copy_beside_its_tensors_keeps_them_together():
    # one deep copy of a plan and of the tensors that the program holds: the copied plan steps the copied tensors
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    flat = torch.zeros(1024, device="cuda")
    params, grads = [flat[:300], flat[512:]], [torch.ones(300, device="cuda"), torch.ones(512, device="cuda")]
    both = copy.deepcopy({"flat": flat, "plan": ss1.AdamWPlan.make(params, grads)})
    step(both["plan"], 1)
    assert (flat == 0).all() and (both["flat"][:300] != 0).all() and (both["flat"][512:] != 0).all()
    assert (both["flat"][300:512] == 0).all()
