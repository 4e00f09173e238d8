"""The operators' binding on a machine of several GPUs (no GPU here: the tensors
only say where they are): a call runs with the GPU of its tensors as the current
one, and refuses tensors, workspaces and streams of another."""
import contextlib

import pytest

import sketched_parameter_sharing_amd as ss1
from sketched_parameter_sharing_amd import _ops

torch = pytest.importorskip("torch")


class On:
    """A host tensor that says it lies on GPU ``index``."""

    def __init__(self, t, index):
        self.t, self.index = t, index

    def get_device(self):
        return self.index

    def is_contiguous(self):
        return self.t.is_contiguous()

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self.t, name)


def calls(place):
    """Every call with each of its tensors on place.get(name, 1); no kernel is reached."""
    M, K, N, f = 4, 8, 16, torch.float32
    sizes = dict(x=(M, K), y=(M, K), dy=(M, K), dx=(M, K), gamma=(K,), beta=(K,), dgamma=(K,), dbeta=(K,), mean=(M,),
                 rstd=(M,), A=(2, K), B=(2, N), base=(M, N), out=(M, N), v=(M, 2), ady=(M, N), dxb=(M, K), dA=(2, K),
                 dB=(2, N), ws=(1 << 16,), p=(K,), g=(K,), m=(K,), s=(K,))
    t = {k: On(torch.zeros(s, dtype=f), place.get(k, 1)) for k, s in sizes.items()}
    for k, values in (("row", [0, 2]), ("seg", [0, M]), ("ids", [0])):
        t[k] = On(torch.tensor(values, dtype=torch.int32), place.get(k, 1))
    t["scale"] = On(torch.ones(1), place.get("scale", 1))
    ad = ss1.AdapterSet(t["A"], t["B"], t["row"], t["scale"], 2, (2,))
    return {
        "layernorm_forward": (lambda **kw: ss1.layernorm_forward(
            t["x"], t["gamma"], t["beta"], y=t["y"], mean=t["mean"], rstd=t["rstd"], **kw),
            "x gamma beta y mean rstd"),
        "layernorm_backward": (lambda **kw: ss1.layernorm_backward(
            t["dy"], t["x"], t["gamma"], t["mean"], t["rstd"], dx=t["dx"], dgamma=t["dgamma"], dbeta=t["dbeta"],
            workspace=t["ws"], **kw), "x dy gamma mean rstd dx dgamma dbeta ws"),
        "adapter_forward": (lambda **kw: ss1.adapter_forward(
            t["x"], ad, t["seg"], t["ids"], base=t["base"], y=t["out"], v=t["v"], workspace=t["ws"], **kw),
            "x A B row scale seg ids base out v ws"),
        "adapter_backward": (lambda **kw: ss1.adapter_backward(
            t["ady"], t["x"], t["v"], ad, t["seg"], t["ids"], dx_base=t["dxb"], dx=t["dx"], dA=t["dA"], dB=t["dB"],
            workspace=t["ws"], **kw), "x ady v A B row scale seg ids dxb dx dA dB ws"),
        "make": (lambda **kw: ss1.AdamWPlan.make([t["p"]], [t["g"]], [t["m"]], [t["s"]], **kw), "p g m s"),
    }


NAMES = list(calls({}))


@pytest.fixture(autouse=True)
def two_gpus(monkeypatch):
    """The current one is 1, and nothing may be launched."""
    _ops._setup()
    monkeypatch.setattr(_ops, "_current_device", lambda: 1)
    monkeypatch.setattr(_ops, "_raw_stream", lambda index: pytest.fail("a launch"))


@pytest.mark.parametrize("name", NAMES)
def test_a_tensor_of_another_gpu_or_of_the_host_is_refused(name):
    for which in calls({})[name][1].split()[1:]:
        for index, error in ((0, "one GPU"), (-1, "GPU tensors")):
            with pytest.raises(ValueError, match=error):
                calls({which: index})[name][0]()
                pytest.fail(f"{which} on {index}")


@pytest.mark.parametrize("name", NAMES[:-1])
def test_the_gpu_of_the_tensors_becomes_the_current_one(name, monkeypatch):
    seen = []

    @contextlib.contextmanager
    def device(index):
        monkeypatch.setattr(_ops, "_current_device", lambda: index)
        yield
        monkeypatch.setattr(_ops, "_current_device", lambda: 1)

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(_ops, "_raw_stream", lambda index: seen.append((index, _ops._current_device())) or 1 / 0)
    with pytest.raises(ZeroDivisionError):
        calls({k: 0 for k in calls({})[name][1].split()})[name][0]()
    assert seen == [(0, 0)]


@pytest.mark.parametrize("name", NAMES[:-1])
def test_a_stream_of_another_gpu_is_refused(name):
    class Stream:
        device_index, cuda_stream = 0, 0

    with pytest.raises(ValueError, match="stream"):
        calls({})[name][0](stream=Stream())


def test_a_step_on_another_gpu(monkeypatch):
    plan = ss1.AdamWPlan(On(torch.zeros(88, dtype=torch.uint8), 0), On(torch.zeros((1, 2)), 0), 1, 1, (), [], [], None,
                         None, None, [0.0])
    asked = []
    monkeypatch.setattr(torch.cuda, "device", lambda index: asked.append(index) or 1 / 0)
    with pytest.raises(ZeroDivisionError):
        plan.step(step=1, lr=0.1)
    assert asked == [0]
    monkeypatch.setattr(_ops, "_current_device", lambda: 0)
    with pytest.raises(ValueError, match="one GPU"):
        plan.step(step=1, lr=0.1, grad_scale=On(torch.ones(1), 1))


def test_a_workspace_of_strides_is_refused():
    call = lambda ws: ss1.layernorm_backward(*[  # noqa: E731
        On(torch.zeros(s), 1) for s in ((4, 8), (4, 8), (8,), (4,), (4,))], **{
        k: On(torch.zeros(s), 1) for k, s in (("dx", (4, 8)), ("dgamma", (8,)), ("dbeta", (8,)))}, workspace=On(ws, 1))
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        call(torch.zeros(1 << 16)[::2])
