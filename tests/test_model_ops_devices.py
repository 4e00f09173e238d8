"""The binding of the embedding, the block-scaled matrices, the dense layer and the
gradient norm on a machine of several GPUs (no GPU here: the tensors only say
where they are): a call runs with the GPU of its tensors as the current one, and
refuses tensors, workspaces and streams of another."""
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

    is_cuda = True

    def __getattr__(self, name):
        return getattr(self.t, name)


def calls(place):
    """Every call with each of its tensors on place.get(name, 1); no kernel is reached."""
    M, K, N, V, f, u8 = 40, 8, 16, 6, torch.float32, torch.uint8
    sizes = dict(x=(M, K), table=(V, K), y=(M, K), dy=(M, K), dE=(V, K), out=(M, N), up=(M, N), dx=(M, K), dW=(N, K),
                 ws=(1 << 18,), norm=(1,), coef=(1,))
    t = {k: On(torch.zeros(s, dtype=f), place.get(k, 1)) for k, s in sizes.items()}
    t["ids"] = On(torch.zeros(M, dtype=torch.int64), place.get("ids", 1))

    def blocks(name, rows, cols):
        return ss1.Fp8Blocks(On(torch.zeros((rows, 128), dtype=u8), place.get(name, 1)),
                             On(torch.zeros((rows, 4), dtype=u8), place.get(name + "s", 1)), 1, cols)

    a, b = blocks("a", M, K), blocks("b", N, K)
    q, qt = blocks("q", M, K), blocks("qt", K, M)
    xt, wt = blocks("xt", K, M), blocks("wt", K, N)
    plan = ss1.GradNormPlan(On(torch.zeros(24, dtype=u8), place.get("entries", 1)),
                            On(torch.zeros((1, 2), dtype=torch.int32), 1), 1, 1, 64, [])
    return {
        "embedding_forward": (lambda **kw: ss1.embedding_forward(t["ids"], t["table"], y=t["y"], **kw),
                              "table ids y"),
        "embedding_backward": (lambda **kw: ss1.embedding_backward(t["dy"], t["ids"], V, dE=t["dE"], workspace=t["ws"],
                                                                   **kw), "dy ids dE ws"),
        "quantize": (lambda **kw: ss1.quantize_fp8_blocks(t["x"], q=q, qt=qt, **kw), "x q qs qt qts"),
        "matmul": (lambda **kw: ss1.matmul_fp8_blocks(a, b, y=t["out"], workspace=t["ws"], **kw), "a as b bs out ws"),
        "dense_forward": (lambda **kw: ss1.dense_forward_fp8(t["x"], b, y=t["out"], xt=xt, workspace=t["ws"], **kw),
                          "x b bs out xt xts ws"),
        "dense_backward": (lambda **kw: ss1.dense_backward_fp8(t["up"], xt, wt, dx=t["dx"], dW=t["dW"],
                                                               workspace=t["ws"], **kw),
                           "up xt xts wt wts dx dW ws"),
        "norm": (lambda **kw: plan.norm(1.0, norm=t["norm"], coef=t["coef"], workspace=t["ws"], **kw),
                 "entries norm coef ws"),
        "clip": (lambda **kw: plan.clip(1.0, norm=t["norm"], coef=t["coef"], workspace=t["ws"], **kw),
                 "entries norm coef ws"),
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


@pytest.mark.parametrize("name", NAMES)
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


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_gpu_is_refused(name):
    class Stream:
        device_index, cuda_stream = 0, 0

    with pytest.raises(ValueError, match="stream"):
        calls({})[name][0](stream=Stream())


def test_a_workspace_of_strides_is_refused():
    x = On(torch.zeros((2000, 8)), 1)
    ids = On(torch.zeros(2000, dtype=torch.int32), 1)
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        ss1.embedding_backward(x, ids, 6, dE=On(torch.zeros((6, 8)), 1), workspace=On(torch.zeros(1 << 18)[::2], 1))


def test_gradients_want_what_they_are_made_of():
    dy = On(torch.zeros((4, 8)), 1)
    with pytest.raises(ValueError, match="needs"):
        ss1.dense_backward_fp8(dy, None, None, dW=None)
    with pytest.raises(ValueError, match="needs"):
        ss1.dense_backward_fp8(dy, None, None, dx=None)
