"""Calls with a stream of the caller's: results, and whose memory they allocate."""
import pytest
import torch

import sketched_parameter_sharing_amd as ss1

pytestmark = pytest.mark.gpu


def pool_of(t):
    """Handle of the stream whose memory holds t."""
    at = t.data_ptr()
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= at < seg["address"] + seg["total_size"]:
            return seg["stream"]
    raise AssertionError("not in the allocator's memory")


def calls(M=96, K=64, N=96, rank=8):
    g = torch.Generator(device="cuda").manual_seed(5)

    def draw(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    x, dy, gamma, beta = draw(M, K), draw(M, N), draw(K), draw(K)
    seg = torch.tensor([0, 40, M], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    adapters = ss1.AdapterSet.make(draw(2 * rank, K), draw(2 * rank, N), [rank, rank], [0.5, 2.0])
    _, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
    _, v = ss1.adapter_forward(x, adapters, seg, ids, save_v=True)
    return {
        "layernorm_forward": lambda s: ss1.layernorm_forward(x, gamma, beta, stream=s),
        "layernorm_backward": lambda s: ss1.layernorm_backward(x, x, gamma, mean, rstd, stream=s),
        "adapter_forward": lambda s: ss1.adapter_forward(x, adapters, seg, ids, save_v=True, stream=s),
        "adapter_backward": lambda s: ss1.adapter_backward(dy, x, v, adapters, seg, ids, stream=s),
    }


@pytest.mark.parametrize("name", ["layernorm_forward", "layernorm_backward", "adapter_forward", "adapter_backward"])
def test_a_given_stream_owns_what_the_call_allocates(name, monkeypatch):
    call = calls()[name]
    want = call(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    made = []
    for maker in ("empty", "empty_like"):
        real = getattr(torch, maker)

        def wrapped(*args, real=real, **kwargs):
            made.append(real(*args, **kwargs))
            return made[-1]

        monkeypatch.setattr(torch, maker, wrapped)
    got = call(side)
    monkeypatch.undo()
    before = torch.cuda.current_stream().cuda_stream
    side.synchronize()
    # outputs and workspace alike
    assert len(made) >= len(got)
    assert all(pool_of(t) == side.cuda_stream for t in made if t.numel())
    assert torch.cuda.current_stream().cuda_stream == before
    for a, b in zip(got, want):
        assert torch.equal(a, b)
