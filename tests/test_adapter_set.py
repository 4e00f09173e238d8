"""The C view that an adapter set keeps: a tensor of the set that was given other
memory, another type or another layout is seen at the next call."""
import pytest

import sketched_parameter_sharing_amd as ss1
from sketched_parameter_sharing_amd import _lib

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ss1.load()


def used_set(dtype=F, K=64, N=72, rank=8):
    """A set that a call has used, and a call with it."""
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda").to(dtype)  # noqa: E731
    s = ss1.AdapterSet.make(r(2 * rank, K), r(2 * rank, N), [rank, rank], [0.5, 2.0])
    x = r(5, K)
    seg = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    call = lambda of=s: ss1.adapter_forward(x, of, seg, ids)[0]  # noqa: E731
    call()
    return s, call


def fresh(s):
    """A set over the same tensors that keeps no view."""
    return ss1.AdapterSet(s.A, s.B, s.row, s.scale, s.max_rank, s.ranks)


def test_other_memory_of_each_tensor():
    for change in (lambda s: setattr(s.scale, "data", s.scale * 3), lambda s: setattr(s.A, "data", s.A * 2),
                   lambda s: setattr(s.B, "data", s.B * 2),
                   lambda s: setattr(s.row, "data", torch.tensor([0, 3, 16], dtype=torch.int32, device="cuda"))):
        s, call = used_set()
        y = call()
        old = s.row.data, s.scale.data  # alive, so that the new memory is elsewhere
        change(s)
        assert torch.equal(call(), call(fresh(s))) and not torch.equal(call(), y)
        del old


def test_values_written_in_place_need_no_new_view():
    s, call = used_set()
    y, view = call(), s._struct(0)
    s.scale.mul_(3)
    assert s._struct(0) is view and torch.equal(call(), call(fresh(s))) and not torch.equal(call(), y)


def test_a_transposed_factor_is_refused():
    # a square A of the same memory and sizes, read the other way round
    s, call = used_set(K=16)
    s.A.data = s.A.t()
    with pytest.raises(ValueError, match="contiguous"):
        call()


def test_another_type_in_the_same_memory_is_refused():
    s, call = used_set(BF)
    s.A.data = s.A.view(torch.float16)
    with pytest.raises(TypeError, match="unsupported dtype"):
        call()
    s, call = used_set(BF)
    s.A.data, s.B.data = s.A.view(F), s.B.view(F)
    with pytest.raises(_lib.SS1Error):  # x is bf16
        call()


def test_a_set_made_by_hand_is_checked():
    # the dataclass is public: its index and scale arrays go to the kernels by address alone
    s, call = used_set()
    for change, error in ((dict(row=s.row.long()), "row must be torch.int32"), (dict(row=s.row[:2]), "row must hold 3"),
                          (dict(row=s.row.cpu()), "GPU tensors"), (dict(scale=s.scale.double()), "scale must be"),
                          (dict(scale=s.scale[:1]), "scale must hold 2"), (dict(scale=s.scale.cpu()), "GPU tensors"),
                          (dict(row=s.row.repeat(2)[::2]), "row must be contiguous"),
                          (dict(ranks=(8, 4, 4)), "row must hold 4")):
        fields = {k: getattr(s, k) for k in ("A", "B", "row", "scale", "max_rank", "ranks")}
        with pytest.raises(ValueError, match=error):
            ss1.AdapterSet(**{**fields, **change})._struct(0)  # the view alone: nothing is launched
    for name, value in (("row", s.row.long()), ("scale", s.scale.cpu())):
        was = getattr(s, name)
        setattr(s, name, value)
        with pytest.raises(ValueError):
            s._struct(0)
        setattr(s, name, was)
    call()
