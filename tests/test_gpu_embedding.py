"""The token embedding and its gradient against their definitions in 64 bits.

Tolerances.  Forward: one float32 product and one rounding to y's type, together
(2^-24 + half a step of y) of the value.  Backward: a row's n tokens are added in
float32 (at most n roundings of partial sums, each at most 2^-24 of the sum of
|dy|), scaled (2^-24), added to what was there (2^-24 of that sum) and rounded
to dE's type."""
import math

import pytest
import torch

import sketched_parameter_sharing_amd as ss1

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # torch.finfo(t).eps / 2
F, H = torch.float32, torch.bfloat16
TINY = 2.0 ** -126


def gen(seed=3):
    return torch.Generator(device="cuda").manual_seed(seed)


def ids_of(kind, M, V, dtype, seed=5):
    g = gen(seed)
    if kind == "text":  # number i about 1 / (i + 1) as often as number 0, some padding
        u = torch.rand((M,), generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * math.log(V + 1)) - 1).floor().long().clamp(0, V - 1)
        ids[torch.rand((M,), generator=g, device="cuda") < 0.05] = -1
    elif kind == "same":
        ids = torch.full((M,), V // 2, device="cuda")
    elif kind == "all":  # every row in turn, descending
        ids = V - 1 - torch.arange(M, device="cuda") % V
    elif kind == "none":
        ids = torch.where(torch.arange(M, device="cuda") % 2 == 0, -1, V)
    else:
        ids = torch.randint(-2, V + 2, (M,), generator=g, device="cuda")
    return ids.to(dtype)


def forward64(ids, table, scale):
    real = (ids >= 0) & (ids < table.shape[0])
    y = torch.zeros((ids.numel(), table.shape[1]), dtype=torch.float64, device="cuda")
    y[real] = table.double()[ids[real].long()] * scale
    return y


@pytest.mark.parametrize("M,V,K", [(1, 1, 1), (1, 1000, 4096), (64, 300, 128), (333, 2003, 1283), (5, 7, 2056),
                                   (1000, 50, 8), (17, 3, 65536), (0, 10, 64), (3, 0, 64), (4097, 129, 72)])
@pytest.mark.parametrize("table_t,out_t", [(H, H), (H, F), (F, H), (F, F)])
@pytest.mark.parametrize("id_t", [torch.int32, torch.int64])
def test_forward(M, V, K, table_t, out_t, id_t):
    table = (torch.randn((V, K), generator=gen(), device="cuda")).to(table_t)
    ids = ids_of("any", M, V, id_t)
    for scale in (1.0, math.sqrt(K), -0.37):
        y = ss1.embedding_forward(ids, table, scale=scale, dtype=out_t)
        assert y.dtype == out_t and y.shape == (M, K)
        want = forward64(ids, table, float(torch.tensor(scale, dtype=F)))
        assert ((y.double() - want).abs() <= (EPS + HALF[out_t]) * want.abs() + TINY).all()
        if scale == 1.0 and table_t == out_t:
            assert torch.equal(y.double(), want)


def test_forward_special_values_and_given_output():
    table = torch.tensor([[float("inf"), float("nan"), -0.0, 1.0] * 2, [2.0] * 8], device="cuda")
    home = torch.full((5, 8), 9.0, device="cuda")
    y = ss1.embedding_forward(torch.tensor([1, 0, 5], device="cuda"), table, scale=2.0, y=home[1:4])
    assert y.data_ptr() == home[1:4].data_ptr()
    assert (home[0] == 9).all() and (home[4] == 9).all() and (home[1] == 4).all() and (home[3] == 0).all()
    assert math.isinf(home[2, 0].item()) and math.isnan(home[2, 1].item()) and home[2, 3].item() == 2.0


def check_backward(M, V, K, kind, dy_t, dE_t, id_t, accumulate, scale=0.75, seed=3):
    g = gen(seed)
    dy = torch.randn((M, K), generator=g, device="cuda").to(dy_t)
    ids = ids_of(kind, M, V, id_t)
    home = torch.full((V + 2, K), 7.0, device="cuda", dtype=dE_t)
    off = 1 if K * home.element_size() % 16 == 0 else 0  # a view is aligned or the call refuses it
    dE = home[off:off + V]
    dE.copy_(torch.randn((V, K), generator=g, device="cuda").to(dE_t))
    before = dE.double().clone()
    got = ss1.embedding_backward(dy, ids, V, scale=scale, dE=dE, accumulate=accumulate)
    assert got.data_ptr() == dE.data_ptr()
    assert (home[off + V:] == 7).all() and (home[:off] == 7).all()
    real = (ids >= 0) & (ids < V)
    rows = ids[real].long()
    # on the host: float64 additions to one row from many threads of the GPU take seconds
    at, shares = rows.cpu(), dy.double()[real].cpu()
    total = torch.zeros((V, K), dtype=torch.float64).index_add_(0, at, shares).cuda()
    size = torch.zeros((V, K), dtype=torch.float64).index_add_(0, at, shares.abs()).cuda()
    count = torch.bincount(at, minlength=V).double().cuda()
    want = scale * total
    slack = EPS * (count[:, None] + 1) * size * scale
    if accumulate:
        want = want + before
        slack = slack + EPS * want.abs()
    out = dE.double()
    assert ((out - want).abs() <= slack * 1.01 + HALF[dE_t] * (want.abs() + slack) + TINY).all()
    empty = count == 0
    if accumulate:
        assert torch.equal(out[empty], before[empty])
    else:
        assert (out[empty] == 0).all()
    return dE


SHAPES = [(1023, 300, 2056), (1024, 3000, 1283), (1100, 70, 33), (2000, 900, 1032), (1, 1, 1), (1, 1000, 512), (2, 5, 8), (15, 300, 72), (16, 300, 520), (17, 2003, 1283), (333, 2003, 1283),
          (1024, 700, 256), (1025, 31, 1000), (3000, 50000, 64), (8192, 1000, 136), (20000, 4000, 24), (0, 40, 64),
          (40, 0, 64), (512, 140000, 8),
          # one launch: rows that a block's waves share; and the last sizes of it
          (511, 700, 1000), (130, 5, 4032), (512, 50, 1024), (512, 50, 1025), (513, 50, 9), (8, 300, 65536),
          # tokens dealt out before the sort: chunks of one step and of several, 256, 512 and (not dealt) 1024 owners
          (16384, 3000, 40), (16383, 3000, 40), (40000, 200000, 8), (17000, 300000, 4), (150000, 900, 16)]


@pytest.mark.parametrize("M,V,K", SHAPES)
@pytest.mark.parametrize("kind", ["text", "same", "all", "any", "none"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_backward(M, V, K, kind, accumulate):
    if V == 0 and kind != "any":
        pytest.skip("no rows")
    n = SHAPES.index((M, V, K)) + 3 * ["text", "same", "all", "any", "none"].index(kind)
    dy_t, dE_t = [(H, H), (F, F), (H, F), (F, H)][n % 4]
    check_backward(M, V, K, kind, dy_t, dE_t, (torch.int32, torch.int64)[n % 2], accumulate)


@pytest.mark.parametrize("dy_t", [H, F])
@pytest.mark.parametrize("dE_t", [H, F])
def test_backward_many_tokens(dy_t, dE_t):
    """More tokens than a sorting wave keeps, and tiles of more than 16."""
    check_backward(70001, 3000, 72, "text", dy_t, dE_t, torch.int32, False)
    check_backward(70001, 300, 9, "same", dy_t, dE_t, torch.int64, True)


def test_backward_gives_equal_bits_and_new_tensors():
    g = gen()
    dy = torch.randn((5000, 264), generator=g, device="cuda").to(H)
    ids = ids_of("text", 5000, 900, torch.int64)
    first = ss1.embedding_backward(dy, ids, 900)
    assert first.dtype == H and ss1.embedding_backward(dy, ids, 900, dtype=F).dtype == F
    for _ in range(5):
        torch.empty(1 << 22, device="cuda").normal_()
        assert torch.equal(ss1.embedding_backward(dy, ids, 900), first)


def test_gradient_against_differences():
    """<dy, y(E + d) - y(E)> = <dE, d> for this linear map, with values that float32 holds exactly."""
    g = gen()
    V, K, M = 40, 24, 200
    ids = ids_of("any", M, V, torch.int64)
    E, d = (torch.randint(-8, 9, (V, K), generator=g, device="cuda").float() for _ in range(2))
    dy = torch.randint(-8, 9, (M, K), generator=g, device="cuda").float()
    change = ss1.embedding_forward(ids, E + d, scale=0.5) - ss1.embedding_forward(ids, E, scale=0.5)
    dE = ss1.embedding_backward(dy, ids, V, scale=0.5)
    assert (dy.double() * change.double()).sum().item() == (dE.double() * d.double()).sum().item()


def test_one_row_with_an_infinity_stays_apart():
    dy = torch.ones((100, 16), device="cuda")
    ids = torch.arange(100, device="cuda") // 10
    dy[57, 3], dy[22, 0] = float("inf"), float("nan")
    ids[80:] = -1
    dy[85] = float("nan")  # padding
    dE = ss1.embedding_backward(dy, ids, 12)
    assert math.isinf(dE[5, 3].item()) and math.isnan(dE[2, 0].item())
    dE[5, 3], dE[2, 0] = 10, 10
    assert (dE[:8] == 10).all() and (dE[8:] == 0).all()


def test_offsets_past_32_bits():
    V, K = 300_007, 8192  # 2.46e9 elements
    table = torch.zeros((V, K), dtype=H, device="cuda")
    table[V - 1], table[262_145] = 3.0, 5.0
    ids = torch.tensor([V - 1, 262_145, 0, V - 1], device="cuda")
    y = ss1.embedding_forward(ids, table, scale=2.0)
    assert [y[i].unique().tolist() for i in range(4)] == [[6.0], [10.0], [0.0], [6.0]]
    dE = ss1.embedding_backward(y, ids, V, scale=0.5, dE=table, accumulate=True)
    assert dE[V - 1].unique().tolist() == [9.0] and dE[262_145].unique().tolist() == [10.0]
    ss1.embedding_backward(y, ids, V, dE=table)
    assert table[V - 1].unique().tolist() == [12.0] and table[262_145].unique().tolist() == [10.0]
    assert table[:262_145].abs().max().item() == 0 and table[262_146:V - 1].abs().max().item() == 0


def test_captured_calls_replay_on_new_tokens():
    V, K, M = 700, 128, 900
    table = torch.randn((V, K), generator=gen(), device="cuda")
    dy = torch.randn((M, K), generator=gen(8), device="cuda")
    ids = ids_of("text", M, V, torch.int32)
    ss1.embedding_backward(dy, ids, V)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = ss1.embedding_forward(ids, table, scale=3.0)
        dE = ss1.embedding_backward(dy, ids, V)
    for k, kind in enumerate(("any", "same", "text", "all", "none")):
        ids.copy_(ids_of(kind, M, V, torch.int32, seed=20 + k))
        dy.normal_()
        graph.replay()
        want_y, want = ss1.embedding_forward(ids, table, scale=3.0), ss1.embedding_backward(dy, ids, V)
        torch.cuda.synchronize()
        assert torch.equal(y, want_y) and torch.equal(dE, want)


@pytest.mark.parametrize("V,K,M", [(700, 128, 300), (900, 72, 20000)])
@pytest.mark.parametrize("id_t", [torch.int32, torch.int64])
def test_captured_gradients_of_few_and_of_many_tokens(V, K, M, id_t):
    dy = torch.randn((M, K), generator=gen(8), device="cuda").to(H)
    ids, shared = ids_of("text", M, V, id_t), torch.zeros((V, K), device="cuda")
    ss1.embedding_backward(dy, ids, V)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dE = ss1.embedding_backward(dy, ids, V)
        ss1.embedding_backward(dy, ids, V, dE=shared, accumulate=True)
    for k, kind in enumerate(("any", "same", "text", "all", "none")):
        ids.copy_(ids_of(kind, M, V, id_t, seed=20 + k))
        dy.normal_()
        shared.fill_(k)
        graph.replay()
        want = ss1.embedding_backward(dy, ids, V)
        more = ss1.embedding_backward(dy, ids, V, dE=torch.full((V, K), float(k), device="cuda"), accumulate=True)
        torch.cuda.synchronize()
        assert torch.equal(dE, want) and torch.equal(shared, more)


def test_gradient_rows_past_32_bits():
    M, K, V = 300_007, 8192, 8  # 2.46e9 elements
    dy, ids = torch.zeros((M, K), dtype=H, device="cuda"), torch.zeros(M, dtype=torch.int32, device="cuda")
    for m, v in ((0, 3), (262_145, 5), (262_146, 3), (M - 1, 7)):
        dy[m], ids[m] = m % 7 + 1, v
    dE = ss1.embedding_backward(dy, ids, V, dtype=F)
    want = torch.zeros((V, K), device="cuda")
    want[3], want[5], want[7] = 1 + 262_146 % 7 + 1, 262_145 % 7 + 1, (M - 1) % 7 + 1
    assert torch.equal(dE, want)


def test_another_stream():
    V, K, M = 700, 128, 900
    table, ids = torch.randn((V, K), generator=gen(), device="cuda"), ids_of("text", M, V, torch.int32)
    y = ss1.embedding_forward(ids, table)
    dE = ss1.embedding_backward(y, ids, V)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2 = ss1.embedding_forward(ids, table, stream=side)
    dE2 = ss1.embedding_backward(y2, ids, V, stream=side)
    side.synchronize()
    assert torch.equal(y, y2) and torch.equal(dE, dE2)


def test_refusals_on_the_gpu():
    x = torch.zeros((4, 16), device="cuda")
    ids = torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ss1.SS1Error):
        ss1.embedding_forward(ids, x, scale=float("inf"))
    with pytest.raises(ss1.SS1Error):
        ss1.embedding_forward(ids, x, y=torch.zeros((5, 16), device="cuda"))
    with pytest.raises(ss1.SS1Error):
        ss1.embedding_backward(x, ids[:3], 9)
    with pytest.raises(ss1.SS1Error):
        ss1.embedding_backward(x.repeat(500, 1), ids.repeat(500), 9,
                               workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ss1.SS1Error):
        ss1.embedding_forward(ids, torch.zeros(65, device="cuda")[1:].view(4, 16))
