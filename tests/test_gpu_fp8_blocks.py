"""Quantisation to block-scaled E4M3: codes and scales equal to the definition,
worked out in 64 bits from a table of the format's values."""
import math

import pytest
import torch

import sketched_parameter_sharing_amd as ss1

pytestmark = pytest.mark.gpu
F, H = torch.float32, torch.bfloat16


def e4m3_table():
    """The nonnegative finite values of E4M3, by code 0 .. 126."""
    return torch.tensor([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                         for c in range(127)], dtype=torch.float64, device="cuda")


def nearest(v):
    """Codes (uint8) of 64-bit values |v| <= 448 by search: nearest, ties to the even code."""
    table = e4m3_table()
    a = v.abs()
    hi = torch.searchsorted(table, a.contiguous()).clamp(max=126)  # first value >= a
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - table[lo], table[hi] - a
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = torch.where(table[hi] == a, hi, code)
    return (code + 128 * torch.signbit(v)).to(torch.uint8)


def two_to(e):
    return torch.tensor([math.ldexp(1.0, k) for k in range(-300, 301)], dtype=torch.float64, device="cuda")[e + 300]


def expected(x, block):
    """(codes, scale bytes) of x [R][C] by the definition."""
    R, C = x.shape
    v = x.double()
    nb = -(-C // 128)
    finite = torch.where(v.isfinite(), v.abs(), 0.0)
    pad = torch.zeros((-(-R // block) * block, nb * 128), dtype=torch.float64, device="cuda")
    pad[:R, :C] = finite
    top = pad.view(-1, block, nb, 128).amax((1, 3))
    e = torch.full(top.shape, -126, dtype=torch.int64, device="cuda")
    for k in range(-126, 128):  # the smallest exponent that fits
        e = torch.where(top > 448 * two_to(torch.tensor(k, device="cuda")), k + 1, e)
    e = torch.where(top > 0, e, 0)
    scale = torch.full((top.shape[0], -(-nb // 4) * 4), 127, dtype=torch.uint8, device="cuda")
    scale[:, :nb] = (e + 127).to(torch.uint8)
    by = e.repeat_interleave(block, 0)[:R].repeat_interleave(128, 1)[:, :C]
    codes = torch.zeros((R, nb * 128), dtype=torch.uint8, device="cuda")
    q = nearest(torch.where(v.isfinite(), v / two_to(by), 0.0))
    codes[:, :C] = torch.where(v.isfinite(), q, 0x7F)
    return codes, scale


def same(got, x, block):
    codes, scale = expected(x, block)
    mine = got.codes.view(torch.uint8)
    nan = codes == 0x7F
    assert torch.equal(mine[~nan], codes[~nan]) and (mine[nan] & 0x7F == 0x7F).all()
    assert torch.equal(got.scale, scale)


def values(rows, cols, dtype, seed=4):
    """Rows of very unequal size, with exact ties, zeros and a few large columns."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, cols), generator=g, device="cuda") * torch.exp2(
        torch.randint(-20, 20, (rows, 1), generator=g, device="cuda").float())
    x = torch.where(torch.rand((rows, cols), generator=g, device="cuda") < 0.2,
                    torch.randint(-300, 300, (rows, cols), generator=g, device="cuda") / 16.0, x)
    x = torch.where(torch.rand((1, cols), generator=g, device="cuda") < 0.03, x * 50, x)
    x[torch.rand((rows, cols), generator=g, device="cuda") < 0.05] = 0
    if rows > 2:
        x[1] = 0
        x[2] = -0.0
    return x.to(dtype)


SHAPES = [(1, 1), (1, 128), (3, 127), (128, 128), (129, 257), (64, 1000), (257, 513), (1111, 1283), (16, 4096),
          (640, 72), (4, 2048)]


@pytest.mark.parametrize("R,C", SHAPES)
@pytest.mark.parametrize("dtype", [H, F])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("which", ["q", "qt", "both"])
def test_codes_and_scales(R, C, dtype, tile, which):
    x = values(R, C, dtype)
    q, qt = ss1.quantize_fp8_blocks(x, tile=tile, q=None if which == "qt" else True, qt=None if which == "q" else True)
    if which == "qt":
        assert q is None
    else:
        assert q.codes.shape == (R, -(-C // 128) * 128) and q.cols == C and q.block == (128 if tile else 1)
        same(q, x, q.block)
    if which == "q":
        assert qt is None
    else:
        assert qt.codes.shape[0] == C and qt.cols == R
        same(qt, x.t().contiguous(), qt.block)
    if tile and which == "both":
        assert torch.equal(q.codes[:, :C].view(torch.uint8).t(), qt.codes[:, :R].view(torch.uint8))


@pytest.mark.parametrize("R,C", [(1, 1), (129, 257), (300, 72)])
@pytest.mark.parametrize("dtype", [H, F])
@pytest.mark.parametrize("of_q,of_qt", [(1, 128), (128, 1)])
def test_a_scale_of_rows_and_one_of_tiles_in_one_call(R, C, dtype, of_q, of_qt):
    x = values(R, C, dtype)
    q, qt = ss1.Fp8Blocks.empty(R, C, of_q), ss1.Fp8Blocks.empty(C, R, of_qt)
    ss1.quantize_fp8_blocks(x, q=q, qt=qt)
    same(q, x, of_q)
    same(qt, x.t().contiguous(), of_qt)


@pytest.mark.parametrize("dtype", [H, F])
def test_special_values(dtype):
    x = values(256, 256, dtype)
    x[3, 5], x[3, 200], x[130, 7], x[250, 255] = float("inf"), float("nan"), float("-inf"), float("nan")
    x[9] = float("nan")
    for tile in (False, True):
        q, qt = ss1.quantize_fp8_blocks(x, tile=tile, qt=True)
        same(q, x, q.block)
        same(qt, x.t().contiguous(), qt.block)


def test_borders_of_the_scale():
    """Largest values next to 448 times a power of two, the smallest and the largest numbers."""
    rows = []
    for e in (-149, -140, -126, -120, -100, -1, 0, 1, 60, 118, 119):
        for m in (1.0, 1.75, 1.7500001, 1.9999999):
            rows.append(min(math.ldexp(m, e), 3.4028234e38))
    rows += [3.4028234e38, 1.17549435e-38, 1.4e-45, 448.0, 448.0001]
    x = torch.tensor(rows, dtype=torch.float64, device="cuda")[:, None] * torch.tensor([1, -0.5, 0.25, 1 / 3],
                                                                                        device="cuda").double()
    x = x.float()
    q, qt = ss1.quantize_fp8_blocks(x, qt=True)
    same(q, x, 1)
    same(qt, x.t().contiguous(), 1)
    xb = x.to(H)
    same(ss1.quantize_fp8_blocks(xb)[0], xb, 1)


def test_every_tie_goes_to_the_even_code():
    table = e4m3_table()
    mid = (table[1:] + table[:-1]) / 2
    x = torch.cat([mid, -mid, table, torch.nextafter(mid.float(), torch.tensor(1e9, device="cuda")).double(),
                   torch.tensor([448.0], device="cuda")]).float()
    x = torch.cat([x, x.new_zeros(-x.numel() % 64)]).view(-1, 64)
    x = torch.cat([x, torch.full_like(x[:, :1], 448.0)], 1).contiguous()  # scale 1 in every row
    same(ss1.quantize_fp8_blocks(x)[0], x, 1)


def test_given_outputs_and_their_neighbours():
    x = values(130, 200, H)
    homes = [torch.full((134, 256), 9, dtype=torch.uint8, device="cuda"),
             torch.full((204, 256), 9, dtype=torch.uint8, device="cuda")]
    scales = [torch.full((8, 4), 9, dtype=torch.uint8, device="cuda"),
              torch.full((210, 4), 9, dtype=torch.uint8, device="cuda")]
    q = ss1.Fp8Blocks(homes[0][2:132], scales[0][1:3], 128, 200)     # tiles of x
    qt = ss1.Fp8Blocks(homes[1][1:201], scales[1][4:204], 1, 130)    # rows of its transpose
    got = ss1.quantize_fp8_blocks(x, q=q, qt=qt)
    assert got[0] is q and got[1] is qt
    same(q, x, 128)
    same(qt, x.t().contiguous(), 1)
    for t, a, b in ((homes[0], 2, 132), (homes[1], 1, 201), (scales[0], 1, 3), (scales[1], 4, 204)):
        assert (t[:a] == 9).all() and (t[b:] == 9).all()


def test_empty_matrices():
    for shape in ((0, 300), (300, 0), (0, 0)):
        q, qt = ss1.quantize_fp8_blocks(torch.zeros(shape, device="cuda"), qt=True)
        assert q.codes.shape[0] == shape[0] and qt.codes.shape[0] == shape[1]


def test_offsets_past_32_bits():
    x = torch.zeros((300_000, 8192), dtype=H, device="cuda")
    x[-1, 5], x[262_145, 8191] = 3.0, -5.0
    q, qt = ss1.quantize_fp8_blocks(x, qt=True)
    assert (q.codes[-1, 5].item(), q.scale[-1, 0].item()) == (384.0, 127 - 7)
    assert (q.codes[262_145, 8191].item(), q.scale[262_145, 63].item()) == (-320.0, 127 - 6)
    assert (qt.codes[5, 299_999].item(), qt.codes[8191, 262_145].item()) == (384.0, -320.0)
    assert q.codes.view(torch.uint8).count_nonzero().item() == 2
    assert qt.codes.view(torch.uint8).count_nonzero().item() == 2


def test_capture_and_another_stream():
    x = values(300, 500, H)
    q, qt = ss1.quantize_fp8_blocks(x, qt=True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gq, gqt = ss1.quantize_fp8_blocks(x, qt=True)
    for k in range(3):
        x.copy_(values(300, 500, H, seed=30 + k))
        graph.replay()
        q, qt = ss1.quantize_fp8_blocks(x, qt=True)
        torch.cuda.synchronize()
        for a, b in ((gq, q), (gqt, qt)):
            assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scale, b.scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sq, _ = ss1.quantize_fp8_blocks(x, stream=side)
    side.synchronize()
    assert torch.equal(sq.codes.view(torch.uint8), q.codes.view(torch.uint8))
