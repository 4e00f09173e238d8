"""The low-rank adapters of many requests on the GPU against their formula in
64 bits: random values with derived tolerances, small integers bit for bit,
and the gradients against central differences of the forward.

Tolerances: a float32 sum of n products has an error of at most about
(8 sqrt(n) + 64) 2^-24 of the sum of the products' sizes; v enters the second
product with a relative error of 2^-17 (bf16) or 2^-24 (float32); each output
adds its rounding, 2^-8 of its value in bf16 and 2^-23 in float32.
"""
import math

import pytest

import sketched_parameter_sharing_amd as ss1

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ss1.load()


def n_eff(n):
    return 8 * math.sqrt(n) + 64


class Case:
    """One batch: segments as (length, adapter) pairs."""

    def __init__(self, segs, ranks, K, N, dtype, seed=0, integers=False, max_rank=None):
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        R, M = sum(ranks), sum(n for n, _ in segs)
        if integers:
            r = lambda *s: torch.randint(-2, 3, s, generator=g, device="cuda").float()  # noqa: E731
            scale = [float(1 << (i % 2)) for i in range(len(ranks))]
            a = b = 1.0
        else:
            r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
            scale = [0.5 + 0.25 * i for i in range(len(ranks))]
            a, b = 1 / math.sqrt(K), 0.1
        self.x, self.A, self.B = r(M, K).to(dtype), (a * r(R, K)).to(dtype), (b * r(R, N)).to(dtype)
        self.base, self.dy, self.dxb = r(M, N).to(dtype), r(M, N).to(dtype), r(M, K).to(dtype)
        self.set = ss1.AdapterSet.make(self.A, self.B, ranks, scale)
        if max_rank is not None:
            self.set.max_rank = max_rank
        ends, at = [0], 0
        for n, _ in segs:
            at += n
            ends.append(at)
        self.seg = torch.tensor(ends, dtype=torch.int32, device="cuda")
        self.ids = torch.tensor([e for _, e in segs], dtype=torch.int32, device="cuda")
        self.M, self.K, self.N, self.R, self.dtype = M, K, N, R, dtype
        row = [0]
        for q in ranks:
            row.append(row[-1] + q)
        self.spans = [(ends[i], ends[i + 1], row[e], row[e + 1], scale[e])
                      for i, (n, e) in enumerate(segs) if 0 <= e < len(ranks) and n > 0]

    def forward64(self, base=True):
        """(y, v, tolerance of y, tolerance of v)."""
        x, A, B = self.x.double(), self.A.double(), self.B.double()
        y = self.base.double().clone() if base else torch.zeros((self.M, self.N), dtype=torch.float64, device="cuda")
        v = torch.zeros((self.M, self.set.max_rank), dtype=torch.float64, device="cuda")
        tv, ty = torch.zeros_like(v), 2 * U * y.abs()
        split = 2.0 ** -17 if self.dtype == BF else U
        for b, e, r0, r1, s in self.spans:
            if r1 == r0:
                continue
            w = x[b:e] @ A[r0:r1].t()
            tw = n_eff(self.K) * U * (x[b:e].abs() @ A[r0:r1].abs().t())
            v[b:e, :r1 - r0], tv[b:e, :r1 - r0] = w, tw
            y[b:e] += s * (w @ B[r0:r1])
            ty[b:e] += s * ((tw + w.abs() * (split + n_eff(r1 - r0) * U)) @ B[r0:r1].abs())
        ty += (2.0 ** -8 if self.dtype == BF else 2.0 ** -23) * y.abs() + 2 * U * y.abs()
        return y, v, ty + 1e-30, tv + 1e-30

    def backward64(self, v, base=True):
        """((dx, dA, dB), their tolerances)."""
        x, A, B, dy, v = (t.double() for t in (self.x, self.A, self.B, self.dy, v))
        dx = self.dxb.double().clone() if base else torch.zeros((self.M, self.K), dtype=torch.float64, device="cuda")
        dA, dB = torch.zeros_like(A), torch.zeros_like(B)
        tx, tA, tB = 2 * U * dx.abs(), torch.zeros_like(A), torch.zeros_like(B)
        split = 2.0 ** -17 if self.dtype == BF else U
        for b, e, r0, r1, s in self.spans:
            if r1 == r0:
                continue
            w = v[b:e, :r1 - r0]
            dv = s * (dy[b:e] @ B[r0:r1].t())
            tdv = s * n_eff(self.N) * U * (dy[b:e].abs() @ B[r0:r1].abs().t())
            dx[b:e] += dv @ A[r0:r1]
            tx[b:e] += (tdv + dv.abs() * (split + n_eff(r1 - r0) * U)) @ A[r0:r1].abs()
            dA[r0:r1] += dv.t() @ x[b:e]
            tA[r0:r1] += (tdv + dv.abs() * (split + n_eff(self.M) * U)).t() @ x[b:e].abs()
            dB[r0:r1] += s * (w.t() @ dy[b:e])
            tB[r0:r1] += s * ((w.abs() * (split + (n_eff(self.M) + 2) * U)).t() @ dy[b:e].abs())
        o = 2.0 ** -8 if self.dtype == BF else 2.0 ** -23
        return (dx, dA, dB), tuple(t + (o + 2 * U) * r.abs() + 1e-30 for t, r in ((tx, dx), (tA, dA), (tB, dB)))

    def forward(self, **kw):
        return ss1.adapter_forward(self.x, self.set, self.seg, self.ids, **kw)

    def backward(self, v, **kw):
        return ss1.adapter_backward(self.dy, self.x, v, self.set, self.seg, self.ids, **kw)


def check(c):
    y, v = c.forward(base=c.base, save_v=True)
    ry, rv, ty, tv = c.forward64()
    assert y.dtype == c.dtype and y.shape == (c.M, c.N) and v.dtype == F and v.shape == (c.M, c.set.max_rank)
    assert ((v.double() - rv).abs() <= tv).all(), "v"
    assert ((y.double() - ry).abs() <= ty).all(), "y"
    y2, none = c.forward(base=c.base)
    assert none is None and torch.equal(y, y2)
    got = c.backward(v, dx_base=c.dxb)
    want, tol = c.backward64(v)
    for name, g, w, t in zip(("dx", "dA", "dB"), got, want, tol):
        assert g.dtype == c.dtype and g.shape == w.shape
        assert ((g.double() - w).abs() <= t).all(), name


ONES = [(1, i % 3) for i in range(7)]
BATCHES = [
    # (segments, ranks): one token; a decode batch; ragged lengths; adapters of unequal ranks, none, empty segments
    ([(1, 0)], [16]),
    ([(1, 0)], [1]),
    (ONES, [8, 16, 3]),
    ([(1, -1), (1, 1), (1, -1), (1, 0)], [5, 64]),
    ([(5, 0), (0, 1), (12, 1), (1, -1), (33, 0)], [16, 24]),
    ([(64, 0), (64, 1)], [32, 32]),
    ([(0, 0), (130, 0), (0, 0)], [17]),
    ([(300, 2), (3, 0), (0, 1), (77, 2)], [64, 128, 40]),
    ([(40, 0), (40, 7), (40, -5)], [4, 4]),            # adapters outside the set: none
    ([(20, 0), (21, 1)], [0, 12]),                     # an adapter of rank 0
    ([(257, 0)], [128]),
    ([(33, 0), (2, 1), (70, 0)], [50, 7]),             # rows of v that are no whole number of 16 bytes
    ([(1, 0), (40, 1), (2, 0)], [2, 47]),
]
SIZES = [(8, 8), (64, 40), (256, 256), (72, 1288), (1280, 520), (4096, 264)]


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("K,N", SIZES)
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_random_values(batch, K, N, dtype):
    segs, ranks = BATCHES[batch]
    check(Case(segs, ranks, K, N, dtype, seed=batch * 31 + K))


@pytest.mark.parametrize("segs,ranks,K,N", [
    ([(1500, 0)], [16], 1280, 640),                                    # one adapter, a long sequence
    ([(1, i % 37) for i in range(200)], [8 + i % 57 for i in range(37)], 2048, 1288),
    ([(511, 1), (513, 0), (1, 2), (1024, 1)], [64, 32, 8], 640, 2056),
    ([(2, 0)], [64], 14336, 4096),                                     # the Llama-3-8B down projection
    ([(3, 0), (2, 1)], [16, 8], 4096, 14336),
])
@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_larger(segs, ranks, K, N, dtype):
    check(Case(segs, ranks, K, N, dtype, seed=K + N))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
@pytest.mark.parametrize("K,N", [(64, 40), (264, 72)])
def test_integers_bit_for_bit(batch, K, N, dtype):
    # values in -2..2 and scales of 1 or 2: every sum is a whole number below 2^24 (float32 holds it) and v below
    # 2^16 (two bf16 values hold it), so only the last rounding counts, and that is the reference's own
    segs, ranks = BATCHES[batch]
    c = Case(segs, ranks, K, N, dtype, seed=batch, integers=True)
    y, v = c.forward(base=c.base, save_v=True)
    ry, rv, _, _ = c.forward64()
    assert torch.equal(v.double(), rv)
    assert torch.equal(y, ry.float().to(dtype))
    for got, want in zip(c.backward(v, dx_base=c.dxb), c.backward64(v)[0]):
        assert torch.equal(got, want.float().to(dtype))


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_many_segments_and_adapters(dtype):
    # more segments and adapters than a block has threads, and one adapter with many times the others' tokens
    g = torch.Generator().manual_seed(5)
    ranks = [1 + i % 5 for i in range(300)]
    ids = torch.randint(-1, 300, (700,), generator=g)
    ids[torch.rand(700, generator=g) < 0.3] = 7
    segs = [(int(n), int(e)) for n, e in zip(torch.randint(0, 5, (700,), generator=g), ids)]
    check(Case(segs, ranks, 264, 136, dtype, seed=3))
    c = Case(segs, ranks, 64, 40, dtype, seed=3, integers=True)
    y, v = c.forward(base=c.base, save_v=True)
    ry, rv, _, _ = c.forward64()
    assert torch.equal(v.double(), rv) and torch.equal(y, ry.float().to(dtype))
    for got, want in zip(c.backward(v, dx_base=c.dxb), c.backward64(v)[0]):
        assert torch.equal(got, want.float().to(dtype))


@pytest.mark.parametrize("segs,ranks", [
    ([(2500, 0), (300, 1), (2700, 0)], [16, 24]),                     # parts of an adapter in several segments
    ([(1, 2), (6000, 1), (31, 0), (33, 2), (1, 1)], [100, 64, 5]),
    ([(40, i % 2) for i in range(150)], [3, 128]),
])
def test_uneven_sharing(segs, ranks):
    # adapters whose tokens are cut into several parts beside adapters of one part
    check(Case(segs, ranks, 520, 264, BF, seed=len(segs)))
    c = Case(segs, ranks, 72, 40, BF, seed=1, integers=True)
    _, v = c.forward(save_v=True)
    for got, want in zip(c.backward(v), c.backward64(v, base=False)[0]):
        assert torch.equal(got, want.float().to(BF))
    only = c.backward(v, dx=None, dA=None)[2]                          # dB alone: no shrink runs before it
    assert torch.equal(only, c.backward64(v)[0][2].float().to(BF))


def test_offsets_past_32_bits():
    # 2.4 GB of x: the tokens of one adapter lie at both ends, over 2^31 bytes apart
    M, K, N, tail = 73001, 16384, 64, 300
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn((M, K), generator=g, device="cuda", dtype=BF)
    A = (torch.randn((40, K), generator=g, device="cuda") / 128).to(BF)
    B = (0.1 * torch.randn((40, N), generator=g, device="cuda")).to(BF)
    s = ss1.AdapterSet.make(A, B, [16, 24], [1.0, 2.0])
    seg = torch.tensor([0, 200, 500, M - tail, M], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 1, -1, 0], dtype=torch.int32, device="cuda")
    dy = torch.randn((M, N), generator=g, device="cuda", dtype=BF)
    y, v = ss1.adapter_forward(x, s, seg, ids, save_v=True)
    dx, dA, dB = ss1.adapter_backward(dy, x, v, s, seg, ids)
    assert (y[500:M - tail] == 0).all() and (dx[500:M - tail] == 0).all()
    at = torch.cat([torch.arange(200), torch.arange(M - tail, M)]).cuda()
    xs, dys, vs = x[at].double(), dy[at].double(), v[at, :16].double()
    A0, B0 = A[:16].double(), B[:16].double()
    # rounding of y and dx (2^-8), and of the sums as above
    assert ((vs - xs @ A0.t()).abs() <= n_eff(K) * U * (xs.abs() @ A0.abs().t())).all()
    want = vs @ B0
    assert ((y[at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * (vs.abs() @ B0.abs())).all()
    dv = dys @ B0.t()
    want = dv @ A0
    assert ((dx[at].double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * (dv.abs() @ A0.abs())).all()
    for got, l, r in ((dA[:16], dv, xs), (dB[:16], vs, dys)):
        want = l.t() @ r
        assert ((got.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -15 * (l.abs().t() @ r.abs())).all()


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_without_base_and_in_place(dtype):
    c = Case([(30, 0), (7, -1), (1, 1)], [16, 40], 128, 264, dtype, seed=9)
    y, v = c.forward(save_v=True)
    ry, _, ty, _ = c.forward64(base=False)
    assert ((y.double() - ry).abs() <= ty).all() and (y[30:37] == 0).all()
    dx, dA, dB = c.backward(v)
    (rx, _, _), (tx, _, _) = c.backward64(v, base=False)
    assert ((dx.double() - rx).abs() <= tx).all()
    full, _ = c.forward(base=c.base)
    buf = c.base.clone()
    assert c.forward(base=buf, y=buf)[0] is buf and torch.equal(buf, full)
    want, _, _ = c.backward(v, dx_base=c.dxb)
    buf = c.dxb.clone()
    c.backward(v, dx_base=buf, dx=buf)
    assert torch.equal(buf, want)


def test_skipped_gradients():
    c = Case([(100, 0), (60, 1)], [16, 40], 256, 264, BF, seed=4)
    _, v = c.forward(save_v=True)
    dx, dA, dB = c.backward(v, dx_base=c.dxb)
    only = c.backward(v, dx_base=c.dxb, dA=None, dB=None)
    assert only[1] is None and only[2] is None and torch.equal(only[0], dx)
    only = c.backward(None, dx=None, dB=None)
    assert only[0] is None and torch.equal(only[1], dA)
    only = c.backward(v, dx=None, dA=None)
    assert torch.equal(only[2], dB)


def test_unused_adapters_get_zero_gradients_and_empty_batches():
    c = Case([(9, 1), (3, -1)], [4, 8, 16], 64, 72, BF, seed=6)
    _, v = c.forward(save_v=True)
    _, dA, dB = c.backward(v)
    for d in (dA, dB):
        assert (d[:4] == 0).all() and (d[12:] == 0).all() and (d[4:12] != 0).any()
    e = Case([(0, 0)], [4], 64, 72, BF)
    y, v = e.forward(save_v=True)
    assert y.shape == (0, 72) and v.shape == (0, 4)
    dx, dA, dB = e.backward(v)
    assert dx.shape == (0, 64) and (dA == 0).all() and (dB == 0).all()
    n = Case([(5, -1), (4, 0)], [0], 64, 72, BF)        # no adapter rows at all
    y, _ = n.forward(base=n.base)
    assert torch.equal(y, n.base)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    y, _ = ss1.adapter_forward(c.x, c.set, torch.zeros(1, dtype=torch.int32, device="cuda"), none, base=c.base)
    assert torch.equal(y, c.base)                       # no segments: nobody has an adapter


def test_wider_max_rank_leaves_zero_columns():
    c = Case([(20, 0), (3, 1)], [5, 9], 64, 72, BF, seed=2, max_rank=50)
    check(c)
    _, v = c.forward(save_v=True)
    assert v.shape == (23, 50) and (v[:20, 5:] == 0).all() and (v[20:, 9:] == 0).all()


def test_index_arrays_out_of_order_stay_inside():
    # arrays that break the rules leave y unspecified, but every read and write stays inside the buffers
    c = Case([(50, 0), (14, 1)], [16, 40], 128, 264, BF, seed=3)
    guard = torch.full((c.M + 2, c.N), 7.0, dtype=BF, device="cuda")
    row = c.set.row.clone()
    for seg, r in (([0, 1000, 64], row), ([-5, 30, 20], row), ([10, 20, 30], row), ([0, 50, 64], row.flip(0)),
                   ([0, 50, 64], row + 1000), ([0, 50, 64], row - 1000)):
        c.set.row.copy_(r)
        s = torch.tensor(seg, dtype=torch.int32, device="cuda")
        _, v = ss1.adapter_forward(c.x, c.set, s, c.ids, base=c.base, y=guard[1:-1], save_v=True)
        ss1.adapter_backward(c.dy, c.x, v, c.set, s, c.ids)
        torch.cuda.synchronize()
        assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    c.set.row.copy_(row)
    check(c)


def test_special_values_stay_with_their_tokens_and_adapters():
    # an infinity or a NaN in one token's row, or in one adapter's factors, reaches no other token or adapter
    for dtype in (BF, F):
        c = Case([(5, 0), (6, 1), (5, 2)], [16, 7, 16], 128, 136, dtype, seed=12)
        y0, v0 = c.forward(base=c.base, save_v=True)
        g0 = c.backward(v0)
        c.x[7, 3] = float("nan")
        c.dy[7, 5] = float("inf")
        y, v = c.forward(base=c.base, save_v=True)
        keep = [i for i in range(16) if i != 7]
        assert torch.equal(y[keep], y0[keep]) and torch.isnan(y[7]).all()
        dx, dA, dB = c.backward(v)
        assert torch.equal(dx[keep], g0[0][keep])
        for d, d0 in ((dA, g0[1]), (dB, g0[2])):
            assert torch.equal(d[:16], d0[:16]) and torch.equal(d[23:], d0[23:])
        c = Case([(5, 0), (6, 1), (5, 2)], [16, 7, 16], 128, 136, dtype, seed=12)
        c.A[16:23] = float("nan")
        c.B[16:23] = float("inf")
        y, _ = c.forward(base=c.base)
        keep = [i for i in range(16) if not 5 <= i < 11]
        assert torch.equal(y[keep], y0[keep])


@pytest.mark.parametrize("dtype", [BF, F], ids=["bf16", "f32"])
def test_gradient_against_differences(dtype):
    # L = sum(dy y) is linear in each of x, A and B, so a central difference is exact up to rounding; steps of 2
    # in integer values keep the bf16 inputs exact.  float32 y: the sums are whole numbers, the difference exact.
    # bf16: y without a base in float32 is not available, so the float32 set carries the bf16 values
    c = Case([(9, 0), (14, 1), (3, -1)], [8, 5], 64, 40, dtype, seed=1, integers=True)
    _, v = c.forward(save_v=True)
    dx, dA, dB = c.backward(v)
    g = torch.Generator(device="cuda").manual_seed(3)
    f = {k: getattr(c, k).float() for k in ("x", "A", "B")}
    for name, grad in (("x", dx), ("A", dA), ("B", dB)):
        d = torch.randint(-1, 2, f[name].shape, generator=g, device="cuda").float()

        def loss(sign):
            t = dict(f)
            t[name] = f[name] + sign * d
            s = ss1.AdapterSet.make(t["A"], t["B"], c.set.ranks, c.set.scale.tolist())
            return (ss1.adapter_forward(t["x"], s, c.seg, c.ids)[0].double() * c.dy.double()).sum()

        num = (loss(1) - loss(-1)) / 2
        ana = (grad.double() * d.double()).sum()
        tol = 2.0 ** -8 * (grad.double() * d.double()).abs().sum() if dtype == BF else 0.0
        assert abs(num - ana) <= tol, (name, float(num), float(ana))


def test_equal_calls_give_equal_bits_and_other_streams():
    c = Case([(700, 0), (300, 1), (1, 0)], [16, 64], 1280, 520, BF, seed=21)
    y, v = c.forward(base=c.base, save_v=True)
    a = c.backward(v, dx_base=c.dxb)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, v2 = c.forward(base=c.base, save_v=True)
        b = c.backward(v2, dx_base=c.dxb)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(v, v2)
    for p, q in zip(a, b):
        assert torch.equal(p, q)


@pytest.mark.parametrize("segs", [[(1, i % 3) for i in range(16)], [(200, 0), (90, 2)]])
def test_graph_replays(segs):
    c = Case(segs, [16, 8, 32], 512, 264, BF, seed=14)
    outs = {}

    def call():
        outs["y"], outs["v"] = c.forward(base=c.base, save_v=True)
        outs["dx"], outs["dA"], outs["dB"] = c.backward(outs["v"], dx_base=c.dxb)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    held = dict(outs)
    x0 = c.x.clone()
    for r in range(3):
        c.x.copy_(x0 * (1 + 0.5 * r))
        c.ids.copy_(c.ids.roll(1))           # other requests, the same buffers
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        got = {k: t.clone() for k, t in held.items()}
        call()
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k], outs[k]), (r, k)
