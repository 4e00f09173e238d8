"""The AdamW step over many tensors on the GPU against its formula in 64 bits.

Tolerances: every value is a handful of float32 operations on values that the
formula holds in 64 bits, so each is within 16 units of 2^-24 of the sizes of
the terms it is made of; bf16 params add their rounding (half a unit, 2^-8, to
nearest; one unit, 2^-7, where it is random).  8-bit states lie within one
quantum of the value: 2^-3 of it, or 2^-9 of the block's scale.
"""
import math

import pytest

import sketched_parameter_sharing_amd as ss1

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
HYPER = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ss1.load()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def quantize(t):
    """float32 [n] -> (E4M3 codes, scales), to nearest: a starting state."""
    n = t.numel()
    p = torch.zeros(-(-n // 256) * 256, device="cuda")
    p[:n] = t
    top = p.view(-1, 256).abs().amax(1)
    s = torch.where(top > 0, top / 448, torch.ones_like(top))
    return (p.view(-1, 256) / s[:, None]).clamp(-448, 448).view(-1)[:n].to(E4), s


def per_element(s, n):
    return s.double().repeat_interleave(256)[:n]


def make(sizes, param, master, grad, state, seed=0, decay=0.1):
    g = gen(seed)
    r = lambda n, std: std * torch.randn(n, generator=g, device="cuda")  # noqa: E731
    full = [r(n, 0.1) for n in sizes]
    d = dict(params=[t.to(param) for t in full], grads=[r(n, 1.0).to(grad) for n in sizes],
             masters=[t.clone() for t in full] if master else None)
    m, v = [r(n, 0.1) for n in sizes], [r(n, 0.5).abs() for n in sizes]
    if state == "f32":
        d["m"], d["v"] = m, [t.square() for t in v]
    else:
        for k, q in (("m", m), ("v", v)):
            pairs = [quantize(t) for t in q]
            d[k], d[k + "_scales"] = [p[0] for p in pairs], [p[1] for p in pairs]
    return d, ss1.AdamWPlan.make(**d, weight_decay=decay)


def value(codes, scales, n):
    return codes.float().double() * per_element(scales, n)


def snapshot(d):
    return {k: None if v is None else [t.clone() for t in v] for k, v in d.items()}


def step64(d, i, decay, step, lr, beta1, beta2, eps, grad_scale=1.0):
    """(p, m, v) in 64 bits and bounds of their float32 errors, of tensor i of a snapshot."""
    n = d["params"][i].numel()
    p = (d["params"] if d["masters"] is None else d["masters"])[i].double()
    g = d["grads"][i].double() * grad_scale
    if "m_scales" in d:
        m, v = value(d["m"][i], d["m_scales"][i], n), value(d["v"][i], d["v_scales"][i], n).square()
    else:
        m, v = d["m"][i].double(), d["v"][i].double()
    em = 16 * U * (beta1 * m.abs() + (1 - beta1) * g.abs())
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    den = v.sqrt() / math.sqrt(1 - beta2 ** step) + eps
    upd = lr / (1 - beta1 ** step) / den
    ep = 16 * U * (p.abs() + upd * m.abs()) + upd * em
    return (p * (1 - lr * decay) - upd * m, m, v), (ep, em, 16 * U * v)


FORMATS = [(F, False, F, "f32"), (F, False, BF, "f32"), (BF, True, BF, "f32"), (BF, True, F, "fp8"),
           (BF, False, BF, "f32"), (BF, False, BF, "fp8"), (F, False, F, "fp8"), (F, False, BF, "fp8"),
           (BF, True, F, "f32"), (BF, True, BF, "fp8"), (BF, False, F, "f32"), (BF, False, F, "fp8")]
SIZES = [[1], [255, 256, 257], [4095, 4096, 4097, 3, 0, 8], [100003], [7] * 70, [12289, 1, 65536, 511]]


@pytest.mark.parametrize("fmt", FORMATS, ids=lambda f: f"{f[0]}-{f[1]}-{f[2]}-{f[3]}".replace("torch.", ""))
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_step(sizes, fmt):
    param, master, grad, state = fmt
    decay = [0.1 * (i % 2) for i in range(len(sizes))]
    d, plan = make(sizes, *fmt, seed=len(sizes) + sizes[0], decay=decay)
    for step in (1, 30):
        before = snapshot(d)
        plan.step(step=step, seed=step, grad_scale=0.5, **HYPER)
        for i, n in enumerate(sizes):
            (p, m, v), (ep, em, ev) = step64(before, i, decay[i], step, grad_scale=0.5, **HYPER)
            if n == 0:
                continue
            got = d["params"][i].double()
            if master:
                assert ((d["masters"][i].double() - p).abs() <= ep).all()
                assert torch.equal(d["params"][i], d["masters"][i].to(BF))
            elif param == F:
                assert ((got - p).abs() <= ep).all()
            else:
                assert ((got - p).abs() <= ep + 2.0 ** -7 * p.abs()).all()
            if state == "f32":
                assert ((d["m"][i].double() - m).abs() <= em).all()
                assert ((d["v"][i].double() - v).abs() <= ev).all()
                continue
            for k, want in (("m", m), ("v", v.sqrt())):
                sc = d[k + "_scales"][i].double()
                pad = torch.zeros(sc.numel() * 256, dtype=torch.float64, device="cuda")
                pad[:n] = want.abs()
                top = pad.view(-1, 256).amax(1) / 448
                assert ((sc - torch.where(top > 0, top, torch.ones_like(top))).abs() <= 32 * U * top).all()
                err = (value(d[k][i], d[k + "_scales"][i], n) - want).abs()
                quantum = torch.maximum(want.abs() / 8, per_element(sc, n) * 2.0 ** -9)
                assert (err <= quantum * (1 + 1e-5) + em).all(), k


def test_random_rounding_is_unbiased():
    # the mean over many steps' seeds of a rounded value is the value: with n draws the mean of a rounding that
    # is one of two neighbours q apart is off by at most 6 q / (2 sqrt(n)) (six standard deviations)
    n, trials = 2048, 400
    g = gen(3)
    p0 = 0.1 * torch.randn(n, generator=g, device="cuda")
    grad = torch.randn(n, generator=g, device="cuda")
    (m0, ms), (v0, vs) = quantize(0.1 * torch.randn(n, generator=g, device="cuda")), quantize(
        torch.rand(n, generator=g, device="cuda"))
    p = p0.to(BF)
    d = dict(params=[p], grads=[grad], masters=None, m=[m0.clone()], v=[v0.clone()], m_scales=[ms.clone()],
             v_scales=[vs.clone()])
    plan = ss1.AdamWPlan.make(**d)
    start = snapshot(d)
    (rp, rm, rv), _ = step64(start, 0, 0.0, 10, **HYPER)
    total = {k: torch.zeros(n, dtype=torch.float64, device="cuda") for k in "pmv"}
    for t in range(trials):
        for k in ("params", "m", "v", "m_scales", "v_scales"):
            d[k][0].copy_(start[k][0])
        plan.step(step=10, seed=1000 + t, **HYPER)
        total["p"] += d["params"][0].double()
        total["m"] += value(d["m"][0], d["m_scales"][0], n)
        total["v"] += value(d["v"][0], d["v_scales"][0], n)
    sm, sv = per_element(d["m_scales"][0], n), per_element(d["v_scales"][0], n)
    for k, want, q in (("p", rp, rp.abs() * 2.0 ** -7), ("m", rm, torch.maximum(rm.abs() / 8, sm * 2.0 ** -9)),
                       ("v", rv.sqrt(), torch.maximum(rv.sqrt() / 8, sv * 2.0 ** -9))):
        off = (total[k] / trials - want).abs()
        limit = 6 * q / (2 * math.sqrt(trials)) + 1e-5 * want.abs()
        if k == "v":     # values that would round to zero keep the smallest code
            limit = limit + sv * 2.0 ** -9
        assert (off <= limit).all(), k
    assert total["m"].ne(0).any()


def test_states_of_zeros_and_a_first_step():
    # a fresh plan: zero states; a zero gradient moves nothing but the decay, whatever the format
    for fmt in FORMATS:
        p = torch.full((1000,), 0.5, device="cuda").to(fmt[0])
        grad = torch.zeros(1000, device="cuda", dtype=fmt[2])
        plan = ss1.AdamWPlan.make([p], [grad], masters=[p.float()] if fmt[1] else None, state=fmt[3])
        plan.step(step=1, seed=1, **HYPER)
        assert (p == 0.5).all() and (plan.m[0].float() == 0).all() and (plan.v[0].float() == 0).all()
        if fmt[3] == "fp8":
            assert (plan.m_scales[0] == 1).all() and (plan.v_scales[0] == 1).all()
        # the first step of a constant gradient is lr in size
        grad.fill_(0.25)
        plan.step(step=1, seed=2, **HYPER)
        got = (plan.masters[0] if fmt[1] else p).float()
        tol = 2.0 ** -7 * 0.5 if fmt[0] == BF and not fmt[1] else 1e-6
        assert ((got - 0.49).abs() <= tol).all(), fmt


def test_eight_bit_states_follow_32_bits():
    # 300 steps of a noisy quadratic: the second moment has to move with beta2 = 0.999 (rounding to nearest would
    # hold it), and the params have to get as near the optimum as with float32 states, up to a factor
    n, target = 4096, 0.3
    dist = {}
    for state in ("f32", "fp8"):
        p = torch.zeros(n, device="cuda")
        grad = torch.empty(n, device="cuda")
        plan = ss1.AdamWPlan.make([p], [grad], state=state)
        g = gen(1)
        for t in range(1, 301):
            grad.copy_(p - target + 0.1 * torch.randn(n, generator=g, device="cuda"))
            plan.step(step=t, lr=1e-2, beta1=0.9, beta2=0.999, seed=t)
        v = plan.v[0] if state == "f32" else value(plan.v[0], plan.v_scales[0], n).square()
        dist[state] = (float((p - target).abs().mean()), float(v.double().mean()))
    assert dist["fp8"][0] <= 2 * dist["f32"][0] + 1e-3, dist
    assert 0.8 <= dist["fp8"][1] / dist["f32"][1] <= 1.25, dist


def test_grad_scale_on_the_device_and_mixed_formats():
    # tensors of every format in one plan; a clip coefficient in device memory gives the bits of the same number
    out = []
    for scale in (0.25, torch.full((1,), 0.25, device="cuda")):
        lists = {k: [] for k in ("params", "grads", "m", "v", "masters")}
        for i, (param, master, grad, state) in enumerate(f for f in FORMATS if f[3] == "f32"):
            d, _ = make([300 + 77 * i], param, master, grad, state, seed=i)
            for k in lists:
                lists[k] += [None] if d[k] is None else d[k]
        plan = ss1.AdamWPlan.make(**lists, weight_decay=0.01)
        plan.step(step=3, grad_scale=scale, seed=5, **HYPER)
        out.append([t.clone() for k in ("params", "m", "v") for t in lists[k]])
    for a, b in zip(*out):
        assert torch.equal(a, b)


def test_special_gradients_stay_with_their_elements():
    for state in ("f32", "fp8"):
        d, plan = make([600, 300], F, False, F, state, seed=8)
        e, other = make([600, 300], F, False, F, state, seed=8)
        d["grads"][0][300] = float("nan")
        plan.step(step=2, seed=1, **HYPER)
        other.step(step=2, seed=1, **HYPER)
        assert torch.isnan(d["params"][0][300])
        keep = torch.ones(600, dtype=torch.bool, device="cuda")
        keep[300] = False
        assert torch.equal(d["params"][0][keep], e["params"][0][keep])
        assert torch.equal(d["params"][1], e["params"][1])
        if state == "f32":
            assert torch.equal(d["m"][0][keep], e["m"][0][keep])
        else:             # a block's scale is its own: the first and last blocks are as they were
            for k in ("m", "v"):
                a, b = d[k][0].view(torch.uint8), e[k][0].view(torch.uint8)
                assert torch.equal(a[:256], b[:256]) and torch.equal(a[512:], b[512:])


def test_same_seed_same_bits_other_seed_other_bits():
    res = []
    for seed in (7, 7, 8):
        d, plan = make([5000], BF, False, BF, "fp8", seed=4)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            plan.step(step=5, seed=seed, **HYPER)
        s.synchronize()
        res.append([d["params"][0].clone(), d["m"][0].view(torch.uint8).clone(), d["v"][0].view(torch.uint8).clone()])
    for a, b, c in zip(*res):
        assert torch.equal(a, b) and not torch.equal(a, c)


def test_writes_stay_inside_the_tensors():
    # views of one buffer with guards between them
    sizes, at, spans = [5, 256, 1000, 4097], 0, []
    for n in sizes:
        spans.append((at, at + n))
        at += -(-n // 256) * 256 + 256
    bufs = {k: torch.full((at,), 3.0, device="cuda") for k in ("p", "g", "m", "v")}
    view = lambda k: [bufs[k][a:b] for a, b in spans]  # noqa: E731
    for k in ("m", "v"):
        for t in view(k):
            t.fill_(0.5)
    ss1.AdamWPlan.make(view("p"), view("g"), view("m"), view("v")).step(step=1, **HYPER)
    inside = torch.zeros(at, dtype=torch.bool, device="cuda")
    for a, b in spans:
        inside[a:b] = True
    for k in ("p", "m", "v"):
        assert (bufs[k][~inside] == 3).all()
        assert (bufs[k][inside] != 3).all()


def test_more_than_2_to_31_elements():
    n = 2 ** 31 + 777
    p, grad = torch.zeros(n, device="cuda", dtype=BF), torch.zeros(n, device="cuda", dtype=BF)
    plan = ss1.AdamWPlan.make([p], [grad], state="fp8")
    grad[-9:] = 1.0
    grad[5] = -1.0
    plan.step(step=1, lr=0.5, seed=1)
    assert p.count_nonzero() == 10 and ((p[-9:].float() + 0.5).abs() <= 2.0 ** -8).all()
    assert abs(float(p[5]) - 0.5) <= 2.0 ** -8 and plan.m[0].view(torch.uint8).count_nonzero() == 10


def test_empty_plan_and_graph_replays():
    ss1.AdamWPlan.make([], []).step(step=1, lr=1e-3)
    d, plan = make([3000, 17], BF, True, BF, "fp8", seed=2)
    e, other = make([3000, 17], BF, True, BF, "fp8", seed=2)
    plan.step(step=4, seed=9, **HYPER)
    other.step(step=4, seed=9, **HYPER)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan.step(step=5, seed=9, **HYPER)
    for r in range(3):
        for a, b in zip(d["grads"], e["grads"]):
            a.mul_(0.5)
            b.mul_(0.5)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        other.step(step=5, seed=9, **HYPER)
        torch.cuda.synchronize()
        for k in ("params", "masters", "m_scales", "v_scales"):
            for a, b in zip(d[k], e[k]):
                assert torch.equal(a, b), (r, k)
