"""The AdamW step bit for bit: codes, scales, states, masters and randomly rounded
bf16 parameters against the header's formula in IEEE float32 on the host (numpy:
each product, sum, quotient and root rounded once), with the header's random bits.

Gradients of many sizes bring every branch of the step: small codes, quotients and
roots on both sides of the bounds of their short forms, zeros, values that leave
float32's normal range, infinities and NaN.
"""
import math

import numpy as np
import pytest

import sketched_parameter_sharing_amd as ss1

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF, F, E4 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
BLOCK = 256
f32 = np.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ss1.load()


def splitmix(seed, counter):
    """SplitMix64's output for state seed + (counter + 1) * golden."""
    u = lambda v: np.uint64(v & (2 ** 64 - 1))  # noqa: E731
    z = u(seed) + (counter + u(1)) * u(0x9E3779B97F4A7C15)
    z = (z ^ (z >> u(30))) * u(0xBF58476D1CE4E5B9)
    z = (z ^ (z >> u(27))) * u(0x94D049BB133111EB)
    return z ^ (z >> u(31))


DECODE = torch.arange(256, dtype=torch.uint8).view(E4).float().numpy()


def encode(r):
    """Codes of values that E4M3 holds; 127 for NaN."""
    with np.errstate(invalid="ignore"):
        code = torch.from_numpy(r).to(E4).view(torch.uint8).numpy()
    assert (np.isnan(r) | (DECODE[code] == r)).all()
    return np.where(np.isnan(r), np.uint8(127), code)


def quantize(t, u16, root):
    """(codes, scales) of the float32 values t with 16 random bits each."""
    n = len(t)
    good = np.isfinite(t)
    pad = np.zeros(-(-n // BLOCK) * BLOCK, f32)
    pad[:n] = np.where(good, np.abs(t), 0)
    top = pad.reshape(-1, BLOCK).max(1)
    scale = np.where(top > 0, top * (f32(1) / f32(448)), f32(1)).astype(f32)
    q = t / np.repeat(scale, BLOCK)[:n]
    a = np.abs(q)
    high = ((a.view(np.uint32) + (u16.astype(np.uint32) << np.uint32(4))) & np.uint32(0xFFF00000)).view(f32)
    high = np.fmin(high, f32(448))
    low = np.floor(np.where(a < f32(2 ** -6), a, 0).astype(f32) * f32(512) + u16.astype(f32) * f32(2 ** -16)) * f32(2 ** -9)
    r = np.where(a < f32(2 ** -6), low, high).astype(f32)
    if root:
        r = np.where(t > 0, np.fmax(r, f32(2 ** -9)), r)
    r = np.where(good, np.copysign(r, q), f32(np.nan)).astype(f32)
    return encode(r), scale


def host_step(d, i, fmt, decay, h):
    """The step of tensor i of the host copies d: what its arrays become."""
    param, master, _, state = fmt
    n = len(d["grads"][i])
    b1, b2, t = h["beta1"], h["beta2"], h["step"]
    step_size, root_c2 = f32(h["lr"] / (1 - b1 ** t)), f32(1 / math.sqrt(1 - b2 ** t))
    keep = f32(1 - h["lr"] * float(f32(decay)))
    g = d["grads"][i] * f32(h["grad_scale"])
    m, v = d["m"][i], d["v"][i]
    if state == "fp8":
        m = DECODE[m] * np.repeat(d["m_scales"][i], BLOCK)[:n]
        v = DECODE[v] * np.repeat(d["v_scales"][i], BLOCK)[:n]
        v = v * v
    m = f32(b1) * m + f32(1 - b1) * g
    v = f32(b2) * v + f32(1 - b2) * g * g
    r = np.sqrt(v)
    p = (d["masters"] if master else d["params"])[i]
    p = p * keep - step_size * m / (r * root_c2 + f32(h["eps"]))
    e = np.arange(n, dtype=np.uint64)
    stream = np.uint64(i << 40)
    out = {}
    if state == "fp8":
        z = splitmix(h["seed"], stream + (e >> np.uint64(1))) >> ((e & np.uint64(1)) * np.uint64(32))
        out["m"], out["m_scales"] = quantize(m, z & np.uint64(0xFFFF), False)
        out["v"], out["v_scales"] = quantize(r, (z >> np.uint64(16)) & np.uint64(0xFFFF), True)
    else:
        out["m"], out["v"] = m, v
    if param == F:
        out["params"] = p
    elif master:
        out["masters"] = p
        out["params"] = torch.from_numpy(p).to(BF).float().numpy()
    else:
        z = splitmix(h["seed"], stream + np.uint64(1 << 39) + (e >> np.uint64(2))) >> ((e & np.uint64(3)) * np.uint64(16))
        bits = (p.view(np.uint32) + (z & np.uint64(0xFFFF)).astype(np.uint32)) & np.uint32(0xFFFF0000)
        out["params"] = np.where(np.isfinite(p), bits.view(f32), p)
    return out


def host(t):
    return t.view(torch.uint8).cpu().numpy() if t.dtype == E4 else t.float().cpu().numpy()


def same(got, want):
    if got.dtype == np.uint8:  # a NaN code of either sign
        return np.array_equal(np.where(got & 127 == 127, 127, got), want)
    return np.array_equal(got, want, equal_nan=True) and np.array_equal(
        np.signbit(got[~np.isnan(want)]), np.signbit(want[~np.isnan(want)]))


FORMATS = [(p, master, g, s) for p, master in ((F, False), (BF, True), (BF, False)) for g in (F, BF)
           for s in ("f32", "fp8")]
# sizes of the gradients of each tensor: all elements near it, or spread by factors up to e^6 around it
SIZES = [(1, 1.0), (255, 1.0), (256, 1e-3), (0, 1.0), (257, 1e-12), (1001, 1e-20), (777, 1e-26), (4099, 1e9),
         (513, 1e17), (300, 1e18), (2049, 3e18), (260, 1e38), (70, 0.0)]


def make(fmt, seed):
    g = torch.Generator().manual_seed(seed)
    param, master, grad, state = fmt
    d = {k: [] for k in ("params", "grads", "m", "v")}
    d["masters"] = [] if master else None
    if state == "fp8":
        d["m_scales"], d["v_scales"] = [], []
    for n, size in SIZES:
        r = lambda: torch.randn(n, generator=g)  # noqa: E731
        p = 0.1 * r()
        d["params"].append(p.to(param))
        if master:
            d["masters"].append(p)
        values = size * r() * torch.exp(2 * r() if n % 2 else torch.zeros(n))
        if n == 2049:
            values[[5, 600, 601, 2048]] = torch.tensor([float("nan"), float("inf"), -float("inf"), float("nan")])
        d["grads"].append(values.to(grad))
        if state == "f32":
            d["m"].append(0.3 * size * r())
            d["v"].append((0.5 * size * r()).square())
        else:
            blocks = -(-n // BLOCK)
            codes = torch.randint(0, 127, (2, n), generator=g, dtype=torch.uint8)
            d["m"].append((codes[0] | (torch.randint(0, 2, (n,), generator=g, dtype=torch.uint8) << 7)).view(E4))
            d["v"].append(codes[1].view(E4))
            for k in ("m_scales", "v_scales"):
                d[k].append((0.5 + torch.rand(blocks, generator=g)) * max(size, 1e-30) / 448)
    return {k: None if ts is None else [t.cuda() for t in ts] for k, ts in d.items()}


@pytest.mark.parametrize("eps", [1e-8, 1e-14, 0.0, 1e6], ids=lambda e: f"eps{e:g}")
@pytest.mark.parametrize("fmt", FORMATS, ids=lambda f: f"{f[0]}-{f[1]}-{f[2]}-{f[3]}".replace("torch.", ""))
def test_bit_for_bit(fmt, eps):
    d = make(fmt, seed=17)
    decay = [0.1 * (i % 3) for i in range(len(SIZES))]
    plan = ss1.AdamWPlan.make(**d, weight_decay=decay)
    h = dict(lr=1e-2, beta1=0.9, beta2=0.999, eps=eps, grad_scale=0.5)
    for step in (1, 2, 40):
        h.update(step=step, seed=(1 << 63) + 12345 * step)
        before = {k: None if ts is None else [host(t) for t in ts] for k, ts in d.items()}
        plan.step(**h)
        torch.cuda.synchronize()
        with np.errstate(all="ignore"):
            for i, (n, size) in enumerate(SIZES):
                for k, want in host_step(before, i, fmt, decay[i], h).items():
                    got = host(d[k][i])
                    assert same(got, want), (step, i, n, size, k, int((got != want).sum()))


def test_random_rounding_near_the_ends_of_the_codes():
    # one block whose quotients run over the whole range, small codes and both neighbours of 448 among them
    n = BLOCK
    for seed in range(8):
        m = torch.exp(torch.linspace(-16, 0, n)) * torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)
        fmt, d = (F, False, F, "fp8"), {}
        start, sm = quantize(m.numpy().astype(f32), np.zeros(n, np.uint64), False)
        d["params"], d["grads"] = [torch.zeros(n).cuda()], [m.cuda()]
        d["m"] = [torch.from_numpy(start).view(E4).cuda()]
        d["v"] = [torch.from_numpy(start & 127).view(E4).cuda()]
        d["m_scales"], d["v_scales"] = [torch.from_numpy(sm).cuda()], [torch.from_numpy(sm).cuda()]
        d["masters"] = None
        plan = ss1.AdamWPlan.make(**d)
        h = dict(lr=1e-3, beta1=0.0, beta2=0.0, eps=1e-8, grad_scale=1.0, step=1, seed=seed)
        before = {k: None if ts is None else [host(t) for t in ts] for k, ts in d.items()}
        plan.step(**h)
        with np.errstate(all="ignore"):
            for k, want in host_step(before, 0, fmt, 0.0, h).items():
                assert same(host(d[k][0]), want), (seed, k)


@pytest.mark.parametrize("beta1", [0.0, 0.5])
def test_zeros_keep_their_sign(beta1):
    # moments of both zeros beside others: the codes are those of the formula's quotients
    d = make((F, False, F, "fp8"), seed=5)
    for t in d["m"]:
        t.view(torch.uint8)[::3] &= 128
    plan = ss1.AdamWPlan.make(**d)
    h = dict(lr=1e-2, beta1=beta1, beta2=0.5, eps=1e-8, grad_scale=0.0, step=3, seed=11)
    before = {k: None if ts is None else [host(t) for t in ts] for k, ts in d.items()}
    plan.step(**h)
    with np.errstate(all="ignore"):
        for i, (n, size) in enumerate(SIZES):
            for k, want in host_step(before, i, (F, False, F, "fp8"), 0.0, h).items():
                assert same(host(d[k][i]), want), (i, n, size, k)
