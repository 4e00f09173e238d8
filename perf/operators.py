"""Workloads of the training and serving operators around an SS1 layer: the low-rank adapters of many requests beside
the shared projection, layer norm's forward and backward pass, and the AdamW step over many tensors.

Each case is a dict of sizes; ``prepare`` draws its inputs on the GPU from a seed, ``run`` is one pass, in elementary
torch operations (``own`` false) or through the package's entry points (``own`` true), ``exact`` is the definition in
64 bits, ``work`` the bytes and operations a pass cannot do without.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
STATE_BLOCK = 256  # elements that share one scale of an 8-bit optimizer state


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one decoded token of one request on the Llama-3-8B gate/up projection: latency
        {"name": "adapter_forward_one", "op": "adapter_forward", "dtype": "bf16", "M": 1, "K": 4096, "N": 14336,
         "S": 1, "E": 1, "rank": 16, "save": False},
        # a decode step: 64 requests of one token each, 48 adapters of ranks up to 64 loaded
        {"name": "adapter_forward_decode", "op": "adapter_forward", "dtype": "bf16", "M": 64, "K": 4096, "N": 14336,
         "S": 64, "E": 48, "rank": 64, "save": False},
        # a prefill step: 12 prompts of ragged lengths, 8 adapters, and v kept for a backward pass
        {"name": "adapter_forward_prefill", "op": "adapter_forward", "dtype": "bf16", "M": 4096, "K": 4096, "N": 14336,
         "S": 12, "E": 8, "rank": 64, "save": True},
        # gradients on the small float32 layer (256 -> 256): latency of the training direction
        {"name": "adapter_backward_small", "op": "adapter_backward", "dtype": "f32", "M": 64, "K": 256, "N": 256,
         "S": 3, "E": 2, "rank": 8},
        # finetuning six adapters on the GPT-2 L up-projection, ragged sequences
        {"name": "adapter_backward_finetune", "op": "adapter_backward", "dtype": "bf16", "M": 8192, "K": 1280,
         "N": 5120, "S": 24, "E": 6, "rank": 64},
        # the norm before a decode step's projections
        {"name": "layernorm_forward_decode", "op": "layernorm_forward", "dtype": "bf16", "affine": "f32", "M": 16,
         "K": 4096},
        # the norm of a large prefill or training batch
        {"name": "layernorm_forward_large", "op": "layernorm_forward", "dtype": "bf16", "affine": "f32", "M": 16384,
         "K": 4096},
        # an odd width and row count in float32
        {"name": "layernorm_backward_odd", "op": "layernorm_backward", "dtype": "f32", "affine": "f32", "M": 1111,
         "K": 1283},
        # the training direction of the large batch
        {"name": "layernorm_backward_large", "op": "layernorm_backward", "dtype": "bf16", "affine": "f32", "M": 16384,
         "K": 4096},
        # the parameters of many adapters and norms: hundreds of small tensors of odd sizes
        {"name": "adamw_many_small", "op": "adamw", "param": "f32", "master": False, "state": "f32", "grad": "bf16",
         "tensors": 400, "elements": 1500000},
        # every compressed MLP weight of a GPT-2 L at c = 4 (36 blocks, 2 x 1280 x 5120 / 4), bf16 with float32 masters
        {"name": "adamw_master", "op": "adamw", "param": "bf16", "master": True, "state": "f32", "grad": "bf16",
         "tensors": 72, "elements": 118000000},
        # the same weights with both states in 8 bits
        {"name": "adamw_eight_bit", "op": "adamw", "param": "bf16", "master": True, "state": "fp8", "grad": "bf16",
         "tensors": 72, "elements": 118000000},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["adapter_forward", "adapter_forward", "adapter_backward", "adapter_backward", "layernorm_forward",
                     "layernorm_backward", "adamw", "adamw"])
    if op.startswith("adapter"):
        forward = op == "adapter_forward"
        while True:
            dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
            K, N = (8 * _log(rng, 32, 1792) for _ in range(2))
            M = _log(rng, 1, 4096 if forward else 8192)
            S = M if M <= 256 and rng.random() < 0.4 else _log(rng, 1, min(M, 64))
            case = {"op": op, "dtype": dtype, "M": M, "K": K, "N": N, "S": S, "E": _log(rng, 1, 48),
                    "rank": rng.randint(1, 64)}
            if forward:
                case["save"] = rng.random() < 0.5
            top = 4096 * (4096 + 14336) if forward else 8192 * (1280 + 5120)
            if M * (K + N) * (2 if dtype == "f32" else 1) <= top:
                return case
    if op.startswith("layernorm"):
        while True:
            K = _log(rng, 48, 16384)
            case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "affine": "f32", "M": _log(rng, 1, 16384),
                    "K": K if rng.random() < 0.4 else K // 8 * 8}
            if case["dtype"] == "bf16" and rng.random() < 0.3:
                case["affine"] = "bf16"
            if case["M"] * K * (2 if case["dtype"] == "f32" else 1) <= 16384 * 4096:
                return case
    param, master, state, grad = rng.choice([
        ("f32", False, "f32", "f32"), ("f32", False, "f32", "bf16"), ("bf16", True, "f32", "bf16"),
        ("bf16", True, "fp8", "bf16"), ("bf16", False, "fp8", "bf16"), ("f32", False, "fp8", "f32"),
        ("bf16", False, "f32", "bf16")])
    tensors = _log(rng, 1, 600)
    return {"op": op, "param": param, "master": master, "state": state, "grad": grad, "tensors": tensors,
            "elements": max(4 * tensors, _log(rng, 2000, 80000000))}


# --------------------------------------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _host(seed):
    g = torch.Generator()
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _ranks(case):
    """Ranks of the adapters, a function of the case alone: the first has the largest, the others from a quarter up."""
    r = case["rank"]
    g = _host(case["E"] * 1000 + r)
    rest = torch.randint(max(1, r // 4), r + 1, (case["E"],), generator=g)
    rest[0] = r
    return rest.tolist()


def _segments(case, seed):
    """Token offsets of the segments (requests) and each one's adapter, -1 for none."""
    M, S, E = case["M"], case["S"], case["E"]
    g = _host(seed + 17)
    if S == M:
        seg = torch.arange(M + 1)
    else:
        seg = torch.cat([torch.zeros(1, dtype=torch.int64),
                         torch.randint(0, M + 1, (S - 1,), generator=g).sort().values, torch.tensor([M])])
    ids = torch.randint(0, E, (S,), generator=g)
    if S > 3:
        ids[torch.randint(0, S, (S // 8,), generator=g)] = -1
    return seg.to(torch.int32), ids.to(torch.int32)


def _prepare_adapter(case, seed):
    M, K, N, dt = case["M"], case["K"], case["N"], DTYPES[case["dtype"]]
    g = _gen(seed)
    ranks = _ranks(case)
    R = sum(ranks)
    seg, ids = _segments(case, seed)
    scale = 1.0 + torch.rand(case["E"], generator=_host(seed + 3))
    row = torch.tensor([0] + ranks).cumsum(0).to(torch.int32)
    s = {"A": _normal(g, (R, K), dt, 1.0 / math.sqrt(K)), "B": _normal(g, (R, N), dt, 0.02), "row": row.cuda(),
         "scale": scale.cuda(), "max_rank": case["rank"], "seg": seg.cuda(), "ids": ids.cuda(),
         "x": _normal(g, (M, K), dt)}
    if case["op"] == "adapter_forward":
        s["base"] = _normal(g, (M, N), dt)
        s["save"] = case["save"]
    else:
        s["dy"] = _normal(g, (M, N), dt, 0.1)
        s["dx_base"] = _normal(g, (M, K), dt, 0.1)
        # v as the forward pass kept it: float32 [M][max_rank], zero beyond a token's rank
        tok, mask = _owners(s)
        s["v"] = _by_rank(s, (s["x"].float() @ s["A"].float().t()) * mask, tok)
    if own:
        import sketched_parameter_sharing_amd as ss1
        s["set"] = ss1.AdapterSet.make(s["A"], s["B"], ranks, scale.tolist())
    return s


def _prepare_layernorm(case, seed):
    M, K, dt, at = case["M"], case["K"], DTYPES[case["dtype"]], DTYPES[case["affine"]]
    g = _gen(seed)
    # rows of unequal mean and size, as a residual stream's
    x = (_normal(g, (M, K), torch.float32) * (0.5 + torch.rand((M, 1), generator=g, device="cuda"))
         + _normal(g, (M, 1), torch.float32)).to(dt)
    s = {"x": x, "gamma": (1.0 + _normal(g, (K,), torch.float32, 0.1)).to(at),
         "beta": _normal(g, (K,), torch.float32, 0.1).to(at), "eps": 1e-5}
    if case["op"] == "layernorm_backward":
        s["dy"] = _normal(g, (M, K), dt, 0.1)
        xf = x.float()
        s["mean"] = xf.mean(1)
        s["rstd"] = 1.0 / torch.sqrt((xf - s["mean"][:, None]).square().mean(1) + s["eps"])
    return s


def _sizes(case):
    """Element counts of the tensors, a function of the case alone: spread over a factor of about 50, odd ones among
    them."""
    T, total = case["tensors"], case["elements"]
    w = torch.exp(torch.rand(T, generator=_host(T * 7 + 1), dtype=torch.float64) * 4.0)
    n = (w / w.sum() * total).floor().long().clamp(min=1)
    return n.tolist()


def _prepare_adamw(case, seed):
    """The tensors are views of flat buffers, every tensor starting at a multiple of 256 elements."""
    g = _gen(seed)
    sizes = _sizes(case)
    starts, at = [], 0
    for n in sizes:
        starts.append(at)
        at += (n + STATE_BLOCK - 1) // STATE_BLOCK * STATE_BLOCK
    pdt, gdt = DTYPES[case["param"]], DTYPES[case["grad"]]
    real = torch.zeros(at, dtype=torch.bool, device="cuda")
    for a, n in zip(starts, sizes):
        real[a:a + n] = True

    def flat(std, dtype=torch.float32):
        return (_normal(g, (at,), torch.float32, std) * real).to(dtype)

    master = flat(0.02)
    s = {"param": master.to(pdt), "grad": flat(0.01, gdt), "starts": starts, "sizes": sizes,
         "decay": [0.1 if n > 2000 else 0.0 for n in sizes], "step": 20, "seed": int(seed) * 1000,
         "lr": 1e-3, "beta1": 0.9, "beta2": 0.999, "eps": 1e-8, "grad_scale": 0.5}
    s["master"] = master if case["master"] else None
    m, r = flat(0.002), flat(0.004).abs()
    if case["state"] == "f32":
        s["m"], s["v"] = m, r.square()
    else:
        for name, t in (("m", m), ("v", r)):
            top = t.view(-1, STATE_BLOCK).abs().amax(1)
            sc = torch.where(top > 0, top / 448.0, torch.ones_like(top))
            s[name] = (t.view(-1, STATE_BLOCK) / sc[:, None]).clamp(-448, 448).view(-1).to(torch.float8_e4m3fn)
            s[name + "_scale"] = sc
    if own:
        import sketched_parameter_sharing_amd as ss1

        def views(t, unit=1):
            return None if t is None else [t[a // unit:a // unit + -(-n // unit)] for a, n in zip(starts, sizes)]

        s["plan"] = ss1.AdamWPlan.make(views(s["param"]), views(s["grad"]), views(s["m"]), views(s["v"]),
                                       masters=views(s["master"]), m_scales=views(s.get("m_scale"), STATE_BLOCK),
                                       v_scales=views(s.get("v_scale"), STATE_BLOCK), weight_decay=s["decay"])
    else:
        # the flat form's own tables: each element's tensor, its place there and its decay
        s["start_of"] = torch.tensor(starts, device="cuda")
        s["decay_of"] = torch.tensor(s["decay"], device="cuda")
    return s


def prepare(case, seed):
    if case["op"].startswith("adapter"):
        return dict(_prepare_adapter(case, seed), op=case["op"])
    if case["op"].startswith("layernorm"):
        return dict(_prepare_layernorm(case, seed), op=case["op"])
    return dict(_prepare_adamw(case, seed), op=case["op"])


# ---------------------------------------------------------------------------------------------------------- plain forms
def _owners(s):
    """Each token's adapter (-1: none), and whether row j of A and B is one of token i's adapter."""
    dev = s["x"].device
    where = torch.searchsorted(s["seg"][1:].contiguous(), torch.arange(s["x"].shape[0], device=dev, dtype=torch.int32),
                               right=True)
    tok = s["ids"][where]
    owner = torch.searchsorted(s["row"][1:].contiguous(),
                               torch.arange(s["A"].shape[0], device=dev, dtype=torch.int32), right=True)
    return tok, (tok[:, None] == owner[None, :]).float()


def _by_rank(s, V, tok):
    """[M][R] with one adapter's columns in use a row -> [M][max_rank]."""
    first = s["row"].long()[tok.clamp(min=0).long()]
    rank = s["row"].long()[tok.clamp(min=0).long() + 1] - first
    j = torch.arange(s["max_rank"], device=V.device)
    at = (first[:, None] + j).clamp(max=V.shape[1] - 1)
    return V.gather(1, at) * ((j < rank[:, None]) & (tok[:, None] >= 0))


def _by_adapter(s, v, tok):
    """[M][max_rank] -> [M][R]: the inverse of _by_rank."""
    R = s["A"].shape[0]
    first = s["row"].long()[tok.clamp(min=0).long()]
    j = torch.arange(R, device=v.device)[None, :] - first[:, None]
    return v.gather(1, j.clamp(0, v.shape[1] - 1))


def _plain_adapter_forward(s):
    tok, mask = _owners(s)
    V = (s["x"].float() @ s["A"].float().t()) * mask
    scaled = V * s["scale"][tok.clamp(min=0).long()][:, None]
    y = (s["base"].float() + scaled @ s["B"].float()).to(s["base"].dtype)
    return (y, _by_rank(s, V, tok)) if s["save"] else y


def _plain_adapter_backward(s):
    tok, mask = _owners(s)
    sc = s["scale"][tok.clamp(min=0).long()][:, None]
    dy, x = s["dy"].float(), s["x"].float()
    V = _by_adapter(s, s["v"], tok) * mask
    dV = (dy @ s["B"].float().t()) * mask * sc
    dx = (s["dx_base"].float() + dV @ s["A"].float()).to(s["x"].dtype)
    dA = (dV.t() @ x).to(s["A"].dtype)
    dB = ((V * sc).t() @ dy).to(s["B"].dtype)
    return dx, dA, dB


def _plain_layernorm_forward(s):
    x = s["x"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / torch.sqrt(d.square().mean(1) + s["eps"])
    y = d * rstd[:, None] * s["gamma"].float() + s["beta"].float()
    return y.to(s["x"].dtype), mean, rstd


def _plain_layernorm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    g = dy * s["gamma"].float()
    dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx.to(s["x"].dtype), (dy * xh).sum(0).to(s["gamma"].dtype), dy.sum(0).to(s["gamma"].dtype)


def _s64(c):
    return c - (1 << 64) if c >= 1 << 63 else c


def _splitmix(seed, counter):
    """SplitMix64's output for state seed + (counter + 1) * golden (Steele, Lea, Flood 2014), int64 bits."""
    z = (counter + 1) * _s64(0x9E3779B97F4A7C15) + seed
    z = (z ^ ((z >> 30) & ((1 << 34) - 1))) * _s64(0xBF58476D1CE4E5B9)
    z = (z ^ ((z >> 27) & ((1 << 37) - 1))) * _s64(0x94D049BB133111EB)
    return z ^ ((z >> 31) & ((1 << 33) - 1))


def _to_e4m3(t, u16, keep_nonzero):
    """Blocks of t as (E4M3 codes, scales): scale = max |t| / 448 of the block (1 for a zero block), the quotient rounded
    up with the probability of its distance, by the 16 random bits u16; a value that must not vanish keeps at least the
    smallest code."""
    b = t.view(-1, STATE_BLOCK)
    top = b.abs().amax(1)
    sc = torch.where(top > 0, top / 448.0, torch.ones_like(top))
    q = (b / sc[:, None]).view(-1)
    a = q.abs()
    high = ((a.view(torch.int32) + (u16.to(torch.int32) << 4)) & ~0xFFFFF).view(torch.float32)
    low = torch.floor(a * 512.0 + u16.float() / 65536.0) / 512.0
    r = torch.where(a < 2.0 ** -6, low, high).clamp(max=448.0)
    if keep_nonzero:
        r = torch.where(t > 0, r.clamp(min=2.0 ** -9), r)
    return torch.copysign(r, t).to(torch.float8_e4m3fn), sc


def _plain_adamw(s):
    s["step"] += 1
    t, b1, b2, lr = s["step"], s["beta1"], s["beta2"], s["lr"]
    c1, c2 = 1 - b1 ** t, 1 - b2 ** t
    n = s["param"].numel()
    i = torch.arange(n, device="cuda")
    tensor = torch.searchsorted(s["start_of"], i, right=True) - 1
    decay = s["decay_of"][tensor]
    place = i - s["start_of"][tensor]
    p = (s["param"] if s["master"] is None else s["master"]).float()
    g = s["grad"].float() * s["grad_scale"]
    eight = "m_scale" in s
    if eight:
        m0 = (s["m"].float().view(-1, STATE_BLOCK) * s["m_scale"][:, None]).view(-1)
        v0 = (s["v"].float().view(-1, STATE_BLOCK) * s["v_scale"][:, None]).view(-1).square()
    else:
        m0, v0 = s["m"], s["v"]
    m = b1 * m0 + (1 - b1) * g
    v = b2 * v0 + (1 - b2) * g * g
    root = torch.sqrt(v)
    p = p * (1 - lr * decay) - (lr / c1) * m / (root * (1 / math.sqrt(c2)) + s["eps"])
    seed = s["seed"] + t
    if eight:
        z = _splitmix(seed, (tensor << 40) + (place >> 1)) >> ((place & 1) * 32)
        codes, scale = _to_e4m3(m, z & 0xFFFF, False)
        s["m"].copy_(codes)
        s["m_scale"].copy_(scale)
        codes, scale = _to_e4m3(root, (z >> 16) & 0xFFFF, True)
        s["v"].copy_(codes)
        s["v_scale"].copy_(scale)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    if s["master"] is not None:
        s["master"].copy_(p)
        s["param"].copy_(p)
    elif s["param"].dtype == torch.float32:
        s["param"].copy_(p)
    else:  # bf16 without a master: rounded up with the probability of its distance
        z = _splitmix(seed, (tensor << 40) + (1 << 39) + (place >> 2)) >> ((place & 3) * 16)
        bits = (p.contiguous().view(torch.int32) + (z & 0xFFFF).to(torch.int32)) & ~0xFFFF
        s["param"].copy_(bits.view(torch.float32))
    return _adamw_outputs(s)


def _adamw_outputs(s):
    return {k: s[k] for k in ("param", "master", "m", "v", "m_scale", "v_scale") if s.get(k) is not None}


# ------------------------------------------------------------------------------------------- through the entry points
def _own(s):
    import sketched_parameter_sharing_amd as ss1
    op = s["op"]
    if op == "adapter_forward":
        y, v = ss1.adapter_forward(s["x"], s["set"], s["seg"], s["ids"], base=s["base"], save_v=s["save"])
        return (y, v) if s["save"] else y
    if op == "adapter_backward":
        return ss1.adapter_backward(s["dy"], s["x"], s["v"], s["set"], s["seg"], s["ids"], dx_base=s["dx_base"])
    if op == "layernorm_forward":
        return ss1.layernorm_forward(s["x"], s["gamma"], s["beta"], eps=s["eps"])
    if op == "layernorm_backward":
        return ss1.layernorm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"])
    s["step"] += 1
    s["plan"].step(step=s["step"], lr=s["lr"], beta1=s["beta1"], beta2=s["beta2"], eps=s["eps"],
                   grad_scale=s["grad_scale"], seed=s["seed"] + s["step"])
    return _adamw_outputs(s)


def run(state):
    if own:
        return _own(state)
    return {"adapter_forward": _plain_adapter_forward, "adapter_backward": _plain_adapter_backward,
            "layernorm_forward": _plain_layernorm_forward, "layernorm_backward": _plain_layernorm_backward,
            "adamw": _plain_adamw}[state["op"]](state)


# ------------------------------------------------------------------------------------------------------------ in 64 bits
def _inputs_only(case, seed):
    """prepare()'s inputs; nothing of the package is wanted here."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def exact(case, seed):
    s = _inputs_only(case, seed)
    f64 = {k: t.double() for k, t in s.items() if isinstance(t, torch.Tensor) and t.is_floating_point()}
    op = case["op"]
    if op.startswith("adapter"):
        seg, ids, row = s["seg"].tolist(), s["ids"].tolist(), s["row"].tolist()
        scale = f64["scale"].tolist()
        spans = [(b, e, row[a], row[a + 1], scale[a]) for b, e, a in zip(seg, seg[1:], ids) if a >= 0 and e > b]
        if op == "adapter_forward":
            y, v = f64["base"], torch.zeros((case["M"], case["rank"]), dtype=torch.float64, device="cuda")
            for b, e, r0, r1, a in spans:
                v[b:e, :r1 - r0] = f64["x"][b:e] @ f64["A"][r0:r1].t()
                y[b:e] += a * (v[b:e, :r1 - r0] @ f64["B"][r0:r1])
            return (y, v) if case["save"] else y
        dx, dA, dB = f64["dx_base"], torch.zeros_like(f64["A"]), torch.zeros_like(f64["B"])
        for b, e, r0, r1, a in spans:
            dv = a * (f64["dy"][b:e] @ f64["B"][r0:r1].t())
            dx[b:e] += dv @ f64["A"][r0:r1]
            dA[r0:r1] += dv.t() @ f64["x"][b:e]
            dB[r0:r1] += a * (f64["v"][b:e, :r1 - r0].t() @ f64["dy"][b:e])
        return dx, dA, dB
    if op == "layernorm_forward":
        x = f64["x"]
        var, mean = torch.var_mean(x, dim=1, correction=0)
        rstd = (var + s["eps"]).rsqrt()
        return torch.addcmul(f64["beta"], (x - mean[:, None]) * rstd[:, None], f64["gamma"]), mean, rstd
    if op == "layernorm_backward":
        xh = (f64["x"] - f64["mean"][:, None]) * f64["rstd"][:, None]
        w = f64["dy"] * f64["gamma"]
        along = (w * xh).sum(1, keepdim=True) / case["K"]
        dx = (w - w.sum(1, keepdim=True) / case["K"] - along * xh) * f64["rstd"][:, None]
        return dx, (f64["dy"] * xh).sum(0), f64["dy"].sum(0)
    eight, t = "m_scale" in s, s["step"] + 1
    m, v = f64["m"], f64["v"]
    if eight:
        m = m * f64["m_scale"].repeat_interleave(STATE_BLOCK)
        v = (v * f64["v_scale"].repeat_interleave(STATE_BLOCK)) ** 2
    p = f64["param"] if s["master"] is None else f64["master"]
    g = f64["grad"] * s["grad_scale"]
    m = torch.lerp(g, m, s["beta1"])
    v = torch.lerp(g * g, v, s["beta2"])
    for a, n, w in zip(s["starts"], s["sizes"], s["decay"]):
        p[a:a + n] *= 1 - s["lr"] * w
    hat = (v / (1 - s["beta2"] ** t)).sqrt()
    p = p - s["lr"] * (m / (1 - s["beta1"] ** t)) / (hat + s["eps"])
    out = {"param": p}
    if s["master"] is not None:
        out["master"] = p
    if eight:  # the codes depend on random bits; the scales do not
        def scales(a):
            top = a.view(-1, STATE_BLOCK).abs().amax(1) / 448
            return torch.where(top > 0, top, torch.ones_like(top))
        out.update(m=None, v=None, m_scale=scales(m), v_scale=scales(v.sqrt()))
    else:
        out.update(m=m, v=v)
    return out


# ------------------------------------------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op.startswith("adapter"):
        M, K, N, e = case["M"], case["K"], case["N"], 2 if case["dtype"] == "bf16" else 4
        ranks = _ranks(case)
        # adapters that no request names need not be read: S segments name this many different ones on average
        mean = sum(ranks) / len(ranks)
        touched = mean * len(ranks) * (1 - (1 - 1 / len(ranks)) ** case["S"])
        weights = touched * (K + N) * e
        if op == "adapter_forward":
            saved = M * case["rank"] * 4 if case["save"] else 0
            return {"bytes": M * (K + 2 * N) * e + weights + saved, "flops": 2 * M * mean * (K + N)}
        grads = sum(ranks) * (K + N) * e
        return {"bytes": M * (3 * K + N) * e + M * case["rank"] * 4 + weights + grads,
                "flops": 4 * M * mean * (K + N)}
    if op.startswith("layernorm"):
        M, K, e, a = case["M"], case["K"], 2 if case["dtype"] == "bf16" else 4, 2 if case["affine"] == "bf16" else 4
        if op == "layernorm_forward":
            return {"bytes": 2 * M * K * e + 8 * M + 2 * K * a, "flops": 8 * M * K}
        return {"bytes": 3 * M * K * e + 8 * M + 3 * K * a, "flops": 14 * M * K}
    n = sum(_sizes(case))
    size = {"bf16": 2, "f32": 4}
    per = size[case["grad"]] + (size[case["param"]] + 8 if case["master"] else 2 * size[case["param"]])
    per += 16 if case["state"] == "f32" else 4 + 16 / STATE_BLOCK
    return {"bytes": n * per, "flops": 16 * n}
