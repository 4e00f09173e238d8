"""Workloads of the operators that stand where a model with projected layers begins and ends, and between them: the
token embedding and its gradient, the layers that stay dense (in 8-bit floating point with a scale for each block of
128, forward and backward, and the quantising itself), and the global gradient norm with its clipping.

Each case is a dict of sizes; ``prepare`` draws its inputs on the GPU from a seed, ``run`` is one pass, in elementary
torch operations (``own`` false) or through the package's entry points (``own`` true), ``exact`` is the definition in
64 bits, ``work`` the bytes and operations a pass cannot do without.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
IDS = {"i32": torch.int32, "i64": torch.int64}
BLOCK = 128  # elements that share one scale of an 8-bit matrix


# ---------------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the gradients of many adapters and norms, hundreds of small tensors of odd sizes: their norm and the clip
        # coefficient that the optimizer's step takes
        {"name": "grad_norm_many_small", "op": "grad_norm", "grad": "f32", "tensors": 400, "elements": 1500000,
         "clip": False},
        # the gradients of every compressed MLP weight of a GPT-2 L at c = 4, clipped in place
        {"name": "grad_clip_large", "op": "grad_norm", "grad": "bf16", "tensors": 72, "elements": 118000000,
         "clip": True},
        # one decode step of 64 requests, at the width of Llama-3-8B: latency
        {"name": "embedding_forward_decode", "op": "embedding_forward", "table": "bf16", "out": "bf16", "ids": "i64",
         "V": 128000, "K": 4096, "M": 64},
        # a large prefill or training batch
        {"name": "embedding_forward_large", "op": "embedding_forward", "table": "bf16", "out": "bf16", "ids": "i32",
         "V": 128000, "K": 4096, "M": 16384},
        # a small table of odd width in float32, one short odd batch
        {"name": "embedding_backward_odd", "op": "embedding_backward", "dy": "f32", "dE": "f32", "ids": "i64",
         "V": 2003, "K": 1283, "M": 333, "add": False},
        # finetuning at the width of GPT-2 L: 8192 tokens, some of them very frequent
        {"name": "embedding_backward_large", "op": "embedding_backward", "dy": "bf16", "dE": "bf16", "ids": "i32",
         "V": 50000, "K": 1280, "M": 8192, "add": False},
        # the activations of an odd batch and width in float32, for the product and for the weight's gradient
        {"name": "quantize_rows_odd", "op": "quantize", "x": "f32", "R": 1111, "C": 1283, "tile": False, "q": True,
         "qt": True},
        # a Llama-3-8B gate/up weight after an optimizer step, for the forward and the input's gradient
        {"name": "quantize_tiles_large", "op": "quantize", "x": "bf16", "R": 14336, "C": 4096, "tile": True, "q": True,
         "qt": True},
        # one decoded token on the same layer
        {"name": "dense_forward_one", "op": "dense_forward", "x": "bf16", "M": 1, "K": 4096, "N": 14336, "tile": True,
         "save": False},
        # a prefill step on it
        {"name": "dense_forward_prefill", "op": "dense_forward", "x": "bf16", "M": 4096, "K": 4096, "N": 14336,
         "tile": True, "save": False},
        # gradients of a small float32 layer, an odd batch
        {"name": "dense_backward_odd", "op": "dense_backward", "dy": "f32", "dW": "f32", "M": 333, "K": 500, "N": 768,
         "tile": False},
        # finetuning a dense layer of GPT-2 L's up-projection shape
        {"name": "dense_backward_finetune", "op": "dense_backward", "dy": "bf16", "dW": "f32", "M": 8192, "K": 1280,
         "N": 5120, "tile": True},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: most are multiples of 64, some of 8, some odd."""
    n, kind = _log(rng, lo, hi), rng.random()
    return n if kind < 0.2 else max(8, n // 8 * 8) if kind < 0.5 else max(64, n // 64 * 64)


def draw(rng):
    op = rng.choice(["grad_norm", "embedding_forward", "embedding_backward", "quantize", "dense_forward",
                     "dense_forward", "dense_backward"])
    if op == "grad_norm":
        tensors, clip = _log(rng, 1, 600), rng.random() < 0.5
        return {"op": op, "grad": rng.choice(["f32", "bf16", "mixed"]), "tensors": tensors,
                "elements": _log(rng, 4000000 if clip else max(2000, 4 * tensors), 59000000), "clip": clip}
    if op == "embedding_forward":
        while True:
            table = rng.choice(["bf16", "bf16", "f32"])
            case = {"op": op, "table": table, "out": rng.choice([table, table, "bf16", "f32"]),
                    "ids": rng.choice(["i32", "i64"]), "V": _log(rng, 200, 128000), "K": _width(rng, 32, 8192),
                    "M": _log(rng, 1, 16384)}
            if case["M"] * case["K"] <= 16384 * 2048 and case["V"] * case["K"] <= 128000 * 4096:
                return case
    if op == "embedding_backward":
        while True:
            dy = rng.choice(["bf16", "bf16", "f32"])
            case = {"op": op, "dy": dy, "dE": rng.choice([dy, "f32"]), "ids": rng.choice(["i32", "i64"]),
                    "V": _log(rng, 200, 128000), "K": _width(rng, 32, 4096), "M": _log(rng, 1, 16384),
                    "add": rng.random() < 0.3}
            if case["M"] * case["K"] <= 8192 * 1280 and case["V"] * case["K"] <= 50000 * 640:
                return case
    if op == "quantize":
        while True:
            q = rng.random() < 0.75
            case = {"op": op, "x": rng.choice(["bf16", "bf16", "f32"]), "R": _log(rng, 1, 16384),
                    "C": _width(rng, 64, 14336), "tile": rng.random() < 0.4, "q": q,
                    "qt": not q or rng.random() < 0.5}
            if case["R"] * case["C"] * (2 if case["x"] == "f32" else 1) <= 14336 * 4096:
                return case
    if op == "dense_forward":
        while True:
            case = {"op": op, "x": rng.choice(["bf16", "bf16", "bf16", "f32"]), "M": _log(rng, 1, 8192),
                    "K": _width(rng, 64, 14336), "N": _width(rng, 64, 14336), "tile": rng.random() < 0.7,
                    "save": rng.random() < 0.3}
            if case["M"] * case["K"] * case["N"] <= 4096 * 4096 * 8192 and case["K"] * case["N"] <= 4096 * 14336:
                return case
    while True:
        dy = rng.choice(["bf16", "bf16", "f32"])
        case = {"op": op, "dy": dy, "dW": rng.choice(["f32", "f32", dy]), "M": _log(rng, 1, 8192),
                "K": _width(rng, 64, 8192), "N": _width(rng, 64, 8192), "tile": rng.random() < 0.7}
        if case["M"] * case["K"] * case["N"] <= 8192 * 1280 * 5120 and case["K"] * case["N"] <= 4096 * 4096:
            return case


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


def _sizes(case):
    """Element counts of the tensors, a function of the case alone: spread over a factor of about 50, odd ones among
    them."""
    T, total = case["tensors"], case["elements"]
    w = torch.exp(torch.rand(T, generator=_host(T * 7 + 1), dtype=torch.float64) * 4.0)
    n = (w / w.sum() * total).floor().long().clamp(min=1)
    return n.tolist()


def _prepare_grad_norm(case, seed):
    """Gradients as a backward pass leaves them: the tensors, views of a flat buffer for each type, each starting at a
    multiple of 256 elements, differ in size and in scale."""
    g = _gen(seed)
    sizes = _sizes(case)
    std = (0.001 * 2.0 ** (4 * torch.rand(len(sizes), generator=_host(seed + 5)))).tolist()
    kinds = ["bf16", "f32"] if case["grad"] == "mixed" else [case["grad"]]
    flats, grads = [], []
    for i, kind in enumerate(kinds):
        mine = list(zip(sizes, std))[i::len(kinds)]
        flats.append(torch.zeros((sum(n + -n % 256 for n, _ in mine),), dtype=DTYPES[kind], device="cuda"))
        at = 0
        for n, a in mine:
            grads.append(flats[-1][at:at + n])
            grads[-1].copy_(_normal(g, (n,), torch.float32, a))
            at += n + -n % 256
    # half of the norm that these gradients have on average: every pass clips
    s = {"flats": flats, "clip": case["clip"],
         "max_norm": 0.5 * math.sqrt(sum(n * a * a for n, a in zip(sizes, std)))}
    if own:
        import sketched_parameter_sharing_amd as ss1
        s["plan"] = ss1.GradNormPlan.make(grads)
    return s


def _token_ids(case, seed):
    """Token numbers as text has them: number i about 1 / (i + 1) as often as number 0, and one in 64 is padding (-1)."""
    g = _gen(seed + 29)
    V, M = case["V"], case["M"]
    u = torch.rand((M,), generator=g, device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(V + 1)) - 1).floor().long().clamp(0, V - 1)
    ids[torch.rand((M,), generator=g, device="cuda") < 1 / 64] = -1
    return ids.to(IDS[case["ids"]])


def _prepare_embedding(case, seed):
    g = _gen(seed)
    V, K, M = case["V"], case["K"], case["M"]
    s = {"ids": _token_ids(case, seed), "scale": math.sqrt(K)}
    if case["op"] == "embedding_forward":
        s["table"] = _normal(g, (V, K), DTYPES[case["table"]], 0.02)
        s["out"] = DTYPES[case["out"]]
    else:
        s["dy"] = _normal(g, (M, K), DTYPES[case["dy"]], 0.01)
        s["V"], s["dE_dtype"] = V, DTYPES[case["dE"]]
        # with "add" the table's gradient holds the share of an output layer tied to it, and the lookup's is added
        s["dE"] = _normal(g, (V, K), s["dE_dtype"], 0.01) if case["add"] else None
    return s


def _activations(g, shape, dtype, std=1.0):
    """Rows of unequal size, and a few columns that are much larger than the rest."""
    x = _normal(g, shape, torch.float32, std) * torch.exp(_normal(g, (shape[0], 1), torch.float32, 0.5))
    return (x * torch.where(torch.rand((1, shape[1]), generator=g, device="cuda") < 0.01, 20.0, 1.0)).to(dtype)


def _blocks(pair, cols, tile):
    """The package's form of codes and scales."""
    import sketched_parameter_sharing_amd as ss1
    return ss1.Fp8Blocks(pair[0], pair[1], BLOCK if tile else 1, cols)


def _prepare_dense(case, seed):
    g = _gen(seed)
    M, K, N, tile = case["M"], case["K"], case["N"], case["tile"]
    W = _normal(g, (N, K), torch.float32, 0.02)
    s = {"K": K, "N": N, "M": M, "tile": tile}
    if case["op"] == "dense_forward":
        s["x"], s["save"] = _activations(g, (M, K), DTYPES[case["x"]]), case["save"]
        s["w"] = _quantize(W, tile)
        if own:
            s["w_own"] = _blocks(s["w"], K, tile)
        return s
    # what a training step kept from its forward pass: the codes of x and of W along the other side
    s["dy"], s["dW_dtype"] = _activations(g, (M, N), DTYPES[case["dy"]], 0.01), DTYPES[case["dW"]]
    s["xt"], s["wt"] = _quantize(_activations(g, (M, K), DTYPES[case["dy"]]).t(), False), _quantize(W.t(), tile)
    if own:
        s["xt_own"], s["wt_own"] = _blocks(s["xt"], M, False), _blocks(s["wt"], N, tile)
    return s


def prepare(case, seed):
    op = case["op"]
    if op == "grad_norm":
        s = _prepare_grad_norm(case, seed)
    elif op.startswith("embedding"):
        s = _prepare_embedding(case, seed)
    elif op == "quantize":
        s = {"x": _activations(_gen(seed), (case["R"], case["C"]), DTYPES[case["x"]]), "tile": case["tile"],
             "q": case["q"], "qt": case["qt"]}
    else:
        s = _prepare_dense(case, seed)
    return dict(s, op=op)


# ---------------------------------------------------------------------------------------------------------- plain forms
def _plain_grad_norm(s):
    total = torch.stack([t.float().square().sum(dtype=torch.float64) for t in s["flats"]]).sum()
    norm = total.sqrt()
    coef = torch.where(norm > s["max_norm"], s["max_norm"] / norm, torch.ones_like(norm)).float().reshape(1)
    if s["clip"]:
        [t.copy_(t.float() * coef) for t in s["flats"]]
    return norm.float().reshape(1), coef


def _grad_norm_outputs(s, norm, coef):
    """norm and coefficient, and the gradients where they were clipped; the next pass over the same gradients has a bound
    just below this one's, so that it clips too."""
    s["max_norm"] *= 0.9999
    return (norm, coef, *s["flats"]) if s["clip"] else (norm, coef)


def _plain_embedding_forward(s):
    ids = s["ids"].long()
    real = (ids >= 0) & (ids < s["table"].shape[0])
    rows = s["table"][ids.clamp(min=0)].float() * s["scale"]
    return torch.where(real[:, None], rows, torch.zeros_like(rows)).to(s["out"])


def _plain_embedding_backward(s):
    ids = s["ids"].long()
    real = (ids >= 0) & (ids < s["V"])
    dy = torch.where(real[:, None], s["dy"].float() * s["scale"], 0.0)
    total = torch.zeros((s["V"], dy.shape[1]), device="cuda").index_add_(0, ids.clamp(min=0), dy)
    if s["dE"] is None:
        return total.to(s["dE_dtype"])
    return s["dE"].copy_(s["dE"].float() + total)


def _exponent(top):
    """Exponent of the smallest power of two s with top / s <= 448, the largest E4M3 value; 0 for a block of zeros."""
    m, e = torch.frexp(top)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-126, 127)
    return torch.where(top > 0, e, torch.zeros_like(e))


def _two_to(e):
    """2^e in float32, made of its bits (exp2 need not be exact)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantize(x, tile):
    """x [R][C] as E4M3 codes [R][C up to a multiple of 128] and scale bytes (power of two + 127), one for 128 elements
    of a row or, with ``tile``, for a tile of 128 x 128; rows of scale bytes are as long as a multiple of 4."""
    R, C = x.shape
    nb, rb = -(-C // BLOCK), -(-R // BLOCK)
    xf = torch.zeros((rb * BLOCK if tile else R, nb * BLOCK), device=x.device)
    xf[:R, :C] = x
    a = xf.abs()
    a = torch.where(torch.isfinite(a), a, 0.0)
    if tile:
        e = _exponent(a.view(rb, BLOCK, nb, BLOCK).amax((1, 3)))
        inv = _two_to(-e).repeat_interleave(BLOCK, 0)[:R]
    else:
        e = _exponent(a.view(R, nb, BLOCK).amax(2))
        inv = _two_to(-e)
    codes = (xf[:R].view(R, nb, BLOCK) * inv[:, :, None]).view(R, nb * BLOCK).to(torch.float8_e4m3fn)
    scale = torch.full((e.shape[0], -(-nb // 4) * 4), 127, dtype=torch.uint8, device=x.device)
    scale[:, :nb] = (e + 127).to(torch.uint8)
    return codes, scale


def _values(pair, tile):
    """The float32 matrix that codes and scales stand for, padding columns included."""
    codes, scale = pair
    R, C = codes.shape
    s = _two_to(scale[:, :C // BLOCK].to(torch.int32) - 127)
    if tile:
        s = s.repeat_interleave(BLOCK, 0)[:R]
    return (codes.float().view(R, C // BLOCK, BLOCK) * s[:, :, None]).view(R, C)


def _plain_quantize(s):
    out = _quantize(s["x"], s["tile"]) if s["q"] else ()
    return out + (_quantize(s["x"].t(), s["tile"]) if s["qt"] else ())


def _plain_dense_forward(s):
    x = s["x"]
    y = (_values(_quantize(x, False), False) @ _values(s["w"], s["tile"]).t()).to(x.dtype)
    return (y, *_quantize(x.t(), False)) if s["save"] else y


def _plain_dense_backward(s):
    dy = s["dy"]
    dx = (_values(_quantize(dy, False), False) @ _values(s["wt"], s["tile"]).t()).to(dy.dtype)
    dW = (_values(_quantize(dy.t(), False), False) @ _values(s["xt"], False).t()).to(s["dW_dtype"])
    return dx, dW


# ------------------------------------------------------------------------------------------- through the entry points
def _own(s):
    import sketched_parameter_sharing_amd as ss1
    op = s["op"]
    if op == "grad_norm":
        return s["plan"].clip(s["max_norm"]) if s["clip"] else s["plan"].norm(s["max_norm"])
    if op == "embedding_forward":
        return ss1.embedding_forward(s["ids"], s["table"], scale=s["scale"], dtype=s["out"])
    if op == "embedding_backward":
        return ss1.embedding_backward(s["dy"], s["ids"], s["V"], scale=s["scale"], dE=s["dE"], dtype=s["dE_dtype"],
                                      accumulate=s["dE"] is not None)
    if op == "quantize":
        q, qt = ss1.quantize_fp8_blocks(s["x"], tile=s["tile"], q=s["q"] or None, qt=s["qt"] or None)
        return sum(((b.codes, b.scale) for b in (q, qt) if b is not None), ())
    if op == "dense_forward":
        y, xt = ss1.dense_forward_fp8(s["x"], s["w_own"], save_xt=s["save"])
        return (y, xt.codes, xt.scale) if s["save"] else y
    return ss1.dense_backward_fp8(s["dy"], s["xt_own"], s["wt_own"], dW_dtype=s["dW_dtype"])


def run(state):
    if own:
        out = _own(state)
    else:
        out = {"grad_norm": _plain_grad_norm, "embedding_forward": _plain_embedding_forward,
               "embedding_backward": _plain_embedding_backward, "quantize": _plain_quantize,
               "dense_forward": _plain_dense_forward, "dense_backward": _plain_dense_backward}[state["op"]](state)
    return _grad_norm_outputs(state, *out) if state["op"] == "grad_norm" else out


# ------------------------------------------------------------------------------------------------------------ in 64 bits
def _inputs_only(case, seed):
    """prepare()'s inputs; nothing of the package is wanted here."""
    global own
    was, own = own, False
    try:
        return prepare(case, seed)
    finally:
        own = was


def _two_to_64(e):
    return torch.ldexp(torch.ones((), dtype=torch.float64), torch.arange(-1022, 1024)).to(e.device)[e.long() + 1022]


def _exact_scales(x):
    """x [R][B][128] (or tiles [R][B][128*128]): the largest power-of-two divisor's exponent, from logarithms."""
    top = x.abs().amax(2)
    e = torch.ceil(torch.log2(top / 448.0)).clamp(min=-1000.0)
    # a logarithm next to a whole number may fall on either side of it
    e = torch.where(448.0 * _two_to_64(e - 1) >= top, e - 1, e)
    e = torch.where(448.0 * _two_to_64(e) < top, e + 1, e)
    return torch.where(top > 0, e.clamp(min=-126.0), torch.zeros_like(e))


def _exact_codes(x, tile):
    """(values of the codes, scale exponents, quantised values) of x in 64 bits: nearest multiple of the E4M3 step at each
    value, ties to even."""
    R, C = x.shape
    padded = torch.nn.functional.pad(x.double(), (0, -C % BLOCK))
    nb = padded.shape[1] // BLOCK
    if tile:
        t = torch.nn.functional.pad(padded, (0, 0, 0, -R % BLOCK)).view(-1, BLOCK, nb, BLOCK).transpose(1, 2)
        e = _exact_scales(t.reshape(t.shape[0], nb, BLOCK * BLOCK))
        by_row = e[torch.arange(R, device=x.device) // BLOCK]
    else:
        e = by_row = _exact_scales(padded.view(R, nb, BLOCK))
    by_row = by_row.repeat_interleave(BLOCK, 1)
    q = padded * _two_to_64(-by_row)
    step = _two_to_64(torch.frexp(q.abs().clamp(min=2.0 ** -6)).exponent - 4)
    q = torch.round(q / step) * step
    return q, e, q * _two_to_64(by_row)


def _exact_pair(x, tile):
    q, e, _ = _exact_codes(x, tile)
    scale = torch.full((e.shape[0], -(-e.shape[1] // 4) * 4), 127, dtype=torch.uint8, device=x.device)
    scale[:, :e.shape[1]] = (e + 127).to(torch.uint8)
    return q, scale


def _decoded(pair, tile):
    """Codes and scale bytes as 64-bit values."""
    v = pair[0].double()
    s = _two_to_64(pair[1].long() - 127).repeat_interleave(BLOCK, 1)[:, :v.shape[1]]
    return v * (s.repeat_interleave(BLOCK, 0)[:v.shape[0]] if tile else s)


def exact(case, seed):
    s = _inputs_only(case, seed)
    op = case["op"]
    if op == "grad_norm":
        norm = torch.linalg.vector_norm(torch.stack([torch.linalg.vector_norm(t.double()) for t in s["flats"]]))
        coef = (s["max_norm"] / norm).clamp(max=1.0)
        out = (norm.reshape(1), coef.reshape(1))
        return (*out, *(t.double() * coef for t in s["flats"])) if s["clip"] else out
    if op == "embedding_forward":
        y = torch.zeros((case["M"], case["K"]), dtype=torch.float64, device="cuda")
        at = torch.nonzero(s["ids"] >= 0)[:, 0]
        y[at] = s["table"][s["ids"][at].long()].double() * s["scale"]
        return y
    if op == "embedding_backward":
        dE = torch.zeros((case["V"], case["K"]), dtype=torch.float64, device="cuda") if s["dE"] is None \
            else s["dE"].double()
        at = torch.nonzero(s["ids"] >= 0)[:, 0]
        return dE.index_put_((s["ids"][at].long(),), s["dy"][at].double() * s["scale"], accumulate=True)
    if op == "quantize":
        return sum((_exact_pair(x, s["tile"]) for x, want in ((s["x"], s["q"]), (s["x"].t(), s["qt"])) if want), ())
    if op == "dense_forward":
        y = _exact_codes(s["x"], False)[2] @ _decoded(s["w"], s["tile"]).t()
        return (y, *_exact_pair(s["x"].t(), False)) if s["save"] else y
    return (_exact_codes(s["dy"], False)[2] @ _decoded(s["wt"], s["tile"]).t(),
            _exact_codes(s["dy"].t(), False)[2] @ _decoded(s["xt"], False).t())


# ------------------------------------------------------------------------------------------------------------------ work
def _codes_bytes(R, C, tile):
    """Codes and scales of an [R][C] matrix."""
    nb = -(-C // BLOCK)
    return R * nb * BLOCK + (-(-R // BLOCK) if tile else R) * nb


def work(case):
    op, size, many = case["op"], {"bf16": 2, "f32": 4}, {"i32": 4, "i64": 8}
    if op == "grad_norm":
        n = sum(_sizes(case))
        per = 3 if case["grad"] == "mixed" else size[case["grad"]]
        return {"bytes": n * per * (2 if case["clip"] else 1), "flops": n * (3 if case["clip"] else 2)}
    if op == "embedding_forward":
        M, K = case["M"], case["K"]
        # token numbers of frequency 1 / (i + 1): how many different rows M of them name
        rows = min(M, _different(case["V"], M))
        return {"bytes": M * many[case["ids"]] + rows * K * size[case["table"]] + M * K * size[case["out"]],
                "flops": M * K}
    if op == "embedding_backward":
        M, K, V = case["M"], case["K"], case["V"]
        rows = 2 * _different(V, M) if case["add"] else V
        return {"bytes": M * many[case["ids"]] + M * K * size[case["dy"]] + rows * K * size[case["dE"]],
                "flops": 2 * M * K}
    if op == "quantize":
        R, C = case["R"], case["C"]
        out = (_codes_bytes(R, C, case["tile"]) if case["q"] else 0) + (_codes_bytes(C, R, case["tile"])
                                                                       if case["qt"] else 0)
        return {"bytes": R * C * size[case["x"]] + out, "flops": 3 * R * C}
    M, K, N = case["M"], case["K"], case["N"]
    if op == "dense_forward":
        e = size[case["x"]]
        return {"bytes": M * (K + N) * e + _codes_bytes(N, K, case["tile"])
                + (_codes_bytes(K, M, False) if case["save"] else 0), "flops": 2 * M * K * N}
    e = size[case["dy"]]
    return {"bytes": M * (N + K) * e + _codes_bytes(K, M, False) + _codes_bytes(K, N, case["tile"])
            + N * K * size[case["dW"]], "flops": 4 * M * K * N}


def _different(V, M):
    """Expected number of different tokens among M of frequency log((i + 2) / (i + 1)) / log(V + 1)."""
    i = torch.arange(V, dtype=torch.float64)
    p = torch.log((i + 2) / (i + 1)) / math.log(V + 1)
    return int((1 - (1 - p * 63 / 64) ** M).sum().item())
