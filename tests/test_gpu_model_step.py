"""The operators in a training step of a small model, as they would be used: token
embedding, layer norm, a projected SS1 layer, a layer that stays dense in 8 bits,
their gradients, the global norm and the clipped AdamW step; then the same step
captured and replayed.

Every stage's outputs are checked against its definition in 64 bits on the
tensors that the stage was given, so that a stage's tolerance is its own
roundings (stated at the stage)."""
import math

import pytest
import torch

import sketched_parameter_sharing_amd as ss1

pytestmark = pytest.mark.gpu
F, H = torch.float32, torch.bfloat16
V, K, N, O, M = 900, 256, 384, 320, 700
SCALE = math.sqrt(K)


def value(b):
    two = torch.tensor([math.ldexp(1.0, k - 127) for k in range(256)], dtype=torch.float64, device="cuda")
    v = b.codes.double()
    s = two[b.scale.long()].repeat_interleave(b.block, 0)[:v.shape[0]].repeat_interleave(128, 1)[:, :v.shape[1]]
    return (v * s)[:, :b.cols]


class Model:
    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.plan = ss1.DevicePlan.make(seed, K, N, 2, 32, 32)
        self.E, self.gamma, self.beta = (0.05 * randn(V, K)).to(H), 1 + 0.1 * randn(K), 0.1 * randn(K)
        self.W_c, self.W = (0.06 * randn(N, K // 2)).to(H), (0.05 * randn(O, N)).to(H)
        self.params = [self.E, self.gamma, self.beta, self.W_c, self.W]
        self.grads = [torch.empty_like(p) for p in self.params]
        self.grads[-1] = torch.empty((O, N), device="cuda")  # the dense weight's gradient in float32
        self.opt = ss1.AdamWPlan.make(self.params, self.grads, masters=[p.float() if p.dtype == H else None
                                                                        for p in self.params])
        self.norm = ss1.GradNormPlan.make(self.grads)

    def step(self, ids, dy, number):
        """One step for the loss <dy, y>; returns every intermediate."""
        dE, dgamma, dbeta, dW_c, dW = self.grads
        w, wt = ss1.quantize_fp8_blocks(self.W, tile=True, qt=True)
        h = ss1.embedding_forward(ids, self.E, scale=SCALE)
        n, mean, rstd = ss1.layernorm_forward(h, self.gamma, self.beta)
        u = self.plan.forward(n, self.W_c)
        y, xt = ss1.dense_forward_fp8(u, w, save_xt=True)
        du, _ = ss1.dense_backward_fp8(dy, xt, wt, dW=dW)
        dn, _ = ss1.backward(n, self.W_c, self.plan.hash, self.plan.sign, 2, 32, 32, du, dW_c=dW_c)
        dh, _, _ = ss1.layernorm_backward(dn, h, self.gamma, mean, rstd, dgamma=dgamma, dbeta=dbeta)
        ss1.embedding_backward(dh, ids, V, scale=SCALE, dE=dE)
        norm, coef = self.norm.norm(0.5)
        self.opt.step(step=number, lr=1e-2, grad_scale=coef)
        return dict(w=w, wt=wt, h=h, n=n, u=u, y=y, xt=xt, du=du, dn=dn, dh=dh, norm=norm, coef=coef)


def batch(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    ids = torch.randint(-1, V, (M,), generator=g, device="cuda")
    ids[::7] = 5  # a frequent token
    return ids, (0.01 * torch.randn((M, O), generator=g, device="cuda")).to(H)


def within(x, want, slack):
    off = (x.double() - want).abs()
    assert (off <= slack).all(), (off / slack).max().item()


def test_every_stage_of_a_step():
    m = Model(3)
    ids, dy = batch(4)
    before = [p.clone() for p in m.params]
    t = m.step(ids, dy, 1)
    dE, _, _, _, dW = m.grads
    real = ids >= 0
    # embedding: a float32 product, bf16 (2^-24 + 2^-8 of the value)
    want = torch.zeros((M, K), dtype=torch.float64, device="cuda")
    want[real] = before[0].double()[ids[real]] * float(torch.tensor(SCALE, dtype=F))
    within(t["h"], want, (2.0 ** -24 + 2.0 ** -8) * want.abs() + 2.0 ** -126)
    # dense layer: its codes' product; 2^-10 of the largest product of each block of 128, float32 sums, bf16
    q, qt = ss1.quantize_fp8_blocks(t["u"], qt=True)
    assert torch.equal(qt.codes.view(torch.uint8), t["xt"].codes.view(torch.uint8))

    def product(x, a, b, bf16):
        want, size = a @ b.t(), a.abs() @ b.abs().t()
        slack = a.shape[1] * 2.0 ** -23 * size + 2.0 ** -126
        if bf16:
            for k in range(0, a.shape[1], 128):
                slack += 2.0 ** -10 * a[:, k:k + 128].abs().amax(1)[:, None] * b[:, k:k + 128].abs().amax(1)[None]
            slack += 2.0 ** -8 * (want.abs() + slack)
        within(x, want, slack)

    product(t["y"], value(q), value(t["w"]), True)
    dq, dqt = ss1.quantize_fp8_blocks(dy, qt=True)
    product(t["du"], value(dq), value(t["wt"]), True)
    product(dW, value(dqt), value(t["xt"]), False)
    # the codes themselves: within half a step of what was quantised, 2^-4 of the value or 2^-10 of the scale's unit
    for b, x in ((q, t["u"]), (dq, dy), (t["w"], before[4])):
        unit = torch.exp2(b.scale.double() - 127).repeat_interleave(b.block, 0)[:x.shape[0]]
        unit = unit.repeat_interleave(128, 1)[:, :x.shape[1]]
        within(value(b), x.double(), torch.maximum(2.0 ** -4 * x.double().abs(), 2.0 ** -10 * unit))
    # embedding's gradient: float32 sums over a token's rows, bf16
    rows, shares = ids[real].cpu(), t["dh"].double()[real].cpu()
    want = torch.zeros((V, K), dtype=torch.float64).index_add_(0, rows, shares).cuda() * SCALE
    size = torch.zeros((V, K), dtype=torch.float64).index_add_(0, rows, shares.abs()).cuda() * SCALE
    n = torch.bincount(rows, minlength=V).cuda()[:, None]
    slack = 2.0 ** -24 * (n + 2) * size
    within(dE, want, slack + 2.0 ** -8 * (want.abs() + slack) + 2.0 ** -126)
    # norm and coefficient: one rounding to float32
    want = math.sqrt(sum(g.double().square().sum().item() for g in m.grads))
    assert abs(t["norm"].item() - want) <= 2.0 ** -24 * 1.001 * want
    c = min(1.0, 0.5 / want)
    assert abs(t["coef"].item() - c) <= 2.0 ** -24 * 1.001 * c and c < 1.0
    # the step took the clipped gradients: its first moment is 0.1 of them (float32: two products, 2^-23)
    for g, s in zip(m.grads, m.opt.m):
        want = 0.1 * g.double() * t["coef"].double()
        within(s, want, 2.0 ** -22 * want.abs() + 2.0 ** -149)
    assert all((p != b).any() for p, b in zip(m.params, before))


def test_a_captured_step_replays():
    eager, other = Model(3), Model(3)
    ids, dy = batch(4)
    one_ids, one_dy = ids.clone(), dy.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        Model(5).step(one_ids, one_dy, 1)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = other.step(one_ids, one_dy, 1)
    for k in range(4):  # the optimizer's step number stays the captured one
        ids, dy = batch(10 + k)
        one_ids.copy_(ids)
        one_dy.copy_(dy)
        graph.replay()
        want = eager.step(ids, dy, 1)
        torch.cuda.synchronize()
        for name in ("h", "u", "y", "du", "dh", "norm", "coef"):
            assert torch.equal(out[name], want[name]), (k, name)
        assert all(torch.equal(a, b) for a, b in zip(eager.params, other.params))
        assert all(torch.equal(a, b) for a, b in zip(eager.grads, other.grads))


@pytest.mark.parametrize("name", ["norm", "clip", "embedding_forward", "embedding_backward", "quantize", "matmul",
                                  "dense_forward", "dense_backward"])
def test_a_given_stream_owns_what_the_call_allocates(name, monkeypatch):
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn((300, 256), generator=g, device="cuda")
    ids = torch.randint(0, 40, (1500,), generator=g, device="cuda")
    dy = torch.randn((1500, 64), generator=g, device="cuda")
    plan = ss1.GradNormPlan.make([x.clone()])
    a, at = ss1.quantize_fp8_blocks(x, qt=True)
    b, bt = ss1.quantize_fp8_blocks(torch.randn((100, 256), generator=g, device="cuda"), tile=True, qt=True)
    up = torch.randn((300, 100), generator=g, device="cuda")
    call = {"norm": lambda s: plan.norm(0.1, stream=s), "clip": lambda s: plan.clip(1e9, stream=s),
            "embedding_forward": lambda s: (ss1.embedding_forward(ids, x, stream=s),),
            "embedding_backward": lambda s: (ss1.embedding_backward(dy, ids, 40, stream=s),),
            "quantize": lambda s: [t for q in ss1.quantize_fp8_blocks(x, qt=True, stream=s) for t in
                                   (q.codes.view(torch.uint8), q.scale)],
            "matmul": lambda s: (ss1.matmul_fp8_blocks(a, b, stream=s),),
            "dense_forward": lambda s: (ss1.dense_forward_fp8(x, b, stream=s)[0],),
            "dense_backward": lambda s: ss1.dense_backward_fp8(up, at, bt, stream=s)}[name]
    want = call(None)
    torch.cuda.synchronize()
    side, made, real = torch.cuda.Stream(), [], torch.empty_strided

    def wrapped(*args, **kwargs):
        made.append(real(*args, **kwargs))
        return made[-1]

    monkeypatch.setattr(torch, "empty_strided", wrapped)
    got = call(side)
    monkeypatch.undo()
    side.synchronize()
    assert made
    for t in made:
        at_ = t.data_ptr()
        home = [s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= at_ < s["address"] + s["total_size"]]
        assert home == [side.cuda_stream]
    assert all(torch.equal(p, q) for p, q in zip(got, want))
