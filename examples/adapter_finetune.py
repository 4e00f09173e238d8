"""Finetunes low-rank adapters beside a projected SS1 layer, then serves them.

A dense layer is projected onto SS1 (``ss1.project``); what the projection lost is
learned back by low-rank adapters, one for each of several tasks, trained together
in one batch of ragged sequences:

    h = LayerNorm(x);  y = SS1(h) + adapter of the sequence(h);  loss = |y - target|^2 / 2

with ``layernorm_forward/backward``, ``forward``/``backward`` of the SS1 layer,
``adapter_forward/backward`` beside it, the global gradient norm by
``GradNormPlan.norm``, and one ``AdamWPlan.step``, clipped by it, over the norm's
parameters, the compressed weight and both factors of the adapters.  Afterwards a
decode batch of one token a request runs each request's own adapter.

    python examples/adapter_finetune.py [--steps 60] [--state fp8]
"""
import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import sketched_parameter_sharing_amd as ss1  # noqa: E402


def finetune(steps=60, K=512, N=768, c=2, tasks=3, rank=16, tokens=1536, state="f32", seed=0, report=None):
    """Returns (first loss, last loss, served): served is y of a decode batch and its reference."""
    dev, bf16 = "cuda", torch.bfloat16
    g = torch.Generator(device=dev).manual_seed(seed)
    randn = lambda *s: torch.randn(s, generator=g, device=dev)  # noqa: E731

    # the layer: a dense weight projected onto the sharing pattern
    plan = ss1.DevicePlan.make(seed + 1, K, N, c, 64, 64)
    dense = 0.04 * randn(N, K)
    W_c = ss1.project(dense, plan.hash, plan.sign, c, 64, 64).to(bf16)
    gamma, beta = torch.ones(K, device=dev), torch.zeros(K, device=dev)
    A, B = (randn(tasks * rank, K) / K ** 0.5).to(bf16), torch.zeros((tasks * rank, N), device=dev, dtype=bf16)
    adapters = ss1.AdapterSet.make(A, B, [rank] * tasks, [1.0] * tasks)

    # ragged sequences, each of one task; a task's target is the dense layer changed by a low-rank update
    lengths = torch.randint(20, 200, (32,), generator=torch.Generator().manual_seed(seed)).cumsum(0)
    ends = lengths[lengths < tokens].tolist() + [tokens]
    seg = torch.tensor([0] + ends, dtype=torch.int32, device=dev)
    task_of = torch.arange(len(ends), dtype=torch.int32, device=dev) % tasks
    x = randn(tokens, K).to(bf16)
    tok_task = torch.repeat_interleave(task_of.long(), (seg[1:] - seg[:-1]).long())
    xh = torch.nn.functional.layer_norm(x.float(), (K,))
    updates = [0.02 * randn(N, 4) @ randn(4, K) for _ in range(tasks)]
    target = xh @ dense.t()
    for t in range(tasks):
        target[tok_task == t] += xh[tok_task == t] @ updates[t].t()

    # gradients live in fixed buffers, so one plan of the optimizer serves every step
    params = [gamma, beta, W_c, A, B]
    grads = [torch.empty_like(p) for p in params]
    masters = [None, None] + [p.float() for p in params[2:]]
    opt = ss1.AdamWPlan.make(params, grads, masters=masters, weight_decay=[0.0, 0.0, 0.01, 0.0, 0.0], state=state)
    clip = ss1.GradNormPlan.make(grads)
    dgamma, dbeta, dW, dA, dB = grads
    losses = []
    for step in range(1, steps + 1):
        h, mean, rstd = ss1.layernorm_forward(x, gamma, beta)
        y = plan.forward(h, W_c)
        y, v = ss1.adapter_forward(h, adapters, seg, task_of, base=y, y=y, save_v=True)
        err = y.float() - target
        losses.append(0.5 * err.square().mean())
        dy = (err / err.shape[1]).to(bf16)
        dh, _ = ss1.backward(h, W_c, plan.hash, plan.sign, c, 64, 64, dy, dW_c=dW)
        dh, _, _ = ss1.adapter_backward(dy, h, v, adapters, seg, task_of, dx_base=dh, dx=dh, dA=dA, dB=dB)
        ss1.layernorm_backward(dh, x, gamma, mean, rstd, dx=None, dgamma=dgamma, dbeta=dbeta)
        # clip by the global norm; the coefficient stays on the device
        _, coef = clip.norm(max_norm=1.0)
        opt.step(step=step, lr=2e-3, grad_scale=coef, seed=step)
        if report and (step == 1 or step % 10 == 0):
            report(f"step {step:4d}  loss {float(losses[-1]):.5f}")

    # serving: one token a request, each with its task's adapter, and one request without any
    requests = 24
    q = randn(requests, K).to(bf16)
    who = torch.arange(requests, dtype=torch.int32, device=dev) % (tasks + 1) - 1
    one = torch.arange(requests + 1, dtype=torch.int32, device=dev)
    h, _, _ = ss1.layernorm_forward(q, gamma, beta)
    served = ss1.adapter_forward(h, adapters, one, who, base=plan.forward(h, W_c))[0]
    want = plan.forward(h, W_c).float()
    for t in range(tasks):
        rows = slice(t * rank, (t + 1) * rank)
        want[who == t] += (h[who == t].float() @ A[rows].float().t()) @ B[rows].float()
    return float(losses[0]), float(losses[-1]), (served, want)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--state", choices=("f32", "fp8"), default="f32", help="the optimizer's states")
    a = ap.parse_args()
    first, last, (served, want) = finetune(steps=a.steps, state=a.state, report=print)
    print(f"loss {first:.5f} -> {last:.5f}")
    print(f"serving: largest difference to the plain form {float((served.float() - want).abs().max()):.4f} "
          f"at values up to {float(want.abs().max()):.2f}")


if __name__ == "__main__":
    main()
