"""Training steps of a small mixture of experts behind an adapted projection.

Sequences of several tenants share one frozen input projection, each tenant
with a low-rank adapter of its own; a router then sends every token to one of
several experts. All matrix products run on the library's segmented products:

    h = x W_in + s (x A_t) B_t          lora_matmul      t: the token's tenant
    y = silu(h)[by expert] E_e           grouped_matmul   e: the token's expert

and the backward pass of both (grouped_matmul with transb, grouped_wgrad,
lora_backward). Prints the loss of every step; the adapters and the experts
learn to imitate a random teacher.

    python examples/expert_adapters.py [--dtype bf16] [--steps 30]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp32_gemm_major_gb300 as gemm  # noqa: E402


def offsets_of(keys, count):
    """Where each key's rows start, for keys sorted in ascending order."""
    return torch.searchsorted(keys, torch.arange(count + 1, device=keys.device))


def by_expert(h, router, experts):
    """Tokens sorted by their expert: the order, and the experts' offsets. Stays
    on the device: the products read the offsets there."""
    choice, order = (h.float() @ router).argmax(1).sort(stable=True)
    return order, offsets_of(choice, experts)


class Layer:
    def __init__(self, width, hidden, rank, tenants, experts, dtype, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

        self.w = normal(width, hidden, scale=width ** -0.5)
        self.a = normal(tenants, width, rank, scale=width ** -0.5)
        self.b = normal(tenants, rank, hidden, scale=rank ** -0.5)
        self.e = normal(experts, hidden, width, scale=hidden ** -0.5)
        self.router = torch.randn(hidden, experts, generator=gen, device="cuda")
        self.scales = torch.full((tenants,), 0.5, device="cuda")

    def forward(self, x, tenants):
        u = torch.empty(x.shape[0], self.a.shape[2], dtype=x.dtype, device=x.device)
        h = gemm.lora_matmul(x, self.w, self.a, self.b, tenants, scales=self.scales, shrink_out=u)
        order, experts = by_expert(h, self.router, self.e.shape[0])
        z = h[order]
        act = torch.nn.functional.silu(z)
        y = torch.empty_like(x)
        y[order] = gemm.grouped_matmul(act, self.e, experts)
        return y, (x, tenants, u, order, experts, z, act)

    def backward(self, dy, saved):
        """Gradients of the adapters and the experts (the router is fixed)."""
        x, tenants, u, order, experts, z, act = saved
        dy = dy[order]
        de = gemm.grouped_wgrad(act, dy, experts)
        dact = gemm.grouped_matmul(dy, self.e, experts, transb=True)
        sig = torch.sigmoid(z.float())
        dh = torch.empty_like(dact)
        dh[order] = (dact.float() * sig * (1 + z.float() * (1 - sig))).to(dact.dtype)
        _, da, db = gemm.lora_backward(dh, x, u, self.w, self.a, self.b, tenants, self.scales)
        return da, db, de


def train(dtype=torch.float32, steps=30, tokens=2048, width=512, hidden=1024, rank=16, tenants=4,
          experts=8, rate=0.05):
    teacher = Layer(width, hidden, rank, tenants, experts, dtype, seed=1)
    layer = Layer(width, hidden, rank, tenants, experts, dtype, seed=2)
    layer.w, layer.router = teacher.w, teacher.router
    master = [t.float() for t in (layer.a, layer.b, layer.e)]
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(tokens, width, generator=gen, device="cuda").to(dtype)
    owner = torch.randint(tenants, (tokens,), generator=gen, device="cuda").sort().values
    segments = offsets_of(owner, tenants)
    target = teacher.forward(x, segments)[0].float()
    losses = []
    for _ in range(steps):
        y, saved = layer.forward(x, segments)
        error = y.float() - target
        losses.append(error.square().mean())
        grads = layer.backward((error * (2 / tokens)).to(dtype), saved)
        for m, g in zip(master, grads):
            m.sub_(g.float(), alpha=rate)
        layer.a, layer.b, layer.e = (m.to(dtype) for m in master)
    return torch.stack(losses).tolist()


if __name__ == "__main__":
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    p.add_argument("--steps", type=int, default=30)
    args = p.parse_args()
    dt = torch.float32 if args.dtype == "f32" else torch.bfloat16
    for step, loss in enumerate(train(dt, args.steps)):
        print(f"step {step:3d}  loss {loss:.5f}")
