"""A block of expert MLPs trained by the bank update, on the library's operators alone.

    python -m orthogonalizing_polynomial_cascade_amd.expert_block [--steps N] [--rows R] [--experts E]

Forward, for rows sorted by expert:  h = norm(x);  y = x + relu2(h up_e^T + b_e) down_e.
The weight gradients leave the backward pass as the [experts, hidden, width] gradient stacks of two
banks, which anvil_bank_update orthogonalises and applies; the norm's weight and bias and the experts'
biases take plain gradient steps.  The command fits a fixed random block of the same shape on random
inputs.  What it minimises is the squared error summed over the columns and averaged over the rows; what
it prints is the mean over both, smaller by the width.
"""
from __future__ import annotations

import argparse

from . import anvil


class ExpertBlock:
    """Parameters, forward and backward pass of the block, and its update.

    up and down are bf16 [experts, hidden, width], each the high half of fp32 master weights whose
    low half is `mantissa` (what anvil_bank_update keeps)."""

    def __init__(self, experts, width, hidden, seed=0, lr=0.01):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)

        def stack(scale):
            return (torch.randn(experts, hidden, width, generator=g, device="cuda") * scale).to(torch.bfloat16)

        self.banks = {"up": stack(width ** -0.5), "down": stack(hidden ** -0.5)}
        self.bias = torch.zeros(experts, hidden, device="cuda")
        self.norm_weight = torch.ones(width, device="cuda")
        self.norm_bias = torch.zeros(width, device="cuda")
        self.lr = lr
        self.eff_lr = torch.full((experts,), lr, device="cuda")
        self.state = {}
        for name, w in self.banks.items():
            self.state[name] = {
                "velocity": torch.zeros(2, *w.shape, device="cuda"),
                "energy": torch.zeros(experts * anvil.equalizer_lanes(hidden, width), device="cuda"),
                "mantissa": torch.zeros(w.shape, dtype=torch.int16, device="cuda"),
            }

    def forward(self, x, offsets):
        """(y, what the backward pass needs) for bf16 rows x [rows, width] sorted by expert."""
        h, mean, rstd = anvil.anvil_layer_norm(x, self.norm_weight, self.norm_bias)
        a, z = anvil.anvil_expert_linear(h, self.banks["up"], offsets, self.bias, act="relu2", keep_preact=True)
        y, _ = anvil.anvil_expert_linear(a, self.banks["down"], offsets, residual=x, w_kn=True)
        return y, (x, offsets, h, mean, rstd, a, z)

    def backward(self, dy, kept):
        """(dx, gradients by name) from the bf16 gradient of y."""
        x, offsets, h, mean, rstd, a, z = kept
        ddown, _ = anvil.anvil_expert_grad_weight(dy, a, offsets, w_kn=True, want_bias=False)
        dz = anvil.anvil_expert_grad_input(dy, self.banks["down"], offsets, preact=z, act="relu2", w_kn=True)
        dup, dbias = anvil.anvil_expert_grad_weight(dz, h, offsets)
        dh = anvil.anvil_expert_grad_input(dz, self.banks["up"], offsets)
        dx, dweight, dnorm = anvil.anvil_layer_norm_grad(dh, x, self.norm_weight, mean, rstd)
        return dx + dy, {"up": dup, "down": ddown, "bias": dbias, "norm_weight": dweight, "norm_bias": dnorm}

    def update(self, grads, step):
        """One bank update of each stack and a gradient step of the vectors."""
        momentum, fast_beta, fast_weight = anvil.rail_scalars(step)
        for name, w in self.banks.items():
            s = self.state[name]
            anvil.anvil_bank_update(grads[name], s["velocity"], momentum, fast_beta, fast_weight, s["energy"], 0.95,
                                    w, s["mantissa"], 0.0, self.eff_lr)
        for name in ("bias", "norm_weight", "norm_bias"):
            getattr(self, name).sub_(grads[name], alpha=self.lr)


def groups(rows, experts, seed):
    """Row offsets [experts + 1] of an uneven assignment of rows to experts, on the GPU."""
    import torch
    g = torch.Generator().manual_seed(seed)
    owner = torch.multinomial(torch.rand(experts, generator=g) + 0.1, rows, replacement=True, generator=g)
    counts = torch.bincount(owner, minlength=experts)
    return torch.cat([torch.zeros(1, dtype=torch.long), counts.cumsum(0)]).to(torch.int32).cuda()


def train(steps=20, rows=4096, experts=8, width=256, hidden=768, seed=0):
    """Fits a fixed random block; returns the squared error before each step, averaged over rows and
    columns (the gradients are those of its sum over the columns, which the vectors' plain steps see)."""
    import torch
    teacher, block = ExpertBlock(experts, width, hidden, seed + 1), ExpertBlock(experts, width, hidden, seed)
    losses = []
    for step in range(steps):
        g = torch.Generator(device="cuda").manual_seed(100 + step)
        x = torch.randn(rows, width, generator=g, device="cuda").to(torch.bfloat16)
        offsets = groups(rows, experts, step)
        want, _ = teacher.forward(x, offsets)
        y, kept = block.forward(x, offsets)
        diff = y.float() - want.float()
        losses.append(diff.square().mean())
        _, grads = block.backward((diff * (2.0 / rows)).to(torch.bfloat16), kept)
        block.update(grads, step)
    return [float(v) for v in losses]


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--rows", type=int, default=4096)
    p.add_argument("--experts", type=int, default=8)
    p.add_argument("--width", type=int, default=256)
    p.add_argument("--hidden", type=int, default=768)
    a = p.parse_args()
    for step, loss in enumerate(train(a.steps, a.rows, a.experts, a.width, a.hidden)):
        print(f"step {step:3d}  mean squared error {loss:.5f}")


if __name__ == "__main__":
    main()
