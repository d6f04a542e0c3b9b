"""A small next-token model trained on the library's operators: gated feed-forward blocks whose matrices are one
bank, a linear head with cross entropy, AdamW for what is no bank.

    python -m orthogonalizing_polynomial_cascade_amd.token_model [--steps N] [--rows R] [--blocks L] [--state-bits 8|32]

Forward, for each token t of a batch:  x = embedding[t];  x += (silu(h gate^T) * (h up^T)) down  with
h = norm(x), for every block;  loss = cross entropy of norm(x) head^T against the next token.
The gate, up and down matrices [hidden, width] of all blocks are one bank: their gradients are written
straight into its [3 * blocks, hidden, width] stack, which anvil_bank_update orthogonalises and applies.
Embedding, head and the norms' weights and biases take AdamW, all in one launch, the first two with the
low halves of their fp32 masters; their gradients are clipped to a norm of 1 without leaving the device.
"""
from __future__ import annotations

import argparse

from . import anvil

CLIP = 1.0


class TokenModel:
    """Parameters, loss, gradients and updates.

    bank is bf16 [3 * blocks, hidden, width] (gate, up, down of each block), embedding and head are bf16
    [vocab, width], all of them high halves of fp32 masters; the norms' vectors are fp32 rows of `norms`
    [blocks + 1, 2, width]."""

    def __init__(self, vocab, width, hidden, blocks, seed=0, lr=0.02, adam_lr=3e-3, state_bits=32):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

        self.vocab, self.width, self.hidden, self.blocks = vocab, width, hidden, blocks
        self.bank = normal(3 * blocks, hidden, width, scale=width ** -0.5)
        self.embedding = normal(vocab, width, scale=1.0)
        self.head = normal(vocab, width, scale=width ** -0.5)
        self.norms = torch.zeros(blocks + 1, 2, width, device="cuda")
        self.norms[:, 0] = 1.0
        # what the gradients are written to, step after step
        self.grads = {"bank": torch.zeros(self.bank.shape, device="cuda"),
                      "embedding": torch.zeros(vocab, width, device="cuda"),
                      "head": torch.zeros(vocab, width, dtype=torch.bfloat16, device="cuda"),
                      "norms": torch.zeros(self.norms.shape, device="cuda")}
        stack = 3 * blocks
        self.velocity = torch.zeros(2, *self.bank.shape, device="cuda")
        self.energy = torch.zeros(stack * anvil.equalizer_lanes(hidden, width), device="cuda")
        self.mantissa = torch.zeros(self.bank.shape, dtype=torch.int16, device="cuda")
        self.eff_lr = torch.full((stack,), lr, device="cuda")
        self.adam_lr = adam_lr
        others = ("embedding", "head", "norms")
        self.low = [torch.zeros(vocab, width, dtype=torch.int16, device="cuda") for _ in range(2)]
        self.adam = anvil.AdamW([getattr(self, name) for name in others], [self.grads[name] for name in others],
                                mantissas=self.low + [None], state_bits=[state_bits, state_bits, 32], wd_mul=[1.0, 1.0, 0.0])

    def _matrices(self, stack, block):
        """(gate and up as one [2 * hidden, width], down [hidden, width]) of a block in a [3 * blocks, ...] stack."""
        three = stack[3 * block:3 * block + 3]
        return three[:2].view(2 * self.hidden, self.width), three[2]

    def loss(self, tokens, targets):
        """(loss of each token fp32 [rows], what the gradients need)."""
        x = self.embedding[tokens]
        kept = []
        for b in range(self.blocks):
            gate_up, down = self._matrices(self.bank, b)
            h, mean, rstd = anvil.anvil_layer_norm(x, self.norms[b, 0], self.norms[b, 1])
            a, z = anvil.anvil_gated_linear(h, gate_up, act="silu", keep_preact=True)
            kept.append((x, h, mean, rstd, a, z))
            x, _ = anvil.anvil_linear(a, down, residual=x, w_kn=True)
        h, mean, rstd = anvil.anvil_layer_norm(x, self.norms[-1, 0], self.norms[-1, 1])
        loss, lse = anvil.anvil_cross_entropy(h, self.head, targets)
        return loss, (tokens, targets, kept, x, h, mean, rstd, lse)

    def gradients(self, dloss, kept):
        """Writes the gradients of sum(loss * dloss) to self.grads."""
        tokens, targets, blocks, x, h, mean, rstd, lse = kept
        g = self.grads
        dh, _ = anvil.anvil_cross_entropy_grad(h, self.head, targets, lse, dloss, dw_out=g["head"])
        dx, dweight, dbias = anvil.anvil_layer_norm_grad(dh, x, self.norms[-1, 0], mean, rstd)
        g["norms"][-1, 0], g["norms"][-1, 1] = dweight, dbias
        for b in reversed(range(self.blocks)):
            x, h, mean, rstd, a, z = blocks[b]
            gate_up, down = self._matrices(self.bank, b)
            dgate_up, ddown = self._matrices(g["bank"], b)
            anvil.anvil_linear_grad_weight(dx, a, w_kn=True, out=ddown, want_bias=False)
            dz = anvil.anvil_gated_grad_input(dx, down, z, act="silu", w_kn=True)
            anvil.anvil_linear_grad_weight(dz, h, out=dgate_up, want_bias=False)
            dh = anvil.anvil_linear_grad_input(dz, gate_up)
            through, dweight, dbias = anvil.anvil_layer_norm_grad(dh, x, self.norms[b, 0], mean, rstd)
            g["norms"][b, 0], g["norms"][b, 1] = dweight, dbias
            dx = dx + through
        g["embedding"].zero_().index_add_(0, tokens, dx.float())
        return g

    def update(self, step):
        """The bank update of the blocks' matrices and the AdamW step of everything else; step counts from 0."""
        import torch
        momentum, fast_beta, fast_weight = anvil.rail_scalars(step)
        anvil.anvil_bank_update(self.grads["bank"], self.velocity, momentum, fast_beta, fast_weight, self.energy, 0.95,
                                self.bank, self.mantissa, 0.0, self.eff_lr)
        norm = torch.stack([self.grads[name].float().norm() for name in ("embedding", "head", "norms")]).norm()
        clip = torch.clamp(CLIP / (norm + 1e-6), max=1.0)
        anvil.anvil_adamw(self.adam, self.adam_lr, step + 1, weight_decay=0.01, grad_scale=clip)


def sequence(rows, vocab, seed):
    """Tokens of a fixed random chain, on the GPU: each has four likely successors, the same for every seed."""
    import torch
    g = torch.Generator().manual_seed(1234)
    after = torch.randint(0, vocab, (vocab, 4), generator=g)
    g = torch.Generator().manual_seed(seed)
    choice = torch.randint(0, 4, (rows + 1,), generator=g).tolist()
    table, at, out = after.tolist(), int(torch.randint(0, vocab, (1,), generator=g)), []
    for c in choice:
        out.append(at)
        at = table[at][c]
    return torch.tensor(out).cuda()


def train(steps=20, rows=4096, vocab=1024, width=256, hidden=768, blocks=2, seed=0, state_bits=32):
    """Trains a model; returns the mean loss before each step."""
    import torch
    model = TokenModel(vocab, width, hidden, blocks, seed, state_bits=state_bits)
    dloss = torch.full((rows,), 1 / rows, device="cuda")
    losses = []
    for step in range(steps):
        tokens = sequence(rows, vocab, seed + 10 + step)
        loss, kept = model.loss(tokens[:-1], tokens[1:])
        losses.append(loss.mean())
        model.gradients(dloss, kept)
        model.update(step)
    return [float(v) for v in losses]


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=20)
    p.add_argument("--rows", type=int, default=4096)
    p.add_argument("--vocab", type=int, default=1024)
    p.add_argument("--width", type=int, default=256)
    p.add_argument("--hidden", type=int, default=768)
    p.add_argument("--blocks", type=int, default=2)
    p.add_argument("--state-bits", type=int, default=32, choices=(8, 32))
    a = p.parse_args()
    for step, loss in enumerate(train(a.steps, a.rows, a.vocab, a.width, a.hidden, a.blocks, state_bits=a.state_bits)):
        print(f"step {step:3d}  loss {loss:.4f}")


if __name__ == "__main__":
    main()
