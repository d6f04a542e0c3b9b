"""The expert block: its operators chained forward and backward against the same block in 64 bits
under autograd, and its training by the bank update."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _reference(block, x, offsets, dy):
    leaves = {name: w.double().cpu().requires_grad_() for name, w in block.banks.items()}
    for name in ("bias", "norm_weight", "norm_bias"):
        leaves[name] = getattr(block, name).double().cpu().requires_grad_()
    xd = x.double().cpu().requires_grad_()
    d = xd - xd.mean(1, keepdim=True)
    h = d * (d.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * leaves["norm_weight"] + leaves["norm_bias"]
    ends = offsets.tolist()
    parts = []
    for e in range(len(ends) - 1):
        s = slice(ends[e], ends[e + 1])
        a = torch.relu(h[s] @ leaves["up"][e].T + leaves["bias"][e]) ** 2
        parts.append(xd[s] + a @ leaves["down"][e])
    y = torch.cat(parts)
    y.backward(dy.double().cpu())
    return y.detach(), xd.grad, {name: v.grad for name, v in leaves.items()}


def test_block_against_autograd(gpu_lib):
    """Between the operators the activations are bf16: each of the chain's four roundings (norm, hidden
    activation, kept preactivation, hidden gradient) is off by at most 2^-9 of a step's size and they
    are independent, so the relative Frobenius error stays within 4 * 2^-8 (the derivative of the
    squared rectifier doubles one of them) plus the result's own half step."""
    from orthogonalizing_polynomial_cascade_amd import expert_block as B
    block = B.ExpertBlock(4, 64, 136, seed=3)
    g = torch.Generator(device="cuda").manual_seed(5)
    block.bias.copy_(0.1 * torch.randn(4, 136, generator=g, device="cuda"))
    block.norm_weight.add_(0.1 * torch.randn(64, generator=g, device="cuda"))
    x = torch.randn(300, 64, generator=g, device="cuda").to(torch.bfloat16)
    offsets = torch.tensor([0, 10, 10, 210, 300], dtype=torch.int32, device="cuda")
    dy = torch.randn(300, 64, generator=g, device="cuda").to(torch.bfloat16)
    y, kept = block.forward(x, offsets)
    dx, grads = block.backward(dy, kept)
    want_y, want_dx, want = _reference(block, x, offsets, dy)
    pairs = [("y", y, want_y), ("dx", dx, want_dx)] + [(name, grads[name], want[name]) for name in want]
    for name, got, ref in pairs:
        err = float((got.double().cpu() - ref).norm() / ref.norm())
        assert err <= 5 * 2.0 ** -8, (name, err)


def test_block_learns(gpu_lib):
    """Forty updates take the error of the untrained block down by more than a quarter, with no
    non-finite value on the way."""
    from orthogonalizing_polynomial_cascade_amd import expert_block as B
    losses = B.train(steps=40, rows=2048, experts=4, width=128, hidden=256)
    assert all(v == v and v < float("inf") for v in losses)
    assert sum(losses[-5:]) / 5 < 0.75 * losses[0], losses
