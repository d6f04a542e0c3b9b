"""The token model: gated blocks, head and both updates chained, against the same model in 64 bits under autograd."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def _reference(model, tokens, targets, dloss):
    leaves = {name: getattr(model, name).double().cpu().requires_grad_() for name in ("bank", "embedding", "head", "norms")}

    def norm(x, row):
        d = x - x.mean(1, keepdim=True)
        return d * (d.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * row[0] + row[1]

    x = leaves["embedding"][tokens.cpu()]
    for b in range(model.blocks):
        gate, up, down = leaves["bank"][3 * b:3 * b + 3]
        h = norm(x, leaves["norms"][b])
        x = x + (torch.nn.functional.silu(h @ gate.T) * (h @ up.T)) @ down
    loss = torch.nn.functional.cross_entropy(norm(x, leaves["norms"][-1]) @ leaves["head"].T, targets.long().cpu(),
                                             reduction="none", ignore_index=-1)
    (loss * dloss.double().cpu()).sum().backward()
    return loss.detach(), {name: v.grad for name, v in leaves.items()}


@pytest.mark.parametrize("vocab,width,hidden,blocks", [(500, 64, 136, 2), (1001, 72, 64, 1)])
def test_gradients_against_autograd(gpu_lib, vocab, width, hidden, blocks):
    """Between the operators activations and their gradients are bf16.  A forward block rounds four times (norm, z, gated
    value, sum), a backward one four times (dz, dh, the norm's gradient, the sum), each by at most 2^-9 of the value on a
    relative half step of 2^-8 and independently: with the norm and the head's P and dh that is at most
    8 * blocks + 5 roundings, whose root sum of squares stays within sqrt(8 * blocks + 5) * 2^-8 of the result, the
    layers' Jacobians being of order one; twice that is allowed."""
    from orthogonalizing_polynomial_cascade_amd import token_model as M
    model = M.TokenModel(vocab, width, hidden, blocks, seed=3)
    g = torch.Generator().manual_seed(5)
    model.norms.add_(0.1 * torch.randn(model.norms.shape, generator=g).cuda())
    tokens = torch.randint(0, vocab, (300,), generator=g).cuda()
    targets = torch.randint(0, vocab, (300,), generator=g)
    targets[::7] = -1
    targets = targets.cuda()
    dloss = torch.full((300,), 1 / 300, device="cuda")
    loss, kept = model.loss(tokens, targets)
    grads = model.gradients(dloss, kept)
    want_loss, want = _reference(model, tokens, targets, dloss)
    bar = 2 * (8 * blocks + 5) ** 0.5 * 2.0 ** -8
    for name, got, ref in [("loss", loss, want_loss)] + [(name, grads[name], want[name]) for name in want]:
        err = float((got.double().cpu() - ref).norm() / ref.norm())
        assert err <= bar, (name, err)


@pytest.mark.parametrize("state_bits", [32, 8])
def test_training_runs(gpu_lib, state_bits):
    """Both updates move every parameter, and the losses stay finite."""
    from orthogonalizing_polynomial_cascade_amd import token_model as M
    model = M.TokenModel(300, 64, 128, 2, seed=1, state_bits=state_bits)
    before = {name: getattr(model, name).clone() for name in ("bank", "embedding", "head", "norms")}
    dloss = torch.full((256,), 1 / 256, device="cuda")
    for step in range(3):
        tokens = M.sequence(256, 300, step)
        loss, kept = model.loss(tokens[:-1], tokens[1:])
        assert torch.isfinite(loss).all()
        model.gradients(dloss, kept)
        model.update(step)
    for name, old in before.items():
        now = getattr(model, name)
        assert torch.isfinite(now.float()).all() and not torch.equal(now, old), name
    losses = M.train(steps=2, rows=128, vocab=200, width=64, hidden=64, blocks=1, state_bits=state_bits)
    assert len(losses) == 2 and all(v == v and abs(v) < float("inf") for v in losses)


@pytest.mark.parametrize("state_bits", [32, 8])
def test_updates_are_the_operators(gpu_lib, state_bits):
    """Two steps: every parameter goes against its gradient in the first, the bank's as a bank update of a copy with the
    same gradients and settings and the others' as the AdamW formula on the CPU, bit for bit."""
    from orthogonalizing_polynomial_cascade_amd import token_model as M
    from tests import adamw_helpers as A
    model = M.TokenModel(300, 64, 128, 2, seed=1, state_bits=state_bits)
    names, dloss = ("embedding", "head", "norms"), torch.full((256,), 1 / 256, device="cuda")
    flat = lambda t: None if t is None else t.detach().cpu().reshape(-1).clone()  # noqa: E731
    for step in range(2):
        tokens = M.sequence(256, 300, step)
        _, kept = model.loss(tokens[:-1], tokens[1:])
        grads = {name: g.clone() for name, g in model.gradients(dloss, kept).items()}
        before = {name: getattr(model, name).clone() for name in names + ("bank",)}
        adam, states = model.adam, []
        for i, name in enumerate(names):
            s = {k: flat(v[i]) for k, v in (("param", adam.params), ("mantissa", adam.mantissas), ("grad", adam.grads), ("m", adam.m),
                                            ("v", adam.v), ("m_scale", adam.m_scale), ("v_scale", adam.v_scale))}
            assert torch.equal(s["grad"], flat(grads[name]))
            states.append(s | {"lr_mul": 1.0, "wd_mul": 0.0 if name == "norms" else 1.0})
        bank = [t.clone() for t in (model.velocity, model.energy, model.bank, model.mantissa)]
        model.update(step)
        # the clipping coefficient as a model's user would have it: a norm over all that AdamW takes
        norm = torch.stack([grads[name].float().norm() for name in names]).norm()
        clip = float(torch.clamp(M.CLIP / (norm + 1e-6), max=1.0))
        for i, name in enumerate(names):
            want = A.step32(states[i], i, model.adam_lr, 0.01, (0.9, 0.95), 1e-8, step + 1, clip, step + 1)
            for key, have in (("param", adam.params), ("mantissa", adam.mantissas), ("m", adam.m), ("v", adam.v)):
                if want[key] is not None:
                    kind = {1: torch.uint8, 2: torch.int16, 4: torch.int32}[want[key].element_size()]
                    assert torch.equal(flat(have[i]).view(kind), want[key].view(kind)), (step, name, key)
        velocity, energy, weights, mantissa = bank
        gpu_lib.anvil_bank_update(grads["bank"], velocity, *gpu_lib.rail_scalars(step), energy, 0.95, weights, mantissa, 0.0,
                                  model.eff_lr)
        assert torch.equal(weights.view(torch.int16), model.bank.view(torch.int16)) and torch.equal(mantissa, model.mantissa)
        if step == 0:   # no state yet that could point elsewhere
            for name, old in before.items():
                assert float(((getattr(model, name).double() - old.double()) * grads[name].double()).sum()) < 0, name
