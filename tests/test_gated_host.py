"""Refusals of the gated linear layer's entry points, before any HIP call (fake pointers, never followed)."""
import pytest
import torch

from orthogonalizing_polynomial_cascade_amd import anvil

X, W, B, Y, Z, O = (0x10000000 * i for i in range(1, 7))
OK, INVALID, UNSUPPORTED, MISALIGNED, ALIAS = 0, 1, 2, 3, 4
BF16, F16, F32 = anvil.ANVIL_BF16, anvil.ANVIL_F16, anvil.ANVIL_F32


@pytest.fixture(scope="module")
def lib():
    return anvil.load()


@pytest.mark.parametrize("off", [None, O])
def test_forward_refusals(lib, off):
    def call(x=X, ldx=64, w=W, kn=0, bias=B, bt=F32, act=4, y=Y, ldy=32, z=Z, ldz=64, t=BF16, rows=10, n=32, k=64, off=off,
             bits=32, experts=4):
        if off is None:
            return lib.anvil_gated_linear(x, ldx, w, kn, bias, bt, act, y, ldy, z, ldz, t, rows, n, k, None)
        return lib.anvil_expert_gated_linear(x, ldx, w, kn, off, bits, experts, bias, bt, act, y, ldy, z, ldz, t, rows, n, k, None)
    assert call(rows=0) == OK and call(n=0) == OK and call(rows=0, x=None, w=None, y=None) == OK
    for bad in ({"rows": -1}, {"n": -1}, {"n": -(1 << 63)}, {"k": -1}, {"x": None}, {"w": None}, {"y": None}, {"act": 5},
                {"act": -1}, {"kn": 2}, {"t": 9}, {"bt": F16}):
        assert call(**bad) == INVALID, bad
    for bad in ({"t": F32}, {"ldx": 63}, {"ldy": 31}, {"ldz": 63}, {"rows": 1 << 31}, {"n": 1 << 15, "k": 1 << 15},
                {"n": (1 << 21) + 1}, {"n": 1 << 62}, {"ldy": (1 << 22) + 8}):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in ({"x": X + 1}, {"w": W + 1}, {"y": Y + 1}, {"z": Z + 1}, {"bias": B + 2}):
        assert call(**bad) == MISALIGNED, bad
    # the second halves of the weight, the bias and z count too
    for bad in ({"y": X}, {"y": W + 2 * 63 * 64}, {"y": B + 4 * 63}, {"z": Y}, {"z": X + 128}, {"y": Z + 2 * 40}):
        assert call(**bad) == ALIAS, bad
    if off is not None:
        assert call(off=0) == INVALID and call(bits=16) == INVALID and call(experts=65536) == UNSUPPORTED
        assert call(off=Y + 64) == ALIAS and call(off=O + 2) == MISALIGNED


@pytest.mark.parametrize("off", [None, O])
def test_grad_refusals(lib, off):
    def call(dy=X, w=W, kn=0, z=Z, act=4, dz=Y, t=BF16, rows=10, n=32, k=64, lddy=32, ldz=128, lddz=128, off=off, bits=32,
             experts=4):
        if off is None:
            return lib.anvil_gated_grad_input(dy, lddy, w, kn, z, ldz, act, dz, lddz, t, rows, n, k, None)
        return lib.anvil_expert_gated_grad_input(dy, lddy, w, kn, off, bits, experts, z, ldz, act, dz, lddz, t, rows, n, k, None)
    assert call(rows=0) == OK and call(k=0) == OK
    for bad in ({"dy": None}, {"w": None}, {"dz": None}, {"z": None}, {"act": 6}, {"kn": -1}, {"rows": -2}, {"z": None, "act": 0}):
        assert call(**bad) == INVALID, bad
    for bad in ({"t": F32}, {"lddy": 31}, {"ldz": 127}, {"lddz": 127}, {"k": (1 << 21) + 1}):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in ({"dz": X}, {"dz": W}, {"dz": Z}, {"dz": Z + 2 * 64}):
        assert call(**bad) == ALIAS, bad
    assert call(z=Z + 1) == MISALIGNED


def test_activation_grad_refusals(lib):
    def call(dh=X, z=Z, act=4, dz=Y, t=BF16, rows=10, n=32, lddh=32, ldz=64, lddz=64):
        return lib.anvil_gated_activation_grad(dh, lddh, z, ldz, act, dz, lddz, t, rows, n, None)
    assert call(rows=0) == OK and call(n=0) == OK
    for bad in ({"dh": None}, {"z": None}, {"dz": None}, {"act": 9}, {"n": -1}):
        assert call(**bad) == INVALID, bad
    for bad in ({"t": F32}, {"lddh": 31}, {"ldz": 63}, {"lddz": 63}):
        assert call(**bad) == UNSUPPORTED, bad
    assert call(dz=X) == ALIAS and call(dz=Z) == ALIAS and call(dh=X + 1) == MISALIGNED


def test_binding_refuses_before_the_library():
    cpu = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: anvil.anvil_gated_linear(cpu, cpu), lambda: anvil.anvil_gated_grad_input(cpu, cpu, cpu),
                 lambda: anvil.anvil_gated_activation_grad(cpu, cpu), lambda: anvil.anvil_expert_gated_linear(cpu, cpu, cpu),
                 lambda: anvil.anvil_expert_gated_grad_input(cpu, cpu, cpu, cpu)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        anvil.anvil_gated_linear([1.0], cpu)
