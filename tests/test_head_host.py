"""Refusals of the cross entropy's entry points, before any HIP call (fake pointers, never followed)."""
import pytest
import torch

from orthogonalizing_polynomial_cascade_amd import anvil

X, W, T, L, E, D, DX, DW, S = (0x10000000 * i for i in range(1, 10))
OK, INVALID, UNSUPPORTED, MISALIGNED, ALIAS = 0, 1, 2, 3, 4
BF16, F16, F32 = anvil.ANVIL_BF16, anvil.ANVIL_F16, anvil.ANVIL_F32


@pytest.fixture(scope="module")
def lib():
    return anvil.load()


def _forward(lib, x=X, ldx=64, w=W, kn=0, t=T, bits=64, loss=L, lse=E, dt=BF16, rows=10, vocab=32, k=64, ws=S, wsb=1 << 40):
    return lib.anvil_cross_entropy(x, ldx, w, kn, t, bits, loss, lse, dt, rows, vocab, k, ws, wsb, None)


def _grad(lib, x=X, ldx=64, w=W, kn=0, t=T, bits=64, lse=E, dl=D, dx=DX, lddx=64, dw=DW, wt=F32, dt=BF16, rows=10, vocab=32, k=64,
          ws=S, wsb=1 << 40):
    return lib.anvil_cross_entropy_grad(x, ldx, w, kn, t, bits, lse, dl, dx, lddx, dw, wt, dt, rows, vocab, k, ws, wsb, None)


def test_forward_refusals(lib):
    assert _forward(lib, rows=0, x=None, w=None, t=None, loss=None, lse=None, ws=None) == OK
    for bad in ({"rows": -1}, {"vocab": 0}, {"vocab": -5}, {"k": -1}, {"x": None}, {"w": None}, {"t": None}, {"loss": None},
                {"lse": None}, {"ws": None}, {"kn": 2}, {"bits": 16}, {"dt": 9}):
        assert _forward(lib, **bad) == INVALID, bad
    for bad in ({"dt": F32}, {"ldx": 63}, {"ldx": (1 << 22) + 1}, {"rows": (1 << 22) + 1}, {"vocab": (1 << 22) + 1},
                {"vocab": 1 << 20, "k": 1 << 11, "ldx": 1 << 11}, {"rows": 1 << 22, "vocab": (1 << 15) + 1, "k": 8},
                {"rows": 1 << 22, "k": (1 << 15) + 1, "ldx": 1 << 16, "vocab": 16}):
        assert _forward(lib, **bad) == UNSUPPORTED, bad
    for bad in ({"x": X + 1}, {"w": W + 1}, {"t": T + 4}, {"loss": L + 2}, {"lse": E + 1}, {"ws": S + 64}):
        assert _forward(lib, **bad) == MISALIGNED, bad
    for bad in ({"loss": X}, {"loss": E + 8}, {"lse": W + 64}, {"loss": T}, {"ws": X}, {"ws": W}, {"lse": S}):
        assert _forward(lib, **bad) == ALIAS, bad


def test_grad_refusals(lib):
    assert _grad(lib, rows=0, dw=None) == OK and _grad(lib, k=0) == OK and _grad(lib, dx=None, dw=None, x=None) == OK
    for bad in ({"rows": -1}, {"vocab": 0}, {"k": -1}, {"x": None}, {"w": None}, {"t": None}, {"lse": None}, {"dl": None},
                {"ws": None}, {"kn": -1}, {"bits": 8}, {"wt": F16}):
        assert _grad(lib, **bad) == INVALID, bad
    for bad in ({"dt": F32}, {"ldx": 63}, {"lddx": 63}, {"rows": (1 << 22) + 1}):
        assert _grad(lib, **bad) == UNSUPPORTED, bad
    for bad in ({"dx": DX + 1}, {"dw": DW + 2}, {"dl": D + 2}, {"ws": S + 128}):
        assert _grad(lib, **bad) == MISALIGNED, bad
    for bad in ({"dx": X}, {"dw": W}, {"dx": DW}, {"dw": E}, {"ws": D}, {"dx": T}, {"dx": S}):
        assert _grad(lib, **bad) == ALIAS, bad


def test_workspaces(lib):
    need = lib.anvil_cross_entropy_workspace(0, 3, 10, 32, 64)
    assert need > 0 and _forward(lib, wsb=need - 1) == UNSUPPORTED
    # operands that are copied first take more, and the call sees for itself whether they are
    more = lib.anvil_cross_entropy_workspace(0, 0, 10, 32, 64)
    assert more >= need + (10 + 32) * 64 * 2
    assert _forward(lib, x=X + 2, w=W + 2, wsb=more - 1) == UNSUPPORTED
    assert lib.anvil_cross_entropy_workspace(0, 2, 10, 32, 64) >= need + 10 * 64 * 2
    assert _forward(lib, ldx=65, wsb=need) == UNSUPPORTED
    # a single row has no pitch
    one = lib.anvil_cross_entropy_workspace(0, 3, 1, 32, 64)
    assert _forward(lib, rows=1, ldx=3, wsb=one - 1) == UNSUPPORTED
    assert lib.anvil_cross_entropy_workspace(0, 3, 0, 32, 64) == 0 and lib.anvil_cross_entropy_workspace(0, 3, 10, 0, 64) == 0
    # the gradients' grows with what they keep of P, not with the whole of it
    g = lib.anvil_cross_entropy_grad_workspace
    assert g(1, 1, 0, 3, BF16, 16384, 50304, 768) < 16384 * 50304 * 2
    assert g(0, 0, 0, 3, BF16, 10, 32, 64) == 0 and g(1, 1, 0, 3, F32, 10, 32, 64) == 0
    assert _grad(lib, wsb=g(1, 1, 0, 3, BF16, 10, 32, 64) - 1) == UNSUPPORTED


def test_binding_refuses_before_the_library():
    cpu, t = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        anvil.anvil_cross_entropy(cpu, cpu, t)
    with pytest.raises(ValueError):
        anvil.anvil_cross_entropy_grad(cpu, cpu, t, t.float(), t.float())
    with pytest.raises(TypeError):
        anvil.anvil_cross_entropy([1.0], cpu, t)


@pytest.mark.parametrize("rows,vocab", [(1, 1 << 22), (16384, 50304), (1 << 18, 1 << 19), ((1 << 19) - 1, 100000),
                                        (1 << 20, 1 << 17), (1 << 22, 1 << 15)])
def test_what_the_probabilities_take(lib, rows, vocab):
    """P takes up to 1 GiB, or 2 KiB a row; beside it dx's sums (one for each of 8 columns here) and planes of partial sums,
    of which dx's end at 2.7e8 bytes and dw's at 1.1e9."""
    for want in ((1, 0), (0, 1), (1, 1)):
        need = lib.anvil_cross_entropy_grad_workspace(*want, 0, 3, BF16, rows, vocab, 8)
        p = max(1 << 30, 2048 * rows)
        assert 0 < need <= p + want[0] * (rows * 32 + 270_000_000) + want[1] * 1_100_000_000 + 4096


def test_heads_of_more_than_2_30_weights(lib):
    """A vocabulary of 152064 entries at a width of 8192 is taken; 2^31 weights are not."""
    for kn in (0, 1):
        for vocab, k in ((152064, 8192), (1 << 22, 511), (511, 1 << 22), ((1 << 20) - 1, 1 << 11)):
            assert lib.anvil_cross_entropy_workspace(kn, 3, 10, vocab, k) > 0, (vocab, k)
            assert lib.anvil_cross_entropy_grad_workspace(1, 1, kn, 3, BF16, 10, vocab, k) > 0, (vocab, k)
        for vocab, k in ((1 << 20, 1 << 11), (1 << 22, 512)):
            assert lib.anvil_cross_entropy_workspace(kn, 3, 10, vocab, k) == 0
            assert lib.anvil_cross_entropy_grad_workspace(1, 1, kn, 3, BF16, 10, vocab, k) == 0
