"""Host-side checks of the training operators' entry points: every refusal happens before any HIP
call, so these run without a GPU.  Fake, never dereferenced pointer values are used."""
import pytest
import torch

from orthogonalizing_polynomial_cascade_amd import anvil

X, W, B, R, Y, Z, O, S = (0x10000000 * i for i in range(1, 9))
OK, INVALID, UNSUPPORTED, MISALIGNED, ALIAS = 0, 1, 2, 3, 4
BF16, F16, F32 = anvil.ANVIL_BF16, anvil.ANVIL_F16, anvil.ANVIL_F32


@pytest.fixture(scope="module")
def lib():
    return anvil.load()


def _norm(lib, x=X, ldx=64, w=W, b=B, pt=F32, y=Y, ldy=64, mean=R, rstd=Z, t=BF16, rows=10, cols=64):
    return lib.anvil_layer_norm(x, ldx, w, b, pt, 1e-5, y, ldy, mean, rstd, t, rows, cols, None)


def _norm_grad(lib, dy=X, x=W, w=B, mean=R, rstd=Z, dx=Y, dw=O, db=O + 4096, t=BF16, rows=10, cols=64, ld=64,
               ws=S, wsb=1 << 30):
    return lib.anvil_layer_norm_grad(dy, ld, x, ld, w, F32, mean, rstd, dx, ld, dw, db, t, rows, cols, ws, wsb, None)


def test_norm_refusals(lib):
    assert _norm(lib, rows=0) == OK and _norm(lib, cols=0, x=None, y=None) == OK
    assert _norm(lib, rows=-1) == INVALID and _norm(lib, cols=-1) == INVALID
    assert _norm(lib, x=None) == INVALID and _norm(lib, y=None) == INVALID
    assert _norm(lib, t=7) == INVALID and _norm(lib, pt=F16) == INVALID
    assert _norm(lib, ldx=63) == UNSUPPORTED and _norm(lib, ldy=63) == UNSUPPORTED
    assert _norm(lib, ldx=(1 << 22) + 1) == UNSUPPORTED
    assert _norm(lib, cols=(1 << 22) + 1, ldx=1 << 22) == UNSUPPORTED and _norm(lib, rows=1 << 31) == UNSUPPORTED
    assert _norm(lib, x=X + 1) == MISALIGNED and _norm(lib, w=W + 2) == MISALIGNED
    assert _norm(lib, mean=R + 2) == MISALIGNED and _norm(lib, t=F32, y=Y + 2) == MISALIGNED
    assert _norm(lib, y=X) == ALIAS and _norm(lib, y=W) == ALIAS and _norm(lib, mean=Y + 64) == ALIAS
    assert _norm(lib, rstd=R + 20) == ALIAS
    # column ranges at one pitch: overlapping by one element, by wrapping round, or not at all
    assert _norm(lib, ldx=128, ldy=128, y=X + 2 * 63) == ALIAS
    assert _norm(lib, ldx=128, ldy=128, y=X + 2 * 65) == ALIAS
    assert _norm(lib, ldx=128, ldy=120, y=X + 2 * 64) == ALIAS


def test_norm_grad_refusals(lib):
    need = lib.anvil_layer_norm_grad_workspace(10, 64)
    assert need > 0 and lib.anvil_layer_norm_grad_workspace(0, 64) > 0
    assert lib.anvil_layer_norm_grad_workspace(10, 0) == 0 and lib.anvil_layer_norm_grad_workspace(-1, 64) == 0
    assert _norm_grad(lib, cols=0) == OK and _norm_grad(lib, rows=0, dw=None, db=None) == OK
    for name in ("dy", "x", "mean", "rstd", "dx", "ws"):
        assert _norm_grad(lib, **{name: None}) == INVALID, name
    assert _norm_grad(lib, wsb=need - 1) == UNSUPPORTED and _norm_grad(lib, ws=S + 64) == MISALIGNED
    assert _norm_grad(lib, ld=60) == UNSUPPORTED
    assert _norm_grad(lib, dx=X) == ALIAS and _norm_grad(lib, db=O + 16) == ALIAS and _norm_grad(lib, ws=O) == ALIAS
    assert _norm_grad(lib, dw=O + 2) == MISALIGNED


def _linear(lib, x=X, ldx=64, w=W, kn=0, bias=B, bt=F32, act=0, r=R, ldr=32, y=Y, ldy=32, z=Z, ldz=32, t=BF16, rows=10,
            n=32, k=64, off=None, bits=32, experts=4):
    if off is None:
        return lib.anvil_linear(x, ldx, w, kn, bias, bt, act, r, ldr, y, ldy, z, ldz, t, rows, n, k, None)
    return lib.anvil_expert_linear(x, ldx, w, kn, off, bits, experts, bias, bt, act, r, ldr, y, ldy, z, ldz, t, rows, n,
                                   k, None)


@pytest.mark.parametrize("off", [None, O])
def test_linear_refusals(lib, off):
    def call(**kw):
        return _linear(lib, **{"off": off, **kw})
    assert call(rows=0) == OK and call(n=0) == OK and call(rows=0, x=None, w=None, y=None) == OK
    for bad in ({"rows": -1}, {"n": -1}, {"k": -1}, {"x": None}, {"w": None}, {"y": None}, {"act": 5}, {"act": -1},
                {"kn": 2}, {"t": 9}, {"bt": F16}):
        assert call(**bad) == INVALID, bad
    for bad in ({"t": F32}, {"ldx": 63}, {"ldy": 31}, {"ldr": 31}, {"ldz": 31}, {"rows": 1 << 31}, {"n": 1 << 16, "k": 1 << 15},
                {"ldy": (1 << 22) + 8}):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in ({"x": X + 1}, {"w": W + 1}, {"y": Y + 1}, {"z": Z + 1}, {"r": R + 1}, {"bias": B + 2}):
        assert call(**bad) == MISALIGNED, bad
    for bad in ({"y": X}, {"y": W + 64}, {"y": B}, {"y": R}, {"z": Y}, {"z": X + 128}):
        assert call(**bad) == ALIAS, bad


def test_expert_refusals(lib):
    assert _linear(lib, off=0, experts=4) == INVALID          # no offsets
    assert _linear(lib, off=O, bits=16) == INVALID
    assert _linear(lib, off=O, experts=-1) == INVALID
    assert _linear(lib, off=O, experts=65536) == UNSUPPORTED
    assert _linear(lib, off=O + 2) == MISALIGNED and _linear(lib, off=O + 4, bits=64) == MISALIGNED
    assert _linear(lib, off=Y + 64) == ALIAS
    assert _linear(lib, y=B + 4 * 32 * 3, off=O) == ALIAS      # the last expert's bias


def _grad_input(lib, dz=X, w=W, kn=0, pre=R, act=2, add=Z, dx=Y, t=BF16, rows=10, n=32, k=64, lddz=32, ld=64, off=None,
                bits=32, experts=4):
    if off is None:
        return lib.anvil_linear_grad_input(dz, lddz, w, kn, pre, ld, act, add, ld, dx, ld, t, rows, n, k, None)
    return lib.anvil_expert_grad_input(dz, lddz, w, kn, off, bits, experts, pre, ld, act, add, ld, dx, ld, t, rows, n, k,
                                       None)


@pytest.mark.parametrize("off", [None, O])
def test_grad_input_refusals(lib, off):
    def call(**kw):
        return _grad_input(lib, **{"off": off, **kw})
    assert call(rows=0) == OK and call(k=0) == OK
    for bad in ({"dz": None}, {"w": None}, {"dx": None}, {"pre": None}, {"act": 6}, {"kn": -1}, {"rows": -2}):
        assert call(**bad) == INVALID, bad
    for bad in ({"t": F32}, {"lddz": 31}, {"ld": 63}):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in ({"dx": X}, {"dx": W}, {"dx": R}, {"dx": Z}):
        assert call(**bad) == ALIAS, bad
    assert call(pre=R + 1) == MISALIGNED
    if off is not None:
        assert call(off=0) == INVALID


def _grad_weight(lib, dz=X, x=W, kn=0, dw=Y, wt=F32, db=B, t=BF16, rows=4096, n=32, k=64, lddz=32, ldx=64, ws=S,
                 wsb=1 << 30, off=None, bits=32, experts=4):
    if off is None:
        return lib.anvil_linear_grad_weight(dz, lddz, x, ldx, kn, dw, wt, db, t, rows, n, k, ws, wsb, None)
    return lib.anvil_expert_grad_weight(dz, lddz, x, ldx, kn, off, bits, experts, dw, wt, db, t, rows, n, k, ws, wsb,
                                        None)


@pytest.mark.parametrize("off", [None, O])
def test_grad_weight_refusals(lib, off):
    def call(**kw):
        return _grad_weight(lib, **{"off": off, **kw})
    assert call(n=0) == OK and call(k=0) == OK
    for bad in ({"dz": None}, {"x": None}, {"dw": None}, {"wt": F16}, {"kn": 3}, {"n": -1}):
        assert call(**bad) == INVALID, bad
    for bad in ({"t": F32}, {"lddz": 31}, {"ldx": 63}):
        assert call(**bad) == UNSUPPORTED, bad
    for bad in ({"dw": X}, {"dw": B}, {"db": W}):
        assert call(**bad) == ALIAS, bad
    assert call(db=B + 2) == MISALIGNED and call(dw=Y + 2) == MISALIGNED
    if off is not None:
        assert call(experts=0) == OK and call(off=0) == INVALID


def test_grad_weight_workspace(lib):
    need = lib.anvil_linear_grad_weight_workspace(0, 4096, 32, 64, 1)
    assert need >= 2 * 4 * (32 * 64 + 32)
    assert _grad_weight(lib, ws=None) == INVALID
    assert _grad_weight(lib, wsb=need - 1) == UNSUPPORTED
    assert _grad_weight(lib, ws=S + 16) == MISALIGNED
    assert _grad_weight(lib, ws=Y) == ALIAS
    assert lib.anvil_linear_grad_weight_workspace(0, 4096, 0, 64, 1) == 0
    assert lib.anvil_linear_grad_weight_workspace(0, -1, 8, 64, 1) == 0


def test_activation_grad_refusals(lib):
    def call(dy=X, z=Z, act=2, dz=Y, t=BF16, rows=4, n=32, ld=32):
        return lib.anvil_activation_grad(dy, ld, z, ld, act, dz, ld, t, rows, n, None)
    assert call(rows=0) == OK and call(n=0) == OK
    assert call(dy=None) == INVALID and call(z=None) == INVALID and call(dz=None) == INVALID and call(act=9) == INVALID
    assert call(t=F32) == UNSUPPORTED and call(ld=31) == UNSUPPORTED
    assert call(dz=X) == ALIAS and call(dz=Z) == ALIAS and call(z=Z + 1) == MISALIGNED


def test_binding_refuses_before_the_library():
    cpu = torch.zeros(4, 8, dtype=torch.bfloat16)
    for call in (lambda: anvil.anvil_layer_norm(cpu), lambda: anvil.anvil_linear(cpu, cpu),
                 lambda: anvil.anvil_linear_grad_input(cpu, cpu), lambda: anvil.anvil_linear_grad_weight(cpu, cpu),
                 lambda: anvil.anvil_activation_grad(cpu, cpu, "relu"), lambda: anvil.anvil_expert_linear(cpu, cpu, cpu)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        anvil.anvil_layer_norm([1.0])
    with pytest.raises(ValueError):
        anvil._act("tanh")


def test_offsets_reference_of_the_gpu_tests():
    """The groups that the GPU tests expect for offsets out of order and out of range."""
    from tests.layer_helpers import clamp_offsets
    assert clamp_offsets([-7, 60, 20, 90, 1 << 30, 100], 150) == [0, 60, 60, 90, 150, 150]
    assert clamp_offsets([5, 37, 37, 100], 131) == [5, 37, 37, 100]
