"""The AdamW plan and the refusals of its step, without a GPU (fake pointers, never followed)."""
import ctypes

import pytest
import torch

from orthogonalizing_polynomial_cascade_amd import anvil
from tests import adamw_helpers as A

OK, INVALID, UNSUPPORTED, MISALIGNED, ALIAS = 0, 1, 2, 3, 4
F32, BF16, F16 = anvil.ANVIL_F32, anvil.ANVIL_BF16, anvil.ANVIL_F16


@pytest.fixture(scope="module")
def lib():
    return anvil.load()


def _tensor(base=0x10000000, count=1000, bits=32, **kw):
    t = anvil.AdamwTensor()
    far = 0x1000000
    fields = dict(param=base, mantissa=None, grad=base + far, m=base + 2 * far, v=base + 3 * far, m_scale=None, v_scale=None,
                  count=count, param_dtype=F32, grad_dtype=F32, lr_mul=1.0, wd_mul=1.0, state_bits=bits)
    if bits == 8:
        fields |= dict(m_scale=base + 4 * far, v_scale=base + 5 * far)
    for k, v in {**fields, **kw}.items():
        setattr(t, k, v)
    return t


def _plan(lib, *tensors, size=None):
    table = (anvil.AdamwTensor * max(1, len(tensors)))(*tensors)
    at = ctypes.cast(table, ctypes.c_void_p)
    need = lib.anvil_adamw_plan_bytes(at, len(tensors))
    room = torch.zeros(max(1, need // 8 + 2), dtype=torch.int64)
    return lib.anvil_adamw_plan(at, len(tensors), room.data_ptr(), need if size is None else size), need, room


def test_layout(lib):
    assert ctypes.sizeof(anvil.AdamwTensor) == 88
    status, need, room = _plan(lib, _tensor(count=5000), _tensor(0x40000000, count=0), _tensor(0x80000000, count=2048))
    assert status == OK and need == 3 * 88 + 4 * 8
    words = room.view(torch.int32)[3 * 22:3 * 22 + 8].tolist()
    assert words == [0, 0, 0, 1, 0, 2, 2, 0]
    assert _plan(lib)[0] == OK and lib.anvil_adamw_plan_bytes(None, 3) == 0


def test_plan_refusals(lib):
    for bad in ({"count": -1}, {"param": None}, {"grad": None}, {"m": None}, {"v": None}, {"param_dtype": 7}, {"grad_dtype": -1},
                {"state_bits": 16}, {"mantissa": 0x7000000}, {"bits": 8, "m_scale": None}, {"bits": 8, "v_scale": None}):
        assert _plan(lib, _tensor(**bad))[0] == INVALID, bad
    assert _plan(lib, _tensor(count=(1 << 40) + 1))[0] == UNSUPPORTED
    assert _plan(lib, _tensor(), size=88)[0] == UNSUPPORTED
    for bad in ({"param": 0x10000002}, {"grad": 0x11000001, "grad_dtype": BF16}, {"m": 0x12000002},
                {"mantissa": 0x17000001, "param_dtype": BF16}, {"bits": 8, "v_scale": 0x15000002}):
        assert _plan(lib, _tensor(**bad))[0] == MISALIGNED, bad
    far = 0x1000000
    for bad in ({"m": 0x10000000 + 3996}, {"grad": 0x10000000 + 400}, {"v": 0x10000000 + 2 * far}, {"bits": 8, "m_scale": 0x15000000},
                {"param_dtype": BF16, "mantissa": 0x10000000}):
        assert _plan(lib, _tensor(**bad))[0] == ALIAS, bad
    # side by side is not shared; another tensor's state is, its gradient only where something writes it
    assert _plan(lib, _tensor(m=0x10000000 + 4000))[0] == OK
    two = 0x40000000
    assert _plan(lib, _tensor(), _tensor(two, grad=0x11000000))[0] == OK
    assert _plan(lib, _tensor(), _tensor(two, m=0x12000000))[0] == ALIAS
    assert _plan(lib, _tensor(), _tensor(two, grad=0x10000000))[0] == ALIAS
    # a long span over short ones, written or not
    assert _plan(lib, _tensor(count=100000), _tensor(0x10000000 + 1024, count=4, grad=two, m=two + 64, v=two + 128))[0] == ALIAS


def test_step_refusals(lib):
    def step(plan=0x10000000, size=88 + 8, tensors=1, lr=1e-3, b1=0.9, b2=0.95, eps=1e-8, wd=0.1, n=1, scale=None):
        return lib.anvil_adamw(plan, size, tensors, lr, b1, b2, eps, wd, n, 7, scale, None)

    def dev(scalars=0x20000000, size=88 + 8, b2=0.9):
        return lib.anvil_adamw_dev(0x10000000, size, 1, scalars, 0.9, b2, 1e-8, None, None)
    assert step(size=88) == OK and step(plan=None, size=0, tensors=0) == OK   # nothing to do
    for bad in ({"plan": None}, {"size": 80}, {"size": 88 + 4}, {"tensors": -1}, {"b1": 1.0}, {"b1": -0.1}, {"b2": 1.5},
                {"b2": float("nan")}, {"eps": -1e-8}, {"n": 0}):
        assert step(**bad) == INVALID, bad
    assert step(plan=0x10000008) == MISALIGNED and step(scale=0x20000002) == MISALIGNED
    assert dev(scalars=None) == INVALID and dev(size=90) == INVALID and dev(b2=1.0) == INVALID
    assert dev(scalars=0x20000001) == MISALIGNED


def test_codes_of_the_reference():
    """The tests' e4m3 encoder against torch's conversion: with the noise of half a step it rounds to the nearest code but
    for ties, without noise it truncates, and decoding gives the value back."""
    g = torch.Generator().manual_seed(1)
    v = torch.randn(20000, generator=g) * torch.exp(3 * torch.randn(20000, generator=g))
    codes, scale = A.encode(v, torch.full((20000,), 1 << 19), 0)
    q = A.rows(v) * (torch.tensor(448.0) / A.rows(v).abs().amax(1, keepdim=True))
    want = q.to(torch.float8_e4m3fn).view(torch.uint8).view(-1)[:20000]
    differ = codes.view(torch.uint8) != want
    assert differ.float().mean() < 1e-3
    down, _ = A.encode(v, torch.zeros(20000, dtype=torch.int64), 0)
    back = A.decode(down, scale)
    assert (back.abs() <= v.abs() * (1 + 2.0 ** -22)).all()
    step = torch.maximum(v.abs() * 2.0 ** -3, scale.repeat_interleave(256)[:20000] * 2.0 ** -9)
    assert ((back - v).abs() <= step * (1 + 2.0 ** -20)).all()


def test_binding_refuses_before_the_library():
    with pytest.raises(ValueError):
        anvil.AdamW([torch.zeros(4)], [torch.zeros(4)])
    with pytest.raises(ValueError):
        anvil.AdamW([], [torch.zeros(4)])
    with pytest.raises(TypeError):
        anvil.AdamW([[1.0]], [torch.zeros(4)])
