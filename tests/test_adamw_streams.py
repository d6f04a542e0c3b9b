"""Which streams are recorded as users of what an AdamW object holds, on stand-ins of torch's tensors, streams and
allocator and of the library's step (nothing is launched)."""
import contextlib
import types

import pytest
import torch

from orthogonalizing_polynomial_cascade_amd import anvil

HOME = 7


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class _Tensor:
    at = 0x10000000

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.users = torch.Size(shape), dtype, []
        self.is_cuda, self.device = True, "cuda:0"
        self.pointer = _Tensor.at
        _Tensor.at += 0x100000

    def numel(self):
        return self.shape.numel()

    def data_ptr(self):
        return self.pointer

    def get_device(self):
        return 0

    def is_contiguous(self):
        return True

    def view(self, *_):
        return self

    def zero_(self):
        return self

    def copy_(self, _):
        return self

    def record_stream(self, stream):
        self.users.append(stream.cuda_stream)


@pytest.fixture
def on(monkeypatch):
    """A context manager that makes the stream of a handle the current one, which is first HOME."""
    anvil._module()
    lib = anvil.load()
    now = [_Stream(HOME)]

    @contextlib.contextmanager
    def switch(handle):
        now.append(_Stream(handle))
        yield now[-1]
        now.pop()

    cuda = types.SimpleNamespace(Stream=_Stream, ExternalStream=lambda handle, *_: _Stream(handle), is_available=lambda: True,
                                 current_device=lambda: 0, current_stream=lambda *_: now[-1],
                                 is_current_stream_capturing=lambda: False)
    fake = types.SimpleNamespace(
        cuda=cuda, Tensor=_Tensor, Size=torch.Size, _C=types.SimpleNamespace(_cuda_getCurrentRawStream=lambda _: now[-1].cuda_stream),
        empty=lambda shape, dtype, device: _Tensor(shape, dtype),
        frombuffer=lambda words, dtype: types.SimpleNamespace(to=lambda _: _Tensor((len(words),), dtype)),
        **{name: getattr(torch, name) for name in ("float32", "bfloat16", "float16", "float8_e4m3fn", "int16", "uint16", "int64",
                                                   "uint8")})
    monkeypatch.setattr(anvil, "_torch", fake)
    monkeypatch.setattr(anvil, "load", lambda: types.SimpleNamespace(
        anvil_adamw_plan_bytes=lib.anvil_adamw_plan_bytes, anvil_adamw_plan=lib.anvil_adamw_plan,
        anvil_adamw=lambda *_: 0, anvil_adamw_dev=lambda *_: 0))
    return switch


def _made(bits=8):
    def t(dtype):
        return _Tensor((300,), dtype)

    plan = anvil.AdamW([t(torch.bfloat16), t(torch.float32)], [t(torch.bfloat16), t(torch.float32)],
                       mantissas=[t(torch.int16), None], state_bits=[bits, 32])
    held = [v for name in ("params", "mantissas", "grads", "m", "v", "m_scale", "v_scale") for v in getattr(plan, name)
            if v is not None] + [plan._plan]
    assert len(held) == 12
    return plan, held


@pytest.mark.parametrize("stream", [None, HOME, _Stream(HOME)])
def test_the_constructors_stream_needs_no_record(on, stream):
    plan, held = _made()
    anvil.anvil_adamw(plan, 1e-3, 1, stream=stream)
    assert not any(t.users for t in held)


@pytest.mark.parametrize("stream", [9, _Stream(9), types.SimpleNamespace(cuda_stream=9)])
def test_a_step_on_another_stream(on, stream):
    """Everything that the launch reads or writes has its stream as a user, once however many steps there are."""
    plan, held = _made()
    anvil.anvil_adamw(plan, 1e-3, 1, stream=stream)
    anvil.anvil_adamw_dev(plan, _Tensor((5,), torch.float32), stream=stream)
    assert all(t.users == [9] for t in held)
    anvil.anvil_adamw(plan, 1e-3, 2, stream=_Stream(11))
    assert all(t.users == [9, 11] for t in held)


def test_another_stream_that_is_the_current_one(on):
    """The memory is the constructor's stream's, whatever stream is current at the step."""
    plan, held = _made()
    with on(9):
        anvil.anvil_adamw(plan, 1e-3, 1)
        anvil.anvil_adamw(plan, 1e-3, 2, stream=9)
        anvil.anvil_adamw(plan, 1e-3, 3, stream=HOME)
    assert all(t.users == [9] for t in held)


def test_gradients_that_are_given_later(on):
    """The streams that a plan has run on are users of the gradients it takes from then on."""
    plan, _ = _made()
    anvil.anvil_adamw(plan, 1e-3, 1, stream=9)
    later = [_Tensor((300,), torch.float32) for _ in range(2)]
    plan.bind(later)
    assert all(t.users == [9] for t in later)
    with on(11):
        anvil.anvil_adamw(plan, 1e-3, 2)
    assert all(t.users == [9, 11] for t in later)


def test_an_empty_plan_has_nothing_to_record(on):
    anvil.anvil_adamw(anvil.AdamW([], []), 1e-3, 1, stream=9)
