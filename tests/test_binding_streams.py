"""Memory that the binding allocates for a call on another stream, on stand-ins of torch's streams and
allocator: which stream's pool a tensor comes from, and who else is recorded as its user."""
import ast
import contextlib
import types

import pytest

from orthogonalizing_polynomial_cascade_amd import anvil


class _Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class _Tensor:
    def __init__(self, pool):
        self.pool, self.users = pool, []

    def record_stream(self, stream):
        self.users.append(stream.cuda_stream)


@pytest.fixture
def streams(monkeypatch):
    """A torch whose current stream has the handle 7."""
    now = [_Stream(7)]

    @contextlib.contextmanager
    def switch(stream):
        now.append(stream)
        yield
        now.pop()

    cuda = types.SimpleNamespace(Stream=_Stream, ExternalStream=_Stream, current_stream=lambda *a: now[-1],
                                 stream=switch)
    fake = types.SimpleNamespace(cuda=cuda, empty=lambda *a, **k: _Tensor(now[-1].cuda_stream))
    monkeypatch.setattr(anvil, "_torch", fake)


@pytest.mark.parametrize("stream", [None, 7, _Stream(7), types.SimpleNamespace(cuda_stream=7)])
def test_current_stream_allocates_for_itself(streams, stream):
    t = anvil._empty((4,), None, None, stream)
    assert t.pool == 7 and t.users == []


@pytest.mark.parametrize("stream", [9, _Stream(9), types.SimpleNamespace(cuda_stream=9)])
def test_another_stream_takes_memory_of_its_own(streams, stream):
    """Memory freed on the current stream may still be in use by what is queued there, and the call's
    stream does not wait for that."""
    t = anvil._empty((4,), None, None, stream)
    assert t.pool == 9 and t.users == [7]


def test_every_allocation_goes_through_the_same_place():
    tree = ast.parse(open(anvil.__file__).read())
    allocating = {"empty", "empty_like", "zeros", "zeros_like", "full", "empty_strided", "new_empty"}
    found = [f.name for f in ast.walk(tree) if isinstance(f, ast.FunctionDef)
             for c in ast.walk(f) if isinstance(c, ast.Call) and isinstance(c.func, ast.Attribute)
             and c.func.attr in allocating]
    assert found and set(found) == {"_empty"}, found
