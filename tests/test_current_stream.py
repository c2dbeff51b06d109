"""How the binding finds torch's current stream: by torch's short internal way only where all of it is there
and it agrees with the public one."""
from types import SimpleNamespace

import pytest

from disaggregated_paged_kv_gb300 import kvx


def fake(current=7, **internal):
    return SimpleNamespace(_C=SimpleNamespace(**internal), cuda=SimpleNamespace(
        is_initialized=lambda: True, current_stream=lambda: SimpleNamespace(cuda_stream=current)))


def raises(*_):
    raise TypeError("another signature")


@pytest.mark.parametrize("internal", [
    {}, {"_cuda_getCurrentRawStream": lambda d: 9}, {"_cuda_getDevice": lambda: 0},
    {"_cuda_getCurrentRawStream": lambda d: 9, "_cuda_getDevice": lambda: 0},
    {"_cuda_getCurrentRawStream": raises, "_cuda_getDevice": lambda: 0},
    {"_cuda_getCurrentRawStream": lambda d: 9, "_cuda_getDevice": raises},
])
def test_public_way(monkeypatch, internal):
    monkeypatch.setitem(__import__("sys").modules, "torch", fake(**internal))
    monkeypatch.setattr(kvx, "_stream_number", None, raising=False)
    assert kvx._stream(None) == 7 and kvx._stream(None) == 7


def test_short_way(monkeypatch):
    t = fake(7, _cuda_getCurrentRawStream=lambda d: 7 if d == 3 else 0, _cuda_getDevice=lambda: 3)
    monkeypatch.setitem(__import__("sys").modules, "torch", t)
    monkeypatch.setattr(kvx, "_stream_number", None, raising=False)
    assert kvx._stream(None) == 7
    t.cuda.current_stream = raises  # not asked again
    assert kvx._stream(None) == 7
    assert kvx._stream(SimpleNamespace(cuda_stream=5)) == 5 and kvx._stream(0) is None
