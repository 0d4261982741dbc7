"""The calls for a batch of many requests work on the operands' GPU, whichever one is current (host logic, as in
test_current_gpu_host)."""
import contextlib
import types

import pytest
import torch

import semi_structured_sparse_gb300 as s
from test_current_gpu_host import cache, gpu  # noqa: F401


def calls(c):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 100, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    cu, shared = torch.tensor([0, 2], dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    slots = torch.zeros(2, dtype=torch.int64)
    y, x = torch.zeros(1100, 16, dtype=torch.bfloat16), torch.zeros(1100, 8, dtype=torch.bfloat16)
    a, b = torch.zeros(3, 8, 8, dtype=torch.bfloat16), torch.zeros(3, 16, 8, dtype=torch.bfloat16)
    ids = torch.zeros(1100, dtype=torch.int32)
    return {
        "sp24_attention_decode_shared": lambda **kw: s.attention_decode_shared(q, c, table, lens, cu, shared, **kw),
        "sp24_cache_copy": lambda **kw: s.cache_copy(c, slots, c, slots, **kw),
        "sp24_add_adapters": lambda **kw: s.add_adapters(y, x, a, b, ids, **kw),
    }


@pytest.mark.parametrize("current", [0, -1])
def test_calls_work_on_the_operands_gpu(gpu, current):  # noqa: F811
    gpu.current = current
    for name, call in calls(cache()).items():
        if name == "sp24_add_adapters":
            continue
        call()
        assert gpu.lib.calls[-1] == (name, -1)
    assert s.attention_decode_shared_workspace_size(cache(), 4, 2, 1) == 64
    assert {at for _, at in gpu.lib.calls} == {-1} and gpu.current == current


def test_calls_refuse_a_stream_of_another_gpu(gpu):  # noqa: F811
    for name, call in calls(cache()).items():
        if name == "sp24_add_adapters":
            continue
        call(stream=types.SimpleNamespace(cuda_stream=7, device_index=-1))
        with pytest.raises(ValueError):
            call(stream=types.SimpleNamespace(cuda_stream=7, device_index=0))
        assert gpu.lib.calls[-1][0] != name or gpu.lib.calls[-1][1] == -1


def test_memory_for_a_call_on_another_stream_is_that_streams(gpu, monkeypatch):  # noqa: F811
    now, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    def recorded(make):
        return lambda *a, **kw: made.append(now[0]) or make(*a, **kw)

    todo = calls(cache())
    monkeypatch.setattr(torch.cuda, "stream", on)
    side = types.SimpleNamespace(cuda_stream=7, device_index=-1)
    empty, zeros = torch.empty, torch.zeros
    monkeypatch.setattr(torch, "empty", recorded(empty))
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: (recorded(zeros) if "device" in kw else zeros)(*a, **kw))
    todo["sp24_attention_decode_shared"](stream=side)
    assert len(made) == 2 and all(x is side for x in made)  # the result and the zeroed workspace


@pytest.mark.parametrize("current", [0, 5])
def test_adapters_work_on_the_operands_gpu(gpu, monkeypatch, current):  # noqa: F811
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 5)
    gpu.current = current
    call = calls(cache())["sp24_add_adapters"]
    call()
    assert gpu.lib.calls == [("sp24_add_adapters_workspace_size", 5), ("sp24_add_adapters", 5)]
    call(stream=types.SimpleNamespace(cuda_stream=7, device_index=5))
    with pytest.raises(ValueError):
        call(stream=types.SimpleNamespace(cuda_stream=7, device_index=0))
    assert {at for _, at in gpu.lib.calls} == {5} and gpu.current == current


def test_adapters_of_another_gpu_are_refused(gpu, monkeypatch):  # noqa: F811
    """Each tensor in turn is another GPU's."""
    y, x = torch.zeros(2, 16, dtype=torch.bfloat16), torch.zeros(2, 8, dtype=torch.bfloat16)
    a, b = torch.zeros(3, 8, 8, dtype=torch.bfloat16), torch.zeros(3, 16, 8, dtype=torch.bfloat16)
    ids, scales, out = torch.zeros(2, dtype=torch.int32), torch.ones(3), torch.zeros(2, 16, dtype=torch.bfloat16)
    for other in (x, a, b, ids, scales, out):
        monkeypatch.setattr(torch.Tensor, "get_device", lambda self, other=other: 4 if self is other else 5)
        with pytest.raises(ValueError):
            s.add_adapters(y, x, a, b, ids, scales, out=out)
        assert gpu.lib.calls == []
