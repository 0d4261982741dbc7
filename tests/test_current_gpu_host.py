"""Calls work on the operands' GPU, whichever one is current (host logic: tensors of the CPU, whose index is -1, and a
library that records which GPU was current when it was called)."""
import contextlib
import types

import pytest
import torch

import semi_structured_sparse_gb300 as s

CPU = torch.device("cpu")


class Library:
    """Stands in for libsp24.so: every call succeeds, or gives a size of 64."""

    def __init__(self, gpu):
        self.gpu, self.calls = gpu, []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, self.gpu.current))
            return 64 if name.endswith("_workspace_size") else 0
        return call


@pytest.fixture
def gpu(monkeypatch):
    g = types.SimpleNamespace(current=0)

    @contextlib.contextmanager
    def device(index):
        index = getattr(index, "index", index)
        before, g.current = g.current, -1 if index is None else index
        yield
        g.current = before

    g.lib = Library(g)
    monkeypatch.setattr(s, "_lib", g.lib)
    monkeypatch.setattr(s, "_current_gpu", lambda: g.current, raising=False)
    monkeypatch.setattr(s, "_raw_stream", lambda index: 100 + index)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "stream", contextlib.nullcontext)
    return g


def cache():
    c = s.KVCache.__new__(s.KVCache)
    c.heads, c.page_size, c.head_dim, c.device, c._index, c._scale, c._address = 2, 16, 64, CPU, -1, 0.125, 0
    return c


def attention_calls(c):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 100, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32)
    qkv = torch.zeros(2, 8 * 64, dtype=torch.bfloat16)
    slots, turn = torch.zeros(2, dtype=torch.int64), torch.zeros(4, 64)
    ws = torch.zeros(64, dtype=torch.uint8)
    return {
        "sp24_qk_norm_rope": lambda **kw: s.qk_norm_rope(qkv, 4, c, lens, slots, turn, **kw),
        "sp24_attention_decode": lambda **kw: s.attention_decode(q, c, table, lens, workspace=ws, **kw),
        "sp24_attention_prompt": lambda **kw: s.attention_prompt(q, cu, c, table, lens, workspace=ws, **kw),
    }


@pytest.mark.parametrize("current", [0, -1])
def test_attention_calls_work_on_the_caches_gpu(gpu, current):
    gpu.current = current
    c = cache()
    for name, call in attention_calls(c).items():
        call()
        assert gpu.lib.calls[-1] == (name, -1)
    assert s.attention_decode_workspace_size(c, 4) == 64
    assert s.attention_prompt_workspace_size(c, 4, 2, 2, 100) == 64
    # a prompt that asks for its workspace itself
    s.attention_prompt(torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.tensor([0, 1, 2], dtype=torch.int32), c,
                       torch.zeros(2, 100, dtype=torch.int32), torch.ones(2, dtype=torch.int32))
    assert len(gpu.lib.calls) == 7 and {at for _, at in gpu.lib.calls} == {-1}
    assert gpu.current == current


def test_attention_calls_refuse_a_stream_of_another_gpu(gpu):
    out = torch.zeros(2, 256, dtype=torch.bfloat16)
    for call in attention_calls(cache()).values():
        call(out=out, stream=types.SimpleNamespace(cuda_stream=7, device_index=-1))
        done = len(gpu.lib.calls)
        with pytest.raises(ValueError):
            call(out=out, stream=types.SimpleNamespace(cuda_stream=7, device_index=0))
        assert len(gpu.lib.calls) == done


def test_device_errors_are_those_of_the_streams_gpu(gpu):
    s.last_device_error(types.SimpleNamespace(cuda_stream=7, device_index=-1))
    gpu.current = 3
    s.last_device_error(types.SimpleNamespace(cuda_stream=7, device_index=3))
    assert gpu.lib.calls == [("sp24_last_device_error", -1), ("sp24_last_device_error", 3)]


def linear_calls():
    u8, f32, bf16, i8 = torch.uint8, torch.float32, torch.bfloat16, torch.int8
    z = lambda *shape, t=u8: torch.zeros(shape, dtype=t)  # noqa: E731
    sx, sw, values, meta = z(1, 4, t=f32), z(1, 256, t=f32), z(256, 64), z(256, 16)
    return {
        "sp24_fp8_compress": lambda **kw: s.compress(z(256, 128, t=bf16), **kw),
        "sp24_fp8_decompress": lambda **kw: s.decompress(values, meta, sw, **kw),
        "sp24_fp8_quantize_act": lambda **kw: s.quantize_act(z(4, 128, t=f32), **kw),
        "sp24_fp8_quantize_act_bf16": lambda **kw: s.quantize_act(z(4, 128, t=bf16), **kw),
        "sp24_fp8_gemm": lambda **kw: s.gemm(z(4, 128), sx, values, meta, sw, **kw),
        "sp24_fp8_gemm_batched": lambda **kw: s.gemm_batched(z(1, 4, 128), sx[None], values[None], meta[None], sw[None], **kw),
        "sp24_int8_compress": lambda **kw: s.compress_int8(z(256, 128, t=bf16), **kw),
        "sp24_int8_quantize_act": lambda **kw: s.quantize_act_int8(z(4, 128, t=f32), **kw),
        "sp24_int8_gemm": lambda **kw: s.gemm_int8(z(4, 128, t=i8), sx, values.to(i8), meta, sw, **kw),
    }


@pytest.mark.parametrize("current", [0, -1])
def test_linear_calls_work_on_the_operands_gpu(gpu, monkeypatch, current):
    gpu.current = current
    asked = []
    monkeypatch.setattr(s, "_dev_tensor", lambda t, *_: t)
    monkeypatch.setattr(torch.cuda, "current_stream",
                        lambda index=None: asked.append(index) or types.SimpleNamespace(cuda_stream=7, device_index=index))
    for name, call in linear_calls().items():
        call()
        assert gpu.lib.calls[-1] == (name, -1) and asked.pop() == -1
        done = len(gpu.lib.calls)
        with pytest.raises(ValueError):
            call(stream=types.SimpleNamespace(cuda_stream=7, device_index=0))
        assert name not in [n for n, _ in gpu.lib.calls[done:]]
    assert {at for _, at in gpu.lib.calls} == {-1} and len(gpu.lib.calls) == 13  # two calls of each GEMM ask for a size
    assert gpu.current == current


def test_memory_for_a_call_on_another_stream_is_that_streams(gpu, monkeypatch):
    """Outputs and zeroed workspaces of a call with `stream` are allocated (and zeroed) on it, not on the current one."""
    now, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        before, now[0] = now[0], stream
        yield
        now[0] = before

    def recorded(make):
        return lambda *a, **kw: made.append(now[0]) or make(*a, **kw)

    calls = {**linear_calls(), **attention_calls(cache())}
    monkeypatch.setattr(s, "_dev_tensor", lambda t, *_: t)
    monkeypatch.setattr(torch.cuda, "stream", on)
    side = types.SimpleNamespace(cuda_stream=7, device_index=-1)
    empty, zeros = torch.empty, torch.zeros
    monkeypatch.setattr(torch, "empty", recorded(empty))
    # (the calls' own inputs here are made with torch.zeros, too, but without a device)
    monkeypatch.setattr(torch, "zeros", lambda *a, **kw: (recorded(zeros) if "device" in kw else zeros)(*a, **kw))
    for name, call in calls.items():
        call(stream=side)
        assert made and all(x is side for x in made), name
        made.clear()
