"""A process whose first call of an operator is captured into a graph (GPU): what is asked of the driver once, on a
kernel's first launch, must not break the capture."""
import subprocess
import sys
from pathlib import Path

import pytest

pytestmark = pytest.mark.gpu

CHILD = """
import sys
import torch
import semi_structured_sparse_gb300 as sp24

what = sys.argv[1]
g = torch.Generator(device="cuda").manual_seed(1)
n = lambda *s: torch.randn(*s, device="cuda", generator=g).bfloat16()
if what == "shared":
    B, tokens = 64, 2048
    k, v = n(tokens // 64, 4, 64, 128), n(tokens // 64, 4, 64, 128)
    cache = sp24.KVCache(k, v)
    q, table = n(B, 8, 128), torch.arange(tokens // 64, device="cuda").int().expand(B, -1).contiguous()
    lens, cu, shared = (torch.tensor(x, device="cuda").int() for x in ([tokens] * B, [0, B], [tokens - 100]))
    call = lambda: sp24.attention_decode_shared(q, cache, table, lens, cu, shared)
elif what == "copy":
    k = n(8, 2, 16, 64)
    to = torch.zeros_like(k)
    cache, other = sp24.KVCache(k, n(8, 2, 16, 64)), sp24.KVCache(to, torch.zeros_like(k))
    slots = torch.arange(128, device="cuda")
    call = lambda: (sp24.cache_copy(cache, slots, other, slots), to)[1]
else:
    T = int(what)
    x, y, a, b = n(T, 256), n(T, 136), n(5, 16, 256) / 16, n(5, 136, 16) / 16
    ids = torch.randint(-1, 5, (T,), device="cuda", generator=g).int()
    call = lambda: sp24.add_adapters(y, x, a, b, ids)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = call()
graph.replay()
torch.cuda.synchronize()
got = captured.clone()
assert torch.isfinite(got.float()).all() and got.float().abs().sum() > 0
assert torch.equal(got, call())
sp24.last_device_error()
"""


@pytest.mark.parametrize("what", ["shared", "copy", "7", "300", "1100"])
def test_first_call_in_a_capture(what):
    root = Path(__file__).resolve().parents[1]
    r = subprocess.run([sys.executable, "-c", CHILD, what], cwd=root, capture_output=True, text=True, timeout=240)
    assert r.returncode == 0, r.stderr[-2000:]
