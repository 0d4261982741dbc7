"""The prompt kernel's give-up paths, exercised without faulting or hanging the GPU.

The fault-test copy of the library (bounded waits of 1 ms) copies nothing for each CTA's first tile of keys, so the waits
of the MMA, softmax, conversion and copy warps run out one after the other: copies in flight land, tensor memory is freed,
the launch ends, and the device error word says so.  In a child process; the parent then checks that the library proper
still computes the definition."""
import json
import subprocess
import sys

import pytest
import torch

from attention_util import Setup, assert_attention, attend, sees

pytestmark = pytest.mark.gpu

SP24_ERR_DEVICE_TIMEOUT = 7

CHILD = r"""
import json, sys
import torch
import semi_structured_sparse_gb300 as s
s._build.LIB = sys.argv[1]
s.load(build_if_missing=False)

def status():
    try:
        s.last_device_error()
    except s.Sp24Error as e:
        return e.status
    return 0

out = []
for d in (64, 128):
    for e4m3 in (False, True):
        kv = torch.zeros(2, 40, 2, 64, d, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
        one = torch.ones(2, device="cuda") if e4m3 else None
        cache = s.KVCache(kv[0], kv[1], one, one)
        # one call with a block per SM at most, one with several
        for new in ([300, 10], [90, 200] * 60):
            B = len(new)
            cu = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
            table = torch.arange(20, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
            lens = torch.full((B,), 1100, dtype=torch.int32, device="cuda")
            q = torch.zeros(sum(new), 4, d, dtype=torch.bfloat16, device="cuda")
            s.attention_prompt(q, cu, cache, table, lens)
            out.append([status(), status()])
ok = torch.arange(1000, device="cuda", dtype=torch.float32).sum().item() == 499500.0
print(json.dumps({"status": out, "context_ok": ok}))
"""


def test_prompt_waits_that_run_out_are_reported(sp24):
    from semi_structured_sparse_gb300 import build as b
    fault_lib = b.build_fault_test()
    assert fault_lib != b.LIB
    r = subprocess.run([sys.executable, "-c", CHILD, fault_lib], capture_output=True, text=True, timeout=300, cwd=b.ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["status"] == [[SP24_ERR_DEVICE_TIMEOUT, 0]] * 8  # reported once, and cleared
    assert out["context_ok"]

    s = Setup(sp24, [300], 2, 128, 64, False, False, seed=3)
    cache = s.upload()
    q = torch.randn(300, 4, 128, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    y = sp24.attention_prompt(q.cuda(), i32(0, 300), cache, s.table.cuda(), i32(300))
    sp24.last_device_error()
    ref, size = attend(q.double(), s.tokens("k", 0), s.tokens("v", 0), sees(torch.arange(300), 300, 0, 0), 128 ** -0.5)
    assert_attention(y, ref, size, "library proper")
