"""The give-up paths of the kernels for a batch of many requests, exercised without faulting or hanging the GPU.

The fault-test copy of the library (bounded waits of 1 ms) copies nothing for each CTA's first stage, so the waits of all
roles run out: copies in flight land, tensor memory is freed, the launches end, and the device error word says so.  In a
child process; the parent then checks that the library proper still computes the definition."""
import json
import subprocess
import sys

import pytest
import torch

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
for r in (16, 64, 128):
    for T in (1100, 5000):
        z = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        ids = (torch.arange(T, device="cuda") // 100 % 3).to(torch.int32)
        s.add_adapters(z(T, 512), z(T, 1024), z(3, r, 1024), z(3, 512, r), ids)
        out.append([status(), status()])
for d in (64, 128):
    for e4m3 in (False, True):
        kv = torch.zeros(2, 4000, 2, 16, d, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")
        one = torch.ones(2, device="cuda") if e4m3 else None
        cache = s.KVCache(kv[0], kv[1], one, one)
        for B in (9, 300):
            i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
            table = torch.arange(4000, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
            lens = torch.full((B,), 20000, dtype=torch.int32, device="cuda")
            q = torch.zeros(B, 4, d, dtype=torch.bfloat16, device="cuda")
            s.attention_decode_shared(q, cache, table, lens, i32(0, B), i32(19000))
            out.append([status(), status()])
ok = torch.arange(1000, device="cuda", dtype=torch.float32).sum().item() == 499500.0
print(json.dumps({"status": out, "context_ok": ok}))
"""


def test_waits_that_run_out_are_reported(sp24):
    from semi_structured_sparse_gb300 import build as b
    fault_lib = b.build_fault_test()
    assert fault_lib != b.LIB
    r = subprocess.run([sys.executable, "-c", CHILD, fault_lib], capture_output=True, text=True, timeout=300, cwd=b.ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    out = json.loads(r.stdout.strip().splitlines()[-1])
    assert out["status"] == [[SP24_ERR_DEVICE_TIMEOUT, 0]] * 14  # reported once, and cleared
    assert out["context_ok"]

    from test_gpu_adapters import assert_adapted, inputs, reference
    y, x, a, b_, scales = inputs(1100, 256, 136, 16, 2, seed=1)
    ids = torch.arange(1100, dtype=torch.int32) // 100 % 2
    got = sp24.add_adapters(*(t.cuda() for t in (y, x, a, b_, ids, scales)))
    sp24.last_device_error()
    assert_adapted(got, *reference(y, x, a, b_, ids, scales), "library proper")
