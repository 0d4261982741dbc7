"""The operators for a batch of many requests in a run, as a served layer uses them (GPU)."""
import importlib.util
import os

import pytest
import torch

from attention_util import E4M3, assert_attention, attend
from test_gpu_adapters import assert_adapted, reference

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("cache,kw", [
    ("bf16", {}),
    ("e4m3", {}),
    ("bf16", dict(width=512, heads=14, kv_heads=2, head_dim=64, requests=70, instruction=2501, page_size=16, rank=24)),
])
def test_shared_steps_agree_with_steps_one_by_one(sp24, cache, kw):
    """Captured and replayed decode steps whose shared tokens are read once, and those in which each sequence has its own
    copy of them.  The two differ as in test_gpu_attention_block: by roundings of attention's output, and by steps of
    e4m3 activations that these move here and there; 3 % of the norm is far above that and far below a missed token."""
    assert example().run_shared(cache, report=lambda *_: None, **dict(dict(steps=6), **kw)) < 0.03


@pytest.mark.parametrize("e4m3", [False, True])
def test_every_stage_of_a_step(sp24, e4m3):
    """Instruction tokens copied (and quantised), adapters on the QKV rows, append, attention behind the shared tokens,
    adapters on the output rows: each stage against its definition, from the stage's own inputs."""
    B, heads, kv, d, page, n, width, rank = 40, 8, 2, 64, 16, 1237, 256, 16
    g = torch.Generator().manual_seed(8)
    rows = (heads + 2 * kv) * d
    bf = lambda *s, by=1.0: (torch.randn(*s, generator=g) * by).bfloat16().cuda()  # noqa: E731
    once = sp24.KVCache(bf(n // page + 1, kv, page, d), bf(n // page + 1, kv, page, d))
    full, wide = n // page, 9000            # tables wide enough for sharing to be worth it
    pages = full + 2 * B
    shape = (pages, kv, page, d)
    scale = torch.tensor([0.031, 0.045], device="cuda") if e4m3 else None
    store = [torch.zeros(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda") for _ in range(2)]
    cache = sp24.KVCache(store[0], store[1], scale, scale)
    table = torch.zeros(B, wide, dtype=torch.int32)
    table[:, :full] = torch.arange(full)
    table[:, full] = full + torch.arange(B)
    table[:, full + 1] = full + B + torch.arange(B)
    at = torch.arange(n)
    tail = at[full * page:]
    to = torch.cat((at[:full * page], (table[:, full, None] * page + tail % page).flatten())).long().cuda()
    of = torch.cat((at[:full * page], tail.repeat(B))).cuda()
    sp24.cache_copy(once, of, cache, to)

    x, ids = bf(B, width), torch.randint(-1, 5, (B,), generator=g, dtype=torch.int32)
    projected = bf(B, rows)
    a, b = bf(5, rank, width, by=width ** -0.5), bf(5, rows, rank, by=rank ** -0.5)
    qkv = sp24.add_adapters(projected, x, a, b, ids.cuda())
    assert_adapted(qkv, *reference(projected.cpu(), x.cpu(), a.cpu(), b.cpu(), ids, None), "qkv")

    angle = torch.rand(n + 1, d // 2, generator=g) * 6.28
    positions = torch.full((B,), n, dtype=torch.int32, device="cuda")
    slots = (table[:, n // page].long() * page + n % page).cuda()
    q = sp24.qk_norm_rope(qkv, heads, cache, positions, slots, torch.cat((angle.cos(), angle.sin()), 1).cuda())
    lens = torch.full((B,), n + 1, dtype=torch.int32, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    y = sp24.attention_decode_shared(q, cache, table.cuda(), lens, i32(0, B), i32(n))
    sp24.last_device_error()

    def tokens(t, s, i):
        v = t.cpu()[table[i, :full + 2].long()].transpose(1, 2).reshape(-1, kv, d)[:n + 1]
        return v.view(E4M3).double() * s.double().cpu()[:, None] if e4m3 else v.double()
    for i in range(B):
        k, v = tokens(cache.k, scale, i), tokens(cache.v, scale, i)
        # the shared tokens are the instruction's
        was = once.v.cpu().transpose(1, 2).reshape(-1, kv, d)[:n].double()
        step = (2.0 ** -4 * was.abs()).clamp(min=2.0 ** -10 * 0.045) if e4m3 else 0.0 * was
        assert ((v[:n] - was).abs() <= step * (1 + 2.0 ** -18)).all()
        want, size = attend(q[i:i + 1].double().cpu(), k, v, torch.ones(1, n + 1, dtype=torch.bool), d ** -0.5)
        assert_attention(y[i:i + 1], want, size, "sequence %d" % i)

    a2, b2 = bf(5, rank, heads * d, by=(heads * d) ** -0.5), bf(5, width, rank, by=rank ** -0.5)
    out = bf(B, width)
    before = out.clone()
    sp24.add_adapters(out, y.flatten(1), a2, b2, ids.cuda(), out=out)
    assert_adapted(out, *reference(before.cpu(), y.flatten(1).cpu(), a2.cpu(), b2.cpu(), ids, None), "out")
