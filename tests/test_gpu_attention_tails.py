"""Many keys whose weights are small beside one key's still count, in either cache (GPU)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def setup(sp24, n, strong, d, page, e4m3):
    """One sequence of n keys: one with k = (1, 0, ...) and v = 0, all others with k = 0 and v = 1."""
    pages = -(-n // page)
    one = 0x38 if e4m3 else 1.0  # 0x38: the e4m3 code of 1
    k, v = (torch.zeros(pages, 1, page, d, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda") for _ in "kv")
    v.fill_(one)
    v[strong // page, 0, strong % page] = 0
    k[strong // page, 0, strong % page, 0] = one
    scale = torch.ones(1, device="cuda") if e4m3 else None
    return sp24.KVCache(k, v, scale, scale), torch.arange(pages, dtype=torch.int32, device="cuda")[None]


# A weight enters the tensor core rounded by up to 2^-8 of itself (bf16: 8 bits), or 2^-11 (f16), whose smallest step rounds
# it by up to 2^-25 besides.  The largest weight is 2^15 in a decode step (a step of 2^-40 of it) and at least 2^7 in a prompt
# (2^-32).  fp32 scores of 30 are off by 30 x 2^-23 at most, so exponentials by less than 2^-16; the result is rounded by
# 2^-8 of it.
def assert_tail(y, others, gap, e4m3, step, what):
    tail = others.double() * math.exp(-gap)
    want = (tail / (1 + tail)).view(-1, 1, 1)
    bound = (2.0 ** -8 * 1.02 + (2.0 ** -11 if e4m3 else 2.0 ** -8) + 2.0 ** -15) * want
    if e4m3:
        bound = bound + (others.double() * step).view(-1, 1, 1)
    off = ((y.double().cpu() - want).abs() / bound).max()
    assert off <= 1, "%s: %.3g times the bound" % (what, off)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,page", [(64, 16), (128, 64)])
@pytest.mark.parametrize("gap", [10.0, 14.0, 17.0, 17.375, 20.0, 24.0, 30.0])
def test_small_weights_count(sp24, d, page, e4m3, gap):
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    for n, strong in ((3001, 0), (3001, 1500), (3001, 2990), (100003, 50000)):
        cache, table = setup(sp24, n, strong, d, page, e4m3)
        q = torch.zeros(9, 3, d, dtype=torch.bfloat16, device="cuda")
        q[:, :, 0] = gap
        # 400 sequences of the same pages: each is one CTA's, so that a quarter of its keys share a warp with the one
        many = table.expand(400, -1).contiguous()
        y = sp24.attention_decode(q[:1].expand(400, -1, -1).contiguous(), cache, many, i32(*[n] * 400), scale=1.0)
        assert_tail(y, torch.full((400,), n - 1), gap, e4m3, 2.0 ** -40, "decode of %d, key %d" % (n, strong))
        rows = torch.arange(n - 9, n)
        for ws in (None, torch.empty(0, dtype=torch.uint8, device="cuda")):  # cut into parts, and not
            y = sp24.attention_prompt(q, i32(0, 9), cache, table, i32(n), scale=1.0, workspace=ws)
            assert_tail(y, rows, gap, e4m3, 2.0 ** -32, "prompt over %d, key %d" % (n, strong))
    sp24.last_device_error()
