"""Prompt calls with more blocks than SMs, so that a CTA works through blocks of every kind, one after the other (GPU)."""
import random

import pytest
import torch

from attention_util import Setup, assert_attention, attend, sees

pytestmark = pytest.mark.gpu


def batch(seed, tok, sequences=110):
    """New tokens and earlier ones of each sequence, where a block takes up to 2 tok tokens: blocks with one and with two
    query tiles, of 1 to 9 key tiles, among rows that see nothing and sequences without new tokens."""
    rng = random.Random(seed)
    new, prefix = [], []
    for _ in range(sequences):
        kind = rng.randrange(8)
        m = rng.randint(1, tok) if kind < 4 else rng.randint(tok + 1, 2 * tok + 1)
        if kind == 3:
            m = 0
        new.append(m)
        prefix.append(-rng.randint(1, 2 * m + 1) if kind == 7 else rng.randint(0, 1100))
    return new, prefix


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 5), (3, 300)])
@pytest.mark.parametrize("hq,hkv,d,page,e4m3", [(4, 2, 128, 64, False), (8, 4, 64, 16, False), (4, 2, 128, 16, True),
                                                (8, 4, 64, 128, True)])
def test_blocks_of_all_kinds_in_turn(sp24, hq, hkv, d, page, e4m3, window, sinks):
    new, prefix = batch(1000 * d + window, 128 // (hq // hkv))
    lens = [max(0, a + b) for a, b in zip(new, prefix)]
    s = Setup(sp24, lens, hkv, d, page, e4m3, False, seed=d + window)
    see = [sees(torch.arange(n - m, n), n, window, sinks) for n, m in zip(lens, new)]
    s.poison([x.any(0) if x.shape[0] else torch.zeros(n, dtype=torch.bool) for x, n in zip(see, lens)])
    cache = s.upload()
    T = sum(new)
    q = (2 * torch.randn(T, hq, d, generator=torch.Generator().manual_seed(d))).to(torch.bfloat16)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    blocks = hkv * sum(-(-m // (2 * (128 // (hq // hkv)))) for m in new)
    assert blocks > torch.cuda.get_device_properties(0).multi_processor_count
    args = (q.cuda(), cu.cuda(), cache, s.table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda())
    y = sp24.attention_prompt(*args, window=window, sinks=sinks)
    for _ in range(5):  # whichever CTA takes a block
        assert torch.equal(sp24.attention_prompt(*args, window=window, sinks=sinks), y)
    sp24.last_device_error()
    for b, m in enumerate(new):
        rows = slice(int(cu[b]), int(cu[b + 1]))
        ref, size = attend(q[rows].double(), s.tokens("k", b), s.tokens("v", b), see[b], d ** -0.5)
        assert_attention(y[rows], ref, size, "sequence %d" % b)
