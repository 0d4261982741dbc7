"""The example's layer, row by row: attention's own output of every decoded token, in steps and as one prompt (GPU)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# Both ways round the softmax weights and the result to bf16, errors of up to 2^-9 to 2^-8 of each weight and of the result
# that have no preferred sign: some 2^-8.5 / sqrt(3) each, 0.23 % of a row's norm each way, 0.33 % between them.  (The QKV rows are the same but for a
# bf16 rounding here and there, where the linear sums in another order for another number of tokens.)  One of the 62 keys
# that a row sees is 1/62 of the weight in the mean, about 1/62 |v| beside a row of 1.6 / sqrt(62) |v| (weights exp of
# scores with a deviation of 1): 8 % of the norm.
ROW = 0.01


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("width,heads,kv_heads,d", [(512, 14, 2, 64), (1024, 8, 4, 128)])
def test_every_decoded_row_agrees(sp24, e4m3, width, heads, kv_heads, d):
    spec = importlib.util.spec_from_file_location("attention_block", os.path.join(ROOT, "examples", "attention_block.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    torch.manual_seed(7)
    block = example.AttentionBlock(width, heads, kv_heads, d)
    prompts, steps, mask = [130, 1, 63], 70, dict(window=60, sinks=2)
    B, most = len(prompts), max(prompts) + steps
    hidden = [torch.randn(n + steps, width, device="cuda").bfloat16() for n in prompts]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    def prompt(pages, xs):
        """Attention of the rows `xs` of each sequence, in one call."""
        n = [len(x) for x in xs]
        at = torch.cat([torch.arange(m, device="cuda") for m in n])
        which = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(n, device="cuda"))
        q = block._heads(torch.cat(xs), pages.cache, at.int(), pages.slots(which, at))
        cu = torch.tensor([0] + n, device="cuda").cumsum(0).to(torch.int32)
        return sp24.attention_prompt(q, cu, pages.cache, pages.table, i32(n), **mask).split(n)

    pages = example.PagedCache(B, most, kv_heads, d, page_size=16, e4m3=e4m3)
    first = prompt(pages, [h[:n] for h, n in zip(hidden, prompts)])
    got = [[y] for y in first]
    rows = torch.arange(B, device="cuda")
    for i in range(steps):
        at = torch.tensor([n + i for n in prompts], device="cuda")
        x = torch.stack([h[n + i] for h, n in zip(hidden, prompts)])
        q = block._heads(x, pages.cache, at.int(), pages.slots(rows, at))
        y = sp24.attention_decode(q, pages.cache, pages.table, (at + 1).int(), **mask)
        for b in range(B):
            got[b].append(y[b:b + 1])
    want = prompt(example.PagedCache(B, most, kv_heads, d, page_size=16, e4m3=e4m3), hidden)
    sp24.last_device_error()
    for b in range(B):
        a, w = torch.cat(got[b]).double(), want[b].double()
        off = (a - w).norm(dim=-1) / w.norm(dim=-1)  # [tokens, heads]
        assert off.max() < ROW, "sequence %d: row %s off by %.3g" % (b, divmod(int(off.argmax()), heads), off.max())
