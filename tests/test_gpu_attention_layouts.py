"""Valid layouts of the attention calls' arguments that are easily refused (GPU)."""
import pytest
import torch

from attention_util import Setup

pytestmark = pytest.mark.gpu


def test_a_page_table_of_one_column(sp24):
    """With one page per sequence no row of the table is stepped along, so its column stride may be anything."""
    s = Setup(sp24, [13, 16, 2], 2, 64, 16, False, False, seed=91)
    cache = s.upload()
    lens = torch.tensor(s.lens, dtype=torch.int32, device="cuda")
    q = torch.randn(3, 4, 64, generator=torch.Generator().manual_seed(92)).to(torch.bfloat16).cuda()
    cu = torch.arange(4, dtype=torch.int32, device="cuda")
    table = s.table.cuda()
    column = table.view(1, 3).clone().T
    assert column.shape == (3, 1) and column.stride() == (1, 3) and table.stride() == (1, 1)
    for t in (column, torch.stack((table[:, 0], table[:, 0]), 1)[:, :1]):
        assert torch.equal(sp24.attention_decode(q, cache, t, lens), sp24.attention_decode(q, cache, table, lens))
        assert torch.equal(sp24.attention_prompt(q, cu, cache, t, lens), sp24.attention_prompt(q, cu, cache, table, lens))
    wide = torch.zeros(2, 3, dtype=torch.int32, device="cuda").T  # two columns do have to be next to each other
    for call in (lambda: sp24.attention_decode(q, cache, wide, lens),
                 lambda: sp24.attention_prompt(q, cu, cache, wide, lens)):
        with pytest.raises(ValueError):
            call()
    sp24.last_device_error()


def test_keys_and_values_that_differ_in_a_lone_axis_stride(sp24):
    """With one kv head, pages of tokens and pages of heads are the same memory: k may be one and v the other."""
    s = Setup(sp24, [40, 7], 1, 64, 16, False, False, seed=93)
    cache, table = s.upload(), s.table.cuda()
    lens = torch.tensor(s.lens, dtype=torch.int32, device="cuda")
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(94)).to(torch.bfloat16).cuda()
    want = sp24.attention_decode(q, cache, table, lens)
    k = cache.k.transpose(1, 2).clone(memory_format=torch.contiguous_format).transpose(1, 2)
    assert k.stride(1) != cache.v.stride(1)
    assert torch.equal(sp24.attention_decode(q, sp24.KVCache(k, cache.v), table, lens), want)
    one = sp24.KVCache(k[:1].as_strided((1, 1, 16, 64), (5, 7, 64, 1)), cache.v[:1])
    first = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    assert torch.equal(sp24.attention_decode(q[:1], one, first, lens[1:]),
                       sp24.attention_decode(q[:1], cache, first, lens[1:]))
    two = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16, device="cuda")  # a stride that is stepped along does count
    with pytest.raises(ValueError):
        sp24.KVCache(two, two.transpose(1, 2).contiguous().transpose(1, 2))
    sp24.last_device_error()
