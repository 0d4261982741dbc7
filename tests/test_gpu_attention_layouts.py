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
