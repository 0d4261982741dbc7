"""The operators for a batch of many requests over strides and offsets past 32 bits (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

FAR = (1 << 31) + 64  # elements


@pytest.mark.parametrize("T", [5, 300, 600, 1100])
def test_adapters_and_rows_far_apart(sp24, T):
    """Adapters FAR apart, and rows so far apart that the last begin behind 2^31 elements: the same bits as packed ones."""
    K, N, r, count = 136, 72, 24, 2
    g = torch.Generator().manual_seed(T)
    x, y, a, b = (torch.randn(*s, generator=g).bfloat16().cuda() for s in ((T, K), (T, N), (count, r, K), (count, N, r)))
    ids = torch.randint(-1, count, (T,), generator=g).int().cuda()
    want = sp24.add_adapters(y, x, a, b, ids)
    step = (FAR // T + 1 + 7) // 8 * 8
    rows = torch.empty(T * step, dtype=torch.bfloat16, device="cuda")       # x and y in turn
    xv, yv = (torch.as_strided(rows, (T, c), (step, 1), at) for c, at in ((K, 0), (N, K)))
    stack = torch.empty(FAR + r * (K + N), dtype=torch.bfloat16, device="cuda")
    av = torch.as_strided(stack, (count, r, K), (FAR, K, 1), 0)
    bv = torch.as_strided(stack, (count, N, r), (FAR, r, 1), r * K)
    for view, values in ((xv, x), (yv, y), (av, a), (bv, b)):
        view.copy_(values)
    got = sp24.add_adapters(yv, xv, av, bv, ids, out=yv)
    sp24.last_device_error()
    assert torch.equal(got, want) and torch.equal(xv, x)


@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_far_apart(sp24, e4m3):
    """Tokens copied into pages that begin behind 2^31 elements, and attended there as shared ones: the same bits."""
    heads, page, d, pages, B = 2, 64, 64, 20, 70
    g = torch.Generator().manual_seed(7)
    n = pages * page
    kv = [torch.randn(pages, heads, page, d, generator=g) for _ in range(2)]
    scale = torch.full((heads,), 1 / 64).cuda() if e4m3 else None
    kv = [(x / scale[0].item()).to(torch.float8_e4m3fn).view(torch.uint8).cuda() if e4m3 else x.bfloat16().cuda() for x in kv]
    step = (FAR // (pages - 8) + 127) // 128 * 128
    room = torch.zeros(pages * step, dtype=kv[0].dtype, device="cuda")      # keys and values in turn
    far = [torch.as_strided(room, kv[0].shape, (step, page * d, d, 1), i * heads * page * d) for i in range(2)]
    scales = (scale, scale) if e4m3 else ()
    near_cache, far_cache = sp24.KVCache(*kv, *scales), sp24.KVCache(*far, *scales)
    slots = torch.randperm(n, generator=g).cuda()
    sp24.cache_copy(near_cache, slots, far_cache, slots)
    sp24.last_device_error()
    assert all(torch.equal(a, b) for a, b in zip(far, kv))
    q = torch.randn(B, 8, d, generator=g).bfloat16().cuda()
    width = 2 * pages if not e4m3 else 4 * pages                           # (columns that nobody reads: enough to share)
    table = torch.zeros(B, width, dtype=torch.int32)
    table[:, :pages] = torch.arange(pages)
    lens = torch.randint(n - 300, n, (B,), generator=g).int().cuda()
    cu, shared = torch.tensor([0, B]).int().cuda(), torch.tensor([n - 400]).int().cuda()
    y = [sp24.attention_decode_shared(q, c, table.cuda(), lens, cu, shared) for c in (near_cache, far_cache)]
    plain = sp24.attention_decode(q, near_cache, table.cuda(), lens)
    sp24.last_device_error()
    assert torch.equal(y[0], y[1])
    # Two bf16 results of one definition: within an ulp of each other, and the weights' rounding (2^-9 of a value of
    # at most 5, halved many times over in a sum of a thousand keys).
    assert (y[0].double() - plain.double()).abs().max() < 2.0 ** -8 * (plain.double().abs().max() + 1)
