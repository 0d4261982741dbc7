"""Tokens copied between caches against plain arithmetic (GPU)."""
import pytest
import torch

from attention_util import E4M3, Setup

pytestmark = pytest.mark.gpu


def expected(x, from_scale, to_scale):
    """x [T, heads, d] as the source holds it -> as the destination does.  Products and quotients of fp32 values, each
    rounded once to fp32 as the definition has it: 64-bit arithmetic gives them exactly enough to round (a product of
    24 and 4 bits is exact; a quotient of 24-bit numbers is never closer to a tie of fp32 than 2^-48 of it)."""
    if from_scale is not None:
        x = (x.contiguous().view(E4M3).double() * from_scale.double()[:, None]).float()
    if to_scale is None:
        return x.to(torch.bfloat16)
    q = (x.double() / to_scale.double()[:, None]).float()
    return q.clamp(-448, 448).to(E4M3).view(torch.uint8)


@pytest.mark.parametrize("T,heads,d,page,e4m3,token_major,to_page,to_e4m3,to_token_major", [
    (1, 1, 64, 16, False, False, 16, False, False),
    (1, 8, 128, 64, False, False, 64, True, False),
    (1, 8, 128, 64, True, False, 16, False, True),
    (15, 3, 64, 16, False, True, 32, True, False),
    (17, 5, 64, 32, True, False, 16, False, True),
    (64, 8, 128, 64, False, False, 64, False, False),
    (100, 7, 128, 128, True, True, 16, True, False),
    (333, 1, 128, 16, False, False, 128, True, True),
    (700, 2, 64, 64, True, True, 64, False, False),
    (3001, 4, 128, 64, False, True, 64, True, False),   # the many-token form
    (5003, 9, 64, 16, True, False, 32, False, False),
    (6000, 3, 64, 16, False, False, 64, False, True),
    (9001, 1, 128, 32, True, False, 64, True, True),
])
def test_copy(sp24, T, heads, d, page, e4m3, token_major, to_page, to_e4m3, to_token_major):
    s = Setup(sp24, [T + 5], heads, d, page, e4m3, token_major, seed=T)
    t = Setup(sp24, [T + 9], heads, d, to_page, to_e4m3, to_token_major, seed=T + 1)
    src, dst = s.upload(), t.upload()
    g = torch.Generator().manual_seed(T)
    i = torch.randperm(s.store["k"].shape[0] * page, generator=g)[:T]
    j = torch.randperm(t.store["k"].shape[0] * to_page, generator=g)[:T]
    if T > 10:
        i[3], j[7] = -1, -2                             # left out
    sp24.cache_copy(src, i.cuda(), dst, j.cuda())
    sp24.last_device_error()
    ok = (i >= 0) & (j >= 0)
    for name, got in (("k", dst.k.cpu()), ("v", dst.v.cpu())):
        want = t.store[name].clone()
        x = s.store[name].transpose(1, 2)[i[ok] // page, i[ok] % page]
        want.transpose(1, 2)[j[ok] // to_page, j[ok] % to_page] = expected(x, s.scale.get(name), t.scale.get(name))
        assert torch.equal(got.contiguous().view(torch.uint8), want.contiguous().view(torch.uint8)), name
    for name, x in (("k", src.k.cpu()), ("v", src.v.cpu())):
        assert torch.equal(x, s.store[name]), name + " of the source"


def test_special_values(sp24):
    """Values past the largest code saturate, NaN stays NaN, bf16 to bf16 keeps every bit; -0 stays -0."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).cuda()
    x = torch.zeros(8, 16, 8, 64, dtype=torch.bfloat16, device="cuda")
    x.view(-1)[:] = bits
    x = x.transpose(1, 2)                               # [8, 8 heads, 16, 64]
    one = torch.full((8,), 0.75, device="cuda")
    src = sp24.KVCache(x, x)
    slots = torch.arange(128, device="cuda")
    same = sp24.KVCache(torch.zeros_like(x), torch.zeros_like(x))
    sp24.cache_copy(src, slots, same, slots)
    assert torch.equal(same.k.view(torch.int16), x.view(torch.int16))
    code = torch.zeros(x.shape, dtype=torch.uint8, device="cuda")
    small = sp24.KVCache(code, torch.zeros_like(code), one, one)
    sp24.cache_copy(src, slots, small, slots)
    sp24.last_device_error()
    got, q = small.k.contiguous().view(E4M3).float().cpu(), (x.double() / 0.75).float().cpu()
    assert torch.equal(got.isnan(), q.isnan())
    fine = ~q.isnan()
    assert torch.equal(got[fine], q[fine].clamp(-448, 448).to(E4M3).float())
    # every code with its own scale: back and forth it stays what it is
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).repeat(64).view(2, 2, 64, 64).cuda()
    sc = torch.tensor([0.0371, 1.7], device="cuda")
    a = sp24.KVCache(codes, codes.clone(), sc, sc)
    b = sp24.KVCache(torch.zeros_like(codes), torch.zeros_like(codes), sc, sc)
    sp24.cache_copy(a, slots, b, slots)
    was, now = codes.view(E4M3).float(), b.v.view(E4M3).float()
    assert torch.equal(was.isnan(), now.isnan()) and torch.equal(was[~was.isnan()], now[~was.isnan()])


def test_within_one_cache_and_by_graph(sp24):
    """A page copied for a new sequence, inside one cache, replayed with other slots."""
    k = torch.randn(6, 2, 16, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
    cache = sp24.KVCache(k.clone(), -k)
    i, j = torch.arange(16, 30, device="cuda"), torch.arange(48, 62, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    sp24.cache_copy(cache, i, cache, j, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp24.cache_copy(cache, i, cache, j)
    j.add_(32)                                          # page 5
    graph.replay()
    sp24.last_device_error()
    want = k.clone()
    want[3, :, :14] = k[1, :, :14]
    want[5, :, :14] = k[1, :, :14]
    assert torch.equal(cache.k, want) and torch.equal(cache.v, -want)


def test_index_errors(sp24):
    k = torch.randn(3, 1, 16, 64).bfloat16().cuda()
    a, b = sp24.KVCache(k, k), sp24.KVCache(torch.zeros_like(k), torch.zeros_like(k))
    i64 = lambda *v: torch.tensor(v, dtype=torch.int64, device="cuda")  # noqa: E731
    for i, j in ((i64(48, 1), i64(0, 2)), (i64(0, 1), i64(1 << 40, 2)), (i64(1 << 62, 1), i64(0, 2))):
        sp24.cache_copy(a, i, b, j)
        with pytest.raises(sp24.Sp24Error) as e:
            sp24.last_device_error()
        assert e.value.status == 8
        want = torch.zeros_like(k)
        want[0, :, 2] = k[0, :, 1]                      # the other token is copied
        assert torch.equal(b.k, want)
    sp24.cache_copy(a, i64(-1, 0), b, i64(5, -9))       # left out: no error
    sp24.cache_copy(a, i64(), b, i64())
    sp24.last_device_error()
