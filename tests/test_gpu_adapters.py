"""Low-rank adapters of many requests against their definition in 64 bits (GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def inputs(T, K, N, r, count, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    x, y = n(T, K + pad)[:, :K], n(T, N + pad)[:, :N]
    a = (torch.randn(count, r, K, generator=g) * K ** -0.5).bfloat16()
    b = (torch.randn(count, N, r, generator=g) * r ** -0.5).bfloat16()
    return y, x, a, b, torch.rand(count, generator=g) + 0.5


def reference(y, x, a, b, ids, scales):
    """(out, sum of the magnitudes that were added up) in 64 bits."""
    out, size = y.double(), torch.zeros(y.shape, dtype=torch.float64)
    for i in set(ids.tolist()):
        if i < 0 or i >= a.shape[0]:
            continue
        rows = ids == i
        h, hs = x[rows].double() @ a[i].double().T, x[rows].double().abs() @ a[i].double().abs().T
        s = 1.0 if scales is None else float(scales[i])
        out[rows] += s * (h @ b[i].double().T)
        size[rows] += abs(s) * (hs @ b[i].double().abs().T)
    return out, size


# bf16's half an ulp is at most 2^-8 of the result.  Within, as a share of the sum of magnitudes: fp32 sums in chains of
# at most 128 additions, each off by 2^-23 of the sum so far at most (a tensor core may cut off instead of rounding),
# 2^-16; A x in two bf16 parts, each within 2^-8 of what it stands for, 2^-16; the second product's 17 additions, 2^-18.
def assert_adapted(got, out, size, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), what + ": not finite"
    bound = 2.0 ** -8 * out.abs() * (1 + 2.0 ** -7) + (2.0 ** -15 + 2.0 ** -18) * size + 1e-30
    err = (got - out).abs()
    bad = err > bound
    assert not bad.any(), "%s: %d of %d outside the bound, worst %.3g of it at %s" % (
        what, int(bad.sum()), bad.numel(), float((err / bound).max()), bad.nonzero()[0].tolist())


def ids_of(T, count, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "any":
        return torch.randint(-1, count, (T,), generator=g, dtype=torch.int32)
    if kind == "runs":
        out = torch.empty(0, dtype=torch.int64)
        while len(out) < T:
            out = torch.cat((out, torch.randint(-1, count, (1,), generator=g).repeat(int(torch.randint(1, 90, (1,), generator=g)))))
        return out[:T].to(torch.int32)
    if kind == "none":
        return torch.full((T,), -3, dtype=torch.int32)
    return torch.full((T,), count - 1, dtype=torch.int32)


@pytest.mark.parametrize("T,K,N,r,count,kind", [
    (1, 8, 8, 8, 1, "one"),
    (1, 4096, 4096, 16, 3, "one"),
    (1, 128, 256, 128, 1, "none"),
    (2, 136, 72, 24, 2, "any"),
    (7, 1000, 520, 8, 4, "any"),          # no multiple of 16 anywhere
    (8, 264, 8, 40, 8, "any"),
    (9, 8, 1032, 16, 3, "any"),
    (17, 4096, 1024, 64, 20, "any"),
    (33, 520, 2056, 72, 5, "runs"),
    (64, 2048, 3080, 16, 64, "any"),
    (65, 14336, 256, 32, 6, "any"),
    (100, 1024, 1024, 128, 7, "runs"),
    (257, 512, 776, 56, 9, "any"),
    (300, 2048, 512, 64, 1, "one"),
    (700, 1032, 1032, 16, 6, "runs"),     # two blocks of rows
    (513, 136, 200, 128, 30, "any"),
    (1024, 520, 264, 48, 12, "any"),
    (1025, 520, 264, 48, 12, "any"),      # the many-row form
    (1100, 1032, 1032, 16, 6, "runs"),
    (1200, 64, 64, 32, 2, "none"),
    (1030, 256, 2048, 104, 40, "any"),
    (1500, 3000, 640, 8, 3, "runs"),
    (2049, 640, 1000, 128, 5, "runs"),
    (600, 64, 64, 32, 2, "none"),
])
@pytest.mark.parametrize("scaled", [True, False])
def test_add_adapters(sp24, T, K, N, r, count, kind, scaled):
    y, x, a, b, scales = inputs(T, K, N, r, count, seed=T + K)
    ids = ids_of(T, count, kind, T)
    s = scales if scaled else None
    got = sp24.add_adapters(y.cuda(), x.cuda(), a.cuda(), b.cuda(), ids.cuda(), None if s is None else s.cuda())
    sp24.last_device_error()
    assert got.shape == (T, N) and got.dtype == torch.bfloat16
    out, size = reference(y, x, a, b, ids, s)
    assert_adapted(got, out, size, "adapters")
    bare = ids < 0
    assert torch.equal(got.cpu()[bare], y[bare])        # rows without an adapter keep every bit


@pytest.mark.parametrize("T", [5, 40, 900, 1300])
def test_strides_in_place_and_bounds(sp24, T):
    """Rows and adapters further apart than their length; the result in place; nothing else is written, and NaN in what
    belongs to no row's adapter, or lies between, reaches no result."""
    K, N, r, count = 520, 264, 24, 6
    y, x, a, b, scales = inputs(T, K, N, r, count, seed=T)
    ids = ids_of(T, count, "runs" if T > 100 else "any", T)
    ids[ids == 4] = 2                                   # nobody's
    nan = float("nan")
    xb, yb = torch.full((T + 2, K + 40), nan), torch.full((T + 2, N + 16), nan)
    xb[1:T + 1, 16:16 + K], yb[1:T + 1, 8:8 + N] = x.float(), y.float()
    ab, bb = torch.full((count, r * K + 64), nan), torch.full((count, N * r + 8), nan)
    ab[:, :r * K], bb[:, :N * r] = a.float().flatten(1), b.float().flatten(1)
    ab[4], bb[4] = nan, nan
    xd, yd, ad, bd = (t.bfloat16().cuda() for t in (xb, yb, ab, bb))
    av = torch.as_strided(ad, (count, r, K), (r * K + 64, K, 1))
    bv = torch.as_strided(bd, (count, N, r), (N * r + 8, r, 1))
    yv = yd[1:T + 1, 8:8 + N]
    sc = scales.cuda()
    sc[4] = nan
    got = sp24.add_adapters(yv, xd[1:T + 1, 16:16 + K], av, bv, ids.cuda(), sc, out=yv)
    sp24.last_device_error()
    assert got is yv
    out, size = reference(y, x, a, b, ids, scales)
    assert_adapted(got, out, size, "in place")
    rest = yd.clone()
    rest[1:T + 1, 8:8 + N] = nan
    assert rest.isnan().all()


def test_a_row_that_is_not_finite_keeps_to_itself(sp24):
    for T in (20, 800, 1200):
        y, x, a, b, scales = inputs(T, 256, 136, 16, 2, seed=T)
        ids = torch.zeros(T, dtype=torch.int32)
        ids[1::3] = 1
        clean = sp24.add_adapters(y.cuda(), x.cuda(), a.cuda(), b.cuda(), ids.cuda())
        x[7, 3] = float("inf")
        y[9, 5] = float("nan")
        got = sp24.add_adapters(y.cuda(), x.cuda(), a.cuda(), b.cuda(), ids.cuda())
        sp24.last_device_error()
        assert not torch.isfinite(got[7].float()).any() and got[9, 5].isnan()
        keep = torch.ones(T, 136, dtype=torch.bool)
        keep[7], keep[9, 5] = False, False
        assert torch.equal(got.cpu()[keep], clean.cpu()[keep])


@pytest.mark.parametrize("T", [1, 48, 700, 1100])
def test_the_same_every_time_streams_and_graphs(sp24, T):
    y, x, a, b, scales = inputs(T, 1024, 520, 32, 5, seed=T)
    ids = ids_of(T, 5, "any", 1)
    yd, xd, ad, bd, sd, idd = (t.cuda() for t in (y, x, a, b, scales, ids))
    first = sp24.add_adapters(yd, xd, ad, bd, idd, sd)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    on_side = sp24.add_adapters(yd, xd, ad, bd, idd, sd, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, on_side)
    out = torch.empty_like(yd)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sp24.add_adapters(yd, xd, ad, bd, idd, sd, out=out)
    graph.replay()
    assert torch.equal(first, out)
    other = ids_of(T, 5, "any", 2)
    idd.copy_(other)
    graph.replay()
    sp24.last_device_error()
    want, size = reference(y, x, a, b, other, scales)
    assert_adapted(out, want, size, "replayed with other adapters")


def test_ids_out_of_range(sp24):
    for T in (6, 600, 1100):
        y, x, a, b, _ = inputs(T, 64, 72, 8, 2, seed=T)
        ids = torch.zeros(T, dtype=torch.int32)
        ids[3], ids[4] = 2, 2 ** 31 - 1
        got = sp24.add_adapters(y.cuda(), x.cuda(), a.cuda(), b.cuda(), ids.cuda())
        with pytest.raises(sp24.Sp24Error) as e:
            sp24.last_device_error()
        assert e.value.status == 8
        out, size = reference(y, x, a, b, ids, None)
        assert_adapted(got, out, size, "bad ids")
        assert torch.equal(got.cpu()[3:5], y[3:5])


def test_no_rows(sp24):
    y, x, a, b, _ = inputs(3, 64, 72, 8, 2, seed=1)
    got = sp24.add_adapters(y.cuda()[:0], x.cuda()[:0], a.cuda(), b.cuda(), torch.zeros(0, dtype=torch.int32, device="cuda"))
    sp24.last_device_error()
    assert got.shape == (0, 72)


@pytest.mark.parametrize("T,K,N,r,count", [(2300, 1088, 1600, 64, 9), (4000, 512, 2112, 24, 5), (1700, 2112, 1024, 128, 7)])
def test_tiles_of_several_adapters_again_and_again(sp24, T, K, N, r, count):
    """Runs that end inside a tile, so that its rows have two, three and more adapters, beside tiles of one and of none:
    the same bits every time."""
    y, x, a, b, scales = inputs(T, K, N, r, count, seed=r)
    g = torch.Generator().manual_seed(r)
    ids = torch.cat([torch.randint(-1, count, (1,), generator=g).repeat(n) for n in (3, 500, 37, 41, 600, 50, 1, 2, 60, 300,
                                                                                     90, 45, 30, 25, 700, 2000)])
    ids = ids[:T].to(torch.int32)
    args = [t.cuda() for t in (y, x, a, b, ids, scales)]
    first = sp24.add_adapters(*args)
    out, size = reference(y, x, a, b, ids, scales)
    assert_adapted(first, out, size, "several adapters")
    workspace = torch.empty(sp24.add_adapters_workspace_size(T, K, r), dtype=torch.uint8, device="cuda")
    for _ in range(30):
        again = sp24.add_adapters(*args, workspace=workspace)
        assert torch.equal(first, again)
    sp24.last_device_error()


def test_workspace(sp24):
    y, x, a, b, scales = (t.cuda() for t in inputs(1100, 256, 136, 16, 2, seed=1))
    ids = torch.zeros(1100, dtype=torch.int32, device="cuda")
    need = sp24.add_adapters_workspace_size(1100, 256, 16)
    assert need > 0 and sp24.add_adapters_workspace_size(1024, 256, 16) == 0
    short = torch.empty(need - 16, dtype=torch.uint8, device="cuda")
    with pytest.raises(sp24.Sp24Error, match="WORKSPACE"):
        sp24.add_adapters(y, x, a, b, ids, workspace=short)
    with pytest.raises(ValueError, match="unit stride"):
        sp24.add_adapters(y, x, a, b, ids, workspace=torch.empty(2 * need, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(ValueError, match="alignment|ALIGNMENT"):
        sp24.add_adapters(y, x, a, b, ids, workspace=torch.empty(need + 16, dtype=torch.uint8, device="cuda")[1:])


@pytest.mark.parametrize("T,K,N,r,count", [
    (513, 264, 136, 24, 31),       # the last row's block has no other
    (1023, 520, 264, 16, 300),
    (1025, 264, 136, 24, 31),      # the last row's tile has no other
    (1300, 520, 264, 16, 300),     # two bytes of ids
    (1100, 1032, 1096, 40, 90),
    (2175, 256, 328, 72, 2),       # two adapters in turn
    (8191, 72, 200, 8, 20),
    (8193, 64, 136, 16, 6),        # one row in a window of its own
    (20000, 64, 72, 8, 70000),     # three bytes, most adapters nobody's
])
def test_many_rows_in_no_order(sp24, T, K, N, r, count):
    """Adapters scattered over the rows, some rows without one and one id out of range; in place and not, the same bits
    every time."""
    y, x, a, b, scales = inputs(T, K, N, r, min(count, 300), seed=T)
    used = torch.randint(0, count, (300,), generator=torch.Generator().manual_seed(T))
    if count > 300:                                     # 300 different ones
        a = a[torch.arange(count) % 300]
        b = b[torch.arange(count) % 300]
        scales = scales[torch.arange(count) % 300]
    ids = ids_of(T, count, "any", T)
    if count == 2:
        ids = (torch.arange(T) % 2).to(torch.int32)
    if count == 70000:
        ids = torch.where(ids < 0, ids, used[torch.arange(T) % 300].to(torch.int32))
    ids[T // 2] = count
    args = [t.cuda() for t in (y, x, a, b, ids, scales)]
    first = sp24.add_adapters(*args)
    with pytest.raises(sp24.Sp24Error) as e:
        sp24.last_device_error()
    assert e.value.status == 8
    out, size = reference(y, x, a, b, torch.where(ids == count, -1, ids), scales)
    assert_adapted(first, out, size, "scattered")
    bare = (ids < 0) | (ids == count)
    assert torch.equal(first.cpu()[bare], y[bare])
    for _ in range(5):
        again = args[0].clone()
        sp24.add_adapters(again, *args[1:], out=again)
        assert torch.equal(first, again)
    with pytest.raises(sp24.Sp24Error):
        sp24.last_device_error()


@pytest.mark.parametrize("r", [16, 80])
@pytest.mark.parametrize("first", [True, False])
def test_rows_in_order_beside_rows_in_none(sp24, first, r):
    """Tiles that stay as they are beside tiles put together from everywhere, and windows that are sorted beside ones
    that are not."""
    T, K, N, count = 9300, 136, 200, 460
    g = torch.Generator().manual_seed(5)
    short = torch.arange(2000) // 5                       # in order, but in short runs
    mixed = torch.randint(400, count, (6192,), generator=g)
    runs = torch.arange(T - 8192) // 300
    ids = torch.cat((short, mixed, runs) if first else (mixed, short, runs)).to(torch.int32)
    y, x, a, b, scales = inputs(T, K, N, r, count, seed=6)
    args = [t.cuda() for t in (y, x, a, b, ids, scales)]
    got = sp24.add_adapters(*args)
    sp24.last_device_error()
    out, size = reference(y, x, a, b, ids, scales)
    assert_adapted(got, out, size, "in order and in none")
    again = args[0].clone()
    assert torch.equal(got, sp24.add_adapters(again, *args[1:], out=again))


@pytest.mark.parametrize("K", [64, 1000])
@pytest.mark.parametrize("r", [16, 104])
def test_tiles_of_very_different_cost(sp24, K, r):
    """One tile of 128 adapters, some of few, some of none: every part of every sum is there."""
    T, N, count = 8192 + 640, 136, 140
    ids = torch.full((T,), 3)
    ids[1280:1408] = torch.arange(128)
    ids[2000:4000] = -1
    ids[4100:4110] = torch.arange(10) + 128
    ids[8000:8300] = 139
    ids = ids.to(torch.int32)
    y, x, a, b, scales = inputs(T, K, N, r, count, seed=r + K)
    args = [t.cuda() for t in (y, x, a, b, ids, scales)]
    need = sp24.add_adapters_workspace_size(T, K, r)
    workspace = torch.full((need,), 255, dtype=torch.uint8, device="cuda")   # parts that nobody writes are no numbers
    got = sp24.add_adapters(*args, workspace=workspace)
    sp24.last_device_error()
    out, size = reference(y, x, a, b, ids, scales)
    assert_adapted(got, out, size, "tiles of different cost")
    assert torch.equal(got, sp24.add_adapters(*args, workspace=workspace))


def test_an_infinite_value_has_the_sign_of_its_products(sp24):
    """Ranks that are no multiple of 16: what pads them adds nothing, not even to a row with an infinite value."""
    for T in (20, 800, 1200):
        y, x, a, b, _ = inputs(T, 64, 136, 8, 2, seed=T)
        a, b = a.abs() + 0.5, b.abs() + 0.5
        x[7, 3], x[11, 3] = float("inf"), float("-inf")
        got = sp24.add_adapters(y.cuda(), x.cuda(), a.cuda(), b.cuda(), torch.zeros(T, dtype=torch.int32, device="cuda"))
        sp24.last_device_error()
        assert (got[7] == float("inf")).all() and (got[11] == float("-inf")).all()
        rest = torch.ones(T, dtype=torch.bool)
        rest[7], rest[11] = False, False
        assert torch.isfinite(got.cpu()[rest].float()).all()
