"""Attention of one new token per sequence behind shared first tokens, against its definition in 64 bits (GPU)."""
import pytest
import torch

from attention_util import Setup, assert_attention, attend, sees

pytestmark = pytest.mark.gpu


def widened(table, page, hkv, d, e4m3, seed=1):
    """The table with more columns, of pages that are not to be read: a call whose tables could hold so much that
    sharing may save more than 32 MB (fewer, and the sequences are attended one by one)."""
    B = table.shape[0]
    tokens = (32 << 20) // (max(1, B - 1) * hkv * 2 * d * (1 if e4m3 else 2)) + 1
    width = max(table.shape[1], -(-tokens // page))
    out = torch.full((B, width), 1 << 28, dtype=torch.int32)
    out[:, :table.shape[1]] = table
    return out


def batch(sp24, cu, shared, lens, hkv, d, page, e4m3, token_major, window, sinks, seed, one_by_one=False):
    """A cache in which the groups' shared tokens are in the pages of each group's first sequence: whole pages in all
    the group's tables, the page that they end in as a copy.  All that is not to be read is NaN.  Returns the setup and
    each sequence's keys and values in 64 bits."""
    s = Setup(sp24, lens, hkv, d, page, e4m3, token_major, seed)
    by_itself = [True] * len(lens)
    for g, n in enumerate(shared):
        for b in range(cu[g], cu[g + 1]):
            by_itself[b] = one_by_one or lens[b] < n or (window > 0 and lens[b] > window)
            lead = cu[g]
            m = min(n, lens[b])
            full = min(m, lens[lead]) // page
            s.table[b, :full] = s.table[lead, :full]
            if m > full * page and b != lead:
                for x in ("k", "v"):
                    s.store[x][int(s.table[b, full]), :, :m - full * page] = \
                        s.store[x][int(s.table[lead, full]), :, :m - full * page]
    tokens = [(s.tokens("k", b), s.tokens("v", b)) for b in range(len(lens))]
    seen = []
    for b, n in enumerate(lens):
        see = sees([n - 1], n, window, sinks)[0] if n else torch.zeros(0, dtype=torch.bool)
        seen.append(see.clone())
    for g, n in enumerate(shared):
        for b in range(cu[g], cu[g + 1]):
            if not by_itself[b]:
                seen[b][:n] = False
        if any(not by_itself[b] for b in range(cu[g], cu[g + 1])):
            assert lens[cu[g]] >= n, "the first sequence has the shared tokens"
            seen[cu[g]][:n] = True
    s.poison(seen)
    return s, tokens


def run(sp24, cu, shared, lens, hq, hkv, d, page, e4m3=False, token_major=False, window=0, sinks=0, seed=0, q=None,
        scale=None, wide=True, **kw):
    s, tokens = batch(sp24, cu, shared, lens, hkv, d, page, e4m3, token_major, window, sinks, seed, not wide)
    table = widened(s.table, page, hkv, d, e4m3) if wide else s.table
    cache = s.upload()
    g = torch.Generator().manual_seed(seed + 1)
    if q is None:
        q = (2 * torch.randn(len(lens), hq, d, generator=g)).to(torch.bfloat16)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    y = sp24.attention_decode_shared(q.cuda(), cache, table.cuda(), i32(lens), i32(cu), i32(shared), scale=scale,
                                     window=window, sinks=sinks, **kw)
    sp24.last_device_error()
    want, size = torch.zeros(len(lens), hq, d, dtype=torch.float64), torch.zeros(len(lens), hq, d, dtype=torch.float64)
    for b, n in enumerate(lens):
        see = sees([n - 1], n, window, sinks) if n else torch.zeros(1, 0, dtype=torch.bool)
        k, v = tokens[b]
        out, sz = attend(q[b:b + 1].double(), k, v, see, scale or d ** -0.5)
        want[b], size[b] = out[0], sz[0]
    assert_attention(y, want, size, "shared")
    return y


CASES = [
    # cu, shared, lens, hq, hkv, d, page, e4m3, token_major, window, sinks
    ([0, 1], [1], [1], 1, 1, 64, 16, False, False, 0, 0),                        # one key in all
    ([0, 2], [1], [1, 2], 4, 2, 128, 64, False, False, 0, 0),
    ([0, 2], [1000], [1001, 1030], 32, 8, 128, 64, False, False, 0, 0),
    ([0, 3], [1000], [1000, 1001, 1300], 32, 8, 128, 64, True, False, 0, 0),     # nothing of its own
    ([0, 5], [127], [128, 200, 127, 130, 400], 7, 1, 64, 16, False, True, 0, 0),  # a tile but one key
    ([0, 5], [129], [129, 200, 130, 131, 400], 5, 1, 64, 16, True, True, 0, 0),
    ([1, 4, 4, 9], [300, 77, 512], [5, 301, 310, 400, 513, 514, 600, 700, 512, 40], 12, 4, 64, 32, False, False, 0, 0),
    ([0, 4, 8], [0, 640], [1, 2, 300, 0, 641, 650, 700, 900], 8, 2, 128, 16, True, False, 0, 0),   # nothing shared
    ([0, 6], [500], [501, 30, 0, 499, 500, 700], 6, 2, 128, 32, False, True, 0, 0),   # sequences shorter than that
    ([0, 6], [500], [600, 30, 0, 499, 520, 700], 6, 2, 64, 32, True, True, 0, 0),
    ([0, 40], [333], [334 + 5 * i for i in range(40)], 28, 4, 64, 16, False, True, 0, 0),  # rows of three tiles
    ([0, 70], [200], [201 + 3 * i for i in range(70)], 16, 2, 128, 64, True, False, 0, 0),  # three blocks of rows
    ([0, 2], [150], [151, 160], 128, 1, 64, 128, False, False, 0, 0),             # a token's heads fill a tile
    ([0, 3], [260], [261, 270, 280], 96, 1, 128, 16, True, False, 0, 0),          # ... or leave the rest of it empty
    ([0, 4], [900], [901, 950, 1000, 1200], 8, 4, 64, 16, False, False, 1000, 4),  # some see all of it, some do not
    ([0, 4], [900], [901, 950, 1000, 1200], 8, 4, 128, 64, True, False, 940, 130),
    ([0, 4], [900], [901, 950, 1000, 1200], 4, 4, 64, 16, False, True, 50, 0),     # windows within what is their own
    ([2, 2], [5], [20, 30], 4, 2, 64, 16, False, False, 0, 0),                    # a group without sequences
    ([0, 17, 33], [2100, 1500], [2101 + 40 * i for i in range(17)] + [1501 + 9 * i for i in range(16)], 8, 1, 128, 128,
     False, False, 0, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "%dx%s-%d/%dx%d-p%d%s%s%s" % (
    len(c[2]), "+".join(map(str, c[1])), c[3], c[4], c[5], c[6], "-e4m3" * c[7], "-tok" * c[8], "-w%d" % c[9] if c[9] else ""))
def test_shared(sp24, case):
    cu, shared, lens, hq, hkv, d, page, e4m3, token_major, window, sinks = case
    run(sp24, cu, shared, lens, hq, hkv, d, page, e4m3, token_major, window, sinks, seed=len(lens) + d)


@pytest.mark.parametrize("case", CASES[1:9:2] + CASES[14:16], ids=str)
def test_little_to_share(sp24, case):
    """The same sizes where the tables could not hold much: one by one, through each sequence's own pages."""
    cu, shared, lens, hq, hkv, d, page, e4m3, token_major, window, sinks = case
    run(sp24, cu, shared, lens, hq, hkv, d, page, e4m3, token_major, window, sinks, seed=len(lens) + d, wide=False)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_every_visible_key_counts_once(sp24, d, e4m3):
    """Queries of zero: a row is the plain mean of the values that it sees, whichever way they are read."""
    lens = [700 + 37 * i for i in range(9)]
    s = Setup(sp24, lens, 2, d, 16, e4m3, False, seed=4)
    for b in range(9):
        s.table[b, :37] = s.table[0, :37]
    for x in ("k", "v"):  # 600 shared tokens: 37 pages and 8 places
        for b in range(1, 9):
            s.store[x][int(s.table[b, 37]), :, :8] = s.store[x][int(s.table[0, 37]), :, :8]
    cache = s.upload()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    table = widened(s.table, 16, 2, d, e4m3).cuda()
    y = sp24.attention_decode_shared(torch.zeros(9, 4, d, device="cuda").bfloat16(), cache, table, i32(*lens),
                                     i32(0, 9), i32(600))
    sp24.last_device_error()
    for b in range(9):
        v = s.tokens("v", b)
        mean = v.mean(0).repeat_interleave(2, 0)
        # weights are exactly 1 (a power of two in f16): what is left is the sum's fp32 rounding and the result's to bf16
        size = v.abs().mean(0).repeat_interleave(2, 0)
        assert ((y[b].double().cpu() - mean).abs() <= 2.0 ** -8 * mean.abs() + 2.0 ** -14 * size).all(), b


def test_agrees_with_decode_and_is_the_same_every_time(sp24):
    """The same call again, with the same workspace, after calls of other shapes: the same bits."""
    cu, shared, lens = [1, 30], [3000], [40] + [3001 + 17 * i for i in range(29)]
    s = Setup(sp24, lens, 2, 128, 64, False, False, 7)
    for b in range(1, 30):
        s.table[b, :46] = s.table[1, :46]
        for x in ("k", "v"):
            s.store[x][int(s.table[b, 46]), :, :56] = s.store[x][int(s.table[1, 46]), :, :56]
    cache = s.upload()
    q = (2 * torch.randn(30, 8, 128, generator=torch.Generator().manual_seed(1))).bfloat16().cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    size = max(sp24.attention_decode_shared_workspace_size(cache, 8, 30, 1),
               sp24.attention_decode_shared_workspace_size(cache, 8, 30, 3))
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    args = (q, cache, widened(s.table, 64, 2, 128, False).cuda(), i32(lens))
    first = sp24.attention_decode_shared(*args, i32(cu), i32(shared), workspace=ws)
    other = sp24.attention_decode_shared(*args, i32([1, 4, 20, 30]), i32([3000, 100, 2999]), workspace=ws)
    plain = sp24.attention_decode(*args)
    again = sp24.attention_decode_shared(*args, i32(cu), i32(shared), workspace=ws)
    sp24.last_device_error()
    assert torch.equal(first, again)
    # three ways to add up the same rows: each within the bound of assert_attention of the true row, where |v| is of
    # order 1 and the rows' values are below 4
    for y in (first, other):
        assert (y.float() - plain.float()).abs().max() < 2 * (2.0 ** -8 * 4 + 2.0 ** -7 * 2)


def test_graph_replays_follow_the_lengths(sp24):
    """A captured call reads lengths, tables and groups anew each time."""
    lens = [400, 410, 500, 450]
    s = Setup(sp24, lens, 1, 64, 16, False, False, 3)
    for b in range(4):
        s.table[b, :20] = s.table[0, :20]
    cache = s.upload()
    q = torch.randn(4, 4, 64, generator=torch.Generator().manual_seed(2)).bfloat16()
    qd, table = q.cuda(), widened(s.table, 16, 1, 64, False).cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    n, cu, sh = i32(*lens), i32(0, 4), i32(320)
    ws = torch.zeros(sp24.attention_decode_shared_workspace_size(cache, 4, 4, 1), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(qd)
    call = lambda: sp24.attention_decode_shared(qd, cache, table, n, cu, sh, out=out, workspace=ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for now, shared, groups in ((lens, 320, (0, 4)), ([330, 320, 321, 400], 320, (0, 4)), ([400, 3, 0, 450], 300, (0, 4)),
                                ([400, 410, 500, 450], 16, (1, 3))):
        n.copy_(i32(*now))
        sh.fill_(shared)
        cu.copy_(i32(*groups))
        out.fill_(7)
        graph.replay()
        sp24.last_device_error()
        for b in range(4):
            k, v = s.tokens("k", b)[:now[b]], s.tokens("v", b)[:now[b]]
            see = torch.ones(1, now[b], dtype=torch.bool)
            y, size = attend(q[b:b + 1].double(), k, v, see, 0.125)
            assert_attention(out[b:b + 1], y, size, "replay %s, row %d" % (now, b))


def test_index_errors(sp24):
    """Groups, shared lengths and pages out of range are kept in bounds and reported."""
    lens = [64, 70, 80]
    s = Setup(sp24, lens, 1, 64, 16, False, False, 5)
    for b in range(3):
        s.table[b, :4] = s.table[0, :4]
    cache = s.upload()
    q = torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(3)).bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    bad = s.table.clone()
    bad[0, 1] = 1 << 30
    worse = s.table.clone()
    worse[2, 4] = -5
    good = s.table
    for cu, shared, table, n in ((i32(0, 9), i32(64), good, i32(*lens)), (i32(-3, 3), i32(64), good, i32(*lens)),
                                 (i32(2, 1), i32(64), good, i32(*lens)), (i32(0, 3), i32(-1), good, i32(*lens)),
                                 (i32(0, 3), i32(1 << 30), good, i32(*lens)), (i32(0, 3), i32(64), bad, i32(*lens)),
                                 (i32(0, 3), i32(64), worse, i32(*lens)), (i32(0, 3), i32(64), good, i32(64, -1, 80)),
                                 (i32(0, 3), i32(64), good, i32(64, 1 << 30, 80))):
        y = sp24.attention_decode_shared(q.cuda(), cache, widened(table, 16, 1, 64, False).cuda(), n, cu, shared)
        with pytest.raises(sp24.Sp24Error) as e:
            sp24.last_device_error()
        assert e.value.status == 8
        assert torch.isfinite(y.float()).all()
    # and all is well afterwards
    y = sp24.attention_decode_shared(q.cuda(), cache, widened(good, 16, 1, 64, False).cuda(), i32(*lens), i32(0, 3), i32(64))
    sp24.last_device_error()
    for b in range(3):
        want, size = attend(q[b:b + 1].double(), s.tokens("k", b), s.tokens("v", b),
                            torch.ones(1, lens[b], dtype=torch.bool), 0.125)
        assert_attention(y[b:b + 1], want, size, "after errors")


def test_layouts_and_empty_calls(sp24):
    """Rows further apart than their length, a wide table, 2-D queries, another stream, no groups, no sequences."""
    lens = [70, 90, 130]
    s = Setup(sp24, lens, 2, 64, 16, False, False, 6)
    for b in range(3):
        s.table[b, :4] = s.table[0, :4]
    cache = s.upload()
    q = torch.randn(3, 4 * 64 + 24, generator=torch.Generator().manual_seed(3)).bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    wide = widened(s.table, 16, 2, 64, False)
    columns = wide.shape[1]
    wide = torch.cat((wide, wide[:, :7]), 1)            # rows further apart than their length
    out = torch.zeros(3, 4 * 64 + 8, device="cuda").bfloat16()
    qd, wd, n, cu, sh = q.cuda(), wide.cuda(), i32(*lens), i32(0, 3), i32(64)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = sp24.attention_decode_shared(qd[:, 8:264], cache, wd[:, :columns], n, cu, sh, scale=0.3, out=out[:, :256], stream=side)
    sp24.last_device_error(side)
    none = sp24.attention_decode_shared(qd[:, 8:264], cache, wd[:, :columns], n, i32(0), i32(), scale=0.3)
    sp24.last_device_error()
    for b in range(3):
        want, size = attend(q[b:b + 1, 8:264].double().view(1, 4, 64), s.tokens("k", b), s.tokens("v", b),
                            torch.ones(1, lens[b], dtype=torch.bool), 0.3)
        assert_attention(y[b], want, size, "layout")
        assert_attention(none[b], want, size, "no groups")
    assert (out[:, 256:] == 0).all()
    empty = sp24.attention_decode_shared(qd[:0, 8:264], cache, wd[:0], n[:0], i32(0), i32())
    assert empty.shape == (0, 256)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("cu", [[0, 7, 3, 8], [5, 2, 8, 8], [0, 3, 3, 9], [-1, 4, 6, 8], [2, 1, 0, 8], [0, 8, 0, 8]], ids=str)
def test_groups_out_of_order(sp24, cu, e4m3):
    """Groups that are not in order share nothing and are reported: no row takes what an earlier call has left in the
    workspace, or loses its first tokens."""
    lens = [113, 150, 200, 260, 170, 121, 300, 240]
    s = Setup(sp24, lens, 2, 64, 16, e4m3, False, 11)
    for b in range(8):
        s.table[b, :7] = s.table[0, :7]      # the first 112 tokens are everyone's
    cache = s.upload()
    g = torch.Generator().manual_seed(12)
    q, other = ((2 * torch.randn(8, 6, 64, generator=g)).bfloat16() for _ in range(2))
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    table, n = widened(s.table, 16, 2, 64, e4m3).cuda(), i32(*lens)
    ws = torch.zeros(sp24.attention_decode_shared_workspace_size(cache, 6, 8, 3), dtype=torch.uint8, device="cuda")
    wants = []
    for x in (q, other):
        rows = [attend(x[b:b + 1].double(), s.tokens("k", b), s.tokens("v", b), torch.ones(1, lens[b], dtype=torch.bool), 0.125)
                for b in range(8)]
        wants.append([torch.cat([r[i] for r in rows]) for i in range(2)])
    y = sp24.attention_decode_shared(other.cuda(), cache, table, n, i32(0, 8, 8, 8), i32(112, 0, 0), workspace=ws)
    sp24.last_device_error()
    assert_attention(y, *wants[1], "a call before")
    y = sp24.attention_decode_shared(q.cuda(), cache, table, n, i32(*cu), i32(112, 96, 112), workspace=ws)
    with pytest.raises(sp24.Sp24Error) as e:
        sp24.last_device_error()
    assert e.value.status == 8
    assert_attention(y, *wants[0], "groups %s" % cu)
    y = sp24.attention_decode_shared(q.cuda(), cache, table, n, i32(0, 3, 3, 8), i32(112, 96, 112), workspace=ws)
    sp24.last_device_error()
    assert_attention(y, *wants[0], "a call after")


@pytest.mark.parametrize("shared,lens,window,sinks,one_by_one", [
    (700, [1100 + 6 * i for i in range(70)], 500, 0, True),            # nobody sees all shared tokens
    (700, [701 + 6 * i for i in range(70)], 500, 20, True),
    (300, [900] + [301 + 3 * i for i in range(69)], 500, 20, True),    # the first sequence does not, others would
    (300, [560] + [301 + 3 * i for i in range(69)], 500, 20, True),    # ... by three pages
    (480, [520] + [481 + 2 * i for i in range(69)], 500, 20, False),   # the first does, some do not
    (480, [485] + [481 + 9 * i for i in range(69)], 500, 40, False),
    (0, [900] + [301 + 3 * i for i in range(69)], 500, 20, True),
])
@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_before_a_window(sp24, shared, lens, window, sinks, one_by_one, e4m3):
    """Neither a page without a visible key nor its entry in the table is read, whoever else is in the group."""
    hq, hkv, d, page, B = 16, 8, 64, 16, len(lens)
    s, tokens = batch(sp24, [0, B], [shared], lens, hkv, d, page, e4m3, False, window, sinks, 21, one_by_one)
    table = widened(s.table, page, hkv, d, e4m3)
    see = [sees([n - 1], n, window, sinks) for n in lens]
    hidden = 0
    for b, n in enumerate(lens):
        for i in range(-(-n // page)):
            if not see[b][0, i * page:(i + 1) * page].any():
                table[b, i] = -1 if (b + i) % 2 else 1 << 28
                hidden += 1
    assert hidden
    cache = s.upload()
    q = (2 * torch.randn(B, hq, d, generator=torch.Generator().manual_seed(22))).bfloat16()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    y = sp24.attention_decode_shared(q.cuda(), cache, table.cuda(), i32(lens), i32([0, B]), i32([shared]), window=window,
                                     sinks=sinks)
    sp24.last_device_error()
    rows = [attend(q[b:b + 1].double(), *tokens[b], see[b], d ** -0.5) for b in range(B)]
    assert_attention(y, torch.cat([r[0] for r in rows]), torch.cat([r[1] for r in rows]), "window")
