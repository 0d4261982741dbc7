"""Every visible key counts once, and no other does (GPU).

With queries of zero all weights are equal, so a row that sees n keys gives 1/n of the sum of their values.  A value is 1
at one key's own (head, dim) and 0 elsewhere: the row then holds 1/n there if it sees that key, and 0 if not, whatever the
length.  heads x dims keys are looked at per call, and all of them over the calls."""
import pytest
import torch

from attention_util import sees

pytestmark = pytest.mark.gpu


class Tokens:
    """Sequences in a paged cache whose keys are zero and whose values a call sets."""

    def __init__(self, sp24, lens, hkv, d, page, e4m3, token_major, seed, width=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.d, self.e4m3 = lens, hkv, d, e4m3
        width = max([1, width] + [-(-n // page) for n in lens])
        own = len(lens) * max(1, max(-(-n // page) for n in lens))
        pages = torch.randperm(own + 2, generator=g)[:own].view(len(lens), -1).to(torch.int32)
        self.table = torch.zeros(len(lens), width, dtype=torch.int32)
        self.table[:, :pages.shape[1]] = pages
        shape = (own + 2, page, hkv, d) if token_major else (own + 2, hkv, page, d)
        make = lambda: torch.zeros(shape, dtype=torch.uint8 if e4m3 else torch.bfloat16, device="cuda")  # noqa: E731
        self.k, self.v = (make().transpose(1, 2) if token_major else make() for _ in range(2))
        one = torch.ones(hkv, device="cuda") if e4m3 else None
        self.cache = sp24.KVCache(self.k, self.v, one, one)
        self.table, self.page = self.table.cuda(), page
        self.n = torch.tensor(lens, dtype=torch.int32).cuda()
        self.calls = -(-max(lens) // (hkv * d))

    def set(self, call):
        """Values of one at the keys of this call; returns the key of each (head, dim)."""
        key = call * self.hkv * self.d + torch.arange(self.hkv * self.d, device="cuda").view(self.hkv, self.d)
        self.v.zero_()
        h, i = torch.meshgrid(torch.arange(self.hkv, device="cuda"), torch.arange(self.d, device="cuda"), indexing="ij")
        for b, n in enumerate(self.lens):
            at = key < n
            p = self.table[b, (key[at] // self.page)].long()
            self.v[p, h[at], key[at] % self.page, i[at]] = 0x38 if self.e4m3 else 1  # 0x38: the e4m3 code of 1
        return key


def check(y, key, see, hq, what):
    """y [m, hq, d]; see [m, n]: 1/n of the row's keys, exactly but for the rounding to bf16 (2^-8 of it) and a few
    2^-24 of the quotient; exactly zero where the key is not seen."""
    m, n = see.shape
    hkv, d = key.shape
    got = y.double().view(m, hkv, hq // hkv, d)
    count = see.sum(1).double().cuda().clamp(min=1).view(m, 1, 1, 1)
    sight = torch.zeros(m, hkv, d, dtype=torch.bool, device="cuda")
    at = key < n
    sight[:, at] = see.cuda()[:, key[at]]
    bad = ((got * count - sight[:, :, None].double()).abs() > 2.0 ** -8 * 1.01 * sight[:, :, None].double())
    assert not bad.any(), "%s: %d wrong, first (row, head, in group, dim) %s" % (what, int(bad.sum()),
                                                                              bad.nonzero()[0].tolist())


LAYOUTS = [(8, 4, 64, 16, False, True), (8, 2, 128, 64, False, False), (14, 2, 64, 32, True, False),
           (8, 4, 128, 16, True, True)]


@pytest.mark.parametrize("hq,hkv,d,page,e4m3,token_major", LAYOUTS)
@pytest.mark.parametrize("lens,window,sinks", [
    ([1, 15, 16, 17, 63, 64, 65, 129, 1000], 0, 0),
    ([5000, 31], 0, 0),
    ([20011], 0, 0),
    ([5000, 700, 2047], 1029, 7),
    ([3001, 900], 64, 1100),
    ([2500], 1, 33),
])
def test_decode_counts_every_key_once(sp24, hq, hkv, d, page, e4m3, token_major, lens, window, sinks):
    t = Tokens(sp24, lens, hkv, d, page, e4m3, token_major, seed=len(lens))
    q = torch.zeros(len(lens), hq, d, dtype=torch.bfloat16, device="cuda")
    for call in range(t.calls):
        key = t.set(call)
        y = sp24.attention_decode(q, t.cache, t.table, t.n, window=window, sinks=sinks)
        for b, n in enumerate(lens):
            check(y[b:b + 1], key, sees([n - 1], n, window, sinks), hq, "call %d, sequence %d" % (call, b))
    sp24.last_device_error()


@pytest.mark.parametrize("hq,hkv,d,page,e4m3,token_major", LAYOUTS)
@pytest.mark.parametrize("new,prefix,width,window,sinks", [
    ([1, 15, 130, 260], [0, 500, 0, 1], 0, 0, 0),
    ([300, 20], [1500, 2100], 0, 0, 0),
    ([300, 20], [1500, 2100], 0, 517, 9),
    ([150], [700], 0, 64, 300),
    ([40], [-15], 0, 0, 0),
    ([7, 1], [9000, 3000], 9216, 0, 0),        # few rows over a long cache: cut into parts
    ([33], [9000], 9216, 4000, 700),
    ([70, 2], [140, 5], 20000, 0, 0),          # parts without keys
])
def test_prompt_counts_every_key_once(sp24, hq, hkv, d, page, e4m3, token_major, new, prefix, width, window, sinks):
    lens = [a + b for a, b in zip(new, prefix)]
    t = Tokens(sp24, lens, hkv, d, page, e4m3, token_major, seed=len(new), width=width // page)
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).cuda()
    q = torch.zeros(sum(new), hq, d, dtype=torch.bfloat16, device="cuda")
    need = sp24.attention_prompt_workspace_size(t.cache, hq, sum(new), len(new), t.table.shape[1], window, sinks)
    assert need > 0 or not width
    for call in range(t.calls):
        key = t.set(call)
        y = sp24.attention_prompt(q, cu, t.cache, t.table, t.n, window=window, sinks=sinks)
        for b, m in enumerate(new):
            see = sees(torch.arange(lens[b] - m, lens[b]), lens[b], window, sinks)
            check(y[int(cu[b]):int(cu[b + 1])], key, see, hq, "call %d, sequence %d" % (call, b))
    sp24.last_device_error()
