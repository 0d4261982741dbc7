"""The attention operators from their definitions in 64 bits, and inputs for them."""
import torch

E4M3 = torch.float8_e4m3fn


class Setup:
    """A paged cache on the GPU, its decoded values in 64 bits, and page tables.

    Every place that no sequence's visible token occupies can be poisoned with NaN."""

    def __init__(self, sp24, lens, hkv, d, page, e4m3, token_major, seed, extra_pages=3):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.d, self.page, self.e4m3 = list(lens), hkv, d, page, e4m3
        width = max([1] + [-(-n // page) for n in lens])
        pages = len(lens) * width + extra_pages
        self.table = torch.randperm(pages, generator=g)[:len(lens) * width].view(len(lens), width).to(torch.int32)
        shape = (pages, page, hkv, d) if token_major else (pages, hkv, page, d)
        self.store, self.value, self.scale = {}, {}, {}
        for name in ("k", "v"):
            x = torch.randn(shape, generator=g)
            if e4m3:
                x = (32 * x).clamp(-448, 448).to(E4M3).view(torch.uint8)
                self.scale[name] = torch.rand(hkv, generator=g) * 0.02 + 0.02
            else:
                x = x.to(torch.bfloat16)
            self.store[name] = x.transpose(1, 2) if token_major else x
        self.sp24 = sp24

    def poison(self, seen):
        """NaN everywhere but at each sequence's tokens for which seen[b][j] holds."""
        for name in ("k", "v"):
            old = self.store[name].clone()
            self.store[name].copy_(torch.full_like(old, 0x7F if self.e4m3 else float("nan")))
            for b, n in enumerate(self.lens):
                for j in range(n):
                    if bool(seen[b][j]):
                        p = int(self.table[b, j // self.page])
                        self.store[name][p, :, j % self.page] = old[p, :, j % self.page]

    def upload(self):
        up = {}
        for name, x in self.store.items():  # keeps the strides
            y = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device="cuda")
            up[name] = y.copy_(x)
        sc = {n: s.cuda() for n, s in self.scale.items()}
        self.cache = self.sp24.KVCache(up["k"], up["v"], sc.get("k"), sc.get("v"))
        return self.cache

    def tokens(self, name, b):
        """[n, hkv, d] in 64 bits: what the cache stands for."""
        n = self.lens[b]
        x = self.store[name][self.table[b].long()]            # [width, hkv, page, d]
        x = x.transpose(1, 2).reshape(-1, self.hkv, self.d)[:n]
        if self.e4m3:
            return x.contiguous().view(E4M3).double() * self.scale[name].double()[:, None]
        return x.double()


def sees(at, n, window, sinks):
    """[len(at), n]: whether the query at each position sees each key."""
    j = torch.arange(n)
    at = torch.as_tensor(at)[:, None]
    see = j[None] <= at
    return see & ((j[None] > at - window) | (j[None] < sinks)) if window else see


def attend(q, k, v, see, scale):
    """q [m, hq, d], k and v [n, hkv, d] in 64 bits -> (y, softmax-weighted mean of |v|), both [m, hq, d]."""
    m, hq, d = q.shape
    y, size = torch.zeros(m, hq, d, dtype=torch.float64), torch.zeros(m, hq, d, dtype=torch.float64)
    if k.shape[0] == 0:
        return y, size
    group = hq // k.shape[1]
    some = see.any(1)
    for h in range(hq):
        kk, vv = torch.nan_to_num(k[:, h // group]), torch.nan_to_num(v[:, h // group])
        s = (q[:, h] @ kk.T * scale).masked_fill(~see, -torch.inf)
        p = torch.softmax(s, -1)
        p[~some] = 0
        y[:, h], size[:, h] = p @ vv, p @ vv.abs()
    return y, size


# bf16 has 8 significant bits: half an ulp is at most 2^-8 of a value.  Weights enter the tensor core rounded to it, so
# the weighted sum moves by at most 2^-8 of the weighted mean of |v|, and the result is rounded to it (2^-8 of it).  fp32 scores, exponentials and sums: scores of at most some tens off by a few 2^-24 times that
# and by an ulp of the exponential, far below 2^-12 of the weighted mean.
def assert_attention(got, y, size, what):
    got = got.double().cpu().view(y.shape)
    assert torch.isfinite(got).all(), what + ": not finite"
    bound = 2.0 ** -8 * (1 + 2.0 ** -6) * y.abs() + (2.0 ** -8 + 2.0 ** -12) * size + 1e-30
    err = (got - y).abs()
    bad = err > bound
    assert not bad.any(), "%s: %d of %d outside the bound, worst %.3g of it at %s" % (
        what, int(bad.sum()), bad.numel(), float((err / bound).max()), bad.nonzero()[0].tolist())
