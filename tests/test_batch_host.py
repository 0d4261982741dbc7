"""Refusals of the operators for a batch of many requests, on the host, before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

from test_attention_host import BAD_CACHES, cache

INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 1, 2, 3, 6
P, ODD, ODD4 = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def lib():
    import semi_structured_sparse_gb300 as s
    return s.load()


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_caches(lib, kw, status):
    bad, good = cache(**kw), cache()
    a, g = ctypes.addressof(bad), ctypes.addressof(good)
    assert lib.sp24_attention_decode_shared(P, 1, 256, 4, a, P, 3, 3, P, P, P, 1, 1.0, 0, 0, P, 256, P, 1 << 40,
                                            None) == status
    assert lib.sp24_cache_copy(a, P, g, P, 1, None) == status
    assert lib.sp24_cache_copy(g, P, a, P, 1, None) == status


def test_shared_arguments(lib):
    keep = cache()

    def call(**kw):
        a = dict(q=P, B=2, ldq=256, hq=4, c=ctypes.addressof(keep), table=P, width=3, ld=3, lens=P, cu=P, shared=P, G=1,
                 scale=1.0, window=0, sinks=0, y=P, ldy=256, ws=P, bytes=1 << 40)
        a.update(kw)
        return lib.sp24_attention_decode_shared(*a.values(), None)

    for kw in (dict(q=None), dict(B=-1), dict(hq=0), dict(hq=3), dict(c=None), dict(table=None), dict(width=0), dict(ld=2),
               dict(lens=None), dict(cu=None), dict(shared=None), dict(G=-1), dict(G=1 << 30), dict(scale=0.0),
               dict(scale=float("inf")), dict(window=-1), dict(sinks=-1), dict(y=None), dict(ldq=248), dict(ldy=248)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(q=ODD), dict(y=ODD), dict(cu=ODD4), dict(shared=ODD4), dict(ldq=260), dict(lens=ODD4)):
        assert call(**kw) == ALIGNMENT, kw
    assert call(hq=2 * 129, ldq=2 * 129 * 64, ldy=2 * 129 * 64) == UNSUPPORTED
    size = lib.sp24_attention_decode_shared_workspace_size
    for bad in ((-1, 1, 4, 2, 64), (1, -1, 4, 2, 64), (1, 1, 0, 2, 64), (1, 1, 3, 2, 64), (1, 1, 4, 0, 64), (1, 1, 4, 2, 96),
                (1, 1, 258, 2, 64)):
        assert size(*bad) == 0, bad


def test_copy_arguments(lib):
    a, b = cache(), cache(heads=1)
    at = ctypes.addressof
    assert lib.sp24_cache_copy(at(a), P, at(b), P, 1, None) == INVALID
    wide = cache(head_dim=128, token_stride=128, head_stride=16 * 128, page_stride=2 * 16 * 128)
    assert lib.sp24_cache_copy(at(a), P, at(wide), P, 1, None) == INVALID
    assert lib.sp24_cache_copy(at(a), None, at(a), P, 1, None) == INVALID
    assert lib.sp24_cache_copy(at(a), P, at(a), None, 1, None) == INVALID
    assert lib.sp24_cache_copy(at(a), P, at(a), P, -1, None) == INVALID
    assert lib.sp24_cache_copy(at(a), P, at(a), P, 1 << 31, None) == INVALID
    assert lib.sp24_cache_copy(at(a), ctypes.c_void_p(0x10004), at(a), P, 1, None) == ALIGNMENT


def test_adapter_arguments(lib):
    def call(**kw):
        a = dict(y=P, ldy=64, x=P, ldx=128, T=2, K=128, N=64, a=P, sa=1024, b=P, sb=512, r=8, count=3, ids=P, scales=P, out=P,
                 ldo=64, ws=None, bytes=0)
        a.update(kw)
        return lib.sp24_add_adapters(*a.values(), None)

    for kw in (dict(y=None), dict(x=None), dict(a=None), dict(b=None), dict(ids=None), dict(out=None), dict(T=-1),
               dict(T=1 << 31), dict(K=0), dict(N=0), dict(r=0), dict(count=0), dict(ldy=56), dict(ldx=120), dict(ldo=56),
               dict(sa=1016), dict(sb=504), dict(K=(1 << 24) + 8, ldx=1 << 25), dict(ldx=1 << 39)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(K=124), dict(N=60), dict(r=12, sa=2048, sb=2048), dict(r=136, sa=1 << 16, sb=1 << 16)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(y=ODD), dict(x=ODD), dict(a=ODD), dict(b=ODD), dict(out=ODD), dict(ids=ODD4), dict(scales=ODD4),
               dict(ldy=68), dict(ldx=132), dict(ldo=68), dict(sa=1028), dict(sb=516)):
        assert call(**kw) == ALIGNMENT, kw


def test_python_refuses_what_is_not_on_a_gpu():
    import semi_structured_sparse_gb300 as s
    t = torch.zeros(2, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="y must be a CUDA tensor"):
        s.add_adapters(t, t, t[None], t[None], torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError, match="y must be a CUDA tensor"):
        s.add_adapters(None, t, t[None], t[None], torch.zeros(2, dtype=torch.int32))
