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


def fake_gpu_tensors(monkeypatch):
    """Tensors of the CPU that say that they are GPU 0's: what the binding checks of shapes, types and strides."""
    import semi_structured_sparse_gb300 as s
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0)
    monkeypatch.setattr(torch.Tensor, "is_cuda", property(lambda self: True))

    class Library:
        def __getattr__(self, name):
            return lambda *a: pytest.fail("the library was called")
    monkeypatch.setattr(s, "_lib", Library())
    return s


def test_adapter_shapes_are_refused(monkeypatch):
    s = fake_gpu_tensors(monkeypatch)
    z = lambda *shape, t=torch.bfloat16: torch.zeros(shape, dtype=t)  # noqa: E731
    good = dict(y=z(4, 16), x=z(4, 24), a=z(3, 8, 24), b=z(3, 16, 8), ids=z(4, t=torch.int32), scales=z(3, t=torch.float32),
                out=z(4, 16))
    bad = [dict(y=z(4, 16, t=torch.float16)), dict(y=z(5, 16)), dict(y=z(4, 32)[:, ::2]), dict(y=z(4)), dict(x=z(3, 24)),
           dict(x=z(4, 32)), dict(x=z(24, 4).T), dict(x=z(4, 24, t=torch.float32)), dict(a=z(3, 8, 16)), dict(a=z(2, 8, 24)),
           dict(a=z(3, 24, 8).transpose(1, 2)), dict(a=z(8, 24)), dict(a=z(1, 8, 24).expand(3, 8, 24)), dict(b=z(3, 16, 16)),
           dict(b=z(3, 8, 8)), dict(b=z(3, 8, 16).transpose(1, 2)), dict(ids=z(4, t=torch.int64)), dict(ids=z(3, t=torch.int32)),
           dict(ids=z(8, t=torch.int32)[::2]), dict(scales=z(2, t=torch.float32)), dict(scales=z(3)), dict(out=z(4, 24)),
           dict(out=z(4, 16, t=torch.float32)), dict(out=z(16, 4).T), dict(y=None), dict(a=None), dict(ids=None)]
    for kw in bad:
        with pytest.raises(ValueError):
            s.add_adapters(**dict(good, **kw))


def test_shared_and_copy_shapes_are_refused(monkeypatch):
    s = fake_gpu_tensors(monkeypatch)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    k = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    c, other = s.KVCache(k, k), s.KVCache(k[:, :1], k[:, :1])
    q, table, lens = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.zeros(2, 3, dtype=torch.int32), i32(1, 1)
    ws = torch.zeros(64, dtype=torch.uint8)
    for cu, shared in ((i32(0), i32(1)), (i32(0, 1, 2), i32(1)), (i32(0, 1).long(), i32(1)), (i32(0, 1), i32(1).float()),
                       (i32(0, 9, 1)[::2], i32(1)), (i32(0, 1)[None], i32(1)), (None, i32(1)), (i32(0, 1), None)):
        with pytest.raises(ValueError):
            s.attention_decode_shared(q, c, table, lens, cu, shared, workspace=ws)
    with pytest.raises(ValueError, match="sequences"):
        s.attention_decode_shared(q[:1], c, table, lens, i32(0, 2), i32(1), workspace=ws)
    with pytest.raises(ValueError):
        s.attention_decode_shared(q, c, table, lens, i32(0, 2), i32(1), workspace=ws.float())
    slots = torch.zeros(2, dtype=torch.int64)
    for i, j in ((slots, slots[:1]), (slots.int(), slots), (slots, slots.int()), (slots[None], slots[None]), (None, slots),
                 (slots, torch.zeros(4, dtype=torch.int64)[::2])):
        with pytest.raises(ValueError):
            s.cache_copy(c, i, c, j)
    with pytest.raises(ValueError, match="same heads"):
        s.cache_copy(c, slots, other, slots)


def test_copy_takes_as_many_heads_as_a_grid_has(lib):
    n = 1 << 16
    a = cache(heads=n, page_stride=n * 16 * 64)
    assert lib.sp24_cache_copy(ctypes.addressof(a), P, ctypes.addressof(a), P, 1, None) == INVALID
    n -= 1
    a = cache(heads=n, page_stride=n * 16 * 64)
    assert lib.sp24_cache_copy(ctypes.addressof(a), P, ctypes.addressof(a), P, 0, None) != INVALID
