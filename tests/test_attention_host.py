"""The attention entry points' checks of arguments: refused on the host, before any launch (no GPU needed)."""
import ctypes

import pytest

INVALID, UNSUPPORTED, ALIGNMENT = 1, 2, 3
P, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)


@pytest.fixture(scope="module")
def lib():
    import semi_structured_sparse_gb300 as s
    return s.load()


def cache(**kw):
    import semi_structured_sparse_gb300 as s
    a = dict(k=0x10000, v=0x20000, k_scale=None, v_scale=None, num_pages=9, page_stride=2 * 16 * 64,
             head_stride=16 * 64, token_stride=64, heads=2, page_size=16, head_dim=64, dtype=0)
    a.update(kw)
    return s._KVCacheStruct(*(a[f] for f, _ in s._KVCacheStruct._fields_))


BAD_CACHES = [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(heads=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_pages=1 << 31), INVALID), (dict(dtype=2), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(dtype=1), INVALID), (dict(dtype=1, k_scale=0x100), INVALID), (dict(k_scale=0x100, v_scale=0x100), INVALID),
    (dict(page_stride=0), INVALID), (dict(head_stride=-64), INVALID), (dict(page_stride=1 << 40), INVALID),
    (dict(token_stride=32), INVALID), (dict(head_stride=16 * 64 + 4), ALIGNMENT), (dict(k=0x10008), ALIGNMENT),
]


@pytest.mark.parametrize("kw,status", BAD_CACHES)
def test_caches(lib, kw, status):
    c = ctypes.addressof(cache(**kw)), cache(**kw)
    keep = c[1]
    a = ctypes.addressof(keep)
    assert lib.sp24_qk_norm_rope(P, 1, 512, 4, None, None, 1e-6, P, 9, 64, 0, P, P, P, 256, a, None) == status
    assert lib.sp24_attention_decode(P, 1, 256, 4, a, P, 3, 3, P, 1.0, 0, 0, P, 256, P, 1 << 30, None) == status
    assert lib.sp24_attention_prompt(P, 1, 256, 4, P, 1, a, P, 3, 3, P, 1.0, 0, 0, P, 256, None, 0, None) == status
    assert lib.sp24_attention_prompt_workspace_size(1, 1, 4, a, 3, 0, 0) == 0


def test_rope_arguments(lib):
    keep = cache()

    def call(**kw):
        a = dict(x=P, T=2, ldx=512, hq=4, qw=P, kw=P, eps=1e-6, cs=P, mp=9, rot=64, inter=0, pos=P, slots=P, q=P, ldq=256,
                 c=ctypes.addressof(keep))
        a.update(kw)
        return lib.sp24_qk_norm_rope(*a.values(), None)

    for kw in (dict(x=None), dict(q=None), dict(slots=None), dict(pos=None), dict(cs=None), dict(mp=0), dict(T=-1),
               dict(T=1 << 31), dict(hq=0), dict(ldx=504), dict(ldq=248), dict(rot=-16), dict(rot=80), dict(qw=None),
               dict(kw=None), dict(eps=-1.0), dict(eps=float("nan")), dict(c=None)):
        assert call(**kw) == INVALID, kw
    assert call(rot=24) == UNSUPPORTED
    for kw in (dict(x=ODD), dict(q=ODD), dict(ldx=516), dict(ldq=260), dict(qw=ODD), dict(cs=ODD),
               dict(slots=ctypes.c_void_p(0x10004)), dict(pos=ctypes.c_void_p(0x10002))):
        assert call(**kw) == ALIGNMENT, kw


def test_attention_arguments(lib):
    keep = cache()

    def decode(**kw):
        a = dict(q=P, B=2, ldq=256, hq=4, c=ctypes.addressof(keep), t=P, w=3, ldt=3, n=P, scale=1.0, window=0, sinks=0,
                 y=P, ldy=256)
        a.update(kw)
        return lib.sp24_attention_decode(*a.values(), P, 1 << 30, None)

    def prompt(**kw):
        a = dict(q=P, T=2, ldq=256, hq=4, cu=P, B=2, c=ctypes.addressof(keep), t=P, w=3, ldt=3, n=P, scale=1.0, window=0,
                 sinks=0, y=P, ldy=256)
        a.update(kw)
        return lib.sp24_attention_prompt(*a.values(), None, 0, None)

    for call in (decode, prompt):
        for kw in (dict(q=None), dict(y=None), dict(t=None), dict(n=None), dict(c=None), dict(B=-1), dict(hq=0),
                   dict(hq=3), dict(ldq=248), dict(ldy=248), dict(w=0), dict(ldt=2), dict(w=1 << 27, ldt=1 << 27),
                   dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(window=-1), dict(sinks=-1)):
            assert call(**kw) == INVALID, kw
        assert call(hq=2 * 129, ldq=2 * 129 * 64, ldy=2 * 129 * 64) == UNSUPPORTED
        for kw in (dict(q=ODD), dict(y=ODD), dict(ldq=260), dict(ldy=260), dict(t=ctypes.c_void_p(0x10002)),
                   dict(n=ctypes.c_void_p(0x10001))):
            assert call(**kw) == ALIGNMENT, kw
    assert prompt(T=-1) == INVALID
    assert prompt(cu=None) == INVALID
    assert prompt(cu=ctypes.c_void_p(0x10002)) == ALIGNMENT


def test_workspace_size_of_bad_layouts(lib):
    f = lib.sp24_attention_decode_workspace_size
    assert f(0, 1, 64) == 0 and f(3, 2, 64) == 0 and f(4, 2, 96) == 0 and f(129, 1, 64) == 0


def test_status_of_an_index_out_of_range(lib):
    assert lib.sp24_status_string(8).startswith(b"SP24_ERR_DEVICE_INDEX")


def test_binding_refuses_host_tensors():
    import torch
    import semi_structured_sparse_gb300 as s
    k = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        s.KVCache(k, k.clone())
