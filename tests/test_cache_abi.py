"""The 8-bit cache's C ABI without a GPU: every bad argument is refused on the
host and nothing is launched."""
import ctypes

import pytest

FAKE = 0x100000  # never dereferenced: every call below fails validation or has nothing to do


@pytest.fixture(scope="module")
def api():
    from speculative_decoding_verification_02_gb300 import api, build
    build.build()
    api.lib()
    return api


def cache(api, **kw):
    a = dict(k=FAKE, v=FAKE, k_scale=FAKE, v_scale=FAKE, page_stride=8 * 64 * 128, scale_stride=8, num_pages=10, kv_heads=8,
             page_size=64, head_dim=128, table=FAKE, table_stride=4)
    a.update(kw)
    return api._CacheStruct(*a.values())


def s3(*s):
    return (ctypes.c_int64 * 3)(*s)


def s2(*s):
    return (ctypes.c_int64 * 2)(*s)


BAD_CACHES = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(num_pages=0), dict(kv_heads=0),
              dict(table=None), dict(table_stride=-1), dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(page_size=0),
              dict(head_dim=8), dict(head_dim=120), dict(head_dim=272), dict(head_dim=0), dict(page_stride=8 * 64 * 128 - 16),
              dict(page_stride=8 * 64 * 128 + 8), dict(scale_stride=7), dict(k=FAKE + 8), dict(v=FAKE + 1),
              dict(table_stride=1 << 25)]


def append(api, c=None, **kw):
    a = dict(k=FAKE, ks=s3(1 << 14, 1 << 10, 128), v=FAKE, vs=s3(1 << 14, 1 << 10, 128), dtype=1, B=2, n=9, index=None, ist=0, rows=9,
             counts=None, len=FAKE, new=FAKE + 64, status=None, stream=None)
    a.update(kw)
    c = c or cache(api)
    return api.lib().spec_cache_append(ctypes.byref(c), *a.values())


def attend(api, c=None, **kw):
    a = dict(q=FAKE, qs=s3(1 << 16, 1 << 12, 128), dtype=1, B=2, N=9, Hq=32, len=FAKE, nq=None, mask=None, scale=0.1, cap=0.0,
             out=FAKE, os=s3(1 << 16, 1 << 12, 128), lse=None, status=None, ws=FAKE, wsb=1 << 40, stream=None)
    a.update(kw)
    c = c or cache(api)
    return api.lib().spec_cache_attend(ctypes.byref(c), *a.values())


def weights(api, c=None, **kw):
    a = dict(q=FAKE, qs=s3(1 << 16, 1 << 12, 128), dtype=1, B=2, N=9, Hq=32, lse=FAKE, ls=s3(288, 32, 1), index=None, ist=0, rows=9,
             counts=None, len=FAKE, scale=0.1, cap=0.0, prev=None, ps=None, out=FAKE, os=s2(2048, 256), pos=256, status=None, ws=FAKE,
             wsb=1 << 40, stream=None)
    a.update(kw)
    c = c or cache(api)
    return api.lib().spec_cache_weights(ctypes.byref(c), *a.values())


def evict(api, c=None, d=None, **kw):
    a = dict(B=2, len=FAKE, w=FAKE, ws=s2(2048, 256), pos=256, keep=16, recent=4, kept=FAKE, kw=None, new=FAKE + 64, status=None,
             wsp=FAKE, wsb=1 << 40, stream=None)
    a.update(kw)
    c, d = c or cache(api), d or cache(api)
    return api.lib().spec_cache_evict(ctypes.byref(c), ctypes.byref(d), *a.values())


@pytest.mark.parametrize("call", [append, attend, weights, evict])
def test_bad_caches(api, call):
    n0 = api.launch_count()
    for bad in BAD_CACHES:
        assert call(api, cache(api, **bad)) == api.SPEC_EINVAL, bad
    assert api.launch_count() == n0


def test_no_cache(api):
    L = api.lib()
    assert L.spec_cache_append(None, *[None] * 4, 1, 1, 1, None, 0, 1, None, None, None, None, None) == api.SPEC_EINVAL
    assert L.spec_cache_workspace_size(api.OP_CACHE_ATTEND, None, 1, 1, 1) == 0


@pytest.mark.parametrize("call,bad", [
    (append, dict(B=-1)), (append, dict(n=-1)), (append, dict(rows=8)), (append, dict(index=FAKE, ist=4)), (append, dict(len=None)),
    (append, dict(new=None)), (append, dict(new=FAKE)), (append, dict(k=None)), (append, dict(v=None)), (append, dict(k=FAKE + 1)),
    (append, dict(ks=None)), (append, dict(vs=s3(-1, 0, 0))), (append, dict(dtype=0, k=FAKE + 2)),
    (attend, dict(B=-1)), (attend, dict(N=-1)), (attend, dict(N=4097)), (attend, dict(Hq=0)), (attend, dict(Hq=12)),
    (attend, dict(q=None)), (attend, dict(out=None)), (attend, dict(len=None)), (attend, dict(scale=float("nan"))),
    (attend, dict(scale=float("inf"))), (attend, dict(cap=-1.0)), (attend, dict(cap=1e-30)), (attend, dict(cap=float("inf"))), (attend, dict(cap=float("nan"))), (attend, dict(q=FAKE + 1)),
    (attend, dict(qs=s3(0, -1, 0))), (attend, dict(os=None)),
    (weights, dict(B=-1)), (weights, dict(N=4097)), (weights, dict(rows=8)), (weights, dict(index=FAKE, ist=8)), (weights, dict(Hq=9)),
    (weights, dict(q=None)), (weights, dict(lse=None)), (weights, dict(out=None)), (weights, dict(len=None)),
    (weights, dict(cap=-0.5)), (weights, dict(scale=float("nan"))), (weights, dict(prev=FAKE)), (weights, dict(pos=-1)),
    (weights, dict(os=s2(-1, 0))), (weights, dict(ls=None)), (weights, dict(ls=s3(288, 32, -1))),
    (evict, dict(B=-1)), (evict, dict(keep=0)), (evict, dict(keep=-3)), (evict, dict(recent=-1)), (evict, dict(recent=17)),
    (evict, dict(len=None)), (evict, dict(w=None)), (evict, dict(kept=None)), (evict, dict(new=None)), (evict, dict(new=FAKE)),
    (evict, dict(pos=-1)), (evict, dict(ws=None)),
])
def test_bad_arguments(api, call, bad):
    n0 = api.launch_count()
    assert call(api, **bad) == api.SPEC_EINVAL
    assert api.launch_count() == n0


@pytest.mark.parametrize("other", [dict(kv_heads=4), dict(page_size=32), dict(head_dim=64)])
def test_evict_needs_one_geometry(api, other):
    assert evict(api, d=cache(api, **other)) == api.SPEC_EINVAL


def test_dtypes(api):
    for call, codes in ((append, (3, 7, -1)), (attend, (0, 3, 7)), (weights, (0, 3, -1))):
        for code in codes:
            assert call(api, dtype=code) == api.SPEC_EDTYPE, (call, code)


def test_nothing_to_do(api):
    n0 = api.launch_count()
    for call in (append, attend, weights, evict):
        assert call(api, B=0) == api.SPEC_OK
    assert attend(api, N=0) == api.SPEC_OK
    assert api.launch_count() == n0


def test_workspaces(api):
    """A call whose geometry asks for a workspace refuses one that is missing, misaligned or too small."""
    c = cache(api)
    for call, op, args in ((attend, api.OP_CACHE_ATTEND, (2, 9, 32)), (weights, api.OP_CACHE_WEIGHTS, (2, 9, 32)),
                           (evict, api.OP_CACHE_EVICT, (2, 16, 0))):
        need = api.lib().spec_cache_workspace_size(op, ctypes.byref(c), *args)
        assert need % 256 == 0
        if need:
            key = "wsp" if call is evict else "ws"
            assert call(api, wsb=need - 1) == api.SPEC_EWORKSPACE
            assert call(api, **{key: None}) == api.SPEC_EWORKSPACE
            assert call(api, **{key: FAKE + 16}) == api.SPEC_EWORKSPACE
    size = api.lib().spec_cache_workspace_size
    assert size(99, ctypes.byref(c), 2, 9, 32) == 0
    assert size(api.OP_CACHE_ATTEND, ctypes.byref(c), -1, 9, 32) == 0
    assert size(api.OP_CACHE_ATTEND, ctypes.byref(cache(api, page_size=24)), 2, 9, 32) == 0


def test_status_strings(api):
    text = api.lib().spec_status_string
    assert b"page" in text(100 + api.STATUS_BAD_PAGE) and b"index" in text(100 + api.STATUS_BAD_INDEX)
