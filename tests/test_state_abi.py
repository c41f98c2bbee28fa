"""The linear-attention states' C ABI and binding without a GPU: every bad argument is refused on the host and nothing is
launched."""
import ctypes

import pytest
import torch

FAKE = 0x100000  # never dereferenced: every call below fails validation or has nothing to do


@pytest.fixture(scope="module")
def api():
    from speculative_decoding_verification_02_gb300 import api, build
    build.build()
    api.lib()
    return api


def pool(api, **kw):
    a = dict(state=FAKE, slot_stride=48 * 128 * 128, num_slots=4, heads=48, key_dim=128, value_dim=128, slots=None)
    a.update(kw)
    return api._StateStruct(*a.values())


def s3(*s):
    return (ctypes.c_int64 * 3)(*s)


ROW = s3(1 << 20, 16 * 128, 128)
WIDE = s3(1 << 20, 48 * 128, 128)


def ref(x):
    return None if x is None else ctypes.byref(x)


def forward(api, c="pool", d="pool", **kw):
    c, d = (pool(api) if x == "pool" else x for x in (c, d))
    a = dict(q=FAKE, qs=ROW, k=FAKE, ks=ROW, v=FAKE, vs=WIDE, dtype=1, B=2, n=9, Hk=16, g=FAKE, gs=s3(1 << 10, 48, 1), counts=None,
             scale=0.1, out=FAKE, os=WIDE, status=None, ws=FAKE, wsb=1 << 40, stream=None)
    a.update(kw)
    return api.lib().spec_state_forward(ref(c), ref(d), *a.values())


def attend(api, c="pool", d=None, **kw):
    c = pool(api) if c == "pool" else c
    a = dict(q=FAKE, qs=ROW, k=FAKE, ks=ROW, v=FAKE, vs=WIDE, dtype=1, B=2, n=9, Hk=16, g=FAKE, gs=s3(1 << 10, 48, 1), parents=None,
             nq=None, scale=0.1, out=FAKE, os=WIDE, status=None, ws=FAKE, wsb=1 << 40, stream=None)
    a.update(kw)
    return api.lib().spec_state_attend(ref(c), *a.values())


def commit(api, c="pool", d="pool", **kw):
    c, d = (pool(api) if x == "pool" else x for x in (c, d))
    a = dict(k=FAKE, ks=ROW, v=FAKE, vs=WIDE, dtype=1, B=2, n=9, Hk=16, g=FAKE, gs=s3(1 << 10, 48, 1), index=None, ist=0, rows=9,
             counts=None, status=None, stream=None)
    a.update(kw)
    return api.lib().spec_state_commit(ref(c), ref(d), *a.values())


BAD_POOLS = [dict(heads=0), dict(heads=1 << 16), dict(key_dim=8), dict(key_dim=120), dict(key_dim=272), dict(value_dim=0),
             dict(value_dim=72), dict(value_dim=512), dict(num_slots=0), dict(slot_stride=48 * 128 * 128 - 4),
             dict(slot_stride=48 * 128 * 128 + 2), dict(state=FAKE + 4)]


@pytest.mark.parametrize("call", [forward, attend, commit])
def test_bad_pools(api, call):
    n0 = api.launch_count()
    for bad in BAD_POOLS:
        assert call(api, c=pool(api, **bad)) == api.SPEC_EINVAL, bad
        if call is not attend:
            assert call(api, d=pool(api, **bad)) == api.SPEC_EINVAL, bad
    assert call(api, c=None) == api.SPEC_EINVAL
    assert api.launch_count() == n0


@pytest.mark.parametrize("call", [forward, commit])
def test_pools_that_differ(api, call):
    for other in (dict(heads=16), dict(key_dim=64), dict(value_dim=64)):
        assert call(api, d=pool(api, **other)) == api.SPEC_EINVAL


@pytest.mark.parametrize("call", [forward, attend, commit])
@pytest.mark.parametrize("bad", [dict(B=-1), dict(n=-1, rows=-1), dict(Hk=0), dict(Hk=5), dict(Hk=96), dict(ks=None), dict(vs=s3(-1, 0, 0)),
                                 dict(gs=s3(0, -1, 0)), dict(gs=None), dict(k=None), dict(v=None), dict(g=None), dict(g=FAKE + 2),
                                 dict(k=FAKE + 1), dict(v=FAKE + 1), dict(B=1 << 30)])
def test_bad_arguments(api, call, bad):
    n0 = api.launch_count()
    bad = {k: v for k, v in bad.items() if k != "rows" or call is commit}
    assert call(api, **bad) == api.SPEC_EINVAL
    assert api.launch_count() == n0


@pytest.mark.parametrize("call", [forward, attend])
@pytest.mark.parametrize("bad", [dict(q=None), dict(qs=None), dict(out=None), dict(os=s3(0, 0, -2)), dict(q=FAKE + 1), dict(out=FAKE + 1),
                                 dict(scale=float("nan")), dict(scale=float("inf"))])
def test_bad_outputs(api, call, bad):
    assert call(api, **bad) == api.SPEC_EINVAL


@pytest.mark.parametrize("call", [forward, attend, commit])
def test_bad_dtypes(api, call):
    for dtype in (0, 3, -1):
        assert call(api, dtype=dtype) == api.SPEC_EDTYPE


def test_bad_rows_and_sizes(api):
    assert commit(api, rows=8) == api.SPEC_EINVAL
    assert commit(api, index=FAKE, ist=4, rows=5) == api.SPEC_EINVAL
    assert commit(api, d=None) == api.SPEC_EINVAL
    assert commit(api, d=pool(api, state=None)) == api.SPEC_EINVAL
    assert attend(api, n=4097) == api.SPEC_EINVAL


@pytest.mark.parametrize("call", [forward, attend, commit])
def test_no_requests(api, call):
    n0 = api.launch_count()
    assert call(api, B=0) == api.SPEC_OK
    assert api.launch_count() == n0


def test_workspace_of_invalid_calls(api):
    size = api.lib().spec_state_workspace_size
    c = pool(api)
    assert size(api.OP_STATE_FORWARD, None, 1, 1) == 0
    for bad in BAD_POOLS[:8]:
        p = pool(api, **bad)
        assert size(api.OP_STATE_FORWARD, ctypes.byref(p), 2, 1000) == 0
    assert size(api.OP_STATE_FORWARD, ctypes.byref(c), -1, 10) == 0 and size(api.OP_STATE_FORWARD, ctypes.byref(c), 1, -1) == 0
    assert size(77, ctypes.byref(c), 1, 10) == 0


def test_status_text(api):
    assert b"slot" in api.lib().spec_status_string(100 + api.STATUS_BAD_SLOT)


def test_binding_packs_the_struct(api):
    """The packed bytes are those of the struct."""
    s = pool(api, slots=FAKE + 64)
    assert bytes(s) == api._pack_state(FAKE, 48 * 128 * 128, 4, 48, 128, 128, FAKE + 64)


def test_binding_refuses_pools(api):
    """What the binding looks at before it reaches the library."""
    dev = torch.device("cpu")

    class Dev:  # a device whose index is the host tensors' get_device()
        index = -1

    dims = (2, 16, 32)
    x = torch.zeros(3, 2, 16, 32)
    ok = api._state_struct(x, None, 3, dims, Dev, "state")
    assert len(ok) == ctypes.sizeof(api._StateStruct)
    for bad in (x.double(), x.half()):
        with pytest.raises(TypeError):
            api._state_struct(bad, None, 3, dims, Dev, "state")
    for bad in (x[0], x.transpose(2, 3), torch.zeros(3, 3, 16, 32), torch.zeros(3, 2, 16, 64)[..., ::2], torch.zeros(3, 4, 16, 32)[:, ::2]):
        with pytest.raises(ValueError):
            api._state_struct(bad, None, 3, dims, Dev, "state")
    with pytest.raises(TypeError):
        api._state_struct(x, torch.zeros(3, dtype=torch.int64), 3, dims, Dev, "state")
    with pytest.raises(ValueError):
        api._state_pools(None, None, None, torch.zeros(3, dtype=torch.int32), 3, dims, dev)
