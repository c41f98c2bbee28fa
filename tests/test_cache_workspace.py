"""Workspaces of the 8-bit cache's operators, on the host: sizes, and calls that are given none, too little or a misaligned one."""
import ctypes

import pytest

from test_cache_abi import FAKE, api, attend, cache, evict, weights  # noqa: F401

ROOMY = 400  # pages to a request: contexts for which attention is cut over the SMs


def test_attention_that_is_cut_over_the_gpu_needs_a_workspace(api):  # noqa: F811
    c = cache(api, table_stride=ROOMY)
    need = api.lib().spec_cache_workspace_size(api.OP_CACHE_ATTEND, ctypes.byref(c), 2, 9, 32)
    assert need > 0 and need % 256 == 0
    n0 = api.launch_count()
    for bad in (dict(ws=None), dict(ws=FAKE + 16), dict(ws=FAKE + 128), dict(wsb=need - 1), dict(wsb=0), dict(ws=None, wsb=0)):
        assert attend(api, c, **bad) == api.SPEC_EWORKSPACE, bad
    assert api.launch_count() == n0


@pytest.mark.parametrize("rows", [1, 9, 60])
@pytest.mark.parametrize("head_dim", [64, 128])
def test_sizes_do_not_grow_with_the_batch(api, rows, head_dim):  # noqa: F811
    """A workspace is the size of what the SMs hand on, whatever the batch; a call of the same geometry asks for the same."""
    c = cache(api, table_stride=ROOMY, head_dim=head_dim)
    size = api.lib().spec_cache_workspace_size
    sizes = {size(api.OP_CACHE_ATTEND, ctypes.byref(c), B, rows, 32) for B in (32, 64, 300)}
    assert len(sizes) == 1


@pytest.mark.parametrize("head_dim", [16, 80, 256])
def test_other_widths_need_none(api, head_dim):  # noqa: F811
    c = cache(api, table_stride=ROOMY, head_dim=head_dim, page_stride=8 * 64 * 256)
    assert api.lib().spec_cache_workspace_size(api.OP_CACHE_ATTEND, ctypes.byref(c), 2, 9, 32) == 0


def test_weights_and_eviction_need_none(api):  # noqa: F811
    c = cache(api, table_stride=ROOMY)
    size = api.lib().spec_cache_workspace_size
    assert size(api.OP_CACHE_WEIGHTS, ctypes.byref(c), 2, 9, 32) == 0
    assert size(api.OP_CACHE_EVICT, ctypes.byref(c), 2, 16, 0) == 0
    n0 = api.launch_count()
    assert weights(api, c, B=0, ws=None, wsb=0) == evict(api, c, B=0, wsp=None, wsb=0) == api.SPEC_OK
    assert api.launch_count() == n0
