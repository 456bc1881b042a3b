"""The 8-bit paged cache's entry points refuse bad arguments on the host (no GPU needed)."""
import pytest

import __graft_entry__


@pytest.fixture(scope="module")
def wi():
    __graft_entry__._load_build_module().build()
    import clustered_sparse_kv_gb300 as m
    return m


def test_calls_on_null_handle(wi):
    lib = wi.lib
    assert lib.wi_paged_axes(None, 1, None) == -1 and lib.wi_last_error()
    assert lib.wi_paged_write8(None, 1, 16, 8, 16, 8, 16, 8, None, None, 16, 16, 16, 16, 16, 16, 16, None) == -1
    assert lib.wi_paged_attention8(None, 1, 1, 16, 16, 16, 16, 16, 16, 16, 16, 16, None, None) == -1
    assert lib.wi_paged_gather8(None, 1, 1, 16, 16, 16, 16, 16, 16, 0, 1, 16, 16, None) == -1


def test_python_calls_check_their_tensors_before_the_library(wi):
    """The Python calls' checks, without a device: a context of handle 0 that no checked call reaches."""
    import torch

    from clustered_sparse_kv_gb300 import _paged
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros((4, 4, 128), dtype=torch.bfloat16)
    ctx = _paged.context(0, 0, 4, 2, 16, 8, 4)
    for call, n in ((_paged.write8, 14), (_paged.attention8, 12), (_paged.gather8, 11)):
        with pytest.raises(TypeError, match="arguments"):
            call(ctx, *[x] * (n - 2))
        with pytest.raises(ValueError, match="freed"):
            call(None, *[x] * (n - 1))
    with pytest.raises(ValueError, match=r"q must be .*\(4, 4, 128\) .*on cpu"):
        _paged.attention8(ctx, x, x, x, x, x, i, i, i, x, None, 0)
    with pytest.raises(ValueError, match="q must be .*contiguous heads"):
        _paged.write8(ctx, x.transpose(0, 1), x, x, i, i, x, x, x, x, x, None, None, 0)
    with pytest.raises(ValueError, match="k_out must have shape"):
        _paged.gather8(ctx, x, x, x, x, i, i, 0, x, x, 0)


def test_axes_are_checked_before_a_cache_is_made(wi):
    cfg = wi.make_paged_config(4, 2, 16, 8, 2, 4)
    for bad in ([0] * 63, [], [0] * 65, [-1] + [0] * 63):
        with pytest.raises(ValueError, match="rotary_dim"):
            wi.PagedCache(cfg, axes=bad)
