"""The paged cache's entry points refuse bad arguments on the host with the documented codes (no GPU needed),
and wi_paged_config has the same layout in C as in the binding."""
import ctypes
import os
import subprocess

import pytest

import __graft_entry__

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def wi():
    __graft_entry__._load_build_module().build()
    import clustered_sparse_kv_gb300 as m
    return m


def good(wi, **kw):
    base = dict(n_q_heads=8, n_kv_heads=2, page_size=16, n_pages=64, max_batch=4, max_pages=8)
    return wi.make_paged_config(**{**base, **kw})


@pytest.mark.parametrize("kw,code", [
    (dict(head_dim=64), -1),
    (dict(n_q_heads=7), -1),
    (dict(n_kv_heads=0), -1),
    (dict(page_size=8), -1),
    (dict(page_size=24), -1),
    (dict(page_size=-16), -1),
    (dict(n_pages=0), -1),
    (dict(max_batch=0), -1),
    (dict(max_pages=0), -1),
    (dict(rotary_dim=132), -1),
    (dict(rotary_dim=20), -1),
    (dict(rotary_dim=-8, inv_freq=[]), -1),
    (dict(eps=0.0), -1),
    (dict(eps=float("nan")), -1),
    (dict(eps=1e-60), -1),
    (dict(rope_scale=float("inf")), -1),
    (dict(rotary_dim=8, inv_freq=[1.0, 0.5, float("nan"), 0.1]), -1),
    (dict(n_q_heads=18), -4),
    (dict(max_batch=4097), -4),
    (dict(n_pages=1 << 26), -4),       # 2^26 pages of 2 heads and 16 positions: 2^31 rows
    (dict(max_pages=1 << 27), -4),
])
def test_create_refuses_bad_config(wi, kw, code):
    out = ctypes.c_void_p(123)
    assert wi.lib.wi_paged_create(ctypes.byref(good(wi, **kw)), ctypes.byref(out)) == code
    assert out.value is None and wi.lib.wi_last_error()


def test_create_refuses_null_and_reserved(wi):
    out = ctypes.c_void_p(123)
    assert wi.lib.wi_paged_create(None, ctypes.byref(out)) == -1 and out.value is None
    assert wi.lib.wi_paged_create(ctypes.byref(good(wi)), None) == -1
    cfg = good(wi)
    cfg.interleaved = 2
    assert wi.lib.wi_paged_create(ctypes.byref(cfg), ctypes.byref(out)) == -1
    cfg = good(wi)
    cfg.reserved[1] = 1
    assert wi.lib.wi_paged_create(ctypes.byref(cfg), ctypes.byref(out)) == -1
    cfg = good(wi)
    cfg.inv_freq = None
    assert wi.lib.wi_paged_create(ctypes.byref(cfg), ctypes.byref(out)) == -1
    with pytest.raises(ValueError):
        good(wi, inv_freq=[1.0])


def test_calls_on_null_handle(wi):
    lib = wi.lib
    assert lib.wi_paged_check(None) == -1
    assert lib.wi_paged_tables(None, 1, 16, 16, 16, 16, 1, 16, 16, 16, 16, 16, 1, 16, None) == -1
    assert lib.wi_paged_write(None, 1, 16, 8, 16, 8, 16, 8, None, None, 16, 16, 16, 16, 16, None) == -1
    assert lib.wi_paged_attention(None, 1, 1, 16, 16, 16, 16, 16, 16, 16, None, None) == -1
    assert lib.wi_paged_gather(None, 1, 1, 16, 16, 16, 16, 0, 1, 16, 16, None) == -1
    lib.wi_paged_free(None)  # no-op


def test_config_layout_matches_binding(wi, tmp_path):
    fields = [n for n, _ in wi.wi_paged_config._fields_]
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "wave_index.h"\nint main(void) {\n'
                   '  printf("size %zu\\n", sizeof(wi_paged_config));\n'
                   + "".join(f'  printf("{f} %zu\\n", offsetof(wi_paged_config, {f}));\n' for f in fields)
                   + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"), str(src), "-o",
                    str(exe)], check=True)
    out = dict(line.split() for line in subprocess.run([str(exe)], check=True, capture_output=True,
                                                       text=True).stdout.splitlines())
    assert int(out["size"]) == ctypes.sizeof(wi.wi_paged_config)
    for f in fields:
        assert int(out[f]) == getattr(wi.wi_paged_config, f).offset, f


def test_python_calls_check_their_tensors_before_the_library(wi):
    """The Python calls' checks, without a device: a context of handle 0 that no checked call reaches."""
    import torch

    from clustered_sparse_kv_gb300 import _paged
    i = torch.zeros(4, dtype=torch.int32)
    x = torch.zeros((4, 4, 128), dtype=torch.bfloat16)
    ctx = _paged.context(0, 0, 4, 2, 16, 8, 4)
    for c in (None, 3):
        with pytest.raises(ValueError, match="freed"):
            _paged.tables(c, i, i, i, i, i, i, i, i, i, i, 0)
    with pytest.raises(TypeError, match="arguments"):
        _paged.attention(ctx, x)
    with pytest.raises(ValueError, match="ctx_len must be a tensor"):
        _paged.tables(ctx, [1], i, i, i, i, i, i, i, i, i, 0)
    with pytest.raises(ValueError, match="ctx_len .* on cuda:0 .*on cpu"):
        _paged.tables(ctx, i, i, i, i, i, i, i, i, i, i, 0)
    with pytest.raises(ValueError, match="dimension"):
        _paged.tables(ctx, torch.zeros((), dtype=torch.int32), i, i, i, i, i, i, i, i, i, 0)
    with pytest.raises(ValueError, match=r"q must be .*\(4, 4, 128\) .*on cpu"):
        _paged.attention(ctx, x, x, x, i, i, i, x, None, 0)
    with pytest.raises(ValueError, match="q must be .*contiguous heads"):
        _paged.write(ctx, x.transpose(0, 1), x, x, i, i, x, x, x, None, None, 0)
    with pytest.raises(ValueError, match="k_out must have shape"):
        _paged.gather(ctx, x, x, i, i, 0, x, x, 0)
