"""The paged cache's extension module is loaded by the paged cache alone, and built again for another torch (no GPU
needed)."""
import os
import subprocess
import sys

import __graft_entry__

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_package_does_without_the_extension_module():
    """With a _paged.so that cannot be loaded the rest of the package works; a paged cache says what is wrong."""
    __graft_entry__._load_build_module().build()
    code = """
import sys
sys.modules["clustered_sparse_kv_gb300._paged"] = None      # an import of it raises
import clustered_sparse_kv_gb300 as wi
assert wi.lib.wi_free and wi.make_config(1, 1, 4, 1, 1024) and wi.WaveIndex
p = wi.LruPolicy(4, 2, 1)
assert p.round([1], 0) == ([], [(1, 0)])
try:
    wi.PagedCache(wi.make_paged_config(4, 1, 16, 8, 1, 4))
except ImportError as e:
    assert "_paged.so" in str(e)
    print("said so")
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and "said so" in r.stdout, r.stdout + r.stderr


def test_another_torch_or_python_means_another_build(monkeypatch, tmp_path):
    """Files newer than every source are kept only while the extension module's Python and torch are those of now."""
    b = __graft_entry__._load_build_module()
    b.build()
    assert b.is_current()
    for name in ("LIB", "EXT", "STAMP"):
        f = tmp_path / name
        f.write_text(open(b.STAMP).read() if name == "STAMP" else "")
        monkeypatch.setattr(b, name, str(f))
    assert b.is_current()
    monkeypatch.setattr(b, "_torch_of_this_python", lambda: "3.12 | torch 0.0")
    assert not b.is_current()
    monkeypatch.undo()
    monkeypatch.setattr(b, "STAMP", str(tmp_path / "none"))
    assert not b.is_current()
