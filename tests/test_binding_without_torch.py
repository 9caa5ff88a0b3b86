"""The binding and its build where torch is not installed: the host calls, and
the per-step calls that take plain addresses, need none of it."""
import importlib.util
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
sys.modules["torch"] = None                      # as if it were not installed
import numpy as np
import paged_kv_cache_153_gb300 as pkv

pool = pkv.BlockPool(8)
a, b = pool.alloc(), pool.alloc()
pool.incref(b)
tables = np.array([[a, b], [b, -1]], dtype=np.int32)
src, dst = pkv.pkv_prepare_append(pool, tables, [20, 5])
assert len(src) == 1 and src[0] == b and pool.num_free == 5, (src, dst, pool.num_free)
assert pkv.pkv_blocks_needed(33) == 3 and pkv.pkv_version() > 0 and pkv.pkv_status_string(0)
turns, amplitude = pkv.pkv_rope_plan(64)
assert turns[0] > 0 and amplitude == 1.0

class Array:                                     # some other library's device array, with no tokens in it
    def __init__(self, *shape):
        self.shape = shape
    def numel(self):
        return int(np.prod(self.shape))
    def data_ptr(self):
        return 0
cache = Array(4, 2, 16, 64)
pkv.pkv_kv_append(Array(0, 2, 64), Array(0, 2, 64), Array(0), cache, cache, dtype=pkv.PKV_F16, stream=0)
try:
    pkv.pkv_select_blocks(Array(1, 2, 4), Array(1), Array(1, 2, 2), stream=0)
except ImportError as e:                         # a call that takes torch tensors
    assert "torch" in str(e), e
else:
    raise AssertionError("a tensor call without torch")
print("fine")
"""


def builder():
    spec = importlib.util.spec_from_file_location("pkv_build_probe", os.path.join(ROOT, "paged_kv_cache_153_gb300",
                                                                                 "_build.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_import_and_calls():
    builder().build()
    r = subprocess.run([sys.executable, "-c", SCRIPT], cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr


def test_importing_does_not_import_torch():
    builder().build()
    r = subprocess.run([sys.executable, "-c", "import sys, paged_kv_cache_153_gb300; print('torch' in sys.modules)"],
                       cwd=ROOT, capture_output=True, text=True, timeout=120)
    assert r.stdout.strip() == "False", r.stdout + r.stderr


def test_build_without_torch(monkeypatch):
    m = builder()
    with_torch = m.outputs()
    assert m.TENSOR_PATH in with_torch
    monkeypatch.setitem(sys.modules, "torch", None)
    without = m.outputs()
    assert m.TENSOR_PATH not in without and set(without) < set(with_torch) and m.CALL_PATH in without
    assert m._source_digest()


def test_a_missing_tensor_module_fails_at_import(tmp_path):
    # (torch is there, the module that takes its tensors is not)
    import shutil
    m = builder()
    m.build()
    pkg = tmp_path / "paged_kv_cache_153_gb300"
    pkg.mkdir()
    for name in ("__init__.py", "libpkv.so", "_call.so"):
        shutil.copy(os.path.join(m.PKG_DIR, name), pkg / name)
    r = subprocess.run([sys.executable, "-c", "import paged_kv_cache_153_gb300"], cwd=tmp_path, capture_output=True,
                       text=True, timeout=120)
    assert r.returncode != 0 and "ImportError" in r.stderr and "_tensor" in r.stderr, r.stderr


