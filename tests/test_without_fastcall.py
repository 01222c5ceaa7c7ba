"""The library without the _fastcall extension (another interpreter's build, or
one without Python's headers): the calls that go through ctypes work, the
others say what is missing."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CODE = """
import torch
from paged_kv_cache_480_b200 import binding as b
b.FASTCALL_PATH = b.FASTCALL_PATH + ".none"
b.load_library()
m = b.BlockManager(4, 16)
m.allocate(1, 20)
assert m.num_free() == 2
assert b.paged_attention_workspace_size(8, 8, 8, 64, 16, 512, 1) > 0
f, att = b.rotary_frequencies(64)
assert f.shape == (32,)
try:
    b._load_fast()
except FileNotFoundError as e:
    assert "_fastcall" in str(e)
else:
    raise AssertionError("no error")
b.FASTCALL_PATH = b.FASTCALL_PATH[:-len(".none")]
assert b._load_fast() is b._fast is not None     # built since
"""


def test_calls_without_the_extension():
    run = subprocess.run([sys.executable, "-c", CODE], cwd=ROOT, capture_output=True, text=True)
    assert run.returncode == 0, run.stderr


def test_building_without_pythons_headers(monkeypatch, tmp_path, capsys):
    """The library is built, the extension left out."""
    from paged_kv_cache_480_b200 import build
    built = []
    monkeypatch.setattr(build, "_run", lambda cmd: built.append(cmd[-1]) or "")
    monkeypatch.setattr(build, "_stale", lambda *a: False)
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    monkeypatch.setattr(build.os, "replace", lambda a, b: None)
    assert build.build() == build.LIB
    assert not any("fastcall" in c for c in built) and "Python.h" in capsys.readouterr().err
