"""The host extension is rebuilt for another torch, and refuses one it was not built for."""
import subprocess
import sys

from mla_latent_kv_07_gb300 import build


def test_it_is_stale_for_another_torch(tmp_path, monkeypatch):
    built = tmp_path / "_mla_native.so"
    monkeypatch.setattr(build, "NATIVE", str(built))
    stamp = tmp_path / "_mla_native.so.stamp"
    built.write_bytes(b"")
    assert build.native_stale()                      # no record of what it was built against
    stamp.write_text(build.native_stamp())
    assert not build.native_stale()
    version = build.torch_version()
    monkeypatch.setattr(build, "torch_version", lambda: version + "1")
    assert build.native_stale()
    stamp.write_text(build.native_stamp())
    assert not build.native_stale()
    built.unlink()
    assert build.native_stale()


def test_it_is_not_used_with_another_torch():
    build.build()
    code = """
import torch
import mla_latent_kv_07_gb300 as mla
right = torch.__version__
torch.__version__ = "1.0.0"
try:
    mla.native()
    raise SystemExit("used")
except RuntimeError as e:
    assert "built against torch" in str(e) and mla._host is None
torch.__version__ = right
assert mla.native().torch_version == right
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=build.ROOT)
    assert r.returncode == 0, r.stdout + r.stderr
