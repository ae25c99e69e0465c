"""The build's and the import's needs (no GPU needed): libattn.so takes nvcc alone, and
only the calls of the binding's native part need that part."""
import importlib.util
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def b(tmp_path, monkeypatch):
    """The build module with a folder of its own and a compiler that only writes its output."""
    from transformer_attention_fwd_gb300 import build
    spec = importlib.util.spec_from_file_location("build_under_test", build.__file__)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    fake = tmp_path / "cc"
    fake.write_text("#!/bin/sh\nwhile [ $# -gt 0 ]; do [ \"$1\" = -o ] && echo built > \"$2\"; shift; done\n")
    fake.chmod(0o755)
    monkeypatch.setattr(m, "BUILD", str(tmp_path / "out"))
    monkeypatch.setattr(m, "LIB", str(tmp_path / "out" / "libattn.so"))
    monkeypatch.setattr(m, "BINDING", str(tmp_path / "out" / "_attn_binding.so"))
    monkeypatch.setattr(m, "nvcc", lambda: str(fake))
    return m


def _hide_torch(monkeypatch):
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))


def test_the_library_builds_without_torch(b, monkeypatch):
    _hide_torch(monkeypatch)
    assert b.is_stale()
    assert b.build() == b.LIB and os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
    assert not b.is_stale()


def test_the_library_is_there_when_the_binding_fails(b, monkeypatch):
    monkeypatch.setattr(b, "_binding_compile", lambda obj: ["false"])
    with pytest.raises(RuntimeError, match="binding"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)
    assert b.is_stale()


def test_a_missing_binding_alone_is_built(b, monkeypatch):
    for name in ("_binding_compile", "_binding_link"):
        monkeypatch.setattr(b, name, lambda *a: [b.nvcc(), "-o", a[-1]])
    b.build()
    assert os.path.exists(b.BINDING) and not b.is_stale()
    first = os.stat(b.LIB).st_mtime_ns
    os.remove(b.BINDING)
    assert b.is_stale()
    b.build()
    assert os.path.exists(b.BINDING) and os.stat(b.LIB).st_mtime_ns == first


def test_the_older_calls_import_without_the_native_part(tmp_path):
    from transformer_attention_fwd_gb300 import build
    build.build()
    package = tmp_path / "transformer_attention_fwd_gb300"
    (package / "_build").mkdir(parents=True)
    for name in ("__init__.py", "attn.py", "build.py", "inputs.py"):
        os.symlink(os.path.join(ROOT, "transformer_attention_fwd_gb300", name), package / name)
    os.symlink(build.LIB, package / "_build" / "libattn.so")
    code = """
import torch
from transformer_attention_fwd_gb300 import attn
print(attn.rope_turns(64)[1], attn.last_launch_info())
try:
    attn.Rotation(torch.zeros(32, dtype=torch.int64))
except RuntimeError as e:
    print(e)
"""
    r = subprocess.run([sys.executable, "-c", code], cwd=tmp_path, capture_output=True, text=True,
                       env={**os.environ, "PYTHONPATH": str(tmp_path)})
    assert r.returncode == 0, r.stderr
    assert "_attn_binding.so is missing" in r.stdout


def test_a_binding_of_another_torch_is_stale_and_refused(b, monkeypatch):
    import torch
    from transformer_attention_fwd_gb300 import attn, build
    build.build()
    assert build.installed_torch() == torch.__version__ and not build.is_stale()
    for name in ("_binding_compile", "_binding_link"):
        monkeypatch.setattr(b, name, lambda *a: [b.nvcc(), "-o", a[-1]])
    b.build()
    assert not b.is_stale()
    first = os.stat(b.BINDING).st_ino
    monkeypatch.setattr(b, "installed_torch", lambda: "0.1")
    assert b.is_stale()
    b.build()
    assert not b.is_stale() and os.stat(b.BINDING).st_ino != first
    monkeypatch.setattr(build, "binding_built_for", lambda: "torch 0.1, other")
    with pytest.raises(RuntimeError, match="built for torch 0.1"):
        attn._load_binding()


def test_a_rebuild_never_leaves_the_binding_without_its_mark(b, monkeypatch):
    """Another process may load the binding while this one builds it again."""
    for name in ("_binding_compile", "_binding_link"):
        monkeypatch.setattr(b, name, lambda *a: [b.nvcc(), "-o", a[-1]])
    b.build()
    seen, link = [], b._link

    def watched(cmd, target):
        seen.append(b.binding_built_for())
        link(cmd, target)
        seen.append(b.binding_built_for())

    monkeypatch.setattr(b, "_link", watched)
    b.build(force=True)
    assert len(seen) == 4 and set(seen) == {b.binding_for(b.installed_torch())}
