"""The build's reuse of objects, with a stand-in for nvcc."""
import os
import stat
import sys
import time

import pytest

from kv_cache_retrieval_b200 import build as kbuild

NVCC = """#!{python}
import os, sys, time
a = sys.argv[1:]
out = a[a.index("-o") + 1]
root = {root!r}
with open(os.path.join(root, "calls"), "a") as f:
    f.write(("link" if "-shared" in a else os.path.basename(a[a.index("-c") + 1])) + "\\n")
text = ""
for f in a:
    if os.path.isfile(f) and f != out:
        text += open(f).read()
if os.path.exists(os.path.join(root, "edit")):      # someone saves a source while it is compiled
    os.remove(os.path.join(root, "edit"))
    time.sleep(0.05)
    with open(os.path.join(root, "csrc", "a.cu"), "a") as f:
        f.write("// edited\\n")
    time.sleep(0.05)
if os.path.exists(os.path.join(root, "fail")):
    open(out, "w").write("half a f")
    sys.exit(1)
open(out, "w").write(text)
"""


@pytest.fixture
def tree(tmp_path, monkeypatch):
    for d in ("csrc", "include"):
        (tmp_path / d).mkdir()
    (tmp_path / "include" / "hhr.h").write_text("// api\n")
    (tmp_path / "csrc" / "x.cuh").write_text("// x\n")
    (tmp_path / "csrc" / "a.cu").write_text('#include "x.cuh"\n')
    (tmp_path / "csrc" / "b.cu").write_text('#include "hhr.h"\n')
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(NVCC.format(python=sys.executable, root=str(tmp_path)))
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    for name, value in (("CSRC", "csrc"), ("INCLUDE", "include"), ("BUILD", "_build"), ("LIB", "lib.so")):
        monkeypatch.setattr(kbuild, name, str(tmp_path / value))
    monkeypatch.setattr(kbuild, "SOURCES", ["a.cu", "b.cu"])
    monkeypatch.setattr(kbuild, "_nvcc", lambda: str(nvcc))

    def calls():
        at = tmp_path / "calls"
        done = sorted(at.read_text().split()) if at.exists() else []
        at.write_text("")
        return done
    old = time.time() - 100
    for d in ("csrc", "include"):
        for f in (tmp_path / d).iterdir():
            os.utime(f, (old, old))
    return tmp_path, calls


def touch(f):
    time.sleep(0.02)
    f.write_text(f.read_text() + "// more\n")


def test_only_what_changed_is_compiled(tree):
    at, calls = tree
    kbuild.build()
    assert calls() == ["a.cu", "b.cu", "link"]
    kbuild.build()
    assert calls() == []
    touch(at / "csrc" / "x.cuh")
    kbuild.build()
    assert calls() == ["a.cu", "link"]
    touch(at / "include" / "hhr.h")
    kbuild.build()
    assert calls() == ["b.cu", "link"]


def test_a_source_saved_during_the_build_is_compiled_again(tree):
    at, calls = tree
    kbuild.build()
    touch(at / "csrc" / "a.cu")
    (at / "edit").write_text("")
    kbuild.build()
    calls()
    kbuild.build()
    assert calls() == ["a.cu", "link"]
    assert "edited" in (at / "lib.so").read_text()


def test_a_failed_compilation_leaves_no_object(tree):
    at, calls = tree
    (at / "fail").write_text("")
    with pytest.raises(RuntimeError):
        kbuild.build()
    (at / "fail").unlink()
    calls()
    kbuild.build()
    assert "a.cu" in calls() and "half" not in (at / "lib.so").read_text()
