"""The build's order and what makes it stale (no compiler is run: its commands are answered here)."""

import os
import subprocess
import warnings

import pytest
import torch

from attention_fa2_attn_gb300 import _lib, build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Outputs go to a directory of their own, and a command makes the file that follows its -o."""
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    monkeypatch.setattr(build, "BUILD_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / build.LIB_NAME))
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    ran = []

    def run(cmd, **kw):
        bad = tree_state["refuse"] and any(tree_state["refuse"] in c for c in cmd)
        ran.append(cmd)
        if not bad:
            open(cmd[cmd.index("-o") + 1], "w").write("x")
        return subprocess.CompletedProcess(cmd, 1 if bad else 0, "", "no" if bad else "")

    tree_state = {"refuse": None, "ran": ran}
    monkeypatch.setattr(build.subprocess, "run", run)
    return tree_state


def _extensions():
    return [f for f in os.listdir(build.HERE) if f.startswith("_fast") and f.endswith(".so")]


def test_a_whole_build_makes_both(tree):
    assert build.needs_build()
    build.build()
    assert os.path.exists(build.LIB_PATH) and len(_extensions()) == 1
    assert not build.needs_build()
    n = len(tree["ran"])
    build.build()
    assert len(tree["ran"]) == n


def test_the_library_does_not_need_the_extension(tree):
    # the C ABI needs neither the host compiler nor torch's headers
    tree["refuse"] = "fast_calls"
    with pytest.warns(RuntimeWarning, match="fast_calls"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not _extensions()
    # not tried again by every process that loads the library, but by a build that is asked for
    assert not build.needs_build()
    tree["refuse"] = None
    build.build(force=True)
    assert len(_extensions()) == 1


def test_the_library_is_what_a_build_is_for(tree):
    tree["refuse"] = "rope.cu"
    with pytest.raises(RuntimeError, match="rope.cu"):
        build.build()
    assert not os.path.exists(build.LIB_PATH)


def test_another_torch_makes_the_extension_stale(tree, monkeypatch):
    build.build()
    n = len(tree["ran"])
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert build.needs_build()
    build.build()
    new = tree["ran"][n:]
    assert new and not any(".cu" in c for cmd in new for c in cmd), "the library was not stale"
    assert not build.needs_build()
    assert len(_extensions()) == 2  # each torch loads its own


def test_sources_make_their_own_part_stale(tree):
    build.build()
    old = os.path.getmtime(build.FAST_SRC) - 100
    os.utime(build.fast_path(), (old, old))
    n = len(tree["ran"])
    assert build.needs_build()
    build.build()
    assert not any(c.endswith(".cu") for cmd in tree["ran"][n:] for c in cmd)


def test_without_the_extension_the_python_checks_take_the_calls(monkeypatch, tmp_path):
    _lib.lib()
    for path, text in ((tmp_path / "none.so", None), (tmp_path / "broken.so", "no library")):
        if text:
            path.write_text(text)
        monkeypatch.setattr(_lib._build, "fast_path", lambda p=path: str(p))
        monkeypatch.setattr(_lib, "_fast_calls", None)
        with pytest.warns(RuntimeWarning, match="extension"):
            f = _lib.fast()
        for call in ("paged_plan", "tree_mask", "rope", "rope_append_paged", "tree_decode_paged"):
            assert getattr(f, call)(1, 2, 3) is None
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            assert _lib.fast() is f  # said once
