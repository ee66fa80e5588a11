"""The binding without the C++ side of its per-token calls, on the CPU: everything
imports and refuses as it does with it, and a build that cannot make it says so."""
import os
import subprocess
import sys

import pytest

from long_sequence_context_b200 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = (
    "import sys, types, warnings\n"
    "name = 'long_sequence_context_b200._calls'\n"
    "{plant}\n"
    "with warnings.catch_warnings(record=True) as seen:\n"
    "    warnings.simplefilter('always')\n"
    "    from long_sequence_context_b200 import cpattn as cp\n"
    "assert any('_calls.so is not used' in str(w.message) and {why!r} in str(w.message) for w in seen), seen\n"
    "assert cp.plan(256, 2, True) and cp.status_str(cp.ERR_PAGE)\n"
    "import pytest, torch\n"
    "sys.path.insert(0, {root!r})\n"
    "from tests import test_paged_cpu as t\n"
    "for fn, args, names in t.CALLS:\n"
    "    t.test_with_everything_right_only_the_device_is_left_to_refuse(fn, args)\n"
    "    for n in names:\n"
    "        t.test_each_tensor_argument_is_checked(fn, args, n)\n"
    "t.test_shapes_that_do_not_belong_together()\n"
    "print('done')\n")


@pytest.mark.parametrize("plant,why", [
    ("sys.modules[name] = None", "import"),
    ("m = sys.modules[name] = types.ModuleType(name)\n"
     "import long_sequence_context_b200 as p; p._calls = m; m.tag = 'torch 0.1, python 3.0'", "built for torch 0.1"),
    ("m = sys.modules[name] = types.ModuleType(name)\nimport long_sequence_context_b200 as p; p._calls = m", "tag"),
], ids=["missing", "another torch", "without a tag"])
def test_the_binding_works_without_calls(plant, why):
    r = subprocess.run([sys.executable, "-c", WITHOUT.format(plant=plant, why=why, root=ROOT)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("done"), r.stdout + r.stderr


@pytest.fixture
def folder(tmp_path, monkeypatch):
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    return tmp_path


def test_a_compiler_that_fails_is_reported_and_leaves_no_old_module(folder, monkeypatch):
    (folder / "_calls.so").write_bytes(b"of other sources")
    for cxx in ("/bin/false", str(folder / "missing")):
        monkeypatch.setattr(build, "CXX", cxx)
        with pytest.warns(UserWarning, match="_calls.so was not built"):
            build._try_calls(False)
        assert not (folder / "_calls.so").exists() and not (folder / "calls.tag").exists()


def test_another_torch_or_newer_sources_rebuild(folder, monkeypatch):
    made = []

    def fake(cmd, **kw):
        made.append(cmd)
        (folder / "_calls.so.tmp").write_bytes(b"x")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", fake)
    build._try_calls(False)
    build._try_calls(False)
    assert len(made) == 1
    path, version = build._torch()
    assert build.calls_tag(version) in (folder / "calls.tag").read_text()
    monkeypatch.setattr(build, "_torch", lambda: (path, "99.0"))
    build._try_calls(False)
    build._try_calls(False)
    assert len(made) == 2 and any("torch 99.0" in x for x in made[1])
    os.utime(folder / "_calls.so", (1, 1))
    build._try_calls(False)
    assert len(made) == 3


def test_version_read_from_the_file_is_the_installed_one():
    import torch
    assert build._torch()[1] == torch.__version__
