"""What the build and the import need, on the CPU: the C library does without torch, and the binding's older parts
without the module that checks lists of tensors."""
import importlib.util
import os
import subprocess
import sys

import pytest

from tests.conftest import ROOT


def _script():
    """The build script by path, as a module of its own."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, "fp4_rollout_guided_amd", "build.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("torch_there", [True, False])
def test_build_without_torch(monkeypatch, tmp_path, torch_there):
    build = _script()
    started, put = [], []

    class Done:
        returncode, stdout, stderr = 0, "", ""

        def __init__(self, cmd, **_):
            started.append(cmd)

        def communicate(self):
            return "", ""
    monkeypatch.setattr(build.subprocess, "Popen", Done)
    monkeypatch.setattr(build.subprocess, "run", Done)
    monkeypatch.setattr(build.os, "replace", lambda a, b: put.append(b))
    monkeypatch.setattr(build, "CEILING_BIN", str(tmp_path / "ceiling" / "bin"))
    if not torch_there:
        monkeypatch.setitem(sys.modules, "torch", None)
        find = importlib.util.find_spec
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda n, *a: None if n == "torch" else find(n, *a))
    assert build.build() == build.LIB
    assert build.LIB in put and build.SMALLGRID_LIB in put
    assert (build.LISTS_LIB in put) == torch_there
    assert any("tensor_lists.cpp" in str(c) for c in started) == torch_there


def test_binding_without_its_list_module():
    """What does not use the module (built for another torch, say) is there without it; what does says what is missing."""
    code = ("import sys; sys.modules['fp4_rollout_guided_amd._tensor_lists'] = None\n"
            "import torch, fp4_rollout_guided_amd as tr\n"
            "assert tr.abi_version() > 0 and tr.step_revision() > 0\n"
            "t = torch.zeros(4)\n"
            "try:\n"
            "    tr._outs(t, 16, None, (None, 'out', (4,), torch.float32))\n"
            "except ImportError as e:\n"
            "    assert 'build.py' in str(e)\n"
            "    print('refused')\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert out.returncode == 0 and out.stdout.strip().endswith("refused"), out.stdout


def test_list_module_built_after_the_first_import():
    """Loaded again, the binding finds the module that was missing before."""
    code = ("import importlib, sys; name = 'fp4_rollout_guided_amd._tensor_lists'; sys.modules[name] = None\n"
            "import fp4_rollout_guided_amd as tr\n"
            "del sys.modules[name]\n"
            "importlib.reload(tr)\n"
            "assert tr._tensor_lists.changed([]) is None\n")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert out.returncode == 0, out.stdout
