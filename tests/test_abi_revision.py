"""A C caller can tell a library with the products and the routed rows from an
older one of the same ABI version (no GPU call)."""
import os
import shutil
import subprocess

import pytest

import fp4_rollout_guided_amd as tr

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CALLER = ('#include "trace.h"\n'
          "int main(void) {\n"
          "  return trace_abi_version() == TRACE_ABI_VERSION && trace_abi_revision() >= TRACE_ABI_REVISION ? 0 : 1;\n"
          "}\n")
OLDER = "int trace_abi_version(void) { return 10; }\n"


def _link(cc, src, libdir, lib, exe):
    return subprocess.run([cc, "-std=c99", "-Wall", "-Wextra", "-Werror", "-pedantic", "-I", os.path.join(ROOT, "include"),
                           str(src), "-L", str(libdir), f"-l:{lib}", f"-Wl,-rpath,{libdir}", "-o", str(exe)],
                          capture_output=True, text=True)


def test_revision(tmp_path):
    assert tr.abi_revision() == 1
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    src, exe = tmp_path / "caller.c", tmp_path / "caller"
    src.write_text(CALLER)
    built = _link(cc, src, os.path.dirname(tr.LIB_PATH), os.path.basename(tr.LIB_PATH), exe)
    assert built.returncode == 0, built.stderr
    assert subprocess.run([str(exe)]).returncode == 0
    # a library of the same version without the additions: the caller does not link, and, linked before, does not run
    (tmp_path / "older.c").write_text(OLDER)
    subprocess.run([cc, "-shared", "-fPIC", str(tmp_path / "older.c"), "-o", str(tmp_path / "libtrace.so")], check=True)
    refused = _link(cc, src, tmp_path, "libtrace.so", tmp_path / "other")
    assert refused.returncode != 0 and "trace_abi_revision" in refused.stderr
    env = dict(os.environ, LD_LIBRARY_PATH=str(tmp_path))
    again = subprocess.run([cc, str(src), "-I", os.path.join(ROOT, "include"), "-L", os.path.dirname(tr.LIB_PATH),
                            "-l:libtrace.so", "-o", str(exe)], capture_output=True, text=True)
    assert again.returncode == 0, again.stderr
    assert subprocess.run([str(exe)], env=env, capture_output=True).returncode != 0
