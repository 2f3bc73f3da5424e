"""What the build needs: the library nvcc alone, the binding torch and a C++ compiler.  Compilers are stand-ins here."""
import os
import shutil
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def tree(tmp_path):
    """A copy of the package's build files, and a PATH whose nvcc writes its output file and whose g++ fails."""
    pkg = tmp_path / "exact_attention_128_b200"
    (tmp_path / "bin").mkdir()
    pkg.mkdir()
    shutil.copy(os.path.join(ROOT, "exact_attention_128_b200", "build.py"), pkg)
    shutil.copytree(os.path.join(ROOT, "exact_attention_128_b200", "csrc"), pkg / "csrc")
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    for name, body in (("nvcc", 'while [ "$1" != -o ]; do shift; done; echo built > "$2"'), ("g++", "exit 1")):
        f = tmp_path / "bin" / name
        f.write_text("#!/bin/sh\n" + body + "\n")
        f.chmod(0o755)
    return pkg, {"PATH": f"{tmp_path / 'bin'}:/usr/bin:/bin", "HOME": str(tmp_path)}


def test_the_library_is_built_on_a_host_without_torch(tree):
    pkg, env = tree
    r = subprocess.run([sys.executable, "-S", str(pkg / "build.py")], env=env, capture_output=True, text=True)  # no site-packages
    assert r.returncode == 0, r.stderr
    assert (pkg / "libfa_b200.so").exists() and not (pkg / "_binding.so").exists()
    assert "torch is not installed" in r.stderr


def test_the_library_is_there_when_the_binding_fails(tree):
    pkg, env = tree
    r = subprocess.run([sys.executable, str(pkg / "build.py")], env=env, capture_output=True, text=True)
    assert r.returncode != 0 and "g++" in r.stderr
    assert (pkg / "libfa_b200.so").exists() and not (pkg / "_binding.so").exists()
