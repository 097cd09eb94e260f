"""What the package needs to load and what its build leaves behind (CPU): the calls on device arrays of pointers need
libmuon.so alone; only the calls on lists of tensors need the extension module and the newer entry points."""
import os
import re
import shutil
import subprocess
import sys

import pytest

import matrix_orthogonalizing_optimizer_step_amd as mu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.dirname(os.path.abspath(mu.__file__))

# Calls that worked before there was an extension module, then one call of each kind that needs it.
PROBE = """
import torch
import matrix_orthogonalizing_optimizer_step_amd as mu
assert mu.abi_version() == 6
assert mu.workspace_size(1, 256, 512) > 0 and mu.grasp_workspace_size(1, 256, 512, 0) > 0
for call in (lambda: mu.adamw_step([], [], [], [], 1, 1e-3),
             lambda: mu.adamw8_step([], mu.AdamW8State([], [], [], []), [], 1, 1e-3),
             lambda: mu.mx4_quantize([torch.zeros(2, 2)]), lambda: mu.mx4_matmul(mu.MX4([], [], 1), mu.MX4([], [], 1))):
    try:
        call()
    except ImportError as e:
        print("refused:", e)
    else:
        raise SystemExit("a call on a list ran")
"""


def run_probe(cwd, **env):
    out = subprocess.run([sys.executable, "-c", PROBE], cwd=cwd, env=dict(os.environ, PYTHONPATH=str(cwd), **env),
                         capture_output=True, text=True, timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr
    return [line for line in out.stdout.splitlines() if line.startswith("refused:")]


def copy_package(to):
    shutil.copytree(PACKAGE, os.path.join(to, os.path.basename(PACKAGE)),
                    ignore=shutil.ignore_patterns("__pycache__", "csrc", "native", "_native*"))
    return os.path.join(to, os.path.basename(PACKAGE))


@pytest.mark.parametrize("kind", ["missing", "unfit"])
def test_muon_calls_need_no_extension_module(tmp_path, kind):
    package = copy_package(str(tmp_path))
    if kind == "unfit":
        with open(os.path.join(package, "_native.so"), "wb") as f:
            f.write(b"not a shared object")
    refusals = run_probe(tmp_path)
    assert len(refusals) == 4 and all("_native.so is missing or does not fit" in r for r in refusals)


def test_muon_calls_need_no_newer_entry_points(tmp_path):
    """A library without the calls on lists (a stand-in with the other functions only)."""
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "muon.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b([a-z_][a-z0-9_]*)\s*\(", text)) - {"sizeof"})
    old = [n for n in names if "adamw" not in n and "mx4" not in n]
    assert len(names) - len(old) == 7
    source = tmp_path / "old.c"
    source.write_text("\n".join(f"unsigned long {n}(void) {{ return {6 if n == 'muon_abi_version' else 256}; }}" for n in old))
    lib = tmp_path / "libold.so"
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(lib), str(source)], check=True)
    refusals = run_probe(ROOT, MUON_LIBRARY=str(lib))
    assert len(refusals) == 4 and all("older build of the library" in r for r in refusals)
