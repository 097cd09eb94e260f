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


# --- build ---------------------------------------------------------------------------------------------------------
@pytest.fixture
def fake_build(tmp_path, monkeypatch):
    """_build with a stand-in compiler: it fails on a source whose name is in a list, and otherwise writes its output."""
    from matrix_orthogonalizing_optimizer_step_amd import _build

    compiler = tmp_path / "fakecc"
    compiler.write_text("""#!/bin/sh
for a in "$@"; do
  case "$a" in *bad*) echo "bad source"; exit 3;; esac
  if [ "$last" = "-o" ]; then out="$a"; fi
  last="$a"
done
echo new > "$out"
""")
    compiler.chmod(0o755)
    lib, native = tmp_path / "libmuon.so", tmp_path / "_native.so"
    lib.write_text("old")
    native.write_text("old")
    monkeypatch.setattr(_build, "LIB", str(lib))
    monkeypatch.setattr(_build, "NATIVE", str(native))
    monkeypatch.setattr(_build, "SOURCES", ["one.hip", "two.hip"])
    monkeypatch.setattr(_build, "hipcc", lambda: str(compiler))
    monkeypatch.setattr(_build, "_native_command", lambda out: [str(compiler), "module.cpp", "-o", out])
    return _build, lib, native, compiler


def test_build_replaces_library_and_extension_together(fake_build):
    build, lib, native, compiler = fake_build
    assert build.build(lib=str(lib)) == str(lib)
    assert (lib.read_text(), native.read_text()) == ("new\n", "new\n")
    native.write_text("old")
    other = lib.with_name("libvariant.so")
    build.build(lib=str(other))  # a variant leaves the extension module as it is
    assert (other.read_text(), native.read_text()) == ("new\n", "old")


def test_failed_extension_leaves_the_old_pair(fake_build, monkeypatch):
    build, lib, native, compiler = fake_build
    monkeypatch.setattr(build, "_native_command", lambda out: ["/bin/sh", str(compiler), "bad.cpp", "-o", out])
    with pytest.raises(RuntimeError, match="sh failed on muon_native.cpp"):
        build.build(lib=str(lib))
    assert (lib.read_text(), native.read_text()) == ("old", "old")
    assert not list(lib.parent.glob("*.tmp"))


def test_failed_source_leaves_no_process_behind(fake_build, monkeypatch):
    build, lib, native, compiler = fake_build
    pid = lib.with_name("pid")
    monkeypatch.setattr(build, "SOURCES", ["one.hip", "bad.hip"])
    monkeypatch.setattr(build, "_native_command", lambda out: ["/bin/sh", "-c", f"echo $$ > {pid}; exec sleep 60"])
    with pytest.raises(RuntimeError, match="fakecc failed on bad.hip"):
        build.build(lib=str(lib))
    assert (lib.read_text(), native.read_text()) == ("old", "old")
    if pid.exists() and pid.read_text():  # it may have been ended before it wrote its number
        assert not os.path.exists(f"/proc/{pid.read_text().strip()}")
    assert not list(lib.parent.glob("*.tmp"))


def test_library_builds_without_torch_or_a_host_compiler(fake_build, monkeypatch, capsys):
    build, lib, native, compiler = fake_build
    monkeypatch.setattr(build, "_native_command", lambda out: None)
    build.build(lib=str(lib))
    assert lib.read_text() == "new\n" and not native.exists()
    assert "extension module is left out" in capsys.readouterr().err


def test_extension_command_needs_torch_and_a_compiler(monkeypatch):
    from matrix_orthogonalizing_optimizer_step_amd import _build

    assert _build._native_command("x.so") is not None
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)
        assert _build._native_command("x.so") is None
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(_build.shutil, "which", lambda name: None)
    assert _build._native_command("x.so") is None
