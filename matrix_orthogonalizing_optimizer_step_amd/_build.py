"""Compile the HIP sources of the Muon library into ``libmuon.so`` (gfx950) and
the list-marshalling extension module ``_native.so``.

``python -m matrix_orthogonalizing_optimizer_step_amd._build`` builds in
place; the shared libraries sit next to this file so they travel with the
source tree.
"""
from __future__ import annotations

import os
import shutil
import signal
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libmuon.so")
SOURCES = ["muon_gemm_bf16.hip", "muon_gemm_f16.hip", "muon_gemm_f32.hip", "muon_gemm.hip",
           "muon_elementwise.hip", "muon_grasp.hip", "muon_adamw.hip", "muon_mx4.hip", "muon_mx4_gemm.hip",
           "muon_api.hip", "muon_schedule.cpp", "muon_ceiling.hip"]
ARCH = os.environ.get("MUON_OFFLOAD_ARCH", "gfx950")

HIPCC_FLAGS = [
    "-O3", "-std=c++17", "-fPIC", "-Wall",
    f"--offload-arch={ARCH}",
    # keep the compiler from forming packed fp32 instructions
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), shutil.which("hipcc"), "/opt/rocm/bin/hipcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: install ROCm or set HIPCC")


def _run(cmd: list[str], verbose: bool) -> subprocess.Popen:
    if verbose:
        print(" ".join(cmd), flush=True)
    # a process group of its own: a compiler driver's passes end with it
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, start_new_session=True)


def _finish(proc: subprocess.Popen, what: str, verbose: bool) -> None:
    out, _ = proc.communicate()
    noise = "is not a recognized feature for this target"
    msgs = "\n".join(l for l in out.splitlines() if noise not in l)
    if proc.returncode != 0:
        raise RuntimeError(f"{os.path.basename(proc.args[0])} failed on {what} ({proc.returncode}):\n{msgs}")
    if verbose and msgs.strip():
        print(msgs, file=sys.stderr)


# Host-side AddressSanitizer and UndefinedBehaviorSanitizer (the device code is
# built as usual): for checking the argument checks, workspace planning and
# schedule derivation on the CPU.  Load the result with the clang sanitizer
# runtime preloaded (see sanitizer_runtime()).
SANITIZE_COMPILE = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
                    "-Xarch_host", "-fno-sanitize-recover=undefined", "-Xarch_host", "-fno-omit-frame-pointer"]
SANITIZE_LINK = ["-fsanitize=address", "-fsanitize=undefined", "-fno-gpu-sanitize", "-shared-libsan"]


def sanitizer_runtime() -> str:
    """Path of clang's shared AddressSanitizer runtime that a sanitized build links against."""
    out = subprocess.run([hipcc(), "--print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True, text=True)
    return out.stdout.strip()


NATIVE_SOURCE = os.path.join(HERE, "native", "muon_native.cpp")
NATIVE = os.path.join(HERE, "_native.so")


def _native_command(out: str) -> list[str] | None:
    """Host compiler line of the extension module (torch's headers and ABI, no device code); None without torch or a
    host compiler, which the library itself does not need."""
    import sysconfig

    cxx = os.environ.get("CXX") or shutil.which("g++") or shutil.which("c++")
    try:
        import torch
        from torch.utils.cpp_extension import include_paths, library_paths
    except ImportError:
        return None
    if cxx is None:
        return None
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return [cxx, "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-fvisibility=hidden",
            f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-DTORCH_API_INCLUDE_EXTENSION_H",
            *[f"-isystem{p}" for p in include_paths()], f"-isystem{sysconfig.get_paths()['include']}",
            NATIVE_SOURCE, "-o", out, *[f"-L{p}" for p in library_paths()], "-lc10", "-ltorch_cpu", "-ltorch",
            "-ltorch_python"]


def build(verbose: bool = False, csrc: str = CSRC, lib: str = LIB, defines=(), sanitize: bool = False) -> str:
    """Always recompiles (one process per source, in parallel); once all of it
    has compiled, puts the library (default libmuon.so next to this file, and
    with it the extension module) in place atomically and returns its path.  ``csrc``, ``lib`` and ``defines`` (-D flags) build a variant;
    ``sanitize`` instruments the host code (see SANITIZE_COMPILE)."""
    objdir = tempfile.mkdtemp(prefix="muon_build_")
    san = SANITIZE_COMPILE if sanitize else []
    started, made = [], {}  # processes; finished outputs and where they go

    def start(cmd):
        started.append(_run(cmd, verbose))
        return started[-1]

    try:
        native = None
        if lib == LIB:  # a variant of the library uses the same extension module
            made[NATIVE] = NATIVE + ".tmp"
            command = _native_command(made[NATIVE])
            native = start(command) if command is not None else None
        objs = [os.path.join(objdir, os.path.splitext(src)[0] + ".o") for src in SOURCES]
        procs = [(src, start([hipcc(), *HIPCC_FLAGS, *san, *[f"-D{d}" for d in defines], "-c", "-o", obj,
                              os.path.join(csrc, src)])) for src, obj in zip(SOURCES, objs)]
        for src, proc in procs:
            _finish(proc, src, verbose)
        made[lib] = lib + ".tmp"
        _finish(start([hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *(SANITIZE_LINK if sanitize else []),
                       "-o", made[lib], *objs]), "link", verbose)
        if native is not None:
            _finish(native, os.path.basename(NATIVE_SOURCE), verbose)
        elif NATIVE in made:  # one of an earlier build must not stay beside this library
            del made[NATIVE]
            if os.path.exists(NATIVE):
                os.remove(NATIVE)
            print("the extension module is left out: it needs PyTorch and a C++ compiler", file=sys.stderr)
        for target, tmp in made.items():  # all of it has compiled
            os.replace(tmp, target)
    finally:
        for proc in started:  # after a failure the others may still run
            if proc.poll() is None:
                os.killpg(proc.pid, signal.SIGKILL)
                proc.communicate()
        for tmp in made.values():
            if os.path.exists(tmp):
                os.remove(tmp)
        shutil.rmtree(objdir, ignore_errors=True)
    return lib


if __name__ == "__main__":
    if "--sanitize" in sys.argv[1:]:
        print(build(verbose=True, lib=os.path.join(HERE, "libmuon_sanitized.so"), sanitize=True))
        print("runtime to preload:", sanitizer_runtime())
    else:
        print(build(verbose=True))
