"""Build libconvrot.so in-tree with nvcc for sm_100a (B200).

``python -m w8a8_rotated_int8_token_b200.build`` or ``build()`` compiles every
``csrc/*.cu`` into ``w8a8_rotated_int8_token_b200/libconvrot.so``. No GPU is
needed to build. The CUDA runtime is linked statically and its symbols are
kept private, so the library does not clash with the runtime PyTorch loads.
Beside it, g++ compiles ``csrc/binding.cpp`` against the installed PyTorch into
the extension ``_binding``, the Python binding's short way to the calls of a
decoding step. Both carry the hash of ``convrot.h``, whose structs they share.
The library needs no PyTorch to build; without one, or where g++ fails, it is
built alone, and the Python form of the binding serves.
"""

from __future__ import annotations

import glob
import hashlib
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
LIB_PATH = os.path.join(PKG_DIR, "libconvrot.so")
# with the tag of this Python's binary interface, so that no other one loads it
BINDING_PATH = os.path.join(PKG_DIR, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))
BINDING_SOURCE = os.path.join(PKG_DIR, "csrc", "binding.cpp")

NVCC_FLAGS = [
    "-gencode", "arch=compute_100a,code=sm_100a",
    "-O3", "-lineinfo", "-std=c++17",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
    "-shared",
    "-cudart", "static",
    "-Xlinker", "--exclude-libs=ALL",
    "-Xlinker", "-Bsymbolic",
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or install the CUDA toolkit)")


def _header_flag() -> str:
    with open(os.path.join(ROOT, "include", "convrot.h"), "rb") as f:
        return f'-DCONVROT_HEADER="{hashlib.sha256(f.read()).hexdigest()[:16]}"'


def sources() -> list[str]:
    return sorted(glob.glob(os.path.join(PKG_DIR, "csrc", "*.cu")))


def _deps() -> list[str]:
    return sources() + sorted(glob.glob(os.path.join(PKG_DIR, "csrc", "*.cuh"))) + [
        os.path.join(ROOT, "include", "convrot.h")]


def _newer(path: str, deps: list[str]) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in deps)


def up_to_date() -> bool:
    return _newer(LIB_PATH, _deps())


def _torch_works() -> bool:
    try:
        import torch  # noqa: F401
    except (ImportError, OSError):  # none, or one whose libraries do not load
        return False
    return True


def _binding_up_to_date() -> bool:
    import torch

    installed = os.path.join(os.path.dirname(torch.__file__), "version.py")  # another torch may have come since
    return _newer(BINDING_PATH, [BINDING_SOURCE, os.path.join(ROOT, "include", "convrot.h"), installed])


def _binding_command(out: str) -> list[str]:
    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(_nvcc()))
    include = [os.path.join(ROOT, "include"), os.path.join(base, "include"), os.path.join(cuda, "include"),
               sysconfig.get_paths()["include"]]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
            f'-DBUILT_FOR_TORCH="{torch.__version__}"', _header_flag(),
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", *(f"-I{d}" for d in include),
            BINDING_SOURCE, "-o", out, f"-L{os.path.join(base, 'lib')}", "-lc10", "-lc10_cuda", "-ltorch_cpu",
            "-ltorch_python"]


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile the library and the binding if a source is newer than them; return the library's path.
    Raises if the library cannot be built, warns if the binding cannot."""
    jobs = []
    if force or not up_to_date():
        tmp = LIB_PATH + ".tmp"
        jobs.append((LIB_PATH, [_nvcc(), *NVCC_FLAGS, _header_flag(), "-I", os.path.join(ROOT, "include"), "-o", tmp,
                                *sources()]))
    if _torch_works() and (force or not _binding_up_to_date()):
        jobs.append((BINDING_PATH, _binding_command(BINDING_PATH + ".tmp")))
    running = []
    for path, cmd in jobs:
        if verbose:
            print(" ".join(cmd), file=sys.stderr)
        try:
            p = subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.PIPE, text=True)
        except OSError as e:  # no such compiler
            p = subprocess.CompletedProcess(cmd, 127, "", str(e))
        running.append((path, cmd[0], p))
    ended = [(path, tool, *(p.communicate() if isinstance(p, subprocess.Popen) else (p.stdout, p.stderr)), p.returncode)
             for path, tool, p in running]
    for path, tool, out, err, code in ended:
        if code != 0:
            failed = f"{os.path.basename(tool)} failed ({code}):\n{out}\n{err}"
            if path == LIB_PATH:
                raise RuntimeError(failed)
            warnings.warn(f"calls go through the Python form of the binding; {failed}")
            if os.path.exists(path):
                os.remove(path)  # of older sources
            continue
        if verbose and (out or err):
            print(out + err, file=sys.stderr)
        os.replace(path + ".tmp", path)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
