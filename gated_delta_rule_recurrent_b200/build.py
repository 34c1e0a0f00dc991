"""Build libgdr.so in-tree with nvcc for sm_100a.

``python -m gated_delta_rule_recurrent_b200.build`` compiles
``csrc/gdr_api.cu`` and ``csrc/gdr_linear_api.cu`` (which include the kernel
headers) into objects and links them into
``gated_delta_rule_recurrent_b200/libgdr.so``. Sidecar files record a hash of
the sources and of the flags, so ``ensure_built()`` rebuilds exactly what
changed (file times are not trusted across copies).
"""
from __future__ import annotations

import concurrent.futures
import hashlib
import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
REPO_DIR = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(REPO_DIR, "include")
LIB_PATH = os.path.join(PKG_DIR, "libgdr.so")
HASH_PATH = LIB_PATH + ".srchash"
# A second build with -DGDR_TEST_HOOKS, for the failure-path tests only: the
# same kernels with a shortened budget for abandonable waits and a switch that
# holds one tile back. The shipped libgdr.so never contains the hooks.
TEST_HOOKS_LIB_PATH = os.path.join(PKG_DIR, "libgdr_testhooks.so")
TEST_HOOKS_FLAGS = ["-DGDR_TEST_HOOKS"]

_COMMON = [os.path.join(CSRC, name) for name in (
    "gdr_decode.cuh", "gdr_host.h", "gdr_ptx.cuh", "gdr_umma.cuh")] + [
    os.path.join(INCLUDE, "gdr.h")]
# Each source with the files it is compiled from, itself first.
UNITS = {os.path.join(CSRC, source): [os.path.join(CSRC, name) for name in (source, *headers)]
         + _COMMON for source, headers in (
    ("gdr_api.cu", ("gdr_decode_tma.cuh", "gdr_decode_chunk.cuh", "gdr_decode_chunk_tc.cuh",
                    "gdr_decode_rows.cuh", "gdr_gate.cuh", "gdr_prefill_tc.cuh")),
    ("gdr_linear_api.cu", ("gdr_linear.cuh", "gdr_linear_decode.cuh", "gdr_linear_plan.h",
                           "gdr_linear_prefill.cuh", "gdr_state_cache.cuh")))}
SOURCES = list(UNITS)
DEPS = list(dict.fromkeys(path for files in UNITS.values() for path in files))
OBJ_DIR = os.path.join(PKG_DIR, "_build")

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = [
    "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
    "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found; it is needed to build libgdr.so")


def compile_command(source, obj, extra=()) -> list:
    return [nvcc_path(), *ARCH_FLAGS, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC,
            "-c", "-o", obj, source]


def link_command(objs, out=LIB_PATH) -> list:
    return [nvcc_path(), *ARCH_FLAGS, "-shared", "-o", out, *objs]


def source_hash(flags=(), files=None) -> str:
    h = hashlib.sha256()
    for path in DEPS if files is None else files:
        with open(path, "rb") as f:
            h.update(os.path.basename(path).encode())
            h.update(f.read())
    h.update(" ".join(ARCH_FLAGS + NVCC_FLAGS + list(flags)).encode())
    return h.hexdigest()


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError(f"nvcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    if verbose and (res.stdout or res.stderr):
        print(res.stdout + res.stderr, flush=True)


def _forget(path) -> None:
    """Remove the sidecar file of something that is about to be written again: an
    interruption in between must not leave the old hash beside the new file."""
    if os.path.exists(path + ".srchash"):
        os.remove(path + ".srchash")


def build(verbose: bool = False, extra=(), test_hooks: bool = False, reuse: bool = False) -> str:
    """Compile every source, side by side, and link the library. With ``reuse``
    an object whose sources and flags are unchanged is not compiled again."""
    out = TEST_HOOKS_LIB_PATH if test_hooks else LIB_PATH
    flags = TEST_HOOKS_FLAGS if test_hooks else []
    os.makedirs(OBJ_DIR, exist_ok=True)

    def one(source):
        name = os.path.splitext(os.path.basename(source))[0]
        obj = os.path.join(OBJ_DIR, name + ("_testhooks" if test_hooks else "") + ".o")
        key = source_hash([*flags, *extra], UNITS[source])
        if reuse and os.path.exists(obj) and os.path.exists(obj + ".srchash"):
            with open(obj + ".srchash") as f:
                if f.read().strip() == key:
                    return obj
        _forget(obj)
        _run(compile_command(source, obj, [*flags, *extra]), verbose)
        with open(obj + ".srchash", "w") as f:
            f.write(key + "\n")
        return obj

    with concurrent.futures.ThreadPoolExecutor(len(UNITS)) as pool:
        objs = list(pool.map(one, UNITS))
    _forget(out)
    _run(link_command(objs, out), verbose)
    with open(out + ".srchash", "w") as f:
        f.write(source_hash(flags) + "\n")
    return out


def is_current(test_hooks: bool = False) -> bool:
    out = TEST_HOOKS_LIB_PATH if test_hooks else LIB_PATH
    if not (os.path.exists(out) and os.path.exists(out + ".srchash")):
        return False
    with open(out + ".srchash") as f:
        return f.read().strip() == source_hash(TEST_HOOKS_FLAGS if test_hooks else [])


def ensure_built(verbose: bool = False, test_hooks: bool = False) -> str:
    if not is_current(test_hooks):
        build(verbose=verbose, test_hooks=test_hooks, reuse=True)
    return TEST_HOOKS_LIB_PATH if test_hooks else LIB_PATH


if __name__ == "__main__":
    ptxas_info = "--ptxas-info" in sys.argv
    hooks = "--test-hooks" in sys.argv
    print(build(verbose=True, extra=("-Xptxas", "-v") if ptxas_info else (), test_hooks=hooks))
