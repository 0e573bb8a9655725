"""Build libgdncp.so (the C-ABI CUDA library) in-tree for sm_103a.

Each translation unit is compiled by nvcc in parallel into ``_build/`` and
linked into ``libgdncp.so`` next to this file.  Only sources or headers that
changed since the last build are recompiled.  Sources whose kernels must stay in
registers (NO_LOCAL) fail to build when one of them does not.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import re
import shutil
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libgdncp.so")
SOURCES = ["api.cu", "plan.cu", "conv.cu", "chunk_bf16.cu", "chunk_f32.cu", "chunk_tc.cu", "schedule.cu",
           "combine.cu", "noalloc.cu", "layout.cu", "backward.cu", "shard_bwd.cu", "mchain.cu",
           "ssm_conv.cu", "ssm_scan.cu", "ssm_scan_bwd.cu", "block_norm.cu",
           "rule_step.cu", "embed.cu", "vocab_loss.cu", "vocab_few.cu"]
# Kernels without local memory: two builds of vocab_loss.cu's product kernel that kept accumulators there ended
# with an illegal address, for a reason that was not found.
NO_LOCAL = {"vocab_loss.cu"}
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-rdc=true", "-Xcompiler", "-fPIC", "-I", INCLUDE,
              "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    hs = [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]
    hs += [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    return hs


def _stale(target, deps):
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def local_memory(ptxas_v: str) -> dict:
    """Bytes of stack and spills of every kernel that has any, from what -Xptxas -v prints."""
    found, name = {}, None
    for line in ptxas_v.splitlines():
        m = re.search(r"(?:Compiling entry function '|Function properties for )(\w+)", line)
        if m:
            name = m.group(1)
        m = re.search(r"(\d+) bytes stack frame, (\d+) bytes spill stores, (\d+) bytes spill loads", line)
        if m and any(map(int, m.groups())):
            found[name] = tuple(map(int, m.groups()))
    return found


def compile_command(src: str, obj: str, extra_flags=()) -> list:
    report = ["-Xptxas", "-v"] if os.path.basename(src) in NO_LOCAL else []
    return [nvcc(), *ARCH, *NVCC_FLAGS, *report, *extra_flags, "-c", src, "-o", obj]


def compile_unit(src: str, obj: str, extra_flags=()) -> str:
    """Compiles one source; what the compiler printed."""
    out = _run(compile_command(src, obj, extra_flags))
    if os.path.basename(src) in NO_LOCAL:
        if "bytes stack frame" not in out:
            os.remove(obj)
            raise RuntimeError(f"{src}: the compiler reports nothing of its kernels' local memory")
        bad = local_memory(out)
        if bad:
            os.remove(obj)  # or the next build would link it
            raise RuntimeError(f"{src}: kernels in local memory (stack, spill stores, spill loads): {bad}")
    return out


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("nvcc failed:\n" + " ".join(cmd) + "\n" + r.stdout + r.stderr)
    return r.stdout + r.stderr


def build_library(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    hdrs = _headers()
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, [s] + hdrs):
            jobs.append((s, obj, extra_flags))

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for out in ex.map(lambda job: compile_unit(*job), jobs):
            if verbose and out.strip():
                print(out)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".{os.getpid()}.tmp"
        _run([nvcc(), *ARCH, "-rdc=true", "-shared", "-o", tmp, *objs])
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    import sys
    print(build_library(force="--force" in sys.argv, verbose=True,
                        extra_flags=["-Xptxas", "-v"] if "--ptxas" in sys.argv else []))
