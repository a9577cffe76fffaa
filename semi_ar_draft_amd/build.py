"""Build libdspark.so for gfx950 with hipcc, and the binding's compiled part
with the host compiler (in-tree, no JIT cache).

Usage: python -m semi_ar_draft_amd.build   (or call build()).
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(HERE, "libdspark.so")
NATIVE_PATH = os.path.join(HERE, "_native.so")
SOURCES = ["api.hip", "sweep.hip", "verify.hip", "confidence.hip", "schedule.hip", "gru.hip", "sts.hip",
           "stream.hip", "pages.hip", "cache.hip", "attend.hip", "constrain.hip"]
ARCH = os.environ.get("DSPARK_OFFLOAD_ARCH", "gfx950")

COMMON_FLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC",
    # no packed fp32 arithmetic in device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", INCLUDE, "-I", CSRC,
]

# The attention's running results stay in the registers that its vector code
# can reach; by default they are copied there and back around every step.
FILE_FLAGS = {"attend.hip": ["-mllvm", "-amdgpu-mfma-vgpr-form=1"]}


def _hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found")


def _run(cmd):
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    lines = [ln for ln in p.stdout.splitlines() if "packed-fp32-ops" not in ln]
    return p.returncode, "\n".join(lines)


def _native_cmds(obj: str, out: str):
    """The host compiler's commands for the binding's compiled part (no device code in it)."""
    import torch
    from torch.utils import cpp_extension
    gxx = shutil.which("g++") or "g++"
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    compile_ = [gxx, "-O2", "-std=c++17", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", INCLUDE,
                "-I", sysconfig.get_paths()["include"],
                "-isystem", os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include")]
    for inc in cpp_extension.include_paths():
        compile_ += ["-isystem", inc]
    link = [gxx, "-shared", obj, "-o", out, "-L", HERE, "-l:libdspark.so", "-Wl,-rpath,$ORIGIN",
            "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10"]
    return compile_ + ["-c", os.path.join(CSRC, "binding.cpp"), "-o", obj], link


def build(verbose: bool = False, extra_flags=()) -> str:
    """Compile every source for gfx950 and link libdspark.so; returns its path."""
    hipcc = _hipcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    jobs = []
    for src in SOURCES:
        obj = os.path.join(BUILD_DIR, src.replace(".hip", ".o"))
        cmd = [hipcc, *COMMON_FLAGS, *FILE_FLAGS.get(src, ()), *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        jobs.append((src, obj, cmd))
    native_obj = os.path.join(BUILD_DIR, "binding.o")
    native_compile, native_link = _native_cmds(native_obj, NATIVE_PATH + ".tmp")
    work = [("binding.cpp", native_obj, native_compile), *jobs]
    with concurrent.futures.ThreadPoolExecutor(max_workers=min(8, len(work))) as ex:
        results = list(ex.map(lambda j: (j[0], *_run(j[2])), work))
    for src, rc, out in results:
        if verbose and out.strip():
            print(out)
        if rc != 0:
            raise RuntimeError(f"the compiler failed on {src}:\n{out}")
    tmp = LIB_PATH + ".tmp"
    rc, out = _run([hipcc, f"--offload-arch={ARCH}", "-shared", "-fPIC",
                    *[j[1] for j in jobs], "-ldl", "-o", tmp])
    if rc != 0:
        raise RuntimeError(f"link failed:\n{out}")
    os.replace(tmp, LIB_PATH)
    rc, out = _run(native_link)
    if rc != 0:
        raise RuntimeError(f"link of the binding failed:\n{out}")
    os.replace(NATIVE_PATH + ".tmp", NATIVE_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
