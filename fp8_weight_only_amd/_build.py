"""Build libfp8w.so and libfp8w_moe.so (the HIP kernels + C ABIs) in-tree for gfx950 with hipcc.

Every source under csrc/ is compiled to an object in parallel, then linked into
``fp8_weight_only_amd/libfp8w.so`` (the FP8 linear layer, include/fp8w.h); those
under csrc/moe/ go into ``fp8_weight_only_amd/libfp8w_moe.so`` (routing, products
grouped by expert, the int8 layer, include/fp8w_moe.h). Flags: -O3, IEEE fp32 division (no
fast-math), hidden visibility except the C ABI, packed-fp32 instructions
disabled (the compiler's own choice of v_pk_*_f32 is switched off), and kernel
arguments preloaded into SGPRs at wave launch (up to 16 SGPRs' worth). With
preloading a wave computes its first addresses without waiting for a load of
its arguments; the decode GEMV, whose one-wave workgroups each issue a single
round of loads, measured 0.1-0.2 us faster per launch on MI355X (4096 x 4096:
5.04 -> 4.82 us) and the skinny kernels the same. The compiler also emits a
header that loads the arguments itself, for firmware that does not preload.
"""
import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libfp8w.so")
MOE_LIB = os.path.join(HERE, "libfp8w_moe.so")
OBJDIR = os.path.join(ROOT, "_build", "fp8w")
ARCH = os.environ.get("FP8W_ARCH", "gfx950")

CFLAGS = [
    f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    "-Wall", "-Wextra", "-Wno-unused-parameter",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-mllvm", "-amdgpu-kernarg-preload-count=16",
    "-I", os.path.join(ROOT, "include"),
]


def _hipcc() -> str:
    p = shutil.which("hipcc") or "/opt/rocm/bin/hipcc"
    if not os.path.exists(p):
        raise RuntimeError("hipcc not found: the ROCm toolchain is required to build libfp8w.so")
    return p


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def moe_sources():
    return sorted(glob.glob(os.path.join(CSRC, "moe", "*.hip")))


def _compile(src: str, verbose: bool) -> str:
    obj = os.path.join(OBJDIR, os.path.relpath(src, CSRC).replace(os.sep, "_") + ".o")
    cmd = [_hipcc(), *CFLAGS, "-c", src, "-o", obj]
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    # the host pass does not know the packed-fp32 feature and says so; keep real diagnostics
    out = "\n".join(l for l in r.stdout.splitlines() if "packed-fp32-ops" not in l and l.strip())
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{out}")
    if out and verbose:
        print(out, flush=True)
    return obj


def _link(objs, lib: str, verbose: bool) -> None:
    tmp = lib + ".tmp"
    cmd = [_hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)


def build(verbose: bool = False) -> str:
    os.makedirs(OBJDIR, exist_ok=True)
    libs = [(LIB, sources()), (MOE_LIB, moe_sources())]
    srcs = [s for _, part in libs for s in part]
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs))) as ex:
        objs = dict(zip(srcs, ex.map(lambda s: _compile(s, verbose), srcs)))
    for lib, part in libs:
        _link([objs[s] for s in part], lib, verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
