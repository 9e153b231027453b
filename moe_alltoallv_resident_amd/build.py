"""Compile the gfx950 library in-tree with hipcc: liba2av.so (release) and
liba2av_debug.so (the same sources with -DA2AV_DEBUG=1: device-side bounds checks on
every row index and table value the kernels turn into an address, failures reported as
status bit A2AV_ST_BOUNDS).  All sources of both compile side by side.

Flags: -O3 for gfx950 only; packed-FP32 instruction selection switched off (the
kernels' float code is scalar FMA); no fast-math.
"""
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
ROOT = os.path.dirname(HERE)
LIB = os.path.join(HERE, "liba2av.so")
DEBUG_LIB = os.path.join(HERE, "liba2av_debug.so")
SOURCES = ["a2av_api.hip", "a2av_kernels.hip", "a2av_measure.hip", "a2av_norm.hip", "a2av_experts.hip",
           "a2av_experts_few.hip", "a2av_experts_tile.hip"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC", "-shared",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
         "-Wall", "-Wno-unused-command-line-argument",
         "-I", os.path.join(ROOT, "include")]


def build(verbose: bool = False) -> str:
    """Builds both libraries (every source of both at once); returns the release library's path."""
    compile_flags = [f for f in FLAGS if f != "-shared"]
    with tempfile.TemporaryDirectory() as tmp:
        jobs = []
        for out, extra in ((LIB, []), (DEBUG_LIB, ["-DA2AV_DEBUG=1"])):
            for s in SOURCES:
                obj = os.path.join(tmp, os.path.basename(out) + "." + s + ".o")
                cmd = [HIPCC] + compile_flags + extra + ["-c", "-o", obj, os.path.join(CSRC, s)]
                if verbose:
                    print(" ".join(cmd), flush=True)
                jobs.append((out, obj, cmd, subprocess.Popen(cmd)))
        failed = [cmd for _, _, cmd, p in jobs if p.wait() != 0]
        if failed:
            raise subprocess.CalledProcessError(1, failed[0])
        for lib in (LIB, DEBUG_LIB):
            objs = [obj for out, obj, _, _ in jobs if out == lib]
            cmd = [HIPCC, f"--offload-arch={ARCH}", "-fPIC", "-shared", "-o", lib + ".tmp"] + objs
            if verbose:
                print(" ".join(cmd), flush=True)
            subprocess.run(cmd, check=True)
    for lib in (LIB, DEBUG_LIB):
        os.replace(lib + ".tmp", lib)
    return LIB


def device_asm(out_dir: str) -> list:
    """Write the gfx950 assembly of every source into out_dir (for inspection)."""
    os.makedirs(out_dir, exist_ok=True)
    outs = []
    for s in SOURCES:
        o = os.path.join(out_dir, s.replace(".hip", f"-{ARCH}.s"))
        cmd = [HIPCC] + [f for f in FLAGS if f not in ("-shared", "-fPIC")] + \
              ["--offload-device-only", "-S", "-o", o, os.path.join(CSRC, s)]
        subprocess.run(cmd, check=True)
        outs.append(o)
    return outs


if __name__ == "__main__":
    print(build(verbose=True))
