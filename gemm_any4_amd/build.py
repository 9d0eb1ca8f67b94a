"""Compile libany4.so (HIP, gfx950 only) in-tree with hipcc."""
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
SRCS = [os.path.join(HERE, "csrc", f) for f in ("any4.hip", "lora.hip", "gemm_dx.hip", "ffn.hip",
                                               "route.hip")]
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libany4.so")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    # no packed-fp32 instructions anywhere in the device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp"
    with tempfile.TemporaryDirectory() as work:
        objs = [os.path.join(work, os.path.basename(s) + ".o") for s in SRCS]
        running = []
        for src, obj in zip(SRCS, objs):
            cmd = [HIPCC, *FLAGS, "-I", INCLUDE, "-c", "-o", obj, src]
            if verbose:
                print(" ".join(cmd), flush=True)
            running.append(subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT,
                                            text=True))
        out = [p.communicate()[0] for p in running]
        for p, o in zip(running, out):
            if p.returncode != 0:
                raise RuntimeError(f"hipcc failed ({p.returncode}):\n{o}")
        # hipBLASLt: the plain bf16 GEMM of the prefill path
        cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp, *objs, "-lhipblaslt"]
        if verbose:
            print(" ".join(cmd), flush=True)
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError(f"hipcc failed ({res.returncode}):\n{res.stdout}\n{res.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
