"""Build libgdn_cpr.so and libgdn_policy.so in-tree with hipcc for gfx950 (cross-compiles without a GPU).

Flags that the contract depends on:
  -ffp-contract=off                  no fusion other than the explicit fmaf
  -fno-gpu-flush-denormals-to-zero   binary32 denormals kept on the GPU
  -Xclang -target-feature -Xclang -packed-fp32-ops
                                     no packed fp32 (v_pk_*) instructions in the kernels
No -ffast-math anywhere.
"""

from __future__ import annotations

import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgdn_cpr.so")

SOURCES = ["cpr_kernels.hip", "cpr_backward.hip", "cpr2.hip", "linear.hip", "api.cpp",
           "contract.cpp"]
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950",
    "-O3",
    "-std=c++17",
    "-fPIC",
    "-shared",
    "-fvisibility=hidden",
    "-ffp-contract=off",
    "-fno-fast-math",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall",
]


POLICY_LIB = os.path.join(PKG, "libgdn_policy.so")
POLICY_BINDING = os.path.join(PKG, "_policy_binding.so")
POLICY_SOURCES = ["norm.hip", "linear_i8.hip", "logprob.hip", "policy_loss.hip", "policy_api.cpp"]


def _build(sources, lib, verbose):
    """Compile the sources to objects side by side (one hipcc per source), then link them."""
    from concurrent.futures import ThreadPoolExecutor

    objdir = os.path.join(ROOT, "_build")
    os.makedirs(objdir, exist_ok=True)
    compile_flags = [f for f in FLAGS if f != "-shared"]

    def compile_one(src):
        obj = os.path.join(objdir, src + ".o")
        cmd = [HIPCC, *compile_flags, "-c", "-I", INCLUDE, "-I", CSRC, "-o", obj,
               os.path.join(CSRC, src)]
        if verbose:
            print(" ".join(cmd), flush=True)
        return obj, subprocess.run(cmd, capture_output=True, text=True)

    jobs = max(1, min(len(sources), os.cpu_count() or 1))
    with ThreadPoolExecutor(jobs) as pool:
        results = list(pool.map(compile_one, sources))
    for (obj, res), src in zip(results, sources):
        if res.returncode != 0:
            sys.stderr.write(res.stdout + res.stderr)
            raise RuntimeError(f"hipcc failed to compile {src}")
    tmp = lib + ".tmp"
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp,
           *[obj for obj, _ in results]]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed to link {os.path.basename(lib)}")
    os.replace(tmp, lib)
    return lib


def build(verbose: bool = False) -> str:
    """Build bitwise_consistent_linear_amd/libgdn_cpr.so; return its path."""
    return _build(SOURCES, LIB, verbose)


def build_policy(verbose: bool = False) -> str:
    """Build bitwise_consistent_linear_amd/libgdn_policy.so, the policy-head operators, with
    the same flags; return its path. A library of its own: libgdn_cpr.so holds exactly the
    contract's entry points and only its binary32 instructions."""
    lib = _build(POLICY_SOURCES, POLICY_LIB, verbose)
    build_policy_binding(verbose)
    return lib


PROBE_LIB = os.path.join(PKG, "libgdn_probe.so")


def build_probe(verbose: bool = False) -> str:
    """Compile the measurement probes (csrc/probe.hip) into libgdn_probe.so, which bench.py
    uses for the vector-issue ceiling and shader clock; the library proper does not link it."""
    tmp = PROBE_LIB + ".tmp"
    cmd = [HIPCC, *FLAGS, "-o", tmp, os.path.join(CSRC, "probe.hip")]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("hipcc failed to build libgdn_probe.so")
    os.replace(tmp, PROBE_LIB)
    return PROBE_LIB


KERNEL_SOURCES = [s for s in SOURCES if s.endswith(".hip")]


def build_policy_binding(verbose: bool = False) -> str:
    """Build _policy_binding.so, the policy head's Python calls, against the installed torch;
    return its path. Host code only. libgdn_policy.so is found beside it."""
    import sysconfig

    import torch

    base = os.path.dirname(torch.__file__)
    abi = int(torch.compiled_with_cxx11_abi())
    tmp = POLICY_BINDING + ".tmp"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           "-fvisibility=hidden", "-Wall", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", "-I", INCLUDE,
           "-isystem", os.path.join(base, "include"),
           "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           os.path.join(CSRC, "policy_binding.cpp"), "-o", tmp,
           "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_hip", "-ltorch_cpu",
           "-ltorch", "-lc10",
           "-L", PKG, "-l:" + os.path.basename(POLICY_LIB), "-Wl,-rpath,$ORIGIN"]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError("failed to build _policy_binding.so")
    os.replace(tmp, POLICY_BINDING)
    return POLICY_BINDING


def device_asm(out_path: str, sources=None) -> str:
    """Write the gfx950 assembly of the kernel sources (default: libgdn_cpr.so's),
    concatenated (for instruction-mix checks)."""
    parts = []
    for src in KERNEL_SOURCES if sources is None else sources:
        one = out_path + "." + src + ".s"
        cmd = [HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-ffp-contract=off",
               "-fno-fast-math", "-fno-gpu-flush-denormals-to-zero",
               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
               "--cuda-device-only", "-S", "-I", INCLUDE, "-I", CSRC, "-o", one,
               os.path.join(CSRC, src)]
        subprocess.run(cmd, check=True, capture_output=True)
        with open(one) as f:
            parts.append(f.read())
        os.remove(one)
    with open(out_path, "w") as f:
        f.write("\n".join(parts))
    return out_path


if __name__ == "__main__":
    print(build(verbose=True))
    print(build_probe(verbose=True))
    print(build_policy(verbose=True))
