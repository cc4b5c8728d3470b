"""Build libfp8gemm.so (gfx950) in-tree with hipcc.

    python -m fp8_block_scaled_x128_amd.build        # or: python fp8_block_scaled_x128_amd/build.py

Besides compiling, it checks the generated gfx950 assembly for two properties the kernels rely
on: M0 is written only by the direct-to-LDS load sequences (which set it themselves), and no
nested loop (the K loop, the split-K sums) spills to scratch memory.
"""
from __future__ import annotations

import concurrent.futures
import os
import re
import shutil
import subprocess
import sys
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(HERE, "libfp8gemm.so")
# the benchmark's streaming-read kernel (read floor), a library of its own
PROBE_LIB = os.path.join(HERE, "libreadprobe.so")
PROBE_SOURCE = os.path.join(HERE, "csrc", "read_probe.hip")
SOURCES = [os.path.join(CSRC, "fp8gemm_kernels.hip"), os.path.join(CSRC, "stream_kernels.hip"),
           os.path.join(CSRC, "quantize_kernels.hip"), os.path.join(CSRC, "scratch.hip"),
           os.path.join(CSRC, "route_kernels.hip"), os.path.join(CSRC, "permute_kernels.hip"),
           os.path.join(CSRC, "w4_kernels.hip"), os.path.join(CSRC, "gated_kernels.hip"),
           os.path.join(CSRC, "lora_kernels.hip"),
           os.path.join(CSRC, "fp8gemm_api.cpp"), os.path.join(CSRC, "moe_api.cpp"),
           os.path.join(CSRC, "ffn_api.cpp"),
           os.path.join(CSRC, "fp8gemm_jit.cpp")]
# the Python module of the short path from torch tensors to the library (host code)
NATIVE_LIB = os.path.join(HERE, "_native.so")
NATIVE_SOURCE = os.path.join(CSRC, "binding.cpp")
# headers of the tiled kernel, compiled into the library as text for the run-time build
JIT_HEADERS = ["fp8gemm_args.h", "fp8gemm_device.h", "fp8gemm_tiled.h"]
JIT_DELIM = "FP8GEMM_SRC"
DEVICE_SOURCES = [p for p in SOURCES if p.endswith(".hip")]
ARCH = "gfx950"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
# Packed fp32 VALU ops are kept out of the device code on purpose.
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                # MFMA results in VGPRs, so the promotion FMAs read them without AGPR copies
                "-mllvm", "-amdgpu-mfma-vgpr-form"]
COMMON = ["-O3", "-std=c++17", "-fPIC", "-I", INCLUDE, "-I", CSRC, "-Wall", "-Wno-unused-result"]


def _run(cmd):
    r = subprocess.run(cmd, capture_output=True, text=True)
    noise = ("is not a recognized feature for this target", "packed-fp32-ops")
    err = "\n".join(l for l in r.stderr.splitlines() if not any(n in l for n in noise))
    if r.returncode != 0:
        raise RuntimeError("command failed: %s\n%s" % (" ".join(cmd), err))
    return err


def check_isa(asm_text: str) -> None:
    """M0 may only be set by the LDS-DMA sequences, and no nested loop may touch scratch."""
    lines = asm_text.splitlines()
    for i, line in enumerate(lines):
        code = line.split(";", 1)[0]
        if re.search(r"\bm0\b", code):
            ok = (re.match(r"\s*s_mov_b32 m0, (s\d+|vcc_lo|vcc_hi)\s*$", code) and i + 2 < len(lines)
                  and "s_nop" in lines[i + 1] and "global_load_lds_dword" in lines[i + 2])
            if not ok:
                raise RuntimeError("unexpected use of M0 in generated code: line %d: %s" % (i + 1, line.strip()))
    # Spills are tolerated only outside nested loops: a value kept across the per-tile loop may be
    # reloaded once per tile, but nothing in the K loop (loop depth >= 2) may touch scratch.
    depth = 0
    for i, line in enumerate(lines):
        if re.match(r"^(\.LBB\w+:|; %bb\.\d+:)", line):
            m = re.search(r"Depth=(\d+)", line)
            depth = int(m.group(1)) if m else 0
        elif re.match(r"^\S+:", line):
            depth = 0
        code = line.split(";", 1)[0]
        if depth >= 2 and re.search(r"\bscratch_(load|store)", code):
            raise RuntimeError("scratch access inside a nested loop: line %d: %s" % (i + 1, line.strip()))


def jit_sources_inc() -> str:
    """C++ text of fp8gemm_jit_sources.inc: the tiled kernel's headers as raw string literals."""
    names, texts = [], []
    for h in JIT_HEADERS:
        text = open(os.path.join(CSRC, h)).read()
        if ")" + JIT_DELIM + '"' in text:
            raise RuntimeError("%s contains the raw-string delimiter" % h)
        names.append('"%s"' % h)
        texts.append('R"%s(%s)%s"' % (JIT_DELIM, text, JIT_DELIM))
    return ("// generated by build.py from %s\n" % ", ".join(JIT_HEADERS) +
            "static const int kJitSourceCount = %d;\n" % len(JIT_HEADERS) +
            "static const char* const kJitSourceNames[] = {%s};\n" % ", ".join(names) +
            "static const char* const kJitSources[] = {\n%s};\n" % ",\n".join(texts))


def build_native(tmp: str) -> None:
    """_native.so: needs libfp8gemm.so beside it (found by $ORIGIN) and torch loaded before it."""
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    include = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.environ.get("ROCM_PATH", "/opt/rocm"), "include"), sysconfig.get_paths()["include"]]
    _run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
          "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, "-I", INCLUDE] +
         [x for d in include for x in ("-isystem", d)] +
         [NATIVE_SOURCE, "-o", tmp, "-L" + HERE, "-l:" + os.path.basename(LIB), "-L" + os.path.join(root, "lib"), "-lc10", "-lc10_hip",
          "-ltorch_cpu", "-ltorch_python", "-Wl,-rpath,$ORIGIN"])
    os.replace(tmp, NATIVE_LIB)


def build(verbose: bool = False) -> str:
    tmp = LIB + ".tmp%d" % os.getpid()
    gen = tempfile.mkdtemp(prefix="fp8gemm_gen")
    try:
        with open(os.path.join(gen, "fp8gemm_jit_sources.inc"), "w") as f:
            f.write(jit_sources_inc())
        hipcc = [HIPCC, "--offload-arch=" + ARCH] + COMMON + DEVICE_FLAGS
        with tempfile.TemporaryDirectory() as td, concurrent.futures.ThreadPoolExecutor(min(8, os.cpu_count() or 1)) as pool:
            def out(src, ext):
                return os.path.join(td, os.path.basename(src) + ext)
            jobs = [pool.submit(_run, hipcc + ["-I", gen, "-c", "-o", out(src, ".o"), src]) for src in SOURCES]
            jobs += [pool.submit(_run, hipcc + ["--cuda-device-only", "-S", "-o", out(src, ".s"), src]) for src in DEVICE_SOURCES]
            for job in jobs:
                job.result()
            for src in DEVICE_SOURCES:
                with open(out(src, ".s")) as f:
                    check_isa(f.read())
            _run(hipcc + ["-shared", "-o", tmp] + [out(src, ".o") for src in SOURCES] + ["-ldl"])
        os.replace(tmp, LIB)
        _run([HIPCC, "--offload-arch=" + ARCH] + COMMON + DEVICE_FLAGS + ["-shared", "-o", tmp, PROBE_SOURCE])
        os.replace(tmp, PROBE_LIB)
        build_native(tmp)
    finally:
        if os.path.exists(tmp):
            os.remove(tmp)
        shutil.rmtree(gen, ignore_errors=True)
    if verbose:
        print("built", LIB, NATIVE_LIB, "and", PROBE_LIB)
    return LIB


if __name__ == "__main__":
    build(verbose=True)
    sys.exit(0)
