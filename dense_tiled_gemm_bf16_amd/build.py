"""Build libtgemm.so and libtgemm_ffn.so in-tree with hipcc for gfx950, and the
compiled part of the Python binding, _ffn_binding.so, with the host compiler.

    python -m dense_tiled_gemm_bf16_amd.build
"""
from __future__ import annotations

import os
import subprocess
import sys
import tempfile
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "libtgemm.so")
SOURCES = [os.path.join(CSRC, "tgemm_kernels.hip"), os.path.join(CSRC, "tgemm_quant.hip"),
           os.path.join(CSRC, "tgemm_clock.hip"), os.path.join(CSRC, "tgemm_scratch.hip"),
           os.path.join(CSRC, "tgemm_abi.cpp")]
FFN_LIB = os.path.join(PKG, "libtgemm_ffn.so")
FFN_SOURCES = [os.path.join(CSRC, "tgemm_ffn_gemm_bf16.hip"), os.path.join(CSRC, "tgemm_ffn_gemm_f16.hip"),
               os.path.join(CSRC, "tgemm_ffn_gemm.hip"), os.path.join(CSRC, "tgemm_ffn_rows.hip"),
               os.path.join(CSRC, "tgemm_ffn_rowops.hip"), os.path.join(CSRC, "tgemm_ffn_route.hip"),
               os.path.join(CSRC, "tgemm_ffn_norm.hip"), os.path.join(CSRC, "tgemm_ffn_quant.hip"),
               os.path.join(CSRC, "tgemm_ffn_mx_bf16.hip"), os.path.join(CSRC, "tgemm_ffn_mx_f16.hip"),
               os.path.join(CSRC, "tgemm_ffn_mx_bf16_64.hip"), os.path.join(CSRC, "tgemm_ffn_mx_f16_64.hip"),
               os.path.join(CSRC, "tgemm_ffn_mx_rows.hip"), os.path.join(CSRC, "tgemm_ffn_mx.hip"),
               os.path.join(CSRC, "tgemm_ffn_abi.cpp")]
BINDING = os.path.join(PKG, "_ffn_binding.so")
BINDING_SOURCE = os.path.join(CSRC, "tgemm_ffn_binding.cpp")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    "-Wall", "-Wno-unused-command-line-argument", "-fvisibility=hidden",
    # (Device helpers are unused in the host pass, which compiles no kernel bodies.)
    "-Wno-unneeded-internal-declaration",
    # No packed-fp32 VALU instructions (v_pk_*_f32) in device code.
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I", os.path.join(ROOT, "include"),
]


def _run(cmd, verbose):
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    # hipcc's host pass does not know the packed-fp32 feature and says so; drop that line.
    noise = "is not a recognized feature for this target"
    err = "\n".join(l for l in res.stderr.splitlines() if noise not in l)
    if res.returncode != 0:
        raise RuntimeError(f"{os.path.basename(cmd[0])} failed ({res.returncode}):\n{err}")
    if verbose and err.strip():
        print(err, file=sys.stderr)


def build_binding(verbose: bool = False) -> str:
    """Links against libtgemm_ffn.so (found beside it) and torch's libraries."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    torch_lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    includes = [sysconfig.get_paths()["include"], *cpp_extension.include_paths(), "/opt/rocm/include",
                os.path.join(ROOT, "include")]
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden", "-Wall",
           "-D__HIP_PLATFORM_AMD__", "-DUSE_ROCM", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    for path in includes:
        cmd += ["-isystem", path]
    cmd += [BINDING_SOURCE, "-o", BINDING + ".tmp", "-L" + PKG, "-l:libtgemm_ffn.so", "-L" + torch_lib, "-lc10",
            "-lc10_hip", "-ltorch_cpu", "-ltorch_hip", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    _run(cmd, verbose)
    os.replace(BINDING + ".tmp", BINDING)
    return BINDING


def build(verbose: bool = False) -> str:
    """Compiles every source (several at a time) and links the two libraries."""
    with tempfile.TemporaryDirectory(prefix="tgemm_build_") as tmp:
        def obj(src):
            return os.path.join(tmp, os.path.basename(src) + ".o")

        # The longest first: the tiled MXFP4 products, the dense products.
        order = sorted(SOURCES[:1] + FFN_SOURCES + SOURCES[1:], key=lambda src: "_mx_" not in src)
        with ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as pool:
            list(pool.map(lambda src: _run([HIPCC, *FLAGS, "-c", src, "-o", obj(src)], verbose), order))
        for lib, sources in ((LIB, SOURCES), (FFN_LIB, FFN_SOURCES)):
            _run([HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", lib + ".tmp", *map(obj, sources)], verbose)
            os.replace(lib + ".tmp", lib)
    build_binding(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose=True))
