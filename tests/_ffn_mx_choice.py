"""Which kernel an MXFP4 product takes, asked of the library's own rule
(tgemm_ffn_mx.hip, host code) built here with the launches left out; and sizes
for each kernel."""
import ctypes
import os
import subprocess
import tempfile

import _ffn_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "dense_tiled_gemm_bf16_amd", "csrc")

SOURCE = r"""
#include "tgemm_ffn_internal.hpp"
namespace tgemm {
namespace ffn {
static int taken;  // the tile's rows; 65: 64 x 64 tiles two to a CU; 1: K is split
hipError_t launch_mx_rows(const MxGemm &) { return taken = 16, hipSuccess; }
hipError_t launch_mx_split(const MxGemm &) { return taken = 1, hipSuccess; }
hipError_t launch_join(const Gemm &) { return hipSuccess; }
template <>
hipError_t launch_mx_64<0>(const MxGemm &, bool two) { return taken = two ? 65 : 64, hipSuccess; }
template <>
hipError_t launch_mx_64<1>(const MxGemm &, bool two) { return taken = two ? 65 : 64, hipSuccess; }
template <>
hipError_t launch_mx_large<0>(const MxGemm &, int tm) { return taken = tm, hipSuccess; }
template <>
hipError_t launch_mx_large<1>(const MxGemm &, int tm) { return taken = tm, hipSuccess; }
}  // namespace ffn
}  // namespace tgemm
#include "tgemm_ffn_mx.hip"
extern "C" int choice(int64_t M, int64_t N, int64_t K, int64_t groups, int act, int bias, int residual, int preact,
                      int dtype) {
  using namespace tgemm::ffn;
  static char p[16] __attribute__((aligned(16)));
  MxGemm g{};
  g.dtype = dtype;
  g.M = M, g.N = N, g.K = K, g.groups = groups, g.act = act;
  g.A = g.B = g.SA = g.SB = g.C = p;
  g.stride_sb = N * (K / 32);
  if (bias) g.bias = p;
  if (residual) g.residual = p;
  if (preact) g.preact = p;
  g.cus = 256;
  g.splits = groups ? 1 : mx_splits(M, N, K);
  taken = 0;
  launch_mx(g);
  return taken;
}
"""

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4, "swiglu": 5, "geglu": 6}
_rule = None


def choice(M, N, K, groups=0, act="none", bias=False, residual=False, preact=False, f16=False):
    """16, 64, 65 (64 x 64, two to a compute unit), 128, 256, or 1 where K is split."""
    global _rule
    if _rule is None:
        with tempfile.TemporaryDirectory() as d:
            src, so = os.path.join(d, "choice.cpp"), os.path.join(d, "choice.so")
            with open(src, "w") as f:
                f.write(SOURCE)
            subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                            "-I" + CSRC, src, "-o", so], check=True)
            lib = ctypes.CDLL(so)
        lib.choice.argtypes = [ctypes.c_int64] * 4 + [ctypes.c_int] * 5
        _rule = lib.choice
    return _rule(M, N, K, groups, ACTS[act], bias, residual, preact, f16)


#: (kernel, M, N, K, act, bias, residual, preact) of dense products, K in every kernel's own steps and outside them.
DENSE = [
    (16, 1, 4096, 4096, "silu", True, True, False), (16, 16, 4104, 1056, "gelu", True, False, True),
    (16, 7, 8272, 160, "swiglu", False, False, False),
    (64, 64, 4096, 1088, "gelu", True, True, True), (64, 48, 8192, 4096, "swiglu", False, False, False),
    (65, 600, 3000, 320, "none", True, True, True), (65, 1030, 2056, 288, "relu", True, False, False),
    (65, 1, 32768, 4096, "none", False, False, False),
    (128, 1500, 4112, 544, "gelu", True, True, False), (128, 4100, 4104, 288, "none", False, False, False),
    (128, 4095, 8176, 1024, "geglu", True, False, True),
    (256, 4095, 4088, 4096, "gelu", True, True, True), (256, 4095, 4088, 1024, "none", False, False, False),
    (256, 4001, 4096, 2048, "none", True, False, False), (256, 4095, 8176, 4096, "swiglu", False, False, False),
    (1, 48, 520, 16384, "silu", True, True, True),
]
#: (kernel, rows, groups, N, K, act, bias, preact) of products by group.
GROUPED = [
    (16, 20, 4, 264, 512, "gelu", True, True), (16, 150, 64, 2048, 1024, "swiglu", False, False),
    (64, 60, 8, 1024, 4096, "none", False, False),
    (65, 2000, 8, 512, 544, "relu", True, True), (65, 150, 64, 2048, 2048, "swiglu", False, False),
    (128, 3000, 16, 2048, 1536, "none", True, False), (128, 8192, 4, 4096, 2048, "swiglu", False, False),
    (256, 6000, 4, 2048, 2048, "none", False, False), (256, 7000, 3, 8192, 4096, "none", True, False),
    (256, 7000, 3, 8192, 4096, "silu", False, True),
]
