"""Which kernel a 4-bit product runs, and calls that run each of them.

The choice is the library's own: csrc/layers_api.cpp is compiled for the host
with launchers that only note what they were asked for, on a device of 256
compute units.
"""
import ctypes
import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "communication_gemm_amd", "csrc")

LAUNCHERS = r"""
#include "layers.hpp"
extern "C" {
int noted;
hipError_t hipGetDevice(int* dev) { *dev = 0; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* n, hipDeviceAttribute_t, int) { *n = 256; return hipSuccess; }
}
namespace agg {
hipError_t launch_sort(const SortArgs&, bool wide, hipStream_t) { noted = wide; return hipSuccess; }
hipError_t launch_dispatch(const DispatchArgs&, int unit, hipStream_t) { noted = unit; return hipSuccess; }
hipError_t launch_combine(const CombineArgs&, int, int, bool wide, hipStream_t) { noted = wide; return hipSuccess; }
hipError_t launch_combine_grad(const CombineArgs&, int, bool wide, hipStream_t) { noted = wide; return hipSuccess; }
hipError_t launch_norm(const NormArgs&, int, bool wide, hipStream_t) { noted = wide; return hipSuccess; }
hipError_t launch_norm_grad(const NormGradArgs&, int, bool wide, hipStream_t) { noted = wide; return hipSuccess; }
hipError_t launch_mx_quant(const MxQuantArgs&, int, bool wide, hipStream_t) { noted = wide; return hipSuccess; }
hipError_t launch_mx_dequant(const MxQuantArgs&, int, bool wide, hipStream_t) { noted = wide; return hipSuccess; }
hipError_t launch_mx(const MxArgs&, int variant, bool shift, hipStream_t)
{
    noted = variant + 16 * shift;
    return hipSuccess;
}
}
"""

VARIANTS = ["any layout", "large", "128 x 128", "64 x 256", "64 x 64", "16 rows", "32 rows",
            "split 32 x 32", "split 32 x 64", "split 64 x 64", "split 64 x 128"]
TYPES = {"f16": 0, "bf16": 2, "f32": 4}
P = 1 << 20     # stands for every matrix; never read


class Chooser:
    def __init__(self, folder):
        src, lib = os.path.join(folder, "launchers.cpp"), os.path.join(folder, "libchoice.so")
        with open(src, "w") as f:
            f.write(LAUNCHERS)
        rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
        subprocess.run([shutil.which("g++"), "-std=c++17", "-O1", "-fPIC", "-shared",
                        "-D__HIP_PLATFORM_AMD__", "-Wno-attributes", f"-I{rocm}/include",
                        f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", src,
                        os.path.join(CSRC, "layers_api.cpp"), "-Wl,-Bsymbolic", "-o", lib], check=True)
        self.lib = ctypes.CDLL(lib)
        self.noted = ctypes.c_int.in_dll(self.lib, "noted")

    def call(self, fn, *args):
        """What the call's launcher was asked for."""
        def as_c(x):
            return ctypes.c_float(x) if isinstance(x, float) else ctypes.c_int64(x) if isinstance(x, int) \
                else ctypes.c_void_p(x)
        self.noted.value = -1
        rc = getattr(self.lib, fn)(*(as_c(x) for x in args))
        assert rc == 0, (fn, rc)
        return self.noted.value

    def product(self, counts, K, N, out="bf16", lda=None, lds=None, ldc=None):
        T, E, kb = sum(counts), len(counts), -(-K // 32)
        lda, lds, ldc = lda or K // 2, lds or -(-kb // 4) * 4, ldc or N
        if E == 1:
            v = self.call("ag_gemm_mxfp4", P, lda, P, lds, P, K // 2, P, lds, P, ldc, TYPES[out], T, K, N, None)
        else:
            v = self.call("ag_gemm_grouped_mxfp4", P, lda, P, lds, P, K // 2, N * K // 2, P, lds, N * lds, P, E,
                          P, ldc, TYPES[out], T, K, N, None)
        return VARIANTS[v % 16] + (", shifted" if v >= 16 else "")


# Calls: rows of each group, K's, N, and what they run.  Every number of slices
# of 256 modulo four, ends inside tiles, blocks and slices, groups without rows.
PRODUCTS = {
    "16 rows": dict(counts=[5], K=[32, 7168], N=264, kernel="16 rows"),
    "16 rows, whole": dict(counts=[16], K=[4096], N=1032, kernel="16 rows"),
    "16 rows, groups": dict(counts=[5, 3, 8, 1, 0, 7, 16, 2], K=[160, 1184], N=520, kernel="16 rows"),
    "16 rows, several": dict(counts=[200], K=[544, 1184], N=296, kernel="16 rows"),
    "32 rows": dict(counts=[32], K=[64, 2080], N=4088, kernel="32 rows"),
    "32 rows, several": dict(counts=[40], K=[1184], N=2040, kernel="32 rows"),
    "32 rows, groups": dict(counts=[17, 0, 32, 33], K=[544, 1312], N=520, kernel="32 rows"),
    "split 32 x 32": dict(counts=[64], K=[1056, 2336, 7168], N=4088, kernel="split 32 x 32"),
    "split 32 x 32, groups": dict(counts=[1, 40, 33, 0, 70], K=[1056, 1312], N=520, kernel="split 32 x 32"),
    "split 32 x 64": dict(counts=[200], K=[1184, 2080, 3104], N=2056, kernel="split 32 x 64"),
    "split 32 x 64, groups": dict(counts=[5, 40, 1, 33, 0, 64, 32, 25], K=[1056], N=968, kernel="split 32 x 64"),
    "split 64 x 64": dict(counts=[300], K=[1056, 2080, 4128], N=2568, kernel="split 64 x 64"),
    "split 64 x 64, groups": dict(counts=[300, 257, 0, 511, 132], K=[1312], N=456, kernel="split 64 x 64"),
    "split 64 x 128": dict(counts=[500], K=[4096, 4128], N=4088, kernel="split 64 x 128"),
    "split 64 x 128, groups": dict(counts=[300, 257, 0, 511, 132], K=[4352], N=776, kernel="split 64 x 128"),
    "64 x 64": dict(counts=[300, 257, 0, 511, 132], K=[32, 416, 1056, 1312], N=776, kernel="64 x 64"),
    "64 x 64, one group": dict(counts=[200], K=[288, 800], N=2056, kernel="64 x 64"),
    "64 x 256": dict(counts=[3, 0, 64, 65, 17] * 12, K=[32, 288, 544, 1056], N=776, kernel="64 x 256"),
    "128 x 128": dict(counts=[700, 300, 129, 1, 100, 0, 128], K=[96, 544, 1056, 1312], N=2312,
                      kernel="128 x 128"),
    "128 x 128, one group": dict(counts=[1024], K=[2048], N=4096, kernel="128 x 128"),
    "large, a cut round": dict(counts=[700, 300, 129, 1, 100, 0, 128], K=[32, 288, 800], N=4360, kernel="large"),
    "large, a cut second round": dict(counts=[1500, 1025, 1100, 300, 129], K=[544, 1056], N=4360, kernel="large"),
    "large, two rounds and halves": dict(counts=[3000, 3328, 70], K=[256], N=4360, kernel="large"),
    "large, one group, cut": dict(counts=[600], K=[1312], N=8200, kernel="large"),
    "large, one group, rounds": dict(counts=[4900], K=[288], N=8200, kernel="large"),
}
