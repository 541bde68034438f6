"""Which kernel an expert product runs, and calls that run each of them.

The choice is the library's own: csrc/experts_api.cpp is compiled for the host
with launchers that only note what they were asked for, on a device of 256
compute units.  What the kernels decide from the group boundaries (whole, half
and cut tiles) is counted here by the same rule, from sizes.
"""
import ctypes
import os
import shutil
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "communication_gemm_amd", "csrc")
CUS = 256

LAUNCHERS = r"""
#include "experts.hpp"
extern "C" {
int noted[4];   // kind of call, element type, variant, narrow strips
hipError_t hipGetDevice(int* dev) { *dev = 0; return hipSuccess; }
hipError_t hipDeviceGetAttribute(int* n, hipDeviceAttribute_t, int) { *n = 256; return hipSuccess; }
}
namespace agg {
hipError_t launch_grouped(const ProductArgs& a, int type, bool q_strided, int variant, hipStream_t)
{
    const int rows = variant == kSkinny16 ? 16 : 32;
    const int64_t more = a.groups < a.rows ? a.groups : a.rows;
    const int64_t tiles = a.offsets ? a.rows / rows + more : (a.rows + rows - 1) / rows;
    noted[0] = q_strided; noted[1] = type; noted[2] = variant;
    noted[3] = tiles * ((a.J + 31) / 32) < a.cus;
    return hipSuccess;
}
hipError_t launch_wgrad(const ProductArgs&, int type, int variant, hipStream_t)
{
    noted[0] = 2; noted[1] = type; noted[2] = variant; noted[3] = 0;
    return hipSuccess;
}
hipError_t launch_quant(const QuantArgs&, int type, int block_rows, bool wide, hipStream_t)
{
    noted[0] = 3; noted[1] = type; noted[2] = block_rows; noted[3] = wide;
    return hipSuccess;
}
}
"""

TYPES = {"f16": 0, "bf16": 2, "fp8": 3, "f32": 4}
VARIANTS = ["any layout", "large", "128 x 128", "64 x 256", "64 x 64", "16 rows", "32 rows"]
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
                        os.path.join(CSRC, "experts_api.cpp"), "-Wl,-Bsymbolic", "-o", lib], check=True)
        self.lib = ctypes.CDLL(lib)
        self.noted = (ctypes.c_int * 4).in_dll(self.lib, "noted")

    def _call(self, fn, *args):
        kinds = [ctypes.c_int64 if isinstance(x, int) else ctypes.c_void_p for x in args]
        rc = getattr(self.lib, fn)(*(k(x) for k, x in zip(kinds, args)))
        assert rc == 0, (fn, rc)
        return list(self.noted)

    def grouped(self, typ, out, counts, K, N, trans):
        T, E = sum(counts), len(counts)
        kind, _, variant, narrow = self._call(
            "ag_gemm_grouped", TYPES[typ], P, K, P, K if trans else N, K * N, int(trans), P, E, P, N,
            TYPES[out], T, K, N, None)
        assert kind == (not trans)
        name = f"{typ} {'[N, K]' if trans else '[K, N]'} {VARIANTS[variant]}"
        return name + (" narrow" if narrow else " wide") * (trans and variant == 6)

    def fp8(self, out, counts, K, N):
        T, E, kb, nb = sum(counts), len(counts), -(-K // 128), -(-N // 128)
        if E == 1:
            variant, narrow = self._call("ag_gemm_fp8_block", P, K, P, kb, P, K, P, kb, P, N,
                                         TYPES[out], T, K, N, None)[2:]
        else:
            variant, narrow = self._call(
                "ag_gemm_grouped_fp8_block", P, K, P, kb, P, K, N * K, P, kb, nb * kb, P, E, P, N,
                TYPES[out], T, K, N, None)[2:]
        if out == "f32" and variant == 1:
            variant = 2            # float32 outputs have no large kernel
        name = f"fp8 {'exact' if out == 'f32' else 'native'} {VARIANTS[variant]}"
        return name + (" narrow" if narrow else " wide") * (variant >= 5)

    def wgrad(self, typ, out, counts, K, N):
        T, E = sum(counts), len(counts)
        variant = self._call("ag_gemm_grouped_wgrad", TYPES[typ], P, K, P, N, P, E, P, N, K * N,
                             TYPES[out], T, K, N, None)[2]
        past = E * K * N * (4 if out == "f32" else 2) > 128 << 20
        return f"{typ} weight gradient {VARIANTS[variant]}" + " past the cache" * past


def large_positions(counts, N, cus=CUS):
    """(whole tiles, cut tiles, half tiles) of the large kernel."""
    nj = -(-N // 256)
    whole = sum(c // 256 + (c % 256 > 128) for c in counts) * nj
    half = sum(0 < c % 256 <= 128 for c in counts) * nj
    left = whole % cus
    uncut = max(20 if left else 0, 11 * -(-half // (cus - left)))
    cut = left if left <= cus // 2 and 11 * -(-(half + 2 * left) // cus) < uncut else 0
    return whole - cut, cut, half


# Calls of the grouped products: rows of each group, N, K's, and what they run
# (at K's last value; "large" also: whether tiles are cut, and the rounds).
GROUPED = {
    "large, a cut round": dict(counts=[700, 300, 129, 1, 100, 0, 128], N=4360, K=[64, 528],
                               kernel="large", cut=True, rounds=1),
    "large, a cut second round": dict(counts=[1500, 1025, 1100, 300, 129], N=4360, K=[16, 272],
                                      kernel="large", cut=True, rounds=2),
    "large, two rounds and halves": dict(counts=[3000, 3328, 70], N=4360, K=[128, 144],
                                         kernel="large", cut=False, rounds=2),
    "large, one group, cut": dict(counts=[600], N=8200, K=[272], kernel="large", cut=True, rounds=1),
    "large, one group, rounds": dict(counts=[4900], N=8200, K=[144], kernel="large", cut=False,
                                     rounds=3),
    "large, more than 64 groups": dict(counts=[60] * 30 + [0] + [61] * 35 + [0, 300, 257, 1, 128], N=776,
                                       K=[144, 528], kernel="large", cut=False, rounds=2),
    "128 x 128": dict(counts=[300, 257, 0, 511, 132], N=2056, K=[16, 272, 1168], kernel="128 x 128"),
    "64 x 256": dict(counts=[3, 0, 64, 65, 17] * 12, N=1032, K=[16, 144, 528], kernel="64 x 256"),
    "64 x 64": dict(counts=[100, 64, 65, 171], N=1608, K=[16, 272, 1168], kernel="64 x 64"),
    "64 x 64, one group": dict(counts=[200], N=328, K=[16, 2064], kernel="64 x 64"),
    "16 rows": dict(counts=[5, 3, 8, 1, 0, 7, 16, 2], N=2056, K=[16, 1168, 4112], kernel="16 rows"),
    "16 rows, few strips": dict(counts=[1, 16, 17, 0, 3], N=328, K=[16, 1168, 4112], kernel="16 rows"),
    "32 rows": dict(counts=[32, 33, 20, 18], N=328, K=[16, 272, 4112], kernel="32 rows"),
    "32 rows, one group of 33": dict(counts=[33], N=4104, K=[16, 272, 4112], kernel="32 rows"),
    "32 rows, one group of 64": dict(counts=[64], N=4104, K=[144, 2064], kernel="32 rows"),
    "any layout": dict(counts=[70, 0, 129, 5], N=130, K=[77, 129], kernel="any layout"),
}

# Weight gradients: rows of each group, K, N, and what they run.
WGRAD = {
    "large": dict(counts=[70, 0, 1, 129, 64, 65], K=1544, N=2056, kernel="large"),
    "128 x 128": dict(counts=[70, 0, 1, 129, 64, 65], K=136, N=264, kernel="128 x 128"),
    "past the cache": dict(counts=[70, 0, 1, 65, 64, 3, 9, 20, 0, 128, 5, 0, 33, 17, 2, 2, 64], K=2056,
                           N=2056, kernel="large past the cache"),
    "any layout": dict(counts=[70, 0, 129], K=77, N=130, kernel="any layout"),
}
