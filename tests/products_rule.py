"""Which kernel a product of E4M3 or bf16 rows takes: the library's own rule (products_choice.h), compiled for
the host, so that a case made for a kernel can be held to it."""
import atexit
import collections
import ctypes as C
import functools
import os
import shutil
import subprocess
import tempfile

from quantized_expert_ffn_topk_amd import abi, build

SOURCE = """
#include <cstdio>
#include "products_choice.h"
using namespace moe;
namespace {
struct Named {
    char *to;
    template <int MODE, bool NT, int RT, int TC, int W>
    void stream()
    {
        std::sprintf(to, "stream %d %d %d %d %d", MODE, (int)NT, 8 * TC, 16 * RT, W);
    }
    template <int MODE, bool DMA, int NB, int WT, int WN, int FT, int FN>
    void tiles()
    {
        std::sprintf(to, "tiles %d %d %d %d %d", MODE, (int)DMA, 16 * WT * FT, 16 * WN * FN, NB);
    }
    template <int MODE, bool DMA>
    void groups()
    {
        std::sprintf(to, "groups %d %d 256 256 0", MODE, (int)DMA);
    }
};
}
extern "C" int copies(uint64_t x, uint64_t w, int64_t ldx, int64_t ldw, int64_t w_stride, int64_t gathered)
{
    return copies_rows((const void *)x, (const void *)w, ldx, ldw, w_stride, gathered);
}
extern "C" void choose(int grouped, int f8, int f32, int64_t M, int64_t N, int64_t K, int64_t E, int copied, char *to)
{
    const ProductSizes a{M, N, f8 ? K : 2 * K, E, copied != 0};
    Named n{to};
    if (!grouped && f32)
        choose_dense<F8X, F8X>(a, n);
    else if (!grouped)
        choose_dense<F8X, F8>(a, n);
    else if (f8 && f32)
        choose_grouped<F8X, F8X>(a, n);
    else if (f8)
        choose_grouped<F8X, F8>(a, n);
    else
        choose_grouped<BF16, BF16>(a, n);
}
"""
UNITS = ("f8", "f8x", "bf16")
# flag: non-temporal loads of a stream, or rows copied by the load unit; last: a stream's waves, a tile's buffers
Kernel = collections.namedtuple("Kernel", "way unit flag rows channels last")


@functools.lru_cache(maxsize=None)
def _lib():
    d = tempfile.mkdtemp(prefix="products_rule")
    atexit.register(shutil.rmtree, d, ignore_errors=True)
    source, lib = os.path.join(d, "rule.cpp"), os.path.join(d, "rule.so")
    with open(source, "w") as f:
        f.write(SOURCE)
    subprocess.run(build.CXX.split() + ["-std=c++17", "-O1", "-fPIC", "-shared", "-Wall", "-ffp-contract=off",
                                        "-I" + os.path.join(abi.PKG, "csrc"), source, "-o", lib], check=True)
    L = C.CDLL(lib)
    L.copies.argtypes, L.copies.restype = [C.c_uint64] * 2 + [C.c_int64] * 4, C.c_int
    L.choose.argtypes, L.choose.restype = [C.c_int] * 3 + [C.c_int64] * 4 + [C.c_int, C.c_char_p], None
    return L


def copies(ldx, ldw, shift=0, w_stride=0, gathered=0):
    """Rows of bytes ldx and ldw apart, `shift` bytes past an address of 128 bytes' alignment."""
    return bool(_lib().copies(4096 + shift, 4096 + shift, ldx, ldw, w_stride, gathered))


def _kernel(*args):
    to = C.create_string_buffer(64)
    _lib().choose(*args, to)
    way, unit, flag, *rest = to.value.decode().split()
    return Kernel(way, UNITS[int(unit)], bool(int(flag)), *map(int, rest))


def dense(out, T, N, K, copied=True):
    return _kernel(0, 1, out == "f32", T, N, K, 1, copied)


def grouped(xd, out, M, N, K, E, copied=True):
    return _kernel(1, xd == "fp8", out == "f32", M, N, K, E, copied)
