"""Which tiles and k-splits the shared expert's bf16 products take: the library's own rule (``csrc/shared_tiles.h``, host code),
compiled here, on the products' sizes."""
import ctypes
import functools
import os
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "expert_output_overlap_amd", "csrc")
SOURCE = """
#include "shared_tiles.h"
extern "C" void one(int64_t M, int64_t cols, int nkt, int* got) {
  const Choice c = choose(M, cols, nkt);
  got[0] = c.tile;
  got[1] = c.splits;
}
extern "C" void three(const int64_t* size, int* got) {
  Product p[3];
  for (int i = 0; i < 3; ++i) p[i] = {size[3 * i], size[3 * i + 1], (int)size[3 * i + 2]};
  int splits[3];
  got[0] = choose_grads(p, splits).tile;
  for (int i = 0; i < 3; ++i) got[1 + i] = splits[i];
}
"""


@functools.lru_cache(None)
def _lib():
    with tempfile.TemporaryDirectory() as at:
        src, lib = os.path.join(at, "tiles.cpp"), os.path.join(at, "tiles.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-O2", "-fPIC", "-shared", "-I", CSRC, src, "-o", lib], check=True)
        return ctypes.CDLL(lib)


def _up(n, k):
    return -(-n // k) * k


def tiles(T, d, f):
    """{product: (tile, k-splits)} of a forward (unless few tokens stream the weights) and backward call."""
    D, F, nkt = _up(d, 8), _up(f, 8), lambda k: -(-k // 64)
    got, c = {}, (ctypes.c_int * 4)()
    one = {"gate and up": (T, 2 * F, nkt(D)), "down": (T, _up(d, 4), nkt(F)), "dh": (T, F, nkt(D))}
    few = T <= 32 or T <= 64 and d % 8 == 0 and f % 8 == 0 and 2 * d * f <= 1 << 25
    for name, (M, cols, k) in one.items():
        if name == "dh" or not few:
            _lib().one(ctypes.c_int64(M), ctypes.c_int64(cols), k, c)
            got[name] = c[0], c[1]
    sizes = (ctypes.c_int64 * 9)(T, _up(d, 4), nkt(2 * F), 2 * F, _up(d, 4), nkt(T), d, _up(f, 4), nkt(T))
    _lib().three(sizes, c)
    got["gradients"] = c[0], max(c[1:4])
    return got
