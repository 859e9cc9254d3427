"""The library's choice of a kernel for a 4-bit product, asked on the host: its header compiled by itself."""
import ctypes
import functools
import os
import shutil
import subprocess
import tempfile

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_moe_routing_amd", "csrc")
CUS = 256  # of an MI355X

SOURCE = """
#include "w4_choice.h"
extern "C" void choose(const int *v, int cus, int *out) {
    const moe::W4Sizes s{v[0], v[1], v[2], v[3], v[4], v[5] != 0, v[6] != 0, v[7] != 0, v[8] != 0, v[9] != 0, v[10] != 0};
    const moe::W4Choice c = moe::w4_choose(s, cus);
    out[0] = c.r, out[1] = c.split, out[2] = c.tile_rows;
}
"""


@functools.lru_cache(None)
def _library():
    cc = shutil.which("g++")
    if cc is None:
        import pytest
        pytest.skip("no host compiler")
    out = tempfile.mkdtemp(prefix="w4_choice")
    src, lib = os.path.join(out, "choice.cpp"), os.path.join(out, "choice.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run([cc, "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", "-I" + CSRC, src, "-o", lib], check=True)
    loaded = ctypes.CDLL(lib)
    shutil.rmtree(out)
    return loaded


def choose(n, E, M, K, G, grouped=True, x="bf16", scale="bf16", zero=False, y="bf16", swiglu=False):
    """("stream", rows of a wave, K is split) or ("block", rows of a block)."""
    v = (ctypes.c_int * 11)(n, E, M, K, G, grouped, x == "f32", scale == "f32", zero, y == "f32", swiglu)
    out = (ctypes.c_int * 3)()
    _library().choose(v, CUS, out)
    return ("block", out[2]) if out[0] == 0 else ("stream", 4 * out[0], bool(out[1]))


def block_rows(x, scale, zero):
    """The most rows of a block of a form: what its registers hold."""
    return 128 if x == "f32" else 192 if zero or scale == "f32" else 256
