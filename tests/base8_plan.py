"""csrc_base8/linear_plan.h, host code without CUDA, compiled on its own: ``plan(back, m, n, sms, pairs, wide)`` gives which CTAs a
product takes, ``(ctas of a tile, columns of a tile, columns of an accumulator, k-blocks of a stage)``."""
import ctypes
import functools
import os
import subprocess
import tempfile

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SMS, PAIRS = 152, 76


@functools.lru_cache(None)
def _lib():
    d = tempfile.mkdtemp()
    src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
    with open(src, "w") as f:
        f.write('#include "linear_plan.h"\n'
                'extern "C" void plan(int b, int m, int n, int sms, int pairs, int wide, int* o) {\n'
                '  const mlp::LinPlan p = mlp::lin_plan(b, m, n, sms, pairs, wide);\n'
                '  o[0] = p.cg; o[1] = p.bn; o[2] = p.w; o[3] = p.deep;\n}\n')
    subprocess.run([os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "deterministic_arithmetic_gb300", "csrc_base8"), src, "-o", so], check=True)
    return ctypes.CDLL(so)


def plan(back, m, n, sms=SMS, pairs=PAIRS, wide=True):
    o = (ctypes.c_int * 4)()
    _lib().plan(int(back), m, n, sms, pairs, int(wide), o)
    return tuple(o)
