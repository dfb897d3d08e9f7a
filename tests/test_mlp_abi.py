"""include/lora_mlp.h without a GPU: every declared entry point is exported, bad arguments are refused on
the host before the device is touched, and a valid call without a GPU fails loudly."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lora_mlp.h")
F = 0x10000        # never dereferenced: the cases below fail their host-side checks first
BIG = 1 << 40
OK, NULL, SHAPE, ALIGN, RANK, WORKSPACE = range(6)
VP, INT, I64, F32, SIZE = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
ARGS = {
    "lora_layer_norm_fwd": (VP, INT, VP, VP, INT, F32, I64, I64, VP, VP, VP, VP),
    "lora_layer_norm_bwd": (VP, INT, VP, VP, VP, INT, VP, VP, I64, I64, VP, VP, VP, VP, SIZE, VP),
    "lora_pack8": (VP, INT, I64, I64, VP, VP, VP),
    "lora_unpack8": (VP, VP, I64, I64, VP, INT, VP),
    "lora_pack8_da": (VP, VP, VP, I64, I64, I64, VP, VP, SIZE, VP),
    "lora_delta_bwd_packed8": (VP,) * 6 + (F32,) + (I64,) * 4 + (VP,) * 5 + (SIZE, VP),
    "lora_gated_ffn_fwd": (VP,) * 5 + (INT,) + (I64,) * 3 + (VP, INT) + (VP,) * 5,
    "lora_gated_ffn_bwd": (VP,) * 4 + (INT,) + (VP,) * 4 + (INT,) + (I64,) * 3 + (VP,) * 6,
}


def entry(name):
    from deterministic_arithmetic_gb300 import _capi

    return _capi.fn(name, ARGS[name])



@pytest.fixture(scope="module")
def lib():
    from deterministic_arithmetic_gb300 import build_lib
    from deterministic_arithmetic_gb300 import lora_delta as ld

    build_lib.build()
    return ld.library()


def no_gpu():
    import torch

    return not torch.cuda.is_available()


def declared():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    return sorted(set(re.findall(r"^\s*(?:lora_status|size_t)\s+(lora_[a-z_0-9]+)\s*\(", text, flags=re.M)))


def test_every_declared_symbol_is_exported(lib):
    names = declared()
    assert len(names) >= 10 and all(hasattr(lib, n) for n in names)


def test_layer_norm_refusals(lib):
    from deterministic_arithmetic_gb300 import layer_norm as ln

    f = entry("lora_layer_norm_fwd")

    def fwd(x=F, xt=0, w=F, b=F, wt=0, M=4, N=64, y=F, mean=F, rstd=F):
        return f(x, xt, w, b, wt, 1e-5, M, N, y, mean, rstd, None)

    assert fwd(M=0, x=None) == OK
    assert fwd(N=0) == fwd(M=-1) == fwd(N=1 << 31) == fwd(xt=2) == fwd(wt=-1) == SHAPE
    assert fwd(x=None) == fwd(w=None) == fwd(y=None) == fwd(mean=None) == fwd(rstd=None) == NULL
    assert fwd(x=F + 2) == fwd(b=F + 4) == ALIGN
    g = entry("lora_layer_norm_bwd")
    need = ln.layer_norm_bwd_workspace_size(4, 64)
    assert need > 0 and ln.layer_norm_bwd_workspace_size(4, 0) == 0

    def bwd(dy=F, t=0, x=F, xs=None, w=F, wt=0, M=4, N=64, dx=F, dw=F, db=F, ws=F, size=need):
        return g(dy, t, x, xs, w, wt, F, F, M, N, dx, dw, db, ws, size, None)

    assert bwd(N=-3) == bwd(t=7) == SHAPE
    assert bwd(dy=None) == bwd(dw=None) == bwd(ws=None) == bwd(M=0, dw=None) == NULL
    assert bwd(xs=F + 1) == bwd(db=F + 8) == bwd(dx=F + 2) == ALIGN
    assert bwd(size=need - 1) == WORKSPACE
    if no_gpu():
        assert fwd() in (6, 7) and fwd(b=None) in (6, 7) and bwd() in (6, 7) and bwd(db=None) in (6, 7)


def test_pack8_refusals(lib):
    from deterministic_arithmetic_gb300 import pack8

    f = entry("lora_pack8")
    assert f(None, 0, 0, 64, None, None, None) == OK
    assert f(F, 0, 4, 0, F, F, None) == f(F, 5, 4, 8, F, F, None) == f(F, 0, -1, 8, F, F, None) == SHAPE
    assert f(None, 0, 4, 8, F, F, None) == f(F, 0, 4, 8, F, None, None) == NULL
    assert f(F + 2, 0, 4, 8, F, F, None) == f(F, 0, 4, 8, F + 8, F, None) == ALIGN
    g = entry("lora_unpack8")
    assert g(F, F, 4, 8, F, 3, None) == SHAPE and g(F, None, 4, 8, F, 0, None) == NULL
    h = entry("lora_pack8_da")
    need = pack8.pack8_da_workspace_size(300, 520, 16)
    assert need > 0 and pack8.pack8_da_workspace_size(300, 521, 16) == pack8.pack8_da_workspace_size(300, 520, 12) == 0

    def da(du=F, M=300, K=520, R=16, out=F, ws=F, size=need):
        return h(du, F, F, M, K, R, out, ws, size, None)

    assert da(K=12) == da(M=-1) == SHAPE and da(R=72) == da(R=4) == RANK
    assert da(du=None) == da(M=0, out=None) == NULL and da(out=F + 4) == ALIGN and da(size=need - 1) == WORKSPACE
    b = entry("lora_delta_bwd_packed8")
    size = pack8.lora_delta_bwd_packed8_workspace_size(64, 128, 96, 16)

    def bwd(dy=F, codes=F, M=64, K=128, N=96, R=16, ws=F, n=size):
        return b(dy, codes, F, F, F, F, 2.0, M, K, N, R, F, F, F, F, ws, n, None)

    assert bwd(M=0) == OK and bwd(K=100) == SHAPE and bwd(R=12) == RANK
    assert bwd(dy=None) == bwd(codes=None) == bwd(ws=None) == NULL and bwd(codes=F + 2) == ALIGN
    assert bwd(n=size - 1) == WORKSPACE
    if no_gpu():
        assert f(F, 0, 4, 8, F, F, None) in (6, 7) and da() in (6, 7) and bwd() in (6, 7)


def test_gated_ffn_refusals(lib):
    f = entry("lora_gated_ffn_fwd")

    def fwd(x=F, wg=F, dg=None, du=None, act=0, M=4, K=64, N=32, h=F, keep=0, g=None, u=None, gs=None, us=None):
        return f(x, wg, F, dg, du, act, M, K, N, h, keep, g, u, gs, us, None)

    assert fwd(M=0) == OK
    assert fwd(K=60) == fwd(N=4) == fwd(M=-1) == fwd(act=2) == fwd(keep=3) == fwd(K=1 << 22) == SHAPE
    assert fwd(x=None) == fwd(h=None) == fwd(dg=F) == fwd(du=F) == fwd(keep=1, g=F) == NULL
    assert fwd(keep=2, g=F, u=F, gs=F) == NULL
    assert fwd(wg=F + 2) == fwd(dg=F + 4, du=F) == fwd(keep=1, g=F, u=F + 8) == ALIGN
    b = entry("lora_gated_ffn_bwd")

    def bwd(dh=F, x=F, keep=1, g=F, gs=None, us=None, act=0, M=4, K=64, N=32, dx=F, dwg=F, dwu=F):
        return b(dh, x, F, F, keep, g, F, gs, us, act, M, K, N, dx, F, F, dwg, dwu, None)

    assert bwd(M=0, dwg=None, dwu=None) == OK
    assert bwd(keep=0) == bwd(act=-1) == bwd(N=20) == SHAPE
    assert bwd(dh=None) == bwd(x=None) == bwd(dwg=None) == bwd(dx=None) == bwd(keep=2, gs=F) == NULL
    assert bwd(g=F + 2) == bwd(dwu=F + 8) == ALIGN
    if no_gpu():
        assert fwd() in (6, 7) and bwd() in (6, 7) and bwd(x=None, dwg=None, dwu=None) in (6, 7)
        assert bwd(M=0) in (6, 7)                      # the weights' gradients are still zeros to write


def test_status_calls(lib):
    f = lib.lora_mlp_device_status
    f.argtypes, f.restype = [ctypes.c_void_p], ctypes.c_int
    assert f(None) == NULL
