"""include/lora_base8.h without a GPU: every declared entry point is exported, bad arguments are refused on the host
before the device is touched, a valid call without a GPU fails loudly, and tensors of another device are refused."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "lora_base8.h")
F = 0x10000        # never dereferenced: the cases below fail their host-side checks first
OK, NULL, SHAPE, ALIGN = range(4)
VP, INT, I64, F32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
INF, NAN = float("inf"), float("nan")
ARGS = {
    "lora_block8": (VP, INT, INT, I64, I64, VP, VP, VP),
    "lora_unblock8": (VP, VP, INT, I64, I64, VP, INT, VP),
    "lora_block8_linear_fwd": (VP,) * 5 + (I64,) * 3 + (VP, INT, VP),
    "lora_block8_linear_bwd": (VP,) * 5 + (I64,) * 3 + (VP, INT, VP),
    "lora_distill_topk_fwd": (VP, INT, VP, INT, VP, INT, VP, VP, F32, I64, I64, I64, VP, VP, VP, VP),
    "lora_distill_topk_bwd": (VP, VP, INT, VP, INT, VP, VP, F32, I64, I64, I64, VP, VP, VP),
}


def entry(name):
    from deterministic_arithmetic_gb300 import _capi

    return _capi.fn(name, ARGS[name])


def no_gpu():
    import torch

    return not torch.cuda.is_available()


@pytest.fixture(scope="module", autouse=True)
def lib():
    from deterministic_arithmetic_gb300 import build_lib
    from deterministic_arithmetic_gb300 import lora_delta as ld

    build_lib.build()
    return ld.library()


def test_every_declared_symbol_is_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:lora_status|size_t)\s+(lora_[a-z_0-9]+)\s*\(", text, flags=re.M)))
    assert names == sorted(ARGS) and all(hasattr(lib, n) for n in names)


def test_block8_refusals():
    f, g = entry("lora_block8"), entry("lora_unblock8")
    assert f(None, 0, 1, 0, 64, None, None, None) == g(None, None, 128, 0, 64, None, 1, None) == OK
    for bad in (f(F, 0, 1, 4, 0, F, F, None), f(F, 2, 1, 4, 8, F, F, None), f(F, 0, 1, -1, 8, F, F, None),
                f(F, 0, 64, 4, 8, F, F, None), f(F, 0, 1, 4, 1 << 31, F, F, None), g(F, F, 2, 4, 8, F, 0, None),
                g(F, F, 1, 4, 8, F, 3, None)):
        assert bad == SHAPE
    assert f(None, 0, 1, 4, 8, F, F, None) == f(F, 0, 1, 4, 8, None, F, None) == f(F, 0, 1, 4, 8, F, None, None) == NULL
    assert f(F + 2, 0, 1, 4, 8, F, F, None) == f(F, 0, 1, 4, 8, F + 8, F, None) == g(F, F + 4, 1, 4, 8, F, 0, None) == ALIGN
    if no_gpu():
        assert f(F, 0, 1, 4, 8, F, F, None) in (6, 7) and g(F, F, 128, 4, 8, F, 1, None) in (6, 7)


@pytest.mark.parametrize("name", ["lora_block8_linear_fwd", "lora_block8_linear_bwd"])
def test_linear_refusals(name):
    f = entry(name)

    def call(x=F, xs=F, w=F, ws=F, delta=None, M=4, K=64, N=32, y=F, t=0):
        return f(x, xs, w, ws, delta, M, K, N, y, t, None)

    assert call(M=0, x=None, w=None, y=None) == OK
    for bad in (call(M=-1), call(K=0), call(N=0), call(K=1 << 22), call(N=1 << 22), call(M=1 << 22), call(t=2), call(t=-1)):
        assert bad == SHAPE
    assert call(x=None) == call(xs=None) == call(w=None) == call(ws=None) == call(y=None) == NULL
    assert call(x=F + 8) == call(ws=F + 4) == call(delta=F + 4) == call(y=F + 2) == ALIGN
    if no_gpu():
        assert call() in (6, 7) and call(delta=F, t=1, K=61, N=31) in (6, 7)


def test_distill_refusals():
    f, g = entry("lora_distill_topk_fwd"), entry("lora_distill_topk_bwd")

    def fwd(z=F, t=0, ids=F, ib=8, te=F, tt=1, lse=None, w=None, T=1.0, M=4, V=100, top=5, loss=F, probs=F, stats=F):
        return f(z, t, ids, ib, te, tt, lse, w, T, M, V, top, loss, probs, stats, None)

    def bwd(dl=F, z=F, t=0, ids=F, ib=8, probs=F, stats=F, T=1.0, M=4, V=100, top=5, dz=F, sc=None):
        return g(dl, z, t, ids, ib, probs, stats, T, M, V, top, dz, sc, None)

    assert fwd(M=0, z=None) == bwd(M=0, z=None) == OK
    for call in (fwd, bwd):
        for bad in (call(t=2), call(ib=2), call(T=0.0), call(T=-1.0), call(T=INF), call(T=NAN), call(T=1e-39), call(M=-1), call(V=0),
                    call(V=1 << 22), call(top=0), call(top=1025), call(M=1 << 28)):
            assert bad == SHAPE
        assert call(z=None) == call(ids=None) == call(probs=None) == call(stats=None) == NULL
        assert call(z=F + 2) == call(ids=F + 8) == call(stats=F + 4) == ALIGN
    assert fwd(tt=5) == SHAPE and fwd(te=None) == fwd(loss=None) == bwd(dl=None) == bwd(dz=None) == NULL
    assert fwd(lse=F + 4) == fwd(w=F + 8) == bwd(sc=F + 4) == bwd(dz=F + 2) == ALIGN
    if no_gpu():
        assert fwd() in (6, 7) and fwd(lse=F, w=F, V=101) in (6, 7) and bwd() in (6, 7) and bwd(sc=F, V=101) in (6, 7)


def calls_on(device, monkeypatch):
    """A call of every operator with tensors that claim to be on ``device`` (fake ones: they have no memory)."""
    import torch
    from torch._subclasses import fake_tensor
    from torch._subclasses.fake_tensor import FakeTensorMode

    from deterministic_arithmetic_gb300 import block8 as b8, distill as ds

    # on a machine with a GPU the mode would first touch the device, which is not there
    monkeypatch.setattr(fake_tensor, "init_gpu_context", lambda *_: None, raising=False)
    with FakeTensorMode():
        def t(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device=device)

        x, ids, row = t(4, 64), t(4, 5, dtype=torch.int64), t(4)
        f8 = torch.float8_e4m3fn
        p, w = b8.Block8(t(4, 64, dtype=f8), t(4, 1), 64, 1), b8.Block8(t(64, 64, dtype=f8), t(1, 1), 64, 128)
        top, stats = t(4, 5), t(4, 4)
    return [lambda: b8.block8(x), lambda: b8.unblock8(p), lambda: b8.block8_linear_fwd(p, w), lambda: b8.block8_linear_bwd(p, w),
            lambda: ds.distill_topk_fwd(x, ids, top), lambda: ds.distill_topk_bwd(row, x, ids, top, stats)]


@pytest.mark.parametrize("i", range(6))
def test_tensors_on_another_device_than_the_current_one_are_refused(i, monkeypatch):
    with pytest.raises(ValueError, match="cuda:5, which is not the current device"):
        calls_on("cuda:5", monkeypatch)[i]()


def test_types_are_refused_before_the_device_is_touched():
    import torch

    from deterministic_arithmetic_gb300 import block8 as b8, distill as ds

    x = torch.zeros(4, 64)
    p = b8.Block8(torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 1), 64, 1)
    for bad in (lambda: b8.unblock8(p, dtype=torch.float16), lambda: b8.block8_linear_fwd(p, p, dtype=torch.int8),
                lambda: b8.block8(x), lambda: b8.unblock8(p), lambda: ds.distill_topk_fwd(x, x, x)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: b8.unblock8(x), lambda: b8.block8_linear_fwd(x, p), lambda: b8.block8([1.0]),
                lambda: ds.distill_topk_bwd(x, None, x, x, x)):
        with pytest.raises(TypeError):
            bad()
