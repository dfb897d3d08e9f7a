"""Host-side rules of include/lora_mlp.h and its binding, without a GPU."""
import ctypes

import pytest

F = 0x10000        # never dereferenced: the calls below end before the device is touched
OK, NULL, SHAPE, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module", autouse=True)
def _built():
    from deterministic_arithmetic_gb300 import build_lib

    build_lib.build()


def test_packed_backward_of_no_rows_wants_its_gradients():
    """M = 0: da and db, sums over no rows, are written (as zeros), so they have to be there."""
    from deterministic_arithmetic_gb300 import _capi

    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    f = _capi.fn("lora_delta_bwd_packed8", (vp,) * 6 + (ctypes.c_float,) + (i64,) * 4 + (vp,) * 5 + (ctypes.c_size_t, vp))

    def call(da=F, db=F):
        return f(None, None, None, None, None, None, 1.0, 0, 128, 96, 16, None, da, db, None, None, 0, None)

    assert call(da=None) == call(db=None) == NULL
    assert call(da=F + 4) == call(db=F + 8) == ALIGN


def calls_on(device, monkeypatch):
    """A call of every operator with tensors that claim to be on ``device`` (fake ones: they have no memory)."""
    import torch
    from torch._subclasses import fake_tensor
    from torch._subclasses.fake_tensor import FakeTensorMode

    from deterministic_arithmetic_gb300 import gated_ffn as ffn, layer_norm as ln, pack8

    # on a machine with a GPU the mode would first touch the device, which is not there
    monkeypatch.setattr(fake_tensor, "init_gpu_context", lambda *_: None, raising=False)
    with FakeTensorMode():
        def t(*shape, dtype=torch.bfloat16):
            return torch.empty(*shape, dtype=dtype, device=device)

        x, row, w, f32 = t(4, 64), t(64), t(32, 64), t(4, dtype=torch.float32)
        p = pack8.Packed8(t(4, 64, dtype=torch.int8), t(4, 2, dtype=torch.uint8), 64)
        h, du, a, b = t(4, 32), t(4, 8), t(8, 64), t(32, 8)
    return [lambda: ln.layer_norm_fwd(x, row, row), lambda: ln.layer_norm_bwd(x, x, row, f32, f32),
            lambda: ln.layer_norm_bwd(x, p, row, f32, f32), lambda: pack8.pack8(x), lambda: pack8.unpack8(p),
            lambda: pack8.pack8_da(du, p), lambda: pack8.lora_delta_bwd_packed8(h, p, a, b, du, 1.0),
            lambda: ffn.gated_ffn_fwd(x, w, w), lambda: ffn.gated_ffn_bwd(h, x, w, w, h, h)]


@pytest.mark.parametrize("i", range(9))
def test_tensors_on_another_device_than_the_current_one_are_refused(i, monkeypatch):
    """The library launches on the current device, so tensors of another one must not reach it. Device 5 is
    current nowhere here; the refusal comes before any address is taken."""
    with pytest.raises(ValueError, match="cuda:5, which is not the current device"):
        calls_on("cuda:5", monkeypatch)[i]()


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_differences_along_a_gradient_tell_wrong_ones(act):
    """ffn_off_along on the formulas' own gradients and on planted mistakes, at the GPU test's sizes and tolerance."""
    import numpy as np

    import mlp_ref as R

    rng = np.random.RandomState(3)
    M, K, F = 24, 40, 56
    x, wg, wu = rng.standard_normal((M, K)), rng.standard_normal((F, K)) / K ** 0.5, rng.standard_normal((F, K)) / K ** 0.5
    dh = 0.1 * rng.standard_normal((M, F))
    _, g, u = R.ffn(act, x, wg, wu)
    a, slope = R.act(act, g)
    p = a / g                                             # act(g) = g p: the slope without its second term
    dg, du, short = dh * u * slope, dh * a, dh * u * p

    def off(i, grad):
        return R.ffn_off_along(act, x, wg, wu, dh, i, grad)

    right = (dg @ wg + du @ wu, dg.T @ x, du.T @ x)
    assert all(off(i, v) < 1e-6 for i, v in enumerate(right))
    for i, v in ((0, dg @ wg), (0, du @ wu), (0, short @ wg + du @ wu), (0, -dg @ wg + du @ wu), (1, short.T @ x),
                 (1, 0.5 * right[1]), (1, (dh * slope).T @ x), (2, 0.5 * right[2]), (2, (dh * p).T @ x), (2, (dh * g).T @ x)):
        print(act, i, off(i, v))
        assert off(i, v) > 2 * 2.0 ** -7, i


def ffn_plans(tmp_path, cases):
    """(CTAs of a pair, CTAs of a split, tile columns) that the library's rule gives for (mode, m, n, nk, piece,
    whole groups, SMs, pairs, clusters of two, of eight): its header, compiled on the host."""
    import os
    import subprocess

    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "deterministic_arithmetic_gb300", "csrc_mlp")
    rows = ",".join("{" + ",".join(map(str, c)) + "}" for c in cases)
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text('#include <cstdio>\n#include "ffn_plan.h"\nint main() { static const int c[][10] = {%s};\n'
                   'for (auto& v : c) { const mlp::FfnPlan p = mlp::ffn_plan(v[0], v[1], v[2], v[3], v[4], v[5], '
                   '{v[6], v[7], v[8], v[9]});\nstd::printf("%%d %%d %%d\\n", p.cg, p.split, p.bn); } }\n' % rows)
    subprocess.run(["g++", "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True).stdout
    return [tuple(map(int, line.split())) for line in out.splitlines()]


def test_products_are_taken_without_clusters_that_the_device_cannot_hold(tmp_path):
    """A device (or the part of one that a process has) that can form no cluster of eight, of two, or no pair takes
    the products another way; nothing but the way changes. One that holds them all uses all of them."""
    sizes = (1, 8, 16, 64, 128, 129, 300, 512, 1300, 4096, 17408)
    cols = (8, 96, 520, 2048, 5120, 17408)
    shapes = [(mode, m, n, nk, max(4, -(-nk // 4)), packed) for mode in (0, 1, 2) for m in sizes for n in cols
              for nk in (1, 8, 80, 272) for packed in ((0, 1) if mode == 0 else (0,))]
    seen = set()
    for nsm, pairs, two, eight in ((152, 76, 76, 16), (152, 76, 76, 0), (152, 76, 0, 0), (152, 0, 0, 0), (7, 3, 3, 0), (1, 0, 0, 0)):
        for (mode, m, n, nk, piece, packed), (cg, split, bn) in zip(
                shapes, ffn_plans(tmp_path, [s + (nsm, pairs, two, eight) for s in shapes])):
            assert cg in (1, 2) and split in (0, 2, 8) and (cg == 1 or split == 0) and (mode == 1 or split == 0)
            assert cg == 1 or pairs
            assert split != 2 or two
            assert split != 8 or eight
            most, step = (128, 32 if packed else 8) if mode == 0 else (256, 64)
            assert 0 < bn <= most and bn % step == 0 and (cg == 1 or bn == most) and (split == 0 or bn <= 128)
            if eight:
                seen.add((mode, cg, split))
    assert seen == {(0, 1, 0), (0, 2, 0), (1, 1, 0), (1, 2, 0), (1, 1, 2), (1, 1, 8), (2, 1, 0), (2, 2, 0)}
