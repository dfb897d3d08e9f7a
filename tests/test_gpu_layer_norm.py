"""Layer norm forward and backward on the GPU against the 64-bit form.

Tolerances, from the operations (u = 2^-24; a sum of n terms added in a chain of c additions is off by at
most c u times the sum of the terms' magnitudes). A row's sum: at most 16 additions in a thread of a held
row (N / 512 in a looped one), 5 in a warp, 16 over warps: C = 40 + N / 512. Then
  |mean'|   <= C u mean|x|
  |rstd'|   <= rstd (C + 4) u, plus what the mean's error does to the variance (its square: nothing)
  |y'|      <= |w| rstd (|mean'| + |d| (C + 8) u) + 2 u (|y| + |b|), then half an ulp of the output type
  |dx'|     <= rstd (C + 8) u (|g| + mean|g| + |xh| mean|g xh|), then half an ulp
  |dw'|, |db'| <= (M / 304 + 64) u sum_m |terms| (+ 4 u for forming xh): a thread's rows, a CTA's groups,
                  the partials of a warp and the warps.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mlp_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_arithmetic_gb300 import build_lib

    build_lib.build()


def inputs(M, N, dt, wdt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda")

    x = (rnd(M, N) * torch.exp(0.5 * rnd(N)) + 0.3).to(DT[dt])
    return x, (1 + 0.1 * rnd(N)).to(DT[wdt]), (0.1 * rnd(N)).to(DT[wdt]), (0.1 * rnd(M, N)).to(DT[dt])


def within(name, got, ref, bound):
    err = np.abs(R.f64(got) - ref)
    bad = np.argwhere(~(err <= bound))
    assert not len(bad), f"{name}: {len(bad)} outside, e.g. {tuple(bad[0])}: off by {err[tuple(bad[0])]:.3g}, " \
                         f"allowed {np.broadcast_to(bound, err.shape)[tuple(bad[0])]:.3g}"


def out_ulp(dt, v):
    return (R.U16 if dt == "bf16" else R.U32) * np.abs(v) + 1e-40


SHAPES = [(1, 1), (3, 7), (1, 8), (2, 31), (9, 33), (5, 512), (17, 513), (8, 520), (33, 1024), (4, 4096), (7, 4097),
          (3, 8192), (2, 8193), (3, 8200), (2, 20000), (700, 96), (1300, 40), (641, 1000)]


@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("M,N", SHAPES)
def test_forward(M, N, dt, wdt):
    from deterministic_arithmetic_gb300 import layer_norm as ln

    x, w, b, _ = inputs(M, N, dt, wdt, M + N)
    for bias in (b, None):
        y, mean, rstd = ln.layer_norm_fwd(x, w, bias, 1e-5)
        X, W = R.f64(x), R.f64(w)
        ry, rm, rr = R.layer_norm(X, W, None if bias is None else R.f64(bias), 1e-5)
        C = (40 + N / 512) * R.U32
        em = C * np.abs(X).mean(1)
        within("mean", mean, rm, em + 1e-40)
        d = np.abs(X - rm[:, None])
        # a row of one element, or of equal ones: var is what the mean's error leaves, squared
        within("rstd", rstd, rr, rr * (C + 4 * R.U32) + rr ** 3 * (em ** 2 + 1e-40))
        B = 0 if bias is None else np.abs(R.f64(bias))
        bound = np.abs(W) * rr[:, None] * (em[:, None] + d * (C + 8 * R.U32)) + 2 * R.U32 * (np.abs(ry) + B)
        within("y", y, ry, bound + out_ulp(dt, np.abs(ry) + bound))


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dt,wdt", [("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("M,N", SHAPES)
def test_backward(M, N, dt, wdt, packed):
    from deterministic_arithmetic_gb300 import layer_norm as ln, pack8

    x, w, b, dy = inputs(M, N, dt, wdt, M + N)
    _, mean, rstd = ln.layer_norm_fwd(x, w, b, 1e-5)
    src = pack8.pack8(x) if packed else x
    dx, dw, db = ln.layer_norm_bwd(dy, src, w, mean, rstd)
    X = R.f64(pack8.unpack8(src, dtype=torch.float32)) if packed else R.f64(x)
    DY, rs = R.f64(dy), R.f64(rstd)
    rdx, rdw, rdb, xh, g = R.layer_norm_bwd(DY, X, R.f64(w), R.f64(mean), rs)
    C = (48 + N / 512) * R.U32
    bound = rs[:, None] * C * (np.abs(g) + np.abs(g).mean(1, keepdims=True)
                               + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    within("dx", dx, rdx, bound + out_ulp(dt, np.abs(rdx) + bound))
    D = (M / 304 + 68) * R.U32 if N <= 8192 else (M / 64 + 68) * R.U32
    within("dw", dw, rdw, D * np.abs(DY * xh).sum(0) + 1e-40)
    within("db", db, rdb, D * np.abs(DY).sum(0) + 1e-40)
    dx2, dw2, none = ln.layer_norm_bwd(dy, src, w, mean, rstd, bias_grad=False)
    assert none is None and torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_backward_against_differences():
    """<dx, v> and the sum's central difference along v, for x, weight and bias. Truncation: h^2 / 6 times a third
    derivative of order 1 (unit rows); rounding: sqrt(M N) terms off by 4 u |y|, over h. At h = 2^-6, M N = 320,
    |dy| |y| ~ 1: 4e-5 and 3e-4 of |dy| |v| / sqrt(M N) each; the tolerance is 1e-3 |dy| |v|."""
    from deterministic_arithmetic_gb300 import layer_norm as ln

    torch.manual_seed(0)
    M, N, h = 5, 64, 2.0 ** -6
    x, w, b, dy, v = (torch.randn(*s, device="cuda") for s in ((M, N), (N,), (N,), (M, N), (M, N)))

    def loss(x_, w_, b_):
        return float((ln.layer_norm_fwd(x_, w_, b_)[0].double() * dy.double()).sum())

    _, mean, rstd = ln.layer_norm_fwd(x, w, b)
    dx, dw, db = ln.layer_norm_bwd(dy, x, w, mean, rstd)
    tol = 1e-3 * float(dy.norm() * v.norm())
    assert abs((loss(x + h * v, w, b) - loss(x - h * v, w, b)) / (2 * h) - float((dx.double() * v).sum())) < tol
    assert abs((loss(x, w + h * v[0], b) - loss(x, w - h * v[0], b)) / (2 * h) - float((dw.double() * v[0]).sum())) < tol
    assert abs((loss(x, w, b + h * v[0]) - loss(x, w, b - h * v[0])) / (2 * h) - float((db.double() * v[0]).sum())) < tol


@pytest.mark.parametrize("N", [40, 513, 4096, 9001])
def test_rows_do_not_depend_on_the_batch(N):
    from deterministic_arithmetic_gb300 import layer_norm as ln

    x, w, b, dy = inputs(700, N, "bf16", "bf16")
    y, mean, rstd = ln.layer_norm_fwd(x, w, b)
    dx, dw, db = ln.layer_norm_bwd(dy, x, w, mean, rstd)
    for lo, hi in ((0, 1), (699, 700), (13, 64), (0, 333)):
        y2, m2, r2 = ln.layer_norm_fwd(x[lo:hi].clone(), w, b)
        dx2, _, _ = ln.layer_norm_bwd(dy[lo:hi].clone(), x[lo:hi].clone(), w, m2, r2)
        for a_, b_ in ((y, y2), (mean, m2), (rstd, r2), (dx, dx2)):
            assert torch.equal(a_[lo:hi], b_)
    dx3, dw3, db3 = ln.layer_norm_bwd(dy, x, w, mean, rstd)
    assert torch.equal(dw, dw3) and torch.equal(db, db3) and torch.equal(dx, dx3)


@pytest.mark.parametrize("N", [33, 512, 9001])
def test_nan_and_infinity_stay_in_their_row(N):
    from deterministic_arithmetic_gb300 import layer_norm as ln

    x, w, b, dy = inputs(6, N, "f32", "f32")
    y0, m0, r0 = ln.layer_norm_fwd(x, w, b)
    x[1, N - 1] = float("nan")
    x[4, 0] = float("-inf")
    y, mean, rstd = ln.layer_norm_fwd(x, w, b)
    keep = torch.tensor([0, 2, 3, 5], device="cuda")
    assert torch.equal(y[keep], y0[keep]) and torch.equal(mean[keep], m0[keep])
    assert y[1].isnan().all() and y[4].isnan().all()      # (x - (-inf)) * rstd: rstd is 1 / sqrt(NaN)
    dx, _, _ = ln.layer_norm_bwd(dy, x, w, mean, rstd)
    dx0, _, _ = ln.layer_norm_bwd(dy, x.nan_to_num(0, 0, 0), w, m0, r0)
    assert torch.equal(dx[keep], dx0[keep]) and dx[1].isnan().all()


def test_empty_batch_and_constant_rows():
    from deterministic_arithmetic_gb300 import layer_norm as ln

    w = torch.ones(48, device="cuda")
    e = torch.empty(0, 48, device="cuda")
    y, mean, rstd = ln.layer_norm_fwd(e, w)
    dx, dw, db = ln.layer_norm_bwd(e, e, w, mean, rstd)
    assert y.shape == dx.shape == (0, 48) and not dw.any() and not db.any()
    x = torch.full((3, 48), 2.5, device="cuda")
    y, mean, rstd = ln.layer_norm_fwd(x, w, eps=1e-5)
    assert not y.any() and torch.equal(mean, x[:, 0])
    assert (R.f64(rstd) - 1e-5 ** -0.5 < 1e-3).all()


def test_other_stream_and_given_outputs():
    from deterministic_arithmetic_gb300 import layer_norm as ln

    x, w, b, dy = inputs(300, 1000, "bf16", "bf16")
    y, mean, rstd = ln.layer_norm_fwd(x, w, b)
    ref = ln.layer_norm_bwd(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for st in (s, s.cuda_stream):
        outs = ln.layer_norm_fwd(x, w, b, y=torch.empty_like(y), stream=st)
        got = ln.layer_norm_bwd(dy, x, w, outs[1], outs[2], stream=st)
        s.synchronize()
        assert torch.equal(outs[0], y) and all(torch.equal(p, q) for p, q in zip(got, ref))


def test_refusals():
    from deterministic_arithmetic_gb300 import layer_norm as ln, lora_delta as ld

    x, w, b, dy = inputs(16, 64, "bf16", "bf16")
    y, mean, rstd = ln.layer_norm_fwd(x, w, b)
    for bad in (lambda: ln.layer_norm_fwd(x.half(), w, b), lambda: ln.layer_norm_fwd(x[:, ::2], w[::2].contiguous()),
                lambda: ln.layer_norm_fwd(x, w[:32].contiguous()), lambda: ln.layer_norm_fwd(x, w, b.float()),
                lambda: ln.layer_norm_fwd(x, w.cpu()), lambda: ln.layer_norm_fwd(x, w, y=y.float()),
                lambda: ln.layer_norm_fwd(x[0], w),
                lambda: ln.layer_norm_bwd(dy, x.float(), w, mean, rstd),
                lambda: ln.layer_norm_bwd(dy, x, w, mean[:8].contiguous(), rstd),
                lambda: ln.layer_norm_bwd(dy, x, w, mean.double(), rstd)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ld.LoraDeltaError, match="LORA_ERR_WORKSPACE"):
        ln.layer_norm_bwd(dy, x, w, mean, rstd, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ld.LoraDeltaError, match="LORA_ERR_ALIGN"):
        ln.layer_norm_fwd(torch.empty(17 * 64, dtype=torch.bfloat16, device="cuda")[1:1 + 16 * 64].view(16, 64), w, b)
