"""8-bit blocks and the products with weights held so, on the GPU, against the 64-bit forms of base8_ref.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import base8_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_arithmetic_gb300 import build_lib

    build_lib.build()


@pytest.fixture(autouse=True)
def _no_wait_ran_out():
    yield
    from deterministic_arithmetic_gb300 import _capi

    assert _capi.device_status() == 0


def rnd(*shape, c=1.0, dtype=BF, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return (torch.randn(*shape, generator=g, device="cuda") * c).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def b8():
    from deterministic_arithmetic_gb300 import block8

    return block8


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ------------------------------------------------------------------ blocks
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 128), (3, 8), (5, 100), (130, 136), (129, 257), (300, 24), (7, 1031), (256, 384)])
def test_blocks(m, k, dtype, tile):
    x = rnd(m, k, dtype=dtype) * torch.exp(2 * rnd(m, 1, dtype=F32, seed=9)).to(dtype)
    p = b8().block8(x, tile=tile)
    codes, scales = R.block8(f64(x), tile)
    assert p.cols == k and p.tile == tile and p.codes.shape == (m, -(-k // 16) * 16)
    assert np.array_equal(f64(p.scales), scales)
    got = f64(p.codes.float())
    assert np.array_equal(got[:, :k], codes) and not got[:, k:].any()
    for out in (BF, F32):
        assert np.array_equal(f64(b8().unblock8(p, dtype=out)), R.unblock8(codes, scales, tile))


@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("k", [256, 203])
def test_block_values_at_the_ends_of_the_range(k, tile):
    """Zeros, subnormals, the largest numbers, ties, and the scale's steps at 448 = 1.75 * 2^8."""
    x = torch.zeros(6 * 128, k, device="cuda")
    x[0, :4] = torch.tensor([448.0, 449.0, -1.0, 2.0 ** -9], device="cuda")
    x[128, :4] = torch.tensor([448.0, 17.0, 19.0, 2.0 ** -10 * 3], device="cuda")        # ties
    x[256, :3] = torch.tensor([3.4028234663852886e38, -3e38, 1e30], device="cuda")
    x[384, :3] = torch.tensor([2.0 ** -133, 2.0 ** -126, -2.0 ** -149], device="cuda")
    x[512:, :] = rnd(256, k, dtype=F32)
    for dtype in (F32, BF):
        v = x.to(dtype)
        if dtype == BF:
            v[256, 0] = 3.3895313892515355e38
        p = b8().block8(v, tile=tile)
        codes, scales = R.block8(f64(v), tile)
        assert np.array_equal(f64(p.scales), scales) and np.array_equal(f64(p.codes.float())[:, :k], codes)
        out = b8().unblock8(p)
        assert bool(torch.isfinite(out).all()) and np.array_equal(f64(out), R.unblock8(codes, scales, tile))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("tile", [1, 128])
@pytest.mark.parametrize("k", [264, 201])
def test_a_value_that_is_not_finite_reaches_its_block_only(k, tile, bad):
    x = rnd(260, k)
    clean = b8().unblock8(b8().block8(x, tile=tile))
    x[130, 129] = bad
    out = b8().unblock8(b8().block8(x, tile=tile))
    hit = torch.zeros(260, k, dtype=torch.bool, device="cuda")
    hit[130 if tile == 1 else slice(128, 256), 128:256] = True if tile == 128 else False
    if tile == 1:
        hit[130, 128:256] = True
    assert bool(out[hit].isnan().all()) and same(out[~hit], clean[~hit])


def test_block_outputs_given_and_rows_of_a_batch():
    x = rnd(200, 264)
    p = b8().block8(x)
    q = b8().Block8(torch.empty_like(p.codes), torch.empty_like(p.scales), 264, 1)
    assert b8().block8(x, out=q) is q and same(p.codes, q.codes) and same(p.scales, q.scales)
    one = b8().block8(x[37:38].contiguous())
    assert same(one.codes, p.codes[37:38]) and same(one.scales, p.scales[37:38])
    out = torch.empty(200, 264, device="cuda")
    assert b8().unblock8(p, dtype=F32, out=out) is not None and torch.equal(out, b8().unblock8(p).float())
    assert b8().block8(rnd(0, 264)).codes.shape == (0, 272 // 16 * 16)


# ---------------------------------------------------------------- products
def operands(m, k, n, bwd=False, seed=0):
    """Codes of all sizes and scales that are no powers of two."""
    w = b8().block8(rnd(n, k, c=k ** -0.5, seed=seed), tile=128)
    x = b8().block8(rnd(m, n if bwd else k, seed=seed + 1) * torch.exp(rnd(m, 1, dtype=F32, seed=3)).to(BF))
    w.scales *= 1 + 0.3 * torch.rand_like(w.scales)
    x.scales *= 1 + 0.3 * torch.rand_like(x.scales)
    return x, w


def check_product(x, w, bwd, delta=None):
    a = R.unblock8(f64(x.codes.float())[:, :x.cols], f64(x.scales), 1)
    b = R.unblock8(f64(w.codes.float())[:, :w.cols], f64(w.scales), 128)
    b = b if bwd else b.T
    want, tol = a @ b, R.product_tol(a, b, -(-x.cols // 128))
    if delta is not None:
        want = want + f64(delta)
    tol = tol + 2 * R.U32 * np.abs(want)
    run = b8().block8_linear_bwd if bwd else b8().block8_linear_fwd
    y32 = run(x, w, delta=delta, dtype=F32)
    y16 = run(x, w, delta=delta)
    assert y32.dtype == F32 and y16.dtype == BF and same(y32.to(BF), y16)
    off = np.abs(f64(y32) - want)
    assert (off <= tol).all(), f"off by {np.max(off / np.maximum(tol, 1e-300)):.3g} of the tolerance"
    return y32


SIZES = [(1, 1, 1), (1, 128, 128), (1, 16, 40), (7, 100, 33), (16, 520, 200), (130, 128, 48), (100, 1000, 520),
         (333, 520, 1000), (64, 2049, 131), (129, 257, 300), (1, 5120, 4100), (300, 384, 7000), (1, 1024, 20000)]


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("m,k,n", SIZES)
def test_product(m, k, n, bwd):
    x, w = operands(m, k, n, bwd)
    check_product(x, w, bwd)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("m,k,n", [(5, 136, 200), (200, 260, 130), (33, 131, 77), (2500, 520, 2600)])
def test_product_with_delta(m, k, n, bwd):
    x, w = operands(m, k, n, bwd)
    check_product(x, w, bwd, rnd(m, k if bwd else n, dtype=F32))


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("m,k,n", [(2560, 2600, 2600), (4097, 1300, 1304), (2049, 2500, 2501)])
def test_product_of_pairs(m, k, n, bwd):
    x, w = operands(m, k, n, bwd)
    check_product(x, w, bwd)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("k,n", [(1024, 2600), (2600, 1024), (300, 77)])
def test_rows_are_the_same_bits_in_any_batch(k, n, bwd):
    """Every tile width, a CTA alone or in a pair, whole tiles and halves."""
    x, w = operands(4000, k, n, bwd)
    run = b8().block8_linear_bwd if bwd else b8().block8_linear_fwd
    y = run(x, w, dtype=F32)
    for rows in (slice(0, 1), slice(3, 20), slice(100, 300), slice(1000, 1700), slice(300, 2700), slice(3999, 4000)):
        part = b8().Block8(x.codes[rows].clone(), x.scales[rows].clone(), x.cols, 1)
        assert same(run(part, w, dtype=F32), y[rows])
    assert same(run(x, w, dtype=F32), y)


def test_codes_past_the_last_column_are_not_read():
    x, w = operands(20, 200, 72)
    y = b8().block8_linear_fwd(x, w)
    x.codes.view(torch.uint8)[:, 200:] = 0x7F
    w.codes.view(torch.uint8)[:, 200:] = 0x7F
    assert same(b8().block8_linear_fwd(x, w), y)


@pytest.mark.parametrize("bwd", [False, True])
def test_nan_rows_stay_rows(bwd):
    x, w = operands(200, 256, 256, bwd)
    run = b8().block8_linear_bwd if bwd else b8().block8_linear_fwd
    y = run(x, w)
    x.scales[77, 1] = float("nan")
    z = run(x, w)
    keep = torch.arange(200, device="cuda") != 77
    assert bool(z[77].isnan().all()) and same(z[keep], y[keep])


def test_rows_past_the_last_are_left_alone():
    x, w = operands(37, 264, 100)
    big = torch.full((50, 100), 7.0, device="cuda")
    b8().block8_linear_fwd(x, w, dtype=F32, y=big[:37])
    assert bool((big[37:] == 7).all())
