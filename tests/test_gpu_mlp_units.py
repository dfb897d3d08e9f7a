"""The MLP-block operators at sizes where a CTA takes several units of work: rings that wrap, accumulators and
barriers that are used again, whole and half tiles on pairs of CTAs. Against 64-bit forms, or bit for bit against
the delta's own backward pass for the unpacked x.

Tolerances: those of the operators' own tests (u = 2^-24; test_gpu_layer_norm.py, test_gpu_gated_ffn.py), with
the column sums' chain taken for any number of rows: a thread's rows (M / 152 at most: one row group a CTA on 152
CTAs), 7 additions over row groups, 29 over the partials of a warp, 16 over warps, 4 for forming xh, 8 to spare:
(M / 152 + 64) u of the sum of magnitudes.
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mlp_ref as R  # noqa: E402
from test_gpu_gated_ffn import A22, inputs as ffn_inputs, within  # noqa: E402
from test_gpu_layer_norm import DT, inputs as ln_inputs, out_ulp  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_arithmetic_gb300 import build_lib

    build_lib.build()


@pytest.fixture(autouse=True)
def _status():
    from deterministic_arithmetic_gb300 import _capi

    yield
    assert _capi.device_status() == 0


# ------------------------------------------------------------------------ dA
# Units of 128 columns x 256 rows on 152 CTAs: 2 to 7 each; last chunks of 256, 184, 136, 100 and 48 rows (four to
# one stage of 64); every padded rank.
@pytest.mark.parametrize("M,K,r", [(8192, 4096, 16), (3000, 4104, 32), (5000, 2056, 64), (6500, 1032, 8),
                                   (4400, 3000, 40), (9000, 1096, 24)])
def test_da_of_several_units_a_cta(M, K, r):
    from deterministic_arithmetic_gb300 import lora_delta as ld, pack8

    g = torch.Generator(device="cuda").manual_seed(M + K)

    def rnd(*s, c=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * c).to(torch.bfloat16)

    N = 72
    # scales of many sizes, so that a scale of another unit or stage would show
    x = rnd(M, K) * torch.exp2(torch.randint(-6, 7, (M, 1), generator=g, device="cuda").float()).bfloat16()
    dy, a, b, u = rnd(M, N, c=0.1), rnd(r, K, c=K ** -0.5), rnd(N, r, c=r ** -0.5), rnd(M, r)
    p = pack8.pack8(x)
    x = pack8.unpack8(p)
    ref = ld.lora_delta_bwd(dy, x, a, b, u, 2.0)
    for name, s, t in zip(("dx", "da", "db", "du"), pack8.lora_delta_bwd_packed8(dy, p, a, b, u, 2.0), ref):
        assert torch.equal(s, t), name
    for _ in range(3):
        assert torch.equal(pack8.pack8_da(ref[3], p), ref[1])
    DU, X = ref[3].double(), x.double()
    got = pack8.pack8_da(ref[3], p).double()
    assert bool(((got - DU.t() @ X).abs() <= 1e-6 * (DU.abs().t() @ X.abs())).all())


# ---------------------------------------------------------------------- norm
# Rows of a group, forward and backward: 5 to 16 (the slot rings of 3 wrap). 5120, 6144 and 8192
# columns fill CTAs of 10, 12 and 16 warps; 33, 513, 2049 and 3002 take one or two elements at a time; above 8192
# the column sums are a kernel of their own (64 partials of 8 warps).
ROWS = [(40000, 33), (10000, 513), (4100, 2049), (4100, 3002), (4500, 4096), (2100, 5120), (1900, 6144), (2500, 8192),
        (700, 9001), (1100, 12288)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", ROWS)
def test_norm_of_many_rows(M, N, dt):
    from deterministic_arithmetic_gb300 import layer_norm as ln, pack8

    x, w, b, dy = ln_inputs(M, N, dt, "f32", M + N)
    y, mean, rstd = ln.layer_norm_fwd(x, w, b, 1e-5)
    X, W, B = R.f64(x), R.f64(w), R.f64(b)
    ry, rm, rr = R.layer_norm(X, W, B, 1e-5)
    C = (40 + N / 512) * R.U32
    em = C * np.abs(X).mean(1)
    within("mean", mean, rm, em + 1e-40)
    within("rstd", rstd, rr, rr * (C + 4 * R.U32) + rr ** 3 * (em ** 2 + 1e-40))
    bound = np.abs(W) * rr[:, None] * (em[:, None] + np.abs(X - rm[:, None]) * (C + 8 * R.U32)) \
        + 2 * R.U32 * (np.abs(ry) + np.abs(B))
    within("y", y, ry, bound + out_ulp(dt, np.abs(ry) + bound))
    for src in (x, pack8.pack8(x)):
        dx, dw, db = ln.layer_norm_bwd(dy, src, w, mean, rstd)
        if src is not x:
            X = R.f64(pack8.unpack8(src, dtype=torch.float32))
        rs, DY = R.f64(rstd), R.f64(dy)
        rdx, rdw, rdb, xh, g = R.layer_norm_bwd(DY, X, W, R.f64(mean), rs)
        C = (48 + N / 512) * R.U32
        bound = rs[:, None] * C * (np.abs(g) + np.abs(g).mean(1, keepdims=True)
                                   + np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
        within("dx", dx, rdx, bound + out_ulp(dt, np.abs(rdx) + bound))
        D = (M / 152 + 64) * R.U32
        within("dw", dw, rdw, D * np.abs(DY * xh).sum(0) + 1e-40)
        within("db", db, rdb, D * np.abs(DY).sum(0) + 1e-40)


def test_norm_of_equal_elements():
    """var = 0: rstd is 1 / sqrt(eps), to the few units that its formula takes."""
    from deterministic_arithmetic_gb300 import layer_norm as ln

    x, w = torch.full((3, 48), 2.5, device="cuda"), torch.ones(48, device="cuda")
    rstd = R.f64(ln.layer_norm_fwd(x, w, eps=1e-5)[2])
    ref = 1 / np.sqrt(np.float64(np.float32(1e-5)))
    assert (np.abs(rstd - ref) <= 4 * R.U32 * ref).all()
