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


# -------------------------------------------------------------- gated block
def check_products(M, K, F, act, delta):
    """Forward and backward against 64 bits, the products with torch's 64-bit ones (the sizes are large)."""
    from deterministic_arithmetic_gb300 import gated_ffn as ffn, pack8

    t = ffn_inputs(M, K, F, M + K + F)
    kw = dict(delta_gate=t["dg"], delta_up=t["du"]) if delta else {}
    h, gate, up = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], activation=act, save="bf16", **kw)
    h8, gate8, up8 = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], activation=act, save="packed8", **kw)
    assert torch.equal(h, h8)

    def prod(p, q):                                       # 64-bit, and the sum of the products' magnitudes
        return (p @ q).cpu().numpy(), (p.abs() @ q.abs()).cpu().numpy()

    x, wg, wu = t["x"].double(), t["wg"].double(), t["wu"].double()
    n = (K / 16 + 16) * A22
    pre, err = [], []
    for w, d in ((wg, "dg"), (wu, "du")):
        v, s = prod(x, w.t())
        v = v + (R.f64(t[d]) if delta else 0.0)
        pre.append(v)
        err.append(n * s + R.U32 * np.abs(v))
    (g, u), (eg, eu) = pre, err
    a = np.abs(R.act(act, g)[0])
    rh = R.act(act, g)[0] * u
    bound = (1.2 * eg + 2.0 ** -18 * a) * np.abs(u) + (a + 1.2 * eg) * eu
    within("h", h, rh, bound + R.U16 * (np.abs(rh) + bound) + 1e-38)
    for name, b16, p8, v, e in (("gate", gate, gate8, g, eg), ("up", up, up8, u, eu)):
        within(name, b16, v, e + R.U16 * (np.abs(v) + e))
        top = np.pad(np.abs(v) + e, ((0, 0), (0, -F % 32))).reshape(M, -1, 32).max(2)
        within(name + " in 8 bits", pack8.unpack8(p8), v, e + np.repeat(top, 32, 1)[:, :F] / 127.5)
    del h8, gate8, up8
    dx, dgate, dup, dwg, dwu = ffn.gated_ffn_bwd(t["dh"], t["x"], t["wg"], t["wu"], gate, up, activation=act)
    DG, DU = dgate.double(), dup.double()
    (p, sp), (q, sq) = prod(DG, wg), prod(DU, wu)
    e = (2 * F / 16 + 16) * A22 * (sp + sq)
    within("dx", dx, p + q, e + R.U16 * (np.abs(p + q) + e) + 1e-38)
    for name, got, d in (("dw_gate", dwg, DG), ("dw_up", dwu, DU)):
        rd, s = prod(d.t(), x)
        e = (M / 16 + 16) * A22 * s
        within(name, got, rd, e + R.U16 * (np.abs(rd) + e) + 1e-38)


# With 76 pairs of CTAs (256 x 256 tiles of dx and dW, 256 x 128 of the forward): tiles, and what is left for a last
# round in half tiles where it is at most 38.
#   1300 x 4160 -> 576   dx 102 (26 halved), operands in whole 64-column blocks
#   2100 x 2560 -> 1088  forward 81 (5), dx 90 (14), dW 100 (24), blocks
#   2600 x 1792 -> 896   forward 77 (1), dx 77 (1), blocks
#   2600 x 1792 -> 1408  forward 121, dx 77 (1), dW 84 (8), blocks
#   5000 x 2048 -> 2048  forward 320 (16), dx 160 (8), dW 128, blocks: several tiles a pair
#   2300 x 2312 -> 1096  forward 81 (5), dx 90 (14), dW 100 (24), rows that are not whole blocks
@pytest.mark.parametrize("M,K,F,act,delta", [
    (1300, 4160, 576, "silu", True), (2100, 2560, 1088, "gelu", False), (2600, 1792, 896, "silu", True),
    (2600, 1792, 1408, "gelu", True), (5000, 2048, 2048, "silu", False), (2300, 2312, 1096, "silu", True)])
def test_products_on_pairs(M, K, F, act, delta):
    check_products(M, K, F, act, delta)


@pytest.mark.parametrize("M,K,F", [(2600, 1792, 1408), (4096, 1536, 2112)])
def test_rows_of_pairs_with_blocked_operands_do_not_depend_on_the_batch(M, K, F):
    """The whole batch goes to pairs of CTAs, its parts to lone CTAs and to clusters, all with blocked operands."""
    from deterministic_arithmetic_gb300 import gated_ffn as ffn

    t = ffn_inputs(M, K, F)

    def step(lo, hi):
        x, dh, dg, du = (t[k][lo:hi].clone() for k in ("x", "dh", "dg", "du"))
        h, gate, up = ffn.gated_ffn_fwd(x, t["wg"], t["wu"], delta_gate=dg, delta_up=du, save="bf16")
        return (h, gate, up) + ffn.gated_ffn_bwd(dh, x, t["wg"], t["wu"], gate, up)

    whole = step(0, M)
    for lo, hi in ((0, 1), (M - 1, M), (8, 72), (100, 228), (0, 300), (64, 1100), (300, M)):
        for a, b in zip(whole[:6], step(lo, hi)[:6]):
            assert torch.equal(a[lo:hi], b), (lo, hi)
    assert all(torch.equal(a, b) for a, b in zip(whole, step(0, M)))


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_against_differences_along_themselves(act):
    """The slope of the 64-bit forward along each gradient is that gradient's length. Tolerance: gate, up, dgate (dup)
    and the result are each rounded to bf16, 2^-9 of a value at most; the errors of one gradient's terms are
    independent in sign, so its error's length stays below 2^-9 sqrt(4) = 2^-8 of its own, and 2^-7 allows twice that.
    Truncation (h^2, h = 2^-12) and 64-bit rounding are below 1e-6. A missing or halved term is off by several times
    the tolerance (test_mlp_host.py shows it on planted ones)."""
    from deterministic_arithmetic_gb300 import gated_ffn as ffn

    t = ffn_inputs(24, 40, 56, 3)
    _, gate, up = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], activation=act, save="bf16")
    dx, _, _, dwg, dwu = ffn.gated_ffn_bwd(t["dh"], t["x"], t["wg"], t["wu"], gate, up, activation=act)
    args = [R.f64(t[k]) for k in ("x", "wg", "wu", "dh")]
    for i, grad in enumerate((dx, dwg, dwu)):
        assert R.ffn_off_along(act, *args, i, R.f64(grad)) <= 2.0 ** -7, i
