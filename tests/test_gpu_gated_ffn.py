"""The gated feed-forward block on the GPU against the 64-bit form.

Tolerances. A tensor-core accumulation of n products in steps of 16 is taken to be off by at most
(n / 16 + 16) 2^-22 of the sum of the products' magnitudes S (a step may lose a unit of FP32's last place,
twice over); half an ulp of a bf16 result is at most 2^-8 of it. With e the bound of G or U:
  |h'|    <= (1.2 eG + 2^-18 |a|) |u| + (|a| + 1.2 eG) eU, then half an ulp (|act'| < 1.2; 2^-18: exp and
             divide of the activation, a few units of the last place each)
  kept    <= e, then half an ulp, or half a step of its group (at most 1 / 127.5 of the group's largest)
  |dup'|, |dgate'| <= 2^-16 (|dh| (|a| + 1.2 |u|)), then half an ulp
  dx, dw: against the products of the operator's own rounded dgate and dup: the accumulation, half an ulp
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mlp_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
A22 = 2.0 ** -22


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


def inputs(M, K, F, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s, c=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * c).to(torch.bfloat16)

    return dict(x=rnd(M, K), wg=rnd(F, K, c=K ** -0.5), wu=rnd(F, K, c=K ** -0.5), dh=rnd(M, F, c=0.1),
                dg=rnd(M, F, c=0.3).float(), du=rnd(M, F, c=0.3).float())


def within(name, got, ref, bound):
    err = np.abs(R.f64(got) - ref)
    bad = np.argwhere(~(err <= bound))
    assert not len(bad), f"{name}: {len(bad)} of {err.size} outside, e.g. {tuple(bad[0])}: off by " \
                         f"{err[tuple(bad[0])]:.3g}, allowed {np.broadcast_to(bound, err.shape)[tuple(bad[0])]:.3g}"


SHAPES = [(1, 8, 8), (7, 64, 40), (1, 520, 1000), (16, 72, 128), (128, 128, 256), (129, 200, 136), (300, 520, 264),
          (257, 1000, 72), (64, 5120, 512), (600, 264, 2056), (1000, 640, 1096), (1300, 4104, 520),
          (2600, 72, 4104)]


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("delta,save", [(False, None), (True, "bf16"), (False, "packed8"), (True, "packed8")])
@pytest.mark.parametrize("M,K,F", SHAPES)
def test_forward(M, K, F, delta, save, act):
    from deterministic_arithmetic_gb300 import gated_ffn as ffn, pack8

    t = inputs(M, K, F, M + K + F)
    kw = dict(delta_gate=t["dg"], delta_up=t["du"]) if delta else {}
    h, gate, up = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], activation=act, save=save, **kw)
    x, wg, wu = R.f64(t["x"]), R.f64(t["wg"]), R.f64(t["wu"])
    dg, du = (R.f64(t["dg"]), R.f64(t["du"])) if delta else (0.0, 0.0)
    rh, g, u = R.ffn(act, x, wg, wu, dg, du)
    n = (K / 16 + 16) * A22
    eg = n * (np.abs(x) @ np.abs(wg).T) + R.U32 * np.abs(g)
    eu = n * (np.abs(x) @ np.abs(wu).T) + R.U32 * np.abs(u)
    a = np.abs(R.act(act, g)[0])
    bound = (1.2 * eg + 2.0 ** -18 * a) * np.abs(u) + (a + 1.2 * eg) * eu
    within("h", h, rh, bound + R.U16 * (np.abs(rh) + bound) + 1e-38)
    if save is None:
        assert gate is None and up is None
    elif save == "bf16":
        within("gate", gate, g, eg + R.U16 * (np.abs(g) + eg))
        within("up", up, u, eu + R.U16 * (np.abs(u) + eu))
    else:
        for name, p, v, e in (("gate", gate, g, eg), ("up", up, u, eu)):
            top = np.pad(np.abs(v) + e, ((0, 0), (0, -F % 32))).reshape(M, -1, 32).max(2)
            within(name, pack8.unpack8(p), v, e + np.repeat(top, 32, 1)[:, :F] / 127.5)
            assert not p.codes[:, F:].any()


@pytest.mark.parametrize("M,K,F", [(5, 24, 72), (130, 136, 200), (260, 64, 1032)])
def test_forward_of_integers_is_exact(M, K, F):
    """Small whole numbers: every sum is exact, so what is kept must be equal, code for code."""
    from deterministic_arithmetic_gb300 import gated_ffn as ffn

    g = torch.Generator(device="cuda").manual_seed(M)
    x, wg, wu = (torch.randint(-2, 3, s, generator=g, device="cuda").to(torch.bfloat16)
                 for s in ((M, K), (F, K), (F, K)))
    dg, du = (torch.randint(-4, 5, (M, F), generator=g, device="cuda").float() for _ in range(2))
    _, G, U = R.ffn("silu", R.f64(x), R.f64(wg), R.f64(wu), R.f64(dg), R.f64(du))
    assert np.abs(G).max() < 256 and np.abs(U).max() < 256       # bf16 holds them
    _, gate, up = ffn.gated_ffn_fwd(x, wg, wu, delta_gate=dg, delta_up=du, save="bf16")
    assert np.array_equal(R.f64(gate), G) and np.array_equal(R.f64(up), U)
    _, gate, up = ffn.gated_ffn_fwd(x, wg, wu, delta_gate=dg, delta_up=du, save="packed8")
    for p, v in ((gate, G), (up, U)):
        codes, scales = R.pack8(v)
        assert np.array_equal(p.codes.cpu().numpy(), codes) and np.array_equal(p.scales.cpu().numpy(), scales)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("save", ["bf16", "packed8"])
@pytest.mark.parametrize("M,K,F", SHAPES)
def test_backward(M, K, F, save, act):
    from deterministic_arithmetic_gb300 import gated_ffn as ffn, pack8

    t = inputs(M, K, F, M + K + F)
    _, gate, up = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], activation=act, save=save)
    dx, dgate, dup, dwg, dwu = ffn.gated_ffn_bwd(t["dh"], t["x"], t["wg"], t["wu"], gate, up, activation=act)
    g, u = (R.f64(pack8.unpack8(v, dtype=torch.float32) if save == "packed8" else v) for v in (gate, up))
    dh, x, wg, wu = R.f64(t["dh"]), R.f64(t["x"]), R.f64(t["wg"]), R.f64(t["wu"])
    a, slope = R.act(act, g)
    ref = {"dup": dh * a, "dgate": dh * u * slope}
    loose = 2.0 ** -16 * np.abs(dh) * (np.abs(a) + 1.2 * np.abs(u))
    for name, got in (("dup", dup), ("dgate", dgate)):
        within(name, got, ref[name], loose + R.U16 * (np.abs(ref[name]) + loose) + 1e-38)
    DG, DU = R.f64(dgate), R.f64(dup)
    n = (2 * F / 16 + 16) * A22
    rdx = DG @ wg + DU @ wu
    e = n * (np.abs(DG) @ np.abs(wg) + np.abs(DU) @ np.abs(wu))
    within("dx", dx, rdx, e + R.U16 * (np.abs(rdx) + e) + 1e-38)
    for name, got, d in (("dw_gate", dwg, DG), ("dw_up", dwu, DU)):
        rd, e = d.T @ x, (M / 16 + 16) * A22 * (np.abs(d).T @ np.abs(x))
        within(name, got, rd, e + R.U16 * (np.abs(rd) + e) + 1e-38)
    dx2, dgate2, dup2, none, none2 = ffn.gated_ffn_bwd(t["dh"], None, t["wg"], t["wu"], gate, up, activation=act,
                                                       weight_grads=False)
    assert none is None and none2 is None
    assert torch.equal(dx, dx2) and torch.equal(dgate, dgate2) and torch.equal(dup, dup2)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_backward_against_differences(act):
    """Central differences of the 64-bit forward, h = 2^-12 (truncation 1e-7, rounding 1e-12), against the
    operator's gradients along random directions. bf16: gate, up, dgate, dup and the result are rounded, each to
    2^-8 at most, and the four together, over sums of hundreds of terms of either sign, stay below 2^-6 |a| |b| of
    the two vectors' norms."""
    from deterministic_arithmetic_gb300 import gated_ffn as ffn

    M, K, F, h = 24, 40, 56, 2.0 ** -12
    t = inputs(M, K, F, 3)
    _, gate, up = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], activation=act, save="bf16")
    dx, _, _, dwg, dwu = ffn.gated_ffn_bwd(t["dh"], t["x"], t["wg"], t["wu"], gate, up, activation=act)
    x, wg, wu, dh = (R.f64(t[k]) for k in ("x", "wg", "wu", "dh"))
    rng = np.random.RandomState(0)
    for i, grad in ((0, dx), (1, dwg), (2, dwu)):
        args = [x, wg, wu]
        v = rng.standard_normal(args[i].shape)
        ends = []
        for s in (h, -h):
            moved = list(args)
            moved[i] = args[i] + s * v
            ends.append((R.ffn(act, *moved)[0] * dh).sum())
        got = (R.f64(grad) * v).sum()
        assert abs((ends[0] - ends[1]) / (2 * h) - got) <= 2.0 ** -6 * np.linalg.norm(R.f64(grad)) * np.linalg.norm(v)


@pytest.mark.parametrize("M,K,F", [(700, 264, 520), (1500, 512, 1024), (2600, 128, 4104), (1300, 4104, 520)])
def test_rows_do_not_depend_on_the_batch(M, K, F):
    from deterministic_arithmetic_gb300 import gated_ffn as ffn

    t = inputs(M, K, F)

    def step(rows):
        x, dh, dg, du = (t[k][rows].clone() for k in ("x", "dh", "dg", "du"))
        h, gate, up = ffn.gated_ffn_fwd(x, t["wg"], t["wu"], delta_gate=dg, delta_up=du, save="packed8")
        hb, gb, ub = ffn.gated_ffn_fwd(x, t["wg"], t["wu"], delta_gate=dg, delta_up=du, save="bf16")
        assert torch.equal(h, hb)
        dx, dgate, dup, dwg, dwu = ffn.gated_ffn_bwd(dh, x, t["wg"], t["wu"], gate, up)
        return (h, gb, ub, gate.codes, gate.scales, up.codes, up.scales, dx, dgate, dup), (dwg, dwu)

    whole, dw = step(slice(0, M))
    for lo, hi in ((0, 1), (M - 1, M), (5, 12), (100, 228), (0, 129), (64, 420), (0, 513)):
        for a, b in zip(whole, step(slice(lo, hi))[0]):
            assert torch.equal(a[lo:hi], b)
    again, dw2 = step(slice(0, M))
    assert all(torch.equal(a, b) for a, b in zip(whole + dw, again + dw2))


@pytest.mark.parametrize("F", [72, 520, 1032, 4104])
def test_every_way_of_taking_dx_gives_the_same_bits(F):
    """Alone, a cluster a tile (by product, by piece of one) and in pairs: a batch of 19300 rows is enough for
    pairs at 96 columns, and its parts reach the others. Reductions of one to four pieces, short last ones."""
    from deterministic_arithmetic_gb300 import gated_ffn as ffn

    t = inputs(19300, 96, F)
    gate, up = t["dg"].bfloat16(), t["du"].bfloat16()

    def dx(lo, hi):
        return ffn.gated_ffn_bwd(t["dh"][lo:hi], t["x"][lo:hi], t["wg"], t["wu"], gate[lo:hi], up[lo:hi],
                                 weight_grads=False)[0]

    whole = dx(0, 19300)
    for lo, hi in ((0, 1), (8, 72), (64, 192), (0, 1300), (128, 5000), (19040, 19300)):
        assert torch.equal(dx(lo, hi), whole[lo:hi]), (lo, hi)


def test_pairs_start_while_the_gpu_is_full():
    """Backward passes back to back: the pairs of CTAs of the product dx start on SMs that are full of the
    element-wise step's CTAs, the two of a pair apart from each other. Each pass gives the same bits."""
    from deterministic_arithmetic_gb300 import gated_ffn as ffn

    t = inputs(4096, 2048, 8192)
    _, gate, up = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], save="bf16")
    outs = [ffn.gated_ffn_bwd(t["dh"], None, t["wg"], t["wu"], gate, up, weight_grads=False) for _ in range(30)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs[1:] for a, b in zip(o[:3], outs[0][:3]))


def test_extreme_activations():
    """Large and infinite gates: the tails are act's limits, and no NaN comes of 0 times infinity in a slope."""
    from deterministic_arithmetic_gb300 import gated_ffn as ffn

    vals = [0.0, -0.0, 20.0, -20.0, 90.0, -90.0, 1e4, -1e4, 1e20, -1e20, 3e38, -3e38] + [1.0] * 4
    gate = torch.tensor([vals], device="cuda", dtype=torch.bfloat16)
    up = torch.ones_like(gate)
    dh = torch.ones_like(gate)
    w = torch.zeros(16, 8, device="cuda", dtype=torch.bfloat16)
    for act in ("silu", "gelu"):
        _, dgate, dup, _, _ = ffn.gated_ffn_bwd(dh, None, w, w, gate, up, activation=act, weight_grads=False)
        y = R.f64(gate)
        assert np.array_equal(R.f64(dgate)[0, 4:12], [1, 0, 1, 0, 1, 0, 1, 0])
        assert np.array_equal(R.f64(dup)[0, 6:12:2], y[0, 6:12:2]) and not R.f64(dup)[0, 7:12:2].any()
        assert R.f64(dgate)[0, 0] == R.f64(dgate)[0, 1] == 0.5


def test_empty_batch_streams_and_given_outputs():
    from deterministic_arithmetic_gb300 import gated_ffn as ffn

    t = inputs(200, 136, 264)
    e = torch.empty(0, 136, dtype=torch.bfloat16, device="cuda")
    eh = torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")
    h, gate, up = ffn.gated_ffn_fwd(e, t["wg"], t["wu"], save="bf16")
    dx, dgate, dup, dwg, dwu = ffn.gated_ffn_bwd(eh, e, t["wg"], t["wu"], gate, up)
    assert h.shape == (0, 264) and dx.shape == (0, 136) and not dwg.any() and not dwu.any()
    ref = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], save="bf16")
    back = ffn.gated_ffn_bwd(t["dh"], t["x"], t["wg"], t["wu"], ref[1], ref[2])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for st in (s, s.cuda_stream):
        got = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], save="bf16", h=torch.empty_like(ref[0]), stream=st)
        gb = ffn.gated_ffn_bwd(t["dh"], t["x"], t["wg"], t["wu"], got[1], got[2], dx=torch.empty_like(back[0]), stream=st)
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(ref + back, got + gb))


def test_refusals():
    from deterministic_arithmetic_gb300 import gated_ffn as ffn, pack8

    t = inputs(16, 64, 40)
    x, wg, wu, dh = t["x"], t["wg"], t["wu"], t["dh"]
    _, gate, up = ffn.gated_ffn_fwd(x, wg, wu, save="bf16")
    for bad in (lambda: ffn.gated_ffn_fwd(x.float(), wg, wu), lambda: ffn.gated_ffn_fwd(x, wg, wu[:8].contiguous()),
                lambda: ffn.gated_ffn_fwd(x, wg.t(), wu), lambda: ffn.gated_ffn_fwd(x, wg, wu.cpu()),
                lambda: ffn.gated_ffn_fwd(x, wg, wu, activation="relu"), lambda: ffn.gated_ffn_fwd(x, wg, wu, save="f32"),
                lambda: ffn.gated_ffn_fwd(x, wg, wu, delta_gate=t["dg"].bfloat16(), delta_up=t["du"].bfloat16()),
                lambda: ffn.gated_ffn_fwd(x, wg, wu, save="packed8", gate=gate, up=up),
                lambda: ffn.gated_ffn_bwd(dh, x, wg, wu, gate, pack8.pack8(up)),
                lambda: ffn.gated_ffn_bwd(dh, x[:8].contiguous(), wg, wu, gate, up),
                lambda: ffn.gated_ffn_bwd(dh, x, wg, wu, gate.float(), up.float()),
                lambda: ffn.gated_ffn_bwd(dh.float(), x, wg, wu, gate, up)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        ffn.gated_ffn_fwd(x, wg, wu, delta_gate=t["dg"])          # both deltas or neither
    from deterministic_arithmetic_gb300 import lora_delta as ld
    with pytest.raises(ld.LoraDeltaError, match="LORA_ERR_SHAPE"):
        ffn.gated_ffn_fwd(x[:, :60].contiguous(), wg[:, :60].contiguous(), wu[:, :60].contiguous())


@pytest.mark.parametrize("kind,site", [(16, 65), (17, 65), (18, 65)])
def test_a_wait_that_runs_out_is_reported(kind, site):
    """The producer of one product is made to wait for what never comes (1 ms limit): the kernel returns, the
    status block names the site, and after a reset the next call gives the same bits as before."""
    from deterministic_arithmetic_gb300 import _capi, gated_ffn as ffn

    t = inputs(300, 136, 264)

    def step():
        h, gate, up = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], save="bf16")
        return (h,) + ffn.gated_ffn_bwd(t["dh"], t["x"], t["wg"], t["wu"], gate, up)

    ref = step()
    try:
        _capi.device_status_reset(kind, 1000)
        step()
        assert _capi.device_status() == (site << 8) | 1
    finally:
        _capi.device_status_reset()
    assert _capi.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(ref, step()))


@pytest.mark.parametrize("M,K,F", [(300, 520, 1032), (5, 264, 4104)])      # a CTA a product, a CTA a piece
def test_a_wait_that_runs_out_in_a_cluster_is_reported(M, K, F):
    """The same where the CTAs of dx's cluster send one another their sums."""
    from deterministic_arithmetic_gb300 import _capi, gated_ffn as ffn

    t = inputs(M, K, F)
    _, gate, up = ffn.gated_ffn_fwd(t["x"], t["wg"], t["wu"], save="bf16")

    def dx():
        return ffn.gated_ffn_bwd(t["dh"], t["x"], t["wg"], t["wu"], gate, up, weight_grads=False)[0]

    ref = dx()
    try:
        _capi.device_status_reset(17, 1000)
        dx()
        assert _capi.device_status() == (65 << 8) | 1
    finally:
        _capi.device_status_reset()
    assert _capi.device_status() == 0
    assert torch.equal(ref, dx())
