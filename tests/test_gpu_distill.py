"""The loss against a teacher's top logits on the GPU, forward and backward, against the 64-bit forms of base8_ref.py and
against differences."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import base8_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_arithmetic_gb300 import build_lib

    build_lib.build()


def ops():
    from deterministic_arithmetic_gb300 import distill

    return distill


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def make(m, v, top, dtype=F32, seed=0, tail=False, T=1.0, ids=torch.int64, teacher=F32):
    g = torch.Generator(device="cuda").manual_seed(seed + m + v + top)
    full = -2.2 * torch.log(torch.rand(m, v, generator=g, device="cuda") * v + 0.5)
    t, i = torch.topk(full, min(top, v), dim=1)
    if top > v:
        t, i = (torch.nn.functional.pad(a, (0, top - v), value=x) for a, x in ((t, 0.0), (i, -1)))
    z = (full + torch.randn(m, v, generator=g, device="cuda")).to(dtype)
    w = torch.rand(m, generator=g, device="cuda") + 0.5
    lse = torch.logsumexp(full / T, 1) if tail else None
    return dict(logits=z, ids=i.to(ids), teacher=t.to(teacher), teacher_lse=lse, weight=w, temperature=T)


def fwd(c, **kw):
    return ops().distill_topk_fwd(c["logits"], c["ids"], c["teacher"], temperature=c["temperature"],
                                  teacher_lse=c["teacher_lse"], weight=c["weight"], **kw)


def bwd(c, dloss, probs, stats, **kw):
    return ops().distill_topk_bwd(dloss, c["logits"], c["ids"], probs, stats, temperature=c["temperature"], **kw)


def ref(c):
    return R.distill(f64(c["logits"]), c["ids"].cpu().numpy(), f64(c["teacher"]), np.float64(np.float32(c["temperature"])),
                     f64(c["teacher_lse"]), f64(c["weight"]))


def check(c):
    loss, probs, stats = fwd(c)
    want, p, st, dz, tol = ref(c)
    assert np.array_equal(np.isnan(f64(loss)), np.isnan(want))
    off = np.abs(f64(loss) - want)
    assert (off <= tol).all(), f"loss off by {np.max(off / np.maximum(tol, 1e-300)):.3g} of the tolerance"
    # p: an exponential, 2 ulps, of an argument that is right to an ulp of itself and of the norm's sum
    arg = np.abs(np.log(np.maximum(p, 1e-300)))
    assert (np.abs(f64(probs) - p) <= np.where(p < 0, 0, (2.0 ** -21 + 2 * R.U32 * arg) * np.maximum(p, 2.0 ** -126))).all()
    assert np.array_equal(f64(stats)[:, [0, 3]], st[:, [0, 3]])
    dl = torch.rand(len(want), device="cuda") + 0.1
    got = bwd(c, dl, probs, stats)
    assert got.dtype == c["logits"].dtype
    # The forward's tolerance on log q is in stats; q adds an exponential (2^-21) whose argument, about x log2(e) / T and
    # of at most |x| + |m|, has the roundings of its fma and constants; the entries' q - p cancel.
    w = f64(dl)[:, None] * np.where(st[:, 3] != 0, st[:, 3], 0)[:, None] / c["temperature"]
    z = f64(c["logits"])
    with np.errstate(invalid="ignore", over="ignore"):
        far = np.where(np.isfinite(z), np.abs((z - st[:, :1]) / c["temperature"]), 0)
    q = np.exp(-np.minimum(far, 700) - st[:, 1:2] * np.log(2)) * np.isfinite(z)
    rel = 2.0 ** -20 + 2.0 ** -22 * far + (z.shape[1] / 16384 + 64) * R.U32 + 2.0 ** -22 * np.abs(st[:, 1:2])
    t = np.abs(w) * q * rel * np.maximum(1, np.abs(st[:, 2:3]))
    # 1 - r / rho: r is 2^-21 of the entries' mass off, rho 2^-20 of itself
    kept = np.where(p < 0, 0, p).sum(1, keepdims=True)
    rest = np.maximum(1 - st[:, 2:3], 0)
    if c["teacher_lse"] is not None:
        r_over = np.maximum(1 - kept, 2.0 ** -40)
        t = t + np.abs(w) * q * (2.0 ** -19 * rest + 2.0 ** -21 * rest / r_over)
    at = c["ids"].cpu().numpy()
    for r in range(len(at)):
        ok = p[r] >= 0
        t[r, at[r][ok]] += np.abs(w[r]) * 2.0 ** -21 * (p[r][ok] * (1 + arg[r][ok]) + q[r, at[r][ok]])
    dz = dz * f64(dl)[:, None]
    half = R.U16 if got.dtype == BF else R.U32
    off = np.abs(f64(got) - dz)
    bound = t + half * (np.abs(dz) + t) + 2.0 ** -133
    assert (off <= bound).all(), f"gradient off by {np.max(off / bound):.3g} of the tolerance"
    return loss, probs, stats, got


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("m,v,top", [(1, 1, 1), (1, 5, 3), (3, 256, 1), (2, 257, 40), (5, 1000, 64), (2, 1001, 33), (40, 4098, 20),
                                     (1, 20000, 100), (2, 33333, 256), (3, 65544, 1024), (700, 520, 16), (333, 1030, 8)])
def test_loss_and_gradient(m, v, top, dtype, tail):
    check(make(m, v, top, dtype, tail=tail))


@pytest.mark.parametrize("T", [0.5, 1.7, 4.0])
@pytest.mark.parametrize("tail", [False, True])
def test_temperatures(T, tail):
    check(make(9, 3000, 32, T=T, tail=tail))


@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("teacher", [BF, F32])
def test_types_of_ids_and_teacher(ids, teacher):
    check(make(6, 2000, 24, BF, ids=ids, teacher=teacher))


@pytest.mark.parametrize("tail", [False, True])
def test_what_is_no_entry(tail):
    """Ids outside the vocabulary, logits of -infinity, ids given twice (the first counts), rows with no entry at all."""
    c = make(8, 700, 12, tail=tail)
    i, t = c["ids"], c["teacher"]
    i[0, 3:] = -1
    i[1, 0], i[1, 1] = 700, 2 ** 40
    t[2, 5:] = -INF
    i[3, 7] = i[3, 0]                              # a later entry of the first's id, with another logit
    i[4, :] = i[4, 4]
    i[5, :] = -1
    t[6, :] = -INF
    loss, probs, stats, dz = check(c)
    assert probs[3, 7] == -1 and bool((probs[4, 1:] == -1).all()) and probs[4, 0] > 0
    for r in (5, 6):
        assert loss[r] == 0 and not dz[r].any() and not stats[r].any()


def test_many_entries_of_one_id():
    c = make(3, 5000, 1024)
    c["ids"][1, :] = 4321
    c["ids"][2, 512:] = c["ids"][2, :512].flip(0)
    check(c)


def test_rows_of_weight_0_are_not_read():
    c = make(10, 1003, 8, BF, tail=True)
    ok = [t.clone() for t in fwd(c)]
    c["weight"][4] = 0
    c["logits"][4] = float("nan")
    c["teacher"][4] = float("nan")
    loss, probs, stats = fwd(c)
    assert loss[4] == 0 and bool((probs[4] == -1).all()) and not stats[4].any()
    rows = torch.arange(10, device="cuda") != 4
    assert all(same(a[rows], b[rows]) for a, b in zip((loss, probs, stats), ok))
    dl = torch.ones(10, device="cuda")
    dl[7] = 0
    c["logits"][7] = float("nan")
    for block in (False, True):
        dz = bwd(c, dl, probs, stats, block8=block)
        if block:
            from deterministic_arithmetic_gb300 import block8

            dz = block8.unblock8(dz)
        assert not dz[4].any() and not dz[7].any() and bool(dz[3].any())
    assert fwd(dict(c, weight=None))[2][:, 3].tolist() == [1.0] * 10


def test_masked_and_infinite_logits():
    """Logits of -infinity and of the type's lowest value have no part; +infinity and NaN make their row NaN."""
    for dtype in (BF, F32):
        c = make(6, 900, 10, dtype, tail=True)
        z = c["logits"]
        free = torch.ones(900, dtype=torch.bool, device="cuda")
        free[c["ids"][:2].flatten()] = False
        z[0, free & (torch.arange(900, device="cuda") % 3 == 0)] = -INF
        z[1, free & (torch.arange(900, device="cuda") % 2 == 0)] = torch.finfo(dtype).min
        check({k: (v[:2].clone() if isinstance(v, torch.Tensor) else v) for k, v in c.items()})
        z[3, 7], z[4, 8] = INF, float("nan")
        z[5, c["ids"][5, 0]] = -INF
        loss, probs, stats = fwd(c)
        assert bool(loss[3].isnan()) and bool(loss[4].isnan()) and loss[5] == INF and bool(loss[:3].isfinite().all())
        dz = bwd(c, torch.ones(6, device="cuda"), probs, stats)
        assert bool(dz[:3].isfinite().all()) and bool(dz[5].isfinite().all()) and bool(dz[3].isnan().any())


def test_all_of_the_vocabulary_listed():
    """Nothing is left to the rest: its mass and its gradient are 0."""
    c = make(4, 40, 40, tail=True)
    loss, probs, stats = fwd(c)
    dz = bwd(c, torch.ones(4, device="cuda"), probs, stats)
    w = f64(c["weight"])[:, None]
    q = torch.softmax(c["logits"].double(), 1).cpu().numpy()
    p = np.zeros_like(q)
    np.put_along_axis(p, c["ids"].cpu().numpy(), f64(probs), 1)
    assert np.abs(f64(dz) - w * (q - p)).max() < 2.0 ** -18 and bool((stats[:, 2] == 1).all())


@pytest.mark.parametrize("v", [520, 1001, 1030, 256, 255])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_gradient_in_blocks(v, dtype):
    """What block8 gives for the fp32 gradient, whose roundings the fp32 form of the call shows (from the same values)."""
    from deterministic_arithmetic_gb300 import block8

    c = make(9, v, 12, BF, tail=True)
    c["logits"] = c["logits"].to(dtype)
    c["weight"][2] = 0
    _, probs, stats = fwd(c)
    dl = torch.rand(9, device="cuda")
    p = bwd(c, dl, probs, stats, block8=True)
    full = bwd(dict(c, logits=c["logits"].float()), dl, probs, stats)
    q = block8.block8(full)
    assert p.cols == v and p.tile == 1 and same(p.scales, q.scales) and same(p.codes, q.codes)
    given = block8.Block8(torch.empty_like(p.codes), torch.empty_like(p.scales), v, 1)
    assert bwd(c, dl, probs, stats, block8=True, dlogits=given) is given and same(given.codes, p.codes)


@pytest.mark.parametrize("v", [512, 1001, 40000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_are_the_same_bits_in_any_batch(v, dtype):
    """A row alone (spread over a cluster), in a few and in many; the gradient in place of the logits."""
    c = make(600, v, 17, dtype, tail=True)
    loss, probs, stats = fwd(c)
    dl = torch.rand(600, device="cuda")
    dz = bwd(c, dl, probs, stats)
    for rows in (slice(0, 1), slice(40, 60), slice(100, 350), slice(599, 600)):
        d = {k: (x[rows].clone() if isinstance(x, torch.Tensor) else x) for k, x in c.items()}
        got = fwd(d)
        assert all(same(a, b[rows]) for a, b in zip(got, (loss, probs, stats)))
        assert same(bwd(d, dl[rows].clone(), got[1], got[2], dlogits=d["logits"]), dz[rows])
    assert all(same(a, b) for a, b in zip(fwd(c), (loss, probs, stats)))


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(tail):
    """The loss in 64 bits (the same form that the loss is held to) moved along the gradient and back."""
    c = make(5, 300, 9, tail=tail, T=1.5)
    c["weight"] = None
    _, probs, stats = fwd(c)
    dz = f64(bwd(c, torch.ones(5, device="cuda"), probs, stats))
    z, ids, t = f64(c["logits"]), c["ids"].cpu().numpy(), f64(c["teacher"])
    h, size = 2.0 ** -10, np.sqrt((dz * dz).sum())
    up, down = (R.distill(z + s * h * dz / size, ids, t, 1.5, f64(c["teacher_lse"]))[0].sum() for s in (1, -1))
    assert abs((up - down) / (2 * h) / size - 1) < 1e-4          # h^2 times the third derivative, and fp32's roundings


def test_outputs_given_and_no_rows():
    c = make(4, 300, 5)
    out = dict(loss=torch.empty(4, device="cuda"), probs=torch.empty(4, 5, device="cuda"), stats=torch.empty(4, 4, device="cuda"))
    got = fwd(c, **out)
    assert all(a.data_ptr() == b.data_ptr() for a, b in zip(got, out.values())) and all(same(a, b) for a, b in zip(got, fwd(c)))
    e = make(4, 300, 5)
    e = {k: (x[:0].clone() if isinstance(x, torch.Tensor) else x) for k, x in e.items()}
    loss, probs, stats = fwd(e)
    assert loss.shape == (0,) and bwd(e, torch.empty(0, device="cuda"), probs, stats).shape == (0, 300)


def test_offsets_past_32_bits():
    """Rows that start past 2^32 elements: the same bits as in a batch of their own."""
    m, v = 1030, (1 << 22) - 8
    z = torch.full((m, v), -4.0, dtype=BF, device="cuda")
    z[-2:, ::977] = 3.0
    ids = torch.arange(m * 4, device="cuda").view(m, 4) * 997 % v
    t = torch.linspace(0, 3, 4, device="cuda").expand(m, 4).contiguous()
    c = dict(logits=z, ids=ids, teacher=t, teacher_lse=None, weight=None, temperature=1.0)
    loss, probs, stats = fwd(c)
    few = dict(c, logits=z[-2:].clone(), ids=ids[-2:].clone(), teacher=t[-2:].clone())
    got = fwd(few)
    assert all(same(a, b[-2:]) for a, b in zip(got, (loss, probs, stats)))
    dz = bwd(few, torch.ones(2, device="cuda"), *got[1:])
    bwd(c, torch.ones(m, device="cuda"), probs, stats, dlogits=z)
    assert same(z[-2:], dz)
