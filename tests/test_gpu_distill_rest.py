"""The loss with the teacher's log-sum-exp where its pieces are far apart, against its definition in 64 bits and that one's
automatic differentiation."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_distill import BF, F32, INF, _built, bwd, f64, fwd, make, same  # noqa: E402,F401

pytestmark = pytest.mark.gpu
U32 = 2.0 ** -24


def definition(c, dloss, no_rest=False):
    """(loss, gradient of sum(dloss * loss), parts) in 64 bits, from the formula of include/lora_base8.h; every entry counts.
    no_rest: r is 0."""
    T = c["temperature"]
    z = c["logits"].double().requires_grad_()
    ids = c["ids"].long()
    log_p = c["teacher"].double() / T - c["teacher_lse"].double()[:, None]
    p = log_p.exp()
    log_q = torch.log_softmax(z / T, 1)
    part = p * (log_p - log_q.gather(1, ids))
    loss = part.sum(1)
    r = (1 - p.sum(1)).clamp_min(0)
    listed = torch.zeros_like(z, dtype=torch.bool).scatter_(1, ids, True)
    if no_rest:
        r = torch.zeros_like(r)
    on = r > 0
    log_rho = torch.full_like(r, -math.inf)
    if on.any():
        others = (z[on] / T).masked_fill(listed[on], -math.inf)
        log_rho[on] = torch.logsumexp(others, 1) - torch.logsumexp(z[on] / T, 1)
        loss = loss.index_add(0, on.nonzero()[:, 0], r[on] * (r[on].log() - log_rho[on]))
    w = torch.ones_like(r) if c["weight"] is None else c["weight"].double()
    loss = loss * w
    dz, = torch.autograd.grad((dloss.double() * loss).sum(), z)
    return loss.detach(), dz, dict(p=p, log_p=log_p, part=part.detach(), r=r, log_rho=log_rho.detach(), listed=listed,
                                   log_q=log_q.detach(), w=w, T=T)


def off_by(c, dloss, loss, dz, k):
    """How far fp32 may be off: (loss, gradient before its last rounding). A probability is an exponential (2^-21) of an
    argument right to an ulp of itself; log q adds to that the sums' roundings; r is as far off as the sum of p; a far
    rest's log2(r / rho) is held, and taken from an exponent again, in fp32."""
    z, T, v = c["logits"].double(), k["T"], c["logits"].shape[1]
    far = ((z - z.amax(1, keepdim=True)) / T).abs().clamp_max(1e300)
    q = k["log_q"].exp()
    live = torch.where(q > 0, far, 0.0)
    sums = (v / 16384 + 64) * U32
    d_log = 2.0 ** -21 * (1 + (q * live).sum(1)) + sums
    mass = k["p"].sum(1)
    dr = 2.0 ** -21 * (k["p"] * (1 + k["log_p"].abs())).sum(1)
    r = k["r"]
    on = r > 0
    lr = torch.where(on, (r.clamp_min(1e-300).log() - torch.where(on, k["log_rho"], 0.0)).abs(), 0.0)
    tol = (mass + r) * d_log + 2.0 ** -21 * (k["part"].abs().sum(1) + mass) + dr * (1 + lr) * on + 2.0 ** -20 * r * lr
    tol = tol * k["w"].abs() + 2 * U32 * loss.abs()
    scale = (dloss.double() * k["w"] / T).abs()[:, None]
    own = q * torch.maximum(mass, torch.ones_like(mass))[:, None]
    L = torch.where(on, -torch.where(on, k["log_rho"], 0.0) / math.log(2), 0.0)[:, None]
    rel = 2.0 ** -19 + sums + 2.0 ** -22 * (live + k["log_q"].abs().amin(1, keepdim=True))
    rest = torch.where(on[:, None] & ~k["listed"], (own - dz / (dloss.double() * k["w"] / T)[:, None]).abs(), 0.0)   # r rho_j
    t = own * rel + rest * (rel + 2.0 ** -22 * L + torch.where(on, dr / r.clamp_min(1e-300), 0.0)[:, None])
    t.scatter_add_(1, c["ids"].long(), 2.0 ** -21 * (k["p"] * (1 + k["log_p"].abs()) + own.gather(1, c["ids"].long())))
    return tol, scale * t


def check(c, no_rest=False, seed=1):
    """The loss and its gradient (as it is and in blocks) of c."""
    from deterministic_arithmetic_gb300 import block8

    m = len(c["logits"])
    dl = torch.rand(m, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda") + 0.1
    loss, probs, stats = fwd(c)
    got = bwd(c, dl, probs, stats)
    want, dz, k = definition(c, dl, no_rest)
    tol, t = off_by(c, dl, want, dz, k)
    off = (loss.double() - want).abs()
    assert bool((off <= tol).all()), f"loss off by {float((off / tol).max()):.3g} of the tolerance"
    half = 2.0 ** -8 if got.dtype == BF else U32
    bound = t + half * (dz.abs() + t) + 2.0 ** -133
    off = (got.double() - dz).abs()
    assert bool((off <= bound).all()), f"gradient off by {float((off / bound).max()):.3g} of the tolerance"
    full = bwd(dict(c, logits=c["logits"].float()), dl, probs, stats)
    b, a = bwd(c, dl, probs, stats, block8=True), block8.block8(full)
    assert same(a.codes, b.codes) and same(a.scales, b.scales)
    few = {key: (x[1:3].clone() if isinstance(x, torch.Tensor) else x) for key, x in c.items()}
    alone = fwd(few)
    assert all(same(x, y[1:3]) for x, y in zip(alone, (loss, probs, stats)))
    assert same(bwd(few, dl[1:3].clone(), *alone[1:]), got[1:3])
    return loss, got, k


def on_gpu(a, dtype=F32):
    return torch.from_numpy(a).to("cuda").to(dtype)


# ------------------------------------------ entries whose probabilities sum to more than 1
def peaked(m, v, top, dtype, T, student=None):
    """Rows with a few logits near 24, the teacher's kept in bf16 (half a step is 0.06 there), its log-sum-exp of the fp32 ones."""
    rng = np.random.default_rng(m + v)
    full = rng.standard_normal((m, v)) * 2
    full[:, :3] = 24 + rng.standard_normal((m, 3))
    full = on_gpu(full)
    t, ids = torch.topk(full, top, dim=1)
    z = full + on_gpu(rng.standard_normal((m, v))) if student is None else full
    lse = torch.logsumexp(full.double() / T, 1).float()
    return dict(logits=z.to(dtype), ids=ids, teacher=t.to(BF), teacher_lse=lse, weight=on_gpu(rng.random(m) + 0.5), temperature=T)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0.5, 1.0, 1.5])
@pytest.mark.parametrize("v", [2000, 2001])
def test_a_teacher_in_bf16_whose_entries_sum_to_more_than_1(v, T, dtype):
    c = peaked(64, v, 20, dtype, T)
    _, got, k = check(c)
    over = k["p"].sum(1)
    assert int((over > 1.005).sum()) >= 5 and int((over < 0.995).sum()) >= 5
    if dtype == F32:                               # a softmax's gradient sums to 0: v roundings of values of up to 1
        assert float(got.double().sum(1).abs().max()) < 1.6 / T * (v * U32 + 2.0 ** -16)


def test_the_gradient_where_they_do_is_that_of_the_losses_differences():
    c = peaked(64, 2000, 20, F32, 1.0)
    c["weight"] = None
    _, probs, stats = fwd(c)
    over = probs.clamp_min(0).sum(1) > 1.005
    dl = over.float()
    dz = bwd(c, dl, probs, stats).double()
    assert not dz[~over].any()
    size = dz.norm(dim=1, keepdim=True).clamp_min(1e-30)
    h = 2.0 ** -10
    up, down = (definition(dict(c, logits=c["logits"].double() + s * h * dz / size), dl)[0] for s in (1, -1))
    slope = (up - down)[over] / (2 * h)
    assert float((slope / size[over, 0] - 1).abs().max()) < 1e-4      # h^2 times the third derivative, and fp32's roundings


# ------------------------------------------------------------- a rest far below the entries
def gapped(gap, T, dtype, r=0.05, m=8, v=700, top=12):
    """The student's unlisted logits lie gap * T below the listed ones; the teacher's unlisted mass is r."""
    rng = np.random.default_rng(int(gap * 8) + m)
    z = T * (rng.standard_normal((m, v)) - gap)
    ids = np.argsort(rng.random((m, v)), 1)[:, :top]
    np.put_along_axis(z, ids, T * rng.standard_normal((m, top)), 1)
    t = on_gpu(T * rng.standard_normal((m, top)))
    lse = (torch.logsumexp(t.double() / T, 1) - math.log1p(-r)).float()
    return dict(logits=on_gpu(z, dtype), ids=on_gpu(ids, torch.int64), teacher=t, teacher_lse=lse,
                weight=on_gpu(rng.random(m) + 0.5), temperature=T)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0.1, 0.25, 1.0, 4.0])
@pytest.mark.parametrize("gap", [20, 42, 46, 60, 85, 90, 120, 700, 2500])
def test_a_rest_far_below_the_entries(gap, T, dtype):
    for r in (0.3, 0.01):
        loss, got, k = check(gapped(gap, T, dtype, r))
        assert bool(loss.isfinite().all())
        # the rest's gradient is -r of the row's, however small rho
        at = torch.where(k["listed"], 0.0, got.double()).sum(1)
        assert bool((at < 0).all())


@pytest.mark.parametrize("v", [701, 40000])
def test_a_far_rest_of_rows_of_other_lengths(v):
    for dtype in (BF, F32):
        check(gapped(100, 0.5, dtype, v=v, top=30))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("gap", [5000, 1e6, None])
def test_a_rest_further_down_than_the_gradient_knows(gap, dtype):
    """Below 2^-4096 the rest has no gradient; the loss is still the formula's. None: the type's lowest value."""
    c = gapped(gap or 10, 1.0, dtype)
    if gap is None:
        keep = torch.zeros_like(c["logits"], dtype=torch.bool).scatter_(1, c["ids"], True)
        c["logits"].masked_fill_(~keep, torch.finfo(dtype).min)
    dl = torch.ones(8, device="cuda")
    loss, probs, stats = fwd(c)
    got = bwd(c, dl, probs, stats)
    want, dz, k = definition(c, dl)
    tol, t = off_by(c, dl, want, dz, k)
    assert bool(((loss.double() - want).abs() <= tol).all()) and bool(loss.isfinite().all())
    assert not got[~k["listed"]].any()
    half = 2.0 ** -8 if dtype == BF else U32
    off = (got.double() - dz).abs()
    assert bool((off <= t + half * (dz.abs() + t))[k["listed"]].all())


# -------------------------------------------------------- nothing left to the student's rest
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0.3, 1.0, 3.0])
@pytest.mark.parametrize("mask", ["all listed", "-inf", "lowest"])
@pytest.mark.parametrize("at", [0.0, 30.0, -200.0])
def test_an_r_that_is_rounding_counts_as_0_where_rho_is_nothing(at, mask, T, dtype):
    """The teacher's listed logits are all it has, so r is 0, and what fp32 leaves of 1 - sum p is not: no such row's loss
    may be infinite, or a mask's lowest value times it."""
    m, top, v = 600, 40, 40 if mask == "all listed" else 300
    rng = np.random.default_rng(int(at) + 300)
    ids = on_gpu(np.argsort(rng.random((m, v)), 1)[:, :top], torch.int64)
    t = on_gpu(at + 2 * rng.standard_normal((m, top)))
    z = torch.full((m, v), -INF if mask == "-inf" else torch.finfo(dtype).min, dtype=dtype, device="cuda")
    z.scatter_(1, ids, on_gpu(2 * rng.standard_normal((m, top)), dtype))
    c = dict(logits=z, ids=ids, teacher=t, teacher_lse=torch.logsumexp(t / T, 1), weight=on_gpu(rng.random(m) + 0.5), temperature=T)
    dl = torch.rand(m, device="cuda") + 0.1
    loss, probs, stats = fwd(c)
    got = bwd(c, dl, probs, stats).double()
    sums = probs.double().sum(1)
    assert bool((sums < 1).any()) and bool((sums > 1).any())
    want, _, k = definition(dict(c, logits=z.clamp_min(torch.finfo(dtype).min)), dl, no_rest=True)
    off = (loss.double() - want).abs()
    far = (z.double().clamp_min(-1e300) - z.double().amax(1, keepdim=True)).abs() / T
    q = k["log_q"].exp()
    tol = 2.0 ** -21 * (1 + torch.where(q > 0, q * far, 0.0).sum(1)) + 65 * U32
    tol = k["w"] * (k["p"].sum(1) * tol + 2.0 ** -21 * (k["part"].abs().sum(1) + k["p"].sum(1) * (1 + k["log_p"].abs().amax(1))))
    # (log p - log q as a difference of logits and one of the row's, each of at most 64 there)
    tol = tol + 4 * 64 * U32 * k["w"] * k["p"].sum(1) + 2 * U32 * want.abs()
    assert bool((off <= tol).all()), float((off / tol).max())
    p = torch.zeros_like(q).scatter_(1, ids, k["p"])
    dz = (dl.double() * k["w"] / T)[:, None] * (q * k["p"].sum(1, keepdim=True).clamp_min(1) - p)
    arg = 1 + k["log_p"].abs().amax(1, keepdim=True) + torch.where(q > 0, far, 0.0)
    t_off = (dl.double() * k["w"] / T)[:, None] * (2.0 ** -19 * (q + p) * arg + 70 * U32 * q)
    assert bool(((got - dz).abs() <= t_off + (2.0 ** -8 if dtype == BF else U32) * dz.abs()).all())


def test_a_mass_that_the_student_cannot_have_is_no_rounding():
    """r = 0.01, rho = 0: the definition's infinity; the gradient is that of the entries."""
    c = gapped(10, 1.0, F32, r=0.01)
    keep = torch.zeros_like(c["logits"], dtype=torch.bool).scatter_(1, c["ids"], True)
    c["logits"].masked_fill_(~keep, -INF)
    loss, probs, stats = fwd(c)
    dz = bwd(c, torch.ones(8, device="cuda"), probs, stats)
    assert bool((loss == INF).all()) and bool(dz.isfinite().all()) and not dz[~keep].any() and bool(dz[keep].any())
    c["teacher_lse"][:] = INF                      # the teacher lists nothing of its mass
    assert bool((fwd(c)[0] == INF).all())


# ------------------------------------------------------------- rows without a gradient
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v", [1000, 1003])
@pytest.mark.parametrize("bad", [float("nan"), INF])
def test_rows_of_weight_0_have_no_gradient_whatever_dloss_is(bad, v, dtype):
    """A mean over no rows, say, has a dloss that is not finite; a row of weight 0 is not read, one without entries has none."""
    from deterministic_arithmetic_gb300 import block8

    c = make(10, v, 8, dtype, tail=True)
    c["weight"][4] = 0
    c["logits"][4] = float("nan")
    c["ids"][6] = -1
    loss, probs, stats = fwd(c)
    dl = torch.ones(10, device="cuda")
    ok = bwd(c, dl, probs, stats)
    dl[4] = dl[6] = bad
    for block in (False, True):
        dz = bwd(c, dl, probs, stats, block8=block)
        dz = block8.unblock8(dz) if block else dz
        assert not dz[4].any() and not dz[6].any() and bool(dz.isfinite().all())
        assert block or same(dz, ok)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("r", [2e-6, 1e-5])
@pytest.mark.parametrize("gap", [50, 100, 2500])
def test_a_small_r_beside_a_rest_that_is_not_nothing_is_one(gap, r, dtype):
    """r of a few roundings is the definition's r as long as rho has a logarithm that the gradient knows."""
    for T in (0.25, 1.0):
        c = gapped(gap, T, dtype, r)
        c["teacher"] -= 20 * T
        c["teacher_lse"] -= 20
        _, _, k = check(c)
        # (teacher_lse and the logits near -20 are rounded to 2^-20 each: so far is the r that they give from the one wanted)
        assert bool(((k["r"] - r).abs() < 2.0 ** -18).all()) and bool((k["r"] > 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0.25, 1.0])
@pytest.mark.parametrize("gap", [20, 28, 36, 44, 52])
def test_elements_far_below_a_far_rest(gap, T, dtype):
    """Half of the rest lies 55 T below the other half: q_j is too small for a float, r rho_j is not."""
    c = gapped(gap, T, dtype)
    low = torch.ones_like(c["logits"], dtype=torch.bool).scatter_(1, c["ids"], False)
    low[:, ::2] = False
    c["logits"][low] -= 55 * T
    dl = torch.ones(8, device="cuda")
    loss, probs, stats = fwd(c)
    got = bwd(c, dl, probs, stats).double()
    want, dz, k = definition(c, dl)
    tol, t = off_by(c, dl, want, dz, k)
    # an exponential below 2^-126 is 0, times an r / rho of 2^32 at most (above, its logarithm is part of the exponent)
    flushed = (k["w"] / k["T"])[:, None] * 2.0 ** -94
    assert bool(((got - dz).abs() <= t + flushed + (2.0 ** -8 if dtype == BF else U32) * (dz.abs() + t)).all())
    assert gap < 36 or bool((got[low] < 0).all())
    assert bool(((loss.double() - want).abs() <= tol).all())


# --------------------------------------------------------- a teacher's own masks
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("teacher", [BF, F32])
@pytest.mark.parametrize("T", [0.1, 0.5, 1.0, 2.0])
def test_entries_of_the_teachers_lowest_value_have_probability_0(T, teacher, tail):
    """t / T may pass the type's range; the others' probabilities, the loss and the gradient are those of rows without them."""
    c = make(6, 900, 12, tail=tail, T=T, teacher=teacher)
    c["teacher"][:4, 8:] = torch.finfo(teacher).min
    c["teacher"][1, 3] = torch.finfo(teacher).min
    loss, probs, stats = fwd(c)
    dz = bwd(c, torch.ones(6, device="cuda"), probs, stats)
    gone = c["teacher"] == torch.finfo(teacher).min
    assert bool(loss.isfinite().all()) and bool((probs[gone] == 0).all()) and bool((probs[~gone] > 0).all())
    want = probs.double()
    if not tail:                                   # the same entries without them: p are the same to their roundings
        d = dict(c, teacher=c["teacher"].masked_fill(gone, -INF))
        l2, p2, _ = fwd(d)
        assert bool(((probs - p2.clamp_min(0)).abs() <= 2.0 ** -22 * want).all())
        assert bool(((loss - l2).abs() <= 2.0 ** -20 * l2.abs()).all())
    else:
        k = definition(c, torch.ones(6, device="cuda"))
        assert bool(((want - k[2]["p"]).abs() <= 2.0 ** -20 * k[2]["p"] * (1 + k[2]["log_p"].abs().clamp_max(1e30))).all())
        tol, t = off_by(c, torch.ones(6, device="cuda"), k[0], k[1], {**k[2], "log_p": k[2]["log_p"].clamp_min(-1e30)})
        assert bool(((loss.double() - k[0]).abs() <= tol).all())
        # (an exponential below 2^-126 is 0, times an r / rho of 2^32 at most and weight / T of at most 1.5 / 0.1 < 2^4)
        assert bool(((dz.double() - k[1]).abs() <= t + U32 * k[1].abs() + 2.0 ** -90).all())


# ----------------------------------------------------------------- digits of 1 - sum p
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v,top,T", [(1000, 256, 0.7), (1000, 256, 0.6), (2003, 200, 1 / 3 + 0.3), (3001, 256, 0.7), (700, 30, 0.5), (20000, 64, 1.0), (2000, 1024, 1.0), (5000, 100, 2.0)])
def test_a_small_mass_of_the_rest_has_its_digits(v, top, T, dtype):
    """r = 1 - sum p of 10^-3 to 10^-7, as a teacher leaves whose listed logits have nearly all its mass: r / rho is right to rho's own
    roundings, and to 2^-43 / rho (an entry's p to 2^-44 of itself or of 1)."""
    c = make(200, v, top, dtype, tail=True, T=T)
    _, _, stats = fwd(c)
    _, _, k = definition(c, torch.ones(200, device="cuda"))
    rho = torch.where(k["r"] > 0, k["log_rho"], 0.0).exp()
    off = (stats[:, 2].double() - (1 - k["r"] / rho)).abs()
    # rho: exponentials 2^-21, of arguments up to 64 right to 2^-24 of themselves, and the sums; then the stored value's rounding
    rel = 2.0 ** -21 + 64 * U32 + (v / 16384 + 64) * U32 + 2.0 ** -23
    bound = k["r"] / rho * rel + 2.0 ** -43 / rho + 2.0 ** -22
    assert bool((off <= bound).all())
    if top < 1000:                                 # entries given twice, the second time with another logit: the first counts
        twice = {key: torch.cat([c[key], c[key][:, :5] + more], 1) for key, more in (("ids", 0), ("teacher", 1.0))}
        _, probs, stats = fwd(dict(c, **twice))
        assert bool((probs[:, top:] == -1).all())
        assert bool(((stats[:, 2].double() - (1 - k["r"] / rho)).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("top", [1, 4, 64])
@pytest.mark.parametrize("T", [2.0, 4.0])
def test_a_small_divergence_has_its_digits(T, top, dtype):
    """A flat teacher and student over a long vocabulary: the listed entries have little of the mass, and the loss is what is left of
    terms that cancel. Each is right to 2^-20 of the listed mass: p and q of the entries to 2^-21, the logarithms to 2^-22."""
    c = make(60, 60000, top, dtype, tail=True, T=T)
    loss, _, _ = fwd(c)
    want, _, k = definition(c, torch.ones(60, device="cuda"))
    listed = k["p"].sum(1) + k["log_q"].gather(1, c["ids"]).exp().sum(1)
    assert bool(((loss.double() - want).abs() <= k["w"] * (2.0 ** -20 * listed * (1 + (k["log_p"] - k["log_q"].gather(1, c["ids"])).abs().amax(1)) + 2.0 ** -22 * want)).all())
