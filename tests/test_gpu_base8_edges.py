"""The calls at the edges of what include/lora_base8.h allows: sums that are exact, waits that run out, streams, offsets past
32 bits, masks of the type's lowest value, and what is refused."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from test_gpu_block8 import BF, F32, F8, _built, b8, operands, rnd, same  # noqa: E402,F401
from test_gpu_distill import bwd, check, fwd, make, ops  # noqa: E402

pytestmark = pytest.mark.gpu
# a CTA's tile of 32, 64, 128 and 256 columns; a pair's; a pair's, several tiles each
WAYS = [(100, 520, 4864), (100, 520, 9728), (100, 520, 19456), (100, 520, 38912), (2560, 1300, 2600), (5000, 264, 2600)]


@pytest.fixture(autouse=True)
def _no_wait_ran_out():
    yield
    from deterministic_arithmetic_gb300 import _capi

    assert _capi.device_status() == 0


def whole(m, k, tile, seed):
    """Whole numbers of up to +-6 at scales of whole numbers: every sum below 2^24 is exact in fp32."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.zeros(m, -(-k // 16) * 16, device="cuda")
    codes[:, :k] = torch.randint(-6, 7, (m, k), generator=g, device="cuda").float()
    scales = torch.randint(1, 4, (-(-m // tile), -(-k // 128)), generator=g, device="cuda").float()
    return b8().Block8(codes.to(F8), scales, k, tile), codes[:, :k].double() * scales.repeat_interleave(tile, 0)[:m].repeat_interleave(
        128, 1)[:, :k].double()


@pytest.mark.parametrize("joined", [False, True])
@pytest.mark.parametrize("m,k,n", WAYS + [(2049, 300, 2502)])
def test_whole_numbers_are_exact_and_the_passes_are_adjoint(m, k, n, joined):
    x, xv = whole(m, k, 1, 1)
    w, wv = whole(n, k, 128, 2)
    dy, dyv = whole(m, n, 1, 3)
    assert 36 * 9 * max(k, n) < 2 ** 24
    d = [torch.randint(-99, 99, s, device="cuda").float() if joined else None for s in ((m, n), (m, k))]
    y = b8().block8_linear_fwd(x, w, delta=d[0], dtype=F32).double()
    dx = b8().block8_linear_bwd(dy, w, delta=d[1], dtype=F32).double()
    assert torch.equal(y, xv @ wv.T + (d[0].double() if joined else 0))
    assert torch.equal(dx, dyv @ wv + (d[1].double() if joined else 0))
    if not joined:
        assert (dyv * y).sum() == (dx * xv).sum()


@pytest.mark.parametrize("joined", [False, True])
@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("m,red,cols", WAYS)
def test_a_wait_that_runs_out_is_reported(m, red, cols, back, joined):
    """The producer is made to wait for what never comes (1 ms limit): the kernel returns, the status block names the
    site, and after a reset the next call gives the same bits as before."""
    from deterministic_arithmetic_gb300 import _capi

    x, w = operands(m, *((cols, red) if back else (red, cols)), bwd=back)
    delta = rnd(m, cols, dtype=F32) if joined else None
    run = b8().block8_linear_bwd if back else b8().block8_linear_fwd
    ref = run(x, w, delta=delta)
    y = torch.empty_like(ref)
    try:
        _capi.device_status_reset(25 if back else 24, 1000)
        run(x, w, delta=delta, y=y) if not back else run(x, w, delta=delta, dx=y)
        assert _capi.device_status() == (97 << 8) | 1
    finally:
        _capi.device_status_reset()
    assert _capi.device_status() == 0
    assert same(run(x, w, delta=delta), ref)


def test_streams_and_two_calls_at_once():
    """The streams' calls run side by side, over and over: the same bits as alone."""
    c = make(300, 5000, 20, BF, tail=True)
    dl = torch.rand(300, device="cuda")
    x, w = operands(300, 700, 5000)

    def run(st=None):
        loss, probs, stats = fwd(c, stream=st)
        dz = bwd(c, dl, probs, stats, block8=True, stream=st)
        y = b8().block8_linear_fwd(x, w, stream=st)
        dx = b8().block8_linear_bwd(dz, w, stream=st)
        p = b8().block8(y, stream=st)
        return loss, probs, stats, dz.codes, dz.scales, y, dx, p.codes, b8().unblock8(p, stream=st)

    ref = run()
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [run(st if i % 2 else st.cuda_stream) for i in range(5) for st in streams]
    torch.cuda.synchronize()
    assert all(same(a, b) for g in got for a, b in zip(g, ref))


def test_captured_and_replayed():
    """One graph of the whole run, replayed with other inputs, gives what the calls give; two graphs replayed side by
    side share nothing."""
    def inputs(seed):
        c = make(70, 3000, 9, BF, seed=seed, tail=True)
        c["x"] = rnd(70, 520, seed=seed)
        return c

    w = b8().block8(rnd(3000, 520, c=0.05), tile=128)
    delta = rnd(70, 3000, dtype=F32)
    dl = torch.rand(70, device="cuda")

    def run(c):
        y = b8().block8_linear_fwd(b8().block8(c["x"]), w, delta=delta)
        d = dict(c, logits=y)
        loss, probs, stats = fwd(d)
        return loss, stats, b8().block8_linear_bwd(bwd(d, dl, probs, stats, block8=True), w), bwd(d, dl, probs, stats)

    a, b = inputs(1), inputs(2)
    graphs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for c in (a, b):
            run(c)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = run(c)
            graphs.append((g, out, c))
    torch.cuda.synchronize()
    for new in (inputs(3), inputs(4)):
        for g, _, c in graphs:
            for k in ("x", "ids", "teacher", "teacher_lse", "weight"):
                c[k].copy_(new[k])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graphs[0][0].replay()
        graphs[1][0].replay()
        torch.cuda.synchronize()
        want = run(new)
        assert all(same(x, y) for _, out, _ in graphs for x, y in zip(out, want))


def test_no_rows():
    p, w = b8().block8(torch.empty(0, 200, dtype=BF, device="cuda")), b8().block8(rnd(72, 200), tile=128)
    assert p.codes.shape == (0, 208) and p.scales.shape == (0, 2) and b8().unblock8(p).shape == (0, 200)
    assert b8().block8_linear_fwd(p, w).shape == (0, 72)
    dy = b8().block8(torch.empty(0, 72, device="cuda"))
    assert b8().block8_linear_bwd(dy, w, dtype=F32).shape == (0, 200)


@pytest.mark.parametrize("tile", [1, 128])
def test_blocks_past_32_bits(tile):
    m, k = 66048, 65536 + 8
    x = torch.full((m, k), 0.37, dtype=BF, device="cuda")
    x[-256:] = rnd(256, k)
    p = b8().block8(x, tile=tile)
    few = b8().block8(x[-256:].clone(), tile=tile)
    assert same(p.codes[-256:], few.codes) and same(p.scales[-256 // tile:], few.scales)
    tail = b8().unblock8(few)
    b8().unblock8(p, out=x)
    assert same(x[-256:], tail) and bool((x[:-256].view(-1)[::4099] == x[0, 0]).all())


@pytest.mark.parametrize("back", [False, True])
def test_products_past_32_bits(back):
    """Of the operands and of the output (with delta): the last rows are those of a call of their own."""
    run = b8().block8_linear_bwd if back else b8().block8_linear_fwd
    big, small = 66000, 65536 + 8
    one = torch.ones(big, small + 8, device="cuda").to(F8)        # (a row of codes is a multiple of 16)
    scales = torch.ones(big, -(-small // 128), device="cuda")
    one[-200:] = rnd(200, small + 8).to(F8)
    x = b8().Block8(one, scales, small, 1)
    _, w = operands(1, *((40, small) if back else (small, 40)))
    few = b8().Block8(one[-200:].clone(), scales[-200:].clone(), small, 1)
    assert same(run(x, w, dtype=F32)[-200:], run(few, w, dtype=F32))
    del one, x, few
    a = rnd(big, 40)
    x = b8().block8(a)
    _, w = operands(1, *((small, 40) if back else (40, small)))
    delta = torch.full((big, small), 0.5, device="cuda")
    delta[-200:] = rnd(200, small, dtype=F32)
    few = b8().block8(a[-200:].clone())
    assert same(run(x, w, delta=delta)[-200:], run(few, w, delta=delta[-200:].clone()))
    y = run(x, w, dtype=F32)
    assert same(y[-200:], run(few, w, dtype=F32))


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("T", [0.25, 1.0, 3.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_rows_of_the_lowest_value_and_logits_far_from_0(dtype, T, tail):
    """All logits the type's lowest (the student is uniform); lowest but for a few; all far up or down, where a product with
    1 / T has no digits behind the point."""
    c = make(6, 1500, 12, dtype, tail=tail, T=T)
    z = c["logits"]
    z[0] = torch.finfo(dtype).min
    z[1] = torch.finfo(dtype).min
    z[1, c["ids"][1]] = rnd(12, dtype=dtype)
    z[1, 700:1400] = rnd(700, dtype=dtype)
    z[2] = 2.0 ** 20
    z[3] = -(2.0 ** 24)
    z[4] = torch.finfo(dtype).max
    if dtype == F32:
        z[5] += 300000.0
    check(c)


def test_refusals():
    from deterministic_arithmetic_gb300 import lora_delta as ld

    x, w = operands(40, 200, 300)
    dy = b8().block8(rnd(40, 300))
    t = rnd(40, 200)
    B = b8().Block8
    for bad in (lambda: b8().block8(t.half()), lambda: b8().block8(t[:, ::2]), lambda: b8().block8(t[0]), lambda: b8().block8(t, tile=64),
                lambda: b8().block8(t, out=B(x.codes, x.scales, 100, 1)),
                lambda: b8().block8(t, out=B(x.codes[:20], x.scales, 200, 1)),
                lambda: b8().block8(t, out=B(x.codes, w.scales, 200, 1)),
                lambda: b8().unblock8(x, out=torch.empty(40, 200, device="cuda")),
                lambda: b8().unblock8(B(x.codes, x.scales, 200, 128)),
                lambda: b8().unblock8(B(x.codes, x.scales.double(), 200, 1)),
                lambda: b8().unblock8(B(x.codes, x.scales, 100, 1)),
                lambda: b8().unblock8(B(x.codes.float(), x.scales, 200, 1)),
                lambda: b8().unblock8(B(x.codes, x.scales.cpu(), 200, 1)),
                lambda: b8().block8_linear_fwd(w, x), lambda: b8().block8_linear_fwd(dy, w),
                lambda: b8().block8_linear_bwd(x, w), lambda: b8().block8_linear_fwd(x, w, delta=t),
                lambda: b8().block8_linear_fwd(x, w, delta=rnd(40, 300)),
                lambda: b8().block8_linear_fwd(x, w, y=torch.empty(40, 300, device="cuda")),
                lambda: b8().block8_linear_fwd(x, w, y=torch.empty(39, 300, dtype=BF, device="cuda")),
                lambda: b8().block8_linear_fwd(x, w, dtype=torch.float16)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ld.LoraDeltaError, match="LORA_ERR_ALIGN"):
        b8().block8(rnd(40 * 200 + 1)[1:].view(40, 200))
    for bad in (lambda: b8().unblock8(t), lambda: b8().block8_linear_fwd(x, t), lambda: b8().block8(None)):
        with pytest.raises(TypeError):
            bad()
    c = make(6, 300, 5)
    loss, probs, stats = fwd(c)
    f, z, i, te, d = ops().distill_topk_fwd, c["logits"], c["ids"], c["teacher"], torch.ones(6, device="cuda")
    g = ops().distill_topk_bwd
    for bad in (lambda: f(z.half(), i, te), lambda: f(z, i.short(), te), lambda: f(z, i, te.double()),
                lambda: f(z, i[:, :4], te), lambda: f(z, i[:5], te[:5]), lambda: f(z, i, te, weight=d[:5]),
                lambda: f(z, i, te, teacher_lse=d.double()), lambda: f(z[:, ::2], i, te), lambda: f(z, i.cpu(), te),
                lambda: f(z, i, te, loss=torch.empty(5, device="cuda")), lambda: f(z, i, te, stats=torch.empty(6, 3, device="cuda")),
                lambda: g(d[:5], z, i, probs, stats), lambda: g(d, z, i, probs[:, :4].contiguous(), stats),
                lambda: g(d, z, i, probs, stats[:, :3].contiguous()), lambda: g(d, z, i, probs, stats, dlogits=z.to(BF)),
                lambda: g(d.double(), z, i, probs, stats)):
        with pytest.raises(ValueError):
            bad()
    for T in (0.0, -1.0, float("nan"), float("inf"), 1e-40):
        with pytest.raises(ld.LoraDeltaError, match="LORA_ERR_SHAPE"):
            f(z, i, te, temperature=T)
        with pytest.raises(ld.LoraDeltaError, match="LORA_ERR_SHAPE"):
            g(d, z, i, probs, stats, temperature=T)
    many = torch.zeros(6, 1025, dtype=torch.int64, device="cuda")
    with pytest.raises(ld.LoraDeltaError, match="LORA_ERR_SHAPE"):
        f(z, many, torch.zeros(6, 1025, device="cuda"))
    for bad in (lambda: g(d, z, i, probs, stats, block8=True, dlogits=z), lambda: g(d, z, i, probs, stats, dlogits=x)):
        with pytest.raises((TypeError, ValueError)):
            bad()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v", [1, 2, 3, 5, 7, 9])
def test_what_lies_behind_the_last_row_has_no_part(v, dtype):
    """Rows shorter than a vector, the last of them in one with what is not the tensor's."""
    for m in (1, 2, 5, 13):
        c = make(m, v, 2, dtype, tail=v > 2)
        room = torch.full((m * v + 16,), float("nan"), dtype=dtype, device="cuda")
        room[:m * v] = c["logits"].flatten()
        c["logits"] = room[:m * v].view(m, v)
        check(c)
        _, probs, stats = fwd(c)
        bwd(c, torch.ones(m, device="cuda"), probs, stats, dlogits=c["logits"])
        assert bool(room[:m * v].isfinite().all()) and bool(room[m * v:].isnan().all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("v", [24576, 24577, 32000, 114688, 115001, 131072])
def test_long_rows(v, dtype):
    """Rows of one, two and four places: a row alone, in a few and in many."""
    c = make(400, v, 30, dtype, tail=True)
    loss, probs, stats = fwd(c)
    dl = torch.rand(400, device="cuda")
    dz = bwd(c, dl, probs, stats)
    for rows in (slice(3, 4), slice(5, 30), slice(60, 260)):
        d = {k: (x[rows].clone() if isinstance(x, torch.Tensor) else x) for k, x in c.items()}
        got = fwd(d)
        assert all(same(a, b[rows]) for a, b in zip(got, (loss, probs, stats)))
        assert same(bwd(d, dl[rows].clone(), got[1], got[2]), dz[rows])
    check({k: (x[5:8].clone() if isinstance(x, torch.Tensor) else x) for k, x in c.items()})


def test_outputs_of_one_call_are_tensors_of_their_own():
    """Small outputs may lie in one allocation: each can be written, kept, saved and viewed alone, and outlives the others."""
    import io

    x = rnd(5, 300)
    p = b8().block8(x)
    want = b8().unblock8(p)
    q = b8().Block8(p.codes, p.scales.clone(), p.cols, p.tile)
    p.scales.zero_()
    assert same(b8().unblock8(q), want) and repr(p).startswith("Block8(codes=") and p == p
    assert p.codes.is_contiguous() and p.scales.is_contiguous() and p.codes.data_ptr() % 16 == p.scales.data_ptr() % 16 == 0
    c = make(7, 130, 5)
    loss, probs, stats = fwd(c)
    ref = [t.clone() for t in (loss, probs, stats)]
    f = io.BytesIO()
    torch.save(probs, f)
    f.seek(0)
    assert torch.equal(torch.load(f), ref[1])
    loss.fill_(3.0)
    assert torch.equal(probs, ref[1]) and torch.equal(stats, ref[2])
    del probs, loss
    torch.cuda.synchronize()
    junk = [torch.full((7, 5), 9.0, device="cuda") for _ in range(20)]
    assert torch.equal(stats, ref[2]) and len(junk) == 20
    stats.requires_grad_()
    assert (stats * 2).sum().requires_grad


@pytest.mark.parametrize("m,k,n,back", [(2, (1 << 22) - 1, 8, False), (3, 24, (1 << 22) - 1, True), (2, 40, (1 << 22) - 1, False),
                                        (1, (1 << 22) - 1, 40, True), ((1 << 22) - 1, 24, 16, False)])
def test_products_of_the_largest_sizes(m, k, n, back):
    from test_gpu_block8 import check_product

    x, w = operands(m, k, n, back)
    y = check_product(x, w, back)
    assert bool(y.isfinite().all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_the_longest_rows_and_most_entries(dtype):
    m, v = 320, (1 << 22) - 1
    g = torch.Generator(device="cuda").manual_seed(5)
    z = torch.empty(m, v, dtype=dtype, device="cuda").normal_(generator=g)
    ids = torch.randint(0, v, (m, 1024), generator=g, device="cuda")
    t = torch.randn(m, 1024, generator=g, device="cuda")
    c = dict(logits=z, ids=ids, teacher=t, teacher_lse=torch.logsumexp(t, 1) + 0.5, weight=None, temperature=1.0)
    loss, probs, stats = fwd(c)
    few = {k: (x[-2:].clone() if isinstance(x, torch.Tensor) else x) for k, x in c.items()}
    got = check(few)
    assert all(same(a, b[-2:]) for a, b in zip(got[:3], (loss, probs, stats)))
    dl = torch.rand(m, device="cuda")
    dz = bwd(few, dl[-2:].clone(), *got[1:3])
    bwd(c, dl, probs, stats, dlogits=z)
    assert same(z[-2:], dz)
