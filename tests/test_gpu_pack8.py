"""Activation checkpoints in 8 bits on the GPU: codes and scales equal to the 64-bit form's, unpacked
values exact, and backward passes from a checkpoint bit for bit those of the unpacked tensor."""
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


def data(M, K, dt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(M, K, generator=g, device="cuda") * torch.exp(2 * torch.randn(M, 1, generator=g, device="cuda"))
    return x.to(DT[dt])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 5), (2, 31), (4, 32), (1, 33), (7, 40), (5, 64), (6, 100), (3, 1000),
                                 (40, 257), (2, 4096)])
def test_codes_scales_and_values(M, K, dt):
    from deterministic_arithmetic_gb300 import pack8

    x = data(M, K, dt, K)
    p = pack8.pack8(x)
    codes, scales = R.pack8(R.f64(x))
    assert np.array_equal(p.codes.cpu().numpy(), codes) and np.array_equal(p.scales.cpu().numpy(), scales)
    ref = R.unpack8(codes, scales, K)
    for out in (torch.bfloat16, torch.float32):
        v = pack8.unpack8(p, dtype=out)
        assert v.dtype == out and np.array_equal(R.f64(v), ref)
    again = pack8.pack8(pack8.unpack8(p))          # the values pack to themselves (to a finer step at most)
    assert np.array_equal(R.f64(pack8.unpack8(again)), ref)
    # half a step of the group, a step being at most 2 / 127.5 of its largest magnitude
    pad = np.pad(np.abs(R.f64(x)), ((0, 0), (0, -K % 32))).reshape(M, -1, 32).max(2)
    assert (np.abs(ref - R.f64(x)) <= np.repeat(pad, 32, 1)[:, :K] / 127.5).all()


def edge_rows():
    """Rows of 32: ties, the step's edge at 127.5, subnormals, the largest numbers, zeros, NaN, infinity."""
    rows = []

    def row(*v):
        rows.append(list(v) + [0.0] * (32 - len(v)))

    row()
    row(127.0, 0.5, 1.5, 2.5, -0.5, -1.5)
    row(127.5, 126.5, -127.5, 0.5)
    row(float(np.nextafter(np.float32(127.5), np.float32(200))), 1.0, 2.0, 3.0, -3.0)
    row(2.0 ** -126, 2.0 ** -130, -2.0 ** -133)
    row(2.0 ** -149, -2.0 ** -140)
    row(2.0 ** -127, 3 * 2.0 ** -127, 2.0 ** -128, -1.5 * 2.0 ** -127)
    row(3.3895314e38, -1e38, 1.0)
    row(3.4028235e38, 2e38)
    row(2.0 ** -120, 2.0 ** -121, 127 * 2.0 ** -127, 127.5 * 2.0 ** -127)
    row(float("nan"), 1.0)
    row(1.0, float("inf"))
    row(float("-inf"), float("nan"), 2.0)
    row(-1.0)
    return torch.tensor(rows, dtype=torch.float32)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_edges(dt):
    from deterministic_arithmetic_gb300 import pack8

    x = edge_rows().to(DT[dt])
    for cols in (32, 31):                       # the vector kernel and the one for any width
        xs = x[:, :cols].contiguous().cuda()
        p = pack8.pack8(xs)
        codes, scales = R.pack8(R.f64(xs))
        assert np.array_equal(p.scales.cpu().numpy(), scales) and np.array_equal(p.codes.cpu().numpy(), codes)
        for out in (torch.bfloat16, torch.float32):
            assert np.array_equal(R.f64(pack8.unpack8(p, dtype=out)), R.unpack8(codes, scales, cols), equal_nan=True)


def lora(M, K, N, r, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rnd(*s, c=1.0):
        return (torch.randn(*s, generator=g, device="cuda") * c).to(torch.bfloat16)

    return dict(x=rnd(M, K), a=rnd(r, K, c=K ** -0.5), b=rnd(N, r, c=r ** -0.5), dy=rnd(M, N, c=0.1), u=rnd(M, r),
                du=rnd(M, r, c=0.1))


@pytest.mark.parametrize("M,K,N,r", [(1, 8, 8, 8), (64, 128, 96, 8), (255, 264, 136, 16), (256, 40, 512, 16),
                                     (257, 1000, 72, 24), (700, 520, 264, 32), (130, 72, 1024, 40), (513, 4104, 64, 64),
                                     (3000, 256, 128, 16)])
def test_backward_from_a_checkpoint(M, K, N, r):
    """dA, and the whole backward of the delta, against the unpacked x: the same bits."""
    from deterministic_arithmetic_gb300 import _capi, lora_delta as ld, pack8

    t = lora(M, K, N, r, M + K)
    p = pack8.pack8(t["x"])
    x = pack8.unpack8(p)
    ref = ld.lora_delta_bwd(t["dy"], x, t["a"], t["b"], t["u"], 2.0)
    got = pack8.lora_delta_bwd_packed8(t["dy"], p, t["a"], t["b"], t["u"], 2.0)
    for name, a, b in zip(("dx", "da", "db", "du"), got, ref):
        assert torch.equal(a, b), name
    da = pack8.pack8_da(ref[3], p)
    assert torch.equal(da, ref[1])
    # and against 64 bits, at the contract's 1e-6 of the sum of magnitudes
    DU, X = R.f64(t["du"]), R.f64(x)
    got = R.f64(pack8.pack8_da(t["du"], p))
    assert (np.abs(got - DU.T @ X) <= 1e-6 * (np.abs(DU).T @ np.abs(X))).all()
    assert torch.equal(pack8.pack8_da(t["du"], p), pack8.pack8_da(t["du"], p))
    assert _capi.device_status() == 0


def test_da_of_extreme_steps():
    """Groups whose steps lie at both ends of the range, and zeros, through dA: the same bits as unpacked."""
    from deterministic_arithmetic_gb300 import lora_delta as ld, pack8

    M, K, r = 128, 256, 16
    t = lora(M, K, 64, r)
    x = t["x"].float()
    for j, e in enumerate((-126, -120, -100, -60, 0, 60, 90, 0)):
        x[:, 32 * j:32 * j + 32] *= 2.0 ** e
    x[:, 224:] = 0
    p = pack8.pack8(x.to(torch.bfloat16))
    ref = ld.lora_delta_bwd(t["dy"], pack8.unpack8(p), t["a"], t["b"], t["u"], 1.0)
    assert torch.equal(pack8.pack8_da(ref[3], p), ref[1])


def test_empty_and_nan_groups_in_da():
    from deterministic_arithmetic_gb300 import pack8

    e = pack8.pack8(torch.empty(0, 64, device="cuda"))
    assert e.codes.shape == (0, 64) and pack8.unpack8(e).shape == (0, 64)
    assert not pack8.pack8_da(torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), e).any()
    t = lora(64, 128, 64, 16)
    x = t["x"].clone()
    x[5, 40] = float("nan")
    da = pack8.pack8_da(t["du"], pack8.pack8(x))
    assert da[:, 32:64].isnan().all() and not da[:, :32].isnan().any() and not da[:, 64:].isnan().any()


def test_streams_and_refusals():
    from deterministic_arithmetic_gb300 import lora_delta as ld, pack8

    t = lora(300, 520, 64, 16)
    p = pack8.pack8(t["x"])
    ref = pack8.pack8_da(t["du"], p)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    q = pack8.pack8(t["x"], stream=s)
    got = pack8.pack8_da(t["du"], q, stream=s)
    v = pack8.unpack8(q, stream=s)
    s.synchronize()
    assert torch.equal(got, ref) and torch.equal(v, pack8.unpack8(p))
    for bad in (lambda: pack8.pack8(t["x"].half()), lambda: pack8.pack8(t["x"].t()), lambda: pack8.pack8(t["x"].cpu()),
                lambda: pack8.unpack8(pack8.Packed8(p.codes, p.scales, 512)),
                lambda: pack8.unpack8(pack8.Packed8(p.codes[:, :512], p.scales, 520)),
                lambda: pack8.unpack8(p, dtype=torch.float16),
                lambda: pack8.pack8_da(t["du"][:64].contiguous(), p), lambda: pack8.pack8_da(t["du"].float(), p)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        pack8.unpack8(t["x"])
    with pytest.raises(ld.LoraDeltaError, match="LORA_ERR_RANK"):
        pack8.pack8_da(t["du"][:, :12].contiguous(), p)
    with pytest.raises(ld.LoraDeltaError, match="LORA_ERR_SHAPE"):
        pack8.pack8_da(t["du"], pack8.pack8(t["x"][:, :100].contiguous()))
    with pytest.raises(ld.LoraDeltaError, match="LORA_ERR_WORKSPACE"):
        pack8.pack8_da(t["du"], p, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("M", [200, 1000])
def test_a_wait_that_runs_out_is_reported(M):
    """The copying warp of dA's kernel is made to wait for what never comes (1 ms limit): the kernel returns, the
    status block names the site, and after a reset the next call gives the same bits as before."""
    from deterministic_arithmetic_gb300 import _capi, pack8

    t = lora(M, 264, 72, 16, M)
    p = pack8.pack8(t["x"])
    ref = pack8.pack8_da(t["du"], p)
    try:
        _capi.device_status_reset(13, 1000)
        pack8.pack8_da(t["du"], p)
        assert _capi.device_status() == (56 << 8) | 1
    finally:
        _capi.device_status_reset()
    assert _capi.device_status() == 0
    assert torch.equal(ref, pack8.pack8_da(t["du"], p))
