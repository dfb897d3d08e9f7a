"""Products with 8-bit weights in tiles of 96 columns: an accumulator of 128 whose last 32 nobody reads, and tiles that touch
one or two blocks of scales in turn."""
import pytest

torch = pytest.importorskip("torch")

from base8_plan import plan  # noqa: E402
from test_gpu_base8_edges import whole  # noqa: E402
from test_gpu_block8 import F32, _built, _no_wait_ran_out, b8, check_product, operands, rnd, same  # noqa: E402,F401

pytestmark = pytest.mark.gpu
# one row to a tile's, whole tiles and pieces, columns that vectors fit and that they do not, one k-block to twelve
SHAPES = [(1, 1300, 9760), (7, 100, 12001), (33, 264, 11003), (100, 520, 11008), (128, 1536, 14592), (128, 129, 9794)]


def _takes_96(m, n):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return plan(False, m, n, sms, sms // 2)[1] == 96


@pytest.mark.parametrize("joined", [False, True])
@pytest.mark.parametrize("m,k,n", SHAPES)
def test_against_64_bits(m, k, n, joined):
    assert _takes_96(m, n)
    x, w = operands(m, k, n)
    check_product(x, w, False, rnd(m, n, dtype=F32) if joined else None)


@pytest.mark.parametrize("joined", [False, True])
@pytest.mark.parametrize("m,k,n", SHAPES)
def test_whole_numbers_are_exact(m, k, n, joined):
    assert _takes_96(m, n) and 36 * 9 * k < 2 ** 24
    x, xv = whole(m, k, 1, 1)
    w, wv = whole(n, k, 128, 2)
    d = torch.randint(-99, 99, (m, n), device="cuda").float() if joined else None
    assert torch.equal(b8().block8_linear_fwd(x, w, delta=d, dtype=F32).double(), xv @ wv.T + (d.double() if joined else 0))


@pytest.mark.parametrize("n", [9760, 11003])
def test_rows_are_the_same_bits_as_in_other_tiles(n):
    """In tiles of 96, of 128 and 256 and of pairs; what lies behind the last row stays."""
    x, w = operands(700, 1300, n)
    y = b8().block8_linear_fwd(x, w, dtype=F32)
    for rows in (slice(0, 1), slice(100, 228), slice(300, 600), slice(690, 700)):
        part = b8().Block8(x.codes[rows].clone(), x.scales[rows].clone(), x.cols, 1)
        m = rows.stop - rows.start
        assert (m > 128) != _takes_96(m, n)
        out = torch.full((m + 3, n), 7.0, device="cuda")
        b8().block8_linear_fwd(part, w, dtype=F32, y=out[:m])
        assert same(out[:m], y[rows]) and bool((out[m:] == 7).all())


@pytest.mark.parametrize("joined", [False, True])
def test_a_wait_that_runs_out_is_reported(joined):
    from deterministic_arithmetic_gb300 import _capi

    m, k, n = 100, 520, 11008
    x, w = operands(m, k, n)
    delta = rnd(m, n, dtype=F32) if joined else None
    ref = b8().block8_linear_fwd(x, w, delta=delta)
    try:
        _capi.device_status_reset(24, 1000)
        b8().block8_linear_fwd(x, w, delta=delta, y=torch.empty_like(ref))
        assert _capi.device_status() == (97 << 8) | 1
    finally:
        _capi.device_status_reset()
    assert same(b8().block8_linear_fwd(x, w, delta=delta), ref)
