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
