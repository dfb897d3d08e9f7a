"""Edges of the MLP-block operators on the GPU: batches of no rows, kernels whose CTAs take several units of
work, streams and devices, status, against 64-bit forms or the unpacked tensor's bits."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import mlp_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_arithmetic_gb300 import build_lib

    build_lib.build()


def rnd(*shape, c=1.0, dtype=torch.bfloat16, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + sum(shape))
    return (torch.randn(*shape, generator=g, device="cuda") * c).to(dtype)


@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("r", [8, 40])
def test_packed_backward_of_no_rows_gives_zero_gradients(r, given):
    """da and db are sums over no rows: zeros, whatever the outputs held before."""
    from deterministic_arithmetic_gb300 import pack8

    K, N = 200, 136
    bf = dict(dtype=torch.bfloat16, device="cuda")
    p = pack8.pack8(torch.empty(0, K, **bf))
    nan = {k: torch.full(s, float("nan"), device="cuda") for k, s in (("da", (r, K)), ("db", (N, r)))}
    trash = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]       # what new outputs may get
    del trash
    dx, da, db, du = pack8.lora_delta_bwd_packed8(torch.empty(0, N, **bf), p, rnd(r, K), rnd(N, r),
                                                  torch.empty(0, r, **bf), 2.0, **(nan if given else {}))
    assert dx.shape == (0, K) and du.shape == (0, r)
    assert torch.equal(da, torch.zeros(r, K, device="cuda")) and torch.equal(db, torch.zeros(N, r, device="cuda"))
    if given:
        assert da.data_ptr() == nan["da"].data_ptr() and db.data_ptr() == nan["db"].data_ptr()


def test_status_calls_wait_for_every_stream():
    """A wait that runs out (1 ms) in a call queued on another stream behind 50 ms of idling: the status call comes
    back with its code, and a reset behind such a call leaves nothing of it."""
    from deterministic_arithmetic_gb300 import _capi, pack8

    du, p = rnd(200, 16), pack8.pack8(rnd(200, 264))
    s = torch.cuda.Stream()

    def stalled_call():
        _capi.device_status_reset(13, 1000)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            torch.cuda._sleep(100_000_000)                # cycles, at up to 2.1 GHz
            pack8.pack8_da(du, p)

    try:
        stalled_call()
        assert _capi.device_status() == (56 << 8) | 1
        stalled_call()
    finally:
        _capi.device_status_reset()
    torch.cuda.synchronize()
    assert _capi.device_status() == 0


def test_workspace_status_waits_for_every_stream():
    """The same of the status block of a workspace, which the packed backward's kernels report to."""
    from deterministic_arithmetic_gb300 import lora_delta as ld, pack8

    M, K, N, r = 200, 264, 136, 16
    ws = ld.new_workspace(pack8.lora_delta_bwd_packed8_workspace_size(M, K, N, r), "cuda")
    ws[:16].view(torch.int32).copy_(torch.tensor([0, 0, 13, 1000]))       # dA's copying warp stalls; 1 ms
    args = rnd(M, N), pack8.pack8(rnd(M, K)), rnd(r, K), rnd(N, r), rnd(M, r), 2.0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        torch.cuda._sleep(100_000_000)
        pack8.lora_delta_bwd_packed8(*args, workspace=ws)
    assert ld.lora_delta_device_status(ws) == (56 << 8) | 1


def test_the_readme_step_is_the_examples_step():
    """README.md's lines, run as they stand: the output and every gradient of examples/mlp_block_step.py."""
    import os
    import re
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    sys.path.insert(0, os.path.join(root, "examples"))
    import mlp_block_step as ex

    from deterministic_arithmetic_gb300 import lora_delta as ld

    text = open(os.path.join(root, "README.md"), encoding="utf-8").read()
    step, = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "gated_ffn_bwd" in b]
    p, x, dh = ex.make(300, 256, 520, 16)
    names = dict(torch=torch, ld=ld, x=x, dh=dh, weight=p.ln_weight, bias=p.ln_bias, w_gate=p.w_gate, w_up=p.w_up,
                 a_g=p.a_gate, b_g=p.b_gate, a_u=p.a_up, b_u=p.b_up, alpha=p.alpha)
    exec(step, names)
    h, kept = ex.forward(p, x)
    dx, grads = ex.backward(p, dh, kept)
    mine = dict(ln_weight="dw", ln_bias="db", a_gate="da_g", b_gate="db_g", a_up="da_u", b_up="db_u")
    assert torch.equal(names["h"], h) and torch.equal(names["dx"], dx)
    assert all(torch.equal(names[mine[k]], grads[k]) for k in grads)
