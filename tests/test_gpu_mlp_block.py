"""The operators together, as examples/mlp_block_step.py runs them, against 64-bit automatic differentiation.

What is kept in 8 bits is off by up to half a step, a step at most 2 / 127.5 of its group's largest value:
for normal values (largest of 32 about 2.2 times their size, steps of 1 / 127.5 to 2 / 127.5 of it) about
0.8 % of a value's size, independent from value to value; the bf16 roundings of n, dgate, dup, dn, U and dU add
0.2 % each. Gradients are sums of many such terms: relative errors of the norms stay near 1 %, and are held
to 3 %. h has no 8-bit value in it: bf16 roundings of n (inside the norm's error) and h, held to 1 %."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_arithmetic_gb300 import build_lib

    build_lib.build()


def reference(p, x, dh):
    d = {k: v.double().requires_grad_() for k, v in vars(p).items() if isinstance(v, torch.Tensor)}
    x = x.double().requires_grad_()
    n = torch.nn.functional.layer_norm(x, (x.shape[1],), d["ln_weight"], d["ln_bias"], 1e-5)
    g = n @ d["w_gate"].t() + p.alpha * (n @ d["a_gate"].t()) @ d["b_gate"].t()
    u = n @ d["w_up"].t() + p.alpha * (n @ d["a_up"].t()) @ d["b_up"].t()
    h = torch.nn.functional.silu(g) * u
    h.backward(dh.double())
    return h.detach(), x.grad, {k: v.grad for k, v in d.items()}


@pytest.mark.parametrize("tokens,width,hidden,rank", [(200, 136, 264, 16), (513, 256, 520, 8), (300, 520, 1000, 32)])
def test_step_against_autograd(tokens, width, hidden, rank):
    import mlp_block_step as ex

    p, x, dh = ex.make(tokens, width, hidden, rank, seed=tokens)
    h, kept = ex.forward(p, x)
    dx, grads = ex.backward(p, dh, kept)
    rh, rdx, rg = reference(p, x, dh)

    def off(a, b):
        return float((a.double() - b).norm() / b.norm())

    assert off(h, rh) < 0.01
    assert off(dx, rdx) < 0.03
    for k, g in grads.items():
        assert off(g, rg[k]) < 0.03, (k, off(g, rg[k]))


def test_step_is_batch_invariant_and_repeats():
    import mlp_block_step as ex

    p, x, dh = ex.make(700, 256, 520, 16)
    h, kept = ex.forward(p, x)
    dx, grads = ex.backward(p, dh, kept)
    for lo, hi in ((0, 1), (100, 333), (699, 700)):
        h2, kept2 = ex.forward(p, x[lo:hi].clone())
        dx2, _ = ex.backward(p, dh[lo:hi].clone(), kept2)
        assert torch.equal(h[lo:hi], h2) and torch.equal(dx[lo:hi], dx2)
    h3, kept3 = ex.forward(p, x)
    dx3, grads3 = ex.backward(p, dh, kept3)
    assert torch.equal(h, h3) and torch.equal(dx, dx3) and all(torch.equal(grads[k], grads3[k]) for k in grads)


def test_step_in_a_graph():
    """The whole step captured and replayed: no operator synchronises or allocates outside torch's pool."""
    import mlp_block_step as ex

    p, x, dh = ex.make(300, 256, 520, 16)
    h, kept = ex.forward(p, x)
    dx, grads = ex.backward(p, dh, kept)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        h2, kept2 = ex.forward(p, x)
        dx2, grads2 = ex.backward(p, dh, kept2)
    for t in (h2, dx2, *grads2.values()):
        t.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, h2) and torch.equal(dx, dx2) and all(torch.equal(grads[k], grads2[k]) for k in grads)
