"""The operators together, as examples/distill_step.py runs them, against 64-bit automatic differentiation of the same
function: the values that the 8-bit forms of x and n stand for go into the products, and the gradient passes them by.

What is left to differ. An e4m3 code is off by up to 2^-4 of its value, evenly spread: 2^-4 / sqrt(3), 3.6 %, at most on the
quadratic mean, independent from value to value; gradients are sums of many such terms, and their norms are off by as much.
The gradient by the logits is rounded so, once, and by it all gradients: held to 6 %; dx has dh's rounding too, 5.1 %
together: held to 8 %. The loss has bf16 roundings of h, n (beside its 8-bit form) and the logits only: of the logits, of
size 1, 2^-8 each and independent; the loss, a mean of them over the teacher's distribution, is held to 1 %."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
SIZES = [(200, 136, 1000, 16), (40, 256, 5003, 8), (300, 520, 2056, 32)]


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from deterministic_arithmetic_gb300 import build_lib

    build_lib.build()


def step(p, x, t, dloss):
    import distill_step as ex

    loss, kept = ex.forward(p, x, t)
    dx, grads = ex.backward(p, t, dloss, kept)
    return loss, dx, grads


def reference(p, x, t, dloss):
    from deterministic_arithmetic_gb300 import block8, layer_norm, lora_delta

    def value(b):
        return block8.unblock8(b, dtype=torch.float32).double()

    delta, _ = lora_delta.lora_delta_fwd(x, p.a, p.b, p.alpha)
    h = block8.block8_linear_fwd(block8.block8(x), p.w, delta=delta)
    n8 = value(block8.block8(layer_norm.layer_norm_fwd(h, p.ln_weight, p.ln_bias)[0]))
    d = {k: getattr(p, k).double().requires_grad_() for k in ("ln_weight", "ln_bias", "a", "b")}
    xd = x.double().requires_grad_()
    xq = xd + (value(block8.block8(x)) - xd).detach()
    hd = xq @ value(p.w).t() + p.alpha * (xd @ d["a"].t()) @ d["b"].t()
    n = torch.nn.functional.layer_norm(hd, (x.shape[1],), d["ln_weight"], d["ln_bias"], 1e-5)
    logits = (n + (n8 - n).detach()) @ value(p.head).t()
    log_q = torch.log_softmax(logits / p.temperature, 1)
    log_p = t.logits.double() / p.temperature - t.lse.double()[:, None]
    rest = 1 - log_p.exp().sum(1)
    others = log_q.exp().scatter(1, t.ids, 0.0).sum(1)
    loss = t.weight * ((log_p.exp() * (log_p - log_q.gather(1, t.ids))).sum(1) + rest * (rest.log() - others.log()))
    loss.backward(dloss.double())
    return loss.detach(), xd.grad, {k: v.grad for k, v in d.items()}


@pytest.mark.parametrize("tokens,width,vocabulary,rank", SIZES)
def test_step_against_autograd(tokens, width, vocabulary, rank):
    import distill_step as ex

    p, x, t = ex.make(tokens, width, vocabulary, rank, seed=tokens)
    dloss = torch.rand(tokens, device="cuda") + 0.5
    loss, dx, grads = step(p, x, t, dloss)
    rl, rdx, rg = reference(p, x, t, dloss)

    def off(a, b):
        return float((a.double() - b).norm() / b.norm())

    assert off(loss, rl) < 0.01 and not loss[7::8].any() and not dx[7::8].any()
    assert off(dx, rdx) < 0.08, off(dx, rdx)
    for k, g in grads.items():
        assert off(g, rg[k]) < 0.06, (k, off(g, rg[k]))


def test_step_is_batch_invariant_and_repeats():
    import distill_step as ex

    p, x, t = ex.make(700, 256, 3000, 16)
    dloss = torch.rand(700, device="cuda")
    loss, dx, grads = step(p, x, t, dloss)
    for lo, hi in ((0, 1), (100, 333), (692, 700)):
        part = ex.Teacher(*(v[lo:hi].clone() for v in vars(t).values()))
        l2, dx2, _ = step(p, x[lo:hi].clone(), part, dloss[lo:hi].clone())
        assert torch.equal(loss[lo:hi], l2) and torch.equal(dx[lo:hi], dx2)
    l3, dx3, grads3 = step(p, x, t, dloss)
    assert torch.equal(loss, l3) and torch.equal(dx, dx3) and all(torch.equal(grads[k], grads3[k]) for k in grads)


def test_step_in_a_graph():
    """The whole step captured and replayed: no operator synchronises or allocates outside torch's pool."""
    import distill_step as ex

    p, x, t = ex.make(300, 256, 3000, 16)
    dloss = torch.rand(300, device="cuda")
    loss, dx, grads = step(p, x, t, dloss)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        l2, dx2, grads2 = step(p, x, t, dloss)
    for v in (l2, dx2, *grads2.values()):
        v.zero_()
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    assert torch.equal(loss, l2) and torch.equal(dx, dx2) and all(torch.equal(grads[k], grads2[k]) for k in grads)


def test_the_readme_step_is_the_examples_step():
    """README.md's lines, run as they stand."""
    import re

    import distill_step as ex

    from deterministic_arithmetic_gb300 import layer_norm, lora_delta as ld

    text = open(os.path.join(ROOT, "README.md"), encoding="utf-8").read()
    lines, = [b for b in re.findall(r"```python\n(.*?)```", text, flags=re.S) if "distill_topk_bwd" in b]
    p, x, t = ex.make(300, 256, 3000, 16)
    dloss = torch.rand(300, device="cuda")
    full = {k: torch.randn(r, 256, device="cuda").to(torch.bfloat16) / 16 for k, r in (("w", 256), ("head", 3000))}
    names = dict(torch=torch, ld=ld, layer_norm=layer_norm, x=x, a=p.a, b=p.b, alpha=p.alpha, weight=p.ln_weight, bias=p.ln_bias,
                 T=p.temperature, ids=t.ids, teacher=t.logits, lse=t.lse, row_weight=t.weight, dloss=dloss, **full)
    exec(lines, names)
    from deterministic_arithmetic_gb300 import block8

    p.w, p.head = block8.block8(full["w"], tile=128), block8.block8(full["head"], tile=128)
    loss, dx, grads = step(p, x, t, dloss)
    mine = dict(ln_weight="dw", ln_bias="db", a="da", b="db_a")
    assert torch.equal(names["loss"], loss) and torch.equal(names["dx"], dx)
    assert all(torch.equal(names[mine[k]], grads[k]) for k in grads)
