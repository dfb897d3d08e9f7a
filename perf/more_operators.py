"""Cases, plain forms and 64-bit values of the operators that train adapters on a frozen 8-bit base by
distillation: 8-bit blocks of 128, the products with weights held so, and the loss against a teacher's top
logits.

``own`` selects what ``run`` calls: the plain forms below (elementary torch operations in 32 bits,
rounded once at the end) or the package's operators. ``exact`` gives the same outputs in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128         # elements of a row (and, for weights, rows) that share one scale
TOP = 448.0         # the largest e4m3 value
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
F8 = torch.float8_e4m3fn


# ------------------------------------------------------------------- cases
def listed():
    return [
        # the activations of a serving batch on their way into a projection of the MLP width: latency only
        dict(name="block8 64x5120 bf16", op="block8", M=64, K=5120, dtype="bf16", tile=1),
        # the activations of the training step (8192 tokens, width 4096)
        dict(name="block8 8192x4096 bf16", op="block8", M=8192, K=4096, dtype="bf16", tile=1),
        # a projection's weights of the MLP configuration, once when a base is loaded
        dict(name="block8 17408x5120 bf16 tile 128", op="block8", M=17408, K=5120, dtype="bf16", tile=128),
        # one token through an 8-bit projection of the MLP: the weight's bytes
        dict(name="linear_fwd 1x5120->17408", op="linear_fwd", M=1, K=5120, N=17408, out="bf16", delta=False),
        # a short ragged batch, sizes that no block of 128 divides, fp32 results
        dict(name="linear_fwd 333x520->1000 f32", op="linear_fwd", M=333, K=520, N=1000, out="f32", delta=False),
        # the training step's adapted layer: the frozen base's product plus the adapter's delta
        dict(name="linear_fwd 8192x4096->4096 delta", op="linear_fwd", M=8192, K=4096, N=4096, out="bf16", delta=True),
        # a small batch's gradient through a square projection: the weight's bytes, along its other side
        dict(name="linear_bwd 16x4096->4096", op="linear_bwd", M=16, K=4096, N=4096, out="bf16", delta=False),
        # the MLP configuration's gradient through an up projection, joined with the adapter's
        dict(name="linear_bwd 4096x5120->17408 delta", op="linear_bwd", M=4096, K=5120, N=17408, out="bf16", delta=True),
        # a few positions with an odd vocabulary in fp32, 20 of the teacher's logits: latency
        dict(name="distill_fwd 7x50257 f32 top 20", op="distill_fwd", M=7, V=50257, top=20, dtype="f32", tail=False,
             temperature=1.0),
        # a training batch over a large vocabulary, 64 of the teacher's logits and the mass of the rest
        dict(name="distill_fwd 4096x131072 bf16 top 64 rest", op="distill_fwd", M=4096, V=131072, top=64, dtype="bf16",
             tail=True, temperature=2.0),
        # a ragged batch's gradient, written in 8-bit blocks for the product with the head's 8-bit weights
        dict(name="distill_bwd 333x32000 bf16 top 16 blocks", op="distill_bwd", M=333, V=32000, top=16, dtype="bf16",
             tail=False, temperature=1.0, out="block8"),
        # the gradient of the large training batch
        dict(name="distill_bwd 4096x131072 bf16 top 64 rest", op="distill_bwd", M=4096, V=131072, top=64, dtype="bf16",
             tail=True, temperature=2.0, out="same"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["block8", "linear_fwd", "linear_bwd", "distill_fwd", "distill_bwd"])
    if op == "block8":
        k = _log(rng, 33, 17408)
        if rng.random() < 0.5:
            k = max(16, k // 16 * 16)       # as often a width that vector loads fit
        return dict(op=op, M=_log(rng, 1, min(17408, (1 << 26) // k)), K=k, dtype=rng.choice(["bf16", "f32"]),
                    tile=rng.choice([1, 128]))
    if op.startswith("linear"):
        k, n = _log(rng, 64, 5120), _log(rng, 64, 17408)
        if rng.random() < 0.5:
            k, n = max(64, k // 16 * 16), max(64, n // 16 * 16)
        return dict(op=op, M=_log(rng, 1, 4096), K=k, N=n, out=rng.choice(["bf16", "f32"]), delta=rng.random() < 0.5)
    v = _log(rng, 1000, 131072)
    if rng.random() < 0.5:
        v = v // 8 * 8
    c = dict(op=op, M=_log(rng, 1, min(4096, (1 << 28) // v)), V=v, top=_log(rng, 1, 256), dtype=rng.choice(["bf16", "f32"]),
             tail=rng.random() < 0.5, temperature=rng.choice([0.7, 1.0, 2.0, 4.0]))
    if op == "distill_bwd":
        c["out"] = rng.choice(["same", "block8"])
    return c


# ------------------------------------------------------------------ inputs
def _blocks(k):
    return -(-k // BLOCK)


def _cut(x, tile):
    """x in 32 bits as [row blocks][tile][column blocks][128], padded with zeros."""
    m, k = x.shape
    r, g = -(-m // tile), _blocks(k)
    return torch.nn.functional.pad(x.float(), (0, g * BLOCK - k, 0, r * tile - m)).view(r, tile, g, BLOCK)


def _block8(x, tile):
    """(codes [M][16 ceil(K / 16)] e4m3, scales [ceil(M / tile)][ceil(K / 128)]) of x: a scale is the smallest
    power of two, from 2^-124 to 2^119, of which no value is more than 448 times."""
    m, k = x.shape
    v = _cut(x, tile)
    frac, ex = torch.frexp(v.abs().amax((1, 3)))
    e = (ex - 9 + (frac > 0.875).to(ex.dtype)).clamp(-124, 119)
    scale = torch.ldexp(torch.ones_like(frac), e)
    codes = (v * torch.ldexp(torch.ones_like(frac), -e)[:, None, :, None]).clamp(-TOP, TOP).to(F8)
    full = codes.view(v.shape[0] * tile, -1)[:m]
    pad = -(-k // 16) * 16
    return full[:, :min(pad, full.shape[1])].contiguous(), scale


def _values(codes, scales, m, k, tile):
    """The values that codes and scales stand for, in 32 bits."""
    return codes.float()[:, :k] * scales.repeat_interleave(tile, 0)[:m].repeat_interleave(BLOCK, 1)[:, :k]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def rnd(*shape, s=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * s

    def uneven(m, n):
        """Rows of a residual stream: channels of unequal size, a few of them far larger."""
        ch = torch.exp(0.5 * rnd(n))
        return rnd(m, n) * torch.where(torch.rand(n, generator=gen, device="cuda") < 1 / 256, 20 * ch, ch)

    op, s, m = case["op"], dict(case), case["M"]
    if op == "block8":
        k = case["K"]
        s["x"] = (uneven(m, k) if case["tile"] == 1 else rnd(m, k, s=k ** -0.5)).to(DT[case["dtype"]])
    elif op.startswith("linear"):
        k, n = case["K"], case["N"]
        s["w"] = _block8(rnd(n, k, s=k ** -0.5).to(torch.bfloat16), BLOCK)
        if op == "linear_fwd":
            s["x"] = _block8(uneven(m, k).to(torch.bfloat16), 1)
            s["delta"] = rnd(m, n, s=0.1) if case["delta"] else None
        else:
            s["dy"] = _block8((rnd(m, n) * torch.exp(rnd(m, 1)) * 1e-3).to(torch.bfloat16), 1)
            s["delta"] = rnd(m, k, s=1e-4) if case["delta"] else None
    else:
        v, top, t = case["V"], case["top"], case["temperature"]
        # a few entries far above the rest, as a language model's: the r-th largest near -2.2 log(r)
        full = torch.rand(m, v, generator=gen, device="cuda").mul_(v).add_(0.5).log_().mul_(-2.2)
        s["teacher"], s["ids"] = torch.topk(full, top, dim=1)
        s["teacher_lse"] = torch.logsumexp(full / t, dim=1) if case["tail"] else None
        # shorter lists (a teacher that keeps fewer logits where they are certain), the rest of the row -1
        keep = torch.randint(top // 2, top + 1, (m, 1), generator=gen, device="cuda")
        s["ids"] = torch.where(torch.arange(top, device="cuda") <= keep, s["ids"], -1)
        s["logits"] = (full + rnd(m, v)).to(DT[case["dtype"]])
        del full
        s["weight"] = torch.ones(m, device="cuda")
        s["weight"][: m // 16] = 0.0                         # the prompt's positions
        if op == "distill_bwd":
            _, s["probs"], s["stats"] = _loss(s)
            s["dloss"] = torch.rand(m, generator=gen, device="cuda") / m
            for name in ("teacher", "teacher_lse", "weight"):
                del s[name]
    return s


# ------------------------------------------------------------- plain forms
def _loss(s):
    """(loss, probs, stats): the divergence of the student's distribution from the teacher's, a row each. The
    teacher's few entries in 64 bits: the terms of a small divergence cancel."""
    t, ids, w = s["temperature"], s["ids"], s["weight"]
    z = s["logits"].float()
    valid = (ids >= 0) & (ids < s["V"])
    at = ids.clamp(0, s["V"] - 1)
    log_p = torch.where(valid, s["teacher"].double() / t, -math.inf)
    norm = s["teacher_lse"]
    if norm is None:
        top = log_p.amax(1)
        norm = top + torch.exp(log_p - top[:, None]).sum(1).log()
    log_p = log_p - norm[:, None]
    p = log_p.exp()
    top = z.amax(1)
    e = torch.exp((z - top[:, None]) / t)
    total = e.sum(1, dtype=torch.float64)
    log_q = (z.gather(1, at).double() - top[:, None]) / t - total.log()[:, None]
    loss = torch.where(p > 0, p * (log_p - log_q), 0.0).sum(1)
    rest = torch.ones_like(loss)
    if s["teacher_lse"] is not None:
        of_top = torch.where(valid, log_q.exp(), 0.0).sum(1)
        of_rest = e.scatter_add_(1, at, torch.where(valid, -e.gather(1, at), 0.0)).sum(1, dtype=torch.float64) / total
        r, log_rho = (1 - p.sum(1)).clamp_min(0), -torch.log1p(of_top / of_rest)
        loss = loss + torch.where(r > 0, r * (torch.log(r) - log_rho), 0.0)
        rest = 1 - r * torch.exp(-log_rho)
    on = w != 0
    stats = torch.stack([top, total.log() / math.log(2.0), rest, w], 1)
    return (torch.where(on, loss * w, 0.0).float(), torch.where(valid & on[:, None], p, -1.0).float(),
            torch.where(on[:, None], stats, 0.0).float())


def _grad(s):
    """The gradient of sum(dloss * loss) by the logits, in 32 bits."""
    t, ids, p = s["temperature"], s["ids"], s["probs"]
    top, log2_sum, rest, w = s["stats"].unbind(1)
    z = s["logits"].float()
    g = (s["dloss"] * w / t)[:, None]
    q = torch.exp((z - top[:, None]) / t - (log2_sum * math.log(2.0))[:, None]) * g
    at = ids.clamp(0, s["V"] - 1)
    qi = q.gather(1, at)
    rest = rest[:, None]
    return (q * rest).scatter_add_(1, at, torch.where(p >= 0, qi - p * g - qi * rest, 0.0))


def _plain(s):
    op = s["op"]
    if op == "block8":
        x, tile = s["x"], s["tile"]
        codes, scales = _block8(x, tile)
        return {"values": _values(codes, scales, *x.shape, tile).to(x.dtype), "scales": scales}
    if op.startswith("linear"):
        m, k, n = s["M"], s["K"], s["N"]
        w = _values(*s["w"], n, k, BLOCK)
        if op == "linear_fwd":
            y = _values(*s["x"], m, k, 1) @ w.t()
        else:
            y = _values(*s["dy"], m, n, 1) @ w
        if s["delta"] is not None:
            y = y + s["delta"]
        return {"y" if op == "linear_fwd" else "dx": y.to(DT[s["out"]])}
    if op == "distill_fwd":
        loss, probs, stats = _loss(s)
        return {"loss": loss, "probs": probs, "stats": stats}
    dz = _grad(s)
    if s["out"] == "block8":
        return {"dlogits": _values(*_block8(dz, 1), s["M"], s["V"], 1).to(torch.bfloat16)}
    return {"dlogits": dz.to(s["logits"].dtype)}


# ------------------------------------------------------ the package's calls
def _own(s):
    from deterministic_arithmetic_gb300 import block8 as b8
    from deterministic_arithmetic_gb300 import distill

    op = s["op"]
    if op == "block8":
        p = b8.block8(s["x"], tile=s["tile"])
        return {"values": b8.unblock8(p, dtype=s["x"].dtype), "scales": p.scales}
    if op.startswith("linear"):
        w = b8.Block8(*s["w"], s["K"], BLOCK)
        if op == "linear_fwd":
            return {"y": b8.block8_linear_fwd(b8.Block8(*s["x"], s["K"], 1), w, delta=s["delta"], dtype=DT[s["out"]])}
        return {"dx": b8.block8_linear_bwd(b8.Block8(*s["dy"], s["N"], 1), w, delta=s["delta"], dtype=DT[s["out"]])}
    if op == "distill_fwd":
        loss, probs, stats = distill.distill_topk_fwd(s["logits"], s["ids"], s["teacher"], temperature=s["temperature"],
                                                      teacher_lse=s["teacher_lse"], weight=s["weight"])
        return {"loss": loss, "probs": probs, "stats": stats}
    dz = distill.distill_topk_bwd(s["dloss"], s["logits"], s["ids"], s["probs"], s["stats"],
                                  temperature=s["temperature"], block8=s["out"] == "block8")
    return {"dlogits": b8.unblock8(dz) if s["out"] == "block8" else dz}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work
def work(case):
    op, m = case["op"], case["M"]
    if op == "block8":      # x read, the codes and scales written and read again, the values written
        k, e = case["K"], 2 if case["dtype"] == "bf16" else 4
        held = m * k + 4 * -(-m // case["tile"]) * _blocks(k)
        return {"bytes": 2 * e * m * k + 2 * held, "flops": 4 * m * k}
    if op.startswith("linear"):
        k, n = case["K"], case["N"]
        a, b = (k, n) if op == "linear_fwd" else (n, k)     # the reduction's length, the outputs' columns
        e = (2 if case["out"] == "bf16" else 4) + (4 if case["delta"] else 0)
        return {"bytes": n * k + 4 * _blocks(n) * _blocks(k) + m * a + 4 * m * _blocks(a) + e * m * b,
                "flops": 2 * m * k * n}
    v, top, e = case["V"], case["top"], 2 if case["dtype"] == "bf16" else 4
    on = m - m // 16                                         # rows of weight 0 are not read
    if op == "distill_fwd":
        return {"bytes": on * (e * v + 12 * top + (4 if case["tail"] else 0)) + m * (4 + 4 * top + 20),
                "flops": 4 * on * v}
    if case["out"] == "block8":     # the codes and scales written and read again, the values written
        out = 2 * (v + 4 * _blocks(v)) + 2 * v
    else:
        out = e * v
    return {"bytes": on * (e * v + 12 * top) + m * (out + 20), "flops": 4 * on * v}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    op, m = case["op"], case["M"]
    s = prepare(case, seed)
    f64 = torch.float64

    def nearest(v, top):
        """The nearest e4m3 values of v / scale, times scale, and scale, of blocks whose largest magnitude is top."""
        e = torch.floor(torch.log2(top.clamp_min(2.0 ** -120))) - 10
        for _ in range(4):
            e = torch.where(top > TOP * torch.exp2(e), e + 1, e)
        scale = torch.exp2(e.clamp(-124, 119))
        u = v / scale
        step = torch.exp2(torch.floor(torch.log2(u.abs().clamp_min(2.0 ** -6))) - 3)
        return (torch.round(u / step) * step).clamp(-TOP, TOP) * scale, scale

    def decode(pair, rows, cols, tile):
        codes, scales = pair
        out = codes.to(f64)[:, :cols]
        r = torch.arange(rows, device="cuda") // tile
        c = torch.arange(cols, device="cuda") // BLOCK
        return out.mul_(scales.to(f64)[r][:, c])

    if op == "block8":
        k, tile = case["K"], case["tile"]
        if m * k > 1 << 27:
            return None
        v = _cut(s["x"], tile).to(f64)
        got, scale = nearest(v, v.abs().amax((1, 3), keepdim=True))
        return {"values": got.reshape(-1, got.shape[2] * BLOCK)[:m, :k], "scales": scale[:, 0, :, 0]}
    if op.startswith("linear"):
        k, n = case["K"], case["N"]
        if m * k * n > 1 << 41:
            return None
        w = decode(s["w"], n, k, BLOCK)
        if op == "linear_fwd":
            y = torch.einsum("mk,nk->mn", decode(s["x"], m, k, 1), w)
        else:
            y = torch.einsum("mn,nk->mk", decode(s["dy"], m, n, 1), w)
        return {"y" if op == "linear_fwd" else "dx": y if s["delta"] is None else y.add_(s["delta"])}
    t, ids, v = case["temperature"], s["ids"], case["V"]
    listed_ = ids >= 0
    at = torch.where(listed_, ids, 0)
    if op == "distill_fwd":
        w = s["weight"].to(f64)
        soft = torch.where(listed_, s["teacher"].to(f64) / t, -math.inf)
        norm = torch.logsumexp(soft, 1) if s["teacher_lse"] is None else s["teacher_lse"].to(f64)
        log_p = soft - norm[:, None]
        p = log_p.exp()
        z = s["logits"].to(f64)
        top = z.amax(1)
        log_q = torch.log_softmax(z / t, 1)
        lse = torch.logsumexp(z / t, 1) - top / t
        del z
        loss = torch.where(listed_, p * (log_p - log_q.gather(1, at)), 0.0).sum(1)
        rest = torch.ones_like(loss)
        if case["tail"]:
            r = (1 - p.sum(1)).clamp_min(0)
            hidden = torch.cat([log_q, log_q.new_zeros(m, 1)], 1).scatter_(1, torch.where(listed_, ids, v), -math.inf)
            log_rho = torch.logsumexp(hidden[:, :v], 1)
            loss = loss + torch.where(r > 0, r * (torch.log(r) - log_rho), 0.0)
            rest = 1 - r * torch.exp(-log_rho)
        off = w == 0
        stats = torch.stack([top, lse / math.log(2.0), rest, w], 1)
        return {"loss": loss * w, "probs": torch.where(listed_, p, -1.0).masked_fill(off[:, None], -1.0),
                "stats": stats.masked_fill(off[:, None], 0.0)}
    top, log2_sum, rest, w = s["stats"].to(f64).unbind(1)
    q = s["logits"].to(f64).sub_(top[:, None]).mul_(math.log2(math.e) / t).sub_(log2_sum[:, None]).exp2_()
    qi = q.gather(1, at)
    dz = q.mul_(rest[:, None])
    rows = torch.arange(m, device="cuda")[:, None].expand_as(at)
    p = s["probs"].to(f64)
    use = p >= 0
    dz[rows[use], ids[use]] = (qi - p)[use]
    dz.mul_((s["dloss"].to(f64) * w / t)[:, None])
    if case["out"] == "block8":
        cut = torch.nn.functional.pad(dz, (0, _blocks(v) * BLOCK - v)).view(m, -1, BLOCK)
        dz = nearest(cut, cut.abs().amax(2, keepdim=True))[0].view(m, -1)[:, :v]
    return {"dlogits": dz}
