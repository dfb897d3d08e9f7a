"""Cases, plain forms and 64-bit values of the MLP-block operators: layer norm, 8-bit activation
checkpoints with their use in the backward pass, and the gated feed-forward block.

``own`` selects what ``run`` calls: the plain forms below (elementary torch operations in 32 bits,
rounded once at the end) or the package's operators. ``exact`` gives the same outputs in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

GROUP = 32          # elements of a row that share one 8-bit scale
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one decode-like batch through a norm of the MLP width: latency only
        dict(name="ln_fwd 8x5120 bf16", op="ln_fwd", M=8, N=5120, dtype="bf16", wdtype="bf16", bias=True),
        # the norm before the adapters of the training step (M=8192 tokens, width 4096)
        dict(name="ln_fwd 8192x4096 bf16", op="ln_fwd", M=8192, N=4096, dtype="bf16", wdtype="bf16", bias=True),
        # its backward pass, with the reduction of the weight's and bias's gradients over 8192 rows
        dict(name="ln_bwd 8192x4096 bf16", op="ln_bwd", M=8192, N=4096, dtype="bf16", wdtype="bf16", bias=True,
             packed=False),
        # an odd width and a ragged batch in f32, no bias: rows that no vector load fits
        dict(name="ln_bwd 1000x2049 f32", op="ln_bwd", M=1000, N=2049, dtype="f32", wdtype="f32", bias=False,
             packed=False),
        # keeping the training step's x in 8 bits: written in the forward pass, read back in the backward
        dict(name="pack8 8192x4096 bf16", op="pack8", M=8192, K=4096, dtype="bf16"),
        # a small f32 batch whose rows end inside a group
        dict(name="pack8 100x1000 f32", op="pack8", M=100, K=1000, dtype="f32"),
        # dA of the training step from the kept 8 bits
        dict(name="da 8192x4096 R16", op="da", M=8192, K=4096, R=16),
        # dA of the decode-like configuration: 64 rows, rank 64
        dict(name="da 64x5120 R64", op="da", M=64, K=5120, R=64),
        # one token through the MLP's gated projections: the weights' bytes
        dict(name="ffn_fwd 1x5120x17408", op="ffn_fwd", M=1, K=5120, F=17408, act="silu", delta=False, save="none"),
        # the MLP configuration (4096 tokens, 5120 -> 17408) with gate and up kept in 8 bits for training
        dict(name="ffn_fwd 4096x5120x17408", op="ffn_fwd", M=4096, K=5120, F=17408, act="silu", delta=False,
             save="packed8"),
        # a short ragged batch of an adapter step: frozen weights, so only dx and the adapters' dY are wanted
        dict(name="ffn_bwd 333x520x1000", op="ffn_bwd", M=333, K=520, F=1000, act="gelu", save="bf16", dw=False),
        # the MLP configuration's backward with the weights' gradients, from the kept 8 bits
        dict(name="ffn_bwd 4096x5120x17408", op="ffn_bwd", M=4096, K=5120, F=17408, act="silu", save="packed8",
             dw=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _log8(rng, lo, hi):
    return max(lo, 8 * int(round(_log(rng, lo, hi) / 8)))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "pack8", "da", "ffn_fwd", "ffn_bwd"])
    if op in ("ln_fwd", "ln_bwd"):
        n = _log(rng, 33, 16384)
        m = _log(rng, 1, min(16384, (1 << 26) // n))
        if rng.random() < 0.5:
            n = max(8, n // 8 * 8)          # as often a width that vector loads fit
        c = dict(op=op, M=m, N=n, dtype=rng.choice(["bf16", "f32"]), wdtype=rng.choice(["bf16", "f32"]),
                 bias=rng.random() < 0.5)
        if op == "ln_bwd":
            c["packed"] = rng.random() < 0.5
        return c
    if op == "pack8":
        k = _log(rng, 5, 17408)
        return dict(op=op, M=_log(rng, 1, min(16384, (1 << 26) // k)), K=k, dtype=rng.choice(["bf16", "f32"]))
    if op == "da":
        k = _log8(rng, 64, 17408)
        return dict(op=op, M=_log(rng, 1, min(16384, (1 << 26) // k)), K=k, R=8 * rng.randint(1, 8))
    c = dict(op=op, M=_log(rng, 1, 4096), K=_log8(rng, 64, 5120), F=_log8(rng, 64, 17408),
             act=rng.choice(["silu", "gelu"]))
    if op == "ffn_fwd":
        c.update(delta=rng.random() < 0.5, save=rng.choice(["none", "bf16", "packed8"]))
    else:
        c.update(save=rng.choice(["bf16", "packed8"]), dw=rng.random() < 0.5)
    return c


# ------------------------------------------------------------------ inputs
def _groups(k):
    return -(-k // GROUP)


def _pack(x):
    """8-bit codes [M][32 g] and scale bytes [M][g] of x: a scale is 2^(byte - 127), the smallest that
    brings the group's largest magnitude to at most 127.5."""
    m, k = x.shape
    g = _groups(k)
    v = torch.nn.functional.pad(x.float(), (0, g * GROUP - k)).view(m, g, GROUP)
    amax = v.abs().amax(-1)
    frac, ex = torch.frexp(amax)
    e = ex - 7 + (frac > 127.5 / 128).to(ex.dtype)
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp_min(-127)
    step = torch.ldexp(torch.ones_like(amax), e)
    codes = torch.round(v / step[..., None]).clamp(-127, 127)
    return codes.to(torch.int8).view(m, g * GROUP), (e + 127).to(torch.uint8)


def _values(codes, scales, k):
    """The values that codes and scales stand for, in 32 bits."""
    m, g = scales.shape
    step = torch.ldexp(torch.ones_like(scales, dtype=torch.float32), scales.int() - 127)
    return (codes.view(m, g, GROUP).float() * step[..., None]).view(m, g * GROUP)[:, :k]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def rnd(*shape, s=1.0):
        return torch.randn(*shape, generator=gen, device="cuda") * s

    def stream(m, n):
        """Rows of a residual stream: channels of unequal size, a few of them far larger, a small offset."""
        ch = torch.exp(0.5 * rnd(n))
        ch = torch.where(torch.rand(n, generator=gen, device="cuda") < 1 / 256, 20 * ch, ch)
        return rnd(m, n) * ch + 0.2 * rnd(n)

    op, s = case["op"], dict(case)
    if op in ("ln_fwd", "ln_bwd"):
        m, n, dt, wdt = case["M"], case["N"], DT[case["dtype"]], DT[case["wdtype"]]
        x = stream(m, n).to(dt)
        s["weight"] = (1 + rnd(n, s=0.1)).to(wdt)
        s["bias"] = rnd(n, s=0.1).to(wdt) if case["bias"] else None
        s["eps"] = 1e-5
        if op == "ln_bwd":
            s["dy"] = rnd(m, n, s=0.1).to(dt)
            xf = x.double()
            mean = xf.mean(-1)
            s["mean"] = mean.float()
            s["rstd"] = (1 / torch.sqrt(xf.sub(mean[:, None]).square().mean(-1) + s["eps"])).float()
        if case.get("packed"):
            s["codes"], s["scales"] = _pack(x)
        else:
            s["x"] = x
    elif op == "pack8":
        s["x"] = stream(case["M"], case["K"]).to(DT[case["dtype"]])
    elif op == "da":
        s["codes"], s["scales"] = _pack(rnd(case["M"], case["K"]).to(torch.bfloat16))
        s["du"] = rnd(case["M"], case["R"], s=0.1).to(torch.bfloat16)
    else:
        m, k, f = case["M"], case["K"], case["F"]
        s["x"] = rnd(m, k).to(torch.bfloat16)
        s["w_gate"] = rnd(f, k, s=k ** -0.5).to(torch.bfloat16)
        s["w_up"] = rnd(f, k, s=k ** -0.5).to(torch.bfloat16)
        if op == "ffn_fwd":
            s["delta_gate"] = rnd(m, f, s=0.1) if case["delta"] else None
            s["delta_up"] = rnd(m, f, s=0.1) if case["delta"] else None
        else:
            s["dh"] = rnd(m, f, s=0.1).to(torch.bfloat16)
            for name in ("gate", "up"):
                v = rnd(m, f)
                s[name] = _pack(v) if case["save"] == "packed8" else v.to(torch.bfloat16)
    return s


# ------------------------------------------------------------- plain forms
def _act(name, g):
    if name == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g * g * g)))


def _act_and_slope(name, g):
    if name == "silu":
        sg = 1 / (1 + torch.exp(-g))
        return g * sg, sg * (1 + g * (1 - sg))
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * c * (1 + 3 * 0.044715 * g * g)


def _plain(s):
    op = s["op"]
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(-1)
        d = x - mean[:, None]
        rstd = torch.rsqrt((d * d).mean(-1) + s["eps"])
        y = d * rstd[:, None] * s["weight"].float()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        x = _values(s["codes"], s["scales"], s["N"]) if s["packed"] else s["x"].float()
        dy = s["dy"].float()
        xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * s["weight"].float()
        dx = s["rstd"][:, None] * (g - g.mean(-1, keepdim=True) - xh * (g * xh).mean(-1, keepdim=True))
        out = {"dx": dx.to(s["dy"].dtype), "dw": (dy * xh).sum(0)}
        if s["bias"] is not None:
            out["db"] = dy.sum(0)
        return out
    if op == "pack8":
        return {"values": _values(*_pack(s["x"]), s["K"]).to(s["x"].dtype)}
    if op == "da":
        return {"da": s["du"].float().t() @ _values(s["codes"], s["scales"], s["K"])}
    x, wg, wu = s["x"].float(), s["w_gate"].float(), s["w_up"].float()
    if op == "ffn_fwd":
        g, u = x @ wg.t(), x @ wu.t()
        if s["delta_gate"] is not None:
            g, u = g + s["delta_gate"], u + s["delta_up"]
        out = {"h": (_act(s["act"], g) * u).to(torch.bfloat16)}
        if s["save"] == "bf16":
            out.update(gate=g.to(torch.bfloat16), up=u.to(torch.bfloat16))
        elif s["save"] == "packed8":
            out.update(gate=_values(*_pack(g), s["F"]).to(torch.bfloat16),
                       up=_values(*_pack(u), s["F"]).to(torch.bfloat16))
        return out
    if s["save"] == "packed8":
        g, u = _values(*s["gate"], s["F"]), _values(*s["up"], s["F"])
    else:
        g, u = s["gate"].float(), s["up"].float()
    a, slope = _act_and_slope(s["act"], g)
    dh = s["dh"].float()
    dg, du = dh * u * slope, dh * a
    out = {"dx": (dg @ wg + du @ wu).to(torch.bfloat16), "dgate": dg.to(torch.bfloat16), "dup": du.to(torch.bfloat16)}
    if s["dw"]:
        out.update(dw_gate=(dg.t() @ x).to(torch.bfloat16), dw_up=(du.t() @ x).to(torch.bfloat16))
    return out


# ------------------------------------------------------ the package's calls
def _own(s):
    from deterministic_arithmetic_gb300 import gated_ffn, layer_norm, pack8

    op = s["op"]
    if op == "ln_fwd":
        y, mean, rstd = layer_norm.layer_norm_fwd(s["x"], s["weight"], s["bias"], s["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        x = pack8.Packed8(s["codes"], s["scales"], s["N"]) if s["packed"] else s["x"]
        dx, dw, db = layer_norm.layer_norm_bwd(s["dy"], x, s["weight"], s["mean"], s["rstd"],
                                               bias_grad=s["bias"] is not None)
        out = {"dx": dx, "dw": dw}
        if db is not None:
            out["db"] = db
        return out
    if op == "pack8":
        return {"values": pack8.unpack8(pack8.pack8(s["x"]), dtype=s["x"].dtype)}
    if op == "da":
        return {"da": pack8.pack8_da(s["du"], pack8.Packed8(s["codes"], s["scales"], s["K"]))}
    if op == "ffn_fwd":
        h, gate, up = gated_ffn.gated_ffn_fwd(s["x"], s["w_gate"], s["w_up"], activation=s["act"],
                                              delta_gate=s["delta_gate"], delta_up=s["delta_up"],
                                              save=None if s["save"] == "none" else s["save"])
        out = {"h": h}
        if s["save"] == "bf16":
            out.update(gate=gate, up=up)
        elif s["save"] == "packed8":
            out.update(gate=pack8.unpack8(gate), up=pack8.unpack8(up))
        return out
    if s["save"] == "packed8":
        gate, up = pack8.Packed8(*s["gate"], s["F"]), pack8.Packed8(*s["up"], s["F"])
    else:
        gate, up = s["gate"], s["up"]
    dx, dgate, dup, dwg, dwu = gated_ffn.gated_ffn_bwd(s["dh"], s["x"], s["w_gate"], s["w_up"], gate, up,
                                                       activation=s["act"], weight_grads=s["dw"])
    out = {"dx": dx, "dgate": dgate, "dup": dup}
    if s["dw"]:
        out.update(dw_gate=dwg, dw_up=dwu)
    return out


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------- work
def work(case):
    op, m = case["op"], case["M"]
    if op in ("ln_fwd", "ln_bwd"):
        n, e, w = case["N"], 2 if case["dtype"] == "bf16" else 4, 2 if case["wdtype"] == "bf16" else 4
        if op == "ln_fwd":
            return {"bytes": 2 * e * m * n + w * n * (2 if case["bias"] else 1) + 8 * m, "flops": 8 * m * n}
        x = m * _groups(n) * (GROUP + 1) if case["packed"] else e * m * n
        return {"bytes": x + 2 * e * m * n + 8 * m + w * n + 4 * n * (2 if case["bias"] else 1), "flops": 14 * m * n}
    if op == "pack8":       # x read, the codes and scales written and read again, the values written
        e = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * e * m * case["K"] + 2 * m * _groups(case["K"]) * (GROUP + 1), "flops": 4 * m * case["K"]}
    if op == "da":
        k, r = case["K"], case["R"]
        return {"bytes": m * _groups(k) * (GROUP + 1) + 2 * m * r + 4 * r * k, "flops": 2 * m * r * k}
    k, f = case["K"], case["F"]
    kept = {"none": 0, "bf16": 2 * m * f, "packed8": m * _groups(f) * (GROUP + 1)}[case["save"]]
    if op == "ffn_fwd":
        out = 2 * kept if case["save"] != "packed8" else 4 * kept + 4 * m * f     # written, read back as values
        return {"bytes": 2 * m * k + 4 * k * f + 2 * m * f + out + (8 * m * f if case["delta"] else 0),
                "flops": 4 * m * k * f}
    nbytes = 2 * m * f + 2 * kept + 4 * k * f + 2 * m * k + 4 * m * f
    flops = 4 * m * k * f
    if case["dw"]:
        nbytes += 2 * m * k + 4 * k * f
        flops += 4 * m * k * f
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    op = case["op"]
    if op.startswith("ffn") and case["M"] * case["K"] * case["F"] > 1 << 41:
        return None
    s = prepare(case, seed)
    f64 = torch.float64

    def decode(codes, scales, cols):
        steps = torch.exp2(scales.to(f64) - 127).repeat_interleave(GROUP, dim=1)
        return torch.mul(codes.to(f64), steps)[:, :cols]

    if op == "ln_fwd":
        x = s["x"].to(f64)
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        rstd = (var + s["eps"]).pow(-0.5)
        y = torch.addcmul(torch.zeros((), dtype=f64, device="cuda") if s["bias"] is None else s["bias"].to(f64),
                          (x - mean) * rstd, s["weight"].to(f64))
        return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "ln_bwd":
        n = case["N"]
        x = decode(s["codes"], s["scales"], n) if case["packed"] else s["x"].to(f64)
        mean, rstd, dy = s["mean"].to(f64).unsqueeze(1), s["rstd"].to(f64).unsqueeze(1), s["dy"].to(f64)
        centred = x - mean
        wdy = torch.mul(dy, s["weight"].to(f64))
        along = torch.einsum("mn,mn->m", wdy, centred).unsqueeze(1)
        dx = rstd * wdy - rstd * wdy.sum(1, keepdim=True) / n - rstd.pow(3) * centred * along / n
        out = {"dx": dx, "dw": torch.einsum("mn,mn,m->n", dy, centred, rstd[:, 0])}
        if case["bias"]:
            out["db"] = torch.einsum("mn->n", dy)
        return out
    if op == "pack8":
        # the nearest multiple of the group's step, with the step found by trying each power of two from below
        x = s["x"].to(f64)
        m, k = x.shape
        full = torch.zeros(m, _groups(k) * GROUP, dtype=f64, device="cuda")
        full[:, :k] = x
        full = full.reshape(m, -1, GROUP)
        top = full.abs().max(dim=2, keepdim=True).values
        e = torch.floor(torch.log2(top.clamp_min(2.0 ** -140))) - 8
        for _ in range(3):
            e = torch.where(top > 127.5 * torch.exp2(e), e + 1, e)
        step = torch.exp2(e.clamp_min(-127))
        return {"values": (torch.round(full / step).clamp(-127, 127) * step).reshape(m, -1)[:, :k]}
    if op == "da":
        return {"da": torch.einsum("mr,mk->rk", s["du"].to(f64), decode(s["codes"], s["scales"], case["K"]))}

    gelu = case["act"] == "gelu"

    def act(v):
        if gelu:
            z = math.sqrt(8 / math.pi) * (v + 0.044715 * v.pow(3))
            return v * torch.sigmoid(z)                 # 0.5 (1 + tanh(z / 2)) = sigmoid(z)
        return v * torch.sigmoid(v)

    if op == "ffn_fwd":
        x = s["x"].to(f64)
        pre = []
        for w, d in (("w_gate", "delta_gate"), ("w_up", "delta_up")):
            v = torch.einsum("mk,fk->mf", x, s[w].to(f64))
            pre.append(v if s[d] is None else v + s[d].to(f64))
        h = act(pre[0]) * pre[1]
        if case["save"] == "none":
            return {"h": h}
        if case["save"] == "bf16":
            return {"h": h, "gate": pre[0], "up": pre[1]}
        return {"h": h, "gate": None, "up": None}       # rounded to a step: 64 bits say nothing of a tie in 32
    if case["save"] == "packed8":
        g, u = decode(*s["gate"], case["F"]), decode(*s["up"], case["F"])
    else:
        g, u = s["gate"].to(f64), s["up"].to(f64)
    if gelu:
        z = math.sqrt(8 / math.pi) * (g + 0.044715 * g.pow(3))
        p = torch.sigmoid(z)
        slope = p + g * p * (1 - p) * math.sqrt(8 / math.pi) * (1 + 0.134145 * g.square())
    else:
        p = torch.sigmoid(g)
        slope = p + g * p * (1 - p)
    dh = s["dh"].to(f64)
    dg, du = dh * u * slope, dh * (g * p)
    dx = torch.einsum("mf,fk->mk", dg, s["w_gate"].to(f64))
    dx += torch.einsum("mf,fk->mk", du, s["w_up"].to(f64))
    out = {"dx": dx, "dgate": dg, "dup": du}
    if case["dw"]:
        x = s["x"].to(f64)
        out.update(dw_gate=torch.einsum("mf,mk->fk", dg, x), dw_up=torch.einsum("mf,mk->fk", du, x))
    return out
