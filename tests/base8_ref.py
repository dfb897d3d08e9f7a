"""Plain 64-bit forms of the operators of include/lora_base8.h (NumPy), for their tests. They share nothing with the
CUDA path."""
import numpy as np

U32 = 2.0 ** -24          # half an ulp, relative, of fp32
U16 = 2.0 ** -8           # of bf16
TOP = 448.0


def e4m3(v):
    """v rounded to the nearest e4m3 value, ties to even, held to +-448: 4 significant bits, down to a step of 2^-9."""
    v = np.clip(np.asarray(v, np.float64), -TOP, TOP)
    _, e = np.frexp(v)                                   # |v| in [2^(e-1), 2^e)
    step = np.ldexp(1.0, np.maximum(e - 4, -9))
    return np.clip(np.rint(v / step) * step, -TOP, TOP)


def block8(x, tile):
    """(values of the codes, scales) of a float64 array."""
    m, k = x.shape
    codes = np.zeros((m, k))
    scales = np.zeros((-(-m // tile), -(-k // 128)))
    for i in range(scales.shape[0]):
        for j in range(scales.shape[1]):
            at = np.s_[i * tile:(i + 1) * tile, 128 * j:128 * j + 128]
            v = x[at]
            if not np.isfinite(v).all():
                scales[i, j] = np.nan
                continue
            a, e = np.abs(v).max(), -124
            if a > 0:
                e = max(-124, int(np.floor(np.log2(a))) - 10)
                while a > TOP * 2.0 ** e and e < 119:
                    e += 1
            scales[i, j] = 2.0 ** e
            codes[at] = e4m3(v / 2.0 ** e)
    return codes, scales


def spread(scales, tile, m, k):
    """The scale of each element."""
    return scales.repeat(tile, 0)[:m].repeat(128, 1)[:, :k]


def unblock8(codes, scales, tile):
    return codes * spread(scales, tile, *codes.shape)


def product_tol(a, b, blocks):
    """How far an fp32 result of a @ b, of blocks of 128 each added up by tensor-core instructions and then joined one
    after another, may be off: a block's 128 products are exact and each addition drops less than an ulp, 2^-23, of
    at most the sum of magnitudes; joining rounds the scales' product and every fma by half an ulp."""
    return (128 * 2 * U32 + (blocks + 2) * U32) * (np.abs(a) @ np.abs(b))


def entries(ids, teacher, V):
    """Which of a row's entries count: in the vocabulary, not -infinity, the first of their id."""
    ok, seen = [], set()
    for i, t in zip(ids, teacher):
        good = 0 <= i < V and not t == -np.inf and i not in seen
        if good:
            seen.add(int(i))
        ok.append(good)
    return np.array(ok, bool)


def distill(z, ids, teacher, T, lse=None, weight=None):
    """(loss, probs, stats, dz, tol): dz the gradient of the sum of the losses, tol how far an fp32 loss may be off."""
    M, V = z.shape
    loss, tol, probs = np.zeros(M), np.zeros(M), np.full(ids.shape, -1.0)
    stats, dz = np.zeros((M, 4)), np.zeros((M, V))
    for r in range(M):
        w = 1.0 if weight is None else weight[r]
        ok = entries(ids[r], teacher[r], V)
        if w == 0 or not ok.any():
            continue
        with np.errstate(invalid="ignore"):
            m = z[r].max()
            arg = (z[r] - m) / T
            e = np.exp(arg)
        s = e.sum()
        q, log_q = e / s, arg - np.log(s)
        at, t = ids[r][ok], teacher[r][ok] / T
        norm = np.log(np.exp(t - t.max()).sum()) + t.max() if lse is None else lse[r]
        log_p = t - norm
        p = np.exp(log_p)
        live = p > 0
        part = p[live] * (log_p[live] - log_q[at][live])
        total, keep, mass, spare = part.sum(), 1.0, p.sum(), 0.0
        others = np.ones(V, bool)
        others[at] = False
        if lse is not None:
            rest, rho = max(1 - p.sum(), 0.0), q[others].sum()
            if rest > 0:
                with np.errstate(divide="ignore"):
                    lr = np.log(rest) - np.log(rho)
                total += rest * lr
                mass += rest
                # the rest's mass is 1 less a sum of p, each 2^-21 off at most
                spare = 2.0 ** -21 * p.sum() * (1 + abs(lr)) + 2.0 ** -21 * rest * abs(np.log(rho))
            keep = 1 - rest / rho if rho > 0 else 1.0
        loss[r], probs[r, ok], stats[r] = w * total, p, (m, np.log2(s), keep, w)
        d = q * keep if keep != 1.0 else q.copy()
        d[at] = q[at] - p
        dz[r] = w / T * d
        # log s: every exponential is 2^-21 off at most plus 2^-22 of its argument, and the sums' roundings
        with np.errstate(invalid="ignore"):
            far = np.where(q > 0, q * np.abs(arg), 0).sum()
        d_log = 2.0 ** -21 * (1 + far) + (V / 16384 + 64) * U32
        tol[r] = abs(w) * (mass * d_log + 2.0 ** -21 * (np.abs(part).sum() + p.sum()) + spare) + 2 * U32 * abs(loss[r])
    return loss, probs, stats, dz, tol
