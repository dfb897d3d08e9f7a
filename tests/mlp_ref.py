"""Plain 64-bit forms of the MLP-block operators (NumPy), for the tests of include/lora_mlp.h. They share
nothing with the CUDA path. bf16 arrays are passed as the float64 values they hold."""
import numpy as np

U32 = 2.0 ** -24          # half an ulp, relative, of fp32
U16 = 2.0 ** -8           # of bf16: 8 significant bits, as 2^-24 is for the 24 of fp32


def f64(t):
    return t.detach().to("cpu").double().numpy()


def layer_norm(x, w, b, eps):
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1 / np.sqrt((d * d).mean(1) + eps)
    return d * rstd[:, None] * w + (0 if b is None else b), mean, rstd


def layer_norm_bwd(dy, x, w, mean, rstd):
    xh = (x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = rstd[:, None] * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0), xh, g


def pack8(x):
    """(codes, scale bytes) of a float64 array of fp32 (or bf16) values, group by group."""
    m, k = x.shape
    g = -(-k // 32)
    codes = np.zeros((m, 32 * g), np.int8)
    scales = np.zeros((m, g), np.uint8)
    for r in range(m):
        for j in range(g):
            v = x[r, 32 * j:32 * j + 32]
            if not np.isfinite(v).all():
                scales[r, j] = 255
                continue
            a = np.abs(v).max()
            e = -127
            if a > 0:
                e = max(-127, int(np.floor(np.log2(a))) - 8)
                while a > 127.5 * 2.0 ** e and e < 121:      # 2^121: the largest step whose values stay finite
                    e += 1
            q = np.clip(np.rint(v / 2.0 ** e), -127, 127)     # rint: ties to even
            codes[r, 32 * j:32 * j + len(v)] = q
            scales[r, j] = e + 127
    return codes, scales


def unpack8(codes, scales, k):
    step = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return (codes.astype(np.float64).reshape(len(codes), -1, 32) * step[:, :, None]).reshape(len(codes), -1)[:, :k]


def act(name, y):
    """(act(y), act'(y)); gelu in its tanh form."""
    with np.errstate(over="ignore"):
        if name == "silu":
            p = 1 / (1 + np.exp(-y))
            return y * p, p * (1 + y * (1 - p))
        c = np.sqrt(2 / np.pi)
        t = np.tanh(c * (y + 0.044715 * y ** 3))
        return 0.5 * y * (1 + t), 0.5 * (1 + t) + 0.5 * y * (1 - t * t) * c * (1 + 3 * 0.044715 * y * y)


def ffn(name, x, wg, wu, dg=0.0, du=0.0):
    g, u = x @ wg.T + dg, x @ wu.T + du
    return act(name, g)[0] * u, g, u


def ffn_off_along(name, x, wg, wu, dh, i, grad, h=2.0 ** -12):
    """How far |grad|, the slope that a gradient of sum(dh * h) by argument i (x, wg, wu) claims along itself, is from
    the central difference along it, in units of |grad|. A gradient off by an error e shows it as (e . grad) / |grad|^2."""
    size = np.linalg.norm(grad)
    ends = []
    for s in (h, -h):
        args = [x, wg, wu]
        args[i] = args[i] + s * grad / size
        ends.append((ffn(name, *args)[0] * dh).sum())
    return abs((ends[0] - ends[1]) / (2 * h) / size - 1)
