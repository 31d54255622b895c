"""Plain 64-bit implementations (numpy) of the FP8 layer's operators, for the
tests: block scales and codes, SwiGLU and its gradient, the norm and its gradient,
and the experts' products of E4M3 codes."""
import numpy as np
import torch

BLOCK = 128


def nblocks(cols):
    return -(-cols // BLOCK)


def e4m3(codes):
    """Values of E4M3 codes (uint8), by the format: 1 sign, 4 exponent (bias 7), 3
    mantissa bits; 0x7f and 0xff are NaN, there are no infinities."""
    c = np.asarray(codes, dtype=np.uint8).astype(np.int64)
    s, e, m = c >> 7, c >> 3 & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((e == 15) & (m == 7), np.nan, v)
    return np.where(s == 1, -v, v)


def half_step(t):
    """Half the distance between E4M3 values around |t| (at most 448)."""
    with np.errstate(divide="ignore"):
        ex = np.floor(np.log2(np.abs(t)))
    return 2.0 ** (np.maximum(ex, -6.0) - 4.0)


def widen(scales, cols):
    """Scales [.., blocks] -> one per column."""
    return np.repeat(scales, BLOCK, -1)[..., :cols]


def values(codes, scales):
    return e4m3(codes) * widen(np.asarray(scales, dtype=np.float64), codes.shape[-1])


def block_scales(v):
    """max|v| / 448 of every block of 128 columns, 1 for zeros."""
    rows, cols = v.shape
    out = np.ones((rows, nblocks(cols)))
    for b in range(nblocks(cols)):
        top = np.abs(v[:, b * BLOCK:(b + 1) * BLOCK]).max(1)
        out[:, b] = np.where(top > 0, top / 448.0, 1.0)
    return out


def quantize32(x):
    """The codes and scales of float32 (or bf16) rows, bit for bit: IEEE float32
    quotients, and torch's rounding to E4M3 on the CPU.  x: torch, on the CPU."""
    v = x.float()
    rows, cols = v.shape
    pad = -cols % BLOCK
    b = torch.nn.functional.pad(v, (0, pad)).view(rows, -1, BLOCK)
    top = b.abs().amax(-1)
    scale = top / torch.full_like(top, 448.0)
    scale[scale == 0] = 1.0
    q = (b / scale[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(rows, -1)[:, :cols].contiguous(), scale


def swiglu(x):
    c = x.shape[1] // 2
    with np.errstate(over="ignore"):
        return x[:, :c] / (1.0 + np.exp(-x[:, :c])) * x[:, c:]


def swiglu_grad(x, d):
    """(gradient [rows, 2 cols], magnitude of its terms)."""
    c = x.shape[1] // 2
    g, u = x[:, :c], x[:, c:]
    s, rest = np.exp(-np.logaddexp(0.0, -g)), np.exp(-np.logaddexp(0.0, g))
    grad = np.concatenate([d * u * s * (1.0 + g * rest), d * g * s], 1)
    mag = np.concatenate([np.abs(d * u) * s * (1.0 + np.abs(g) * rest), np.abs(d * g) * s], 1)
    return grad, mag


def norm(z, w, eps):
    """(y, rstd)."""
    r = 1.0 / np.sqrt((z * z).mean(1) + eps)
    return z * r[:, None] * w, r


def norm_grad(dy, z, w, r, dres):
    """(dx, magnitude, dw, magnitude)."""
    n, g = z * r[:, None], dy * w
    dx = r[:, None] * (g - n * (g * n).mean(1, keepdims=True))
    mag = r[:, None] * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
    if dres is not None:
        dx, mag = dx + dres, mag + np.abs(dres)
    return dx, mag, (dy * n).sum(0), np.abs(dy * n).sum(0)


def matmul(x, xs, w, ws, offs, layout, cap, row_src, rows):
    """(out, magnitude, written): x, w codes (uint8); magnitude = the same sum over
    the products' absolute values."""
    E, Nc, Kd = w.shape
    out, mag = np.zeros((rows, Nc)), np.zeros((rows, Nc))
    written = np.zeros(rows, dtype=bool)
    xv = values(x, xs)
    for e in range(E):
        n = int(offs[e + 1]) - int(offs[e])
        if layout == 1:
            n = min(n, cap)
        if n <= 0:
            continue
        wv = values(w[e], np.repeat(ws[e], BLOCK, 0)[:Nc])
        to = e * cap if layout == 1 else int(offs[e])
        src = np.arange(to, to + n) if row_src is None else row_src[int(offs[e]):int(offs[e]) + n]
        ok = (src >= 0) & (src < x.shape[0])
        at = np.arange(to, to + n)
        written[at] = True
        out[at[ok]] = xv[src[ok]] @ wv.T
        mag[at[ok]] = np.abs(xv[src[ok]]) @ np.abs(wv).T
    return out, mag, written


def matmul_tol(Kd, out_bf16):
    """Relative to the magnitude, and to the value.  Each of the four steps of 32
    products of a block may cut every term, the sum so far among them, to 2^-23 of
    the largest: 4 * 33 * 2^-23.  Then a rounding for each scale and block."""
    return 4 * 33 * 2.0 ** -23 + (nblocks(Kd) + 3) * 2.0 ** -24, 2.0 ** -8 if out_bf16 else 2.0 ** -24
