"""Plain 64-bit forms of the 8-bit operators (numpy, CPU): e4m3 rounding, block scales, the
RMS norm and its gradients, the grouped products and the expert layer, with bounds on what
fp32 sums may add. Test infrastructure: shares no code with the GPU path."""
from __future__ import annotations

import numpy as np

B = 128
U32 = 2.0 ** -24  # half a step of fp32
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def e4m3_decode(code: np.ndarray) -> np.ndarray:
    """fp64 values of e4m3 bytes."""
    c = np.asarray(code, np.uint8).astype(np.int64)
    sign = np.where(c & 0x80, -1.0, 1.0)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return np.where((c & 0x7f) == 0x7f, np.nan, sign * v)


def e4m3_round(v: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value, ties to even (|v| <= 448)."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    _, e = np.frexp(np.where(a > 0, a, 1.0))
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(v / step) * step  # rint: ties to even


def scale_of(amax: np.ndarray) -> np.ndarray:
    """Least power of two s with amax <= 448 s, at least 2^-126."""
    amax = np.asarray(amax, np.float64)
    s = np.exp2(np.full(amax.shape, -126.0))
    for _ in range(400):
        low = amax > 448.0 * s
        if not low.any():
            return s
        s = np.where(low, 2.0 * s, s)
    raise AssertionError("amax is not finite")


def block_max(v: np.ndarray) -> np.ndarray:
    """max|v| over the finite values of each block of 128 along the last axis."""
    L = v.shape[-1]
    a = np.where(np.isfinite(v), np.abs(np.where(np.isfinite(v), v, 0.0)), 0.0)
    pad = [(0, 0)] * (a.ndim - 1) + [(0, -L % B)]
    a = np.pad(a, pad)
    return a.reshape(*a.shape[:-1], -1, B).max(-1)


def spread(s: np.ndarray, L: int) -> np.ndarray:
    """Scales [.., blocks] over the values of a row of length L."""
    return np.repeat(s, B, axis=-1)[..., :L]


def quantize_rows(v: np.ndarray):
    """(e4m3 values q, scales): v stands for about q * spread(scale)."""
    s = scale_of(block_max(v))
    w = np.where(np.isfinite(v), v, np.nan)
    return e4m3_round(w / spread(s, v.shape[-1])), s


def spread2(s: np.ndarray, R: int, C: int) -> np.ndarray:
    """Scales [.., blocks, blocks] over [.., R, C]."""
    return np.repeat(np.repeat(s, B, axis=-2)[..., :R, :], B, axis=-1)[..., :C]


def quantize_weights(w: np.ndarray):
    """w [E,K,C] -> e4m3 values [E,C,K], scales [E, ceil(C/128), ceil(K/128)]."""
    t = np.swapaxes(np.asarray(w, np.float64), 1, 2)
    m = block_max(t)  # [E, C, nbk]
    s = scale_of(np.swapaxes(block_max(np.swapaxes(m, 1, 2)), 1, 2))
    return e4m3_round(np.where(np.isfinite(t), t, np.nan) / spread2(s, t.shape[1], t.shape[2])), s


def rmsnorm(r: np.ndarray, w: np.ndarray, eps: float):
    """(y, rstd) of rows r."""
    r = np.asarray(r, np.float64)
    rstd = 1.0 / np.sqrt((r * r).mean(1) + eps)
    return r * rstd[:, None] * np.asarray(w, np.float64), rstd


def rmsnorm_backward(dy, r, w, rstd, dres=None):
    """(dx, dweight) and the sums of magnitudes that bound their fp32 errors."""
    dy, r, w = (np.asarray(a, np.float64) for a in (dy, r, w))
    t = np.asarray(rstd, np.float64)[:, None]
    g = dy * w
    z = 0.0 if dres is None else np.asarray(dres, np.float64)
    dx = t * (g - r * (t * t * (g * r).mean(1, keepdims=True))) + z
    mx = t * (np.abs(g) + np.abs(r) * (t * t * np.abs(g * r).mean(1, keepdims=True))) + np.abs(z)
    n = dy * r * t
    return dx, n.sum(0), mx, np.abs(n).sum(0)


def segments(offsets):
    return [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(len(offsets) - 1)
            if offsets[e + 1] > offsets[e]]


def binades(v, s):
    """2^exponent of the e4m3 value q of each v = q s (2^-6 for subnormals and zeros), times
    the scale."""
    q = np.abs(v) / s
    return np.exp2(np.maximum(np.floor(np.log2(np.maximum(q, 2.0 ** -9))), -6.0)) * s


def grouped(a, sa, w, sw, offsets, rows):
    """out[s] = a[rows[s]] W_e^T for values a, w with scales sa, sw over them, and the bound of
    its sums' error. fp32: at most K + 16 roundings on each product's way into the sum. And
    the matrix cores cut each of eight products next to each other along K off at 2^-13 of
    the largest one's power of two, 2^(ea + eb) with the operands' exponents: each loses less
    than 2^-13 max 2^(ea + eb), the eight less than 8 2^-13 max <= 8 2^-13 sum 2^ea 2^eb."""
    out = np.zeros((int(offsets[-1]), w.shape[1]))
    err = np.zeros_like(out)
    ba = binades(a, sa)
    for e, lo, hi in segments(offsets):
        x = a[rows[lo:hi]]
        out[lo:hi] = x @ w[e].T
        err[lo:hi] = (np.abs(x) @ np.abs(w[e]).T) * ((w.shape[2] + 16) * U32)
        err[lo:hi] += (ba[rows[lo:hi]] @ binades(w[e], sw[e]).T) * 2.0 ** -10
    return out, err


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def experts(x, sx, w_up, su, w_down, sd, offsets, rows, scores, N, concat=False):
    """The expert layer on the values the 8-bit operands stand for: (out, bound of the bf16
    out's error, h interleaved, bound of h's error before its rounding).

    a is put on e4m3 from unrounded h. Where h's fp32 error could carry a past a tie (or a
    block's maximum past the border of a scale) either neighbour may come out: the bound
    takes the largest change of the quantised value over the interval of a's error."""
    I = w_down.shape[2]
    h, eh = grouped(x, sx, w_up, su, offsets, rows)
    if concat:
        h = np.stack([h[:, :I], h[:, I:]], 2).reshape(len(h), 2 * I)
        eh = np.stack([eh[:, :I], eh[:, I:]], 2).reshape(len(eh), 2 * I)
    g, u, eg, eu = h[:, 0::2], h[:, 1::2], eh[:, 0::2], eh[:, 1::2]
    a = silu(g) * u
    # |silu'| <= 1.1; exp, reciprocal and two products in fp32: a few roundings, and the
    # rounding of exp's argument, |g| of them
    ea = 1.1 * np.abs(u) * eg + np.abs(silu(g)) * eu + np.abs(a) * (16 + np.abs(g)) * U32
    q, s = quantize_rows(a)
    v = q * spread(s, I)
    m = block_max(a)
    em = block_max(ea)
    dv = np.zeros_like(v)
    for sc in (scale_of(np.maximum(m - em, 0.0)), scale_of(m + em)):
        w = spread(sc, I)
        for side in (-1.0, 1.0):
            dv = np.maximum(dv, np.abs(e4m3_round(np.clip((a + side * ea) / w, -480, 480)) * w - v))
    y, ey = grouped(v, spread(s, I), w_down, sd, offsets, np.arange(len(v)))
    for e, lo, hi in segments(offsets):
        ey[lo:hi] += dv[lo:hi] @ np.abs(w_down[e]).T
    ey += np.abs(y) * HALF["bf16"]
    out = np.zeros((N, w_down.shape[1]))
    bound = np.zeros_like(out)
    for s_, (t, wt) in enumerate(zip(rows, scores)):
        out[t] += wt * y[s_]
        bound[t] += abs(wt) * (ey[s_] + np.abs(y[s_]) * 72 * U32)  # up to 64 fp32 additions
    return out, bound + np.abs(out) * HALF["bf16"], h, eh
