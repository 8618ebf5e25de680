"""Plain numpy oracles of the FP8 block format, the 8-bit checkpoints and the
balance loss: codes by the formats' own fp32 arithmetic (bit by bit), sums in
float64."""
import numpy as np

BLOCK, CKPT = 128, 32
TINY = np.float32(2.0 ** -126)


def _e4m3_table():
    c = np.arange(127)
    e, m = c >> 3, c & 7
    return np.where(e > 0, np.ldexp(1.0 + m / 8.0, e - 7), np.ldexp(m / 8.0, -6))


E4M3 = _e4m3_table()  # magnitudes of codes 0 .. 126
_MID = (E4M3[1:] + E4M3[:-1]) / 2


def e4m3_encode(v):
    """Codes of float32 values: nearest, ties to the even code; NaN 0x7f."""
    v = np.asarray(v, np.float32)
    a = np.abs(v.astype(np.float64))
    with np.errstate(invalid="ignore"):
        lo = np.searchsorted(_MID, a, side="left")    # ties: the lower code
        hi = np.searchsorted(_MID, a, side="right")   # ties: the upper code
    code = np.where(lo == hi, lo, np.where(lo % 2 == 0, lo, hi))
    code = np.where(np.isnan(v), 0x7F, code)
    return (code | np.where(np.signbit(v) & ~np.isnan(v), 0x80, 0)).astype(np.uint8)


def e4m3_decode(c):
    c = np.asarray(c, np.uint8)
    mag = np.append(E4M3, np.nan)[c & 0x7F]
    return np.where(c & 0x80, -mag, mag)


def _abs_max(x, axis):
    """Largest magnitude, NaN where there is one."""
    return np.max(np.abs(x), axis=axis)  # numpy's maximum hands NaN on


def fp8_rows(x):
    """codes [rows, K], scales [ceil(K/128), rows] of float32 rows."""
    x = np.asarray(x, np.float32)
    rows, K = x.shape
    nb = -(-K // BLOCK)
    p = np.zeros((rows, nb * BLOCK), np.float32)
    p[:, :K] = x
    p = p.reshape(rows, nb, BLOCK)
    with np.errstate(all="ignore"):
        s = np.maximum(_abs_max(p, 2) * np.float32(1 / 448), TINY)
        v = p * (np.float32(1) / s)[:, :, None]
    return e4m3_encode(v).reshape(rows, -1)[:, :K], np.ascontiguousarray(s.T)


def fp8_weights(w):
    """codes [n, N, K], scales [n, ceil(N/128), ceil(K/128)] of w [n, K, N]."""
    w = np.asarray(w, np.float32)
    n, K, N = w.shape
    kb, nb = -(-K // BLOCK), -(-N // BLOCK)
    p = np.zeros((n, nb * BLOCK, kb * BLOCK), np.float32)
    p[:, :N, :K] = w.transpose(0, 2, 1)
    p = p.reshape(n, nb, BLOCK, kb, BLOCK)
    with np.errstate(all="ignore"):
        s = np.maximum(_abs_max(p, (2, 4)) * np.float32(1 / 448), TINY)
        v = p * (np.float32(1) / s)[:, :, None, :, None]
    codes = e4m3_encode(v).reshape(n, nb * BLOCK, kb * BLOCK)[:, :N, :K]
    return np.ascontiguousarray(codes), s


def fp8_row_values(codes, scales):
    K = codes.shape[1]
    with np.errstate(invalid="ignore"):
        return e4m3_decode(codes) * np.repeat(scales.T.astype(np.float64), BLOCK, 1)[:, :K]


def fp8_weight_values(codes, scales):
    """[n, N, K] float64."""
    _, N, K = codes.shape
    s = np.repeat(np.repeat(scales.astype(np.float64), BLOCK, 1)[:, :N], BLOCK, 2)[:, :, :K]
    with np.errstate(invalid="ignore"):
        return e4m3_decode(codes) * s


def silu(g):
    return g / (1 + np.exp(-g))


def grouped(x, w, offsets):
    """x's rows times w [n, N, K] of their expert, and the sum of the products'
    magnitudes; rows past offsets[-1] zero."""
    y = np.zeros((x.shape[0], w.shape[1]))
    mag = np.zeros_like(y)
    for e in range(w.shape[0]):
        a, b = int(offsets[e]), int(offsets[e + 1])
        y[a:b] = x[a:b] @ w[e].T
        mag[a:b] = np.abs(x[a:b]) @ np.abs(w[e]).T
    return y, mag


def ckpt_rows(x):
    """int8 codes [rows, D] and the scales' bf16 bits [rows, D/32]."""
    x = np.asarray(x, np.float32)
    p = x.reshape(x.shape[0], -1, CKPT)
    with np.errstate(all="ignore"):
        s = np.maximum(_abs_max(p, 2) * np.float32(1 / 127), TINY)
        bits = s.view(np.uint32).astype(np.uint64)
        bits = np.where(np.isnan(s), 0x7FC0, (bits + 0xFFFF) >> 16)
        bits = np.where(np.isfinite(s), np.minimum(bits, 0x7C00), bits).astype(np.uint16)
        r = np.float32(1) / bf16_values(bits)
        r = np.where(bits == 0x7C00, np.float32(127 / 128 * 2.0 ** -121), r)
        v = p * r[:, :, None]
        codes = np.where(np.isnan(v), 0, np.rint(v)).astype(np.int8)
    return codes.reshape(x.shape), bits


def bf16_values(bits):
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


def ckpt_values(codes, bits):
    """float32, exact."""
    rows = codes.shape[0]
    with np.errstate(invalid="ignore"):
        return (codes.reshape(rows, -1, CKPT).astype(np.float32)
                * bf16_values(bits)[:, :, None]).reshape(codes.shape)


def swiglu_backward(g, u, dh):
    """dG, dU, H."""
    s = 1 / (1 + np.exp(-g))
    return dh * u * (s + g * s * (1 - s)), dh * g * s, g * s * u


def softmax(z):
    with np.errstate(invalid="ignore"):
        m = z.max(1, keepdims=True)
        e = np.exp(z - np.where(np.isneginf(m), 0, m))
        s = e.sum(1, keepdims=True)
    return np.where(s == 0, 0, e / np.where(s == 0, 1, s))


def balance_loss(z, topk, coef, mask=None):
    """counts, tokens, prob_sum, loss."""
    T, E = z.shape
    on = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    idx = topk[on].ravel()
    counts = np.bincount(idx[(idx >= 0) & (idx < E)], minlength=E)
    N, k = int(on.sum()), topk.shape[1]
    p = softmax(z[on].astype(np.float64)).sum(0) if N else np.zeros(E)
    loss = coef * E / (k * float(N) ** 2) * (counts * p).sum() if N else 0.0
    return counts, N, p, loss


def balance_backward(z, coef, k, counts, tokens, dloss=1.0, mask=None, topk=None, dlogit=None):
    T, E = z.shape
    d = np.zeros((T, E))
    on = np.ones(T, bool) if mask is None else np.asarray(mask) != 0
    if tokens:
        p = softmax(z[on].astype(np.float64))
        f = dloss * coef * E / (k * float(tokens) ** 2) * counts
        d[on] = p * (f - (p * f).sum(1, keepdims=True))
    if topk is not None:
        for t, j in np.ndindex(*topk.shape):
            if 0 <= topk[t, j] < E:
                d[t, topk[t, j]] += dlogit[t, j]
    return d
