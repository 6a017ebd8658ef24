"""Dispatch, combine, block quantisation and block-scaled products in 64 bits
(numpy), written from the definitions, pair by pair and block by block."""
import numpy as np

E4M3_MAX = 448.0


def e4m3_values():
    """What the 256 E4M3 codes stand for."""
    n = np.arange(256)
    e, f = (n >> 3) & 15, (n & 7).astype(np.float64)
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7.0))
    v = np.where((n & 127) == 127, np.nan, v)
    return np.where(n >= 128, -v, v)


def e4m3_code(q):
    """Codes of float32 quotients: nearest even, saturating, NaN 0x7f."""
    q = np.asarray(q, np.float32).astype(np.float64)
    a = np.minimum(np.where(np.isnan(q), 0, np.abs(q)), E4M3_MAX)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -20))), -6)
    step = 2.0 ** (e - 3)
    a = np.minimum(np.rint(a / step) * step, E4M3_MAX)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -20))), -6)
    low = a < 2.0 ** -6
    code = np.where(low, a * 2.0 ** 9, (e + 7) * 8 + (a / 2.0 ** e - 1) * 8).astype(np.int64)
    code = np.where(np.isnan(q), 127, code | np.where(np.signbit(q), 128, 0))
    return code.astype(np.uint8)


def block_scale(x, axis):
    """max(fl32(amax / 448), 2^-126) over the finite magnitudes, 1 if there is none."""
    a = np.where(np.isfinite(x), np.abs(x), 0).max(axis, initial=0).astype(np.float32)
    s = np.maximum(a / np.float32(E4M3_MAX), np.float32(2.0 ** -126))
    return np.where(a == 0, np.float32(1), s).astype(np.float32)


def quantize(x, block_rows=1):
    """x float32 [M, K] -> (codes, scales [row blocks, blocks])."""
    x = np.asarray(x, np.float32)
    M, K = x.shape
    SR, SB = -(-M // block_rows), -(-K // 128)
    codes, scales = np.zeros((M, K), np.uint8), np.zeros((SR, SB), np.float32)
    for i in range(SR):
        r = slice(i * block_rows, (i + 1) * block_rows)
        for b in range(SB):
            c = slice(b * 128, b * 128 + 128)
            scales[i, b] = block_scale(x[r, c], None)
            with np.errstate(invalid="ignore"):
                codes[r, c] = e4m3_code(x[r, c] / scales[i, b])
    return codes, scales


def gated(x):
    g, u = np.split(np.asarray(x, np.float64), 2, 1)
    return g / (1 + np.exp(-g)) * u


def matmul(a, a_scales, w, w_scales):
    """(out, cut, mass): the product in 64 bits; what the E4M3 instructions may
    cut off it (7 of each group of 8 products, by up to 2^-13 of the largest);
    the sum of the products' magnitudes."""
    v = e4m3_values()
    A, W = v[a], v[w]
    M, K = A.shape
    N = W.shape[0]
    out, cut, mass = np.zeros((M, N)), np.zeros((M, N)), np.zeros((M, N))
    rows = np.arange(N) // 128
    for b in range(-(-K // 128)):
        c = slice(b * 128, min(K, b * 128 + 128))
        s = a_scales[:, b, None].astype(np.float64) * w_scales[rows, b].astype(np.float64)
        out += s * (A[:, c] @ W[:, c].T)
        mass += np.abs(s) * (np.abs(A[:, c]) @ np.abs(W[:, c]).T)
        for k in range(c.start, c.stop, 8):
            top = np.zeros((M, N))
            for i in range(k, k + 8):
                top = np.maximum(top, np.abs(A[:, i, None] * W[:, i]))
            cut += np.abs(s) * 7 * 2.0 ** -13 * top
    return out, cut, mass


def dispatch(x, pos, topk, rows, weights=None):
    out = np.zeros((rows, x.shape[1]))
    for f, p in enumerate(pos):
        if 0 <= p < rows:
            out[p] = x[f // topk] * (1.0 if weights is None else weights.reshape(-1)[f])
    return out


def combine(rows, pos, topk, M, weights=None):
    """(out, mass)."""
    out, mass = np.zeros((M, rows.shape[1])), np.zeros((M, rows.shape[1]))
    for f in range(M * topk):
        if 0 <= pos[f] < len(rows):
            y = rows[pos[f]] * (1.0 if weights is None else weights.reshape(-1)[f])
            out[f // topk] += y
            mass[f // topk] += np.abs(y)
    return out, mass


def pair_dots(x, rows, pos, topk):
    """(<token, row> of each pair, mass); 0 without a place."""
    out, mass = np.zeros((len(x), topk)), np.zeros((len(x), topk))
    for f in range(len(x) * topk):
        if 0 <= pos[f] < len(rows):
            p = x[f // topk] * rows[pos[f]]
            out.reshape(-1)[f], mass.reshape(-1)[f] = p.sum(), np.abs(p).sum()
    return out, mass
