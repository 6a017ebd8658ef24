"""fp64 oracle of the rotation, the paged E4M3 cache append and the attention
over it (test infrastructure): plain numpy, token by token and head by head,
sharing nothing with the GPU library.  Caches are dicts of numpy arrays laid
out as include/moe.h documents: k_codes [P, H, S, D] and v_codes
[P, H, S/16, D, 16] uint8, k_scales and v_scales f32 [P, H]."""
import numpy as np

E4M3_MAX = 448.0
MIN_SCALE, MAX_SCALE = 2.0 ** -64, 2.0 ** 48


def _table():
    v = np.zeros(256)
    for n in range(256):
        e, f = (n >> 3) & 15, n & 7
        v[n] = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        if n & 127 == 127:
            v[n] = np.nan
        if n & 128:
            v[n] = -v[n]
    return v


E4M3 = _table()
_MAGS = E4M3[:127]
MIDS = (_MAGS[1:] + _MAGS[:-1]) / 2


def e4m3_codes(x):
    """Nearest E4M3 code of each x, ties to the even code, saturating."""
    a = np.minimum(np.abs(x), E4M3_MAX)
    low = np.searchsorted(MIDS, a, side="left")   # a tie stays below
    high = np.searchsorted(MIDS, a, side="right")
    n = np.where(low % 2 == 0, low, high)
    return (n + np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def angles(positions, inv_freq, pair_axis, inverse):
    """[T, R/2] angles; a pair of no axis turns by 0."""
    axes, T = positions.shape
    a = np.zeros((T, inv_freq.size))
    for i, f in enumerate(inv_freq.astype(np.float64)):
        ax = 0 if pair_axis is None else int(pair_axis[i])
        if 0 <= ax < axes:
            a[:, i] = positions[ax].astype(np.float64) * f
    return -a if inverse else a


def rotate(x, positions, inv_freq, pair_axis=None, interleaved=False, inverse=False):
    """x [T, H, D] (any float) rotated, in fp64."""
    y = x.astype(np.float64).copy()
    half = inv_freq.size
    a = angles(positions, inv_freq, pair_axis, inverse)
    for i in range(half):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, half + i)
        c, s = np.cos(a[:, i])[:, None], np.sin(a[:, i])[:, None]
        u, v = y[:, :, p].copy(), y[:, :, q].copy()
        y[:, :, p], y[:, :, q] = u * c - v * s, v * c + u * s
    return y


def pair_of(D, half, interleaved):
    """The other member of each value's pair (itself where it is not rotated)."""
    d = np.arange(D)
    if interleaved:
        return np.where(d < 2 * half, d ^ 1, d)
    return np.where(d < half, d + half, np.where(d < 2 * half, d - half, d))


def page_scale(amax):
    s = MIN_SCALE
    while E4M3_MAX * s < amax and s < MAX_SCALE:
        s *= 2
    return s


def _v_slot(cache, page, h, slot):
    return cache["v_codes"][page, h, slot // 16, :, slot % 16]


def append(cache, k, v, cu, kv_lens, table, touched=None):
    """k, v [T, H, D] fp64 (k rotated) into a copy of the cache.  touched, if a
    list, gets (page, head, slot, row) of every new token."""
    c = {n: a.copy() for n, a in cache.items()}
    P, H, S, D = c["k_codes"].shape
    for b in range(len(kv_lens)):
        rows = cu[b + 1] - cu[b]
        start = int(kv_lens[b]) - rows
        by_page = {}
        for i in range(rows):
            t = start + i
            if t >= 0 and t // S < table.shape[1] and 0 <= table[b, t // S] < P:
                by_page.setdefault(t // S, []).append((t % S, cu[b] + i))
        for n, got in by_page.items():
            page, old = int(table[b, n]), got[0][0]
            for name, x in (("k", k), ("v", v)):
                for h in range(H):
                    vals = np.abs(np.stack([x[r, h] for _, r in got]))
                    vals = vals[np.isfinite(vals)]
                    s = page_scale(vals.max() if vals.size else 0.0)
                    if old:
                        was = float(c[name + "_scales"][page, h])
                        s = max(s, was)
                        if s != was:
                            for slot in range(old):
                                at = c["k_codes"][page, h, slot] if name == "k" else _v_slot(c, page, h, slot)
                                at[:] = e4m3_codes(E4M3[at] * (was / s))
                    c[name + "_scales"][page, h] = s
                    for slot, r in got:
                        at = c["k_codes"][page, h, slot] if name == "k" else _v_slot(c, page, h, slot)
                        at[:] = e4m3_codes(x[r, h] / s)
                        if touched is not None and name == "k":
                            touched.append((page, h, slot, r))
    return c


def gather(cache, table_row, n, h, hidden):
    """Keys and values [n, D] of a sequence's tokens in fp64, and the values'
    scales [n]; hidden[t] for tokens of no page."""
    P, H, S, D = cache["k_codes"].shape
    k, v, vs = np.zeros((n, D)), np.zeros((n, D)), np.zeros(n)
    for t in range(n):
        page = int(table_row[t // S]) if t // S < len(table_row) else -1
        if not 0 <= page < P:
            hidden[t] = True
            continue
        k[t] = E4M3[cache["k_codes"][page, h, t % S]] * float(cache["k_scales"][page, h])
        vs[t] = float(cache["v_scales"][page, h])
        v[t] = E4M3[_v_slot(cache, page, h, t % S)] * vs[t]
    return k, v, vs


def attention(cache, q, cu, kv_lens, table, scale, causal=True, window=0):
    """(out [T, nH, D], lse [T, nH], bound) in fp64; rows of no sequence are
    NaN.  bound: per row, the largest scale * sum |q||k| over the tokens it
    sees, sum p|v| per value, how many it sees, and the largest p times its
    value's scale."""
    T, nH, D = q.shape
    H, S = cache["k_codes"].shape[1], cache["k_codes"].shape[2]
    G = nH // H
    out, lse = np.full((T, nH, D), np.nan), np.full((T, nH), np.nan)
    reach, mass, seen, heavy = np.zeros((T, nH)), np.zeros((T, nH, D)), np.zeros((T, nH)), np.zeros((T, nH))
    q = q.astype(np.float64)
    for b in range(len(kv_lens)):
        n = min(max(int(kv_lens[b]), 0), table.shape[1] * S)
        rows = cu[b + 1] - cu[b]
        pos = (max(int(kv_lens[b]), 0) - rows + np.arange(rows))[:, None]
        t = np.arange(n)[None]
        for h in range(H):
            hidden = np.zeros(n, bool)
            with np.errstate(invalid="ignore"):
                k, v, vs = gather(cache, table[b], n, h, hidden)
            sees = np.broadcast_to(~hidden[None], (rows, n)).copy()
            if causal:
                sees &= t <= pos
            if window:
                sees &= t > pos - window
            used = sees.any(0)
            k[~used], v[~used], vs[~used] = 0.0, 0.0, 0.0
            for g in range(h * G, h * G + G):
                x = q[cu[b]:cu[b + 1], g]
                with np.errstate(invalid="ignore", divide="ignore"):
                    s = np.where(sees, x @ k.T * scale, -np.inf)
                    top = s.max(1, initial=-np.inf)
                    p = np.exp(s - np.where(np.isneginf(top), 0.0, top)[:, None])
                    total = p.sum(1)
                    p = p / np.where(total == 0, 1.0, total)[:, None]
                    out[cu[b]:cu[b + 1], g] = p @ v
                    lse[cu[b]:cu[b + 1], g] = np.where(total == 0, -np.inf, np.log(total) + top)
                mass[cu[b]:cu[b + 1], g] = p @ np.abs(v)
                reach[cu[b]:cu[b + 1], g] = np.where(sees, np.abs(x) @ np.abs(k).T * abs(scale), 0).max(1, initial=0)
                seen[cu[b]:cu[b + 1], g] = sees.sum(1)
                heavy[cu[b]:cu[b + 1], g] = (p * vs).max(1, initial=0)
    return out, lse, (reach, mass, seen, heavy)
