"""Rotation at far positions and any frequency, by moe_rope_axes and in
moe_kv_append, against sines and cosines in 64-bit mantissas.

The angle is formed in whole units of 2^-32 of a turn (within one unit of the
exact product, so 2^-29.3 rad) and rounded to fp32 in [-1/2, 1/2] of a turn: by
at most 2^-26 of a turn, 2^-23.3 rad.  The sine and cosine instructions are
within 2^-22.9 there.  A product and the sum add 2^-24 of |u| + |v| each at
most.  In all 2^-22.9 + 2^-23.3 + 2^-29.3 + 2^-23 < 2^-21.4 of |u| + |v|."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_13_amd import moe
from oracle import attention_oracle as AO
from tests import attn_harness as A
from tests import test_gpu_kv_append as K

pytestmark = pytest.mark.gpu

BOUND = 2.0 ** -21.4
FREQS = [1.0, 0.7, 1.0, 0.999, 3.0, 10.0, 64.0, 100.0, 1000.0, 1e4, 1e5, 2.0 ** 32, 1e-4, 2.0 ** -30, 0.0, -0.3]
POSITIONS = {
    "to 2^17": (-(1 << 17), 1 << 17), "below 2^24": ((1 << 24) - 4000, 1 << 24), "above -2^24": (-(1 << 24), 4000 - (1 << 24)),
    "above 2^24": (1 << 24, (1 << 24) + 4000), "any": (-(1 << 31), 1 << 31),
}


def cos_sin(pos, freq):
    """Of each position's product with each frequency: exact in a 64-bit
    mantissa (31 and 24 bits), and rounded there."""
    assert np.finfo(np.longdouble).nmant >= 63
    a = pos.astype(np.longdouble)[:, None] * freq.astype(np.float64).astype(np.longdouble)[None]
    return np.cos(a), np.sin(a)


def rotated(x, pos, freq, il, inverse):
    """x [T, H, D] by one axis; and |u| + |v| (0 where a value passes)."""
    half, D = freq.size, x.shape[2]
    c, s = cos_sin(pos, freq)
    if inverse:
        s = -s
    p = np.arange(half) * 2 if il else np.arange(half)
    q = p + 1 if il else p + half
    y, uv = x.astype(np.longdouble), np.zeros(x.shape)
    u, v = y[:, :, p].copy(), y[:, :, q].copy()
    y[:, :, p], y[:, :, q] = u * c[:, None] - v * s[:, None], v * c[:, None] + u * s[:, None]
    uv[:, :, p] = uv[:, :, q] = np.abs(u) + np.abs(v)
    return y, uv


def some_positions(where, T):
    lo, hi = POSITIONS[where]
    pos = np.random.RandomState(5).randint(lo, hi, T, np.int64)
    pos[:2] = lo, hi - 1
    return pos.astype(np.int32)


@pytest.mark.parametrize("where", list(POSITIONS))
@pytest.mark.parametrize("il,inverse", [(False, False), (True, True)])
def test_far_positions_and_high_frequencies(where, il, inverse):
    T, nH, D = 3000, 2, 48
    freq, pos = np.array(FREQS, np.float32), some_positions(where, T)
    x = A.values((T, nH, D), "f32", 3)
    rot = moe.Rotation(A.i32(pos), torch.from_numpy(freq).cuda(), interleaved=il, inverse=inverse)
    got = A.f64(moe.moe_rope_axes(x.cuda(), rot))
    want, uv = rotated(A.f64(x), pos, freq, il, inverse)
    # the result's own rounding is the sum's
    worst = np.max(np.abs(got - want) / (BOUND * uv + 1e-37), axis=(0, 1))
    print(f"  {where}: {worst.max():.3f} of the bound", flush=True)
    assert (worst <= 1).all(), [float(f"{w:.3g}") for w in worst]


@pytest.mark.parametrize("where", ["below 2^24", "any"])
def test_appended_keys(where):
    """Codes of rotated keys: the nearest, but for quotients within the bound of a midpoint."""
    T, H, D, S = 200, 2, 32, 64
    freq, pos = np.array(FREQS, np.float32), some_positions(where, T)
    rot = moe.Rotation(A.i32(pos), torch.from_numpy(freq).cuda())
    append_and_check(T, H, D, S, rot, pos, freq, [0], A.tables([T], S, 5), where)


@pytest.mark.parametrize("first", [(1 << 24) - 50, (1 << 24) + 3, (1 << 29) + 77])
@pytest.mark.parametrize("axes", [False, True])
def test_own_places_past_24_bits(first, axes):
    """The tokens' own places are rotated as exactly as any other positions."""
    T, H, D, S = 150, 1, 32, 128
    freq = np.array(FREQS, np.float32)
    kv, pages = first + T, 4
    table = np.full((1, -(-kv // S)), -1, np.int32)
    used = range(first // S, -(-kv // S))
    table[0, first // S:] = list(range(pages))[:len(used)]
    pair_axis = torch.zeros(16, dtype=torch.int32, device="cuda") if axes else None
    rot = moe.Rotation(None, torch.from_numpy(freq).cuda(), pair_axis)
    append_and_check(T, H, D, S, rot, np.arange(first, kv), freq, [first], (pages, table), f"places from {first}")


def append_and_check(T, H, D, S, rot, pos, freq, past, pages_table, label):
    P, table = pages_table
    kv, cu = [past[0] + T], [0, T]
    k, v = A.values((T, H, D), "f32", 7), A.values((T, H, D), "f32", 8)
    old = A.random_cache(P, H, S, D, 6, pow2=True)
    cache = A.device_cache(old)
    moe.moe_kv_append(cache, k.cuda(), v.cuda(), A.i32(kv), A.i32(table), rotation=rot, cu_q=A.i32(cu))
    torch.cuda.synchronize()
    krot, uv = rotated(A.f64(k), pos, freq, False, False)
    touched = []
    want = AO.append(old, krot.astype(np.float64), A.f64(v), cu, kv, table, touched)
    K.check(A.host_cache(cache), want, krot.astype(np.float64), uv, touched, label)
