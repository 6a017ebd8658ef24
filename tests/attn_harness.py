"""Inputs and tolerances shared by the tests of the rotation, the paged cache
append and the attention over it."""
import numpy as np
import torch

from mixture_experts_layer_13_amd import moe
from oracle import attention_oracle as AO

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


def gen(seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return g


def values(shape, dtype, seed, std=1.0):
    return (torch.randn(shape, generator=gen(seed)) * std).to(DT[dtype])


def f64(t):
    return t.detach().cpu().double().numpy()


def inv_freq(R, base=10000.0):
    return torch.tensor(base ** (-np.arange(0, R, 2, dtype=np.float64) / R), dtype=torch.float32)


def offsets(q):
    return np.concatenate([[0], np.cumsum(q)]).astype(np.int32)


def i32(a, device=DEV):
    return torch.as_tensor(np.asarray(a, np.int32), device=device)


def tables(kv, S, seed, extra_pages=3, extra_columns=0):
    """(pages, table): distinct pages in no order, -1 past a sequence's end."""
    need = [-(-n // S) if n > 0 else 0 for n in kv]
    r = np.random.RandomState(seed)
    pages = sum(need) + extra_pages
    ids = r.permutation(pages)
    table = np.full((len(kv), max(max(need, default=0), 1) + extra_columns), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return pages, table


def random_cache(P, H, S, D, seed, pow2=False):
    """Codes of finite values and scales of all sizes between 2^-7 and 2^-3."""
    r = np.random.RandomState(seed)
    c = {"k_codes": r.randint(0, 256, (P, H, S, D)).astype(np.uint8),
         "v_codes": r.randint(0, 256, (P, H, S // 16, D, 16)).astype(np.uint8)}
    for n in c:
        c[n][(c[n] & 127) == 127] ^= 1
        c[n][(c[n] & 127) > 100] &= 0x9F  # few of the largest
    for n in ("k_scales", "v_scales"):
        e = r.uniform(-7, -3, (P, H))
        c[n] = np.exp2(np.round(e) if pow2 else e).astype(np.float32)
    return c


def poison_unseen(cache, kv, table, q, window=0):
    """NaN codes and NaN scales wherever no row of any sequence looks."""
    P, H, S, D = cache["k_codes"].shape
    seen = np.zeros((P, S), bool)
    for b, n in enumerate(kv):
        lo = max(0, n - q[b] - window + 1) if window else 0
        if q[b] > 0:
            for t in range(lo, max(n, 0)):
                if t // S < table.shape[1] and 0 <= table[b, t // S] < P:
                    seen[table[b, t // S], t % S] = True
    for p in range(P):
        for s in range(S):
            if not seen[p, s]:
                cache["k_codes"][p, :, s] = 0x7F
                cache["v_codes"][p, :, s // 16, :, s % 16] = 0xFF
        if not seen[p].any():
            cache["k_scales"][p] = np.nan
            cache["v_scales"][p] = np.nan
    return cache


def device_cache(c):
    t = {n: torch.from_numpy(a.copy()).to(DEV) for n, a in c.items()}
    return moe.PagedKV(t["k_codes"], t["v_codes"], t["k_scales"], t["v_scales"])


def host_cache(kv):
    return {n: getattr(kv, n).view(torch.uint8).cpu().numpy() if "codes" in n else getattr(kv, n).cpu().numpy()
            for n in ("k_codes", "v_codes", "k_scales", "v_scales")}


def check_attention(out, lse, ref, dtype, D, label):
    """Bounds by arithmetic.  u = 2^-24.  A score is a sum of D exact products
    in fp32 (at most D + 2 roundings of partial sums of size at most `reach`,
    and two of the scaling), so off by at most e = (D + 6) u reach; with the
    maximum subtracted and the hardware base-2 exponential (1 ulp, argument
    rounded: 2 u reach) every p is off by a factor within 2 e + 8 u.  Numerator
    and denominator are fp32 sums over `seen` tokens: (seen + 8) u each.  bf16
    queries: x = p vs over the row's largest p vs (`heavy`) is rounded to fp16,
    by at most 2^-11 of itself, or 2^-32 where it is below 2^-21, which makes
    at most seen 448 2^-32 heavy of the output; that is rounded by 2^-8.  fp32
    queries: 24 bits of p and of the output (u)."""
    o64, l64, (reach, mass, seen, heavy) = ref
    live = ~np.isnan(l64)
    u = 2.0 ** -24
    e = (D + 6) * u * reach
    rel = 2 * (2 * e + 8 * u) + 2 * (seen + 8) * u
    h = HALF_STEP[dtype]
    p = 2.0 ** -11 if dtype == "bf16" else h
    floor = (seen * 448 * 2.0 ** -32 * heavy if dtype == "bf16" else 0 * seen)[:, :, None]
    tol = ((rel + p)[:, :, None] * mass + floor) * (1 + h) + h * np.abs(o64) + 1e-30
    got, glse = f64(out), f64(lse)
    assert np.isfinite(got[live]).all(), label
    worst = np.max((np.abs(got - o64) / tol)[live], initial=0.0)
    assert worst <= 1.0, (label, "out", worst)
    empty = np.isneginf(l64) & live
    assert np.isneginf(glse[empty]).all() and (got[empty] == 0).all(), label
    full = live & ~empty
    ltol = 2 * e + (seen + 16) * u + 8 * u * (np.abs(np.where(full, l64, 0)) + 1)
    lworst = np.max((np.abs(np.where(full, glse - np.where(full, l64, 0), 0)) / ltol)[full], initial=0.0)
    assert lworst <= 1.0, (label, "lse", lworst)
    print(f"  {label}: out {worst:.3f}, lse {lworst:.3f} of their bounds", flush=True)
