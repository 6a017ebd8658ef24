"""Inputs and tolerances shared by the tests of dispatch, combine, block
quantisation and block-scaled products."""
import numpy as np
import torch

from mixture_experts_layer_13_amd import moe
from oracle import blocks_oracle as BO

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
U = 2.0 ** -24


def f64(t):
    return t.detach().cpu().double().numpy()


def values(shape, dtype, seed):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(shape, generator=g).to(DT[dtype])


def aligned(M, topk, E, block_m, seed, keep=1.0):
    """Random expert ids (distinct in a token; a share dropped, -1) through the
    library's alignment: (ids, Alignment, places of the pairs, rows in use)."""
    r = np.random.RandomState(seed)
    ids = np.stack([r.permutation(E)[:topk] for _ in range(M)]) if M else np.zeros((0, topk), int)
    ids[r.rand(M, topk) >= keep] = -1
    t = torch.from_numpy(ids.astype(np.int32)).to(DEV)
    p = moe.make_problem(M, 128, 128, E, topk, block_m, torch.bfloat16, torch.bfloat16, torch.bfloat16)
    ws = torch.empty(max(moe.moe_workspace_size(p), 16), dtype=torch.uint8, device=DEV)
    al = moe.moe_align_permute(t, E, block_m, ws)
    torch.cuda.synchronize()
    return ids, al, al.pair_pos.cpu().numpy()[:M * topk], int(al.num_padded.item())


def strided(t, extra):
    """t [rows, K] as a slice of rows that are `extra` values wider, NaN there."""
    if not extra:
        return t
    wide = torch.full((t.shape[0], t.shape[1] + extra), float("nan"), dtype=t.dtype, device=t.device)
    wide[:, :t.shape[1]] = t
    return wide[:, :t.shape[1]]


def within(got, want, tol, label):
    got = f64(got) if torch.is_tensor(got) else got
    assert got.shape == want.shape, label
    assert np.isfinite(got).all(), label
    worst = np.max(np.abs(got - want) / (tol + 1e-300), initial=0.0)
    assert worst <= 1.0, (label, worst)
    print(f"  {label}: {worst:.3f} of its bound", flush=True)


def codes(shape, seed):
    """Random finite E4M3 codes of all sizes."""
    c = np.random.RandomState(seed).randint(0, 256, shape).astype(np.uint8)
    c[(c & 127) == 127] ^= 1
    return c


def scales(shape, seed):
    """Scales between 2^-12 and 2^4."""
    return np.exp2(np.random.RandomState(seed).uniform(-12, 4, shape)).astype(np.float32)


def product_bound(out, cut, mass, dtype, K):
    """A block's sum, beyond what the E4M3 instructions cut (bf16 results only;
    fp32 ones have bf16 products added in fp32), has at most 128 roundings of
    partial sums no larger than the mass; then come the two scales' product, one
    rounding a block, and the result's own."""
    n = 128 + 3 + -(-K // 128)
    return (cut if dtype == "bf16" else 0) + n * U * mass + HALF_STEP[dtype] * np.abs(out) * (1 + 2.0 ** -7) + 1e-38


def fp8(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV).view(torch.float8_e4m3fn)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)
