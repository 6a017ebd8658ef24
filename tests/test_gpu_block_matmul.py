"""Block-scaled E4M3 products against the 64-bit oracle (bounds in
tests/block_harness.py)."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_13_amd import moe
from oracle import blocks_oracle as BO
from tests import block_harness as B

pytestmark = pytest.mark.gpu

SIZES = [(1, 1, 16), (1, 16, 128), (1, 200, 4096), (2, 129, 144), (16, 64, 256), (17, 300, 400), (32, 128, 1024), (33, 96, 2000),
         (61, 520, 336), (64, 256, 128), (65, 250, 384), (100, 33, 640), (128, 128, 128), (129, 257, 272), (200, 640, 1040),
         (300, 513, 512), (520, 770, 528), (1, 3, 65536)]


def operands(M, N, K, seed, E=None):
    a, w = B.codes((M, K), seed), B.codes((N, K) if E is None else (E, N, K), seed + 1)
    sa = B.scales((M, -(-K // 128)), seed + 2)
    sw = B.scales((*w.shape[:-2], -(-N // 128), -(-K // 128)), seed + 3)
    return a, sa, w, sw


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul(M, N, K, dt):
    a, sa, w, sw = operands(M, N, K, M + N + K)
    out = moe.moe_block_matmul(B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw), out_dtype=B.DT[dt])
    assert out.dtype == B.DT[dt]
    ref = BO.matmul(a, sa, w, sw)
    B.within(out, ref[0], B.product_bound(*ref, dt, K), f"{M} x {N} x {K} {dt}")


@pytest.mark.parametrize("M", [5, 50, 200])
def test_strides(M):
    """Rows of a, of out and scales that are slices of something wider, NaN
    around them; scales by token and by block."""
    N, K = 200, 400
    a, sa, w, sw = operands(M, N, K, 1)
    want = moe.moe_block_matmul(B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw))
    wide = torch.full((M, K + 48), 0x7F, dtype=torch.uint8, device=B.DEV)
    wide[:, :K] = B.dev(a)
    for s in (B.dev(sa.T).t(), B.strided(B.dev(sa), 3), B.dev(sa)):
        out = torch.full((M, N + 24), 5.0, dtype=torch.bfloat16, device=B.DEV)
        got = moe.moe_block_matmul(wide[:, :K], s, B.fp8(w), B.dev(sw), out=out[:, :N])
        assert torch.equal(got, want) and (out[:, N:] == 5).all()
    # rows that are not a multiple of 16 bytes apart
    out = torch.full((M, N + 1), 5.0, dtype=torch.bfloat16, device=B.DEV)
    assert torch.equal(moe.moe_block_matmul(B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw), out=out[:, :N]), want)
    assert (out[:, N:] == 5).all()


@pytest.mark.parametrize("M", [3, 40, 150])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_nan_codes_stay_in_their_rows_and_columns(M, dt):
    N, K = 150, 272
    a, sa, w, sw = operands(M, N, K, 2)
    a[1, 270], w[7, 3] = 0x7F, 0xFF
    out = moe.moe_block_matmul(B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw), out_dtype=B.DT[dt])
    bad = torch.isnan(out).cpu().numpy()
    want = np.zeros((M, N), bool)
    want[1], want[:, 7] = True, True
    assert np.array_equal(bad, want)


@pytest.mark.parametrize("M", [3, 150])
def test_what_lies_behind_a_row_is_not_used(M):
    """K inside a block of 128: the bytes after a row are the next row's."""
    N, K = 130, 144
    a, sa, w, sw = operands(M, N, K, 3)
    want = moe.moe_block_matmul(B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw))
    a2, w2 = a.copy(), w.copy()
    a2[1::2], w2[1::2] = 0x7F, 0x7F
    got = moe.moe_block_matmul(B.fp8(a2), B.dev(sa), B.fp8(w2), B.dev(sw))
    assert torch.equal(got[::2, ::2], want[::2, ::2])


def test_scales_of_zero_and_negative():
    a, sa, w, sw = operands(70, 140, 256, 4)
    sa[3], sw[1, 0], sa[5] = 0, -sw[1, 0], -sa[5]
    out = moe.moe_block_matmul(B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw), out_dtype=torch.float32)
    ref = BO.matmul(a, sa, w, sw)
    B.within(out, ref[0], B.product_bound(*ref, "f32", 256), "zero and negative scales")
    assert (out[3] == 0).all()


def test_no_rows():
    a, sa, w, sw = operands(4, 64, 128, 4)
    assert moe.moe_block_matmul(B.fp8(a)[:0], B.dev(sa)[:0], B.fp8(w), B.dev(sw)).shape == (0, 64)


@pytest.mark.parametrize("M,N", [(40, 128), (300, 256)])
def test_the_gradient_is_the_product_with_the_transposed_weights(M, N):
    """d(sum(out * g)) / da = g w with scales of both, as a second product."""
    K = 384
    _, _, w, sw = operands(1, N, K, 5)
    g = B.codes((M, N), 8)
    sg = B.scales((M, N // 128), 9)
    wt = np.ascontiguousarray(w.T)
    out = moe.moe_block_matmul(B.fp8(g), B.dev(sg), B.fp8(wt), B.dev(np.ascontiguousarray(sw.T)), out_dtype=torch.float32)
    v = BO.e4m3_values()
    W = v[w] * np.kron(sw.astype(np.float64), np.ones((128, 128)))
    G = v[g] * np.repeat(sg.astype(np.float64), 128, 1)
    B.within(out, G @ W, (N + 8) * B.U * (np.abs(G) @ np.abs(W)), "gradient")


#           M    topk E  bm   N    K    keep gather
GROUPED = [(1, 1, 1, 16, 64, 128, 1.0, True), (1, 8, 8, 16, 200, 400, 1.0, True), (8, 2, 4, 16, 128, 256, 1.0, False),
           (64, 4, 16, 16, 136, 272, 1.0, True), (40, 3, 5, 32, 96, 528, 0.7, True), (150, 2, 3, 64, 264, 144, 0.8, False),
           (150, 2, 3, 16, 264, 144, 0.8, True), (200, 4, 6, 128, 130, 256, 1.0, True), (300, 2, 4, 256, 257, 384, 0.6, True),
           (600, 2, 3, 256, 128, 272, 1.0, False), (20, 2, 6, 64, 72, 144, 0.0, True), (500, 6, 9, 32, 80, 128, 1.0, True)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,k,E,bm,N,K,keep,gather", GROUPED)
def test_grouped(M, k, E, bm, N, K, keep, gather, dt):
    ids, al, pos, n = B.aligned(M, k, E, bm, M + N, keep)
    R = al.sorted_pair_ids.numel()
    a, sa, w, sw = operands(M if gather else R, N, K, M + N + K, E)
    sorted_ids = al.sorted_pair_ids.cpu().numpy()
    if not gather:  # what lies in padding rows, and behind, is not looked at
        pad = np.ones(R, bool)
        pad[pos[pos >= 0]] = False
        a[pad], sa[pad] = 0x7F, np.nan
    out = torch.full((R, N), 3.0, dtype=B.DT[dt], device=B.DEV)
    got = moe.moe_block_matmul_grouped(B.fp8(a), B.dev(sa.T).t(), B.fp8(w), B.dev(sw), al, topk=k if gather else None, out=out)
    assert got is out
    off = al.expert_offsets.cpu().numpy()
    want, tol = np.zeros((R, N)), np.zeros((R, N))
    for e in range(E):
        p = np.arange(off[e], off[e + 1])
        p = p[sorted_ids[p] < M * k]
        if len(p):
            at = sorted_ids[p] // k if gather else p
            ref = BO.matmul(a[at], sa[at], w[e], sw[e])
            want[p], tol[p] = ref[0], B.product_bound(*ref, dt, K)
    B.within(out[:n], want[:n], tol[:n], "grouped")
    pad = np.ones(n, bool)
    pad[pos[pos >= 0]] = False
    assert (out[:n].cpu().float().numpy()[pad] == 0).all() and (out[n:] == 3).all()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("bm", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("M,k,E", [(1, 1, 65), (30, 3, 64), (40, 4, 130), (260, 6, 70), (500, 8, 66), (9, 8, 1024)])
def test_many_experts(M, k, E, bm, gather):
    """More experts than a wave has lanes, most of them with few rows or none, in
    blocks shorter and longer than the kernels' spans."""
    test_grouped(M, k, E, bm, 40, 144, 0.9, gather, "bf16")


def on_gpu(a, sa, w, sw):
    """The product and the magnitudes' sum in 64 bits, block by block on the GPU."""
    v = torch.from_numpy(BO.e4m3_values()).to(B.DEV)
    out = torch.zeros(a.shape[0], w.shape[0], dtype=torch.float64, device=B.DEV)
    mass = torch.zeros_like(out)
    rows = torch.arange(w.shape[0], device=B.DEV) // 128
    for b in range(sw.shape[1]):
        c = slice(b * 128, b * 128 + 128)
        x = v[a[:, c].long()] * sa[:, b, None].double()
        y = (v[w[:, c].long()] * sw[rows, b, None].double()).t().contiguous()
        out += x @ y
        mass += x.abs() @ y.abs()
    return out, mass


def near(got, out, mass, dt, K):
    """As product_bound, with all of a group's magnitudes for its largest."""
    n = 128 + 3 + -(-K // 128)
    tol = ((7 * 2.0 ** -13 if dt == "bf16" else 0) + n * B.U) * mass + B.HALF_STEP[dt] * out.abs() * (1 + 2.0 ** -7) + 1e-38
    worst = ((got.double() - out).abs() / tol).max().item()
    assert worst <= 1, worst


LARGE = [(1000, 4000, "bf16"), (2000, 4010, "bf16"), (4000, 4090, "bf16"), (4097, 4104, "bf16"), (300, 4001, "bf16"),
         (600, 4000, "bf16"), (1000, 4001, "f32"), (2500, 4004, "f32"), (700, 3000, "f32")]


@pytest.mark.parametrize("K", [16, 144, 272, 656])
@pytest.mark.parametrize("M,N,dt", LARGE)
def test_large(M, N, dt, K):
    """Sizes for each of the tile kernels, their blocks from one on, odd and even."""
    a, sa, w, sw = (B.dev(x) for x in operands(M, N, K, M + K))
    got = moe.moe_block_matmul(a, sa.t().contiguous().t(), w, sw, out_dtype=B.DT[dt])
    near(got, *on_gpu(a, sa, w, sw), dt, K)


@pytest.mark.parametrize("K", [1536, 1552, 1680, 1920, 4000])
@pytest.mark.parametrize("M,N", [(200, 4000), (70, 4001), (500, 4090), (1000, 4004), (1000, 4001), (1037, 1544)])
def test_long_k_in_fp32(M, N, K):
    """Sizes whose blocks along K are shared out, evenly and unevenly."""
    test_large(M, N, "f32", K)


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("M,k,E,bm,N,K,keep,dt", [
    (3000, 2, 3, 256, 2100, 272, 1.0, "bf16"), (3000, 2, 3, 16, 2100, 144, 0.9, "bf16"), (5000, 4, 5, 128, 1030, 400, 0.7, "bf16"),
    (900, 8, 64, 256, 520, 272, 1.0, "bf16"), (900, 8, 64, 16, 520, 272, 0.3, "bf16"), (2000, 2, 4, 64, 2100, 272, 1.0, "f32"),
    (700, 1, 2, 128, 4100, 528, 1.0, "f32")])
def test_grouped_large(M, k, E, bm, N, K, keep, dt, gather):
    ids, al, pos, n = B.aligned(M, k, E, bm, M + N, keep)
    R = al.sorted_pair_ids.numel()
    a, sa, w, sw = (B.dev(x) for x in operands(M if gather else R, N, K, M + N + K, E))
    out = torch.full((R, N), 3.0, dtype=B.DT[dt], device=B.DEV)
    if not gather:
        pad = torch.ones(R, dtype=torch.bool, device=B.DEV)
        pad[torch.from_numpy(pos[pos >= 0]).to(B.DEV).long()] = False
        a[pad], sa[pad] = 0x7F, float("nan")
    moe.moe_block_matmul_grouped(a, sa.t().contiguous().t(), w, sw, al, topk=k if gather else None, out=out)
    off = al.expert_offsets.cpu().numpy()
    for e in range(E):
        p = torch.arange(off[e], off[e + 1], device=B.DEV)
        f = al.sorted_pair_ids[p].long()
        real = f < M * k
        assert (out[p[~real]] == 0).all()
        if real.any():
            at = f[real] // k if gather else p[real]
            near(out[p[real]], *on_gpu(a[at], sa[at], w[e], sw[e]), dt, K)
    assert (out[n:] == 3).all()


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("M,k,E,bm,N,K", [(700, 1, 3, 64, 1000, 1680), (900, 2, 4, 256, 1001, 1552), (1500, 2, 3, 16, 2050, 1920)])
def test_grouped_long_k_in_fp32(M, k, E, bm, N, K, gather):
    test_grouped_large(M, k, E, bm, N, K, 0.9, "f32", gather)


def test_grouped_rows_trimmed_and_odd_strides():
    M, k, E, bm, N, K = 90, 2, 5, 32, 65, 144
    ids, al, pos, n = B.aligned(M, k, E, bm, 4)
    a, sa, w, sw = operands(M, N, K, 7, E)
    args = (B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw))
    want = moe.moe_block_matmul_grouped(*args, al, topk=k)
    for rows in (n, n - 17, 1):
        cut = moe.Alignment(al.sorted_pair_ids[:rows].clone(), al.block_expert_ids, al.expert_offsets, al.pair_pos,
                            al.num_padded, bm)
        out = torch.full((rows + 3, N + 2), 3.0, dtype=torch.bfloat16, device=B.DEV)
        moe.moe_block_matmul_grouped(*args, cut, topk=k, out=out[:rows, :N])
        assert torch.equal(out[:rows, :N], want[:rows])
        assert (out[rows:] == 3).all() and (out[:, N:] == 3).all()


@pytest.mark.parametrize("bm", [16, 128])
def test_grouped_buffers_made_for_more_tokens(bm):
    """An alignment's buffers used again for fewer tokens: their padding marks are
    fewer pairs than the buffers hold."""
    M, k, E, N, K = 30, 2, 4, 96, 144
    big = moe.alloc_alignment(200, k, E, bm, B.DEV)
    ids, al, pos, n = B.aligned(M, k, E, bm, 5)
    ws = torch.empty(moe.moe_workspace_size(moe.make_problem(M, 128, 128, E, k, bm, *[torch.bfloat16] * 3)), dtype=torch.uint8,
                     device=B.DEV)
    moe.moe_align_permute(B.dev(ids.astype(np.int32)), E, bm, ws, alignment=big)
    R = big.sorted_pair_ids.numel()
    a, sa, w, sw = operands(R, N, K, 3, E)
    want = moe.moe_block_matmul_grouped(B.fp8(a)[:al.sorted_pair_ids.numel()], B.dev(sa)[:al.sorted_pair_ids.numel()], B.fp8(w),
                                        B.dev(sw), al)
    got = moe.moe_block_matmul_grouped(B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw), big, pairs=M * k)
    assert torch.equal(got[:n], want[:n])
    pad = np.ones(n, bool)
    pad[pos[pos >= 0]] = False
    assert pad.any() and (got[:n].cpu().float().numpy()[pad] == 0).all()
    tok = moe.moe_block_matmul_grouped(B.fp8(a)[:200], B.dev(sa)[:200], B.fp8(w), B.dev(sw), big, topk=k, M=M)
    assert (tok[:n].cpu().float().numpy()[pad] == 0).all()


def test_results_repeat_and_streams():
    a, sa, w, sw = operands(300, 512, 1024, 6)
    args = (B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw))
    want = moe.moe_block_matmul(*args)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(3)]
    got = [moe.moe_block_matmul(*args, stream=q) for q in s]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


def test_offsets_past_32_bits():
    """An output of more than 2^31 values, and weights of more than 2^31 bytes."""
    M, N, K = 70000, 32768, 128
    a = torch.randint(0, 100, (M, K), dtype=torch.uint8, device=B.DEV)
    w = torch.randint(0, 100, (N, K), dtype=torch.uint8, device=B.DEV)
    sa, sw = torch.ones(M, 1, device=B.DEV), torch.full((N // 128, 1), 0.5, device=B.DEV)
    out = moe.moe_block_matmul(a, sa, w, sw)
    assert out.numel() > 2 ** 31
    assert torch.equal(out[-300:], moe.moe_block_matmul(a[-300:], sa[-300:], w, sw))
    del out
    E, N, K = 20, 16384, 8192
    w = torch.randint(0, 100, (E, N, K), dtype=torch.uint8, device=B.DEV)
    sw = torch.ones(E, N // 128, K // 128, device=B.DEV)
    ids, al, pos, n = B.aligned(40, 2, E, 16, 4)
    a = torch.randint(0, 100, (40, K), dtype=torch.uint8, device=B.DEV)
    sa = torch.ones(40, K // 128, device=B.DEV)
    got = moe.moe_block_matmul_grouped(a, sa, w, sw, al, topk=2)
    t, j = np.argwhere(ids == ids.max())[0]
    assert ids.max() * N * K > 2 ** 31
    one = moe.moe_block_matmul(a[t:t + 1], sa[t:t + 1], w[ids.max()], sw[ids.max()])
    B.within(got[pos[t * 2 + j]], B.f64(one[0]), 2 * B.HALF_STEP["bf16"] * np.abs(B.f64(one[0])), "last expert")


@pytest.mark.parametrize("rows,N", [(16, 96), (64, 8448)])
def test_gathered_scales_at_the_largest_offset(rows, N):
    """Tokens whose codes and scales lie up to the limits on a_rows times their strides,
    for the few-row kernel and a tile's: the last one's are 2^31 - 64 bytes from the
    first."""
    M, K, stride = (1 << 26) - 1, 32, 8
    a, sa, w, sw = operands(rows, N, K, 3, 1)
    wide = torch.empty(M, stride, device=B.DEV)
    wide[-rows:, :1] = B.dev(sa)
    tokens = torch.empty(M, K, dtype=torch.uint8, device=B.DEV)
    tokens[-rows:] = B.dev(a)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=B.DEV)
    al = moe.Alignment(torch.arange(M - rows, M, dtype=torch.int32, device=B.DEV), i32([0]), i32([0, rows]), i32([0]), i32([rows]),
                       rows)
    got = moe.moe_block_matmul_grouped(tokens, wide[:, :1], B.fp8(w), B.dev(sw), al, topk=1, out_dtype=torch.float32)
    ref = BO.matmul(a, sa, w[0], sw[0])
    B.within(got, ref[0], B.product_bound(*ref, "f32", K), f"{rows} last tokens")


def reused(k, E, bm, M, capacity, seed):
    """An alignment of M tokens in buffers made for more: (Alignment, real places, rows in use)."""
    al = moe.alloc_alignment(capacity, k, E, bm, B.DEV)
    ids, own, pos, n = B.aligned(M, k, E, bm, seed)
    ws = torch.empty(moe.moe_workspace_size(moe.make_problem(M, 128, 128, E, k, bm, *[torch.bfloat16] * 3)), dtype=torch.uint8,
                     device=B.DEV)
    moe.moe_align_permute(B.dev(ids.astype(np.int32)), E, bm, ws, alignment=al)
    return al, ws, pos, n


@pytest.mark.parametrize("bm", [16, 256])
@pytest.mark.parametrize("N", [96, 8300])
def test_grouped_of_reused_buffers_by_default(N, bm):
    """The call without the number of its pairs or tokens, a and the alignment's
    buffers made for more: padding is zero, every expert's rows are written."""
    M, k, E, K, capacity = 30, 2, 4, 144, 200
    al, ws, pos, n = reused(k, E, bm, M, capacity, 5)
    R = al.sorted_pair_ids.numel()
    a, sa, w, sw = operands(max(R, capacity), N, K, 3, E)
    real = np.zeros(R, bool)
    real[pos] = True
    ordered, tokens = a[:R].copy(), a[:capacity].copy()
    ordered[~real], tokens[M:] = 0x7F, 0x7F  # NaN in what no pair reads
    W = (B.fp8(w), B.dev(sw))
    for args, given, more in (((B.fp8(ordered), B.dev(sa[:R]), *W), dict(pairs=M * k), {}),
                              ((B.fp8(tokens), B.dev(sa[:capacity]), *W), dict(topk=k, M=M), dict(topk=k))):
        want = moe.moe_block_matmul_grouped(*args, al, **given)
        out = torch.full((R, N), 3.0, dtype=torch.bfloat16, device=B.DEV)
        moe.moe_block_matmul_grouped(*args, al, out=out, **more)
        assert torch.equal(out[:n], want[:n]) and torch.isfinite(want[:n]).all()
        assert (out[:n][torch.from_numpy(~real[:n]).to(B.DEV)] == 0).all() and (out[n:] == 3).all()


def test_pairs_of_the_last_alignment_count():
    """What a product takes for its pairs is what the buffers were last filled with."""
    k, E, bm, N, K = 2, 4, 64, 96, 144
    al, ws, pos, n = reused(k, E, bm, 30, 200, 5)
    assert al.pairs == 60
    moe.moe_route_align(B.values((11, E), "f32", 1).to(B.DEV), k, True, bm, ws, alignment=al)
    assert al.pairs == 22
    R, n = al.sorted_pair_ids.numel(), int(al.num_padded)
    a, sa, w, sw = operands(R, N, K, 3, E)
    got = moe.moe_block_matmul_grouped(B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw), al)
    pad = (al.sorted_pair_ids[:n] >= 22).cpu().numpy()
    assert pad.sum() == n - 22 and (got[:n].cpu().float().numpy()[pad] == 0).all()


@pytest.mark.parametrize("M,N,K", [(3, 40, 272), (64, 7168, 256), (300, 513, 272), (700, 4000, 144)])
def test_groups_that_cancel(M, N, K):
    """Eight products in a row of 448^2, -448^2 and six of 1 to 9.  Whole numbers
    below 2^24 are exact in fp32 whatever the order; a bf16 result may lose what lies
    below 2^-13 of the largest."""
    r = np.random.RandomState(M + N)
    code = BO.e4m3_code(np.float32([1, 2, 3]))
    a, w = code[r.randint(0, 3, (M, K))], code[r.randint(0, 3, (N, K))]
    at = np.arange(0, K, 8)
    big = BO.e4m3_code(np.float32([448, -448]))
    a[:, at], a[:, at + 1], w[:, at], w[:, at + 1] = big[0], big[0], big[0], big[1]
    sa, sw = np.ones((M, -(-K // 128)), np.float32), np.ones((-(-N // 128), -(-K // 128)), np.float32)
    args = (B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw))
    v = BO.e4m3_values()
    want = v[a] @ v[w].T
    assert want.max() < 9 * K and want.min() > 0
    assert np.array_equal(B.f64(moe.moe_block_matmul(*args, out_dtype=torch.float32)), want)
    cut = K // 8 * 7 * 2.0 ** -13 * 448 ** 2
    got = moe.moe_block_matmul(*args)
    B.within(got, want, cut + (want + cut) * B.HALF_STEP["bf16"], "groups that cancel")
    assert torch.equal(got, moe.moe_block_matmul(*args))


@pytest.mark.parametrize("M", [8, 50])
def test_grouped_of_buffers_filled_with_other_blocks(M):
    """Buffers made for blocks of 16 and many tokens, filled with blocks of 64: the
    product goes by those."""
    k, E, N, K = 2, 4, 96, 144
    al, ws, pos, n = reused(k, E, 16, 20, 300, 5)
    ids, own, pos, n = B.aligned(M, k, E, 64, 8)
    assert n <= al.sorted_pair_ids.numel() and n // 64 <= al.block_expert_ids.numel()
    ws = torch.empty(moe.moe_workspace_size(moe.make_problem(M, 128, 128, E, k, 64, *[torch.bfloat16] * 3)), dtype=torch.uint8,
                     device=B.DEV)
    moe.moe_align_permute(B.dev(ids.astype(np.int32)), E, 64, ws, alignment=al)
    a, sa, w, sw = operands(M, N, K, 3, E)
    args = (B.fp8(a), B.dev(sa), B.fp8(w), B.dev(sw))
    assert torch.equal(moe.moe_block_matmul_grouped(*args, al, topk=k)[:n], moe.moe_block_matmul_grouped(*args, own, topk=k)[:n])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("M,N", [(3, 40), (300, 256)])
def test_products_of_small_scales(M, N, dt):
    """Two scales' product rounded as fp32, subnormal ones too: sums of 128 ones, which
    are exact, times 1.5 and 1.25 times powers of two down to 2^-160."""
    K = 256
    one = np.full((M, K), 0x38, np.uint8), np.full((N, K), 0x38, np.uint8)
    e = -np.arange(100, 161)
    for at in range(0, len(e), 3):
        sa = np.full((M, 2), 1.5 * 2.0 ** -75, np.float32)
        sa[:, 1] *= np.float32(1.25)
        sw = np.full((-(-N // 128), 2), 2.0 ** (e[at] + 75), np.float32)
        both = (sa[0].astype(np.float64) * sw[0]).astype(np.float32).astype(np.float64)
        want = (128 * both[0] + 128 * both[1]).astype(np.float32)
        got = moe.moe_block_matmul(B.fp8(one[0]), B.dev(sa), B.fp8(one[1]), B.dev(sw), out_dtype=B.DT[dt])
        assert (got == torch.tensor(want).to(B.DT[dt]).to(B.DEV)).all(), (e[at], got[0, 0].item(), want)
