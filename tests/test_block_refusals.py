"""What dispatch, combine, block quantisation and the block-scaled products
refuse, decided on the host before anything is enqueued (no GPU), and the
oracle's own closed forms."""
import ctypes

import numpy as np
import pytest
import torch

from mixture_experts_layer_13_amd import moe
from oracle import blocks_oracle as BO

F = 0x7f0000001000
ODD16, ODD4 = F + 8, F + 2
BF, F32 = moe.MOE_BF16, moe.MOE_F32
OK, NULL, SHAPE, DTYPE, ALIGN, UNSUP = (moe.MOE_OK, moe.MOE_ERR_NULL, moe.MOE_ERR_SHAPE, moe.MOE_ERR_DTYPE,
                                        moe.MOE_ERR_ALIGN, moe.MOE_ERR_UNSUPPORTED)


def al(**kw):
    d = dict(sorted_pair_ids=F, block_expert_ids=F, expert_offsets=F, pair_pos=F, num_padded=F, M=9, topk=2, E=4,
             block_m=16, rows=64)
    d.update(kw)
    return moe.moe_alignment(*[d[n] for n, _ in moe.moe_alignment._fields_])


def ref(x):
    return None if x is None else ctypes.byref(x)


def dispatch(a="default", x=F, xt=BF, xs=64, K=64, w=None, rows=F, rt=BF, rs=64):
    return moe.lib().moe_dispatch(ref(al() if a == "default" else a), x, xt, xs, K, w, rows, rt, rs, None)


def dispatch_bwd(a="default", dr=F, rt=BF, drs=64, K=64, x=F, xs=64, w=None, dx=F, xt=BF, dxs=64, dw=F):
    return moe.lib().moe_dispatch_backward(ref(al() if a == "default" else a), dr, rt, drs, K, x, xs, w, dx, xt, dxs, dw, None)


def combine(a="default", rows=F, rt=BF, rs=64, K=64, w=None, out=F, ot=BF, os=64):
    return moe.lib().moe_combine(ref(al() if a == "default" else a), rows, rt, rs, K, w, out, ot, os, None)


def combine_bwd(a="default", g=F, ot=BF, gs=64, K=64, rows=F, rs=64, w=None, dr=F, rt=BF, drs=64, dw=F):
    return moe.lib().moe_combine_backward(ref(al() if a == "default" else a), g, ot, gs, K, rows, rs, w, dr, rt, drs, dw, None)


BAD_ALIGNMENT = [(dict(M=-1), SHAPE), (dict(M=(1 << 22) + 1, topk=1), SHAPE), (dict(topk=0), SHAPE), (dict(topk=65), SHAPE),
                 (dict(M=1 << 22, topk=17), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=(1 << 26) + (1 << 18) + 1), SHAPE),
                 (dict(pair_pos=None), NULL), (dict(pair_pos=ODD4), ALIGN)]
BAD_PLACES = [(dict(sorted_pair_ids=None), NULL), (dict(num_padded=None), NULL), (dict(sorted_pair_ids=ODD4), ALIGN),
              (dict(num_padded=ODD4), ALIGN)]
BAD_K = [(dict(K=0), SHAPE), (dict(K=12), SHAPE), (dict(K=65544), SHAPE), (dict(K=128), SHAPE), (dict(a=None), NULL)]


@pytest.mark.parametrize("call", [dispatch, dispatch_bwd, combine, combine_bwd])
def test_alignment_refusals(call):
    for kw, status in BAD_ALIGNMENT + (BAD_PLACES if call in (dispatch, combine_bwd) else []):
        assert call(a=al(**kw)) == status, kw
        assert moe.moe_last_error()
    for kw, status in BAD_K:
        assert call(**kw) == status, kw
    assert call(a=al(M=0)) == OK
    assert moe.moe_last_error() == ""


@pytest.mark.parametrize("call,kw,status", [
    (dispatch, dict(x=None), NULL), (dispatch, dict(rows=None), NULL), (dispatch, dict(xt=2), DTYPE), (dispatch, dict(rt=9), DTYPE),
    (dispatch, dict(xs=63), SHAPE), (dispatch, dict(xs=68), ALIGN), (dispatch, dict(rs=66), ALIGN), (dispatch, dict(rs=0), SHAPE),
    (dispatch, dict(x=ODD16), ALIGN), (dispatch, dict(rows=ODD16), ALIGN), (dispatch, dict(w=ODD4), ALIGN),
    (dispatch, dict(xs=(1 << 32) + 8), SHAPE),
    (dispatch_bwd, dict(dr=None), NULL), (dispatch_bwd, dict(dx=None), NULL), (dispatch_bwd, dict(x=None), NULL),
    (dispatch_bwd, dict(xs=8), SHAPE), (dispatch_bwd, dict(dw=ODD4), ALIGN), (dispatch_bwd, dict(drs=65), ALIGN),
    (dispatch_bwd, dict(dxs=32), SHAPE), (dispatch_bwd, dict(x=ODD16), ALIGN),
    (combine, dict(rows=None), NULL), (combine, dict(out=None), NULL), (combine, dict(out=ODD16), ALIGN), (combine, dict(os=8), SHAPE),
    (combine, dict(rs=100), ALIGN), (combine, dict(ot=-1), DTYPE),
    (combine_bwd, dict(g=None), NULL), (combine_bwd, dict(dr=None), NULL), (combine_bwd, dict(rows=None), NULL),
    (combine_bwd, dict(rows=ODD16), ALIGN), (combine_bwd, dict(drs=8), SHAPE), (combine_bwd, dict(gs=60), SHAPE),
])
def test_permute_refusals(call, kw, status):
    assert call(**kw) == status
    assert moe.moe_last_error()


def quant(x=F, xt=BF, xs=256, M=9, K=256, gated=0, br=1, n=None, codes=F, scales=F, sr=1, sb=9):
    return moe.lib().moe_quantize_blocks(x, xt, xs, M, K, gated, br, n, codes, scales, sr, sb, None)


@pytest.mark.parametrize("kw,status", [
    (dict(xt=2), DTYPE), (dict(M=-1), SHAPE), (dict(M=(1 << 27) + 1), SHAPE), (dict(K=0), SHAPE), (dict(K=24), SHAPE),
    (dict(K=65552, xs=65552), SHAPE), (dict(br=2), SHAPE), (dict(br=0), SHAPE), (dict(br=128, gated=1, xs=512), UNSUP),
    (dict(br=128, n=F), UNSUP), (dict(gated=1), SHAPE), (dict(xs=250), SHAPE), (dict(xs=260), ALIGN), (dict(sr=0), SHAPE),
    (dict(sb=0), SHAPE), (dict(x=None), NULL), (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(x=ODD16), ALIGN),
    (dict(codes=ODD16), ALIGN), (dict(scales=ODD4), ALIGN), (dict(n=ODD4), ALIGN), (dict(M=1 << 20, K=65536, xs=65536), SHAPE), (dict(M=0, x=None, codes=None), OK),
])
def test_quantize_refusals(kw, status):
    assert quant(**kw) == status
    assert (moe.moe_last_error() != "") == (status != OK)


def matmul(a=F, ast=256, sa=F, sr=1, sb=9, w=F, sw=F, M=9, N=100, K=256, out=F, ot=BF, os=100):
    return moe.lib().moe_block_matmul(a, ast, sa, sr, sb, w, sw, M, N, K, out, ot, os, None)


def grouped(g="default", a=F, ast=256, rows=9, sa=F, sr=1, sb=9, w=F, sw=F, N=100, K=256, gather=1, out=F, ot=BF, os=100):
    return moe.lib().moe_block_matmul_grouped(ref(al() if g == "default" else g), a, ast, rows, sa, sr, sb, w, sw, N, K, gather,
                                              out, ot, os, None)


BAD_PRODUCT = [
    (dict(K=0), SHAPE), (dict(K=24), SHAPE), (dict(K=65552, ast=65552), SHAPE), (dict(N=0), SHAPE), (dict(N=65537, os=65537), SHAPE),
    (dict(ot=2), DTYPE), (dict(ast=240), SHAPE), (dict(ast=264), ALIGN), (dict(ast=(1 << 22) + 16), SHAPE), (dict(sr=0), SHAPE),
    (dict(sr=(1 << 20) + 1), SHAPE), (dict(sb=0), SHAPE), (dict(os=99), SHAPE), (dict(a=None), NULL), (dict(sa=None), NULL),
    (dict(w=None), NULL), (dict(sw=None), NULL), (dict(out=None), NULL), (dict(a=ODD16), ALIGN), (dict(w=ODD16), ALIGN),
    (dict(sa=ODD4), ALIGN), (dict(sw=ODD4), ALIGN), (dict(out=F + 1), ALIGN), (dict(out=ODD4, ot=F32), ALIGN),
]


@pytest.mark.parametrize("kw,status", BAD_PRODUCT + [
    (dict(M=-1), SHAPE), (dict(M=(1 << 27) + 1), SHAPE), (dict(M=1 << 22, N=32768, os=32768), SHAPE), (dict(M=0, a=None, out=None), OK),
])
def test_matmul_refusals(kw, status):
    assert matmul(**kw) == status
    assert (moe.moe_last_error() != "") == (status != OK)


@pytest.mark.parametrize("kw,status", BAD_PRODUCT + [
    (dict(g=None), NULL), (dict(g=al(M=-1)), SHAPE), (dict(g=al(E=0)), SHAPE), (dict(g=al(E=1025)), SHAPE),
    (dict(g=al(block_m=48)), SHAPE), (dict(rows=8), SHAPE), (dict(rows=63, gather=0), SHAPE),
    (dict(rows=1 << 23, ast=256), SHAPE), (dict(rows=1 << 20, sr=1 << 9), SHAPE),
    (dict(g=al(sorted_pair_ids=None)), NULL), (dict(g=al(block_expert_ids=None)), NULL), (dict(g=al(expert_offsets=None)), NULL),
    (dict(g=al(num_padded=None)), NULL), (dict(g=al(expert_offsets=ODD4)), ALIGN),
    (dict(g=al(block_m=16, rows=1 << 26, M=1 << 20), N=65536, os=65536), SHAPE),
    (dict(g=al(M=0)), OK), (dict(g=al(rows=0)), OK), (dict(g=al(M=0, sorted_pair_ids=None)), OK),
])
def test_grouped_refusals(kw, status):
    assert grouped(**kw) == status
    assert (moe.moe_last_error() != "") == (status != OK)


def refused(status, f, *a, **kw):
    with pytest.raises(moe.MoEError) as e:
        f(*a, **kw)
    assert e.value.status == status, e.value


def test_binding_refusals():
    """Tensors of the wrong type, shape, layout or place (all on the host)."""
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    good = moe.Alignment(i32(64), i32(4), i32(5), i32(18), i32(1), 16)
    x, rows, w = torch.zeros(9, 64), torch.zeros(64, 64), torch.zeros(9, 2)
    refused(UNSUP, moe.moe_dispatch, x, good, 2)  # on the host
    refused(DTYPE, moe.moe_dispatch, x.half(), good, 2)
    refused(SHAPE, moe.moe_dispatch, x[0], good, 2)
    refused(UNSUP, moe.moe_dispatch, x.t().contiguous().t(), good, 2)
    refused(SHAPE, moe.moe_dispatch, x, good, 3)
    refused(SHAPE, moe.moe_dispatch, x, good, 2, weights=w[:8])
    refused(DTYPE, moe.moe_dispatch, x, good, 2, weights=w.double())
    refused(UNSUP, moe.moe_dispatch, x, good, 2, weights=torch.zeros(2, 9).t())
    refused(SHAPE, moe.moe_dispatch, x, good, 2, out=rows[:63])
    refused(SHAPE, moe.moe_block_matmul_grouped, torch.zeros(9, 64, dtype=torch.uint8), torch.zeros(9, 1),
            torch.zeros(4, 8, 64, dtype=torch.uint8), torch.zeros(4, 1, 1),
            moe.Alignment(i32(64), i32(3), i32(5), i32(18), i32(1), 16), topk=2)
    refused(DTYPE, moe.moe_dispatch, x, moe.Alignment(i32(64).long(), i32(4), i32(5), i32(18), i32(1), 16), 2)
    refused(SHAPE, moe.moe_combine, rows[:60], good, 9, 2)
    refused(DTYPE, moe.moe_dispatch_backward, rows, good, 9, 2, x=x, out=x.bfloat16())
    refused(DTYPE, moe.moe_combine_backward, x, good, 2, rows=rows, out=rows.bfloat16())
    refused(SHAPE, moe.moe_combine_backward, x, good, 2, rows=rows[:, :32])

    q = torch.zeros(4, 256)
    refused(UNSUP, moe.moe_quantize_blocks, q)
    refused(SHAPE, moe.moe_quantize_blocks, q[None])
    refused(SHAPE, moe.moe_quantize_blocks, q[:, :129], gated=True)
    refused(DTYPE, moe.moe_quantize_blocks, q, codes=torch.zeros(4, 256))
    refused(SHAPE, moe.moe_quantize_blocks, q, codes=torch.zeros(4, 128, dtype=torch.uint8))
    refused(SHAPE, moe.moe_quantize_blocks, q, scales=torch.zeros(4, 3))
    refused(DTYPE, moe.moe_quantize_blocks, q, num_rows=torch.zeros(1))

    a, sa = torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 2)
    b, sb = torch.zeros(200, 256, dtype=torch.uint8), torch.zeros(2, 2)
    refused(UNSUP, moe.moe_block_matmul, a, sa, b, sb)
    refused(DTYPE, moe.moe_block_matmul, a.float(), sa, b, sb)
    refused(SHAPE, moe.moe_block_matmul, a, sa, b[:, :128].contiguous(), sb)
    refused(SHAPE, moe.moe_block_matmul, a, sa, b, sb[:1])
    refused(SHAPE, moe.moe_block_matmul, a, sa[:3], b, sb)
    refused(UNSUP, moe.moe_block_matmul, a, sa, b.t().contiguous().t(), sb)
    refused(SHAPE, moe.moe_block_matmul, a, sa, b, sb, out=torch.zeros(4, 199))
    refused(SHAPE, moe.moe_block_matmul_grouped, a, sa, b, sb, good)
    refused(SHAPE, moe.moe_block_matmul_grouped, a, sa, b[None], sb[None], good, topk=2)  # offsets of four experts


def test_oracle_closed_forms():
    v = BO.e4m3_values()
    fin = np.isfinite(v)
    assert v[0x7E] == 448 and v[1] == 2.0 ** -9 and v[0x38] == 1 and fin.sum() == 254
    c = BO.e4m3_code(v[fin])
    assert np.array_equal(v[c], v[fin])
    t = torch.linspace(-500, 500, 20011)
    want = t.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(BO.e4m3_code(t.numpy()), want)
    # one block: a plain product; identity places: dispatch and combine undo each other
    a, w = np.full((2, 128), 0x38, np.uint8), np.full((3, 128), 0x40, np.uint8)
    assert np.array_equal(BO.matmul(a, np.full((2, 1), 0.5, np.float32), w, np.full((1, 1), 2, np.float32))[0], np.full((2, 3), 256.0))
    x = np.random.RandomState(0).randn(4, 8)
    pos = np.array([5, 0, 3, 1])
    rows = BO.dispatch(x, pos, 1, 6)
    assert np.array_equal(BO.combine(rows, pos, 1, 4)[0], x) and (rows[[2, 4]] == 0).all()
    assert np.allclose(BO.pair_dots(x, rows, pos, 1)[0][:, 0], (x * x).sum(1))


def test_pairs_of_an_alignment():
    """An alignment that knows its pairs: whole tokens of topk, and as many in a."""
    i32 = lambda n: torch.zeros(n, dtype=torch.int32)
    known = moe.Alignment(i32(64), i32(4), i32(5), i32(40), i32(1), 16, 18)
    assert known.pairs == 18 and moe.Alignment(i32(64), i32(4), i32(5), i32(40), i32(1), 16).pairs is None
    w = torch.zeros(4, 8, 64, dtype=torch.uint8), torch.zeros(4, 1, 1)
    a = lambda rows: (torch.zeros(rows, 64, dtype=torch.uint8), torch.zeros(rows, 1))
    refused(SHAPE, moe.moe_block_matmul_grouped, *a(9), *w, known, topk=4)  # 4.5 tokens
    refused(SHAPE, moe.moe_block_matmul_grouped, *a(9), *w, known, topk=0)
    refused(UNSUP, moe.moe_block_matmul_grouped, *a(9), *w, known, topk=2)  # (right, but on the host)
    # the library: fewer tokens than the alignment's, fewer rows than its places
    assert grouped(g=al(M=9), rows=8) == SHAPE and grouped(g=al(rows=64), rows=63, gather=0) == SHAPE


@pytest.mark.parametrize("codes,scales", [((3, 200, 144), None), ((1, 200, 144), None), ((200, 144), None), ((2, 200, 160), None),
                                          (None, (3, 2, 2)), (None, (1, 2, 2)), (None, (2, 2)), (None, (2, 2, 1))])
def test_buffers_for_the_codes_of_experts(codes, scales):
    """Refused as a whole, not after the first experts (or, of too many, never)."""
    made = {}
    if codes:
        made["codes"] = torch.zeros(codes, dtype=torch.uint8)
    if scales:
        made["scales"] = torch.zeros(scales)
    refused(SHAPE, moe.moe_quantize_blocks, torch.zeros(2, 200, 144), block_rows=128, **made)


P = F + (1 << 30)  # apart from F for every call here


@pytest.mark.parametrize("call,kw", [
    # 9 tokens of 64 bf16: 1152 bytes, 64 rows: 8192; weights, places: 72; marks: 256
    (dispatch, dict(a=al(), x=P, rows=P)), (dispatch, dict(x=P + 8176, rows=P)), (dispatch, dict(x=P, rows=P + 1136)),
    (dispatch, dict(x=F, rows=P, w=P + 16)), (dispatch, dict(a=al(pair_pos=P), rows=P)),
    (dispatch, dict(a=al(sorted_pair_ids=P + 8188), rows=P)), (dispatch, dict(a=al(num_padded=P), rows=P)),
    (dispatch, dict(x=P, xs=128, rows=P + 112, rs=128)), (dispatch, dict(x=P + 128 * 2, xs=128, rows=P + 112, rs=128)),
    (dispatch, dict(x=P, xs=1024, rows=P + 8192, rs=64)), (dispatch, dict(x=P + 8176 - 4 * 2048, xs=1024, rows=P, rs=64)),
    (dispatch_bwd, dict(dr=F, x=P, dx=P, dw=P + (1 << 20))), (dispatch_bwd, dict(dr=P, x=F, dx=P + 8000, dw=P + (1 << 20))),
    (dispatch_bwd, dict(dr=F, x=F, dx=P, dw=P + 1148)), (dispatch_bwd, dict(dr=F, x=F, dx=P, dw=F + 1000)),
    (dispatch_bwd, dict(a=al(pair_pos=P), dx=P + (1 << 20), dw=P + 68)),
    (dispatch_bwd, dict(w=P, dx=P + (1 << 20), dw=P)),
    (combine, dict(rows=P, out=P)), (combine, dict(rows=P, out=P + 8176)), (combine, dict(w=P, out=P)),
    (combine_bwd, dict(g=P, rows=F, dr=P, dw=P + (1 << 20))), (combine_bwd, dict(g=F, rows=P, dr=P, dw=P + (1 << 20))),
    (combine_bwd, dict(g=F, rows=F, dr=P, dw=P)),
    # 9 rows of 256 bf16: 4608 bytes, their codes 2304, scales 72
    (quant, dict(x=P, codes=P, scales=P + (1 << 20))), (quant, dict(x=P, codes=P + 4592, scales=P + (1 << 20))),
    (quant, dict(x=F, codes=P, scales=P + 2300)), (quant, dict(x=P, codes=P + (1 << 20), scales=P + 4604)),
    (quant, dict(x=F, codes=P, scales=P - 60, sr=2, sb=1)), (quant, dict(x=F, codes=P, scales=P + 2300, sr=100, sb=1)),
    (quant, dict(x=F, n=P, codes=P, scales=P + (1 << 20))), (quant, dict(x=F, n=P + 4, codes=P + (1 << 20), scales=P)),
    (quant, dict(gated=1, xs=512, x=P, codes=P + 9200, scales=P + (1 << 20))),
    # 9 rows of 256 codes: 2304 bytes; out 9 x 100 bf16: 1800; w 25600
    (matmul, dict(a=P, out=P)), (matmul, dict(sa=P, out=P)), (matmul, dict(w=P, out=P + 25596)), (matmul, dict(sw=P + 1796, out=P)),
    (matmul, dict(a=P, ast=4096, out=P + 4096)), (matmul, dict(sa=P + 1600, sr=1, sb=50, out=P, os=100)),
    (grouped, dict(a=P, out=P)), (grouped, dict(sa=P, out=P)), (grouped, dict(w=P, out=P + 4 * 25600 - 4)),
    (grouped, dict(sw=P + 64 * 200 - 4, out=P)), (grouped, dict(a=P, rows=64, gather=0, out=P + 64 * 256 - 16)),
    *((grouped, dict(g=al(**{n: P + 12796}), out=P)) for n in ("sorted_pair_ids", "block_expert_ids", "expert_offsets", "num_padded")),
])
def test_outputs_that_overlap_inputs(call, kw):
    assert call(**kw) == SHAPE, kw
    assert "overlaps" in moe.moe_last_error()


def test_layer_refusals():
    """Logits of another type, number or place would be read (and places written)
    past their ends; nothing is launched before all of them are looked at."""
    M, K, N, E, k = 9, 128, 64, 4, 2
    codes, scales = lambda *s: torch.zeros(s, dtype=torch.uint8), lambda *s: torch.zeros(s)
    layer = moe.BlockMoE(M, K, N, E, k, codes(E, 2 * N, K), scales(E, 1, 1), codes(E, K, N), scales(E, 1, 1), device="cpu")
    x, logits = torch.zeros(M, K), torch.zeros(M, E)
    refused(DTYPE, layer, x, logits.bfloat16())
    refused(SHAPE, layer, x, torch.zeros(M, E + 1))
    refused(SHAPE, layer, x, logits[:8])
    refused(SHAPE, layer, x[:8], logits)
    refused(UNSUP, layer, x, torch.zeros(E, M).t())
    refused(UNSUP, layer, x, logits.to("meta"))
    refused(UNSUP, layer, x.to("meta"), logits)
    refused(UNSUP, layer, x, logits)  # on the host
    refused(SHAPE, moe.BlockMoE, M, K, N, E, k, codes(E, N, K), scales(E, 1, 1), codes(E, K, N), scales(E, 1, 1), device="cpu")
