"""The attention calls together and with the expert layer, as a serving loop
runs them: a prompt, then single tokens, then a mixed batch, against the fp64
oracle fed with the same inputs (the cache's codes checked on the way)."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_13_amd import moe
from oracle import attention_oracle as AO
from tests import attn_harness as A

pytestmark = pytest.mark.gpu


class Host:
    """The oracle's side of a cache that grows."""

    def __init__(self, P, H, S, D):
        self.c = {"k_codes": np.zeros((P, H, S, D), np.uint8), "v_codes": np.zeros((P, H, S // 16, D, 16), np.uint8),
                  "k_scales": np.ones((P, H), np.float32), "v_scales": np.ones((P, H), np.float32)}

    def step(self, q, k, v, pos, invf, pa, cu, kv, table, window):
        kr = AO.rotate(A.f64(k), pos, invf, pa)
        self.c = AO.append(self.c, kr, A.f64(v), cu, kv, table)
        qr = AO.rotate(A.f64(q), pos, invf, pa)
        return torch.from_numpy(qr).to(q.dtype), kr


@pytest.mark.parametrize("dt,window", [("bf16", 0), ("f32", 0), ("bf16", 40)])
def test_prompt_then_tokens_then_a_mixed_batch(dt, window):
    H, G, D, S, axes = 2, 4, 64, 16, 3
    B, steps = 3, [[37, 1, 90], [1, 1, 1], [1, 1, 1], [20, 1, 3]]
    total = [sum(s[b] for s in steps) for b in range(B)]
    P, table = A.tables(total, S, 1)
    cache = moe.alloc_kv_cache(P, S, H, D)
    for t in (cache.k_codes, cache.v_codes):
        t.view(torch.uint8).fill_(0x7F)  # what was never written is NaN
    invf = A.inv_freq(D)
    pa = torch.randint(0, axes, (D // 2,), generator=A.gen(3), dtype=torch.int32)
    layer = moe.PagedAttention(cache, H * G, invf.cuda(), 160, B, max_q=90, pair_axis=pa.cuda(), window=window,
                               dtype=A.DT[dt])
    host = Host(P, H, S, D)
    kv = [0] * B
    for n, q_lens in enumerate(steps):
        kv = [a + b for a, b in zip(kv, q_lens)]
        T, cu = sum(q_lens), A.offsets(q_lens)
        q, k, v = (A.values((T, h, D), dt, 10 * n + i) for i, h in enumerate((H * G, H, H)))
        pos = torch.randint(0, 5000, (axes, T), generator=A.gen(50 + n), dtype=torch.int32)
        one = all(x == 1 for x in q_lens)
        out = layer(q.cuda(), k.cuda(), v.cuda(), pos.cuda(), A.i32(kv), A.i32(table), cu_q=None if one else A.i32(cu))
        torch.cuda.synchronize()
        qr, _ = host.step(q, k, v, pos.numpy(), invf.numpy(), pa.numpy(), cu, kv, table, window)
        got = A.host_cache(cache)
        # codes: as the append's own test, at most a few at a midpoint differ
        for b in range(B):
            for t in range(kv[b]):
                p, s = table[b, t // S], t % S
                assert np.array_equal(got["v_codes"][p, :, s // 16, :, s % 16], host.c["v_codes"][p, :, s // 16, :, s % 16])
                assert (got["k_codes"][p, :, s] != host.c["k_codes"][p, :, s]).mean() <= 0.05
        # attention from the cache's and the query's own bits
        mine = layer.q[:T].clone()
        assert (A.f64(mine) - A.f64(qr)).__abs__().max() <= 2.0 ** -6 * np.abs(A.f64(qr)).max()
        ref = AO.attention(got, A.f64(mine), cu, kv, table, D ** -0.5, True, window)
        lse = moe.moe_paged_attention(cache, mine, A.i32(kv), A.i32(table), cu_q=A.i32(cu), max_q=90, window=window,
                                      return_lse=True)[1]
        A.check_attention(out, lse, ref, dt, D, f"step {n}")


def test_decoder_step_in_a_graph():
    """Attention and experts of one decode step captured together; replays with
    growing lengths equal the eager calls."""
    B, H, G, D, S = 4, 2, 4, 64, 16
    hidden, I, E, k = H * G * D, 256, 8, 2
    P, table = A.tables([40] * B, S, 1)
    kv0 = [5, 16, 31, 20]
    invf, dev = A.inv_freq(D).cuda(), "cuda"
    w13 = (torch.randn(E, 2 * I, hidden, generator=A.gen(1)) * 0.02).to(torch.bfloat16).cuda()
    w2 = (torch.randn(E, hidden, I, generator=A.gen(2)) * 0.02).to(torch.bfloat16).cuda()
    wr = (torch.randn(E, hidden, generator=A.gen(3)) / hidden ** 0.5).to(torch.bfloat16).cuda()
    start = A.random_cache(P, H, S, D, 4, pow2=True)

    def build():
        cache = A.device_cache(start)
        attn = moe.PagedAttention(cache, H * G, invf, B)
        experts = moe.FusedMoE(B, hidden, I, E, k, w13, w2)
        logits = torch.empty(B, E, device=dev)
        ws = torch.empty(max(moe.moe_route_project_workspace_size(B, hidden, E), 16), dtype=torch.uint8, device=dev)
        ids, wts = torch.empty(B, k, dtype=torch.int32, device=dev), torch.empty(B, k, device=dev)

        def step(qkv, pos, kv, tab, stream=None):
            n = H * G
            y = attn(qkv[:, :n], qkv[:, n:n + H], qkv[:, n + H:], pos, kv, tab, stream=stream).view(B, hidden)
            moe.moe_route_project_topk(y, wr, k, logits=logits, topk_ids=ids, topk_weights=wts, workspace=ws, stream=stream)
            return experts(y, logits, stream=stream)
        return cache, step

    qkv = torch.empty(B, H * G + 2 * H, D, dtype=torch.bfloat16, device=dev)
    pos, kv, tab = A.i32(kv0) - 1, A.i32(kv0), A.i32(table)
    qkv.copy_(A.values(qkv.shape, "bf16", 9))
    cache_g, step_g = build()
    cache_e, step_e = build()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step_g(qkv, pos, kv, tab)  # first calls outside the capture
        step_e(qkv, pos, kv, tab)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = step_g(qkv, pos, kv, tab, stream=s)
    for n in range(4):
        qkv.copy_(A.values(qkv.shape, "bf16", 20 + n))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = step_e(qkv, pos, kv, tab)
        torch.cuda.synchronize()
        assert torch.equal(out, want), n
        a, b = A.host_cache(cache_g), A.host_cache(cache_e)
        assert all(np.array_equal(a[x], b[x]) for x in a), n
        kv += 1
        pos += 1
