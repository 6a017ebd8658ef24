"""moe_paged_attention against the fp64 oracle; the bounds and their
derivation: attn_harness.check_attention.  Everything that no row sees holds
NaN codes and NaN scales."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_13_amd import moe
from oracle import attention_oracle as AO
from tests import attn_harness as A

pytestmark = pytest.mark.gpu


def make(q, kv, H, G, D, page, dt, seed=1, window=0, table=None, pages=None):
    P, tab = A.tables(kv, page, seed, extra_columns=1)
    if table is not None:
        P, tab = pages, table
    host = A.poison_unseen(A.random_cache(P, H, page, D, seed + 1), kv, tab, q, window)
    return host, tab, A.values((sum(q), H * G, D), dt, seed + 2)


def attend(host, tab, x, q, kv, causal=True, window=0, scale=None, cu=True, **kw):
    cache = A.device_cache(host)
    return moe.moe_paged_attention(cache, x.cuda(), A.i32(kv), A.i32(tab), cu_q=A.i32(A.offsets(q)) if cu else None,
                                   max_q=max(max(q), 1), causal=causal, window=window, sm_scale=scale,
                                   return_lse=True, **kw)


def run(q, kv, H, G, D, page, dt, causal=True, window=0, scale=None, **kw):
    host, tab, x = make(q, kv, H, G, D, page, dt, window=window if causal else 0, **kw)
    if not causal and window:
        host = A.random_cache(host["k_codes"].shape[0], H, page, D, 2)
    ref = AO.attention(host, A.f64(x), A.offsets(q), kv, tab, D ** -0.5 if scale is None else scale, causal, window)
    out, lse = attend(host, tab, x, q, kv, causal, window, scale)
    torch.cuda.synchronize()
    A.check_attention(out, lse, ref, dt, D, f"q{q[:4]} kv{kv[:4]} H{H} G{G} D{D} page{page} {dt}")
    if all(n == 1 for n in q):  # without cu_q the same rows, bit for bit
        o2, l2 = attend(host, tab, x, q, kv, causal, window, scale, cu=False)
        torch.cuda.synchronize()
        assert torch.equal(o2, out) and torch.equal(l2, lse)


ONE = [
    # kv (one query each), H, G, D, page, dtype, window
    ([1], 1, 1, 16, 16, "bf16", 0),
    ([0, 1, 2, 15, 16, 17], 2, 4, 64, 16, "bf16", 0),
    ([63, 64, 65, 127, 128, 129], 2, 4, 128, 64, "bf16", 0),
    ([63, 64, 65, 300], 1, 16, 256, 32, "bf16", 0),
    ([1000], 8, 4, 128, 64, "bf16", 0),
    ([700, 3], 2, 7, 80, 128, "bf16", 0),
    ([257, 900], 2, 5, 96, 16, "f32", 0),
    ([0, 65, 1500], 1, 16, 256, 32, "f32", 0),
    ([300, 40], 2, 17, 64, 16, "bf16", 0),
    ([300, 40], 1, 40, 64, 16, "f32", 0),
    ([300, 41], 1, 64, 48, 16, "bf16", 0),
    ([300, 41], 1, 32, 128, 16, "f32", 0),
    ([500, 77], 1, 128, 64, 16, "bf16", 0),
    ([500, 77], 1, 20, 192, 16, "bf16", 0),
    ([500, 1, 64, 200], 2, 4, 128, 16, "bf16", 1),
    ([500, 1, 64, 200], 2, 4, 128, 16, "bf16", 100),
    ([500, 1, 64, 200], 2, 4, 32, 64, "f32", 64),
    ([500, 1], 2, 4, 32, 64, "bf16", 100000),
]


@pytest.mark.parametrize("kv,H,G,D,page,dt,window", ONE)
def test_one_token(kv, H, G, D, page, dt, window):
    run([1] * len(kv), kv, H, G, D, page, dt, window=window)


MANY = [
    # q, kv, H, G, D, page, dtype, causal, window
    ([2], [2], 1, 1, 16, 16, "bf16", True, 0),
    ([64], [64], 1, 2, 64, 16, "bf16", True, 0),
    ([200], [200], 2, 4, 128, 64, "bf16", True, 0),
    ([200], [333], 2, 3, 128, 64, "bf16", True, 0),
    ([1, 100, 0, 17, 3], [500, 130, 60, 17, 260], 2, 4, 128, 32, "bf16", True, 0),
    ([1, 100, 0, 17, 3], [500, 130, 60, 17, 260], 2, 4, 64, 16, "f32", True, 50),
    ([130, 5], [150, 300], 1, 8, 256, 64, "bf16", True, 0),
    ([70, 5], [150, 90], 1, 2, 256, 64, "f32", True, 0),
    ([90, 5], [150, 90], 1, 4, 128, 16, "f32", True, 0),
    ([90, 33], [40, 33], 1, 4, 128, 16, "bf16", True, 0),     # more rows than tokens: the first see nothing
    ([90, 33], [0, 0], 1, 4, 64, 16, "bf16", True, 0),        # nothing at all
    ([90, 33], [95, 200], 2, 4, 96, 16, "bf16", False, 0),
    ([40, 33], [95, 200], 2, 4, 80, 32, "f32", False, 30),
    ([300], [300], 1, 1, 128, 128, "bf16", True, 1),
    ([300], [400], 1, 5, 144, 128, "bf16", True, 33),
    ([3, 2, 4, 1], [70, 9, 300, 64], 2, 8, 128, 64, "bf16", True, 0),   # a few rows each
    ([3, 2, 4, 1], [70, 9, 300, 64], 2, 8, 64, 64, "bf16", True, 20),
    ([130], [130], 1, 100, 32, 16, "bf16", True, 0),
]


@pytest.mark.parametrize("q,kv,H,G,D,page,dt,causal,window", MANY)
def test_many_rows(q, kv, H, G, D, page, dt, causal, window):
    run(q, kv, H, G, D, page, dt, causal, window)


def test_long_sequence_is_shared_out():
    """One sequence over many workgroups, next to one that is all but empty."""
    run([1, 1], [20011, 2], 1, 4, 64, 64, "bf16")
    run([1], [30000], 1, 8, 128, 128, "f32")


@pytest.mark.parametrize("extra", [0, 1])
def test_tables_on_both_sides_of_a_workgroup_of_its_own(extra):
    """Tables of 1024 and 2048 tokens, and of one page more, with few sequences and with many."""
    for kv, cap in (([1000, 3, 0, 777], 1024), ([1500, 0, 2047, 63] * 20, 2048)):
        P, small = A.tables(kv, 32, 1)
        table = np.full((len(kv), cap // 32 + extra), -1, np.int32)
        table[:, :small.shape[1]] = small
        run([1] * len(kv), kv, 8, 2, 16, 32, "bf16", table=table, pages=P)


def test_many_sequences():
    r = np.random.RandomState(1)
    kv = r.randint(0, 90, 600).tolist()
    run([1] * 600, kv, 1, 2, 32, 16, "bf16")
    q = [int(n) for n in r.randint(0, 40, 300)]
    run(q, [n + int(r.randint(0, 50)) for n in q], 1, 4, 32, 16, "bf16")


@pytest.mark.parametrize("q", [[0, 1], [1, 40]])
def test_sequences_that_see_nothing(q):
    """Padding of a batch: sequences without tokens before, between and behind
    the others, in a table long enough for workgroups to share sequences."""
    kv = [0] * 40 + [1500] + [0] * 270 + [70, 0, 2100] + [0] * 30
    rows = [1] * 40 + [1] + [q[i % 2] for i in range(270)] + [1, q[1], 1] + [1] * 30
    run(rows, kv, 2, 4, 32, 16, "bf16")
    # eight workgroups a head, one of which goes from one sequence over the gap to the next
    kv = [0] * 3 + [900] + [0] * 200 + [700] + [0] * 70 + [2100] + [0] * 2
    run([1] * len(kv), kv, 64, 1, 16, 16, "bf16")
    table = np.full((5, 100), 7, np.int32)
    run([1, q[1], 1, 1, 2], [0] * 5, 2, 4, 32, 16, "f32", table=table, pages=8)


@pytest.mark.parametrize("q", [1, 40])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_many_small_probabilities_beside_a_large_one(q, dt):
    """20000 tokens, each 2^-22.2 of one that has no value itself: their sum is
    the output, and fp16 has its smallest step at 2^-24."""
    n, H, D, S = 20000, 1, 64, 64
    P, table = A.tables([n], S, 1)
    host = A.random_cache(P, H, S, D, 2)
    host["k_codes"][:] = 0
    host["v_codes"] = (host["v_codes"] & 7) | 0x58  # 16 to 30
    host["k_codes"][table[0, 0], 0, 5, 9] = 0x38  # 1
    host["v_codes"][table[0, 0], 0, 0, :, 5] = 0
    host["k_scales"][:], host["v_scales"][:] = 1, 0.25
    x = torch.zeros(q, 2, D, dtype=A.DT[dt])
    x[:, :, 9] = 1
    scale = 22.2 * np.log(2)
    ref = AO.attention(host, A.f64(x), [0, q], [n], table, scale, False)
    out, lse = attend(host, table, x, [q], [n], causal=False, scale=scale)
    torch.cuda.synchronize()
    A.check_attention(out, lse, ref, dt, D, f"small beside large q{q} {dt}")


@pytest.mark.parametrize("q", [[1, 1], [40, 30]])
def test_scales_outside_their_bounds_count_as_the_nearest(q):
    kv = [100, 64]
    host, tab, x = make(q, kv, 1, 4, 64, 16, "bf16")
    used = [p for row in tab for p in row if p >= 0]
    host["v_scales"][used[0]], host["k_scales"][used[1]], host["v_scales"][used[2]] = 0, 0, -1
    ref = {n: a.copy() for n, a in host.items()}
    ref["v_scales"][used[0]] = ref["k_scales"][used[1]] = ref["v_scales"][used[2]] = AO.MIN_SCALE
    out, lse = attend(host, tab, x, q, kv)
    want = AO.attention(ref, A.f64(x), A.offsets(q), kv, tab, 64 ** -0.5)
    torch.cuda.synchronize()
    A.check_attention(out, lse, want, "bf16", 64, f"scales outside their bounds q{q}")


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0])
def test_scales(scale):
    run([1, 1], [130, 7], 1, 4, 64, 16, "f32", scale=scale)
    run([80], [130], 1, 4, 64, 16, "f32", scale=scale)


@pytest.mark.parametrize("q", [[1, 1, 1], [60, 50, 44]])
def test_pages_outside_the_cache_hide_their_tokens(q):
    kv = [100, 64, 70]
    P, tab = A.tables(kv, 16, 3)
    tab[0, 2], tab[0, 3], tab[1, :], tab[2, 0] = -1, P, 1 << 30, -(1 << 31)
    run(q, kv, 2, 4, 64, 16, "bf16", table=tab, pages=P)


@pytest.mark.parametrize("q", [[1, 1], [40, 30]])
def test_tokens_past_the_table_are_not_seen(q):
    """Rows stand where kv_lens says; the tokens that the table cannot hold are missing."""
    kv = [200, 70]
    table = np.array([[3, 0, 5], [1, 4, 2]], np.int32)
    run(q, kv, 1, 4, 64, 16, "bf16", table=table, pages=6)
    run(q, kv, 1, 4, 64, 16, "bf16", window=60, table=table, pages=6)


@pytest.mark.parametrize("q", [[2, 1, 3], [50, 60, 1]])
def test_rows_of_no_sequence_keep_their_bytes(q):
    kv = [70, 80, 9]
    host, tab, x = make(q, kv, 1, 4, 64, 16, "bf16")
    T, pad = sum(q), 5
    xp = torch.cat([x, torch.full((pad, 4, 64), float("nan"), dtype=x.dtype)])
    out = torch.full((T + pad, 4, 64), 3.0, dtype=x.dtype, device="cuda")
    lse = torch.full((T + pad, 4), 5.0, device="cuda")
    attend(host, tab, xp, q, kv, out=out, lse=lse)
    want = attend(host, tab, x, q, kv)
    torch.cuda.synchronize()
    assert torch.equal(out[:T], want[0]) and torch.equal(lse[:T], want[1])
    assert (out[T:] == 3).all() and (lse[T:] == 5).all()


@pytest.mark.parametrize("q", [[1, 1], [70, 33]])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_bad_query_spoils_its_own_row_only(q, bad):
    kv = [90, 64]
    host, tab, x = make(q, kv, 1, 4, 64, 16, "bf16")
    y = x.clone()
    y[0, 2, 7] = bad
    a, b = attend(host, tab, x, q, kv), attend(host, tab, y, q, kv)
    torch.cuda.synchronize()
    keep = torch.ones(a[1].shape, dtype=torch.bool, device="cuda")
    keep[0, 2] = False
    assert torch.equal(a[0][keep], b[0][keep]) and torch.equal(a[1][keep], b[1][keep])
    assert not torch.isfinite(b[0][0, 2]).all() or q[0] == 70  # a prompt's first row sees 21 tokens


@pytest.mark.parametrize("q", [[1, 1, 1], [40, 1, 70]])
def test_strides_streams_and_graphs(q):
    kv = [90, 200, 71]
    host, tab, x = make(q, kv, 2, 4, 64, 16, "bf16")
    T = sum(q)
    wide = torch.zeros(T, 13, 64, dtype=x.dtype, device="cuda")
    wide[:, 3:11] = x.cuda()
    cache, lens, table, cu = A.device_cache(host), A.i32(kv), A.i32(tab), A.i32(A.offsets(q))
    out, lse = torch.empty(T, 8, 64, dtype=x.dtype, device="cuda"), torch.empty(T, 8, device="cuda")
    n = moe.moe_paged_attention_workspace_size(cache, T, 3, 8, max(q))
    ws = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
    call = dict(cu_q=cu, max_q=max(q), out=out, lse=lse, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    moe.moe_paged_attention(cache, wide[:, 3:11], lens, table, stream=s, **call)
    s.synchronize()
    want = attend(host, tab, x, q, kv)
    torch.cuda.synchronize()
    assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    g, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        moe.moe_paged_attention(cache, wide[:, 3:11], lens, table, stream=s, **call)
    with torch.cuda.graph(g2, stream=s):  # shares the workspace: replayed in turn
        moe.moe_paged_attention(cache, wide[:, 3:11], lens, table, stream=s, **{**call, "window": 9})
    for step in range(3):  # lengths and queries rewritten between replays
        wide[:, 3:11] = A.values(x.shape, "bf16", 50 + step).cuda()
        lens.copy_(A.i32([n - step for n in kv]))
        for graph, window in ((g, 0), (g2, 9)):
            out.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            e = attend(host, tab, wide[:, 3:11].contiguous(), q, [n - step for n in kv], window=window)
            torch.cuda.synchronize()
            assert torch.equal(out, e[0]) and torch.equal(lse, e[1]), step


def test_defaults_hold_for_any_rows():
    """Without max_q every sequence is worked on; a layer's buffers do for fewer
    rows than they were made for, whichever kernel takes these."""
    H, G, D, S = 1, 8, 64, 16
    for q in ([300, 1], [4], [1, 8, 2], [2, 1]):
        kv = [n + 31 for n in q]
        host, tab, x = make(q, kv, H, G, D, S, "bf16")
        want = attend(host, tab, x, q, kv)[0]
        cache, lens, table, cu = A.device_cache(host), A.i32(kv), A.i32(tab), A.i32(A.offsets(q))
        got = moe.moe_paged_attention(cache, x.cuda(), lens, table, cu_q=cu)
        size = moe.moe_paged_attention_workspace_size(cache, 512, 8, H * G, 512)
        ws = torch.empty(size, dtype=torch.uint8, device="cuda")
        again = moe.moe_paged_attention(cache, x.cuda(), lens, table, cu_q=cu, max_q=512, workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(again, want), q


def test_two_calls_at_once():
    """Two streams, each with its own workspace and output."""
    host, tab, x = make([1, 1], [3000, 900], 2, 4, 128, 64, "bf16")
    cache, lens, table, xd = A.device_cache(host), A.i32([3000, 900]), A.i32(tab), x.cuda()
    want = moe.moe_paged_attention(cache, xd, lens, table)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[moe.moe_paged_attention(cache, xd, lens, table, stream=s) for _ in range(4)] for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for side in got for o in side)


@pytest.mark.parametrize("cap", [100, 40])
def test_a_pool_larger_than_the_caches(cap):
    """Few tokens of a pool of over 256 MB, shared out and by workgroups of their own."""
    H, D, S, kv = 2, 64, 16, [300, 0, 611, 64]
    small, table = A.tables(kv, S, 1)
    host = A.poison_unseen(A.random_cache(small, H, S, D, 2), kv, table, [1] * 4)
    P = (1 << 28) // (2 * H * S * D) + 1000
    where = np.random.RandomState(3).permutation(P)[:small]
    kc = torch.full((P, H, S, D), 0x7F, dtype=torch.uint8, device="cuda")
    vc = torch.full((P, H, S // 16, D, 16), 0x7F, dtype=torch.uint8, device="cuda")
    sc = torch.full((2, P, H), float("nan"), device="cuda")
    at = torch.from_numpy(where).cuda()
    for t, n in ((kc, "k_codes"), (vc, "v_codes"), (sc[0], "k_scales"), (sc[1], "v_scales")):
        t[at] = torch.from_numpy(host[n]).cuda()
    wide = np.full((4, cap), -1, np.int32)
    wide[:, :table.shape[1]] = np.where(table < 0, -1, where[table])
    x = A.values((4, H * 4, D), "bf16", 4)
    out, lse = moe.moe_paged_attention(moe.PagedKV(kc, vc, sc[0], sc[1]), x.cuda(), A.i32(kv), A.i32(wide), return_lse=True)
    torch.cuda.synchronize()
    ref = AO.attention(host, A.f64(x), A.offsets([1] * 4), kv, table, D ** -0.5)
    A.check_attention(out, lse, ref, "bf16", D, f"large pool, table of {cap * S}")


@pytest.mark.parametrize("q", [1, 100])
def test_offsets_past_32_bits(q):
    """A cache of over 4 GiB of codes each, the sequence in its last pages."""
    H, D, S = 2, 128, 128
    P = (1 << 32) // (H * S * D) + 64
    dev = torch.device("cuda")
    kc = torch.zeros(P, H, S, D, dtype=torch.uint8, device=dev)
    vc = torch.zeros(P, H, S // 16, D, 16, dtype=torch.uint8, device=dev)
    sc = torch.ones(2, P, H, device=dev)
    cache = moe.PagedKV(kc, vc, sc[0], sc[1])
    n = 300
    k, v = A.values((n, H, D), "bf16", 1), A.values((n, H, D), "bf16", 2)
    table = np.array([[P - 1, P - 2, P - 3]], np.int32)
    moe.moe_kv_append(cache, k.cuda(), v.cuda(), A.i32([n]), A.i32(table), cu_q=A.i32([0, n]))
    x = A.values((q, 4, D), "bf16", 3)
    out, lse = moe.moe_paged_attention(cache, x.cuda(), A.i32([n]), A.i32(table), cu_q=A.i32([0, q]), max_q=q,
                                       return_lse=True)
    torch.cuda.synchronize()
    small = {n_: a[-3:].cpu().numpy() for n_, a in (("k_codes", kc), ("v_codes", vc), ("k_scales", sc[0]), ("v_scales", sc[1]))}
    low = table - (P - 3)
    blank = {n_: np.zeros_like(a) for n_, a in small.items()}
    want = AO.append(blank, A.f64(k), A.f64(v), [0, n], [n], low)
    for name in small:
        assert np.array_equal(small[name], want[name]), name
    ref = AO.attention(small, A.f64(x), [0, q], [n], low, D ** -0.5)
    A.check_attention(out, lse, ref, "bf16", D, f"past 32 bits q{q}")
    assert int(kc[:-3].max()) == 0 and int(vc[:-3].max()) == 0


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_parts_of_more_than_256_workgroups(dt):
    """One sequence over 313 workgroups of one KV head: the join's second half."""
    run([1], [80003], 1, 4, 64, 64, dt)


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_bad_query_of_a_prompt_shows_in_its_row(bad):
    """The last row of the first sequence sees 90 tokens, the first of the
    second sequence 32, keys of both signs among them: no softmax is left."""
    q, kv = [70, 33], [90, 64]
    host, tab, x = make(q, kv, 1, 4, 64, 16, "bf16")
    clean = attend(host, tab, x, q, kv)
    for row in (69, 70):
        y = x.clone()
        y[row, 1, 7] = bad
        want = AO.attention(host, A.f64(y), A.offsets(q), kv, tab, 64 ** -0.5)
        assert np.isnan(want[0][row, 1]).all()  # the formula's, too
        out, lse = attend(host, tab, y, q, kv)
        torch.cuda.synchronize()
        assert not torch.isfinite(out[row, 1]).any() and not torch.isfinite(lse[row, 1])
        keep = torch.ones(lse.shape, dtype=torch.bool, device="cuda")
        keep[row, 1] = False
        assert torch.equal(out[keep], clean[0][keep]) and torch.equal(lse[keep], clean[1][keep])


@pytest.mark.parametrize("q", [[1, 1], [80, 3]])
@pytest.mark.parametrize("scale", [0.0, 1e-20, -2.0 ** -70])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_tiny_scales_over_pages_of_the_largest_scale(q, scale, dt):
    """Page scales of 2^48: a scale of zero weights every token alike, and the
    smallest others count as they are."""
    kv = [130, 70]
    P, tab = A.tables(kv, 16, 1)
    host = A.random_cache(P, 1, 16, 64, 2)
    host["k_scales"][:] = 2.0 ** 48
    x = A.values((sum(q), 4, 64), dt, 3)
    ref = AO.attention(host, A.f64(x), A.offsets(q), kv, tab, scale)
    out, lse = attend(host, tab, x, q, kv, scale=scale)
    torch.cuda.synchronize()
    A.check_attention(out, lse, ref, dt, 64, f"scale {scale} q{q} {dt}")


def test_tiles_past_32_bits():
    """128 sequences of 2^30 tokens, all in one page: 2^31 tiles in one batch.
    Keys of zero, so that every token weighs the same; values of which one in
    128 is not zero, so that every sum on the way is exact."""
    B, D, S, n = 128, 16, 128, 1 << 30
    kc = torch.zeros(1, 1, S, D, dtype=torch.uint8, device="cuda")
    vc = torch.zeros(1, 1, S // 16, D, 16, dtype=torch.uint8, device="cuda")
    vc[0, 0, 3, :, 5] = torch.arange(D, dtype=torch.uint8, device="cuda") % 15 * 8 + 8  # 2^-6 to 2^8
    one = torch.ones(1, 1, device="cuda")
    table = torch.zeros(B, n // S, dtype=torch.int32, device="cuda")
    out, lse = moe.moe_paged_attention(moe.PagedKV(kc, vc, one, one), A.values((B, 1, D), "bf16", 1).cuda(), A.i32([n] * B),
                                       table, return_lse=True)
    torch.cuda.synchronize()
    want = torch.exp2(torch.arange(D, dtype=torch.float64) % 15 - 6 - 7)
    assert torch.equal(out.cpu().double(), want.expand(B, 1, D))
    assert (lse.cpu().double() - 30 * np.log(2)).abs().max() <= 2.0 ** -20 * 30


@pytest.mark.parametrize("q", [1, 40])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("S", [16, 64])
def test_pages_of_zeros_beside_one_of_the_largest_scale(q, dt, S):
    """40000 tokens of 2^-22.2 of the weight of one whose page has the largest
    scale, in pages of the smallest (what an append of zeros leaves): they have
    no part in the sum of values, but 1/120 of the sum of weights."""
    n, H, D = 40000, 1, 64
    P, table = A.tables([n], S, 1)
    host = A.random_cache(P, H, S, D, 2)
    host["k_codes"][:], host["v_codes"][:] = 0, 0
    host["k_codes"][table[0, 0], 0, 5, 9] = 0x38  # 1
    host["v_codes"][table[0, 0], 0, 0, :, 5] = 0x58  # 16
    host["k_scales"][:], host["v_scales"][:] = 1, AO.MIN_SCALE
    host["v_scales"][table[0, 0]] = AO.MAX_SCALE
    x = torch.zeros(q, 2, D, dtype=A.DT[dt])
    x[:, :, 9] = 1
    scale = 22.2 * np.log(2)
    ref = AO.attention(host, A.f64(x), [0, q], [n], table, scale, False)
    out, lse = attend(host, table, x, [q], [n], causal=False, scale=scale)
    torch.cuda.synchronize()
    A.check_attention(out, lse, ref, dt, D, f"zeros beside the largest q{q} {dt} page{S}")
