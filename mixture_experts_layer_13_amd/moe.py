"""Thin ctypes binding of libmoe.so (include/moe.h).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the hipStream_t, and a non-zero status raises MoEError.  Every
step of the layer runs in the library's HIP kernels; there is no fallback.
"""
import ctypes
import os
from dataclasses import dataclass

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe.so")

MOE_OK, MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_DTYPE, MOE_ERR_ALIGN = 0, 1, 2, 3, 4
MOE_ERR_WORKSPACE, MOE_ERR_UNSUPPORTED, MOE_ERR_HIP = 5, 6, 7
MOE_F32, MOE_BF16, MOE_FP8_E4M3 = 0, 1, 2

EXPORTS = ("moe_status_string", "moe_last_error", "moe_align_capacity", "moe_workspace_size",
           "moe_route_topk", "moe_align_permute", "moe_fused_forward", "moe_quantize_act",
           "moe_fused_forward_profiled", "moe_fused_forward_noalloc", "moe_route_align", "moe_route_project_topk",
           "moe_route_project_workspace_size", "moe_rope_quantize_per_head", "moe_rope_workspace_size",
           "moe_fused_forward_persistent", "moe_rope_axes", "moe_kv_append", "moe_paged_attention",
           "moe_paged_attention_workspace_size")
MOE_QUANT_WORKSPACE_BYTES = 8192
MOE_WORKSPACE_SCALES_OFFSET = 4096
MOE_NOALLOC_SCRATCH_BYTES = 64 << 20
MOE_MAX_SEQS = 65536  # sequences of an append's or attention's batch
MOE_FUSED_SYNC_BYTES = 32768
MOE_FUSED_SYNC_ERROR_OFFSET = 128


class MoEError(RuntimeError):
    def __init__(self, status, detail):
        self.status = status
        super().__init__(f"{moe_status_string(status)}: {detail}")


class moe_problem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in
                ("M", "K", "N", "E", "topk", "block_m", "a_dtype", "w_dtype", "out_dtype")]


class moe_rotation(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("positions", "pair_axis", "inv_freq")] +
                [(n, ctypes.c_int32) for n in ("axes", "rotary_dim", "interleaved", "inverse")])


class moe_kv_cache(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("k_codes", "v_codes", "k_scales", "v_scales")] +
                [(n, ctypes.c_int32) for n in ("num_pages", "page_size", "n_kv_heads", "head_dim")])


class moe_kv_batch(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("cu_q", "kv_lens", "block_table")] +
                [(n, ctypes.c_int32) for n in ("B", "T", "max_pages")])


_lib = None


def lib():
    """The loaded library; raises if it has not been built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run __graft_entry__.build() first")
        L = ctypes.CDLL(LIB_PATH)
        vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        L.moe_status_string.argtypes = [i32]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_last_error.argtypes = []
        L.moe_last_error.restype = ctypes.c_char_p
        L.moe_align_capacity.argtypes = [i32, i32, i32, i32]
        L.moe_align_capacity.restype = i64
        L.moe_workspace_size.argtypes = [ctypes.POINTER(moe_problem), ctypes.POINTER(sz)]
        L.moe_workspace_size.restype = ctypes.c_int
        L.moe_route_topk.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp]
        L.moe_route_topk.restype = ctypes.c_int
        L.moe_align_permute.argtypes = [vp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
        L.moe_align_permute.restype = ctypes.c_int
        L.moe_fused_forward.argtypes = [ctypes.POINTER(moe_problem)] + [vp] * 15 + [sz, vp]
        L.moe_fused_forward.restype = ctypes.c_int
        L.moe_quantize_act.argtypes = [vp, i32, i64, vp, vp, vp, vp, sz, vp]
        L.moe_quantize_act.restype = ctypes.c_int
        L.moe_fused_forward_profiled.argtypes = ([ctypes.POINTER(moe_problem)] + [vp] * 15 +
                                                 [sz, vp, ctypes.POINTER(ctypes.c_void_p)])
        L.moe_fused_forward_profiled.restype = ctypes.c_int
        L.moe_fused_forward_noalloc.argtypes = [ctypes.POINTER(moe_problem)] + [vp] * 15
        L.moe_fused_forward_noalloc.restype = ctypes.c_int
        L.moe_fused_forward_persistent.argtypes = ([ctypes.POINTER(moe_problem)] + [vp] * 15 +
                                                   [sz, vp, sz, vp])
        L.moe_fused_forward_persistent.restype = ctypes.c_int
        L.moe_route_align.argtypes = [vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp,
                                      vp, sz, vp]
        L.moe_route_align.restype = ctypes.c_int
        L.moe_route_project_topk.argtypes = [vp, i32, vp, i32, i32, i32, i32, i32, i32, vp, vp,
                                             vp, vp, sz, vp]
        L.moe_route_project_topk.restype = ctypes.c_int
        L.moe_route_project_workspace_size.argtypes = [i32, i32, i32, ctypes.POINTER(sz)]
        L.moe_route_project_workspace_size.restype = ctypes.c_int
        L.moe_rope_quantize_per_head.argtypes = [vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp,
                                                 vp, vp, sz, vp]
        L.moe_rope_quantize_per_head.restype = ctypes.c_int
        L.moe_rope_workspace_size.argtypes = [i32, i32, i32, ctypes.POINTER(sz)]
        L.moe_rope_workspace_size.restype = ctypes.c_int
        f32 = ctypes.c_float
        L.moe_rope_axes.argtypes = [vp, i32, i64, i64, ctypes.POINTER(moe_rotation), i32, i32, i32, vp, i32,
                                    i64, i64, vp]
        L.moe_rope_axes.restype = ctypes.c_int
        L.moe_kv_append.argtypes = [ctypes.POINTER(moe_kv_cache), ctypes.POINTER(moe_kv_batch), vp, i64, i64,
                                    vp, i64, i64, i32, ctypes.POINTER(moe_rotation), vp]
        L.moe_kv_append.restype = ctypes.c_int
        L.moe_paged_attention.argtypes = [ctypes.POINTER(moe_kv_cache), ctypes.POINTER(moe_kv_batch), vp, i32,
                                          i64, i64, i32, i32, f32, i32, i32, vp, vp, vp, sz, vp]
        L.moe_paged_attention.restype = ctypes.c_int
        L.moe_paged_attention_workspace_size.argtypes = [ctypes.POINTER(moe_kv_cache), i32, i32, i32, i32,
                                                         ctypes.POINTER(sz)]
        L.moe_paged_attention_workspace_size.restype = ctypes.c_int
        _lib = L
    return _lib


def moe_status_string(status):
    return lib().moe_status_string(int(status)).decode()


def moe_last_error():
    return lib().moe_last_error().decode()


def _check(status):
    if status != MOE_OK:
        raise MoEError(status, moe_last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def dtype_code(dt):
    return {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16,
            torch.float8_e4m3fn: MOE_FP8_E4M3}[dt]


def moe_align_capacity(M, topk, E, block_m):
    return int(lib().moe_align_capacity(M, topk, E, block_m))


def make_problem(M, K, N, E, topk, block_m, a_dtype, w_dtype, out_dtype):
    return moe_problem(M, K, N, E, topk, block_m, dtype_code(a_dtype), dtype_code(w_dtype),
                       dtype_code(out_dtype))


def moe_workspace_size(problem):
    n = ctypes.c_size_t(0)
    _check(lib().moe_workspace_size(ctypes.byref(problem), ctypes.byref(n)))
    return int(n.value)


def moe_route_project_workspace_size(M, K, E):
    n = ctypes.c_size_t(0)
    _check(lib().moe_route_project_workspace_size(M, K, E, ctypes.byref(n)))
    return n.value


def moe_route_project_topk(x, w_router, topk, renormalize=True, logits=None, topk_ids=None,
                           topk_weights=None, workspace=None, stream=None):
    """x [M,K] and w_router [E,K] (device, both bf16 or both f32) -> (ids
    int32 [M,k], weights f32 [M,k]); logits f32 [M,E] is written if given."""
    M, K = x.shape
    E = w_router.shape[0]
    if topk_ids is None:
        topk_ids = torch.empty(M, topk, dtype=torch.int32, device=x.device)
    if topk_weights is None:
        topk_weights = torch.empty(M, topk, dtype=torch.float32, device=x.device)
    if workspace is None:
        workspace = torch.empty(max(moe_route_project_workspace_size(M, K, E), 16),
                                dtype=torch.uint8, device=x.device)
    _check(lib().moe_route_project_topk(_ptr(x), dtype_code(x.dtype), _ptr(w_router),
                                        dtype_code(w_router.dtype), M, K, E, topk,
                                        int(bool(renormalize)), _ptr(logits), _ptr(topk_ids),
                                        _ptr(topk_weights), _ptr(workspace), workspace.numel(),
                                        _stream(stream)))
    return topk_ids, topk_weights


def moe_route_topk(logits, topk, renormalize=True, topk_ids=None, topk_weights=None,
                   stream=None):
    """logits f32 [M,E] (device) -> (ids int32 [M,k], weights f32 [M,k])."""
    M, E = logits.shape
    if topk_ids is None:
        topk_ids = torch.empty(M, topk, dtype=torch.int32, device=logits.device)
    if topk_weights is None:
        topk_weights = torch.empty(M, topk, dtype=torch.float32, device=logits.device)
    _check(lib().moe_route_topk(_ptr(logits), M, E, topk, int(bool(renormalize)),
                                _ptr(topk_ids), _ptr(topk_weights), _stream(stream)))
    return topk_ids, topk_weights


def moe_quantize_act(x, static_scale=None, codes=None, scale=None, workspace=None,
                     stream=None):
    """x f32/bf16 (device) -> (E4M3 codes as uint8, f32 scale [1])."""
    n = x.numel()
    dev = x.device
    codes = torch.empty(x.shape, dtype=torch.uint8, device=dev) if codes is None else codes
    scale = torch.empty(1, dtype=torch.float32, device=dev) if scale is None else scale
    if workspace is None:
        workspace = torch.empty(MOE_QUANT_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)
    _check(lib().moe_quantize_act(_ptr(x), dtype_code(x.dtype), n, _ptr(static_scale),
                                  _ptr(codes), _ptr(scale), _ptr(workspace),
                                  workspace.numel() * workspace.element_size(),
                                  _stream(stream)))
    return codes, scale


def moe_fused_forward_noalloc(problem, x, w13, w2, topk_weights, alignment, out,
                              w13_scale=None, w2_scale=None, a1_scale=None, a2_scale=None,
                              stream=None):
    """moe_fused_forward on the library's own per-device scratch array (no
    workspace argument; nothing is allocated by the call)."""
    _check(lib().moe_fused_forward_noalloc(
        ctypes.byref(problem), _ptr(x), _ptr(w13), _ptr(w2), _ptr(w13_scale), _ptr(w2_scale),
        _ptr(a1_scale), _ptr(a2_scale), _ptr(topk_weights), _ptr(alignment.sorted_pair_ids),
        _ptr(alignment.block_expert_ids), _ptr(alignment.expert_offsets),
        _ptr(alignment.pair_pos), _ptr(alignment.num_padded), _ptr(out), _stream(stream)))
    return out


def moe_rope_workspace_size(T, n_heads, head_dim):
    n = ctypes.c_size_t(0)
    _check(lib().moe_rope_workspace_size(T, n_heads, head_dim, ctypes.byref(n)))
    return int(n.value)


def moe_rope_quantize_per_head(x, positions, inv_freq, interleaved=False, inverse=False,
                               static_scales=None, codes=None, scales=None, workspace=None,
                               stream=None):
    """x [T, nH, D] bf16/f32, positions int32 [T], inv_freq f32 [D/2] (device)
    -> (E4M3 codes uint8 [T, nH, D], scales f32 [nH])."""
    T, nH, D = x.shape
    dev = x.device
    codes = torch.empty(x.shape, dtype=torch.uint8, device=dev) if codes is None else codes
    scales = torch.empty(nH, dtype=torch.float32, device=dev) if scales is None else scales
    if workspace is None:
        workspace = torch.empty(max(moe_rope_workspace_size(T, nH, D), 16), dtype=torch.uint8,
                                device=dev)
    _check(lib().moe_rope_quantize_per_head(
        _ptr(x), dtype_code(x.dtype), _ptr(positions), _ptr(inv_freq), T, nH, D,
        int(bool(interleaved)), int(bool(inverse)), _ptr(static_scales), _ptr(codes),
        _ptr(scales), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return codes, scales


_VALUE_CODES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def _index(t, dims, first, name, device):
    """Address of a dense int32 index buffer of this many dimensions, the first
    of this size (None: any), on `device`."""
    if t.dtype is not torch.int32:
        raise MoEError(MOE_ERR_DTYPE, f"{name} must be int32")
    if t.dim() != dims or (first is not None and t.size(0) != first):
        raise MoEError(MOE_ERR_SHAPE, f"{name} has shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise MoEError(MOE_ERR_UNSUPPORTED, f"{name} must be contiguous")
    if t.device != device:
        raise MoEError(MOE_ERR_UNSUPPORTED, f"{name} is on {t.device}, not on {device}")
    return t.data_ptr()


def _heads(t, shape, name, device):
    """(address, dtype code, token stride, head stride) of a [tokens, heads,
    head_dim] tensor of this shape on `device`, the values of a head contiguous."""
    code = _VALUE_CODES.get(t.dtype)
    if code is None:
        raise MoEError(MOE_ERR_DTYPE, f"{name} must be bf16 or f32, not {t.dtype}")
    if t.shape != shape:
        raise MoEError(MOE_ERR_SHAPE, f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    st, sh, sd = t.stride()
    if sd != 1:
        raise MoEError(MOE_ERR_UNSUPPORTED, f"{name}: the values of a head must be contiguous")
    if t.device != device:
        raise MoEError(MOE_ERR_UNSUPPORTED, f"{name} is on {t.device}, not on {device}")
    # the strides of a dimension of size one are torch's to choose
    return t.data_ptr(), code, st if shape[0] > 1 else shape[1] * shape[2], sh if shape[1] > 1 else shape[2]


def _run(device, stream, call, *args):
    """call(*args, stream handle) with `device` current."""
    if device.type != "cuda":
        raise MoEError(MOE_ERR_UNSUPPORTED, f"tensors are on {device}, not on a GPU")
    if device.index != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _run(device, stream, call, *args)
    handle = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    status = call(*args, handle)
    if status != MOE_OK:
        _check(status)


def _made(like, shape, dtype, stream):
    """A tensor of `like`'s device (and type, if dtype is None) made for a call
    that runs on `stream` (None: the current one): from that stream's memory,
    so that nothing still at work on another one holds it, and not given back
    before the current stream is done with it."""
    if stream is None or not like.is_cuda:
        return like.new_empty(shape) if dtype is None else like.new_empty(shape, dtype=dtype)
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype or like.dtype)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


class Rotation:
    """Rotary positions (include/moe.h, moe_rotation): positions int32 [T] or
    [axes, T] (None in an append: the tokens' own places), inv_freq f32
    [rotary_dim / 2], pair_axis int32 [rotary_dim / 2] or None.  Keeps the
    tensors; positions may be rewritten in place between calls."""

    def __init__(self, positions, inv_freq, pair_axis=None, interleaved=False, inverse=False):
        dev = inv_freq.device
        if inv_freq.dtype is not torch.float32:
            raise MoEError(MOE_ERR_DTYPE, "inv_freq must be f32")
        if inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise MoEError(MOE_ERR_SHAPE, "inv_freq must be a dense vector")
        half = inv_freq.size(0)
        axes, at, self.tokens = 1, None, None
        if positions is not None:
            dims = positions.dim()
            if dims not in (1, 2):
                raise MoEError(MOE_ERR_SHAPE, "positions must be [T] or [axes, T]")
            at = _index(positions, dims, None, "positions", dev)
            axes = positions.size(0) if dims == 2 else 1
            self.tokens = positions.size(-1)
        axis_at = None if pair_axis is None else _index(pair_axis, 1, half, "pair_axis", dev)
        self.positions, self.inv_freq, self.pair_axis, self.device = positions, inv_freq, pair_axis, dev
        self.struct = moe_rotation(at, axis_at, inv_freq.data_ptr(), axes, 2 * half, 1 if interleaved else 0,
                                   1 if inverse else 0)

    def _for(self, T, device):
        if self.tokens is not None and self.tokens != T:
            raise MoEError(MOE_ERR_SHAPE, f"positions of {self.tokens} tokens for {T}")
        if self.device != device:
            raise MoEError(MOE_ERR_UNSUPPORTED, f"the rotation is on {self.device}, not on {device}")
        return ctypes.byref(self.struct)


def moe_rope_axes(x, rotation, out=None, out_dtype=None, stream=None):
    """x [T, nH, D] bf16/f32, heads contiguous -> x rotated (out may be x)."""
    shape, dev = x.shape, x.device
    if len(shape) != 3:
        raise MoEError(MOE_ERR_SHAPE, f"x has shape {tuple(shape)}, not [T, heads, head_dim]")
    T, nH, D = shape
    if out is None:
        out = _made(x, shape, out_dtype, stream)
    xp, xc, xt, xh = _heads(x, shape, "x", dev)
    op, oc, ot, oh = _heads(out, shape, "out", dev)
    _run(dev, stream, lib().moe_rope_axes, xp, xc, xt, xh, rotation._for(T, dev), T, nH, D, op, oc, ot, oh)
    return out


class PagedKV:
    """A paged E4M3 key/value cache (include/moe.h, moe_kv_cache) over the
    caller's tensors: k_codes [pages, H, S, D] and v_codes [pages, H, S/16, D,
    16] (float8_e4m3fn or uint8), k_scales and v_scales f32 [pages, H]."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        if k_codes.dim() != 4:
            raise MoEError(MOE_ERR_SHAPE, "k_codes must be [pages, heads, page_size, head_dim]")
        P, H, S, D = k_codes.shape
        for t, shape, name in ((k_codes, (P, H, S, D), "k_codes"), (v_codes, (P, H, S // 16, D, 16), "v_codes"),
                               (k_scales, (P, H), "k_scales"), (v_scales, (P, H), "v_scales")):
            if t.dtype not in ((torch.float8_e4m3fn, torch.uint8) if "codes" in name else (torch.float32,)):
                raise MoEError(MOE_ERR_DTYPE, f"{name} has dtype {t.dtype}")
            if t.shape != shape:
                raise MoEError(MOE_ERR_SHAPE, f"{name} has shape {tuple(t.shape)}, not {shape}")
            if not t.is_contiguous():
                raise MoEError(MOE_ERR_UNSUPPORTED, f"{name} must be contiguous")
            if t.device != k_codes.device:
                raise MoEError(MOE_ERR_UNSUPPORTED, f"{name} is on {t.device}, not on {k_codes.device}")
        self.k_codes, self.v_codes, self.k_scales, self.v_scales = k_codes, v_codes, k_scales, v_scales
        self.num_pages, self.n_kv_heads, self.page_size, self.head_dim = P, H, S, D
        self.device = k_codes.device
        self.struct = moe_kv_cache(k_codes.data_ptr(), v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                   P, S, H, D)

    def _batch(self, T, kv_lens, block_table, cu_q):
        dev = self.device
        lens = _index(kv_lens, 1, None, "kv_lens", dev)
        B = kv_lens.size(0)
        table = _index(block_table, 2, B, "block_table", dev)
        cu = None if cu_q is None else _index(cu_q, 1, B + 1, "cu_q", dev)
        return moe_kv_batch(cu, lens, table, B, T, block_table.size(1))


def alloc_kv_cache(num_pages, page_size, n_kv_heads, head_dim, device="cuda"):
    codes = dict(dtype=torch.float8_e4m3fn, device=device)
    return PagedKV(torch.empty(num_pages, n_kv_heads, page_size, head_dim, **codes),
                   torch.empty(num_pages, n_kv_heads, page_size // 16, head_dim, 16, **codes),
                   torch.empty(num_pages, n_kv_heads, device=device),
                   torch.empty(num_pages, n_kv_heads, device=device))


def moe_kv_append(cache, k, v, kv_lens, block_table, rotation=None, cu_q=None, stream=None):
    """k, v [T, H, D] bf16/f32 into the cache, k rotated first; kv_lens int32
    [B] (these rows included), block_table int32 [B, max_pages], cu_q int32
    [B + 1] or None (one row per sequence)."""
    T, dev = k.shape[0], cache.device
    shape = (T, cache.n_kv_heads, cache.head_dim)
    kp, kc, kt, kh = _heads(k, shape, "k", dev)
    vp, vc, vt, vh = _heads(v, shape, "v", dev)
    if kc != vc:
        raise MoEError(MOE_ERR_DTYPE, f"k is {k.dtype}, v is {v.dtype}")
    batch = cache._batch(T, kv_lens, block_table, cu_q)
    rot = None if rotation is None else rotation._for(T, dev)
    _run(dev, stream, lib().moe_kv_append, ctypes.byref(cache.struct), ctypes.byref(batch), kp, kt, kh, vp, vt, vh,
         kc, rot)


def moe_paged_attention_workspace_size(cache, T, B, n_heads, max_q=1):
    n = ctypes.c_size_t(0)
    _check(lib().moe_paged_attention_workspace_size(ctypes.byref(cache.struct), T, B, n_heads, max_q,
                                                    ctypes.byref(n)))
    return int(n.value)


def moe_paged_attention(cache, q, kv_lens, block_table, cu_q=None, max_q=None, sm_scale=None, causal=True, window=0,
                        out=None, lse=None, return_lse=False, workspace=None, stream=None):
    """q [T, nH, D] bf16/f32 (rotated) over the cache -> out [T, nH, D], and
    with return_lse (or lse given) the log sums lse f32 [T, nH].  max_q: at
    least the rows of every sequence (None: T, or 1 without cu_q).  sm_scale
    None: 1 / sqrt(D)."""
    shape, dev = q.shape, cache.device
    if len(shape) != 3 or shape[2] != cache.head_dim:
        raise MoEError(MOE_ERR_SHAPE, f"q has shape {tuple(shape)}, not [T, heads, {cache.head_dim}]")
    T, nH, D = shape
    qp, qc, qt, qh = _heads(q, shape, "q", dev)
    batch = cache._batch(T, kv_lens, block_table, cu_q)
    if max_q is None:
        max_q = 1 if cu_q is None else max(T, 1)
    if out is None:
        out = _made(q, shape, None, stream)
    elif out.dtype != q.dtype:
        raise MoEError(MOE_ERR_DTYPE, f"out is {out.dtype}, q is {q.dtype}")
    elif out.shape != shape or not out.is_contiguous() or out.device != dev:
        raise MoEError(MOE_ERR_SHAPE, f"out must be a dense {tuple(shape)} on the cache's device")
    if lse is None:
        if return_lse:
            lse = _made(q, (T, nH), torch.float32, stream)
    elif lse.dtype != torch.float32:
        raise MoEError(MOE_ERR_DTYPE, "lse must be f32")
    elif lse.shape != (T, nH) or not lse.is_contiguous() or lse.device != dev:
        raise MoEError(MOE_ERR_SHAPE, f"lse must be a dense {(T, nH)} on the cache's device")
    if workspace is None:
        size = moe_paged_attention_workspace_size(cache, T, batch.B, nH, max_q)
        workspace = _made(q, (max(size, 16),), torch.uint8, stream)
    elif not workspace.is_contiguous() or workspace.device != dev:
        raise MoEError(MOE_ERR_WORKSPACE, "the workspace must be dense and on the cache's device")
    _run(dev, stream, lib().moe_paged_attention, ctypes.byref(cache.struct), ctypes.byref(batch), qp, qc, qt, qh, nH,
         max_q, D ** -0.5 if sm_scale is None else sm_scale, 1 if causal else 0, window, out.data_ptr(),
         None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes)
    return out if lse is None else (out, lse)


@dataclass
class Alignment:
    sorted_pair_ids: torch.Tensor
    block_expert_ids: torch.Tensor
    expert_offsets: torch.Tensor
    pair_pos: torch.Tensor
    num_padded: torch.Tensor
    block_m: int


def alloc_alignment(M, topk, E, block_m, device):
    cap = max(moe_align_capacity(M, topk, E, block_m), 1)
    i32 = dict(dtype=torch.int32, device=device)
    return Alignment(torch.empty(cap, **i32), torch.empty((cap + block_m - 1) // block_m, **i32),
                     torch.empty(E + 1, **i32), torch.empty(max(M * topk, 1), **i32),
                     torch.empty(1, **i32), block_m)


def moe_align_permute(topk_ids, E, block_m, workspace, alignment=None, stream=None):
    M, topk = topk_ids.shape
    al = alignment or alloc_alignment(M, topk, E, block_m, topk_ids.device)
    _check(lib().moe_align_permute(_ptr(topk_ids), M, topk, E, block_m,
                                   _ptr(al.sorted_pair_ids), _ptr(al.block_expert_ids),
                                   _ptr(al.expert_offsets), _ptr(al.pair_pos),
                                   _ptr(al.num_padded), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(),
                                   _stream(stream)))
    return al


def moe_route_align(logits, topk, renormalize, block_m, workspace, topk_ids=None,
                    topk_weights=None, alignment=None, stream=None):
    """Routing and alignment (one launch for M*topk <= 1024)."""
    M, E = logits.shape
    dev = logits.device
    if topk_ids is None:
        topk_ids = torch.empty(M, topk, dtype=torch.int32, device=dev)
    if topk_weights is None:
        topk_weights = torch.empty(M, topk, dtype=torch.float32, device=dev)
    al = alignment or alloc_alignment(M, topk, E, block_m, dev)
    _check(lib().moe_route_align(_ptr(logits), M, E, topk, int(bool(renormalize)), block_m,
                                 _ptr(topk_ids), _ptr(topk_weights), _ptr(al.sorted_pair_ids),
                                 _ptr(al.block_expert_ids), _ptr(al.expert_offsets),
                                 _ptr(al.pair_pos), _ptr(al.num_padded), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))
    return topk_ids, topk_weights, al


def moe_fused_forward(problem, x, w13, w2, topk_weights, alignment, out, workspace,
                      w13_scale=None, w2_scale=None, a1_scale=None, a2_scale=None,
                      stream=None, events=None):
    """events: None, or four hipEvent_t handles (ints or None) recorded around
    the two GEMM launches (moe_fused_forward_profiled)."""
    args = (ctypes.byref(problem), _ptr(x), _ptr(w13), _ptr(w2), _ptr(w13_scale),
            _ptr(w2_scale), _ptr(a1_scale), _ptr(a2_scale), _ptr(topk_weights),
            _ptr(alignment.sorted_pair_ids), _ptr(alignment.block_expert_ids),
            _ptr(alignment.expert_offsets), _ptr(alignment.pair_pos),
            _ptr(alignment.num_padded), _ptr(out), _ptr(workspace),
            workspace.numel() * workspace.element_size(), _stream(stream))
    if events is None:
        _check(lib().moe_fused_forward(*args))
    else:
        ev = (ctypes.c_void_p * 4)(*[(e or None) for e in events])
        _check(lib().moe_fused_forward_profiled(*args, ev))
    return out


def alloc_fused_sync(device="cuda"):
    """A zeroed synchronisation buffer for moe_fused_forward_persistent (one
    per stream; every call leaves it ready for the next)."""
    return torch.zeros(MOE_FUSED_SYNC_BYTES, dtype=torch.uint8, device=device)


def fused_sync_error(sync):
    """The error word of a synchronisation buffer (nonzero: a grid-wide wait
    of an earlier call gave up); reads the device, so it synchronises."""
    o = MOE_FUSED_SYNC_ERROR_OFFSET
    return int(sync[o:o + 4].view(torch.int32).item())


def moe_fused_forward_persistent(problem, x, w13, w2, topk_weights, alignment, out, workspace,
                                 sync, w13_scale=None, w2_scale=None, a1_scale=None,
                                 a2_scale=None, stream=None):
    """moe_fused_forward for E4M3 decode batches in one kernel launch; sync is
    a zero-initialised MOE_FUSED_SYNC_BYTES buffer (alloc_fused_sync)."""
    _check(lib().moe_fused_forward_persistent(
        ctypes.byref(problem), _ptr(x), _ptr(w13), _ptr(w2), _ptr(w13_scale), _ptr(w2_scale),
        _ptr(a1_scale), _ptr(a2_scale), _ptr(topk_weights), _ptr(alignment.sorted_pair_ids),
        _ptr(alignment.block_expert_ids), _ptr(alignment.expert_offsets),
        _ptr(alignment.pair_pos), _ptr(alignment.num_padded), _ptr(out), _ptr(workspace),
        workspace.numel() * workspace.element_size(), _ptr(sync),
        sync.numel() * sync.element_size(), _stream(stream)))
    return out


class FusedMoE:
    """The three calls with their buffers allocated once for a fixed maximum
    M (route -> align -> forward).  Buffers are reused between calls, so
    nothing is allocated or synchronised per call and the sequence can be
    captured into a HIP graph."""

    def __init__(self, M, K, N, E, topk, w13, w2, w13_scale=None, w2_scale=None,
                 block_m=None, a_dtype=torch.bfloat16, out_dtype=torch.bfloat16,
                 renormalize=True, a1_scale=None, a2_scale=None, device="cuda",
                 persistent=False, prequant=None):
        if block_m is None:
            # alignment block: 16 rows for decode-sized batches (the stream and
            # ring kernels), 256 once the experts average 512 rows or more (the
            # 256 x 256 prefill tiles), else 128
            block_m = 16 if M <= 64 else (256 if M * topk >= 512 * E else 128)
        self.M, self.K, self.N, self.E, self.topk = M, K, N, E, topk
        self.block_m, self.renormalize = block_m, renormalize
        self.w13, self.w2, self.w13_scale, self.w2_scale = w13, w2, w13_scale, w2_scale
        self.a1_scale, self.a2_scale = a1_scale, a2_scale
        self.problem = make_problem(M, K, N, E, topk, block_m, a_dtype, w13.dtype, out_dtype)
        ws = moe_workspace_size(self.problem)
        self.workspace = torch.empty(max(ws, 16), dtype=torch.uint8, device=device)
        self.topk_ids = torch.empty(M, topk, dtype=torch.int32, device=device)
        self.topk_weights = torch.empty(M, topk, dtype=torch.float32, device=device)
        self.alignment = alloc_alignment(M, topk, E, block_m, device)
        self.out = torch.empty(M, K, dtype=out_dtype, device=device)
        # persistent: the forward runs as one launch (moe_fused_forward_persistent);
        # prequant (E4M3 weights; default: with the one launch only): the
        # activation codes are made by moe_quantize_act right after the
        # routing, and the forward starts from them (the one launch then
        # starts at gate/up)
        self.persistent = persistent
        self.sync = alloc_fused_sync(device) if persistent else None
        if prequant is None:
            prequant = persistent
        self.prequant = bool(prequant) and w13.dtype == torch.float8_e4m3fn
        if self.prequant:
            self.problem_q = make_problem(M, K, N, E, topk, block_m, torch.float8_e4m3fn,
                                          w13.dtype, out_dtype)
            self.xq = torch.empty(M, K, dtype=torch.uint8, device=device)
            self.xscale = torch.empty(1, dtype=torch.float32, device=device)
            self.qws = torch.empty(MOE_QUANT_WORKSPACE_BYTES, dtype=torch.uint8, device=device)

    def act_scales(self):
        """Device view of the (s_x, s_h) fp32 pair that the last E4M3 forward
        left in the workspace (include/moe.h, MOE_WORKSPACE_SCALES_OFFSET)."""
        o = MOE_WORKSPACE_SCALES_OFFSET
        return self.workspace[o:o + 8].view(torch.float32)

    def __call__(self, x, logits, stream=None, events=None):
        self.prepare(x, logits, stream)
        return self.forward(x, stream, events)

    def prepare(self, x, logits, stream=None):
        """Routing and alignment; in prequant mode then the activation codes."""
        self.route(logits, stream)
        if self.prequant:
            self.quantize(x, stream)

    def route(self, logits, stream=None):
        moe_route_align(logits, self.topk, self.renormalize, self.block_m, self.workspace,
                        self.topk_ids, self.topk_weights, self.alignment, stream)

    def quantize(self, x, stream=None):
        """The activation codes and scale of x (prequant mode)."""
        moe_quantize_act(x, self.a1_scale, self.xq, self.xscale, self.qws, stream)

    def forward(self, x, stream=None, events=None):
        if self.prequant and self.persistent:
            moe_fused_forward_persistent(self.problem_q, self.xq, self.w13, self.w2,
                                         self.topk_weights, self.alignment, self.out,
                                         self.workspace, self.sync, self.w13_scale,
                                         self.w2_scale, self.xscale, self.a2_scale, stream)
        elif self.prequant:
            moe_fused_forward(self.problem_q, self.xq, self.w13, self.w2, self.topk_weights,
                              self.alignment, self.out, self.workspace, self.w13_scale,
                              self.w2_scale, self.xscale, self.a2_scale, stream, events)
        elif self.persistent:
            moe_fused_forward_persistent(self.problem, x, self.w13, self.w2, self.topk_weights,
                                         self.alignment, self.out, self.workspace, self.sync,
                                         self.w13_scale, self.w2_scale, self.a1_scale,
                                         self.a2_scale, stream)
        else:
            moe_fused_forward(self.problem, x, self.w13, self.w2, self.topk_weights,
                              self.alignment, self.out, self.workspace, self.w13_scale,
                              self.w2_scale, self.a1_scale, self.a2_scale, stream, events)
        return self.out


class PagedAttention:
    """The attention of a decoder layer ahead of its experts: queries and keys
    rotated, keys and values into the paged cache, attention over it (the calls
    moe_rope_axes, moe_kv_append and moe_paged_attention), with the buffers
    allocated once for at most max_tokens rows in max_seqs sequences of at most
    max_q rows (None: as many as there are).  Nothing is allocated or synchronised per call, so the sequence
    can be captured into a HIP graph; lengths, tables and positions are read on
    the device and may change between replays.  The rotated queries, out and the
    workspace are the object's: calls of one object, and replays of graphs that
    hold them, must not overlap in time, and out holds until the next."""

    def __init__(self, cache, n_heads, inv_freq, max_tokens, max_seqs=None, max_q=None, pair_axis=None,
                 interleaved=False, sm_scale=None, causal=True, window=0, dtype=torch.bfloat16):
        self.cache, self.n_heads, self.max_q = cache, n_heads, max_q or max_tokens
        self.inv_freq, self.pair_axis, self.interleaved = inv_freq, pair_axis, interleaved
        self.sm_scale, self.causal, self.window = sm_scale, causal, window
        shape = (max_tokens, n_heads, cache.head_dim)
        self.q = torch.empty(shape, dtype=dtype, device=cache.device)
        self.out = torch.empty(shape, dtype=dtype, device=cache.device)
        seqs = max_seqs or min(max_tokens, MOE_MAX_SEQS)
        n = moe_paged_attention_workspace_size(cache, max_tokens, seqs, n_heads, self.max_q)
        self.workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=cache.device)

    def __call__(self, q, k, v, positions, kv_lens, block_table, cu_q=None, stream=None):
        """q [T, n_heads, D], k and v [T, n_kv_heads, D]; positions int32 [T] or
        [axes, T]; kv_lens counts these rows.  Returns out [T, n_heads, D], this
        object's buffer."""
        T = q.shape[0]
        if T > self.out.shape[0]:
            raise MoEError(MOE_ERR_SHAPE, f"T={T} rows, buffers for {self.out.shape[0]}")
        rotation = Rotation(positions, self.inv_freq, self.pair_axis, self.interleaved)
        moe_rope_axes(q, rotation, out=self.q[:T], stream=stream)
        moe_kv_append(self.cache, k, v, kv_lens, block_table, rotation=rotation, cu_q=cu_q, stream=stream)
        return moe_paged_attention(self.cache, self.q[:T], kv_lens, block_table, cu_q=cu_q,
                                   max_q=1 if cu_q is None else self.max_q, sm_scale=self.sm_scale,
                                   causal=self.causal, window=self.window, out=self.out[:T],
                                   workspace=self.workspace, stream=stream)
