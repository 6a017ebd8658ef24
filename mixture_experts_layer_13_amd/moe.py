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
           "moe_paged_attention_workspace_size", "moe_dispatch", "moe_dispatch_backward", "moe_combine",
           "moe_combine_backward", "moe_quantize_blocks", "moe_block_matmul", "moe_block_matmul_grouped")
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


class moe_alignment(ctypes.Structure):
    _fields_ = ([(n, ctypes.c_void_p) for n in ("sorted_pair_ids", "block_expert_ids", "expert_offsets", "pair_pos",
                                                "num_padded")] +
                [(n, ctypes.c_int32) for n in ("M", "topk", "E", "block_m", "rows")])


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
        al = ctypes.POINTER(moe_alignment)
        L.moe_dispatch.argtypes = [al, vp, i32, i64, i32, vp, vp, i32, i64, vp]
        L.moe_dispatch_backward.argtypes = [al, vp, i32, i64, i32, vp, i64, vp, vp, i32, i64, vp, vp]
        L.moe_combine.argtypes = [al, vp, i32, i64, i32, vp, vp, i32, i64, vp]
        L.moe_combine_backward.argtypes = [al, vp, i32, i64, i32, vp, i64, vp, vp, i32, i64, vp, vp]
        L.moe_quantize_blocks.argtypes = [vp, i32, i64, i32, i32, i32, i32, vp, vp, vp, i64, i64, vp]
        L.moe_block_matmul.argtypes = [vp, i64, vp, i64, i64, vp, vp, i32, i32, i32, vp, i32, i64, vp]
        L.moe_block_matmul_grouped.argtypes = [al, vp, i64, i32, vp, i64, i64, vp, vp, i32, i32, i32, vp, i32, i64, vp]
        for f in (L.moe_dispatch, L.moe_dispatch_backward, L.moe_combine, L.moe_combine_backward,
                  L.moe_quantize_blocks, L.moe_block_matmul, L.moe_block_matmul_grouped):
            f.restype = ctypes.c_int
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
    # M * topk of the call that last filled the buffers (moe_align_permute,
    # moe_route_align; a graph's replay is not seen), which may be fewer than they
    # hold; None: not known
    pairs: int | None = None


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
    al.pairs, al.block_m = M * topk, block_m
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
    al.pairs, al.block_m = M * topk, block_m
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


def _rows(t, rows, values, name, device):
    """(address, dtype code, row stride) of a [rows, values] tensor (None: any
    number) on `device`, the values of a row contiguous."""
    code = _VALUE_CODES.get(t.dtype)
    if code is None:
        raise MoEError(MOE_ERR_DTYPE, f"{name} must be bf16 or f32, not {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or (rows is not None and shape[0] != rows) or (values is not None and shape[1] != values):
        raise MoEError(MOE_ERR_SHAPE, f"{name} has shape {tuple(shape)}, not {(rows, values)}")
    st, sv = t.stride()
    if sv != 1 and shape[1] > 1:
        raise MoEError(MOE_ERR_UNSUPPORTED, f"{name}: the values of a row must be contiguous")
    if t.device != device:
        raise MoEError(MOE_ERR_UNSUPPORTED, f"{name} is on {t.device}, not on {device}")
    # the stride of a dimension of size one is torch's to choose
    return t.data_ptr(), code, st if shape[0] > 1 else shape[1]


def _made_rows(like, rows, values, dtype, stream, columns=False):
    """_made of [rows, values], a row's values side by side (columns: a column's)."""
    if stream is None:  # half the time of new_empty with a dtype, and a third of it with t()
        return torch.empty_strided((rows, values), (1, rows or 1) if columns else (values, 1), dtype=dtype,
                                   device=like.device)
    t = _made(like, (values, rows) if columns else (rows, values), dtype, stream)
    return t.t() if columns else t


def _out(out, like, rows, values, dtype, stream):
    """(out, address, dtype code, row stride) of a given [rows, values], or of one
    made of this type."""
    if out is not None:
        return out, *_rows(out, rows, values, "out", like.device)
    code = _VALUE_CODES.get(dtype)
    if code is None:
        raise MoEError(MOE_ERR_DTYPE, f"out must be bf16 or f32, not {dtype}")
    out = _made_rows(like, rows, values, dtype, stream)
    return out, out.data_ptr(), code, values


def _pairs_f32(t, shape, name, device):
    """Address of a dense f32 tensor of this shape on `device` (None: None)."""
    if t is None:
        return None
    if t.dtype is not torch.float32:
        raise MoEError(MOE_ERR_DTYPE, f"{name} must be f32")
    if t.shape != shape:
        raise MoEError(MOE_ERR_SHAPE, f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous() or t.device != device:
        raise MoEError(MOE_ERR_UNSUPPORTED, f"{name} must be contiguous and on {device}")
    return t.data_ptr()


def _places(al, M, topk, device, padding):
    """The moe_alignment of M tokens of topk pairs as far as the movements read it
    (padding: with what tells padding rows), and its rows."""
    pos, rows = _index(al.pair_pos, 1, None, "pair_pos", device), al.sorted_pair_ids.size(0)
    if al.pair_pos.size(0) < M * topk:
        raise MoEError(MOE_ERR_SHAPE, f"pair_pos of {al.pair_pos.size(0)} pairs for {M} x {topk}")
    if not padding:
        return moe_alignment(None, None, None, pos, None, M, topk, 0, 0, rows), rows
    ids = _index(al.sorted_pair_ids, 1, None, "sorted_pair_ids", device)
    used = _index(al.num_padded, 1, 1, "num_padded", device)
    return moe_alignment(ids, None, None, pos, used, M, topk, 0, 0, rows), rows


def _segments(al, M, topk, E, device):
    """The moe_alignment of M * topk pairs and E experts as far as the products
    read it, and its rows."""
    ids = _index(al.sorted_pair_ids, 1, None, "sorted_pair_ids", device)
    rows, bm = al.sorted_pair_ids.size(0), al.block_m
    blocks = _index(al.block_expert_ids, 1, None, "block_expert_ids", device)
    if bm < 1 or al.block_expert_ids.size(0) * bm < rows:
        raise MoEError(MOE_ERR_SHAPE, f"block_expert_ids of {al.block_expert_ids.size(0)} blocks for {rows} rows")
    offsets = _index(al.expert_offsets, 1, E + 1, "expert_offsets", device)
    used = _index(al.num_padded, 1, 1, "num_padded", device)
    return moe_alignment(ids, blocks, offsets, None, used, M, topk, E, bm, rows), rows


def moe_dispatch(x, alignment, topk, weights=None, out=None, out_dtype=None, stream=None):
    """x [M, K] bf16/f32 into expert order: rows [rows, K], rows[place of pair] =
    weight * token; weights f32 [M, topk] or None (1).  Rows of padding are zero,
    those from num_padded on as they were (in a new tensor: anything)."""
    dev = x.device
    xp, xc, xs = _rows(x, None, None, "x", dev)
    M, K = x.shape
    al, rows = _places(alignment, M, topk, dev, True)
    wp = None if weights is None else _pairs_f32(weights, (M, topk), "weights", dev)
    out, op, oc, ost = _out(out, x, rows, K, out_dtype or x.dtype, stream)
    _run(dev, stream, lib().moe_dispatch, al, xp, xc, xs, K, wp, op, oc, ost)
    return out


def moe_dispatch_backward(d_rows, alignment, M, topk, x=None, weights=None, out=None, out_dtype=None, stream=None):
    """The gradient of moe_dispatch: d_rows [rows, K] -> (dx [M, K], d_weights f32
    [M, topk], or None without x, which only they need)."""
    dev = d_rows.device
    al, rows = _places(alignment, M, topk, dev, False)
    rp, rc, rs = _rows(d_rows, rows, None, "d_rows", dev)
    K = d_rows.size(1)
    wp = None if weights is None else _pairs_f32(weights, (M, topk), "weights", dev)
    xp, xc, xs, dw, dwp = None, None, 0, None, None
    if x is not None:
        xp, xc, xs = _rows(x, M, K, "x", dev)
        dw = _made_rows(d_rows, M, topk, torch.float32, stream)
        dwp = dw.data_ptr()
    out, op, oc, ost = _out(out, d_rows, M, K, out_dtype or (d_rows if x is None else x).dtype, stream)
    if xc is not None and xc != oc:
        raise MoEError(MOE_ERR_DTYPE, f"x is {x.dtype}, its gradient {out.dtype}")
    _run(dev, stream, lib().moe_dispatch_backward, al, rp, rc, rs, K, xp, xs, wp, op, oc, ost, dwp)
    return out, dw


def moe_combine(rows, alignment, M, topk, weights=None, out=None, out_dtype=None, stream=None):
    """rows [rows, K] bf16/f32 in expert order back to tokens: out [M, K], out[t] =
    the sum of weight * row over the token's pairs; weights as in moe_dispatch."""
    dev = rows.device
    al, n = _places(alignment, M, topk, dev, False)
    rp, rc, rs = _rows(rows, n, None, "rows", dev)
    K = rows.size(1)
    wp = None if weights is None else _pairs_f32(weights, (M, topk), "weights", dev)
    out, op, oc, ost = _out(out, rows, M, K, out_dtype or rows.dtype, stream)
    _run(dev, stream, lib().moe_combine, al, rp, rc, rs, K, wp, op, oc, ost)
    return out


def moe_combine_backward(d_out, alignment, topk, rows=None, weights=None, out=None, out_dtype=None, stream=None):
    """The gradient of moe_combine: d_out [M, K] -> (d_rows [rows, K], d_weights f32
    [M, topk], or None without rows, which only they need)."""
    dev = d_out.device
    gp, gc, gs = _rows(d_out, None, None, "d_out", dev)
    M, K = d_out.shape
    al, n = _places(alignment, M, topk, dev, True)
    wp = None if weights is None else _pairs_f32(weights, (M, topk), "weights", dev)
    rp, rc, rs, dw, dwp = None, None, 0, None, None
    if rows is not None:
        rp, rc, rs = _rows(rows, n, K, "rows", dev)
        dw = _made_rows(d_out, M, topk, torch.float32, stream)
        dwp = dw.data_ptr()
    out, op, oc, ost = _out(out, d_out, n, K, out_dtype or (d_out if rows is None else rows).dtype, stream)
    if rc is not None and rc != oc:
        raise MoEError(MOE_ERR_DTYPE, f"rows are {rows.dtype}, their gradient {out.dtype}")
    _run(dev, stream, lib().moe_combine_backward, al, gp, gc, gs, K, rp, rs, wp, op, oc, ost, dwp)
    return out, dw


_CODES = (torch.float8_e4m3fn, torch.uint8)


def moe_quantize_blocks(x, gated=False, block_rows=1, num_rows=None, codes=None, scales=None, stream=None):
    """x bf16/f32 [M, K] (gated: [M, 2K], the values are SiLU(gate) * up) -> E4M3
    codes [M, K] and f32 scales, one per row and 128 values: [M, blocks], by
    default the rows of a block side by side (scales.stride(0) == 1); block_rows
    128: one per 128 x 128 block, [row blocks, blocks] dense, and x may be [E, N,
    K], expert by expert.  num_rows int32 [1]: rows from there on are left alone."""
    dev = x.device
    if x.dim() == 3:
        if block_rows != 128:
            raise MoEError(MOE_ERR_SHAPE, "x of three dimensions needs block_rows 128")
        E, N, K = x.shape
        if codes is None:
            codes = _made(x, (E, N, K), torch.float8_e4m3fn, stream)
        elif codes.shape != (E, N, K):
            raise MoEError(MOE_ERR_SHAPE, f"codes have shape {tuple(codes.shape)}, not {(E, N, K)}")
        blocks = (E, -(-N // 128), -(-K // 128))
        if scales is None:
            scales = _made(x, blocks, torch.float32, stream)
        elif scales.shape != blocks:
            raise MoEError(MOE_ERR_SHAPE, f"scales have shape {tuple(scales.shape)}, not {blocks}")
        for e in range(E):
            moe_quantize_blocks(x[e], gated, 128, num_rows, codes[e], scales[e], stream)
        return codes, scales
    xp, xc, xs = _rows(x, None, None, "x", dev)
    M, K = x.shape
    if gated:
        if K % 2:
            raise MoEError(MOE_ERR_SHAPE, f"gated x has {K} values a row")
        K //= 2
    SR, SB = M if block_rows == 1 else -(-M // max(block_rows, 1)), -(-K // 128)
    if codes is None:
        codes = _made_rows(x, M, K, torch.float8_e4m3fn, stream)
    elif codes.dtype not in _CODES:
        raise MoEError(MOE_ERR_DTYPE, f"codes are {codes.dtype}")
    elif codes.shape != (M, K) or not codes.is_contiguous() or codes.device != dev:
        raise MoEError(MOE_ERR_SHAPE, f"codes must be a dense {(M, K)} on {dev}")
    if scales is not None:
        sp, sr, sb = _scales(scales, SR, SB, "scales", dev)
    elif block_rows == 1:
        scales = _made_rows(x, SR, SB, torch.float32, stream, True)
        sp, sr, sb = scales.data_ptr(), 1, SR or 1
    else:
        scales = _made_rows(x, SR, SB, torch.float32, stream)
        sp, sr, sb = scales.data_ptr(), SB, 1
    limit = None if num_rows is None else _index(num_rows, 1, 1, "num_rows", dev)
    _run(dev, stream, lib().moe_quantize_blocks, xp, xc, xs, M, K, 1 if gated else 0, block_rows, limit,
         codes.data_ptr(), sp, sr, sb)
    return codes, scales


def _scales(t, rows, blocks, name, device):
    """(address, row stride, block stride) of f32 scales [rows, blocks]."""
    if t.dtype is not torch.float32:
        raise MoEError(MOE_ERR_DTYPE, f"{name} must be f32")
    if t.shape != (rows, blocks):
        raise MoEError(MOE_ERR_SHAPE, f"{name} have shape {tuple(t.shape)}, not {(rows, blocks)}")
    if t.device != device:
        raise MoEError(MOE_ERR_UNSUPPORTED, f"{name} are on {t.device}, not on {device}")
    sr, sb = t.stride()
    # the strides of a dimension of size one are torch's to choose
    return t.data_ptr(), sr if rows > 1 else 1, sb if blocks > 1 else 1


def _block_operands(a, a_scales, w, w_scales, dims):
    """(M, N, K, addresses and strides of a, its scales, w and its scales)."""
    dev, wshape = a.device, w.shape
    if a.dim() != 2 or len(wshape) != dims or wshape[-1] != a.size(1):
        raise MoEError(MOE_ERR_SHAPE, f"a has shape {tuple(a.shape)}, w {tuple(wshape)}")
    M, K = a.shape
    N, B = wshape[-2], -(-K // 128)
    if a.dtype not in _CODES or w.dtype not in _CODES:
        raise MoEError(MOE_ERR_DTYPE, f"a and w must be E4M3 codes, not {a.dtype} and {w.dtype}")
    st, sv = a.stride()
    if sv != 1 or not w.is_contiguous() or not w_scales.is_contiguous():
        raise MoEError(MOE_ERR_UNSUPPORTED, "the codes of a row must be contiguous, w and w_scales dense")
    if w.device != dev or w_scales.device != dev:
        raise MoEError(MOE_ERR_UNSUPPORTED, f"w and w_scales must be on {dev}")
    want = (-(-N // 128), B) if dims == 2 else (wshape[0], -(-N // 128), B)
    if w_scales.dtype is not torch.float32 or w_scales.shape != want:
        raise MoEError(MOE_ERR_SHAPE, f"w_scales must be f32 {want}")
    return M, N, K, a.data_ptr(), st if M > 1 else K, _scales(a_scales, M, B, "a_scales", dev), w.data_ptr(), w_scales.data_ptr()


def moe_block_matmul(a, a_scales, w, w_scales, out=None, out_dtype=torch.bfloat16, stream=None):
    """a [M, K] and w [N, K] of E4M3 codes, a_scales f32 [M, ceil(K / 128)] (any
    strides), w_scales f32 [ceil(N / 128), ceil(K / 128)] -> out [M, N].  An f32 out
    adds all products in fp32; a bf16 one cuts each eight below 2^-13 of the largest
    (include/moe.h)."""
    dev = a.device
    M, N, K, ap, ast, (sp, sr, sb), wp, wsp = _block_operands(a, a_scales, w, w_scales, 2)
    out, op, oc, ost = _out(out, a, M, N, out_dtype, stream)
    _run(dev, stream, lib().moe_block_matmul, ap, ast, sp, sr, sb, wp, wsp, M, N, K, op, oc, ost)
    return out


def moe_block_matmul_grouped(a, a_scales, w, w_scales, alignment, topk=None, M=None, pairs=None, out=None,
                             out_dtype=torch.bfloat16, stream=None):
    """The rows of an alignment times their experts' weights w [E, N, K], w_scales
    f32 [E, ceil(N / 128), ceil(K / 128)] -> out [rows, N].  With topk, a holds
    tokens (M of them, or more) and a place reads its pair's token; without, a
    [rows, K] is in expert order, of `pairs` pairs.  By default these are those of
    the alignment (alignment.pairs), or where it does not know them all that a or
    pair_pos holds.  Padding rows are zero, those from num_padded on as they were
    (in a new tensor: anything)."""
    dev = a.device
    A, N, K, ap, ast, (sp, sr, sb), wp, wsp = _block_operands(a, a_scales, w, w_scales, 3)
    known = alignment.pairs
    if topk is None:
        if pairs is None:
            pairs = alignment.pair_pos.size(0) if known is None else known
        al, rows = _segments(alignment, pairs, 1, w.size(0), dev)
    else:
        if M is None:
            M = A if known is None else known // max(topk, 1)
            if known is not None and M * topk != known:
                raise MoEError(MOE_ERR_SHAPE, f"an alignment of {known} pairs, topk {topk}")
        al, rows = _segments(alignment, M, topk, w.size(0), dev)
    out, op, oc, ost = _out(out, a, rows, N, out_dtype, stream)
    _run(dev, stream, lib().moe_block_matmul_grouped, al, ap, ast, A, sp, sr, sb, wp, wsp, N, K,
         0 if topk is None else 1, op, oc, ost)
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


class BlockMoE:
    """The layer of FusedMoE with block-scaled E4M3 weights (moe_quantize_blocks
    with block_rows 128 makes them): route and align, activations to E4M3 by token
    and 128 channels, gate/up product, SiLU(gate) * up to E4M3, down product,
    weighted combine.  w13 [E, 2N, K] and w2 [E, K, N] of codes, their scales f32
    [E, ceil(2N / 128), ceil(K / 128)] and [E, ceil(K / 128), ceil(N / 128)].  The
    products' results are held in bf16: a rounding of 2^-8 ahead of E4M3's 2^-4, or
    of the sum over a token's experts; each eight of their products are cut below
    2^-13 of the largest, as for any bf16 result of moe_block_matmul.  Buffers are allocated once for M tokens and
    reused, so that nothing is allocated or synchronised per call and the sequence
    can be captured into a HIP graph; calls of one object, and replays of graphs
    that hold them, must not overlap in time, and out holds until the next."""

    def __init__(self, M, K, N, E, topk, w13, w13_scales, w2, w2_scales, block_m=None, out_dtype=torch.bfloat16,
                 renormalize=True, device="cuda"):
        if w13.shape != (E, 2 * N, K) or w2.shape != (E, K, N):
            raise MoEError(MOE_ERR_SHAPE, f"w13 has shape {tuple(w13.shape)}, w2 {tuple(w2.shape)}")
        if block_m is None:
            # the products' tiles do not depend on it, and more of it is more padding:
            # 64 tokens 176 us (of 256: 254), 8192 1171 (1200)
            block_m = 16
        self.M, self.E, self.topk, self.block_m, self.renormalize = M, E, topk, block_m, renormalize
        self.w13, self.w13_scales, self.w2, self.w2_scales = w13, w13_scales, w2, w2_scales
        like = dict(dtype=torch.bfloat16, device=device)
        # the alignment's part of a workspace does not depend on the layer's sizes
        problem = make_problem(M, 128, 128, E, topk, block_m, torch.bfloat16, torch.bfloat16, torch.bfloat16)
        self.workspace = torch.empty(max(moe_workspace_size(problem), 16), dtype=torch.uint8, device=device)
        self.topk_ids = torch.empty(M, topk, dtype=torch.int32, device=device)
        self.topk_weights = torch.empty(M, topk, device=device)
        self.alignment = alloc_alignment(M, topk, E, block_m, device)
        rows = self.alignment.sorted_pair_ids.size(0)
        codes = dict(dtype=torch.float8_e4m3fn, device=device)
        self.x_codes, self.x_scales = torch.empty(M, K, **codes), torch.empty(-(-K // 128), M, device=device).t()
        self.gate_up = torch.empty(rows, 2 * N, **like)
        self.h_codes, self.h_scales = torch.empty(rows, N, **codes), torch.empty(-(-N // 128), rows, device=device).t()
        self.y = torch.empty(rows, K, **like)
        self.out = torch.empty(M, K, dtype=out_dtype, device=device)

    def __call__(self, x, logits, stream=None):
        """x [M, K] bf16/f32, logits f32 [M, E] -> out [M, K], this object's buffer."""
        dev, al = self.out.device, self.alignment
        if x.shape[0] != self.M:
            raise MoEError(MOE_ERR_SHAPE, f"{x.shape[0]} tokens, buffers for {self.M}")
        if x.device != dev:
            raise MoEError(MOE_ERR_UNSUPPORTED, f"x is on {x.device}, not on {dev}")
        _pairs_f32(logits, (self.M, self.E), "logits", dev)  # (the routing takes them as such)
        if dev.type != "cuda":
            raise MoEError(MOE_ERR_UNSUPPORTED, f"tensors are on {dev}, not on a GPU")
        if dev.index != torch._C._cuda_getDevice():
            with torch.cuda.device(dev):
                return self(x, logits, stream)
        moe_route_align(logits, self.topk, self.renormalize, self.block_m, self.workspace, self.topk_ids,
                        self.topk_weights, al, stream)
        moe_quantize_blocks(x, codes=self.x_codes, scales=self.x_scales, stream=stream)
        moe_block_matmul_grouped(self.x_codes, self.x_scales, self.w13, self.w13_scales, al, topk=self.topk,
                                 out=self.gate_up, stream=stream)
        moe_quantize_blocks(self.gate_up, gated=True, num_rows=al.num_padded, codes=self.h_codes, scales=self.h_scales,
                            stream=stream)
        moe_block_matmul_grouped(self.h_codes, self.h_scales, self.w2, self.w2_scales, al, out=self.y, stream=stream)
        return moe_combine(self.y, al, self.M, self.topk, weights=self.topk_weights, out=self.out, stream=stream)


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
