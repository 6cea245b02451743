"""Python binding of libmoe355 (ctypes).

Argument marshalling only: every step of the layer runs in the HIP kernels of
libmoe355.so.  Tensors are torch CUDA (HIP) tensors; outputs are allocated
here when not passed in, and every call is queued on torch's current stream.
A missing library raises at the first call -- there is no fallback.

Function names and argument order follow include/moe355.h.
"""
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe355.so")
_lib = None

_i32, _i64, _f32, _vp, _sz = ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
_P64, _PSZ = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_size_t)

_SIGNATURES = {
    "moe355_strerror": ([_i32], ctypes.c_char_p),
    "grouped_topk": ([_vp, _i32, _i64, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _f32, _vp, _vp, _i64, _vp], _i32),
    "moe_sort_sizes": ([_i32, _i32, _i32, _i32, _P64, _P64, _PSZ], _i32),
    "moe_block_m": ([_i32, _i32, _i32, ctypes.POINTER(ctypes.c_int)], _i32),
    "moe_sort": ([_vp, _vp, _i64, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "fp8_quant_1x128": ([_vp, _i64, _i32, _i32, _vp, _i64, _vp, _i64, _i64, _vp], _i32),
    "moe_fp8_blockscale_g1u1": ([_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32,
                                 _i64, _vp, _vp, _vp, _vp], _i32),
    "moe_down_combine_workspace": ([_i32, _i32, _i32, _PSZ], _i32),
    "moe_down_combine": ([_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _i64, _vp,
                          _i64, _vp, _sz, _vp], _i32),
    "gemm_fp8_blockscale_workspace": ([_i32, _i32, _i32, _PSZ], _i32),
    "gemm_fp8_blockscale": ([_vp, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _i64, _i32, _vp, _sz, _vp],
                            _i32),
    "shuffle_weight_128x128": ([_vp, _i64, _i32, _vp, _vp], _i32),
    "gemm_fp8_blockscale_noalloc": ([_vp, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _i64, _i32, _vp], _i32),
    "moe_fp8_blockscale_fused_workspace": ([_i32, _i32, _i32, _i32, _i32, _i32, _PSZ], _i32),
    "gemm_fp8_blockscale_tiled": ([_vp, _vp, _i64, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _i64, _i32, _i32, _i32, _i32,
                                   _vp, _sz, _vp], _i32),
    "gemm_fp8_blockscale_tiled_workspace": ([_i32, _i32, _i32, _i32, _PSZ], _i32),
    "gemm_fp8_blockscale_plan": ([_i32, _i32, _i32, _i32, ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int),
                                  ctypes.POINTER(ctypes.c_int)], _i32),
    "moe_fp8_blockscale_fused": ([_vp, _vp, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32,
                                  _i32, _i32, _i64, _vp, _vp, _i64, _vp, _sz, _vp], _i32),
    "fp4_quant_groups": ([_vp, _i32, _i64, _i64, _i32, _i32, _vp, _vp, _i32, _vp], _i32),
    "fp4_dequant_groups": ([_vp, _vp, _i32, _i64, _i32, _i32, _vp, _i32, _i64, _vp], _i32),
    "gemm_fp4_groupscale_workspace": ([_i32, _i32, _i32, _PSZ], _i32),
    "gemm_fp4_groupscale": ([_vp, _i32, _i64, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _sz, _vp], _i32),
    "grouped_gemm_fp4": ([_vp, _i32, _i64, _vp, _vp, _i32, _i32, _vp, _i32, _i32, _i32, _i32, _vp, _i64, _vp], _i32),
    "grouped_gemm": ([_vp, _i32, _i64, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i64, _vp], _i32),
    "grouped_gemm_dgrad": ([_vp, _i32, _i64, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i64, _vp], _i32),
    "grouped_gemm_wgrad": ([_vp, _i32, _i64, _vp, _i64, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _vp], _i32),
    "moe_group_workspace": ([_i32, _i32, _i32, _PSZ], _i32),
    "moe_group": ([_vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "moe_dispatch": ([_vp, _i32, _i64, _i32, _i32, _i32, _vp, _i32, _vp, _i64, _vp], _i32),
    "moe_combine": ([_vp, _i32, _i64, _i32, _i32, _i32, _vp, _i32, _vp, _i64, _vp, _i64, _vp], _i32),
    "moe_combine_grad": ([_vp, _i64, _vp, _i64, _i32, _i32, _i32, _i32, _vp, _i32, _vp, _i64, _vp, _i64, _vp, _vp], _i32),
    "fp8_ragged_blocks": ([_i32, _i32, _P64], _i32),
    "fp8_quant_ragged": ([_vp, _i32, _i64, _vp, _i32, _i32, _i32, _vp, _i64, _vp, _i64, _i64, _vp, _vp, _vp], _i32),
    "fp8_quant_128x128": ([_vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _i32, _vp], _i32),
    "grouped_gemm_fp8": ([_vp, _vp, _i64, _i64, _i64, _vp, _vp, _i32, _vp, _i32, _i32, _i32, _i32, _vp, _i64, _i32, _vp],
                         _i32),
    "grouped_gemm_fp8_wgrad": ([_vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _vp, _i32, _vp], _i32),
}
# the pre-shuffled-weight variants take the same arguments as their plain calls
for _name in ("gemm_fp8_blockscale", "moe_fp8_blockscale_g1u1", "moe_down_combine"):
    _SIGNATURES[_name + "_wpreshuffle"] = _SIGNATURES[_name]
EXPORTED = tuple(_SIGNATURES)


def lib():
    """Load libmoe355.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libmoe355.so not found at %s; build it with "
                               "`python -m fp8_block_scaled_grouped_amd.build`" % LIB_PATH)
        l = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in _SIGNATURES.items():
            fn = getattr(l, name)
            fn.argtypes = args
            fn.restype = res
        _lib = l
    return _lib


class Moe355Error(RuntimeError):
    def __init__(self, code):
        self.code = code
        super().__init__(lib().moe355_strerror(code).decode())


def _check(code):
    if code != 0:
        raise Moe355Error(code)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream():
    # the current stream's handle without a Stream object around it (2.7 us of a 12 us call)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _dev(t, dtype, name):
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    return t


def _need(t, shape, dtype, name):
    """A contiguous device tensor of exactly this shape and dtype (the kernels index it densely)."""
    _dev(t, dtype, name)
    if t.shape != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor of shape %s, got %s" % (name, dtype, tuple(shape),
                                                                                 tuple(t.shape)))
    return t


def _rows(t, name):
    """Row stride of a 2-D tensor whose rows are contiguous."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError("%s must be 2-D with contiguous rows" % name)
    return t.stride(0)


# ----------------------------------------------------------------- routing
def grouped_topk(logits, bias, n_group, topk_group, topk, renorm, routed_scaling_factor,
                 topk_weights=None, topk_ids=None):
    """Biased grouped top-k.  Returns (topk_weights fp32 [T, k], topk_ids int32 [T, k]).

    logits: fp32 or bf16 [T, E].  Outputs may be passed in as row-strided views (same
    row stride for both).
    """
    if logits.dtype != torch.bfloat16:
        _dev(logits, torch.float32, "logits")
    _dev(logits, logits.dtype, "logits")
    T, E = logits.shape
    _need(bias, (E,), torch.float32, "bias")
    if topk_weights is None:
        topk_weights = torch.empty((T, topk), dtype=torch.float32, device=logits.device)
    if topk_ids is None:
        topk_ids = torch.empty((T, topk), dtype=torch.int32, device=logits.device)
    _dev(topk_weights, torch.float32, "topk_weights")
    _dev(topk_ids, torch.int32, "topk_ids")
    if tuple(topk_weights.shape) != (T, topk) or tuple(topk_ids.shape) != (T, topk):
        raise ValueError("top-k outputs must be [T, topk] = %s" % ((T, topk),))
    ld = _rows(topk_weights, "topk_weights")
    if _rows(topk_ids, "topk_ids") != ld:
        raise ValueError("topk_weights and topk_ids must share a row stride")
    _check(lib().grouped_topk(_ptr(logits), int(logits.dtype == torch.bfloat16), _rows(logits, "logits"),
                              _ptr(bias), T, E, n_group,
                              topk_group, topk, int(bool(renorm)), float(routed_scaling_factor),
                              _ptr(topk_weights), _ptr(topk_ids), ld, _stream()))
    return topk_weights, topk_ids


# ----------------------------------------------------------------- sort
def moe_sort_sizes(T, topk, E, block_m):
    """(max_sorted, max_blocks, workspace_bytes) -- host-only."""
    ms, mb, ws = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_size_t()
    _check(lib().moe_sort_sizes(T, topk, E, block_m, ctypes.byref(ms), ctypes.byref(mb), ctypes.byref(ws)))
    return ms.value, mb.value, ws.value


def moe_block_m(T, topk, E):
    """Tuned M tile of the grouped GEMMs for this size (host-only)."""
    b = ctypes.c_int()
    _check(lib().moe_block_m(T, topk, E, ctypes.byref(b)))
    return b.value


def moe_sort(topk_ids, topk_weights, E, block_m, out=None, workspace=None):
    """Returns (sorted_ids, sorted_weights, sorted_expert_ids, num_valid) device tensors."""
    _dev(topk_ids, torch.int32, "topk_ids")
    _dev(topk_weights, torch.float32, "topk_weights")
    T, k = topk_ids.shape
    if tuple(topk_weights.shape) != (T, k):
        raise ValueError("topk_weights must have the shape of topk_ids")
    ms, mb, wsb = moe_sort_sizes(T, k, E, block_m)
    dev = topk_ids.device
    if out is None:
        out = (torch.empty(ms, dtype=torch.int32, device=dev), torch.empty(ms, dtype=torch.float32, device=dev),
               torch.empty(mb, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32, device=dev))
    if workspace is None:
        workspace = torch.empty(wsb, dtype=torch.uint8, device=dev)
    sid, sw, seid, nv = out
    for t, n, dt, name in ((sid, ms, torch.int32, "sorted_ids"), (sw, ms, torch.float32, "sorted_weights"),
                           (seid, mb, torch.int32, "sorted_expert_ids"), (nv, 1, torch.int32, "num_valid")):
        _dev(t, dt, name)
        if not t.is_contiguous() or t.numel() < n:
            raise ValueError("%s must be contiguous with at least %d entries" % (name, n))
    _dev(workspace, torch.uint8, "workspace")
    ld = _rows(topk_ids, "topk_ids")
    if _rows(topk_weights, "topk_weights") != ld:
        raise ValueError("topk_ids and topk_weights must share a row stride")
    _check(lib().moe_sort(_ptr(topk_ids), _ptr(topk_weights), ld, T, k, E, block_m, _ptr(sid), _ptr(sw), _ptr(seid),
                          _ptr(nv), _ptr(workspace), workspace.numel(), _stream()))
    return sid, sw, seid, nv


# ----------------------------------------------------------------- quant
def fp8_quant_1x128(x, q=None, scale=None, scale_layout="row"):
    """bf16 [M, K] -> (e4m3 uint8 [M, K], fp32 scales).

    scale_layout "row": scales [M, KB]; "kblock": scales [KB, M]; KB = ceil(K/128).
    """
    _dev(x, torch.bfloat16, "x")
    M, K = x.shape
    KB = _nblk(K)
    if q is None:
        q = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    shape = (M, KB) if scale_layout == "row" else (KB, M)
    if scale is None:
        scale = torch.empty(shape, dtype=torch.float32, device=x.device)
    _dev(q, torch.uint8, "q")
    if tuple(q.shape) != (M, K):
        raise ValueError("q must be [M, K] = %s, got %s" % ((M, K), tuple(q.shape)))
    _need(scale, shape, torch.float32, "scale")
    ssm, sskb = (KB, 1) if scale_layout == "row" else (1, M)
    _check(lib().fp8_quant_1x128(_ptr(x), _rows(x, "x"), M, K, _ptr(q), _rows(q, "q"), _ptr(scale), ssm, sskb,
                                 _stream()))
    return q, scale


def _nblk(n):
    """ceil(n / 128): scale entries along a dimension of n."""
    return -(-n // 128)


def _scale_strides(a_scale, T, H, scale_layout):
    """Element strides (per row, per K block) of 1x128 activation scales in either layout."""
    KB = _nblk(H)
    if scale_layout == "row":
        _need(a_scale, (T, KB), torch.float32, "a_scale")
        return KB, 1
    if scale_layout != "kblock":
        raise ValueError("scale_layout must be 'row' or 'kblock'")
    _need(a_scale, (KB, T), torch.float32, "a_scale")
    return 1, T


# ----------------------------------------------------------------- grouped GEMMs
def moe_fp8_blockscale_g1u1(a8, a_scale, w1, w1_scale, sorted_ids, sorted_expert_ids, num_valid, topk, block_m,
                            h8=None, h_scale=None, scale_layout="row", fc2_smooth_scale=None, preshuffled=False):
    """Gate/up grouped GEMM + SiLU*up (* fc2_smooth_scale [E, I] if given) + 1x128 requant.

    Returns (h8 [max_sorted, I], h_scale [max_sorted, I/128]).  preshuffled: w1 holds
    shuffle_weight_128x128 output (same shape).
    """
    T, H = a8.shape
    E, twoI, _ = w1.shape
    I = twoI // 2
    _need(a8, (T, H), torch.uint8, "a8")
    _need(w1, (E, 2 * I, H), torch.uint8, "w1")
    _need(w1_scale, (E, _nblk(2 * I), _nblk(H)), torch.float32, "w1_scale")
    ms = sorted_ids.numel()
    _need(sorted_ids, (ms,), torch.int32, "sorted_ids")
    _need(sorted_expert_ids, (sorted_expert_ids.numel(),), torch.int32, "sorted_expert_ids")
    if block_m <= 0 or sorted_expert_ids.numel() < ms // block_m:
        raise ValueError("sorted_expert_ids must hold max_sorted / block_m entries")
    _need(num_valid, (1,), torch.int32, "num_valid")
    if h8 is None:
        h8 = torch.empty((ms, I), dtype=torch.uint8, device=a8.device)
    if h_scale is None:
        h_scale = torch.empty((ms, I // 128), dtype=torch.float32, device=a8.device)
    _need(h8, (ms, I), torch.uint8, "h8")
    _need(h_scale, (ms, _nblk(I)), torch.float32, "h_scale")
    if fc2_smooth_scale is not None:
        _need(fc2_smooth_scale, (E, I), torch.float32, "fc2_smooth_scale")
    ssm, sskb = _scale_strides(a_scale, T, H, scale_layout)
    fn = lib().moe_fp8_blockscale_g1u1_wpreshuffle if preshuffled else lib().moe_fp8_blockscale_g1u1
    _check(fn(_ptr(a8), _ptr(a_scale), ssm, sskb, _ptr(w1), _ptr(w1_scale),
              _ptr(sorted_ids), _ptr(sorted_expert_ids), _ptr(num_valid), T, H, I, E,
              topk, block_m, ms, _ptr(h8), _ptr(h_scale),
              _ptr(fc2_smooth_scale), _stream()))
    return h8, h_scale


def moe_down_combine_workspace(T, H, topk):
    b = ctypes.c_size_t()
    _check(lib().moe_down_combine_workspace(T, H, topk, ctypes.byref(b)))
    return b.value


def moe_down_combine(h8, h_scale, w2, w2_scale, sorted_ids, sorted_weights, sorted_expert_ids, num_valid, T, topk,
                     block_m, out=None, workspace=None, preshuffled=False):
    """Down grouped GEMM + top-k weighted combine.  Returns bf16 [T, H].  preshuffled: w2 holds
    shuffle_weight_128x128 output (same shape)."""
    E, H, I = w2.shape
    _need(w2, (E, H, I), torch.uint8, "w2")
    _need(w2_scale, (E, _nblk(H), _nblk(I)), torch.float32, "w2_scale")
    ms = sorted_ids.numel()
    _need(sorted_ids, (ms,), torch.int32, "sorted_ids")
    _need(sorted_weights, (ms,), torch.float32, "sorted_weights")
    _need(sorted_expert_ids, (sorted_expert_ids.numel(),), torch.int32, "sorted_expert_ids")
    if block_m <= 0 or sorted_expert_ids.numel() < ms // block_m:
        raise ValueError("sorted_expert_ids must hold max_sorted / block_m entries")
    _need(num_valid, (1,), torch.int32, "num_valid")
    _need(h8, (ms, I), torch.uint8, "h8")
    _need(h_scale, (ms, _nblk(I)), torch.float32, "h_scale")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=h8.device)
    if workspace is None:
        workspace = torch.empty(moe_down_combine_workspace(T, H, topk), dtype=torch.uint8, device=h8.device)
    _dev(out, torch.bfloat16, "out")
    if tuple(out.shape) != (T, H):
        raise ValueError("out must be [T, H] = %s, got %s" % ((T, H), tuple(out.shape)))
    _dev(workspace, torch.uint8, "workspace")
    fn = lib().moe_down_combine_wpreshuffle if preshuffled else lib().moe_down_combine
    _check(fn(_ptr(h8), _ptr(h_scale), _ptr(w2), _ptr(w2_scale), _ptr(sorted_ids), _ptr(sorted_weights),
              _ptr(sorted_expert_ids), _ptr(num_valid), T, H, I, E, topk, block_m, ms, _ptr(out), _rows(out, "out"),
              _ptr(workspace), workspace.numel(), _stream()))
    return out


def gemm_fp8_blockscale_plan(M, N, K, measured=True):
    """(tile_m, tile_n, splits) gemm_fp8_blockscale runs for this shape (host-only);
    measured=False: the rule alone, without the table of measured plans."""
    tm, tn, sp = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(lib().gemm_fp8_blockscale_plan(M, N, K, int(bool(measured)), ctypes.byref(tm), ctypes.byref(tn),
                                          ctypes.byref(sp)))
    return tm.value, tn.value, sp.value


def gemm_fp8_blockscale_tiled_workspace(M, N, K, splits):
    b = ctypes.c_size_t()
    _check(lib().gemm_fp8_blockscale_tiled_workspace(M, N, K, splits, ctypes.byref(b)))
    return b.value


def gemm_fp8_blockscale_tiled(a8, a_scale, b8, b_scale, tile_m, tile_n, splits, c=None, workspace=None,
                              scale_layout="row", out_dtype=torch.bfloat16):
    """gemm_fp8_blockscale with a caller-chosen tiling (tile_m rows x tile_n columns, K in
    `splits` runs); workspace None allocates what the split needs."""
    M, K = a8.shape
    N = b8.shape[0]
    _need(a8, (M, K), torch.uint8, "a8")
    _need(b8, (N, K), torch.uint8, "b8")
    _need(b_scale, (_nblk(N), _nblk(K)), torch.float32, "b_scale")
    if c is None:
        c = torch.empty((M, N), dtype=out_dtype, device=a8.device)
    if c.dtype not in (torch.bfloat16, torch.float16) or tuple(c.shape) != (M, N):
        raise ValueError("c must be bf16 or fp16 [M, N]")
    _dev(c, c.dtype, "c")
    if workspace is None:
        n = gemm_fp8_blockscale_tiled_workspace(M, N, K, splits)
        workspace = torch.empty(max(n, 16), dtype=torch.uint8, device=a8.device)
    _dev(workspace, torch.uint8, "workspace")
    ssm, sskb = _scale_strides(a_scale, M, K, scale_layout)
    _check(lib().gemm_fp8_blockscale_tiled(_ptr(a8), _ptr(a_scale), ssm, sskb, _ptr(b8), _ptr(b_scale), M, N, K,
                                           _ptr(c), _rows(c, "c"), int(c.dtype == torch.float16), tile_m, tile_n,
                                           splits, _ptr(workspace), workspace.numel(), _stream()))
    return c


def moe_fp8_blockscale_fused_workspace(T, H, I, E, topk, block_m):
    b = ctypes.c_size_t()
    _check(lib().moe_fp8_blockscale_fused_workspace(T, H, I, E, topk, block_m, ctypes.byref(b)))
    return b.value


def moe_fp8_blockscale_fused(a8, a_scale, w1, w1_scale, w2, w2_scale, sorted_ids, sorted_weights, sorted_expert_ids,
                             num_valid, topk, block_m, out=None, workspace=None, scale_layout="row",
                             fc2_smooth_scale=None):
    """Gate/up + SiLU*up + requant, down projection and combine in one launch.  Returns bf16 [T, H]."""
    T, H = a8.shape
    E, twoI, _ = w1.shape
    I = twoI // 2
    _need(a8, (T, H), torch.uint8, "a8")
    _need(w1, (E, 2 * I, H), torch.uint8, "w1")
    _need(w1_scale, (E, _nblk(2 * I), _nblk(H)), torch.float32, "w1_scale")
    _need(w2, (E, H, I), torch.uint8, "w2")
    _need(w2_scale, (E, _nblk(H), _nblk(I)), torch.float32, "w2_scale")
    ms = sorted_ids.numel()
    _need(sorted_ids, (ms,), torch.int32, "sorted_ids")
    _need(sorted_weights, (ms,), torch.float32, "sorted_weights")
    _need(sorted_expert_ids, (sorted_expert_ids.numel(),), torch.int32, "sorted_expert_ids")
    if block_m <= 0 or sorted_expert_ids.numel() < ms // block_m:
        raise ValueError("sorted_expert_ids must hold max_sorted / block_m entries")
    _need(num_valid, (1,), torch.int32, "num_valid")
    if fc2_smooth_scale is not None:
        _need(fc2_smooth_scale, (E, I), torch.float32, "fc2_smooth_scale")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=a8.device)
    _dev(out, torch.bfloat16, "out")
    if tuple(out.shape) != (T, H):
        raise ValueError("out must be [T, H] = %s, got %s" % ((T, H), tuple(out.shape)))
    if workspace is None:
        workspace = torch.empty(moe_fp8_blockscale_fused_workspace(T, H, I, E, topk, block_m), dtype=torch.uint8,
                                device=a8.device)
    _dev(workspace, torch.uint8, "workspace")
    ssm, sskb = _scale_strides(a_scale, T, H, scale_layout)
    _check(lib().moe_fp8_blockscale_fused(_ptr(a8), _ptr(a_scale), ssm, sskb, _ptr(w1), _ptr(w1_scale), _ptr(w2),
                                          _ptr(w2_scale), _ptr(sorted_ids), _ptr(sorted_weights),
                                          _ptr(sorted_expert_ids), _ptr(num_valid), T, H, I, E, topk, block_m, ms,
                                          _ptr(fc2_smooth_scale), _ptr(out), _rows(out, "out"), _ptr(workspace),
                                          workspace.numel(), _stream()))
    return out


# ----------------------------------------------------------------- weight layout
def shuffle_weight_128x128(w, out=None):
    """e4m3 weights [..., R, K] (R, K multiples of 128) -> the same bytes in the
    pre-shuffled 128x128-tile layout the *_wpreshuffle calls read (new tensor, same shape)."""
    _dev(w, torch.uint8, "w")
    if not w.is_contiguous():
        raise ValueError("w must be contiguous")
    K = w.shape[-1]
    rows = w.numel() // K if K else 0
    if out is None:
        out = torch.empty_like(w)
    _check(lib().shuffle_weight_128x128(_ptr(w), rows, K, _ptr(out), _stream()))
    return out


# ----------------------------------------------------------------- dense
def gemm_fp8_blockscale_workspace(M, N, K):
    b = ctypes.c_size_t()
    _check(lib().gemm_fp8_blockscale_workspace(M, N, K, ctypes.byref(b)))
    return b.value


def gemm_fp8_blockscale(a8, a_scale, b8, b_scale, c=None, scale_layout="row", workspace=None,
                        out_dtype=torch.bfloat16, preshuffled=False):
    """a8 e4m3 [M, K] (1x128 scales), b8 e4m3 [N, K] (128x128 scales) -> [M, N] in out_dtype
    (bf16 or fp16; taken from c when c is given).  K and N need not be multiples of
    128: a_scale [M, ceil(K/128)], b_scale [ceil(N/128), ceil(K/128)].  preshuffled: b8 holds
    shuffle_weight_128x128 output (same shape; N, K multiples of 128).

    workspace: None allocates what gemm_fp8_blockscale_workspace asks for; False runs
    without workspace (no split-K); or a device uint8 tensor.
    """
    M, K = a8.shape
    N = b8.shape[0]
    _need(a8, (M, K), torch.uint8, "a8")
    _need(b8, (N, K), torch.uint8, "b8")
    _need(b_scale, (_nblk(N), _nblk(K)), torch.float32, "b_scale")
    if c is None:
        c = torch.empty((M, N), dtype=out_dtype, device=a8.device)
    if c.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("c must be bf16 or fp16, got %s" % c.dtype)
    _dev(c, c.dtype, "c")
    if tuple(c.shape) != (M, N):
        raise ValueError("c must be [M, N] = %s, got %s" % ((M, N), tuple(c.shape)))
    if workspace is None:
        n = gemm_fp8_blockscale_workspace(M, N, K)
        workspace = torch.empty(n, dtype=torch.uint8, device=a8.device) if n else False
    ws_ptr, ws_n = (None, 0) if workspace is False else (_ptr(workspace), workspace.numel())
    ssm, sskb = _scale_strides(a_scale, M, K, scale_layout)
    fn = lib().gemm_fp8_blockscale_wpreshuffle if preshuffled else lib().gemm_fp8_blockscale
    _check(fn(_ptr(a8), _ptr(a_scale), ssm, sskb, _ptr(b8), _ptr(b_scale), M, N, K, _ptr(c), _rows(c, "c"),
              int(c.dtype == torch.float16), ws_ptr, ws_n, _stream()))
    return c


# ----------------------------------------------------------------- 4-bit weights, ragged groups
_F16 = {torch.bfloat16: 0, torch.float16: 1}


def _half(t, name):
    """0 for a bf16 device tensor, 1 for an fp16 one."""
    f16 = _F16.get(t.dtype)
    if f16 is None or not t.is_cuda:
        raise ValueError("%s must be a bf16 or fp16 GPU tensor, got %s on %s" % (name, t.dtype, t.device))
    return f16


def _out(t, shape, dtype, like, name):
    """The output tensor: allocated when None, else checked (2-D outputs may have strided rows)."""
    if t is None:
        return like.new_empty(shape) if like.dtype == dtype else like.new_empty(shape, dtype=dtype)
    _dev(t, dtype, name)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return t


def _fp4_scale(scale, shape, name="scale"):
    """0 for fp32 scales, 1 for E8M0 bytes, of this shape."""
    e8m0 = int(scale.dtype == torch.uint8)
    _need(scale, shape, torch.uint8 if e8m0 else torch.float32, name)
    return e8m0


def _groups(K, group):
    if group not in (32, 64, 128):
        raise ValueError("group must be 32, 64 or 128, got %s" % (group,))
    return -(-K // group)


def fp4_quant_groups(w, group=128, scale_format="fp32", q=None, scale=None):
    """Pack bf16 or fp16 weights [..., K] to 4 bits: (codes uint8 [..., K/2], scales [..., ceil(K/group)]).

    scale_format "fp32": fp32 scales amax/6; "e8m0": uint8 power-of-two scales (OCP MX with group 32).
    K % 32 == 0; w contiguous, or 2-D with strided rows.
    """
    f16 = _half(w, "w")
    if scale_format not in ("fp32", "e8m0"):
        raise ValueError("scale_format must be 'fp32' or 'e8m0'")
    lead, K = w.shape[:-1], w.shape[-1]
    if w.dim() != 2 and not w.is_contiguous():
        raise ValueError("w must be contiguous, or 2-D with contiguous rows")
    ld = _rows(w, "w") if w.dim() == 2 else K
    rows = lead.numel()
    G, e8m0 = _groups(K, group), scale_format == "e8m0"
    q = _need(_out(q, (*lead, K // 2), torch.uint8, w, "q"), (*lead, K // 2), torch.uint8, "q")
    sdt = torch.uint8 if e8m0 else torch.float32
    scale = _need(_out(scale, (*lead, G), sdt, w, "scale"), (*lead, G), sdt, "scale")
    _check(lib().fp4_quant_groups(_ptr(w), f16, ld if rows > 1 else K, rows, K, group, _ptr(q), _ptr(scale), int(e8m0),
                                  _stream()))
    return q, scale


def fp4_dequant_groups(q, scale, group=128, dtype=torch.bfloat16, out=None):
    """Unpack fp4_quant_groups' output to bf16 or fp16 weights [..., K]."""
    _dev(q, torch.uint8, "q")
    lead, K = q.shape[:-1], 2 * q.shape[-1]
    _need(q, q.shape, torch.uint8, "q")
    e8m0 = _fp4_scale(scale, (*lead, _groups(K, group)))
    out = _out(out, (*lead, K), dtype, q, "out")
    f16 = _half(out, "out")
    if out.dim() != 2 and not out.is_contiguous():
        raise ValueError("out must be contiguous, or 2-D with contiguous rows")
    rows = lead.numel()
    ld = _rows(out, "out") if out.dim() == 2 and rows > 1 else K
    _check(lib().fp4_dequant_groups(_ptr(q), _ptr(scale), e8m0, rows, K, group, _ptr(out), f16, ld, _stream()))
    return out


def _ld(t, name):
    """Row stride of a 2-D tensor; of a single row (whose stride means nothing) its width."""
    if t.dim() == 2 and t.is_contiguous():
        return t.shape[1]
    ld = _rows(t, name)
    return ld if t.shape[0] > 1 else t.shape[1]


def gemm_fp4_groupscale_workspace(M, N, K):
    """Bytes of partial sums with which gemm_fp4_groupscale splits K (host-only)."""
    b = ctypes.c_size_t()
    _check(lib().gemm_fp4_groupscale_workspace(M, N, K, ctypes.byref(b)))
    return b.value


def gemm_fp4_groupscale(x, q, scale, group=128, c=None, workspace=None):
    """x bf16 or fp16 [M, K] times 4-bit weights q [N, K/2] with scales [N, ceil(K/group)] (fp32, or
    uint8 for E8M0), transposed: [M, N] in the type of x.  E8M0 rows of a multiple of 4 scales are fastest.

    workspace: None allocates what gemm_fp4_groupscale_workspace asks for (nothing up to 16
    rows); False runs without (K not split); or a device uint8 tensor.
    """
    f16 = _half(x, "x")
    M, K = x.shape
    N = q.shape[0]
    _need(q, (N, K // 2), torch.uint8, "q")
    e8m0 = _fp4_scale(scale, (N, _groups(K, group)))
    c = _out(c, (M, N), x.dtype, x, "c")
    if workspace is None and M > 16:
        workspace = x.new_empty(gemm_fp4_groupscale_workspace(M, N, K), dtype=torch.uint8)
    ws, wsn = (_ptr(_dev(workspace, torch.uint8, "workspace")), workspace.numel()) if workspace is not None and \
        workspace is not False and workspace.numel() else (None, 0)
    _check(lib().gemm_fp4_groupscale(_ptr(x), f16, _ld(x, "x"), _ptr(q), _ptr(scale), e8m0, group, M, N, K, _ptr(c),
                                     _ld(c, "c"), ws, wsn, _stream()))
    return c


def grouped_gemm_fp4(x, q, scale, offsets, group=128, c=None):
    """Rows of x [R, K] ordered by expert, expert e owning rows [offsets[e], offsets[e+1]) (int32 device
    tensor [E+1]), times its 4-bit weights q [E, N, K/2] with scales [E, N, ceil(K/group)]: [R, N]."""
    f16 = _half(x, "x")
    R, K = x.shape
    E, N, _ = q.shape
    _need(q, (E, N, K // 2), torch.uint8, "q")
    e8m0 = _fp4_scale(scale, (E, N, _groups(K, group)))
    _need(offsets, (E + 1,), torch.int32, "offsets")
    c = _out(c, (R, N), x.dtype, x, "c")
    _check(lib().grouped_gemm_fp4(_ptr(x), f16, _ld(x, "x"), _ptr(q), _ptr(scale), e8m0, group, _ptr(offsets), R, E, N,
                                  K, _ptr(c), _ld(c, "c"), _stream()))
    return c


def grouped_gemm(x, w, offsets, y=None):
    """Rows of x [R, K] ordered by expert (offsets int32 [E+1] on the device) times the experts'
    weights w [E, N, K], transposed: [R, N].  bf16 or fp16; not differentiable (grouped_linear is)."""
    f16 = _half(x, "x")
    R, K = x.shape
    E, N, _ = w.shape
    _need(w, (E, N, K), x.dtype, "w")
    _need(offsets, (E + 1,), torch.int32, "offsets")
    y = _out(y, (R, N), x.dtype, x, "y")
    _check(lib().grouped_gemm(_ptr(x), f16, _ld(x, "x"), _ptr(w), _ptr(offsets), R, E, N, K, _ptr(y), _ld(y, "y"),
                              _stream()))
    return y


def grouped_gemm_dgrad(dy, w, offsets, dx=None):
    """Gradient of grouped_gemm for x: dy [R, N], w [E, N, K] -> [R, K]."""
    f16 = _half(dy, "dy")
    R, N = dy.shape
    E, _, K = w.shape
    _need(w, (E, N, K), dy.dtype, "w")
    _need(offsets, (E + 1,), torch.int32, "offsets")
    dx = _out(dx, (R, K), dy.dtype, dy, "dx")
    _check(lib().grouped_gemm_dgrad(_ptr(dy), f16, _ld(dy, "dy"), _ptr(w), _ptr(offsets), R, E, N, K, _ptr(dx),
                                    _ld(dx, "dx"), _stream()))
    return dx


def grouped_gemm_wgrad(dy, x, offsets, dw=None, out_dtype=None):
    """Gradient of grouped_gemm for w: dy [R, N], x [R, K] -> [E, N, K] in the type of x, or fp32
    (out_dtype, or the type of dw when given).  Experts without rows get zeros."""
    f16 = _half(dy, "dy")
    R, N = dy.shape
    _dev(x, dy.dtype, "x")
    if x.dim() != 2 or x.shape[0] != R:
        raise ValueError("x must be [R, K] with the rows of dy")
    K, E = x.shape[1], offsets.shape[0] - 1
    _need(offsets, (E + 1,), torch.int32, "offsets")
    dt = dw.dtype if dw is not None else out_dtype if out_dtype is not None else x.dtype
    if dt not in (x.dtype, torch.float32):
        raise ValueError("dw must be %s or fp32, got %s" % (x.dtype, dt))
    dw = _need(_out(dw, (E, N, K), dt, x, "dw"), (E, N, K), dt, "dw")
    _check(lib().grouped_gemm_wgrad(_ptr(dy), f16, _ld(dy, "dy"), _ptr(x), _ld(x, "x"), _ptr(offsets), R, E, N, K,
                                    _ptr(dw), int(dt == torch.float32), _stream()))
    return dw


class _GroupedLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, offsets):
        ctx.save_for_backward(x, w, offsets)
        return grouped_gemm(x, w, offsets)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        x, w, offsets = ctx.saved_tensors
        dy = dy.contiguous()
        if dy.data_ptr() % 16:  # a view into a larger gradient may start anywhere
            dy = dy.clone()
        dx = grouped_gemm_dgrad(dy, w, offsets) if ctx.needs_input_grad[0] else None
        dw = grouped_gemm_wgrad(dy, x, offsets) if ctx.needs_input_grad[1] else None
        return dx, dw, None


def grouped_linear(x, w, offsets):
    """grouped_gemm with gradients for x and w, in their type (grouped_gemm_wgrad also gives fp32).  Every row of
    x must lie in a segment (offsets[0] == 0 and offsets[E] == R): rows in none have no defined output or gradient."""
    return _GroupedLinear.apply(x, w, offsets)


# ----------------------------------------------------------------- tokens to rows and back
_ELEM = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2, torch.uint8: 3}


def _elem(t, name, most=2):
    """The library's number of a tensor's element type, among the first `most + 1`."""
    n = _ELEM.get(t.dtype, 9)
    if n > most:
        raise ValueError("%s must be bf16, fp16 or fp32%s, got %s" % (name, " or uint8" if most == 3 else "", t.dtype))
    return n


_MOST = 2 ** 31 - 1


def _cut(*sizes):
    """Sizes that the library's 32-bit arguments would cut."""
    raise ValueError("sizes must be below 2^31, got %s" % (sizes,))


def _queue(*tensors):
    """The current GPU's stream, on which the kernels are queued: every tensor has to be on that GPU."""
    if not tensors[0].is_cuda:
        raise ValueError("tensors must be on a GPU, got one on %s" % tensors[0].device)
    dev = torch._C._cuda_getDevice()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("tensors must be on the current GPU (cuda:%d), got one on %s" % (dev, t.device))
    return torch._C._cuda_getCurrentRawStream(dev)


def _pairs(row_of_pair):
    shape = row_of_pair.shape
    if len(shape) != 2 or shape[1] < 1 or row_of_pair.dtype != torch.int32 or not row_of_pair.is_contiguous():
        raise ValueError("row_of_pair must be a contiguous int32 tensor [T, topk], got %s %s" % (row_of_pair.dtype, tuple(shape)))
    if shape[0] | shape[1] > _MOST:
        _cut(*shape)
    return shape


def _matrix(t, name):
    """(rows, columns, row stride) of a 2-D tensor with contiguous rows."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s must be 2-D, got %s" % (name, tuple(shape)))
    if shape[0] | shape[1] > _MOST:
        _cut(*shape)
    return shape[0], shape[1], shape[1] if t.is_contiguous() else _ld(t, name)


def _grad_wanted(*tensors):
    for t in tensors:
        if t is not None and t.requires_grad:
            return torch.is_grad_enabled()
    return False


@functools.lru_cache(maxsize=256)
def moe_group_workspace(T, topk, E):
    """Bytes of workspace that moe_group needs (host-only)."""
    if T | topk | E > _MOST:
        _cut(T, topk, E)
    b = ctypes.c_size_t()
    _check(lib().moe_group_workspace(T, topk, E, ctypes.byref(b)))
    return b.value


def moe_group(topk_ids, E, out=None, workspace=None):
    """Token-expert pairs in expert order: (offsets [E+1], row_of_pair [T, topk], pair_of_row [T*topk]), all int32.

    topk_ids int32 [T, topk] (rows may be strided).  The pairs of expert e get rows [offsets[e], offsets[e+1])
    in ascending order; pairs whose id is outside [0, E) get row -1, and rows at or past offsets[E] pair -1.
    """
    if topk_ids.dtype != torch.int32:
        raise ValueError("topk_ids must be int32, got %s" % topk_ids.dtype)
    T, k, ld = _matrix(topk_ids, "topk_ids")
    if E > _MOST:
        _cut(E)
    n = T * k
    stream = _queue(topk_ids, *out or (), workspace)
    if out is None:
        offsets, row_of_pair, pair_of_row = topk_ids.new_empty(E + 1), topk_ids.new_empty((T, k)), topk_ids.new_empty(n)
    else:
        offsets, row_of_pair, pair_of_row = out
        for t, shape, name in ((offsets, (E + 1,), "offsets"), (row_of_pair, (T, k), "row_of_pair"), (pair_of_row, (n,), "pair_of_row")):
            _need(t, shape, torch.int32, name)
    if workspace is None and n > 4096:
        workspace = topk_ids.new_empty(moe_group_workspace(T, k, E), dtype=torch.uint8)
    ws, wsn = (None, 0) if workspace is None else (_ptr(_dev(workspace, torch.uint8, "workspace")), workspace.numel())
    _check(lib().moe_group(topk_ids.data_ptr(), ld, T, k, E, offsets.data_ptr(), row_of_pair.data_ptr(), pair_of_row.data_ptr(), ws,
                           wsn, stream))
    return offsets, row_of_pair, pair_of_row


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, row_of_pair):
        ctx.save_for_backward(row_of_pair)
        return moe_dispatch(x, row_of_pair)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, drows):
        return moe_combine(drows.contiguous(), *ctx.saved_tensors), None


def moe_dispatch(x, row_of_pair, rows=None):
    """Tokens x [T, H] (bf16, fp16, fp32 or uint8) to the rows of their pairs: rows[row_of_pair[t, j]] = x[t].

    rows [T*topk, H], or any number of rows when given; rows that no pair has are left as they are.  Differentiable for x
    (moe_combine without weights) when rows is not given.
    """
    if rows is None and x.requires_grad and torch.is_grad_enabled():
        return _Dispatch.apply(x, row_of_pair)
    dt = _elem(x, "x", 3)
    T, k = _pairs(row_of_pair)
    n, H, ld = _matrix(x, "x")
    if n != T:
        raise ValueError("x must have the %d tokens of row_of_pair, got %d" % (T, n))
    if rows is None:
        if T * k > _MOST:
            _cut(T * k)
        stream = _queue(x, row_of_pair)
        R, ld_rows, rows = T * k, H, x.new_empty((T * k, H))
    else:
        R, w, ld_rows = _matrix(rows, "rows")
        stream = _queue(x, row_of_pair, rows)
        if w != H or rows.dtype != x.dtype:
            raise ValueError("rows must be [R, %d] in the type of x" % H)
    _check(lib().moe_dispatch(x.data_ptr(), dt, ld, T, H, k, row_of_pair.data_ptr(), R, rows.data_ptr(), ld_rows, stream))
    return rows


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, row_of_pair, weights):
        ctx.rows = rows.shape[0]
        # the rows themselves are only in the gradient of the weights
        ctx.save_for_backward(row_of_pair, weights, rows if ctx.needs_input_grad[2] else None)
        return moe_combine(rows, row_of_pair, weights)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout):
        row_of_pair, weights, rows = ctx.saved_tensors
        dout = dout.contiguous()
        # rows that no pair has get a gradient of zeros
        drows = dout.new_zeros((ctx.rows, dout.shape[1])) if ctx.needs_input_grad[0] else None
        if weights is None:
            return moe_dispatch(dout, row_of_pair, drows), None, None
        # (without a gradient of the weights the rows are not read)
        drows, dw = moe_combine_grad(dout, drows if rows is None else rows, row_of_pair, weights, drows, want=ctx.needs_input_grad[0::2])
        return drows, None, dw


def _routing_weights(weights, T, k):
    if weights.dtype != torch.float32 or weights.shape != (T, k):
        raise ValueError("weights must be fp32 %s, got %s %s" % ((T, k), weights.dtype, tuple(weights.shape)))
    if weights.is_contiguous():
        return k
    return _ld(weights, "weights")


def moe_combine(rows, row_of_pair, weights=None, out=None):
    """Rows [R, H] (bf16, fp16 or fp32) back to tokens: out[t] = sum over j of weights[t, j] * rows[row_of_pair[t, j]],
    [T, H] in the type of rows; fp32 sums over ascending j.  weights fp32 [T, topk], None for ones.

    Differentiable for rows and weights when out is not given; rows that no pair has get gradients of zeros.
    """
    if out is None and _grad_wanted(rows, weights):
        return _Combine.apply(rows, row_of_pair, weights)
    dt = _elem(rows, "rows")
    T, k = _pairs(row_of_pair)
    R, H, ld = _matrix(rows, "rows")
    w, ld_w = (None, 0) if weights is None else (weights.data_ptr(), _routing_weights(weights, T, k))
    stream = _queue(rows, row_of_pair, weights, out)
    if out is None:
        ld_out, out = H, rows.new_empty((T, H))
    else:
        ld_out = _ld(_out(out, (T, H), rows.dtype, rows, "out"), "out")
    _check(lib().moe_combine(rows.data_ptr(), dt, ld, T, H, k, row_of_pair.data_ptr(), R, w, ld_w, out.data_ptr(), ld_out, stream))
    return out


def moe_combine_grad(dout, rows, row_of_pair, weights, drows=None, dweights=None, want=(True, True)):
    """Gradients of moe_combine: dout [T, H] -> (drows [R, H] in the type of rows, dweights fp32 [T, topk]).

    Rows that no pair has are left as they are (of a new drows: undefined); a pair without a row has a dweights of 0.
    want: which of the two to compute (None for the other).
    """
    dt = _elem(rows, "rows")
    T, k = _pairs(row_of_pair)
    R, H, ld = _matrix(rows, "rows")
    if dout.shape != (T, H) or dout.dtype != rows.dtype:
        raise ValueError("dout must be %s %s, got %s %s" % (rows.dtype, (T, H), dout.dtype, tuple(dout.shape)))
    ld_w = _routing_weights(weights, T, k)
    stream = _queue(dout, rows, row_of_pair, weights, drows, dweights)
    drows = _out(drows, (R, H), rows.dtype, rows, "drows") if want[0] else None
    if not want[1]:
        dweights = None
    elif dweights is None:
        dweights = weights.new_empty((T, k))
    else:
        _need(dweights, (T, k), torch.float32, "dweights")
    _check(lib().moe_combine_grad(dout.data_ptr(), _ld(dout, "dout"), rows.data_ptr(), ld, dt, T, H, k, row_of_pair.data_ptr(), R,
                                  weights.data_ptr(), ld_w, _ptr(drows), 0 if drows is None else _ld(drows, "drows"),
                                  _ptr(dweights), stream))
    return drows, dweights


# ----------------------------------------------------------------- FP8 products over ragged groups
def fp8_ragged_blocks(R, E):
    """Number of 128-row blocks that fp8_quant_ragged's transposed output has room for (host-only)."""
    if R | E > _MOST:
        _cut(R, E)
    n = ctypes.c_int64()
    _check(lib().fp8_ragged_blocks(R, E, ctypes.byref(n)))
    return n.value


def fp8_quant_ragged(x, offsets=None, rows=True, columns=True):
    """Quantise rows x [R, K] (bf16 or fp16) ordered by expert to e4m3 with power-of-two scales (E8M0, uint8).

    rows: (q uint8 [R, K], scale uint8 [R, ceil(K/128)]), one scale for each 1 x 128.  columns (needs offsets): (qt uint8
    [blocks, K, 128], tscale uint8 [blocks, K]), one scale for each 128 rows of an expert x 1 column, as
    grouped_gemm_fp8_wgrad takes them.  Returns (q, scale, qt, tscale) with None for what is not asked for.  Rows in no
    segment are neither read nor written.  scale is stored by K blocks (its transpose is contiguous).
    """
    f16 = _half(x, "x")
    ld = _ld(x, "x")
    R, K = x.shape
    if R | K > _MOST:
        _cut(R, K)
    columns = columns and offsets is not None
    E = 0
    if offsets is not None:
        E = offsets.shape[0] - 1
        _need(offsets, (E + 1,), torch.int32, "offsets")
    q = scale = qt = tscale = None
    if rows:
        q = x.new_empty((R, K), dtype=torch.uint8)
        scale = x.new_empty((_nblk(K), R), dtype=torch.uint8).t()
    if columns:
        blocks = fp8_ragged_blocks(R, E)
        qt, tscale = x.new_empty((blocks, K, 128), dtype=torch.uint8), x.new_empty((blocks, K), dtype=torch.uint8)
    if q is None and qt is None:
        raise ValueError("neither rows nor columns asked for (columns need offsets)")
    stream = _queue(x, offsets)
    _check(lib().fp8_quant_ragged(_ptr(x), f16, ld, _ptr(offsets), R, E, K, _ptr(q), K, _ptr(scale), 1, R, _ptr(qt), _ptr(tscale),
                                  stream))
    return q, scale, qt, tscale


def fp8_quant_128x128(w, scale_format="e8m0", transposed=False):
    """Quantise weights w [E, N, K] (bf16 or fp16) to e4m3 with one scale for each 128 x 128: (q, scale), and with
    transposed=True also (qt [E, K, N], tscale) of the same values.

    scale_format "e8m0": uint8 power-of-two scales; "fp32": fp32 scales amax/448.
    """
    f16 = _half(w, "w")
    if scale_format not in ("fp32", "e8m0"):
        raise ValueError("scale_format must be 'fp32' or 'e8m0'")
    if w.dim() != 3 or not w.is_contiguous():
        raise ValueError("w must be a contiguous [E, N, K] tensor")
    E, N, K = w.shape
    if E | N | K > _MOST:
        _cut(E, N, K)
    sdt = torch.uint8 if scale_format == "e8m0" else torch.float32
    q, scale = w.new_empty((E, N, K), dtype=torch.uint8), w.new_empty((E, _nblk(N), _nblk(K)), dtype=sdt)
    qt = tscale = None
    if transposed:
        qt, tscale = w.new_empty((E, K, N), dtype=torch.uint8), w.new_empty((E, _nblk(K), _nblk(N)), dtype=sdt)
    stream = _queue(w)
    _check(lib().fp8_quant_128x128(_ptr(w), f16, E, N, K, _ptr(q), _ptr(scale), _ptr(qt), _ptr(tscale), int(scale_format == "e8m0"),
                                   stream))
    return (q, scale, qt, tscale) if transposed else (q, scale)


def grouped_gemm_fp8(x8, x_scale, w8, w_scale, offsets, y=None, out_dtype=torch.bfloat16, scale_layout="row"):
    """Rows x8 [R, K] (e4m3 codes, uint8) ordered by expert (offsets int32 [E+1] on the device) times the experts' weights
    w8 [E, N, K], transposed: [R, N] in bf16 or fp16 (out_dtype, or the type of y when given).

    Scales: x_scale [R, ceil(K/128)] of any strides ([ceil(K/128), R] with scale_layout "kblock") and w_scale [E, ceil(N/128),
    ceil(K/128)], both fp32 (fp8_quant_1x128, checkpoints) or both uint8 for E8M0 (fp8_quant_ragged, fp8_quant_128x128).
    Not differentiable (grouped_linear_fp8 is).
    """
    if x8.dtype != torch.uint8 or w8.dtype != torch.uint8:
        raise ValueError("x8 and w8 must be uint8, got %s and %s" % (x8.dtype, w8.dtype))
    ld = _ld(x8, "x8")
    R, K = x8.shape
    E, N, wK = w8.shape
    if R | E | N | K > _MOST:
        _cut(R, E, N, K)
    NB, KB = _nblk(N), _nblk(K)
    if wK != K or not w8.is_contiguous():
        raise ValueError("w8 must be a contiguous [E, N, %d], got %s" % (K, tuple(w8.shape)))
    e8m0 = int(w_scale.dtype == torch.uint8)
    if w_scale.dtype not in (torch.uint8, torch.float32) or w_scale.shape != (E, NB, KB) or not w_scale.is_contiguous():
        raise ValueError("w_scale must be a contiguous fp32 or uint8 %s, got %s %s" % ((E, NB, KB), w_scale.dtype, tuple(w_scale.shape)))
    if scale_layout == "kblock":
        x_scale = x_scale.t()
    elif scale_layout != "row":
        raise ValueError("scale_layout must be 'row' or 'kblock'")
    if x_scale.shape != (R, KB) or x_scale.dtype != w_scale.dtype:
        raise ValueError("x_scale must be %s %s, got %s %s" % (w_scale.dtype, (R, KB), x_scale.dtype, tuple(x_scale.shape)))
    if offsets.dtype != torch.int32 or offsets.shape != (E + 1,) or not offsets.is_contiguous():
        raise ValueError("offsets must be a contiguous int32 tensor of %d, got %s %s" % (E + 1, offsets.dtype, tuple(offsets.shape)))
    y = _out(y, (R, N), out_dtype if y is None else y.dtype, x8, "y")
    stream = _queue(x8, x_scale, w8, w_scale, offsets, y)
    _check(lib().grouped_gemm_fp8(_ptr(x8), _ptr(x_scale), ld, x_scale.stride(0), x_scale.stride(1), _ptr(w8), _ptr(w_scale), e8m0,
                                  _ptr(offsets), R, E, N, K, _ptr(y), _ld(y, "y"), _half(y, "y"), stream))
    return y


def grouped_gemm_fp8_wgrad(dyt, dyt_scale, xt, xt_scale, offsets, R, dw=None, out_dtype=torch.float32):
    """Gradient of grouped_gemm_fp8 for w from the transposed codes of dy and x (fp8_quant_ragged's qt and tscale of R
    rows): [E, N, K] in fp32, bf16 or fp16 (out_dtype, or the type of dw when given).  Experts without rows get zeros."""
    E = offsets.shape[0] - 1
    _need(offsets, (E + 1,), torch.int32, "offsets")
    blocks, N, K = fp8_ragged_blocks(R, E), dyt.shape[1], xt.shape[1]
    if E | N | K > _MOST:
        _cut(E, N, K)
    for t, shape, name in ((dyt, (blocks, N, 128), "dyt"), (dyt_scale, (blocks, N), "dyt_scale"), (xt, (blocks, K, 128), "xt"),
                           (xt_scale, (blocks, K), "xt_scale")):
        _need(t, shape, torch.uint8, name)
    dt = out_dtype if dw is None else dw.dtype
    dw = _need(_out(dw, (E, N, K), dt, dyt, "dw"), (E, N, K), dt, "dw")
    stream = _queue(dyt, dyt_scale, xt, xt_scale, offsets, dw)
    _check(lib().grouped_gemm_fp8_wgrad(_ptr(dyt), _ptr(dyt_scale), _ptr(xt), _ptr(xt_scale), _ptr(offsets), R, E, N, K, _ptr(dw),
                                        _elem(dw, "dw"), stream))
    return dw


def _addresses(buf, sizes):
    """Addresses of places of these bytes, one after the other on 256 bytes, None for a size of None."""
    at, out = buf.data_ptr(), []
    for n in sizes:
        out.append(None if n is None else at)
        at += -(-(n or 0) // 256) * 256
    return out


def _places(like, sizes):
    """A new buffer on `like`'s device for operands of these bytes (each allocation costs the host 1.5 us), and their addresses."""
    buf = like.new_empty(sum(-(-(n or 0) // 256) * 256 for n in sizes), dtype=torch.uint8)
    return buf, _addresses(buf, sizes)


class _GroupedLinearFp8(torch.autograd.Function):
    """fp8_quant_ragged, fp8_quant_128x128, grouped_gemm_fp8 and grouped_gemm_fp8_wgrad on the parts of few buffers."""

    @staticmethod
    def forward(ctx, x, w, offsets, grad):
        need_x, need_w = (grad and n for n in ctx.needs_input_grad[:2])
        f16 = _half(x, "x")
        R, K, ld = _matrix(x, "x")
        if w.dim() != 3 or w.shape[2] != K or not w.is_contiguous():
            raise ValueError("w must be a contiguous [E, N, %d] tensor, got %s" % (K, tuple(w.shape)))
        E, N, _ = w.shape
        if E | N > _MOST:
            _cut(E, N)
        if offsets.dtype != torch.int32 or offsets.shape != (E + 1,) or not offsets.is_contiguous():
            raise ValueError("offsets must be a contiguous int32 tensor of %d, got %s %s" % (E + 1, offsets.dtype, tuple(offsets.shape)))
        stream, off, call = _queue(x, w, offsets), offsets.data_ptr(), lib()
        blocks, NB, KB = R // 128 + E, _nblk(N), _nblk(K)
        # x and w transposed, for the gradients of w and x
        ctx.kept = (blocks * K * 128, blocks * K) if need_w else (None, None)
        ctx.kept += (E * K * N, E * KB * NB) if need_x else (None, None)
        kept, (qt, ts, wt, wts) = _places(x, ctx.kept)
        rest, (q, s, wq, ws) = _places(x, (R * K, KB * R, E * N * K, E * NB * KB))
        y = x.new_empty((R, N))
        _check(call.fp8_quant_ragged(x.data_ptr(), f16, ld, off, R, E, K, q, K, s, 1, R, qt, ts, stream))
        _check(call.fp8_quant_128x128(w.data_ptr(), f16, E, N, K, wq, ws, wt, wts, 1, stream))
        _check(call.grouped_gemm_fp8(q, s, K, 1, R, wq, ws, 1, off, R, E, N, K, y.data_ptr(), N, f16, stream))
        ctx.save_for_backward(offsets, kept)
        ctx.sizes = R, E, N, K
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        offsets, kept = ctx.saved_tensors
        qt, ts, wt, wts = _addresses(kept, ctx.kept)
        R, E, N, K = ctx.sizes
        dy = dy.contiguous()
        if dy.data_ptr() % 16:  # a view into a larger gradient may start anywhere
            dy = dy.clone()
        f16, stream, off, call = _half(dy, "dy"), _queue(dy, kept), offsets.data_ptr(), lib()
        blocks, dx, dw = R // 128 + E, None, None
        rest, (q, s, dyt, dys) = _places(dy, ((None, None) if wt is None else (R * N, _nblk(N) * R)) +
                                         ((None, None) if qt is None else (blocks * N * 128, blocks * N)))
        _check(call.fp8_quant_ragged(dy.data_ptr(), f16, N, off, R, E, N, q, N, s, 1, R, dyt, dys, stream))
        if wt is not None:
            dx = dy.new_empty((R, K))
            _check(call.grouped_gemm_fp8(q, s, N, 1, R, wt, wts, 1, off, R, E, K, N, dx.data_ptr(), K, f16, stream))
        if qt is not None:
            dw = dy.new_empty((E, N, K))
            _check(call.grouped_gemm_fp8_wgrad(dyt, dys, qt, ts, off, R, E, N, K, dw.data_ptr(), f16, stream))
        return dx, dw, None, None


def grouped_linear_fp8(x, w, offsets):
    """grouped_linear in FP8: x [R, K] and w [E, N, K] (bf16 or fp16, the same type) are quantised to e4m3 with a power-of-two
    scale for each block (x 1 x 128, w 128 x 128) and multiplied, and so are the gradients: dx from dy in 1 x 128 and
    the same w, dw from dy and x in blocks of 128 rows x 1.  What the backward pass keeps is x and w in 8 bits.

    N and K multiples of 16.  Rows of x in no segment have no defined output or gradient (moe_combine and the gradient of
    moe_dispatch do not read such rows).
    """
    if x.dtype != w.dtype:
        raise ValueError("x and w must have the same type, got %s and %s" % (x.dtype, w.dtype))
    return _GroupedLinearFp8.apply(x, w, offsets, torch.is_grad_enabled())


# ----------------------------------------------------------------- the layer
class MoELayer:
    """The five calls of one MoE layer on preallocated buffers (no allocation per call).

    forward(hidden bf16 [T, H], logits fp32 [T, E]) -> bf16 [T, H], running
    grouped_topk -> moe_sort -> fp8_quant_1x128 -> moe_fp8_blockscale_g1u1 ->
    moe_down_combine on the current stream.  With overlap_quant the quantisation, which
    does not depend on the routing, runs on a second stream (default priority) beside
    grouped_topk and moe_sort: it starts after everything already queued on the current
    stream (so also after the previous forward's GEMMs, which read a8) and the GEMMs wait
    for it.  Off by default: it measured within noise on the prefill layer (5.10 against
    5.11 ms of serial calls) and 14 us slower on the 64-token decode layer, where the
    cross-stream join costs more than the 6 us quantisation.
    """

    def __init__(self, cfg, bias, w1, w1_scale, w2, w2_scale, T=None, block_m=None, scale_layout="row",
                 fc2_smooth_scale=None, preshuffle=False, fused=False, overlap_quant=False):
        self.cfg = cfg
        self.T = cfg.T if T is None else T
        if block_m is None:
            block_m = cfg.block_m if cfg.block_m else moe_block_m(self.T, cfg.topk, cfg.E)
        self.block_m = block_m
        # preshuffle: the weights are permuted once, here, into the 128x128-tile layout
        self.preshuffle = preshuffle
        if preshuffle:
            w1, w2 = shuffle_weight_128x128(w1), shuffle_weight_128x128(w2)
        self.bias, self.w1, self.w1_scale, self.w2, self.w2_scale = bias, w1, w1_scale, w2, w2_scale
        self.scale_layout = scale_layout
        self.fc2_smooth_scale = fc2_smooth_scale
        dev = w1.device
        T, H, I, E, k = self.T, cfg.H, cfg.I, cfg.E, cfg.topk
        ms, mb, wsb = moe_sort_sizes(T, k, E, self.block_m)
        self.max_sorted = ms
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.sort_out = (torch.empty(ms, dtype=torch.int32, device=dev), torch.empty(ms, dtype=torch.float32,
                                                                                      device=dev),
                         torch.empty(mb, dtype=torch.int32, device=dev), torch.zeros(1, dtype=torch.int32,
                                                                                      device=dev))
        self.sort_ws = torch.empty(max(wsb, 1), dtype=torch.uint8, device=dev)
        self.a8 = torch.empty((T, H), dtype=torch.uint8, device=dev)
        self.a_scale = torch.empty((T, H // 128) if scale_layout == "row" else (H // 128, T), dtype=torch.float32,
                                   device=dev)
        self.out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.side = torch.cuda.Stream(device=dev) if overlap_quant else None
        # fused: the expert computation as one launch (moe_fp8_blockscale_fused), its
        # intermediates in one workspace; else the two calls on h8 / h_scale / down_ws
        self.fused = fused
        if fused:
            if preshuffle:
                raise ValueError("the fused call takes weights as loaded (no pre-shuffled variant)")
            self.fused_ws = torch.empty(moe_fp8_blockscale_fused_workspace(T, H, I, E, k, self.block_m),
                                        dtype=torch.uint8, device=dev)
        else:
            self.h8 = torch.empty((ms, I), dtype=torch.uint8, device=dev)
            self.h_scale = torch.empty((ms, I // 128), dtype=torch.float32, device=dev)
            self.down_ws = torch.empty(moe_down_combine_workspace(T, H, k), dtype=torch.uint8, device=dev)

    def route_and_quantise(self, hidden, logits):
        """grouped_topk, moe_sort and fp8_quant_1x128 (on the side stream with overlap_quant);
        returns the sort outputs.  On return the current stream is ordered after all three."""
        c = self.cfg
        main = torch.cuda.current_stream()
        if self.side is not None:
            self.side.wait_stream(main)
            with torch.cuda.stream(self.side):
                fp8_quant_1x128(hidden, self.a8, self.a_scale, self.scale_layout)
        grouped_topk(logits, self.bias, c.n_group, c.topk_group, c.topk, c.renorm, c.routed_scaling_factor,
                     self.topk_w, self.topk_ids)
        srt = moe_sort(self.topk_ids, self.topk_w, c.E, self.block_m, self.sort_out, self.sort_ws)
        if self.side is not None:
            main.wait_stream(self.side)
        else:
            fp8_quant_1x128(hidden, self.a8, self.a_scale, self.scale_layout)
        return srt

    def forward(self, hidden, logits):
        c = self.cfg
        sid, sw, seid, nv = self.route_and_quantise(hidden, logits)
        if self.fused:
            return moe_fp8_blockscale_fused(self.a8, self.a_scale, self.w1, self.w1_scale, self.w2, self.w2_scale, sid,
                                            sw, seid, nv, c.topk, self.block_m, self.out, self.fused_ws,
                                            self.scale_layout, self.fc2_smooth_scale)
        moe_fp8_blockscale_g1u1(self.a8, self.a_scale, self.w1, self.w1_scale, sid, seid, nv, c.topk, self.block_m,
                                self.h8, self.h_scale, self.scale_layout, self.fc2_smooth_scale, self.preshuffle)
        moe_down_combine(self.h8, self.h_scale, self.w2, self.w2_scale, sid, sw, seid, nv, self.T, c.topk,
                         self.block_m, self.out, self.down_ws, self.preshuffle)
        return self.out
