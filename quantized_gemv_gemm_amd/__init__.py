"""Python binding of libtl, the ternary linear-layer library for MI355X (gfx950).

The functions mirror the C ABI in include/tl.h one to one.  They only check
tensor dtypes/devices/contiguity, allocate outputs with torch when none are
given, and pass raw pointers and the current HIP stream; every step of the
computation runs in the library's HIP kernels.  There is no fallback: if
libtl.so is missing or a call fails, a RuntimeError is raised.

Method: qiita.com/nakanokensetsu/items/ecc183fae033565af7cb ("前提",
"1. TP=2 への移植", "4. 効いた高速化").
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtl.so")

TL_BF16, TL_F32, TL_E4M3 = 0, 1, 2
GROUP, HBLOCK = 128, 1024

_lib = None

_c_i64 = ctypes.c_int64
_c_p = ctypes.c_void_p
_c_sz = ctypes.c_size_t

# name -> (restype, argtypes); mirrors include/tl.h
_SIGS = {
    "tl_abi_version": (ctypes.c_int, []),
    "tl_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "tl_last_kernel_name": (ctypes.c_char_p, []),
    "tl_last_error_detail": (ctypes.c_char_p, []),
    "tl_packed_bytes": (_c_sz, [_c_i64, _c_i64]),
    "tl_pack_weights": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "tl_hadamard_blk": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p]),
    "tl_hadamard_half": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p]),
    "tl_hadamard_join": (ctypes.c_int, [_c_p, _c_p, _c_i64, ctypes.c_int, _c_p, _c_i64, _c_p]),
    "tl_gemv_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "tl_gemv_ternary": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, ctypes.c_int,
                                       _c_p, _c_sz, _c_p]),
    "tl_gemv_prepare": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_sz, _c_p]),
    "tl_gemv_prepared": (ctypes.c_int, [_c_p, _c_sz, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, ctypes.c_int,
                                        _c_p]),
    "tl_gemv_ternary_q8": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, ctypes.c_int,
                                          _c_p]),
    "tl_quant_act_int8": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p]),
    "tl_gemv_prepare_x": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_sz, _c_p]),
    "tl_gemv_ternary_x": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, ctypes.c_int,
                                         _c_p, _c_sz, _c_p]),
    "tl_quant_act_int8_x": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p]),
    "tl_gemm_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "tl_gemm_int8_rescale": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p,
                                            ctypes.c_int, _c_p, _c_p, _c_sz, _c_p]),
    "tl_linear_path": (ctypes.c_int, [_c_i64, _c_i64, _c_i64]),
    "tl_linear_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64]),
    "tl_linear_apply": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p,
                                       ctypes.c_int, _c_p, _c_sz, _c_p]),
    "tl_noalloc_scratch_bytes": (_c_sz, []),
    "tl_read_probe": (ctypes.c_int, [_c_p, _c_sz, _c_p, _c_p]),
    "tl_mfma_probe": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, _c_p, _c_p]),
    "tl_kv_offset": (_c_i64, [ctypes.c_int, ctypes.c_int] + [_c_i64] * 7),
    "tl_step_plan": (ctypes.c_int, [_c_p, _c_p, _c_p, _c_i64, _c_p, _c_i64, _c_i64, _c_p, _c_i64, _c_p, _c_p, _c_i64,
                                    _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p]),
    "tl_kv_write": (ctypes.c_int, [_c_p, _c_i64, _c_p, _c_i64, _c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_i64, _c_i64,
                                   _c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p, ctypes.c_int, _c_i64,
                                   _c_i64, _c_p]),
    "tl_tree_attention_workspace_size": (_c_sz, [_c_i64, _c_i64, _c_i64, ctypes.c_int]),
    "tl_tree_attention": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p,
                                         ctypes.c_int, _c_i64, _c_i64, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p,
                                         ctypes.c_float, _c_i64, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "tl_tree_verify_workspace_size": (_c_sz, [_c_i64, _c_i64]),
    "tl_tree_verify": (ctypes.c_int, [_c_p, ctypes.c_int, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_p, _c_p,
                                      _c_i64, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "tl_kv_commit": (ctypes.c_int, [_c_p, _c_p, _c_i64, _c_p, _c_p, _c_p, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p,
                                    ctypes.c_int, _c_i64, _c_i64, _c_i64, _c_i64, _c_i64, _c_p, _c_p]),
    "tl_linear_apply_noalloc": (ctypes.c_int, [_c_p, _c_i64, _c_i64, _c_i64, _c_p, _c_p, _c_p, _c_p, _c_p,
                                               _c_p, ctypes.c_int, _c_p]),
}

PATH_GEMV, PATH_INT8 = 0, 1


def lib():
    """The loaded libtl.so (ctypes), with argument types declared."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build()")
        # One HIP runtime per process: torch ships its own libamdhip64 (needed as
        # "libamdhip64.so"), libtl needs "libamdhip64.so.7".  Loading torch first makes
        # the dynamic linker resolve libtl's dependency to torch's copy (same SONAME),
        # so device memory, streams and kernels all live in one runtime.
        import torch  # noqa: F401
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in _SIGS.items():
            fn = getattr(L, name)
            fn.restype, fn.argtypes = res, args
        _lib = L
    return _lib


def status_string(s: int) -> str:
    return lib().tl_status_string(s).decode()


def last_kernel_name() -> str:
    return lib().tl_last_kernel_name().decode()


def abi_version() -> int:
    return lib().tl_abi_version()


def _check(name: str, status: int):
    if status != 0:
        detail = lib().tl_last_error_detail().decode() if status == 5 else ""
        raise RuntimeError(f"{name} failed: {status_string(status)} (status {status}) {detail}".rstrip())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(device=None):
    import torch
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtype, ndim=None):
    import torch
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")


def _out_code(dtype):
    import torch
    if dtype == torch.bfloat16:
        return TL_BF16
    if dtype == torch.float32:
        return TL_F32
    raise TypeError("output dtype must be torch.bfloat16 or torch.float32")


# ---------------------------------------------------------------------------
# the five calls
# ---------------------------------------------------------------------------
def packed_words(N: int, K: int) -> int:
    """Number of uint32 words of the packed (tiled) weights of an [N, K] layer."""
    return int(lib().tl_packed_bytes(N, K)) // 4


def _check_packed(packed, N, K):
    import torch
    _need(packed, "packed", torch.int32, 1)
    if packed.numel() != packed_words(N, K):
        raise ValueError(f"packed must hold {packed_words(N, K)} words for N={N}, K={K}")


def pack_weights(codes, scales, packed=None, q=None, row_scale=None, invalid_count=None):
    """codes int8 [N,K], scales fp16 [N,K/128] -> (packed int32 [packed_words(N,K)] (the uint32
    tile words of the layout in include/tl.h), q int8 [N,K/128], row_scale f32 [N])."""
    import torch
    _need(codes, "codes", torch.int8, 2)
    _need(scales, "scales", torch.float16, 2)
    N, K = codes.shape
    dev = codes.device
    packed = torch.empty((packed_words(N, K),), dtype=torch.int32, device=dev) if packed is None else packed
    q = torch.empty((N, K // GROUP), dtype=torch.int8, device=dev) if q is None else q
    row_scale = torch.empty((N,), dtype=torch.float32, device=dev) if row_scale is None else row_scale
    _check_packed(packed, N, K)
    _need(q, "q", torch.int8, 2)
    _need(row_scale, "row_scale", torch.float32, 1)
    if invalid_count is not None:
        _need(invalid_count, "invalid_count", torch.int32, 1)
    if scales.shape != (N, K // GROUP) or q.shape != (N, K // GROUP) or row_scale.shape != (N,):
        raise ValueError("shape mismatch in pack_weights")
    _check("tl_pack_weights", lib().tl_pack_weights(
        _ptr(codes), _ptr(scales), N, K, _ptr(packed), _ptr(q), _ptr(row_scale), _ptr(invalid_count),
        _stream(dev)))
    return packed, q, row_scale


def hadamard_blk(x, signs=None, out=None):
    """x bf16 [T,K] -> xr f32 [T,K]: exact block rotation (1/32) H1024 (d * x), rounded once."""
    import torch
    _need(x, "x", torch.bfloat16, 2)
    T, K = x.shape
    if signs is not None:
        _need(signs, "signs", torch.int8, 1)
        if signs.shape != (K,):
            raise ValueError("signs must be [K]")
    out = torch.empty((T, K), dtype=torch.float32, device=x.device) if out is None else out
    _need(out, "out", torch.float32, 2)
    if out.shape != (T, K):
        raise ValueError("out must be [T, K]")
    _check("tl_hadamard_blk", lib().tl_hadamard_blk(_ptr(x), T, K, _ptr(signs), _ptr(out), _stream(x.device)))
    return out


def _check_x(x, signs):
    import torch
    _need(x, "x", torch.bfloat16, 2)
    if signs is not None:
        _need(signs, "signs", torch.int8, 1)
        if signs.shape != (x.shape[1],):
            raise ValueError("signs must be [K]")


def gemv_prepare_x(x, workspace, signs=None):
    """Fused rotation + GEMV prep: limbs of the rotated x bf16 [b,K] into ``workspace``
    (bit-identical to gemv_prepare(hadamard_blk(x, signs)))."""
    import torch
    _check_x(x, signs)
    _need(workspace, "workspace", torch.uint8, 1)
    b, K = x.shape
    _check("tl_gemv_prepare_x", lib().tl_gemv_prepare_x(_ptr(x), b, K, _ptr(signs), _ptr(workspace),
                                                        workspace.numel(), _stream(x.device)))
    return workspace


def gemv_ternary_x(x, packed, scales, signs=None, out_dtype=None, out=None, workspace=None):
    """Decode layer from the raw input: x bf16 [b,K] -> y [b,N] (rotation fused into the prep)."""
    import torch
    _check_x(x, signs)
    _need(scales, "scales", torch.float16, 2)
    b, K = x.shape
    N = scales.shape[0]
    _check_packed(packed, N, K)
    if scales.shape != (N, K // GROUP):
        raise ValueError("shape mismatch in gemv_ternary_x")
    if out is None:
        out = torch.empty((b, N), dtype=out_dtype or torch.bfloat16, device=x.device)
    code = _out_code(out.dtype)
    _need(out, "out", out.dtype, 2)
    if out.shape != (b, N):
        raise ValueError("out must be [b, N]")
    need = gemv_workspace_size(b, K, N)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=x.device)
    _need(workspace, "workspace", torch.uint8, 1)
    _check("tl_gemv_ternary_x", lib().tl_gemv_ternary_x(
        _ptr(x), b, K, N, _ptr(signs), _ptr(packed), _ptr(scales), _ptr(out), code, _ptr(workspace),
        workspace.numel(), _stream(x.device)))
    return out


def quant_act_int8_x(x, signs=None, xq=None, tok_scale=None):
    """Fused rotation + per-token int8: x bf16 [T,K] -> (xq int8 [T,K], tok_scale f32 [T])
    (bit-identical to quant_act_int8(hadamard_blk(x, signs)))."""
    import torch
    _check_x(x, signs)
    T, K = x.shape
    xq = torch.empty((T, K), dtype=torch.int8, device=x.device) if xq is None else xq
    tok_scale = torch.empty((T,), dtype=torch.float32, device=x.device) if tok_scale is None else tok_scale
    _need(xq, "xq", torch.int8, 2)
    _need(tok_scale, "tok_scale", torch.float32, 1)
    if xq.shape != (T, K) or tok_scale.shape != (T,):
        raise ValueError("shape mismatch in quant_act_int8_x")
    _check("tl_quant_act_int8_x", lib().tl_quant_act_int8_x(_ptr(x), T, K, _ptr(signs), _ptr(xq),
                                                            _ptr(tok_scale), _stream(x.device)))
    return xq, tok_scale


def gemv_workspace_size(b: int, K: int, N: int) -> int:
    return int(lib().tl_gemv_workspace_size(b, K, N))


def gemv_ternary(xr, packed, scales, out_dtype=None, out=None, workspace=None):
    """xr f32 [b,K] (b <= 64), packed tiles, scales fp16 [N,K/128] -> y [b,N]."""
    import torch
    _need(xr, "xr", torch.float32, 2)
    _need(scales, "scales", torch.float16, 2)
    b, K = xr.shape
    N = scales.shape[0]
    _check_packed(packed, N, K)
    if scales.shape != (N, K // GROUP):
        raise ValueError("shape mismatch in gemv_ternary")
    if out is None:
        out = torch.empty((b, N), dtype=out_dtype or torch.bfloat16, device=xr.device)
    code = _out_code(out.dtype)
    _need(out, "out", out.dtype, 2)
    if out.shape != (b, N):
        raise ValueError("out must be [b, N]")
    need = gemv_workspace_size(b, K, N)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=xr.device)
    _need(workspace, "workspace", torch.uint8, 1)
    _check("tl_gemv_ternary", lib().tl_gemv_ternary(
        _ptr(xr), b, K, N, _ptr(packed), _ptr(scales), _ptr(out), code, _ptr(workspace),
        workspace.numel(), _stream(xr.device)))
    return out


def gemv_ternary_q8(xq, tok_scale, packed, scales, out_dtype=None, out=None):
    """Decode GEMV against int8 activations: xq int8 [b,K] and tok_scale f32 [b]
    (from quant_act_int8 / quant_act_int8_x), packed tiles, scales -> y [b,N]."""
    import torch
    _need(xq, "xq", torch.int8, 2)
    _need(tok_scale, "tok_scale", torch.float32, 1)
    _need(scales, "scales", torch.float16, 2)
    b, K = xq.shape
    N = scales.shape[0]
    _check_packed(packed, N, K)
    if scales.shape != (N, K // GROUP) or tok_scale.shape != (b,):
        raise ValueError("shape mismatch in gemv_ternary_q8")
    if out is None:
        out = torch.empty((b, N), dtype=out_dtype or torch.bfloat16, device=xq.device)
    code = _out_code(out.dtype)
    _need(out, "out", out.dtype, 2)
    if out.shape != (b, N):
        raise ValueError("out must be [b, N]")
    _check("tl_gemv_ternary_q8", lib().tl_gemv_ternary_q8(
        _ptr(xq), _ptr(tok_scale), b, K, N, _ptr(packed), _ptr(scales), _ptr(out), code, _stream(xq.device)))
    return out


def gemv_prepare(xr, workspace):
    """First stage of gemv_ternary: activation limbs of xr f32 [b,K] into ``workspace``."""
    import torch
    _need(xr, "xr", torch.float32, 2)
    _need(workspace, "workspace", torch.uint8, 1)
    b, K = xr.shape
    _check("tl_gemv_prepare", lib().tl_gemv_prepare(_ptr(xr), b, K, _ptr(workspace), workspace.numel(),
                                                    _stream(xr.device)))
    return workspace


def gemv_prepared(workspace, b, K, packed, scales, out):
    """Second stage of gemv_ternary: y [b,N] from a workspace filled by gemv_prepare(b, K)."""
    import torch
    _need(workspace, "workspace", torch.uint8, 1)
    _need(scales, "scales", torch.float16, 2)
    N = scales.shape[0]
    _check_packed(packed, N, K)
    if scales.shape != (N, K // GROUP) or out.shape != (b, N):
        raise ValueError("shape mismatch in gemv_prepared")
    code = _out_code(out.dtype)
    _need(out, "out", out.dtype, 2)
    _check("tl_gemv_prepared", lib().tl_gemv_prepared(
        _ptr(workspace), workspace.numel(), b, K, N, _ptr(packed), _ptr(scales), _ptr(out), code,
        _stream(out.device)))
    return out


def quant_act_int8(xr, xq=None, tok_scale=None):
    """xr f32 [T,K] -> (xq int8 [T,K], tok_scale f32 [T])."""
    import torch
    _need(xr, "xr", torch.float32, 2)
    T, K = xr.shape
    xq = torch.empty((T, K), dtype=torch.int8, device=xr.device) if xq is None else xq
    tok_scale = torch.empty((T,), dtype=torch.float32, device=xr.device) if tok_scale is None else tok_scale
    _need(xq, "xq", torch.int8, 2)
    _need(tok_scale, "tok_scale", torch.float32, 1)
    if xq.shape != (T, K) or tok_scale.shape != (T,):
        raise ValueError("shape mismatch in quant_act_int8")
    _check("tl_quant_act_int8", lib().tl_quant_act_int8(_ptr(xr), T, K, _ptr(xq), _ptr(tok_scale),
                                                        _stream(xr.device)))
    return xq, tok_scale


_GEMM_WS = {}


def _gemm_workspace(device, nbytes):
    """A zero-filled GEMM workspace per (device, stream), grown on demand.

    The kernels return the workspace's counters to zero at the end of every
    call, so one buffer serves every call issued on that stream."""
    import torch
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    ws = _GEMM_WS.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros((nbytes,), dtype=torch.uint8, device=device)
        _GEMM_WS[key] = ws
    return ws


def gemm_workspace_size(M: int, K: int, N: int) -> int:
    return int(lib().tl_gemm_workspace_size(M, K, N))


def gemm_int8_rescale(xq, tok_scale, packed, q, row_scale, out_dtype=None, out=None, acc_out=None,
                      want_acc=False, workspace=None):
    """xq int8 [M,K], tok_scale f32 [M], packed/q/row_scale from pack_weights -> y [M,N]
    (and the exact int32 accumulator when ``want_acc`` or ``acc_out`` is given)."""
    import torch
    _need(xq, "xq", torch.int8, 2)
    _need(tok_scale, "tok_scale", torch.float32, 1)
    _need(q, "q", torch.int8, 2)
    _need(row_scale, "row_scale", torch.float32, 1)
    M, K = xq.shape
    N = q.shape[0]
    _check_packed(packed, N, K)
    if tok_scale.shape != (M,) or q.shape != (N, K // GROUP) or row_scale.shape != (N,):
        raise ValueError("shape mismatch in gemm_int8_rescale")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype or torch.bfloat16, device=xq.device)
    code = _out_code(out.dtype)
    _need(out, "out", out.dtype, 2)
    if out.shape != (M, N):
        raise ValueError("out must be [M, N]")
    if acc_out is None and want_acc:
        acc_out = torch.empty((M, N), dtype=torch.int32, device=xq.device)
    if acc_out is not None:
        _need(acc_out, "acc_out", torch.int32, 2)
        if acc_out.shape != (M, N):
            raise ValueError("acc_out must be [M, N]")
    need = gemm_workspace_size(M, K, N)
    if workspace is None and need:
        workspace = _gemm_workspace(xq.device, need)
    ws_bytes = workspace.numel() if workspace is not None else 0
    _check("tl_gemm_int8_rescale", lib().tl_gemm_int8_rescale(
        _ptr(xq), _ptr(tok_scale), M, K, N, _ptr(packed), _ptr(q), _ptr(row_scale), _ptr(out), code,
        _ptr(acc_out), _ptr(workspace), ws_bytes, _stream(xq.device)))
    return (out, acc_out) if acc_out is not None else out


def linear_path(T: int, K: int, N: int) -> int:
    """PATH_GEMV or PATH_INT8: the path linear_apply takes for T tokens of a K -> N layer."""
    return int(lib().tl_linear_path(T, K, N))


def linear_workspace_size(T: int, K: int, N: int) -> int:
    return int(lib().tl_linear_workspace_size(T, K, N))


_LIN_WS = {}


def _linear_workspace(device, nbytes):
    """A zero-filled layer workspace per (device, stream), grown on demand (every
    call leaves its counter region at zero, so one buffer serves every call)."""
    import torch
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    ws = _LIN_WS.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros((nbytes,), dtype=torch.uint8, device=device)
        _LIN_WS[key] = ws
    return ws


def linear_apply(x, packed, scales, q, row_scale, signs=None, out_dtype=None, out=None, workspace=None):
    """The whole layer from the raw input: x bf16 [T,K] -> y [T,N], on the path
    linear_path(T, K, N) names (two-limb GEMV, or int8 quantisation + int8 GEMM)."""
    import torch
    _check_x(x, signs)
    _need(scales, "scales", torch.float16, 2)
    _need(q, "q", torch.int8, 2)
    _need(row_scale, "row_scale", torch.float32, 1)
    T, K = x.shape
    N = scales.shape[0]
    _check_packed(packed, N, K)
    if scales.shape != (N, K // GROUP) or q.shape != (N, K // GROUP) or row_scale.shape != (N,):
        raise ValueError("shape mismatch in linear_apply")
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype or torch.bfloat16, device=x.device)
    code = _out_code(out.dtype)
    _need(out, "out", out.dtype, 2)
    if out.shape != (T, N):
        raise ValueError("out must be [T, N]")
    need = linear_workspace_size(T, K, N)
    if workspace is None:
        workspace = _linear_workspace(x.device, max(need, 1))
    _need(workspace, "workspace", torch.uint8, 1)
    _check("tl_linear_apply", lib().tl_linear_apply(
        _ptr(x), T, K, N, _ptr(signs), _ptr(packed), _ptr(scales), _ptr(q), _ptr(row_scale), _ptr(out), code,
        _ptr(workspace), workspace.numel(), _stream(x.device)))
    return out


def read_probe(src, sink):
    """Measurement helper: one launch that only reads the bytes of ``src`` (see
    tl_read_probe); ``sink`` is a 4-byte (or larger) device tensor."""
    if not (src.is_cuda and sink.is_cuda and src.is_contiguous()):
        raise ValueError("read_probe needs contiguous device tensors")
    nbytes = src.numel() * src.element_size() // 16 * 16
    _check("tl_read_probe", lib().tl_read_probe(_ptr(src), nbytes, _ptr(sink), _stream(src.device)))


def mfma_probe(random_operands, iters, sink):
    """Measurement helper: one launch that only issues int8 matrix instructions
    (see tl_mfma_probe); ``sink`` is a 4-byte (or larger) device tensor."""
    if not sink.is_cuda:
        raise ValueError("mfma_probe needs a device tensor")
    _check("tl_mfma_probe", lib().tl_mfma_probe(1 if random_operands else 0, int(iters), _ptr(sink),
                                                _stream(sink.device)))


def noalloc_scratch_bytes() -> int:
    """Size of the static per-GPU scratch array behind linear_apply_noalloc."""
    return int(lib().tl_noalloc_scratch_bytes())


def linear_apply_noalloc(x, packed, scales, q, row_scale, signs=None, out_dtype=None, out=None):
    """linear_apply without a workspace: the library's static per-GPU scratch array
    serves instead (same kernels, same outputs).  Calls that overlap in time on
    one GPU share that array and race.  ``out`` may be given so that the call
    allocates nothing at all."""
    import torch
    _check_x(x, signs)
    _need(scales, "scales", torch.float16, 2)
    _need(q, "q", torch.int8, 2)
    _need(row_scale, "row_scale", torch.float32, 1)
    T, K = x.shape
    N = scales.shape[0]
    _check_packed(packed, N, K)
    if scales.shape != (N, K // GROUP) or q.shape != (N, K // GROUP) or row_scale.shape != (N,):
        raise ValueError("shape mismatch in linear_apply_noalloc")
    if out is None:
        out = torch.empty((T, N), dtype=out_dtype or torch.bfloat16, device=x.device)
    code = _out_code(out.dtype)
    _need(out, "out", out.dtype, 2)
    if out.shape != (T, N):
        raise ValueError("out must be [T, N]")
    _check("tl_linear_apply_noalloc", lib().tl_linear_apply_noalloc(
        _ptr(x), T, K, N, _ptr(signs), _ptr(packed), _ptr(scales), _ptr(q), _ptr(row_scale), _ptr(out), code,
        _stream(x.device)))
    return out


def _need_rows(t, name, dtype, cols):
    """A 2-D device tensor of ``cols`` contiguous columns whose rows may be further apart."""
    import torch
    if not isinstance(t, torch.Tensor) or t.device.type != "cuda":
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or t.dim() != 2 or t.shape[1] != cols or t.stride(1) != 1:
        raise ValueError(f"{name} must be a {dtype} [T, {cols}] view with unit column stride")


def hadamard_half(x, signs=None, u=None):
    """First split-block stage: x bf16 [T,512] (rows may be a column slice of a wider
    input) -> u f64 [T,512] = H512 (d * x), exact, no 1/32."""
    import torch
    _need_rows(x, "x", torch.bfloat16, 512)
    if signs is not None:
        _need(signs, "signs", torch.int8, 1)
        if signs.shape != (512,):
            raise ValueError("signs must be [512]")
    T = x.shape[0]
    u = torch.empty((T, 512), dtype=torch.float64, device=x.device) if u is None else u
    _need(u, "u", torch.float64, 2)
    if u.shape != (T, 512):
        raise ValueError("u must be [T, 512]")
    _check("tl_hadamard_half", lib().tl_hadamard_half(_ptr(x), T, x.stride(0) if T > 1 else 512, _ptr(signs),
                                                      _ptr(u), _stream(x.device)))
    return u


def hadamard_join(u_lo, u_hi, half, out=None):
    """Second split-block stage: the rank's 512 rotated columns, f32 [T,512]
    (``out`` may be a column slice of the rank's rotated input)."""
    import torch
    _need(u_lo, "u_lo", torch.float64, 2)
    _need(u_hi, "u_hi", torch.float64, 2)
    T = u_lo.shape[0]
    if u_lo.shape != (T, 512) or u_hi.shape != (T, 512):
        raise ValueError("u_lo and u_hi must be [T, 512]")
    out = torch.empty((T, 512), dtype=torch.float32, device=u_lo.device) if out is None else out
    _need_rows(out, "out", torch.float32, 512)
    if out.shape[0] != T:
        raise ValueError("out must have T rows")
    _check("tl_hadamard_join", lib().tl_hadamard_join(_ptr(u_lo), _ptr(u_hi), T, int(half), _ptr(out),
                                                      out.stride(0) if T > 1 else 512, _stream(u_lo.device)))
    return out


# ---------------------------------------------------------------------------
# one step of speculative decoding over a paged cache
# ---------------------------------------------------------------------------
TREE_NODES = 64


def _raw_stream(index):
    """The current HIP stream of GPU ``index``, as an address (a step makes many short calls:
    torch.cuda.current_stream builds an object for 2 us each time)."""
    import torch
    return torch._C._cuda_getCurrentRawStream(index)


def _given(t, name, dtype, shape, index):
    """A contiguous GPU tensor of this dtype and shape, on device number ``index``; its address."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != index or not t.is_contiguous():
        _need(t, name, dtype, len(shape))
        if t.get_device() != index:
            raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    return t.data_ptr()


def _rows(t, name, index):
    """A bf16 [tokens, heads, D] tensor with a token's heads next to each other, tokens a row or
    more apart: its address and that distance."""
    import torch
    if t.dtype is not torch.bfloat16 or t.dim() != 3 or t.get_device() != index:
        _need(t.contiguous(), name, torch.bfloat16, 3)
        raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")
    T, H, D = t.shape
    ld, sh, sd = t.stride()
    if sd != 1 and D > 1 or sh != D and H > 1:
        raise ValueError(f"{name}'s heads must lie next to each other (strides {t.stride()})")
    if T < 2:
        return t.data_ptr(), H * D
    if ld < H * D:
        raise ValueError(f"{name}'s tokens must not overlap (strides {t.stride()}): copy a broadcast tensor first")
    return t.data_ptr(), ld


def _index_of(t, name):
    """The number of the GPU that ``t`` is on."""
    i = t.get_device() if hasattr(t, "get_device") else None
    if i is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    if i < 0:
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return i


def _cache_code(k_cache, k_scale, v_scale):
    import torch
    if k_cache.dtype is torch.bfloat16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("a bfloat16 cache has no scales")
        return TL_BF16
    if k_cache.dtype is torch.float8_e4m3fn:
        if k_scale is None or v_scale is None:
            raise ValueError("an e4m3 cache needs k_scale and v_scale")
        return TL_E4M3
    raise TypeError("the cache must be torch.bfloat16 or torch.float8_e4m3fn")


def _cache_args(k_cache, v_cache, k_scale, v_scale, index, layers=False):
    """Checks a cache; its dtype code and addresses."""
    import torch
    code = _cache_code(k_cache, k_scale, v_scale)
    if k_cache.dim() != (5 if layers else 4):
        raise ValueError(f"k_cache must be [{'layers, ' if layers else ''}pages, heads, block, D]")
    shape = k_cache.shape
    k = _given(k_cache, "k_cache", k_cache.dtype, shape, index)
    v = _given(v_cache, "v_cache", k_cache.dtype, shape, index)
    if code == TL_BF16:
        return code, k, v, None, None
    ks = _given(k_scale, "k_scale", torch.float32, shape[:-1], index)
    return code, k, v, ks, _given(v_scale, "v_scale", torch.float32, shape[:-1], index)


def kv_cache(pages, heads, block, D, dtype=None, layers=None, device="cuda"):
    """A zeroed cache: (k_cache, v_cache, k_scale, v_scale), the caches [pages, heads, block, D]
    of bfloat16 (the default; scales None) or float8_e4m3fn (scales f32 [pages, heads, block]),
    each with a leading dimension if ``layers`` is given."""
    import torch
    dtype = dtype or torch.bfloat16
    shape = ((layers,) if layers is not None else ()) + (pages, heads, block, D)
    bits = {torch.bfloat16: torch.int16, torch.float8_e4m3fn: torch.uint8}.get(dtype)
    if bits is None:
        raise TypeError("the cache must be torch.bfloat16 or torch.float8_e4m3fn")
    k, v = (torch.zeros(shape, dtype=bits, device=device).view(dtype) for _ in "kv")
    if bits is torch.int16:
        return k, v, None, None
    return (k, v, *(torch.zeros(shape[:-1], dtype=torch.float32, device=device) for _ in "kv"))


def kv_offset(which, dtype, heads, D, block, page, head, token, d) -> int:
    """Element offset of (page, head, token in the page, d) in a cache layer; which is "k" or "v"."""
    import torch
    code = {torch.bfloat16: TL_BF16, torch.float8_e4m3fn: TL_E4M3}.get(dtype, -1)
    at = int(lib().tl_kv_offset({"k": 0, "v": 1}.get(which, -1), code, heads, D, block, page, head, token, d))
    if at < 0:
        raise ValueError("kv_offset: argument out of range")
    return at


def step_plan(ctx_lens, new_lens, owned, block_table, free_list, free_head, tokens, block, parents=None):
    """Metadata of a step from the request lengths (int32 [R] each), on the GPU: takes pages from
    ``free_list`` into ``block_table`` int32 [R, width] (in place) and returns (q_start [R+1],
    kv_lens [R], slots int64 [tokens], positions [tokens], tree_mask int64 [tokens] or None,
    owned [R], free_head [1]).  ``tokens`` is the step's token count or more (a graph's capacity); a
    request that does not fit it, the table or the free pages is not served (kv_lens 0, slots -1)."""
    import torch
    i32 = torch.int32
    i = _index_of(ctx_lens, "ctx_lens")
    if ctx_lens.dim() != 1 or block_table.dim() != 2 or free_list.dim() != 1:
        raise ValueError("step_plan needs ctx_lens [R], block_table [R, width] and free_list [F]")
    R, width, T = ctx_lens.shape[0], block_table.shape[1], int(tokens)
    if T < 0:
        raise ValueError("tokens must not be negative")
    p = [_given(ctx_lens, "ctx_lens", i32, (R,), i), _given(new_lens, "new_lens", i32, (R,), i),
         _given(owned, "owned", i32, (R,), i), _given(block_table, "block_table", i32, (R, width), i),
         _given(free_list, "free_list", i32, free_list.shape, i), _given(free_head, "free_head", i32, (1,), i),
         None if parents is None else _given(parents, "parents", i32, (T,), i)]
    dev = ctx_lens.device
    # the outputs share two allocations: each one alone would cost as much as the kernel
    q_start, kv_lens, positions, owned_out, head_out = torch.empty(
        3 * R + T + 2, dtype=i32, device=dev).split_with_sizes((R + 1, R, T, R, 1))
    if parents is None:
        slots, mask = torch.empty(T, dtype=torch.int64, device=dev), None
    else:
        slots, mask = torch.empty((2, T), dtype=torch.int64, device=dev).unbind()
    _check("tl_step_plan", lib().tl_step_plan(
        p[0], p[1], p[2], R, p[3], width, int(block), p[4], free_list.shape[0], p[5], p[6], T, q_start.data_ptr(),
        kv_lens.data_ptr(), slots.data_ptr(), positions.data_ptr(), None if mask is None else mask.data_ptr(),
        owned_out.data_ptr(), head_out.data_ptr(), _raw_stream(i)))
    return q_start, kv_lens, slots, positions, mask, owned_out, head_out


def kv_write(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None, q=None, positions=None, cos_sin=None,
             q_out=None):
    """Writes rows k, v bf16 [T, H, D] (tokens a row or more apart) to the cache at slots int64 [T] and
    returns q_out bf16 [T, Hq, D] if q is given.  With positions int32 [T] and cos_sin f32
    [max_pos, rot] (cosines, then sines) the first rot elements of q and k are rotated first.
    An e4m3 cache gets codes and scales."""
    import torch
    i = _index_of(k, "k")
    code, kc, vc, ks, vs = _cache_args(k_cache, v_cache, k_scale, v_scale, i)
    pages, H, block, D = k_cache.shape
    kp, ldk = _rows(k, "k", i)
    vp, ldv = _rows(v, "v", i)
    T = k.shape[0]
    if k.shape != (T, H, D) or v.shape != (T, H, D):
        raise ValueError(f"k and v must be [T, {H}, {D}]")
    sp = _given(slots, "slots", torch.int64, (T,), i)
    qp, ldq, Hq, qo = None, 0, 0, None
    if q is not None:
        qp, ldq = _rows(q, "q", i)
        Hq = q.shape[1]
        if q.shape != (T, Hq, D):
            raise ValueError(f"q must be [{T}, heads, {D}]")
        q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device) if q_out is None else q_out
        qo = _given(q_out, "q_out", torch.bfloat16, (T, Hq, D), i)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    pp, cp, most, rot = None, None, 0, 0
    if cos_sin is not None:
        if positions is None or cos_sin.dim() != 2:
            raise ValueError("cos_sin must be [max_pos, rot] and needs positions")
        most, rot = cos_sin.shape
        cp = _given(cos_sin, "cos_sin", torch.float32, (most, rot), i)
        pp = _given(positions, "positions", torch.int32, (T,), i)
    _check("tl_kv_write", lib().tl_kv_write(kp, ldk, vp, ldv, sp, T, H, D, qp, ldq, Hq, pp, cp, most, rot, qo, kc, vc,
                                            ks, vs, code, pages, block, _raw_stream(i)))
    return q_out


def tree_attention_workspace_size(max_nodes: int, group: int, D: int, dtype=None) -> int:
    """Bytes of workspace tree_attention needs; dtype is the cache's (bfloat16 by default)."""
    import torch
    code = TL_E4M3 if dtype is torch.float8_e4m3fn else TL_BF16
    return int(lib().tl_tree_attention_workspace_size(max_nodes, group, D, code))


def tree_attention(q, k_cache, v_cache, block_table, q_start, kv_lens, tree_mask=None, k_scale=None, v_scale=None,
                   scale=None, max_nodes=None, out=None, lse=None, workspace=None):
    """Attention of q bf16 [T, Hq, D] (tokens a row or more apart) over the paged cache: request r's tokens
    q_start[r] .. q_start[r+1]-1 see its first kv_lens[r] - n keys and, of its own n, those that
    tree_mask int64 [T] names (or, without a mask or above 64 tokens, those up to themselves).
    Returns out bf16 [T, Hq, D], or (out, lse) if ``lse`` f32 [T, Hq] is given (True: made here).
    ``max_nodes``: the most tokens of a request, as far as known (chooses the kernel)."""
    import torch
    i = _index_of(q, "q")
    code, kc, vc, ks, vs = _cache_args(k_cache, v_cache, k_scale, v_scale, i)
    pages, H, block, D = k_cache.shape
    qp, ldq = _rows(q, "q", i)
    T, Hq, width = q.shape[0], q.shape[1], block_table.shape[-1]
    R = block_table.shape[0]
    if q.shape[2] != D or Hq % H or Hq == 0:
        raise ValueError(f"q must be [T, a multiple of {H}, {D}]")
    G = Hq // H
    tp = _given(block_table, "block_table", torch.int32, (R, width), i)
    sp = _given(q_start, "q_start", torch.int32, (R + 1,), i)
    lp = _given(kv_lens, "kv_lens", torch.int32, (R,), i)
    mp = None if tree_mask is None else _given(tree_mask, "tree_mask", torch.int64, (T,), i)
    out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device) if out is None else out
    op = _given(out, "out", torch.bfloat16, (T, Hq, D), i)
    lse = torch.empty((T, Hq), dtype=torch.float32, device=q.device) if lse is True else lse
    ep = None if lse is None else _given(lse, "lse", torch.float32, (T, Hq), i)
    if max_nodes is None:
        max_nodes = max(1, -(-T // max(R, 1)))
    if workspace is None:
        need = lib().tl_tree_attention_workspace_size(max_nodes, G, D, code)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    wp = _given(workspace, "workspace", torch.uint8, (workspace.numel(),), i)
    _check("tl_tree_attention", lib().tl_tree_attention(
        qp, ldq, T, H, G, D, kc, vc, ks, vs, code, pages, block, tp, width, R, sp, lp, mp,
        D ** -0.5 if scale is None else scale, max_nodes, op, ep, wp, workspace.numel(), _raw_stream(i)))
    return out if lse is None else (out, lse)


def tree_verify(logits, draft, parents, q_start, path_width=TREE_NODES, workspace=None):
    """Greedy check of drafted trees: logits bf16 or f32 [T, V] (any row distance), draft and parents
    int32 [T], q_start int32 [R+1] -> (accepted [R], path [R, path_width], next [R], target [T]).  What
    it says of a request that step_plan did not serve (kv_lens 0) means nothing."""
    import torch
    i = _index_of(logits, "logits")
    code = _out_code(logits.dtype)
    if logits.dim() != 2 or (logits.stride(1) != 1 and logits.shape[1] > 1):
        raise ValueError("logits must be [T, V] with unit column stride")
    T, V = logits.shape
    R = q_start.shape[0] - 1
    i32 = torch.int32
    dp = _given(draft, "draft", i32, (T,), i)
    pp = _given(parents, "parents", i32, (T,), i)
    sp = _given(q_start, "q_start", i32, (R + 1,), i)
    dev = logits.device
    accepted, path, nxt, target = torch.empty(R * (path_width + 2) + T, dtype=i32, device=dev).split_with_sizes(
        (R, R * path_width, R, T))
    path = path.view(R, path_width)
    if workspace is None:
        need = lib().tl_tree_verify_workspace_size(T, V)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    wp = _given(workspace, "workspace", torch.uint8, (workspace.numel(),), i)
    _check("tl_tree_verify", lib().tl_tree_verify(
        logits.data_ptr(), code, logits.stride(0) if T > 1 else V, T, V, dp, pp, sp, R, accepted.data_ptr(),
        path.data_ptr(), path_width, nxt.data_ptr(), target.data_ptr(), wp, workspace.numel(), _raw_stream(i)))
    return accepted, path, nxt, target


def kv_commit(accepted, path, ctx_lens, kv_lens, block_table, k_cache, v_cache, k_scale=None, v_scale=None,
              ctx_out=None):
    """Moves the rows of the accepted nodes (tree_verify's accepted [R] and path [R, width]) to the
    positions after the context, in a cache layer [pages, H, block, D] or all of them
    [L, pages, H, block, D]; returns the new context lengths int32 [R] (a tree's accepted nodes past the
    path's width are not committed)."""
    import torch
    i = _index_of(accepted, "accepted")
    layers = k_cache.dim() == 5
    code, kc, vc, ks, vs = _cache_args(k_cache, v_cache, k_scale, v_scale, i, layers)
    pages, H, block, D = k_cache.shape[-4:]
    R, i32 = accepted.shape[0], torch.int32
    if path.dim() != 2 or block_table.dim() != 2:
        raise ValueError("path must be [R, width] and block_table [R, pages]")
    ctx_out = torch.empty(R, dtype=i32, device=accepted.device) if ctx_out is None else ctx_out
    _check("tl_kv_commit", lib().tl_kv_commit(
        _given(accepted, "accepted", i32, (R,), i), _given(path, "path", i32, (R, path.shape[1]), i), path.shape[1],
        _given(ctx_lens, "ctx_lens", i32, (R,), i), _given(kv_lens, "kv_lens", i32, (R,), i),
        _given(block_table, "block_table", i32, (R, block_table.shape[1]), i), block_table.shape[1], R, kc, vc, ks, vs,
        code, k_cache.shape[0] if layers else 1, pages, H, block, D, _given(ctx_out, "ctx_out", i32, (R,), i),
        _raw_stream(i)))
    return ctx_out
