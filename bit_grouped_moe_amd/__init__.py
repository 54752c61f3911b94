"""Python binding of libgq (grouped MoE matmul on 4-bit packed experts, MI355X).

The functions below carry the names of the C entry points declared in
``include/gq.h`` and only marshal arguments: they check tensor shapes,
dtypes, devices and contiguity, allocate outputs with torch when the caller
passes none, and call the library on torch's current stream.  Every step of
the computation runs in the HIP kernels of ``libgq.so``; there is no CPU or
PyTorch fallback.  If the library is missing, every call raises.

Build the library with ``python -m bit_grouped_moe_amd.build``.
"""

import ctypes
import importlib.machinery
import importlib.util
import os
from collections import namedtuple

import torch

__all__ = [
    "GQError", "load_library", "library_path", "EXPORTED_SYMBOLS", "TILE_M",
    "gq_route_max_tiles", "gq_route_sort", "gq_nf4_decode", "gq_mxfp4_decode",
    "gq_nf4_grouped_gemv", "gq_mxfp4_grouped_gemv", "gq_nf4_grouped_gemm",
    "gq_mxfp4_grouped_gemm", "gq_nf4_grouped_dgrad", "gq_mxfp4_grouped_dgrad",
    "gq_nf4_grouped_gemv_swiglu", "gq_nf4_grouped_gemm_swiglu", "gq_nf4_grouped_gemv_down_combine",
    "gq_moe_combine", "gq_act_split_e4m3", "gq_mxfp4_grouped_gemm_scaled",
    "gq_mxfp4_grouped_gemv_swiglu", "gq_mxfp4_grouped_gemm_scaled_swiglu",
    "gq_mxfp4_grouped_gemm_scaled_swiglu_split",
    "gq_mxfp4_grouped_gemv_down_combine", "gq_nf4_grouped_gemv_host", "gq_mxfp4_grouped_gemv_host",
    "gq_mxfp4_quantize", "gq_moe_topk", "gq_moe_topk_backward", "gq_moe_layer",
    "gq_moe_decode_workspace", "gq_moe_decode", "gq_mxfp4_grouped_gemm_fp4",
    "gq_mxfp4_grouped_gemm_fp4_swiglu", "gq_mxfp4_grouped_gemv_fp4",
    "gq_mxfp4_grouped_gemv_fp4_swiglu",
    "gq_mxfp8_quantize", "gq_rms_norm", "gq_rms_norm_backward", "gq_rms_norm_backward_workspace",
    "gq_mxfp4_grouped_gemm_fp8", "gq_mxfp4_grouped_gemm_fp8_swiglu",
    "gq_mxfp4_grouped_gemv_fp8", "gq_mxfp4_grouped_gemv_fp8_swiglu",
    "gq_moe_route", "gq_moe_route_backward",
    "OSS_ALPHA", "OSS_LIMIT", "Route", "RmsNorm",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
TILE_M = 256                       # the tile height the grouped GEMM kernels use
OSS_ALPHA = 1.702                  # gpt-oss gated unit: sigmoid slope
OSS_LIMIT = 7.0                    # gpt-oss gated unit: clamp

EXPORTED_SYMBOLS = (
    "gq_status_string", "gq_route_max_tiles", "gq_route_sort", "gq_nf4_decode",
    "gq_mxfp4_decode", "gq_nf4_grouped_gemv", "gq_mxfp4_grouped_gemv", "gq_nf4_grouped_gemm",
    "gq_mxfp4_grouped_gemm", "gq_nf4_grouped_dgrad", "gq_mxfp4_grouped_dgrad",
    "gq_nf4_grouped_gemv_swiglu", "gq_nf4_grouped_gemm_swiglu", "gq_nf4_grouped_gemv_down_combine",
    "gq_moe_combine", "gq_act_split_e4m3", "gq_mxfp4_grouped_gemm_scaled",
    "gq_mxfp4_grouped_gemv_swiglu", "gq_mxfp4_grouped_gemm_scaled_swiglu",
    "gq_mxfp4_grouped_gemm_scaled_swiglu_split",
    "gq_mxfp4_grouped_gemv_down_combine", "gq_nf4_grouped_gemv_host", "gq_mxfp4_grouped_gemv_host",
    "gq_mxfp4_quantize", "gq_moe_topk", "gq_moe_topk_backward", "gq_moe_decode_workspace",
    "gq_moe_decode", "gq_mxfp4_grouped_gemm_fp4", "gq_mxfp4_grouped_gemm_fp4_swiglu",
    "gq_mxfp4_grouped_gemv_fp4", "gq_mxfp4_grouped_gemv_fp4_swiglu",
    "gq_mxfp8_quantize", "gq_rms_norm", "gq_rms_norm_backward", "gq_rms_norm_backward_workspace",
    "gq_mxfp4_grouped_gemm_fp8", "gq_mxfp4_grouped_gemm_fp8_swiglu",
    "gq_mxfp4_grouped_gemv_fp8", "gq_mxfp4_grouped_gemv_fp8_swiglu",
    "gq_moe_route", "gq_moe_route_backward",
)

_i32, _i64, _p, _f32 = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float
_SIGNATURES = {
    "gq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "gq_route_max_tiles": (_i32, [_i32, _i32, _i32, _i32]),
    "gq_route_sort": (ctypes.c_int, [_p, _i32, _i32, _i32, _i32, _p, _p, _p, _i32, _p, _p]),
    "gq_nf4_decode": (ctypes.c_int, [_p, _p, _i64, _i32, _p, _p, _p]),
    "gq_mxfp4_decode": (ctypes.c_int, [_p, _p, _i64, _i32, _p, _p, _p]),
    "gq_nf4_grouped_gemv": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _p, _i32,
                                           _p, _p, _p]),
    "gq_mxfp4_grouped_gemv": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _p, _i32,
                                             _p, _p, _p]),
    "gq_nf4_grouped_gemm": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _i32, _p,
                                           _p, _p, _p, _p, _i32, _i32, _p, _p]),
    "gq_mxfp4_grouped_gemm": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _i32, _p,
                                             _p, _p, _p, _p, _i32, _i32, _p, _p]),
    "gq_nf4_grouped_dgrad": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _p, _p,
                                            _p, _p, _i32, _i32, _p, _p]),
    "gq_mxfp4_grouped_dgrad": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _p, _p,
                                              _p, _p, _i32, _i32, _p, _p]),
    "gq_nf4_grouped_gemv_swiglu": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _p,
                                                  _i32, _p, _p]),
    "gq_nf4_grouped_gemm_swiglu": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _i32,
                                                  _p, _p, _p, _p, _i32, _i32, _p, _p]),
    "gq_nf4_grouped_gemv_down_combine": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32,
                                                        _p, _i32, _p, _p, _p]),
    "gq_moe_combine": (ctypes.c_int, [_p, _i32, _i32, _i32, _i64, _p, _p, _p]),
    "gq_act_split_e4m3": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _p]),
    "gq_mxfp4_grouped_gemm_scaled": (ctypes.c_int, [_p, _p, _i32, _i32, _p, _p, _i32, _i32, _i32,
                                                    _p, _p, _p, _p, _p, _i32, _i32, _p, _p]),
    "gq_nf4_grouped_gemv_host": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _p,
                                                _i32, _p, _p, _p]),
    "gq_mxfp4_grouped_gemv_host": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _p,
                                                  _i32, _p, _p, _p]),
    "gq_mxfp4_grouped_gemv_down_combine": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32,
                                                          _i32, _p, _i32, _p, _p, _p]),
    "gq_mxfp4_grouped_gemv_swiglu": (ctypes.c_int, [_p, _i32, _i32, _i64, _p, _p, _i32, _i32, _p,
                                                    _i32, _f32, _f32, _p, _p]),
    "gq_mxfp4_grouped_gemm_scaled_swiglu": (ctypes.c_int, [_p, _p, _i32, _i32, _p, _p, _i32,
                                                           _i32, _i32, _f32, _f32, _p, _p, _p,
                                                           _p, _i32, _i32, _p, _p]),
    "gq_mxfp4_grouped_gemm_scaled_swiglu_split": (ctypes.c_int, [_p, _p, _i32, _i32, _p, _p,
                                                                 _i32, _i32, _i32, _f32, _f32,
                                                                 _p, _p, _p, _p, _i32, _i32, _p,
                                                                 _p, _p]),
    "gq_mxfp4_quantize": (ctypes.c_int, [_p, _i32, _i64, _i32, _i64, _p, _p, _p, _p]),
    "gq_moe_topk": (ctypes.c_int, [_p, _i32, _i64, _i32, _i64, _i32, _i32, _p, _p, _p]),
    "gq_moe_topk_backward": (ctypes.c_int, [_p, _p, _i32, _i64, _i32, _i64, _p, _i32, _i32, _p,
                                            _p]),
    "gq_mxfp4_grouped_gemm_fp4": (ctypes.c_int, [_p, _p, _i32, _i32, _p, _p, _i32, _i32, _i32, _p,
                                                 _p, _p, _p, _p, _i32, _i32, _p, _p]),
    "gq_mxfp4_grouped_gemm_fp4_swiglu": (ctypes.c_int, [_p, _p, _i32, _i32, _p, _p, _i32, _i32,
                                                        _i32, _f32, _f32, _p, _p, _p, _p, _i32,
                                                        _i32, _p, _p]),
    "gq_mxfp4_grouped_gemv_fp4": (ctypes.c_int, [_p, _p, _i32, _i32, _p, _p, _i32, _i32, _p, _i32,
                                                 _p, _p, _p]),
    "gq_mxfp4_grouped_gemv_fp4_swiglu": (ctypes.c_int, [_p, _p, _i32, _i32, _p, _p, _i32, _i32,
                                                        _p, _i32, _f32, _f32, _p, _p]),
    "gq_moe_route": (ctypes.c_int, [_p, _i32, _i64, _i32, _i64, _p, _i32, _i32, _i32, _i32, _i32,
                                    _i32, _f32, _p, _p, _p]),
    "gq_moe_route_backward": (ctypes.c_int, [_p, _p, _i32, _i64, _i32, _i64, _p, _i32, _i32, _i32,
                                             _f32, _p, _p]),
    "gq_mxfp8_quantize": (ctypes.c_int, [_p, _i32, _i64, _i32, _i64, _p, _p, _p, _p]),
    "gq_rms_norm": (ctypes.c_int, [_p, _i64, _p, _i64, _i32, _i64, _i32, _p, _i32, _f32, _p, _p,
                                   _p, _p, _p, _p]),
    "gq_rms_norm_backward_workspace": (_i64, [_i64, _i32]),
    "gq_rms_norm_backward": (ctypes.c_int, [_p, _i64, _p, _i64, _p, _i64, _i32, _i64, _i32, _p,
                                            _i32, _f32, _p, _p, _p, _i64, _p]),
    "gq_moe_decode_workspace": (_i64, [_p, _i32]),
    "gq_moe_decode": (ctypes.c_int, [_p, _p, _i32, _i64, _p, _i64, _p, _p]),
}
for _n in ("gemm_fp4", "gemm_fp4_swiglu", "gemv_fp4", "gemv_fp4_swiglu"):
    _SIGNATURES["gq_mxfp4_grouped_" + _n.replace("fp4", "fp8")] = _SIGNATURES["gq_mxfp4_grouped_"
                                                                              + _n]

_lib = None
_calls = None                      # the short calls (csrc/binding/calls.cpp), when built


class GQError(RuntimeError):
    """A libgq call returned a nonzero status, or the library is missing."""

    def __init__(self, msg, status=None):
        super().__init__(msg)
        self.status = status


def library_path():
    return os.environ.get("GQ_LIBRARY", os.path.join(_HERE, "libgq.so"))


def load_library():
    """Load libgq.so (once) and declare its C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise GQError(f"libgq.so not found at {path}; build it with "
                      "`python -m bit_grouped_moe_amd.build` (no fallback exists)")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    _load_calls(lib)
    return lib


def _load_calls(lib):
    """Load the short calls and hand them the library's entry points.  Without
    them (not built, or built against another torch or another include/gq.h)
    every call takes the Python way, with the same checks, kernels and results."""
    global _calls
    _calls = None
    path = os.path.join(_HERE, "_calls.so")
    if not os.path.exists(path):
        return
    try:
        loader = importlib.machinery.ExtensionFileLoader("_calls", path)
        mod = importlib.util.module_from_spec(importlib.util.spec_from_loader("_calls", loader))
        loader.exec_module(mod)
    except ImportError:
        return
    if mod.torch_version != torch.__version__ or not _same_header(mod):
        return
    mod.bind({n: ctypes.cast(getattr(lib, n), _p).value for n in EXPORTED_SYMBOLS},
             torch.cuda.current_device, _raw_stream)
    _calls = mod


def _same_header(mod):
    """Whether the module was built with the include/gq.h that is there now."""
    from . import build
    try:
        return getattr(mod, "header_id", None) == build.header_id()
    except OSError:
        return False


def _check(status, what):
    if status != 0:
        lib = load_library()
        raise GQError(f"{what}: {lib.gq_status_string(status).decode()} (status {status})", status)


# The raw handle of a device's current stream, without the Stream object that
# torch.cuda.current_stream builds (1.9 us against 0.1 us, of a decode call
# that takes about 10); a torch built without it takes the slower way.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(t):
    return _raw_stream(t.get_device())


def _dev(t, name, dtype, ndim=None):
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype is dtype and t.is_contiguous()
            and (ndim is None or t.dim() == ndim)):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims (got shape {tuple(t.shape)})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _ints(what, *sizes):
    """Sizes that the library takes in 32 bits: ctypes would pass the low half
    of a larger one."""
    for n in sizes:
        if not -(1 << 31) <= n < 1 << 31:
            raise GQError(f"{what}: a size of {n} is not supported", 801)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _done(result, what):
    """A short call's outputs; its status, if it is one, as an error."""
    if type(result) is int:
        _check(result, what)
    return result


Route = namedtuple("Route", "expert_offsets sorted_pairs tiles num_tiles max_tiles tile_m "
                            "rows topk num_experts")


def gq_route_max_tiles(rows, topk, num_experts, tile_m=TILE_M):
    _ints("gq_route_max_tiles", rows, topk, num_experts, tile_m)
    return int(load_library().gq_route_max_tiles(rows, topk, num_experts, tile_m))


def gq_route_sort(topk_ids, num_experts, tile_m=TILE_M, expert_offsets=None, sorted_pairs=None,
                  tiles=None, num_tiles=None):
    """Group the (token, slot) pairs of ``topk_ids`` int32 [rows, topk] by expert."""
    lib = _lib or load_library()
    if _calls and expert_offsets is sorted_pairs is tiles is num_tiles is None:
        r = _calls.route_sort(topk_ids, num_experts, tile_m)
        if r is not None:
            r = _done(r, "gq_route_sort")
            return Route(*r, r[2].shape[0], tile_m, *topk_ids.shape, num_experts)
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    rows, topk = topk_ids.shape
    dev = topk_ids.device
    max_tiles = gq_route_max_tiles(rows, topk, num_experts, tile_m)
    if max_tiles < 0:
        raise GQError("gq_route_max_tiles: invalid arguments", 1)
    if expert_offsets is None:
        expert_offsets = torch.empty(num_experts + 1, dtype=torch.int32, device=dev)
    if sorted_pairs is None:
        sorted_pairs = torch.empty(rows * topk, dtype=torch.int32, device=dev)
    if tiles is None:
        tiles = torch.empty((max_tiles, 2), dtype=torch.int32, device=dev)
    if num_tiles is None:
        num_tiles = torch.empty(1, dtype=torch.int32, device=dev)
    st = lib.gq_route_sort(_ptr(topk_ids), rows, topk, num_experts, tile_m, _ptr(expert_offsets),
                           _ptr(sorted_pairs), _ptr(tiles), tiles.shape[0], _ptr(num_tiles),
                           _stream(topk_ids))
    _check(st, "gq_route_sort")
    return Route(expert_offsets, sorted_pairs, tiles, num_tiles, tiles.shape[0], tile_m, rows,
                 topk, num_experts)


def gq_nf4_decode(codes, absmax, out_f32=True, out_bf16=True):
    """Decode NF4 codes uint8 [..., K/2] with absmax float32 [..., K/64]."""
    lib = _lib or load_library()
    _dev(codes, "codes", torch.uint8)
    _dev(absmax, "absmax", torch.float32)
    K = codes.shape[-1] * 2
    n_rows = codes.numel() // (K // 2) if K else 0
    shape = tuple(codes.shape[:-1]) + (K,)
    f = torch.empty(shape, dtype=torch.float32, device=codes.device) if out_f32 is True else out_f32
    b = torch.empty(shape, dtype=torch.bfloat16, device=codes.device) if out_bf16 is True else out_bf16
    f = None if f is False else f
    b = None if b is False else b
    st = lib.gq_nf4_decode(_ptr(codes), _ptr(absmax), n_rows, K, _ptr(f), _ptr(b), _stream(codes))
    _check(st, "gq_nf4_decode")
    return f, b


def gq_mxfp4_decode(blocks, scales, out_f32=True, out_bf16=True):
    """Decode MXFP4 blocks uint8 [..., K/32, 16] with e8m0 scales uint8 [..., K/32]."""
    lib = _lib or load_library()
    _dev(blocks, "blocks", torch.uint8)
    _dev(scales, "scales", torch.uint8)
    K = blocks.shape[-2] * 32
    n_rows = blocks.numel() // (K // 2) if K else 0
    shape = tuple(blocks.shape[:-2]) + (K,)
    f = torch.empty(shape, dtype=torch.float32, device=blocks.device) if out_f32 is True else out_f32
    b = torch.empty(shape, dtype=torch.bfloat16, device=blocks.device) if out_bf16 is True else out_bf16
    f = None if f is False else f
    b = None if b is False else b
    st = lib.gq_mxfp4_decode(_ptr(blocks), _ptr(scales), n_rows, K, _ptr(f), _ptr(b),
                             _stream(blocks))
    _check(st, "gq_mxfp4_decode")
    return f, b


def _x_args(x, name="x"):
    if not isinstance(x, torch.Tensor) or not x.is_cuda or x.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be a bf16 device tensor")
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError(f"{name} must be 2-D with unit column stride")
    return *x.shape, x.stride(0)


def _nf4_bank(codes, absmax):
    _dev(codes, "codes", torch.uint8, 3)
    _dev(absmax, "absmax", torch.float32, 3)
    E, N, half = codes.shape
    K = half * 2
    if tuple(absmax.shape) != (E, N, K // 64):
        raise ValueError("absmax must be [E, N, K/64]")
    return E, N, K


def _mx_bank(blocks, scales):
    _dev(blocks, "blocks", torch.uint8, 4)
    _dev(scales, "scales", torch.uint8, 3)
    E, N, nb, sixteen = blocks.shape
    if sixteen != 16 or scales.shape != (E, N, nb):
        raise ValueError("blocks must be [E, N, K/32, 16] and scales [E, N, K/32]")
    return E, N, nb * 32


def _out(out, P, N, dev):
    if out is None:
        return torch.empty((P, N), dtype=torch.bfloat16, device=dev)
    _dev(out, "out", torch.bfloat16)
    if out.numel() != P * N:
        raise ValueError("out must hold rows*topk x N elements")
    return out


def _scale(pair_scale, P):
    if pair_scale is None:
        return None
    _dev(pair_scale, "pair_scale", torch.float32)
    if pair_scale.numel() != P:
        raise ValueError("pair_scale must hold one float per pair")
    return pair_scale


def _gemv_pairs(topk_ids, rows):
    """Pair count of a decode GEMV call: ``topk_ids`` must be [rows, topk]
    for the ``rows`` activation rows of x (the kernel reads pair p's row
    p / topk and writes rows*topk output rows)."""
    if topk_ids.dim() != 2 or topk_ids.shape[0] != rows:
        raise ValueError(f"topk_ids must be [rows={rows}, topk] (got {tuple(topk_ids.shape)})")
    return topk_ids.shape[0] * topk_ids.shape[1]


def gq_nf4_grouped_gemv(x, codes, absmax, topk_ids, pair_scale=None, out=None):
    """Decode-time grouped GEMV (<= 256 pairs) on NF4 experts; returns bf16 [rows*topk, N]."""
    lib = _lib or load_library()
    rows, K, xs = _x_args(x)
    E, N, Kw = _nf4_bank(codes, absmax)
    if Kw != K:
        raise ValueError("x and codes disagree on K")
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    P = _gemv_pairs(topk_ids, rows)
    out = _out(out, P, N, x.device)
    st = lib.gq_nf4_grouped_gemv(_ptr(x), rows, K, xs, _ptr(codes), _ptr(absmax), E, N,
                                 _ptr(topk_ids), topk_ids.shape[1], _ptr(_scale(pair_scale, P)),
                                 _ptr(out), _stream(x))
    _check(st, "gq_nf4_grouped_gemv")
    return out


def gq_mxfp4_grouped_gemv(x, blocks, scales, topk_ids, pair_scale=None, out=None):
    """Decode-time grouped GEMV (<= 256 pairs) on MXFP4 experts; returns bf16 [rows*topk, N]."""
    lib = _lib or load_library()
    rows, K, xs = _x_args(x)
    E, N, Kw = _mx_bank(blocks, scales)
    if Kw != K:
        raise ValueError("x and blocks disagree on K")
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    P = _gemv_pairs(topk_ids, rows)
    out = _out(out, P, N, x.device)
    st = lib.gq_mxfp4_grouped_gemv(_ptr(x), rows, K, xs, _ptr(blocks), _ptr(scales), E, N,
                                   _ptr(topk_ids), topk_ids.shape[1], _ptr(_scale(pair_scale, P)),
                                   _ptr(out), _stream(x))
    _check(st, "gq_mxfp4_grouped_gemv")
    return out


def gq_mxfp4_grouped_gemv_swiglu(x, blocks, scales, topk_ids, alpha=OSS_ALPHA, limit=OSS_LIMIT,
                                 out=None):
    """Decode gate_up GEMV on MXFP4 experts with gpt-oss's gated unit fused:
    blocks [E, 2I, K] with gate row 2j and up row 2j + 1; returns bf16
    [rows*topk, I] = gc * sigmoid(alpha gc) * (uc + 1) (gc = min(gate, limit),
    uc = up clipped to [-limit, limit])."""
    lib = _lib or load_library()
    rows, K, xs = _x_args(x)
    E, N2, Kw = _mx_bank(blocks, scales)
    if Kw != K or N2 % 2:
        raise ValueError("x and blocks disagree on K, or the gate_up width is odd")
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    P = _gemv_pairs(topk_ids, rows)
    out = _out(out, P, N2 // 2, x.device)
    st = lib.gq_mxfp4_grouped_gemv_swiglu(_ptr(x), rows, K, xs, _ptr(blocks), _ptr(scales), E, N2,
                                          _ptr(topk_ids), topk_ids.shape[1], float(alpha),
                                          float(limit), _ptr(out), _stream(x))
    _check(st, "gq_mxfp4_grouped_gemv_swiglu")
    return out


def _host_bank(a, b, names):
    """Host-resident bank tensors: CPU, pinned, contiguous (the library maps
    them to device addresses and rejects memory that is not pinned)."""
    for t, n in zip((a, b), names):
        if t.device.type != "cpu" or not t.is_pinned():
            raise ValueError(f"{n} must be a pinned host tensor (pin_memory=True)")
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")


def gq_nf4_grouped_gemv_host(x, codes, absmax, topk_ids, pair_scale=None, out=None):
    """Decode GEMV on NF4 experts resident in pinned host memory: codes uint8
    [E, N, K/2] and absmax float32 [E, N, K/64] are pinned CPU tensors; the
    kernel streams the routed experts' bytes over the host link.  x, topk_ids,
    pair_scale and out are device tensors.  Returns bf16 [rows*topk, N]."""
    lib = _lib or load_library()
    rows, K, xs = _x_args(x)
    _host_bank(codes, absmax, ("codes", "absmax"))
    if codes.dtype != torch.uint8 or absmax.dtype != torch.float32 or codes.dim() != 3:
        raise ValueError("codes uint8 [E, N, K/2] and absmax float32 [E, N, K/64] expected")
    E, N, half = codes.shape
    if half * 2 != K or tuple(absmax.shape) != (E, N, K // 64):
        raise ValueError("x, codes and absmax disagree on the shapes")
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    P = _gemv_pairs(topk_ids, rows)
    out = _out(out, P, N, x.device)
    st = lib.gq_nf4_grouped_gemv_host(_ptr(x), rows, K, xs, _ptr(codes), _ptr(absmax), E, N,
                                      _ptr(topk_ids), topk_ids.shape[1],
                                      _ptr(_scale(pair_scale, P)), _ptr(out), _stream(x))
    _check(st, "gq_nf4_grouped_gemv_host")
    return out


def gq_mxfp4_grouped_gemv_host(x, blocks, scales, topk_ids, pair_scale=None, out=None):
    """Decode GEMV on MXFP4 experts resident in pinned host memory (blocks
    uint8 [E, N, K/32, 16], scales uint8 [E, N, K/32], pinned CPU tensors)."""
    lib = _lib or load_library()
    rows, K, xs = _x_args(x)
    _host_bank(blocks, scales, ("blocks", "scales"))
    if blocks.dtype != torch.uint8 or scales.dtype != torch.uint8 or blocks.dim() != 4:
        raise ValueError("blocks uint8 [E, N, K/32, 16] and scales uint8 [E, N, K/32] expected")
    E, N, nb, sixteen = blocks.shape
    if sixteen != 16 or nb * 32 != K or tuple(scales.shape) != (E, N, nb):
        raise ValueError("x, blocks and scales disagree on the shapes")
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    P = _gemv_pairs(topk_ids, rows)
    out = _out(out, P, N, x.device)
    st = lib.gq_mxfp4_grouped_gemv_host(_ptr(x), rows, K, xs, _ptr(blocks), _ptr(scales), E, N,
                                        _ptr(topk_ids), topk_ids.shape[1],
                                        _ptr(_scale(pair_scale, P)), _ptr(out), _stream(x))
    _check(st, "gq_mxfp4_grouped_gemv_host")
    return out


def _route_ptrs(route):
    return (_ptr(route.expert_offsets), _ptr(route.sorted_pairs), _ptr(route.tiles),
            _ptr(route.num_tiles), route.max_tiles, route.tile_m)


def gq_nf4_grouped_gemm(x, codes, absmax, route, pair_scale=None, out=None):
    """Prefill grouped GEMM on NF4 experts using a ``gq_route_sort`` result."""
    lib = _lib or load_library()
    rows, K, xs = _x_args(x)
    E, N, Kw = _nf4_bank(codes, absmax)
    if Kw != K or route.rows != rows or route.num_experts != E:
        raise ValueError("x, codes and route disagree")
    P = rows * route.topk
    out = _out(out, P, N, x.device)
    st = lib.gq_nf4_grouped_gemm(_ptr(x), rows, K, xs, _ptr(codes), _ptr(absmax), E, N,
                                 route.topk, _ptr(_scale(pair_scale, P)), *_route_ptrs(route),
                                 _ptr(out), _stream(x))
    _check(st, "gq_nf4_grouped_gemm")
    return out


def gq_mxfp4_grouped_gemm(x, blocks, scales, route, pair_scale=None, out=None):
    """Prefill grouped GEMM on MXFP4 experts using a ``gq_route_sort`` result."""
    lib = _lib or load_library()
    rows, K, xs = _x_args(x)
    E, N, Kw = _mx_bank(blocks, scales)
    if Kw != K or route.rows != rows or route.num_experts != E:
        raise ValueError("x, blocks and route disagree")
    P = rows * route.topk
    out = _out(out, P, N, x.device)
    st = lib.gq_mxfp4_grouped_gemm(_ptr(x), rows, K, xs, _ptr(blocks), _ptr(scales), E, N,
                                   route.topk, _ptr(_scale(pair_scale, P)), *_route_ptrs(route),
                                   _ptr(out), _stream(x))
    _check(st, "gq_mxfp4_grouped_gemm")
    return out


def gq_nf4_grouped_dgrad(dy, codes, absmax, route, out=None):
    """dX = dY . W per pair through NF4 experts; ``route`` from gq_route_sort(pair ids [P, 1])."""
    lib = _lib or load_library()
    P, N, ds = _x_args(dy, "dy")
    E, Nw, K = _nf4_bank(codes, absmax)
    if Nw != N or route.rows * route.topk != P or route.topk != 1 or route.num_experts != E:
        raise ValueError("dy, codes and route disagree (route must be built with topk = 1)")
    out = _out(out, P, K, dy.device)
    st = lib.gq_nf4_grouped_dgrad(_ptr(dy), P, N, ds, _ptr(codes), _ptr(absmax), E, K,
                                  *_route_ptrs(route), _ptr(out), _stream(dy))
    _check(st, "gq_nf4_grouped_dgrad")
    return out


def gq_mxfp4_grouped_dgrad(dy, blocks, scales, route, out=None):
    """dX = dY . W per pair through MXFP4 experts; ``route`` from gq_route_sort(pair ids [P, 1])."""
    lib = _lib or load_library()
    P, N, ds = _x_args(dy, "dy")
    E, Nw, K = _mx_bank(blocks, scales)
    if Nw != N or route.rows * route.topk != P or route.topk != 1 or route.num_experts != E:
        raise ValueError("dy, blocks and route disagree (route must be built with topk = 1)")
    out = _out(out, P, K, dy.device)
    st = lib.gq_mxfp4_grouped_dgrad(_ptr(dy), P, N, ds, _ptr(blocks), _ptr(scales), E, K,
                                    *_route_ptrs(route), _ptr(out), _stream(dy))
    _check(st, "gq_mxfp4_grouped_dgrad")
    return out


# ---- MoE-layer epilogues ----------------------------------------------------
def gq_nf4_grouped_gemv_swiglu(x, codes, absmax, topk_ids, out=None):
    """Decode gate_up GEMV with SwiGLU fused: codes [E, 2I, K] (gate rows first);
    returns bf16 [rows*topk, I] = silu(gate) * up."""
    lib = _lib or load_library()
    rows, K, xs = _x_args(x)
    E, N2, Kw = _nf4_bank(codes, absmax)
    if Kw != K or N2 % 2:
        raise ValueError("x and codes disagree on K, or the gate_up width is odd")
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    P = _gemv_pairs(topk_ids, rows)
    out = _out(out, P, N2 // 2, x.device)
    st = lib.gq_nf4_grouped_gemv_swiglu(_ptr(x), rows, K, xs, _ptr(codes), _ptr(absmax), E, N2,
                                        _ptr(topk_ids), topk_ids.shape[1], _ptr(out), _stream(x))
    _check(st, "gq_nf4_grouped_gemv_swiglu")
    return out


def gq_nf4_grouped_gemm_swiglu(x, codes, absmax, route, out=None):
    """Prefill gate_up GEMM with SwiGLU fused; returns bf16 [rows*topk, I]."""
    lib = _lib or load_library()
    rows, K, xs = _x_args(x)
    E, N2, Kw = _nf4_bank(codes, absmax)
    if Kw != K or route.rows != rows or route.num_experts != E or N2 % 2:
        raise ValueError("x, codes and route disagree")
    P = rows * route.topk
    out = _out(out, P, N2 // 2, x.device)
    st = lib.gq_nf4_grouped_gemm_swiglu(_ptr(x), rows, K, xs, _ptr(codes), _ptr(absmax), E, N2,
                                        route.topk, *_route_ptrs(route), _ptr(out), _stream(x))
    _check(st, "gq_nf4_grouped_gemm_swiglu")
    return out


def _weights(topk_weights, rows, topk):
    if topk_weights is None:
        return None
    _dev(topk_weights, "topk_weights", torch.float32)
    if topk_weights.numel() != rows * topk:
        raise ValueError("topk_weights must hold rows x topk floats")
    return topk_weights


def gq_nf4_grouped_gemv_down_combine(act, codes, absmax, topk_ids, topk_weights=None, out=None):
    """Decode down GEMV with the router-weighted combine fused: act bf16 [rows*topk, I]
    (row p is pair p's input), codes [E, H, I]; returns bf16 [rows, H]."""
    lib = _lib or load_library()
    P, I, a_s = _x_args(act, "act")
    E, H, Iw = _nf4_bank(codes, absmax)
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    rows, topk = topk_ids.shape
    if Iw != I or rows * topk != P:
        raise ValueError("act, codes and topk_ids disagree")
    out = _out(out, rows, H, act.device)
    st = lib.gq_nf4_grouped_gemv_down_combine(_ptr(act), rows, I, a_s, _ptr(codes), _ptr(absmax),
                                              E, H, _ptr(topk_ids), topk,
                                              _ptr(_weights(topk_weights, rows, topk)), _ptr(out),
                                              _stream(act))
    _check(st, "gq_nf4_grouped_gemv_down_combine")
    return out


def gq_mxfp4_grouped_gemv_down_combine(act, blocks, scales, topk_ids, topk_weights=None,
                                       out=None):
    """Decode down GEMV on MXFP4 experts with the router-weighted combine fused:
    act bf16 [rows*topk, I] (row p is pair p's input), blocks [E, H, I];
    returns bf16 [rows, H]."""
    lib = _lib or load_library()
    P, I, a_s = _x_args(act, "act")
    E, H, Iw = _mx_bank(blocks, scales)
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    rows, topk = topk_ids.shape
    if Iw != I or rows * topk != P:
        raise ValueError("act, blocks and topk_ids disagree")
    out = _out(out, rows, H, act.device)
    st = lib.gq_mxfp4_grouped_gemv_down_combine(_ptr(act), rows, I, a_s, _ptr(blocks),
                                                _ptr(scales), E, H, _ptr(topk_ids), topk,
                                                _ptr(_weights(topk_weights, rows, topk)),
                                                _ptr(out), _stream(act))
    _check(st, "gq_mxfp4_grouped_gemv_down_combine")
    return out


def gq_moe_combine(y_pairs, topk, topk_weights=None, out=None):
    """y[t] = sum_s w[t, s] * y_pairs[t*topk + s] (plain sum without weights);
    y_pairs bf16 [rows*topk, H]; returns bf16 [rows, H]."""
    lib = _lib or load_library()
    P, H, ys = _x_args(y_pairs, "y_pairs")
    if P % topk:
        raise ValueError("y_pairs must hold rows*topk rows")
    rows = P // topk
    out = _out(out, rows, H, y_pairs.device)
    st = lib.gq_moe_combine(_ptr(y_pairs), rows, topk, H, ys,
                            _ptr(_weights(topk_weights, rows, topk)), _ptr(out), _stream(y_pairs))
    _check(st, "gq_moe_combine")
    return out


# ---- MXFP4 on the block-scaled fp4 matrix instruction ------------------------
def split_sizes(rows, K):
    """Byte shapes of gq_act_split_e4m3's outputs for x [rows, K]:
    (codes [rows, 2*Kp], scales [rows, Kp/16]) with Kp = K rounded up to 64."""
    kp = (K + 63) // 64 * 64
    return (rows, 2 * kp), (rows, kp // 16)


def gq_act_split_e4m3(x, codes=None, scales=None):
    """Two-term e4m3 split of bf16 activations x [rows, K]; returns the
    (codes, scales) uint8 tensors gq_mxfp4_grouped_gemm_scaled takes."""
    lib = _lib or load_library()
    rows, K, xs = _x_args(x)
    cshape, sshape = split_sizes(rows, K)
    if codes is None:
        codes = torch.empty(cshape, dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty(sshape, dtype=torch.uint8, device=x.device)
    _dev(codes, "codes", torch.uint8)
    _dev(scales, "scales", torch.uint8)
    if tuple(codes.shape) != cshape or tuple(scales.shape) != sshape:
        raise ValueError(f"split buffers must be {cshape} and {sshape}")
    st = lib.gq_act_split_e4m3(_ptr(x), rows, K, xs, _ptr(codes), _ptr(scales), _stream(x))
    _check(st, "gq_act_split_e4m3")
    return codes, scales


def gq_mxfp4_grouped_gemm_scaled(x_split, blocks, scales, route, pair_scale=None, out=None):
    """Prefill grouped GEMM on MXFP4 experts through the block-scaled fp4
    instruction; ``x_split`` = gq_act_split_e4m3(x) for x [rows, K]."""
    lib = _lib or load_library()
    xq, xsc = x_split
    _dev(xq, "x_split codes", torch.uint8, 2)
    _dev(xsc, "x_split scales", torch.uint8, 2)
    E, N, K = _mx_bank(blocks, scales)
    rows = xq.shape[0]
    cshape, sshape = split_sizes(rows, K)
    if tuple(xq.shape) != cshape or tuple(xsc.shape) != sshape:
        raise ValueError("x_split does not match the weights' K")
    if route.rows != rows or route.num_experts != E:
        raise ValueError("x_split and route disagree")
    P = rows * route.topk
    out = _out(out, P, N, xq.device)
    st = lib.gq_mxfp4_grouped_gemm_scaled(_ptr(xq), _ptr(xsc), rows, K, _ptr(blocks),
                                          _ptr(scales), E, N, route.topk,
                                          _ptr(_scale(pair_scale, P)), *_route_ptrs(route),
                                          _ptr(out), _stream(xq))
    _check(st, "gq_mxfp4_grouped_gemm_scaled")
    return out


def gq_mxfp4_grouped_gemm_scaled_swiglu(x_split, blocks, scales, route, alpha=OSS_ALPHA,
                                        limit=OSS_LIMIT, out=None):
    """Prefill gate_up GEMM on the block-scaled fp4 instruction with gpt-oss's
    gated unit in the epilogue: blocks [E, 2I, K] (gate row 2j, up row
    2j + 1); returns bf16 [rows*topk, I]."""
    lib = _lib or load_library()
    xq, xsc = x_split
    _dev(xq, "x_split codes", torch.uint8, 2)
    _dev(xsc, "x_split scales", torch.uint8, 2)
    E, N2, K = _mx_bank(blocks, scales)
    if N2 % 2:
        raise ValueError("the gate_up width is odd")
    rows = xq.shape[0]
    cshape, sshape = split_sizes(rows, K)
    if tuple(xq.shape) != cshape or tuple(xsc.shape) != sshape:
        raise ValueError("x_split does not match the weights' K")
    if route.rows != rows or route.num_experts != E:
        raise ValueError("x_split and route disagree")
    P = rows * route.topk
    out = _out(out, P, N2 // 2, xq.device)
    st = lib.gq_mxfp4_grouped_gemm_scaled_swiglu(_ptr(xq), _ptr(xsc), rows, K, _ptr(blocks),
                                                 _ptr(scales), E, N2, route.topk, float(alpha),
                                                 float(limit), *_route_ptrs(route), _ptr(out),
                                                 _stream(xq))
    _check(st, "gq_mxfp4_grouped_gemm_scaled_swiglu")
    return out


def gq_mxfp4_grouped_gemm_scaled_swiglu_split(x_split, blocks, scales, route, alpha=OSS_ALPHA,
                                              limit=OSS_LIMIT, out=None):
    """gq_mxfp4_grouped_gemm_scaled_swiglu with the [rows*topk, I] result
    written as its two-term e4m3 split (the bytes gq_act_split_e4m3 would
    write for it); returns (codes, scales), the down product's x_split.
    ``out``: an optional (codes, scales) pair of the split_sizes shapes."""
    lib = _lib or load_library()
    xq, xsc = x_split
    _dev(xq, "x_split codes", torch.uint8, 2)
    _dev(xsc, "x_split scales", torch.uint8, 2)
    E, N2, K = _mx_bank(blocks, scales)
    if N2 % 2:
        raise ValueError("the gate_up width is odd")
    rows = xq.shape[0]
    cshape, sshape = split_sizes(rows, K)
    if tuple(xq.shape) != cshape or tuple(xsc.shape) != sshape:
        raise ValueError("x_split does not match the weights' K")
    if route.rows != rows or route.num_experts != E:
        raise ValueError("x_split and route disagree")
    P = rows * route.topk
    ocs, oss = split_sizes(P, N2 // 2)
    if out is None:
        out = (torch.empty(ocs, dtype=torch.uint8, device=xq.device),
               torch.empty(oss, dtype=torch.uint8, device=xq.device))
    oq, osc = out
    _dev(oq, "out codes", torch.uint8, 2)
    _dev(osc, "out scales", torch.uint8, 2)
    if tuple(oq.shape) != ocs or tuple(osc.shape) != oss:
        raise ValueError(f"out must be uint8 {ocs} and {oss}")
    st = lib.gq_mxfp4_grouped_gemm_scaled_swiglu_split(
        _ptr(xq), _ptr(xsc), rows, K, _ptr(blocks), _ptr(scales), E, N2, route.topk,
        float(alpha), float(limit), *_route_ptrs(route), _ptr(oq), _ptr(osc), _stream(xq))
    _check(st, "gq_mxfp4_grouped_gemm_scaled_swiglu_split")
    return oq, osc


# ---- MXFP4 quantisation --------------------------------------------------------
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}    # GQ_F32, GQ_BF16, GQ_F16


def _typed(t, name):
    """Type code of a device tensor of one of the three float types."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor (got {t.device})")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16 (got {t.dtype})")
    return code


def _beside(index, *tensors):
    """Every tensor of a call lies on the device that it runs on."""
    for t in tensors:
        if t is not None and t.get_device() != index:
            raise ValueError(f"a tensor of shape {tuple(t.shape)} is on {t.device}, the call runs "
                             f"on cuda:{index}")


def _on(index, fn, what, *args):
    """Call the library on the current stream of device ``index``, with that
    device current."""
    if torch.cuda.current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st != 0:
        _check(st, what)


def _rows(t, name):
    """(rows, width, row stride) of a tensor [..., width] whose leading
    dimensions lie at one stride."""
    shape = t.shape
    if len(shape) == 2 and shape[0] > 1 and t.stride(1) == 1:
        return shape[0], shape[1], t.stride(0)
    if len(shape) < 1 or (shape[-1] > 1 and t.stride(-1) != 1):
        raise ValueError(f"{name} must have unit stride along its last dimension")
    if len(shape) != 2:
        try:
            t = t.view(-1, shape[-1]) if shape[-1] else t.reshape(0, 0)
        except RuntimeError:
            raise ValueError(f"the leading dimensions of {name} must lie at one stride") from None
    rows, width = t.shape
    return rows, width, t.stride(0) if rows > 1 else width


def gq_mxfp4_quantize(x, values=None, blocks=None, scales=None):
    """MXFP4 of x [..., K] (float32, bfloat16 or float16, any row stride):
    returns (blocks uint8 [..., K/32, 16], scales uint8 [..., K/32]), the
    layout that the MXFP4 entry points take.  ``values``: True or a bf16
    tensor of x's shape (x itself, if bf16 and contiguous) also returns the
    values that the codes stand for."""
    lib = _lib or load_library()
    if _calls and blocks is scales is None and (values is None or values is True):
        r = _calls.quantize(x, values is True)
        if r is not None:
            return _done(r, "gq_mxfp4_quantize")
    code = _typed(x, "x")
    dev, index = x.device, x.get_device()
    rows, K, stride = _rows(x, "x")
    nb = K // 32
    lead = (rows,) if x.dim() == 2 else tuple(x.shape[:-1])
    bshape, sshape = (*lead, nb, 16), (*lead, nb)
    if blocks is None:
        blocks = torch.empty(bshape, dtype=torch.uint8, device=dev)
    elif tuple(_dev(blocks, "blocks", torch.uint8).shape) != bshape:
        raise ValueError(f"blocks must be {bshape}")
    if scales is None:
        scales = torch.empty(sshape, dtype=torch.uint8, device=dev)
    elif tuple(_dev(scales, "scales", torch.uint8).shape) != sshape:
        raise ValueError(f"scales must be {sshape}")
    if values is True:
        values = torch.empty(x.shape, dtype=torch.bfloat16, device=dev)
    elif values is False:
        values = None
    elif values is not None and _dev(values, "values", torch.bfloat16).shape != x.shape:
        raise ValueError("values must have x's shape")
    _beside(index, blocks, scales, values)
    if K >= 1 << 31 and stride == K and K % 32 == 0:
        # one long run of blocks, as any number of rows of one block
        rows, K, stride = rows * nb, 32, 32
    _ints("gq_mxfp4_quantize", K)
    _on(index, lib.gq_mxfp4_quantize, "gq_mxfp4_quantize", x.data_ptr(), code, rows, K, stride,
        blocks.data_ptr(), scales.data_ptr(), None if values is None else values.data_ptr())
    return (blocks, scales) if values is None else (blocks, scales, values)


def _like(t, name, dtype, shape, dev):
    """An output: a new tensor where ``t`` is None or True, else ``t`` checked."""
    if t is None or t is True:
        return torch.empty(shape, dtype=dtype, device=dev)
    if _dev(t, name, dtype).shape != shape:
        raise ValueError(f"{name} must be {tuple(shape)}")
    return t


def gq_mxfp8_quantize(x, values=None, codes=None, scales=None):
    """MXFP8 of x [..., K] (float32, bfloat16 or float16, any row stride):
    returns (codes uint8 [..., K], OCP e4m3 in element order, scales uint8
    [..., K/32]), the layout that the _fp8 entry points take.  ``values``: True
    or a bf16 tensor of x's shape (x itself, if bf16 and contiguous) also
    returns the values that the codes stand for."""
    lib = _lib or load_library()
    if _calls and codes is scales is None and (values is None or values is True):
        r = _calls.quantize8(x, values is True)
        if r is not None:
            return _done(r, "gq_mxfp8_quantize")
    code = _typed(x, "x")
    dev, index = x.device, x.get_device()
    rows, K, stride = _rows(x, "x")
    codes = _like(codes, "codes", torch.uint8, x.shape, dev)
    scales = _like(scales, "scales", torch.uint8, torch.Size((*x.shape[:-1], K // 32)), dev)
    values = None if values is False or values is None else _like(values, "values", torch.bfloat16,
                                                                  x.shape, dev)
    _beside(index, codes, scales, values)
    if K >= 1 << 31 and stride == K and K % 32 == 0:
        # one long run of blocks, as any number of rows of one block
        rows, K, stride = rows * (K // 32), 32, 32
    _ints("gq_mxfp8_quantize", K)
    _on(index, lib.gq_mxfp8_quantize, "gq_mxfp8_quantize", x.data_ptr(), code, rows, K, stride,
        codes.data_ptr(), scales.data_ptr(), None if values is None else values.data_ptr())
    return (codes, scales) if values is None else (codes, scales, values)


# ---- root-mean-square norm ---------------------------------------------------------
RmsNorm = namedtuple("RmsNorm", "y residual mxfp8 values")


def _gain(weight, x, H):
    """Type code of a norm's weight."""
    code = _typed(weight, "weight")
    if weight.shape != (H,) or not weight.is_contiguous():
        raise ValueError(f"weight must be [{H}] and contiguous (got shape {tuple(weight.shape)})")
    if weight.dtype not in (x.dtype, torch.float32):
        raise ValueError(f"weight must be {x.dtype} or float32 (got {weight.dtype})")
    return code


def _same_rows(t, like, name):
    """Row stride of a tensor that has the shape and type of another."""
    _typed(t, name)
    if t.shape != like.shape or t.dtype != like.dtype:
        raise ValueError(f"{name} must be {like.dtype} {tuple(like.shape)} "
                         f"(got {t.dtype} {tuple(t.shape)})")
    return _rows(t, name)[2]


def gq_rms_norm(x, weight, eps=1e-6, residual=None, y=True, sum=None, mxfp8=False, values=False):
    """h = x + ``residual`` (rounded to x's type; h = x without one) and its
    root-mean-square norm y = h / sqrt(mean(h^2) + eps) * weight, over the last
    dimension of x [..., H] (float32, bfloat16 or float16; x and residual at any
    row stride).  ``weight`` [H] is of x's type or float32.

    Returns RmsNorm(y, residual, mxfp8, values): y of x's type (None with
    ``y=False``); h, the new residual stream (None where no residual was given);
    with ``mxfp8=True`` the pair (codes uint8 [..., H], scales uint8 [..., H/32])
    of the unrounded y, as gq_mxfp8_quantize lays it out, and with
    ``values=True`` also the bf16 values that the codes stand for.  ``y`` and
    ``sum`` (for h) may be tensors to write to, x or residual among them;
    ``mxfp8`` a pair of tensors and ``values`` a tensor likewise."""
    lib = _lib or load_library()
    if (_calls and y is True and sum is None and (mxfp8 is False or mxfp8 is True)
            and (values is False or values is True)):
        r = _calls.rms_norm(x, weight, eps, residual, mxfp8, values)
        if r is not None:
            y, sum, codes, scales, values = _done(r, "gq_rms_norm")
            return RmsNorm(y, sum, None if codes is None else (codes, scales), values)
    code = _typed(x, "x")
    dev, index = x.device, x.get_device()
    rows, H, stride = _rows(x, "x")
    wcode = _gain(weight, x, H)
    rstride = 0
    if residual is not None:
        rstride = _same_rows(residual, x, "residual")
        sum = _like(sum, "sum", x.dtype, x.shape, dev)
    elif sum is not None:
        raise ValueError("sum goes with a residual")
    y = None if y is False or y is None else _like(y, "y", x.dtype, x.shape, dev)
    codes = scales = None
    if mxfp8 is not False and mxfp8 is not None:
        if H % 32:
            raise ValueError(f"mxfp8 takes rows of whole blocks of 32 (got {H})")
        codes, scales = (None, None) if mxfp8 is True else mxfp8
        codes = _like(codes, "mxfp8 codes", torch.uint8, x.shape, dev)
        scales = _like(scales, "mxfp8 scales", torch.uint8, torch.Size((*x.shape[:-1], H // 32)),
                       dev)
    values = None if values is False or values is None else _like(values, "values", torch.bfloat16,
                                                                  x.shape, dev)
    if values is not None and codes is None:
        raise ValueError("values goes with mxfp8")
    _beside(index, weight, residual, sum, y, codes, scales, values)
    _ints("gq_rms_norm", H)
    _on(index, lib.gq_rms_norm, "gq_rms_norm", x.data_ptr(), stride, _ptr(residual), rstride, code,
        rows, H, weight.data_ptr(), wcode, float(eps), _ptr(sum), _ptr(y), _ptr(codes),
        _ptr(scales), _ptr(values))
    return RmsNorm(y, sum, None if codes is None else (codes, scales), values)


def gq_rms_norm_backward_workspace(rows, H):
    """Bytes of workspace for gq_rms_norm_backward of up to ``rows`` rows; -1 where it does
    not take the sizes."""
    if not 0 <= rows < 1 << 63 or not 0 <= H < 1 << 31:
        return -1
    return int(load_library().gq_rms_norm_backward_workspace(rows, H))


def gq_rms_norm_backward(d_y, h, weight, eps=1e-6, d_residual=None, d_x=None, d_weight=True,
                         workspace=None):
    """Gradients of gq_rms_norm: (d_x, d_weight) from d_y and h [..., H], the
    forward's residual sum (its x, where there was no residual), of one type.
    ``d_residual``: the gradient that reaches h by another way; d_x, the gradient
    of x and of residual alike, includes it.  d_weight [H] is of weight's type;
    ``d_weight=False`` leaves it out (None).  ``d_x`` and ``d_weight`` may be
    tensors to write to (d_x: d_y, h or d_residual among them); ``workspace``: a
    uint8 tensor of at least gq_rms_norm_backward_workspace bytes."""
    lib = _lib or load_library()
    if _calls and d_x is workspace is None and (d_weight is True or d_weight is False):
        r = _calls.rms_norm_backward(d_y, h, weight, eps, d_residual, d_weight)
        if r is not None:
            return _done(r, "gq_rms_norm_backward")
    code = _typed(h, "h")
    dev, index = h.device, h.get_device()
    rows, H, stride = _rows(h, "h")
    wcode = _gain(weight, h, H)
    dstride = _same_rows(d_y, h, "d_y")
    rstride = 0 if d_residual is None else _same_rows(d_residual, h, "d_residual")
    d_x = _like(d_x, "d_x", h.dtype, h.shape, dev)
    d_weight = None if d_weight is False or d_weight is None else _like(
        d_weight, "d_weight", weight.dtype, weight.shape, dev)
    if d_weight is None:
        workspace = None
    elif workspace is None:
        need = gq_rms_norm_backward_workspace(rows, H)
        workspace = torch.empty(need, dtype=torch.uint8, device=dev) if need > 0 else None
    else:
        _dev(workspace, "workspace", torch.uint8)
    _beside(index, weight, d_y, d_residual, d_x, d_weight, workspace)
    _ints("gq_rms_norm_backward", H)
    _on(index, lib.gq_rms_norm_backward, "gq_rms_norm_backward", d_y.data_ptr(), dstride,
        h.data_ptr(), stride, _ptr(d_residual), rstride, code, rows, H, weight.data_ptr(), wcode,
        float(eps), d_x.data_ptr(), _ptr(d_weight), _ptr(workspace),
        0 if workspace is None else workspace.numel())
    return d_x, d_weight


# ---- MXFP4 or MXFP8 x MXFP4 products ------------------------------------------------
def _mx_pair(x, bits, blocks, scales, unit):
    """Checks of a product of MXFP4 or MXFP8 activations with MXFP4 experts: (x
    codes, x scales, rows, E, N, K)."""
    xb, xs = x[0], x[1]
    _dev(xb, "x blocks" if bits == 4 else "x codes", torch.uint8, 3 if bits == 4 else 2)
    _dev(xs, "x scales", torch.uint8, 2)
    E, N, K = _mx_bank(blocks, scales)
    rows, nb = xb.shape[0], K // 32
    if bits == 4 and (xb.shape != (rows, nb, 16) or xs.shape != (rows, nb)):
        raise ValueError(f"x must be (blocks [rows, {nb}, 16], scales [rows, {nb}]) as "
                         "gq_mxfp4_quantize returns them")
    if bits == 8 and (xb.shape != (rows, K) or xs.shape != (rows, nb)):
        raise ValueError(f"x must be (codes [rows, {K}], scales [rows, {nb}]) as "
                         "gq_mxfp8_quantize returns them")
    if unit and N % 2:
        raise ValueError("the gate_up width is odd")
    _beside(xb.get_device(), xs, blocks, scales)
    return xb, xs, rows, E, N, K


def _mx_gemm(what, bits, x, blocks, scales, route, unit, pair_scale, out):
    lib = _lib or load_library()
    if _calls and out is None:
        r = (_calls.fp4_gemm if bits == 4 else _calls.fp8_gemm)(
            x[0], x[1], blocks, scales, route, pair_scale, unit is not None, *(unit or (0.0, 0.0)))
        if r is not None:
            return _done(r, what)
    xb, xs, rows, E, N, K = _mx_pair(x, bits, blocks, scales, unit is not None)
    if route.rows != rows or route.num_experts != E:
        raise ValueError("x, blocks and route disagree")
    index = xb.get_device()
    P = rows * route.topk
    for name, least in (("expert_offsets", E + 1), ("sorted_pairs", P),
                        ("tiles", 2 * route.max_tiles), ("num_tiles", 1)):
        if _dev(getattr(route, name), "route." + name, torch.int32).numel() < least:
            raise ValueError(f"route.{name} is too short for the route's sizes")
    out = _out(out, P, N // 2 if unit else N, xb.device)
    _beside(index, out, pair_scale, route.expert_offsets, route.sorted_pairs, route.tiles,
            route.num_tiles)
    middle = unit or (_ptr(_scale(pair_scale, P)),)
    _ints(what, rows, K, E, N, route.topk, route.max_tiles, route.tile_m)
    _on(index, getattr(lib, what), what, xb.data_ptr(), xs.data_ptr(), rows, K, blocks.data_ptr(),
        scales.data_ptr(), E, N, route.topk, *middle, *_route_ptrs(route), out.data_ptr())
    return out


def gq_mxfp4_grouped_gemm_fp4(x, blocks, scales, route, pair_scale=None, out=None):
    """Prefill grouped GEMM of MXFP4 activations with MXFP4 experts; ``x`` =
    gq_mxfp4_quantize(activations [rows, K]).  Returns bf16 [rows*topk, N]."""
    return _mx_gemm("gq_mxfp4_grouped_gemm_fp4", 4, x, blocks, scales, route, None, pair_scale, out)


def gq_mxfp4_grouped_gemm_fp4_swiglu(x, blocks, scales, route, alpha=OSS_ALPHA, limit=OSS_LIMIT,
                                     out=None):
    """gq_mxfp4_grouped_gemm_fp4 on gate_up experts [E, 2I, K] (gate row 2j,
    up row 2j + 1) with gpt-oss's gated unit: bf16 [rows*topk, I]."""
    return _mx_gemm("gq_mxfp4_grouped_gemm_fp4_swiglu", 4, x, blocks, scales, route,
                     (float(alpha), float(limit)), None, out)


def _mx_gemv(what, bits, x, blocks, scales, topk_ids, unit, pair_scale, out):
    lib = _lib or load_library()
    if _calls and out is None:
        r = (_calls.fp4_gemv if bits == 4 else _calls.fp8_gemv)(
            x[0], x[1], blocks, scales, topk_ids, pair_scale, unit is not None,
            *(unit or (0.0, 0.0)))
        if r is not None:
            return _done(r, what)
    xb, xs, rows, E, N, K = _mx_pair(x, bits, blocks, scales, unit is not None)
    index = xb.get_device()
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    P = _gemv_pairs(topk_ids, rows)
    out = _out(out, P, N // 2 if unit else N, xb.device)
    _beside(index, out, pair_scale, topk_ids)
    middle = unit or (_ptr(_scale(pair_scale, P)),)
    _ints(what, rows, K, E, N, topk_ids.shape[1])
    _on(index, getattr(lib, what), what, xb.data_ptr(), xs.data_ptr(), rows, K, blocks.data_ptr(),
        scales.data_ptr(), E, N, topk_ids.data_ptr(), topk_ids.shape[1], *middle, out.data_ptr())
    return out


def gq_mxfp4_grouped_gemv_fp4(x, blocks, scales, topk_ids, pair_scale=None, out=None):
    """Decode-time product (<= 256 pairs) of MXFP4 activations with MXFP4
    experts; ``x`` = gq_mxfp4_quantize(activations).  Returns bf16 [rows*topk, N]."""
    return _mx_gemv("gq_mxfp4_grouped_gemv_fp4", 4, x, blocks, scales, topk_ids, None, pair_scale,
                     out)


def gq_mxfp4_grouped_gemv_fp4_swiglu(x, blocks, scales, topk_ids, alpha=OSS_ALPHA,
                                     limit=OSS_LIMIT, out=None):
    """gq_mxfp4_grouped_gemv_fp4 on gate_up experts with gpt-oss's gated unit:
    bf16 [rows*topk, I]."""
    return _mx_gemv("gq_mxfp4_grouped_gemv_fp4_swiglu", 4, x, blocks, scales, topk_ids,
                     (float(alpha), float(limit)), None, out)


def gq_mxfp4_grouped_gemm_fp8(x, blocks, scales, route, pair_scale=None, out=None):
    """Prefill grouped GEMM of MXFP8 activations with MXFP4 experts; ``x`` =
    gq_mxfp8_quantize(activations [rows, K]) or gq_rms_norm's ``mxfp8``.
    Returns bf16 [rows*topk, N].  The matrix instruction cuts products far below
    (2^-13) the largest of eight neighbours; gq_mxfp4_grouped_gemv_fp8 does not."""
    return _mx_gemm("gq_mxfp4_grouped_gemm_fp8", 8, x, blocks, scales, route, None, pair_scale, out)


def gq_mxfp4_grouped_gemm_fp8_swiglu(x, blocks, scales, route, alpha=OSS_ALPHA, limit=OSS_LIMIT,
                                     out=None):
    """gq_mxfp4_grouped_gemm_fp8 on gate_up experts [E, 2I, K] (gate row 2j,
    up row 2j + 1) with gpt-oss's gated unit: bf16 [rows*topk, I]."""
    return _mx_gemm("gq_mxfp4_grouped_gemm_fp8_swiglu", 8, x, blocks, scales, route,
                    (float(alpha), float(limit)), None, out)


def gq_mxfp4_grouped_gemv_fp8(x, blocks, scales, topk_ids, pair_scale=None, out=None):
    """Decode-time product (<= 256 pairs) of MXFP8 activations with MXFP4
    experts; ``x`` = gq_mxfp8_quantize(activations).  Returns bf16 [rows*topk, N]."""
    return _mx_gemv("gq_mxfp4_grouped_gemv_fp8", 8, x, blocks, scales, topk_ids, None, pair_scale,
                    out)


def gq_mxfp4_grouped_gemv_fp8_swiglu(x, blocks, scales, topk_ids, alpha=OSS_ALPHA,
                                     limit=OSS_LIMIT, out=None):
    """gq_mxfp4_grouped_gemv_fp8 on gate_up experts with gpt-oss's gated unit:
    bf16 [rows*topk, I]."""
    return _mx_gemv("gq_mxfp4_grouped_gemv_fp8_swiglu", 8, x, blocks, scales, topk_ids,
                    (float(alpha), float(limit)), None, out)


# ---- expert routing --------------------------------------------------------------
def gq_moe_topk(logits, topk, renormalize=True, topk_ids=None, topk_weights=None):
    """The ``topk`` largest logits [rows, E] (float32, bfloat16 or float16) of
    each row, largest first, equal ones by lower index: (topk_ids int32 [rows,
    topk], topk_weights float32 [rows, topk]), the weights a softmax over the
    chosen logits (``renormalize``) or over all.  A logit of -inf is never
    chosen; a slot left without an expert has id -1 and weight 0."""
    lib = _lib or load_library()
    if _calls and topk_ids is topk_weights is None:
        r = _calls.moe_topk(logits, topk, bool(renormalize))
        if r is not None:
            return _done(r, "gq_moe_topk")
    code = _typed(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [rows, E] (got shape {tuple(logits.shape)})")
    rows, E, stride = _rows(logits, "logits")
    dev, index, topk = logits.device, logits.get_device(), int(topk)
    if topk < 1:
        raise ValueError("topk must be at least 1")
    _ints("gq_moe_topk", E, topk)
    shape = (rows, topk)
    if topk_ids is None:
        topk_ids = torch.empty(shape, dtype=torch.int32, device=dev)
    elif tuple(_dev(topk_ids, "topk_ids", torch.int32).shape) != shape:
        raise ValueError(f"topk_ids must be {shape}")
    if topk_weights is None:
        topk_weights = torch.empty(shape, dtype=torch.float32, device=dev)
    elif tuple(_dev(topk_weights, "topk_weights", torch.float32).shape) != shape:
        raise ValueError(f"topk_weights must be {shape}")
    _beside(index, topk_ids, topk_weights)
    _on(index, lib.gq_moe_topk, "gq_moe_topk", logits.data_ptr(), code, rows, E, stride, topk,
        1 if renormalize else 0, topk_ids.data_ptr(), topk_weights.data_ptr())
    return topk_ids, topk_weights


def gq_moe_topk_backward(d_weights, logits, topk_ids, renormalize=True, out=None):
    """Gradient of ``gq_moe_topk``'s weights to its logits, the selection held
    fixed: d_weights float32 [rows, topk] -> [rows, E] of the logits' type."""
    lib = _lib or load_library()
    if _calls and out is None:
        r = _calls.moe_topk_backward(d_weights, logits, topk_ids, bool(renormalize))
        if r is not None:
            return _done(r, "gq_moe_topk_backward")
    code = _typed(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [rows, E] (got shape {tuple(logits.shape)})")
    rows, E, stride = _rows(logits, "logits")
    dev, index = logits.device, logits.get_device()
    _dev(d_weights, "d_weights", torch.float32, 2)
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    if topk_ids.shape[0] != rows or d_weights.shape != topk_ids.shape:
        raise ValueError("d_weights and topk_ids must both be [rows, topk]")
    _ints("gq_moe_topk_backward", E, topk_ids.shape[1])
    if out is None:
        out = torch.empty((rows, E), dtype=logits.dtype, device=dev)
    elif tuple(_dev(out, "out", logits.dtype).shape) != (rows, E):
        raise ValueError("out must be [rows, E]")
    _beside(index, d_weights, topk_ids, out)
    _on(index, lib.gq_moe_topk_backward, "gq_moe_topk_backward", d_weights.data_ptr(),
        logits.data_ptr(), code, rows, E, stride, topk_ids.data_ptr(), topk_ids.shape[1],
        1 if renormalize else 0, out.data_ptr())
    return out


_SCORES = {"softmax": 0, "sigmoid": 1}


def _score(score):
    code = _SCORES.get(score)
    if code is None:
        raise ValueError(f"score must be 'softmax' or 'sigmoid' (got {score!r})")
    return code


def gq_moe_route(logits, topk, score="softmax", bias=None, groups=1, topk_groups=None, group_top=1,
                 renormalize=True, scale=1.0, topk_ids=None, topk_weights=None):
    """Routing with groups: the ``topk`` experts of largest choice score + ``bias``
    among the ``topk_groups`` (all when None) best of ``groups`` groups of
    neighbouring experts, for logits [rows, E] (float32, bfloat16 or float16).
    ``score``: "softmax" or "sigmoid" of the logits; ``bias`` float32 [E] only
    enters the choice; a group counts as the sum of its ``group_top`` (1 or 2)
    largest choices.  Returns (topk_ids int32 [rows, topk], topk_weights float32
    [rows, topk]), the weights ``scale`` times the chosen scores, divided by their
    sum with ``renormalize``.  Ties go to the lower index; a logit of -inf is never
    chosen; a slot left without an expert has id -1 and weight 0."""
    lib = _lib or load_library()
    if _calls and topk_ids is topk_weights is None:
        r = _calls.moe_route(logits, topk, _score(score), bias, groups,
                             groups if topk_groups is None else topk_groups, group_top,
                             bool(renormalize), scale)
        if r is not None:
            return _done(r, "gq_moe_route")
    code = _typed(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [rows, E] (got shape {tuple(logits.shape)})")
    rows, E, stride = _rows(logits, "logits")
    dev, index, topk, groups = logits.device, logits.get_device(), int(topk), int(groups)
    kind = _score(score)
    if topk < 1:
        raise ValueError("topk must be at least 1")
    if groups < 1 or E % groups:
        raise ValueError(f"groups must divide the {E} experts (got {groups})")
    topk_groups = groups if topk_groups is None else int(topk_groups)
    if bias is not None and _dev(bias, "bias", torch.float32).shape != (E,):
        raise ValueError(f"bias must be [{E}]")
    _ints("gq_moe_route", E, topk, groups, topk_groups, int(group_top))
    shape = torch.Size((rows, topk))
    topk_ids = _like(topk_ids, "topk_ids", torch.int32, shape, dev)
    topk_weights = _like(topk_weights, "topk_weights", torch.float32, shape, dev)
    _beside(index, bias, topk_ids, topk_weights)
    _on(index, lib.gq_moe_route, "gq_moe_route", logits.data_ptr(), code, rows, E, stride,
        _ptr(bias), topk, kind, groups, topk_groups, int(group_top), 1 if renormalize else 0,
        float(scale), topk_ids.data_ptr(), topk_weights.data_ptr())
    return topk_ids, topk_weights


def gq_moe_route_backward(d_weights, logits, topk_ids, score="softmax", renormalize=True,
                          scale=1.0, out=None):
    """Gradient of ``gq_moe_route``'s weights to its logits, the selection held
    fixed: d_weights float32 [rows, topk] -> [rows, E] of the logits' type."""
    lib = _lib or load_library()
    if _calls and out is None:
        r = _calls.moe_route_backward(d_weights, logits, topk_ids, _score(score),
                                      bool(renormalize), scale)
        if r is not None:
            return _done(r, "gq_moe_route_backward")
    code = _typed(logits, "logits")
    if logits.dim() != 2:
        raise ValueError(f"logits must be [rows, E] (got shape {tuple(logits.shape)})")
    rows, E, stride = _rows(logits, "logits")
    kind = _score(score)
    _dev(d_weights, "d_weights", torch.float32, 2)
    _dev(topk_ids, "topk_ids", torch.int32, 2)
    if topk_ids.shape[0] != rows or d_weights.shape != topk_ids.shape:
        raise ValueError("d_weights and topk_ids must both be [rows, topk]")
    _ints("gq_moe_route_backward", E, topk_ids.shape[1])
    out = _like(out, "out", logits.dtype, torch.Size((rows, E)), logits.device)
    index = logits.get_device()
    _beside(index, d_weights, topk_ids, out)
    _on(index, lib.gq_moe_route_backward, "gq_moe_route_backward", d_weights.data_ptr(),
        logits.data_ptr(), code, rows, E, stride, topk_ids.data_ptr(), topk_ids.shape[1], kind,
        1 if renormalize else 0, float(scale), out.data_ptr())
    return out


# ---- a whole layer for a few tokens ------------------------------------------------
class _LayerStruct(ctypes.Structure):
    """gq_moe_layer of include/gq.h."""
    _fields_ = ([(n, _i32) for n in ("format", "num_experts", "topk", "hidden", "inner",
                                     "renormalize")]
                + [("alpha", _f32), ("limit", _f32)]
                + [(n, _p) for n in ("router_weight", "router_bias", "gate_up_codes",
                                     "gate_up_scales", "gate_up_bias", "down_codes",
                                     "down_scales", "down_bias")])


class MoeLayer:
    """A layer's checked weights, made by ``gq_moe_layer``; keeps its tensors."""

    def __init__(self, struct, tensors, device):
        self._struct, self.device = struct, device
        # tensors of its own over the same memory: the struct holds addresses, and
        # a caller's tensor that is given other memory (`.data = `, Module.to)
        # would free what they name
        self._tensors = tuple(None if t is None else t.detach() for t in tensors)
        self._ref = ctypes.addressof(struct)
        self.hidden, self.topk = struct.hidden, struct.topk
        self._bytes = {}                         # workspace bytes by token count


def gq_moe_layer(router_weight, gate_up, down, topk, router_bias=None, gate_up_bias=None,
                 down_bias=None, renormalize=True, alpha=OSS_ALPHA, limit=OSS_LIMIT):
    """The weights of one mixture-of-experts layer, for ``gq_moe_decode``.

    ``router_weight`` bf16 [E, H]; ``gate_up`` and ``down`` are (codes, absmax)
    of NF4 experts [E, 2I, H] and [E, H, I] (SwiGLU, gate rows first) or
    (blocks, scales) of MXFP4 experts (the clamped unit, gate and up rows
    interleaved); the optional biases are bf16 [E], [E, 2I] and [E, H].  The
    layer refers to the memory that these tensors have now and keeps it: what is
    written into it later counts, memory that a tensor is given later (``.data =``,
    ``Module.to``) needs a new layer.  The memory itself must not be resized."""
    load_library()
    _dev(router_weight, "router_weight", torch.bfloat16, 2)
    E, H = router_weight.shape
    dev = router_weight.device
    mx = isinstance(gate_up[0], torch.Tensor) and gate_up[0].dim() == 4
    bank = _mx_bank if mx else _nf4_bank
    Eg, N, K = bank(*gate_up)
    Ed, Hd, inner = bank(*down)
    if (Eg, Ed, K, Hd, N) != (E, E, H, H, 2 * inner):
        raise ValueError(f"router [{E}, {H}], gate_up [{Eg}, {N}, {K}] and down [{Ed}, {Hd}, "
                         f"{inner}] are not one layer's")
    for name, b, shape in (("router_bias", router_bias, (E,)),
                           ("gate_up_bias", gate_up_bias, (E, N)), ("down_bias", down_bias, (E, H))):
        if b is not None and tuple(_dev(b, name, torch.bfloat16).shape) != shape:
            raise ValueError(f"{name} must be {shape}")
    tensors = (router_weight, router_bias, *gate_up, gate_up_bias, *down, down_bias)
    _beside(dev.index, *tensors)
    _ints("gq_moe_layer", E, int(topk), H, inner)
    ptr = [None if t is None else t.data_ptr() for t in tensors]
    struct = _LayerStruct(1 if mx else 0, E, int(topk), H, inner, 1 if renormalize else 0,
                          float(alpha), float(limit), *ptr)
    layer = MoeLayer(struct, tensors, dev)
    if gq_moe_decode_workspace(layer, 0) < 0:
        raise GQError(f"gq_moe_layer: not supported (E {E}, topk {topk}, H {H}, I {inner}, "
                      f"alpha {alpha}, limit {limit})", 1)
    return layer


def gq_moe_decode_workspace(layer, rows):
    """Bytes of workspace for ``rows`` tokens; -1 where gq_moe_decode does not take them."""
    if not 0 <= rows < 1 << 31:
        return -1
    return int(load_library().gq_moe_decode_workspace(layer._ref, rows))


def gq_moe_decode(layer, x, out=None, workspace=None):
    """The whole layer for x bf16 [rows, H], at most 8 tokens and 64 (token,
    expert) pairs: bf16 [rows, H].  ``workspace``: a uint8 tensor of at least
    gq_moe_decode_workspace bytes (allocated when None)."""
    lib = _lib or load_library()
    if _calls and out is workspace is None and isinstance(x, torch.Tensor) and x.dim() == 2:
        need = layer._bytes.get(x.shape[0])
        if need:
            r = _calls.moe_decode(layer._ref, layer.device.index, need, x)
            if r is not None:
                return _done(r, "gq_moe_decode")
    rows, H, stride = _x_args(x)
    dev = x.device
    if H != layer.hidden:
        raise ValueError(f"x must be [rows, {layer.hidden}]")
    need = layer._bytes.get(rows)
    if need is None:
        need = layer._bytes[rows] = gq_moe_decode_workspace(layer, rows)
    if need < 0:
        raise GQError(f"gq_moe_decode: {rows} tokens of {layer.topk} experts are not supported "
                      "(at most 8 tokens and 64 pairs)", 801)
    if out is None:
        out = torch.empty((rows, H), dtype=torch.bfloat16, device=dev)
    elif tuple(_dev(out, "out", torch.bfloat16).shape) != (rows, H):
        raise ValueError(f"out must be [{rows}, {H}]")
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _dev(workspace, "workspace", torch.uint8)
    index = layer.device.index
    _beside(index, x, out, workspace)
    _on(index, lib.gq_moe_decode, "gq_moe_decode", layer._ref, x.data_ptr(), rows,
        stride if rows > 1 else H, workspace.data_ptr(), workspace.numel(), out.data_ptr())
    return out
