"""ctypes binding of libmoe_nvfp4.so (include/moe_nvfp4.h): the same entry
points, argument marshalling only. Tensors are torch device tensors (PyTorch
provides device memory and streams); every computation runs in the library's
HIP kernels. There is no fallback: without the built library, or on a failed
call, this raises.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_nvfp4.so")

MOE_OK, MOE_EINVAL, MOE_EUNSUPPORTED, MOE_ELAUNCH = 0, -1, -2, -3
MOE_MX_E2M1, MOE_MX_E4M3 = 0, 1     # MX element formats
MOE_BF16, MOE_F32 = 0, 1            # element types of rows and outputs

# Every symbol include/moe_nvfp4.h declares.
EXPORTS = ("moe_abi_version", "moe_last_error", "moe_rows_max", "moe_meta_layout_get",
           "moe_route", "nvfp4_quant", "moe_route_quant", "moe_pack_w13", "moe_pack_w2",
           "moe_experts_fwd", "moe_finalize", "nvfp4_norm_quant", "moe_router_logits",
           "moe_router_route", "moe_experts_fwd_w4a16", "moe_experts_fwd_bf16",
           "moe_validate_weights", "moe_workspace_bytes", "moe_experts_fwd_noalloc",
           "moe_experts_finalize", "mx_quant", "mx_dequant", "mx_add_norm_quant", "mx_gemm",
           "moe_dispatch", "moe_dispatch_bwd", "moe_combine", "moe_combine_bwd")


class MoeMetaLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "num_tiles", "total_rows", "expert_offsets", "expert_counts", "exp2perm", "perm2tok",
        "tile_expert", "total_ints", "rows_max", "tiles_max", "sync_status", "sub_sync", "subs_max", "perm_counts",
        "tok_sync", "fin_part", "queue")]


class MoeNvfp4Weights(ctypes.Structure):
    _fields_ = [("w13", ctypes.c_void_p), ("w13_sf", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("w2_sf", ctypes.c_void_p)] + \
               [(n, ctypes.c_int64) for n in (
                   "w13_expert_stride_bytes", "w13_pair_stride_bytes",
                   "w13_sf_expert_stride_bytes", "w13_sf_pair_stride_bytes",
                   "w2_expert_stride_bytes", "w2_pair_stride_bytes",
                   "w2_sf_expert_stride_bytes", "w2_sf_pair_stride_bytes")] + \
               [("g1_alphas", ctypes.c_void_p), ("g1_scale_c", ctypes.c_void_p),
                ("g2_alphas", ctypes.c_void_p)]


class MoeWorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int64) for n in (
        "meta", "topk_ids", "topk_weights", "a_codes", "a_sf", "inter_codes", "inter_sf", "rows",
        "total_bytes")]


class MoeError(RuntimeError):
    pass


_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise ImportError(f"{_LIB_PATH} is not built: run python -m nvfp4_block_scaled_route_amd.build")
    L = ctypes.CDLL(_LIB_PATH)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    sig = {
        "moe_abi_version": (i32, []),
        "moe_last_error": (ctypes.c_char_p, []),
        "moe_rows_max": (i64, [i32, i32, i32, i32]),
        "moe_meta_layout_get": (i32, [i32, i32, i32, i32, ctypes.POINTER(MoeMetaLayout)]),
        "moe_route": (i32, [vp, i64, vp, vp, i32, i32, i32, f32, i32, i32, i32, vp, vp, vp, vp]),
        "nvfp4_quant": (i32, [vp, i64, vp, i32, i32, vp, vp, vp]),
        "nvfp4_norm_quant": (i32, [vp, i64, vp, f32, f32, vp, i32, i32, vp, vp, vp]),
        "moe_router_logits": (i32, [vp, i64, vp, i32, i32, i32, vp, vp]),
        "moe_experts_fwd_bf16": (i32, [vp, i64, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp, i64, vp]),
        "moe_experts_fwd_w4a16": (i32, [vp, i64, vp, ctypes.POINTER(MoeNvfp4Weights), i32, i32, i32, i32,
                                        i32, i32, vp, vp, i64, vp]),
        "moe_router_route": (i32, [vp, i64, vp, i32, vp, vp, i32, i32, i32, f32, i32, i32, i32, vp, vp,
                                   vp, vp, vp]),
        "moe_route_quant": (i32, [vp, i64, vp, vp, i32, i32, i32, f32, i32, i32, i32, vp, vp, vp,
                                  vp, i64, vp, i32, vp, vp, vp]),
        "moe_pack_w13": (i32, [vp, vp, i32, i32, i32, vp, vp, vp]),
        "moe_pack_w2": (i32, [vp, vp, i32, i32, i32, vp, vp, vp]),
        "moe_experts_fwd": (i32, [vp, vp, vp, ctypes.POINTER(MoeNvfp4Weights), i32, i32, i32,
                                  i32, i32, i32, vp, vp, vp, i64, vp]),
        "moe_finalize": (i32, [vp, i64, i32, i64, vp, vp, vp, f32, f32, i32, i32, i32, i32, vp, vp]),
        "moe_experts_fwd_noalloc": (i32, [vp, vp, vp, ctypes.POINTER(MoeNvfp4Weights), i32, i32, i32,
                                          i32, i32, i32, vp, i64, vp]),
        "moe_experts_finalize": (i32, [vp, vp, vp, ctypes.POINTER(MoeNvfp4Weights), i32, i32, i32, i32, i32,
                                       i32, vp, vp, vp, i64, i32, i64, vp, vp, f32, f32, i32, vp, vp]),
        "mx_quant": (i32, [vp, i64, i32, i32, i32, vp, vp, vp]),
        "mx_dequant": (i32, [vp, vp, i32, i32, i32, vp, i64, vp]),
        "mx_add_norm_quant": (i32, [vp, i64, vp, i64, vp, f32, f32, i32, i32, i32, vp, i64, vp, vp, vp]),
        "mx_gemm": (i32, [vp, vp, i32, vp, vp, i32, i32, i32, i32, vp, i64, i32, vp]),
        "moe_dispatch": (i32, [vp, i64, i64, vp, vp, vp, i32, i32, i64, vp, i64, vp]),
        "moe_dispatch_bwd": (i32, [vp, i64, i32, vp, i32, i32, i64, i32, vp, i64, vp]),
        "moe_combine": (i32, [vp, i64, i32, vp, vp, i32, i32, i64, i32, vp, i64, vp]),
        "moe_combine_bwd": (i32, [vp, i64, vp, i64, i32, vp, vp, vp, vp, i32, i32, i64, i32, vp, i64, vp, vp]),
        "moe_validate_weights": (i32, [ctypes.POINTER(MoeNvfp4Weights), i32, i32, i32, i32]),
        "moe_workspace_bytes": (i64, [i32, i32, i32, i32, i32, i32, i32, ctypes.POINTER(MoeWorkspaceLayout)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(rc: int, name: str) -> None:
    if rc != MOE_OK:
        msg = lib().moe_last_error().decode(errors="replace")
        raise MoeError(f"{name} failed ({rc}): {msg}")


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch tensor")
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:   # the current stream of the current device, without the objects around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# ------------------------------------------------------------------ sizing
def moe_rows_max(T: int, K: int, E_local: int, tile_m: int) -> int:
    return int(lib().moe_rows_max(T, K, E_local, tile_m))


def moe_workspace_bytes(T: int, K: int, E_local: int, H: int, I: int, tile_m: int,
                        tp: int = 1) -> MoeWorkspaceLayout:
    out = MoeWorkspaceLayout()
    n = lib().moe_workspace_bytes(T, K, E_local, H, I, tile_m, tp, ctypes.byref(out))
    if n < 0:
        _check(MOE_EINVAL, "moe_workspace_bytes")
    return out


def moe_meta_layout_get(T: int, K: int, E_local: int, tile_m: int) -> MoeMetaLayout:
    out = MoeMetaLayout()
    _check(lib().moe_meta_layout_get(T, K, E_local, tile_m, ctypes.byref(out)), "moe_meta_layout_get")
    return out


# ------------------------------------------------------------------ entry points
def moe_route(logits, expert_bias, is_padding, K, route_scale, tile_m, local_expert_offset,
              local_num_experts, topk_ids, topk_weights, meta, stream=None) -> None:
    T, E = logits.shape
    _check(lib().moe_route(_ptr(logits), logits.stride(0), _ptr(expert_bias), _ptr(is_padding),
                           T, E, K, float(route_scale), tile_m, local_expert_offset,
                           local_num_experts, _ptr(topk_ids), _ptr(topk_weights), _ptr(meta),
                           _stream(stream)), "moe_route")


def nvfp4_quant(x, gscale, codes, sf, stream=None) -> None:
    T, H = x.shape
    _check(lib().nvfp4_quant(_ptr(x), x.stride(0), _ptr(gscale), T, H, _ptr(codes), _ptr(sf),
                             _stream(stream)), "nvfp4_quant")


def nvfp4_norm_quant(x, norm_weight, gain_center, eps, gscale, codes, sf, stream=None) -> None:
    T, H = x.shape
    _check(lib().nvfp4_norm_quant(_ptr(x), x.stride(0), _ptr(norm_weight), gain_center, eps,
                                  _ptr(gscale), T, H, _ptr(codes), _ptr(sf), _stream(stream)),
           "nvfp4_norm_quant")


def moe_router_logits(x, w_router, logits, stream=None) -> None:
    T, D = x.shape
    _check(lib().moe_router_logits(_ptr(x), x.stride(0), _ptr(w_router), T, D, w_router.shape[0],
                                   _ptr(logits), _stream(stream)), "moe_router_logits")


def moe_router_route(x, w_router, expert_bias, is_padding, K, route_scale, tile_m, local_expert_offset,
                     local_num_experts, logits, topk_ids, topk_weights, meta, stream=None) -> None:
    T, D = x.shape
    _check(lib().moe_router_route(_ptr(x), x.stride(0), _ptr(w_router), D, _ptr(expert_bias),
                                  _ptr(is_padding), T, w_router.shape[0], K, route_scale, tile_m,
                                  local_expert_offset, local_num_experts, _ptr(logits), _ptr(topk_ids),
                                  _ptr(topk_weights), _ptr(meta), _stream(stream)), "moe_router_route")


def moe_route_quant(logits, expert_bias, is_padding, K, route_scale, tile_m, local_expert_offset,
                    local_num_experts, topk_ids, topk_weights, meta, x, gscale, codes, sf,
                    stream=None) -> None:
    T, E = logits.shape
    H = x.shape[1]
    _check(lib().moe_route_quant(_ptr(logits), logits.stride(0), _ptr(expert_bias),
                                 _ptr(is_padding), T, E, K, float(route_scale), tile_m,
                                 local_expert_offset, local_num_experts, _ptr(topk_ids),
                                 _ptr(topk_weights), _ptr(meta), _ptr(x), x.stride(0),
                                 _ptr(gscale), H, _ptr(codes), _ptr(sf), _stream(stream)),
           "moe_route_quant")


def moe_pack_w13(codes, sf, E, I, H, out_codes, out_sf, stream=None) -> None:
    _check(lib().moe_pack_w13(_ptr(codes), _ptr(sf), E, I, H, _ptr(out_codes), _ptr(out_sf),
                              _stream(stream)), "moe_pack_w13")


def moe_pack_w2(codes, sf, E, H, I, out_codes, out_sf, stream=None) -> None:
    _check(lib().moe_pack_w2(_ptr(codes), _ptr(sf), E, H, I, _ptr(out_codes), _ptr(out_sf),
                             _stream(stream)), "moe_pack_w2")


@dataclass
class Weights:
    """Converted experts (device tensors) plus the strides the kernels read them with."""
    w13: torch.Tensor
    w13_sf: torch.Tensor
    w2: torch.Tensor
    w2_sf: torch.Tensor
    w13_expert_stride: int
    w13_pair_stride: int
    w13_sf_expert_stride: int
    w13_sf_pair_stride: int
    w2_expert_stride: int
    w2_pair_stride: int
    w2_sf_expert_stride: int
    w2_sf_pair_stride: int
    g1_alphas: torch.Tensor
    g1_scale_c: torch.Tensor
    g2_alphas: torch.Tensor
    w13_offset: int = 0       # byte offsets of a view into the tensors above
    w13_sf_offset: int = 0
    w2_offset: int = 0
    w2_sf_offset: int = 0

    def struct(self) -> MoeNvfp4Weights:
        return MoeNvfp4Weights(
            _ptr(self.w13) + self.w13_offset, _ptr(self.w13_sf) + self.w13_sf_offset,
            _ptr(self.w2) + self.w2_offset, _ptr(self.w2_sf) + self.w2_sf_offset,
            self.w13_expert_stride, self.w13_pair_stride, self.w13_sf_expert_stride,
            self.w13_sf_pair_stride, self.w2_expert_stride, self.w2_pair_stride,
            self.w2_sf_expert_stride, self.w2_sf_pair_stride,
            _ptr(self.g1_alphas), _ptr(self.g1_scale_c), _ptr(self.g2_alphas))


def moe_validate_weights(weights: Weights, E_local: int, H: int, I: int, tp: int = 1) -> None:
    """Host-only check of the descriptor (and of its cut into tp slices); raises MoeError."""
    ws = weights.struct()
    _check(lib().moe_validate_weights(ctypes.byref(ws), E_local, H, I, tp), "moe_validate_weights")


def moe_experts_fwd(a_codes, a_sf, meta, weights: Weights, T, K, E_local, H, I, tile_m,
                    inter_codes, inter_sf, rows, stream=None) -> None:
    ws = weights.struct()
    _check(lib().moe_experts_fwd(_ptr(a_codes), _ptr(a_sf), _ptr(meta), ctypes.byref(ws), T, K,
                                 E_local, H, I, tile_m, _ptr(inter_codes), _ptr(inter_sf),
                                 _ptr(rows), rows.stride(0), _stream(stream)), "moe_experts_fwd")


def moe_experts_finalize(a_codes, a_sf, meta, weights: Weights, T, K, E_local, H, I, tile_m,
                         inter_codes, inter_sf, rows, n_partials, partial_stride, topk_weights, norm_weight,
                         gain_center, eps, weight_before_norm, out, stream=None) -> None:
    """rows: the partials' base (partial q at rows + q * partial_stride elements);
    this call writes partial n_partials - 1 and finalizes into out."""
    ws = weights.struct()
    _check(lib().moe_experts_finalize(_ptr(a_codes), _ptr(a_sf), _ptr(meta), ctypes.byref(ws), T, K, E_local,
                                      H, I, tile_m, _ptr(inter_codes), _ptr(inter_sf), _ptr(rows),
                                      rows.stride(-2), n_partials, partial_stride, _ptr(topk_weights),
                                      _ptr(norm_weight), float(gain_center), float(eps),
                                      int(weight_before_norm), _ptr(out), _stream(stream)),
           "moe_experts_finalize")


def moe_experts_fwd_noalloc(a_codes, a_sf, meta, weights: Weights, T, K, E_local, H, I, tile_m,
                            rows, stream=None) -> None:
    ws = weights.struct()
    _check(lib().moe_experts_fwd_noalloc(_ptr(a_codes), _ptr(a_sf), _ptr(meta), ctypes.byref(ws), T, K,
                                         E_local, H, I, tile_m, _ptr(rows), rows.stride(0), _stream(stream)),
           "moe_experts_fwd_noalloc")


def moe_experts_fwd_w4a16(x, meta, weights: Weights, T, K, E_local, H, I, tile_m, inter, rows,
                          stream=None) -> None:
    ws = weights.struct()
    _check(lib().moe_experts_fwd_w4a16(_ptr(x), x.stride(0), _ptr(meta), ctypes.byref(ws), T, K, E_local, H,
                                       I, tile_m, _ptr(inter), _ptr(rows), rows.stride(0), _stream(stream)),
           "moe_experts_fwd_w4a16")


def moe_experts_fwd_bf16(x, meta, w13, w2, T, K, E_local, H, I, tile_m, inter, rows, stream=None) -> None:
    _check(lib().moe_experts_fwd_bf16(_ptr(x), x.stride(0), _ptr(meta), _ptr(w13), _ptr(w2), T, K, E_local, H, I,
                                      tile_m, _ptr(inter), _ptr(rows), rows.stride(0), _stream(stream)),
           "moe_experts_fwd_bf16")


def moe_finalize(rows, n_partials, partial_stride, exp2perm, topk_weights, norm_weight,
                 gain_center, eps, weight_before_norm, T, K, H, out, stream=None) -> None:
    _check(lib().moe_finalize(_ptr(rows), rows.stride(-2), n_partials, partial_stride,
                              _ptr(exp2perm), _ptr(topk_weights), _ptr(norm_weight),
                              float(gain_center), float(eps), int(weight_before_norm), T, K, H,
                              _ptr(out), _stream(stream)), "moe_finalize")


# ------------------------------------------------------------------ MX formats, tokens by expert
# These calls check shapes, types, layouts and devices of their tensors here:
# the library sees addresses only. A decode step's calls are as long as their
# checks, so a tensor that is in order passes one short test (_rows, _flat);
# one that is not goes to _refuse, which finds the reason.
_BF16_TYPES = (torch.bfloat16, torch.int16, torch.uint16)     # int16, uint16: bf16 bit patterns
_TYPED_ROWS = _BF16_TYPES + (torch.float32,)
_U8, _I32, _F32 = (torch.uint8,), (torch.int32,), (torch.float32,)
_E4M3_TYPES = (torch.uint8, torch.float8_e4m3fn)
_SF_TYPES = (torch.uint8, torch.float8_e8m0fnu)
_I32_MAX = 0x7FFFFFFF     # the library's sizes; ctypes would pass the low half of a larger one


def _refuse(call, name, t, dtypes, shape, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{call}: {name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{call}: {name} has type {t.dtype}, not {' or '.join(str(d) for d in dtypes)}")
    if t.shape != shape:
        raise ValueError(f"{call}: {name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{call}: {name} must be a device tensor")
    if t.get_device() != dev:
        raise ValueError(f"{call}: {name} is on {t.device}, not on the current device (or the stream's)")
    raise ValueError(f"{call}: {name} must have contiguous rows{'' if len(shape) == 2 else ' of no stride'}")


def _rows(call, name, t, dtypes, shape, dev) -> int:
    """The row stride in elements of a matrix of one of `dtypes`, of `shape`, on
    device `dev`, with rows of consecutive elements."""
    if isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev:
        if shape[0] <= 1:
            if shape[0] == 0 or shape[1] <= 1 or t.stride(1) == 1:
                return (shape[1] + 15) // 16 * 16       # one row or none: any stride will do
        else:
            s = t.stride()
            if s[1] == 1 or shape[1] <= 1:
                return s[0]
    return _refuse(call, name, t, dtypes, shape, dev)


def _flat(call, name, t, dtypes, shape, dev) -> int:
    """The address of a contiguous tensor of one of `dtypes`, of `shape`, on device `dev`."""
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == dev
            and t.is_contiguous()):
        return t.data_ptr()
    if isinstance(t, torch.Tensor) and not t.is_contiguous() and t.shape == shape:
        raise ValueError(f"{call}: {name} must be contiguous")
    return _refuse(call, name, t, dtypes, shape, dev)


def _where(call, t, stream) -> tuple[int, int]:
    """The device that every tensor has to be on, the current one, and the raw
    stream; a stream object must be of that device. -2 stands for no device: the
    first tensor is a host tensor, which the checks refuse."""
    if t.get_device() < 0:
        return -2, 0
    dev = torch._C._cuda_getDevice()
    if stream is None:
        return dev, torch._C._cuda_getCurrentRawStream(dev)
    if hasattr(stream, "cuda_stream"):
        if stream.device.index != dev:
            raise ValueError(f"{call}: the stream is on {stream.device}, not on the current device")
        return dev, stream.cuda_stream
    return dev, int(stream)


def _shape2(call, name, t):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{call}: {name} must be a tensor of two dimensions")
    shape = t.shape
    if shape[0] > _I32_MAX or shape[1] > _I32_MAX:
        raise MoeError(f"{call}: {name} of shape {tuple(shape)} is too large")
    return shape


def _mx(call, T, H, fmt, codes, sf, dev) -> tuple[int, int]:
    """The addresses of [T, H] values' codes and scales."""
    if H % 32:
        raise MoeError(f"{call}: {H} elements a row are not a multiple of 32")
    if fmt == MOE_MX_E2M1:
        c = _flat(call, "codes", codes, _U8, (T, H // 2), dev)
    elif fmt == MOE_MX_E4M3:
        c = _flat(call, "codes", codes, _E4M3_TYPES, (T, H), dev)
    else:
        raise ValueError(f"{call}: format {fmt!r} is neither MOE_MX_E2M1 nor MOE_MX_E4M3")
    return c, _flat(call, "sf", sf, _SF_TYPES, (T, H // 32), dev)


def mx_quant(x, fmt, codes, sf, stream=None) -> None:
    """bf16 x [T, H] -> MX codes [T, H/2] or [T, H] and e8m0 scales [T, H/32]."""
    shape = T, H = _shape2("mx_quant", "x", x)
    dev, st = _where("mx_quant", x, stream)
    ld = _rows("mx_quant", "x", x, _BF16_TYPES, shape, dev)
    c, s = _mx("mx_quant", T, H, fmt, codes, sf, dev)
    rc = lib().mx_quant(x.data_ptr(), ld, T, H, fmt, c, s, st)
    if rc:
        _check(rc, "mx_quant")


def mx_dequant(codes, sf, fmt, out, stream=None) -> None:
    """MX codes and scales -> bf16 out [T, H]."""
    shape = T, H = _shape2("mx_dequant", "out", out)
    dev, st = _where("mx_dequant", out, stream)
    ld = _rows("mx_dequant", "out", out, _BF16_TYPES, shape, dev)
    c, s = _mx("mx_dequant", T, H, fmt, codes, sf, dev)
    rc = lib().mx_dequant(c, s, T, H, fmt, out.data_ptr(), ld, st)
    if rc:
        _check(rc, "mx_dequant")


def mx_add_norm_quant(x, residual, norm_weight, gain_center, eps, fmt, sum_out, codes, sf, stream=None) -> None:
    """sum_out = bf16(x + residual), and the MX codes and scales of its RMSNorm.
    residual may be None (sum_out then too); sum_out may be residual or x itself."""
    call = "mx_add_norm_quant"
    shape = T, H = _shape2(call, "x", x)
    dev, st = _where(call, x, stream)
    ld = _rows(call, "x", x, _BF16_TYPES, shape, dev)
    ld_res = ld_sum = 0
    res = out = w = None
    if residual is not None:
        ld_res, res = _rows(call, "residual", residual, _BF16_TYPES, shape, dev), residual.data_ptr()
    if sum_out is not None:
        ld_sum, out = _rows(call, "sum_out", sum_out, _BF16_TYPES, shape, dev), sum_out.data_ptr()
    if norm_weight is not None:
        w = _flat(call, "norm_weight", norm_weight, _BF16_TYPES, (H,), dev)
    c, s = _mx(call, T, H, fmt, codes, sf, dev)
    rc = lib().mx_add_norm_quant(x.data_ptr(), ld, res, ld_res, w, gain_center, eps, T, H, fmt, out, ld_sum, c, s, st)
    if rc:
        _check(rc, call)


def mx_gemm(a_codes, a_sf, a_fmt, w_codes, w_sf, w_fmt, out, stream=None) -> None:
    """out [T, N] = a [T, K] times w [N, K] transposed, both MX; out bf16, or fp32
    where both are e2m1."""
    call = "mx_gemm"
    shape = T, N = _shape2(call, "out", out)
    K = _shape2(call, "a_sf", a_sf)[1] * 32
    if K > _I32_MAX:
        raise MoeError(f"{call}: K={K} is too large")
    dev, st = _where(call, out, stream)
    ld = _rows(call, "out", out, _TYPED_ROWS, shape, dev)
    a, asf = _mx(call, T, K, a_fmt, a_codes, a_sf, dev)
    w, wsf = _mx(call, N, K, w_fmt, w_codes, w_sf, dev)
    rc = lib().mx_gemm(a, asf, a_fmt, w, wsf, w_fmt, T, N, K, out.data_ptr(), ld,
                       MOE_F32 if out.dtype == torch.float32 else MOE_BF16, st)
    if rc:
        _check(rc, call)


def mx_gemm_validate(a_fmt, w_fmt, N, K) -> None:
    """Host-only check that mx_gemm takes these formats and K; raises MoeError. (A
    call of no tokens: it checks them, reads nothing and launches nothing.)"""
    if N > _I32_MAX or K > _I32_MAX:
        raise MoeError(f"mx_gemm: N={N} or K={K} is too large")
    _check(lib().mx_gemm(None, None, a_fmt, None, None, w_fmt, 0, N, K, None, N, MOE_BF16, None), "mx_gemm")


def _row_type(call, rows) -> int:
    if rows.dtype == torch.float32:
        return MOE_F32
    if rows.dtype in _BF16_TYPES:
        return MOE_BF16
    raise TypeError(f"{call}: rows of {rows.dtype} are neither bf16 nor fp32")


def moe_dispatch(x, exp2perm, perm2tok, total_rows, rows, stream=None) -> None:
    """rows[exp2perm[t, k]] = x[t]; padding rows below total_rows become zeros.
    x [T, W] and rows [rows_max, W] of one type."""
    call = "moe_dispatch"
    shape = R, W = _shape2(call, "rows", rows)
    maps = T, K = _shape2(call, "exp2perm", exp2perm)
    dev, st = _where(call, rows, stream)
    types, es = (rows.dtype,), rows.element_size()
    ld_x = _rows(call, "x", x, types, (T, W), dev)
    ld_r = _rows(call, "rows", rows, types, shape, dev)
    rc = lib().moe_dispatch(x.data_ptr(), ld_x * es, W * es, _flat(call, "exp2perm", exp2perm, _I32, maps, dev),
                            _flat(call, "perm2tok", perm2tok, _I32, (R,), dev),
                            _flat(call, "total_rows", total_rows, _I32, (1,), dev), T, K, R, rows.data_ptr(),
                            ld_r * es, st)
    if rc:
        _check(rc, call)


def moe_dispatch_bwd(d_rows, exp2perm, d_x, stream=None) -> None:
    """d_x[t] = sum_k d_rows[exp2perm[t, k]]; bf16 or fp32."""
    call = "moe_dispatch_bwd"
    shape = R, H = _shape2(call, "d_rows", d_rows)
    maps = T, K = _shape2(call, "exp2perm", exp2perm)
    dtype, types = _row_type(call, d_rows), (d_rows.dtype,)
    dev, st = _where(call, d_rows, stream)
    ld_r = _rows(call, "d_rows", d_rows, types, shape, dev)
    ld_x = _rows(call, "d_x", d_x, types, (T, H), dev)
    rc = lib().moe_dispatch_bwd(d_rows.data_ptr(), ld_r, dtype, _flat(call, "exp2perm", exp2perm, _I32, maps, dev), T,
                                K, R, H, d_x.data_ptr(), ld_x, st)
    if rc:
        _check(rc, call)


def moe_combine(rows, exp2perm, topk_weights, out, stream=None) -> None:
    """out[t] = sum_k topk_weights[t, k] * rows[exp2perm[t, k]]; bf16 or fp32 rows."""
    call = "moe_combine"
    shape = R, H = _shape2(call, "rows", rows)
    maps = T, K = _shape2(call, "exp2perm", exp2perm)
    dtype, types = _row_type(call, rows), (rows.dtype,)
    dev, st = _where(call, rows, stream)
    ld_r = _rows(call, "rows", rows, types, shape, dev)
    ld_o = _rows(call, "out", out, types, (T, H), dev)
    rc = lib().moe_combine(rows.data_ptr(), ld_r, dtype, _flat(call, "exp2perm", exp2perm, _I32, maps, dev),
                           _flat(call, "topk_weights", topk_weights, _F32, maps, dev), T, K, R, H, out.data_ptr(),
                           ld_o, st)
    if rc:
        _check(rc, call)


def moe_combine_bwd(d_out, rows, exp2perm, perm2tok, total_rows, topk_weights, d_rows, d_weights, stream=None) -> None:
    """moe_combine's gradients: d_rows[exp2perm[t, k]] = topk_weights[t, k] * d_out[t] (padding rows
    below total_rows zero) and d_weights[t, k] = <rows[exp2perm[t, k]], d_out[t]>. d_rows may be rows."""
    call = "moe_combine_bwd"
    shape = R, H = _shape2(call, "rows", rows)
    maps = T, K = _shape2(call, "exp2perm", exp2perm)
    dtype, types = _row_type(call, rows), (rows.dtype,)
    dev, st = _where(call, rows, stream)
    ld_o = _rows(call, "d_out", d_out, types, (T, H), dev)
    ld_r = _rows(call, "rows", rows, types, shape, dev)
    ld_d = _rows(call, "d_rows", d_rows, types, shape, dev)
    rc = lib().moe_combine_bwd(d_out.data_ptr(), ld_o, rows.data_ptr(), ld_r, dtype,
                               _flat(call, "exp2perm", exp2perm, _I32, maps, dev),
                               _flat(call, "perm2tok", perm2tok, _I32, (R,), dev),
                               _flat(call, "total_rows", total_rows, _I32, (1,), dev),
                               _flat(call, "topk_weights", topk_weights, _F32, maps, dev), T, K, R, H,
                               d_rows.data_ptr(), ld_d, _flat(call, "d_weights", d_weights, _F32, maps, dev), st)
    if rc:
        _check(rc, call)
