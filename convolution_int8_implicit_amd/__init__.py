"""MI355X-native fused int8 ResNet convolution: Python binding of libifx.so.

The compute path is the C-ABI library built from csrc/ (hand-written gfx950
HIP kernels); this module only marshals arguments.  Tensors are torch device
tensors (torch supplies memory and streams); every step of the path runs in
the library's kernels.  There is no fallback: if the library is not built the
first call raises.

Entry points mirror include/ifx.h:
    conv_validate, conv_out_dims, act_bytes, wpack_bytes,
    pack_act, unpack_act, pack_weights, conv_fused,
    block_workspace_bytes, block_forward, net_workspace_bytes, net_forward,
    fold_bn, status_string, last_hip_error, version,
    mx4_quantize, mx4_dequantize, mx4_matmul (microscaled 4-bit floating point),
    group_norm, group_norm_mx4, group_norm_backward, group_norm_kernel_name (channels last),
    fp8_quantize, fp8_quantize_t, fp8_dequantize, fp8_matmul (8-bit floating point, a power of two per block of 128),
    gated, gated_fp8, gated_backward (both projections of a gated feed-forward layer),
    rms_norm, rms_norm_fp8, rms_norm_backward
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional, Sequence

import torch

__all__ = [
    "RELU", "RESIDUAL", "MAXPOOL", "OUT_I32", "INPUT_NHWC", "OUT_EVEN", "OUT_PHASE", "IN_PHASE", "IfxError", "ConvDesc", "BlockParams", "NetParams", "lib",
    "conv_desc", "conv_validate", "conv_out_dims", "act_bytes", "wpack_bytes", "pack_act", "unpack_act",
    "pack_weights", "conv_fused", "conv_fused_even", "conv_even_supported", "conv_chain_fused", "conv_chain_kernel_name", "conv_proj_chain_fused",
    "conv_proj_chain_kernel_name", "conv_kernel_name",
    "block_workspace_bytes", "block_forward", "block_forward_noalloc",
    "BLOCK_SCRATCH_BYTES", "net_workspace_bytes",
    "net_forward", "NetGraph", "fold_bn", "BnFold", "status_string", "last_hip_error", "version", "LIB_PATH",
    "ACT_NONE", "ACT_RELU", "ACT_SILU", "Mx4", "mx4_empty", "mx4_quantize", "mx4_dequantize", "mx4_matmul",
    "group_norm", "group_norm_mx4", "group_norm_backward", "GnDesc", "group_norm_kernel_name",
    "FP8_E4M3", "FP8_E5M2", "Fp8", "fp8_empty", "fp8_quantize", "fp8_quantize_t", "fp8_dequantize", "fp8_matmul",
    "gated", "gated_fp8", "gated_backward", "rms_norm", "rms_norm_fp8", "rms_norm_backward",
]

RELU, RESIDUAL, MAXPOOL, OUT_I32, INPUT_NHWC, OUT_EVEN, OUT_PHASE, IN_PHASE = 1, 2, 4, 8, 16, 32, 64, 128
ACT_NONE, ACT_RELU, ACT_SILU = 0, 1, 2
STATUS = {0: "IFX_OK", 1: "IFX_E_NULL", 2: "IFX_E_SHAPE", 3: "IFX_E_UNSUPPORTED", 4: "IFX_E_ALIGN",
          5: "IFX_E_WORKSPACE", 6: "IFX_E_HIP"}

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "lib", "libifx.so")


class IfxError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        name = STATUS.get(status, str(status))
        extra = ""
        if status == 6:
            extra = f" (hipError {last_hip_error()})"
        super().__init__(f"{what}: {name}{extra}")


class ConvDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("h", ctypes.c_int32), ("w", ctypes.c_int32), ("c_in", ctypes.c_int32),
                ("c_out", ctypes.c_int32), ("kh", ctypes.c_int32), ("kw", ctypes.c_int32),
                ("stride", ctypes.c_int32), ("pad", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class BlockParams(ctypes.Structure):
    _fields_ = [("d", ConvDesc * 4), ("has_proj", ctypes.c_int32), ("w_blk", ctypes.c_void_p * 4),
                ("bias", ctypes.c_void_p * 4), ("mult", ctypes.c_void_p * 4), ("shift", ctypes.c_void_p * 4)]


class NetParams(ctypes.Structure):
    _fields_ = [("stem", ConvDesc), ("stem_w", ctypes.c_void_p), ("stem_bias", ctypes.c_void_p),
                ("stem_mult", ctypes.c_void_p), ("stem_shift", ctypes.c_void_p), ("n_blocks", ctypes.c_int32),
                ("blocks", ctypes.POINTER(BlockParams)), ("fc_w_blk", ctypes.c_void_p),
                ("fc_bias", ctypes.c_void_p), ("fc_in", ctypes.c_int32), ("fc_out", ctypes.c_int32),
                ("sub_batch", ctypes.c_int32)]


class BnFold(ctypes.Structure):
    _fields_ = [("c_out", ctypes.c_int32), ("x_scale", ctypes.c_float), ("y_scale", ctypes.c_float),
                ("eps", ctypes.c_float), ("w_per_channel", ctypes.c_int32), ("w_scale", ctypes.c_void_p),
                ("conv_bias", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("beta", ctypes.c_void_p),
                ("mean", ctypes.c_void_p), ("var", ctypes.c_void_p)]


class Mx4Desc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("type", ctypes.c_int32),
                ("act", ctypes.c_int32), ("ld_y", ctypes.c_int64), ("ld_res", ctypes.c_int64)]


class GnDesc(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int32), ("hw", ctypes.c_int32), ("c", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("type", ctypes.c_int32), ("act", ctypes.c_int32), ("eps", ctypes.c_float), ("ld_x", ctypes.c_int64),
                ("ld_y", ctypes.c_int64), ("ld_dy", ctypes.c_int64)]


class Fp8Desc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("a_format", ctypes.c_int32),
                ("type", ctypes.c_int32), ("act", ctypes.c_int32), ("ld_y", ctypes.c_int64), ("ld_res", ctypes.c_int64)]


class GatedDesc(ctypes.Structure):
    _fields_ = [("m", ctypes.c_int32), ("n", ctypes.c_int32), ("k", ctypes.c_int32), ("type", ctypes.c_int32),
                ("act", ctypes.c_int32), ("ld_y", ctypes.c_int64), ("ld_up", ctypes.c_int64), ("ld_dy", ctypes.c_int64)]


class RmsDesc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("c", ctypes.c_int32), ("type", ctypes.c_int32), ("eps", ctypes.c_float),
                ("ld_x", ctypes.c_int64), ("ld_res", ctypes.c_int64), ("ld_h", ctypes.c_int64), ("ld_y", ctypes.c_int64),
                ("ld_dy", ctypes.c_int64), ("ld_dh", ctypes.c_int64)]


_LIB = None


def lib() -> ctypes.CDLL:
    """Load libifx.so (raises if it has not been built)."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"libifx.so not built ({LIB_PATH}); run python -m convolution_int8_implicit_amd.build")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    i64 = ctypes.c_int64
    D = ctypes.POINTER(ConvDesc)
    sigs = {
        "ifx_conv_validate": ([D], i32),
        "ifx_conv_out_dims": ([D, ctypes.POINTER(i32), ctypes.POINTER(i32)], i32),
        "ifx_act_bytes": ([i32, i32, i32, i32], sz),
        "ifx_wpack_bytes": ([D], sz),
        "ifx_pack_act": ([vp, vp, i32, i32, i32, i32, vp], i32),
        "ifx_quantize_f32": ([vp, vp, i64, i32, vp, vp], i32),
        "ifx_quantize_u8": ([vp, vp, i64, i32, vp, vp, vp], i32),
        "ifx_dequantize_i32": ([vp, vp, i64, ctypes.c_float, vp], i32),
        "ifx_unpack_act": ([vp, vp, i32, i32, i32, i32, vp], i32),
        "ifx_pack_weights": ([D, vp, vp, vp], i32),
        "ifx_conv_fused": ([D, vp, vp, vp, vp, vp, vp, vp, vp], i32),
        "ifx_conv_fused_even": ([D, vp, vp, vp, vp, vp, vp, vp, vp, vp], i32),
        "ifx_conv_even_supported": ([D], i32),
        "ifx_conv_proj_fused": ([D, vp, vp, vp, vp, vp, D, vp, vp, vp, vp, vp, vp, vp], i32),
        "ifx_block_workspace_bytes": ([ctypes.POINTER(BlockParams)], sz),
        "ifx_block_forward": ([ctypes.POINTER(BlockParams), vp, vp, vp, sz, vp], i32),
        "ifx_block_forward_noalloc": ([ctypes.POINTER(BlockParams), vp, vp, vp], i32),
        "ifx_net_workspace_bytes": ([ctypes.POINTER(NetParams), i32], sz),
        "ifx_net_forward": ([ctypes.POINTER(NetParams), vp, vp, i32, vp, sz, vp], i32),
        "ifx_fold_bn": ([ctypes.POINTER(BnFold), vp, vp, vp, vp, vp], i32),
        "ifx_net_graph_create": ([ctypes.POINTER(NetParams), vp, vp, i32, vp, sz, ctypes.POINTER(vp)], i32),
        "ifx_graph_launch": ([vp, vp], i32),
        "ifx_graph_destroy": ([vp], i32),
        "ifx_conv_kernel_name": ([D, ctypes.c_char_p, sz], i32),
        "ifx_conv_proj_kernel_name": ([D, D, ctypes.c_char_p, sz], i32),
        "ifx_conv_chain_kernel_name": ([D, D, ctypes.c_char_p, sz], i32),
        "ifx_conv_chain_fused": ([D, vp, vp, vp, vp, vp, vp, vp, D, vp, vp, vp, vp, vp, vp], i32),
        "ifx_conv_proj_chain_kernel_name": ([D, D, D, ctypes.c_char_p, sz], i32),
        "ifx_conv_proj_chain_fused": ([D, vp, vp, vp, vp, vp, D, vp, vp, vp, vp, vp, vp, D, vp, vp, vp, vp, vp,
                                       vp], i32),
        "ifx_mx4_code_bytes": ([i32, i32], sz),
        "ifx_mx4_scale_bytes": ([i32, i32], sz),
        "ifx_mx4_quantize": ([vp, i32, i64, i32, i32, vp, vp, vp], i32),
        "ifx_mx4_dequantize": ([vp, vp, i32, i32, vp, i32, i64, vp], i32),
        "ifx_mx4_matmul": ([ctypes.POINTER(Mx4Desc), vp, vp, vp, vp, vp, vp, vp, vp], i32),
        "ifx_group_norm_workspace_bytes": ([ctypes.POINTER(GnDesc), i32], sz),
        "ifx_group_norm": ([ctypes.POINTER(GnDesc), vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
        "ifx_group_norm_mx4": ([ctypes.POINTER(GnDesc), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
        "ifx_group_norm_backward": ([ctypes.POINTER(GnDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
        "ifx_group_norm_kernel_name": ([ctypes.POINTER(GnDesc), i32, ctypes.c_char_p, sz], i32),
        "ifx_fp8_code_bytes": ([i32, i32], sz),
        "ifx_fp8_scale_bytes": ([i32, i32], sz),
        "ifx_fp8_quantize": ([vp, i32, i64, i32, i32, i32, vp, vp, vp], i32),
        "ifx_fp8_quantize_t": ([vp, i32, i64, i32, i32, i32, vp, vp, vp], i32),
        "ifx_fp8_dequantize": ([vp, vp, i32, i32, i32, vp, i32, i64, vp], i32),
        "ifx_fp8_matmul": ([ctypes.POINTER(Fp8Desc), vp, vp, vp, vp, vp, vp, vp, vp], i32),
        "ifx_gated_workspace_bytes": ([ctypes.POINTER(GatedDesc)], sz),
        "ifx_gated": ([ctypes.POINTER(GatedDesc), vp, vp, vp, vp, vp, vp, vp, vp], i32),
        "ifx_gated_fp8": ([ctypes.POINTER(GatedDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
        "ifx_gated_backward": ([ctypes.POINTER(GatedDesc), vp, vp, vp, vp, vp, vp, vp, vp, vp, vp], i32),
        "ifx_rms_norm_workspace_bytes": ([ctypes.POINTER(RmsDesc)], sz),
        "ifx_rms_norm": ([ctypes.POINTER(RmsDesc), vp, vp, vp, vp, vp, vp, vp], i32),
        "ifx_rms_norm_fp8": ([ctypes.POINTER(RmsDesc), vp, vp, vp, vp, vp, vp, vp, vp], i32),
        "ifx_rms_norm_backward": ([ctypes.POINTER(RmsDesc), vp, vp, vp, vp, vp, vp, vp, vp, sz, vp], i32),
        "ifx_status_string": ([i32], ctypes.c_char_p),
        "ifx_probe_copy": ([vp, vp, sz, vp], i32),
        "ifx_probe_mfma_i8": ([vp, i32, i32, vp], i32),
        "ifx_probe_mfma_i8_data": ([vp, i32, i32, vp], i32),
        "ifx_probe_dma_lds": ([vp, sz, i32, i32, vp, vp], i32),
        "ifx_probe_lds_read": ([vp, i32, i32, vp, vp], i32),
        "ifx_probe_valu": ([i32, vp, i32, i32, vp], i32),
        "ifx_last_hip_error": ([], i32),
        "ifx_version": ([], i32),
    }
    for name, (args, res) in sigs.items():
        fn = getattr(L, name)
        fn.argtypes = args
        fn.restype = res
    _LIB = L
    return L


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> Optional[ctypes.c_void_p]:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check(rc: int, what: str):
    if rc != 0:
        raise IfxError(rc, what)


def _dev(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("libifx takes contiguous device tensors")


def conv_desc(n, h, w, c_in, c_out, kh, kw, stride, pad, flags) -> ConvDesc:
    return ConvDesc(n, h, w, c_in, c_out, kh, kw, stride, pad, flags)


def conv_validate(d: ConvDesc) -> int:
    return lib().ifx_conv_validate(ctypes.byref(d))


def conv_out_dims(d: ConvDesc):
    ho, wo = ctypes.c_int32(), ctypes.c_int32()
    _check(lib().ifx_conv_out_dims(ctypes.byref(d), ctypes.byref(ho), ctypes.byref(wo)), "ifx_conv_out_dims")
    return ho.value, wo.value


def act_bytes(n, h, w, c) -> int:
    return lib().ifx_act_bytes(n, h, w, c)


def wpack_bytes(d: ConvDesc) -> int:
    return lib().ifx_wpack_bytes(ctypes.byref(d))


def pack_act(x_nhwc: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """NHWC int8 -> packed NC/32HW32 [n, ceil(c/32), h, w, 32]."""
    _dev(x_nhwc, out)
    n, h, w, c = x_nhwc.shape
    if out is None:
        out = torch.empty((n, (c + 31) // 32, h, w, 32), dtype=torch.int8, device=x_nhwc.device)
    _check(lib().ifx_pack_act(_ptr(x_nhwc), _ptr(out), n, h, w, c, _stream(stream)), "ifx_pack_act")
    return out


def quantize_f32(x: torch.Tensor, mult: torch.Tensor, out: Optional[torch.Tensor] = None,
                 stream=None) -> torch.Tensor:
    """float32 NHWC image -> int8 codes (ifx_quantize_f32); mult: float32 [c], c the last axis."""
    _dev(x, mult, out)
    assert x.dtype == torch.float32 and mult.dtype == torch.float32
    if out is None:
        out = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    _check(lib().ifx_quantize_f32(_ptr(x), _ptr(out), x.numel(), mult.numel(), _ptr(mult), _stream(stream)),
           "ifx_quantize_f32")
    return out


def quantize_u8(x: torch.Tensor, mean: torch.Tensor, mult: torch.Tensor, out: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    """uint8 NHWC image -> int8 codes (ifx_quantize_u8); mean, mult: float32 [c], c the last axis."""
    _dev(x, mean, mult, out)
    assert x.dtype == torch.uint8 and mean.dtype == torch.float32 and mult.dtype == torch.float32
    assert mean.numel() == mult.numel()
    if out is None:
        out = torch.empty(x.shape, dtype=torch.int8, device=x.device)
    _check(lib().ifx_quantize_u8(_ptr(x), _ptr(out), x.numel(), mult.numel(), _ptr(mean), _ptr(mult),
                                 _stream(stream)), "ifx_quantize_u8")
    return out


def dequantize_i32(q: torch.Tensor, scale: float, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """int32 results (the logits) -> float32 (ifx_dequantize_i32): (float)q * scale."""
    _dev(q, out)
    assert q.dtype == torch.int32
    if out is None:
        out = torch.empty(q.shape, dtype=torch.float32, device=q.device)
    _check(lib().ifx_dequantize_i32(_ptr(q), _ptr(out), q.numel(), float(scale), _stream(stream)),
           "ifx_dequantize_i32")
    return out


def unpack_act(x_blk: torch.Tensor, c: int, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Packed [n, c1, h, w, 32] -> NHWC [n, h, w, c]."""
    _dev(x_blk, out)
    n, _, h, w, _ = x_blk.shape
    if out is None:
        out = torch.empty((n, h, w, c), dtype=torch.int8, device=x_blk.device)
    _check(lib().ifx_unpack_act(_ptr(x_blk), _ptr(out), n, h, w, c, _stream(stream)), "ifx_unpack_act")
    return out


def pack_weights(d: ConvDesc, w_ohwi: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """OHWI int8 -> the packed weight layout of d (flat int8 tensor)."""
    _dev(w_ohwi, out)
    nbytes = wpack_bytes(d)
    if nbytes == 0:
        raise IfxError(conv_validate(d) or 2, "ifx_wpack_bytes")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.int8, device=w_ohwi.device)
    _check(lib().ifx_pack_weights(ctypes.byref(d), _ptr(w_ohwi), _ptr(out), _stream(stream)), "ifx_pack_weights")
    return out


def conv_fused(d: ConvDesc, x_blk, w_blk, bias, mult, shift, residual, y, stream=None) -> None:
    _dev(x_blk, w_blk, bias, mult, shift, residual, y)
    _check(lib().ifx_conv_fused(ctypes.byref(d), _ptr(x_blk), _ptr(w_blk), _ptr(bias), _ptr(mult), _ptr(shift),
                                _ptr(residual), _ptr(y), _stream(stream)), "ifx_conv_fused")


def conv_fused_even(d: ConvDesc, x_blk, w_blk, bias, mult, shift, residual, y, y_even, stream=None) -> None:
    """ifx_conv_fused that also writes the output's even pixels densely to y_even (ifx_conv_fused_even)."""
    _dev(x_blk, w_blk, bias, mult, shift, residual, y, y_even)
    _check(lib().ifx_conv_fused_even(ctypes.byref(d), _ptr(x_blk), _ptr(w_blk), _ptr(bias), _ptr(mult), _ptr(shift),
                                     _ptr(residual), _ptr(y), _ptr(y_even), _stream(stream)), "ifx_conv_fused_even")


def conv_even_supported(d: ConvDesc) -> bool:
    """Whether ifx_conv_fused_even(d, ...) runs (host-only query)."""
    return bool(lib().ifx_conv_even_supported(ctypes.byref(d)))


def conv_proj_fused(d3: ConvDesc, t_blk, w3_blk, bias3, mult3, shift3, dp: ConvDesc, x_blk, wp_blk, biasp, multp,
                    shiftp, y, stream=None) -> None:
    """conv3 of a bottleneck with its 1x1 projection shortcut in one launch (ifx_conv_proj_fused)."""
    _dev(t_blk, w3_blk, bias3, mult3, shift3, x_blk, wp_blk, biasp, multp, shiftp, y)
    _check(lib().ifx_conv_proj_fused(ctypes.byref(d3), _ptr(t_blk), _ptr(w3_blk), _ptr(bias3), _ptr(mult3),
                                     _ptr(shift3), ctypes.byref(dp), _ptr(x_blk), _ptr(wp_blk), _ptr(biasp),
                                     _ptr(multp), _ptr(shiftp), _ptr(y), _stream(stream)), "ifx_conv_proj_fused")


def block_workspace_bytes(p: BlockParams) -> int:
    return lib().ifx_block_workspace_bytes(ctypes.byref(p))


def block_forward(p: BlockParams, x_blk, y_blk, ws: torch.Tensor, stream=None) -> None:
    _dev(x_blk, y_blk, ws)
    _check(lib().ifx_block_forward(ctypes.byref(p), _ptr(x_blk), _ptr(y_blk), _ptr(ws), ws.numel() * ws.element_size(),
                                   _stream(stream)), "ifx_block_forward")


def conv_chain_fused(d3: ConvDesc, t_blk, w3_blk, bias3, mult3, shift3, residual, y, d1: ConvDesc, w1_blk, bias1,
                     mult1, shift1, t1, stream=None) -> None:
    """conv3 (with its shortcut) and the next block's conv1 as one launch (ifx_conv_chain_fused)."""
    ts = (t_blk, w3_blk, bias3, mult3, shift3, residual, y, w1_blk, bias1, mult1, shift1, t1)
    _dev(*ts)
    _check(lib().ifx_conv_chain_fused(ctypes.byref(d3), *[_ptr(t) for t in ts[:7]], ctypes.byref(d1),
                                      *[_ptr(t) for t in ts[7:]], _stream(stream)), "ifx_conv_chain_fused")


def conv_chain_kernel_name(d3: ConvDesc, d1: ConvDesc):
    """The kernel ifx_conv_chain_fused(d3, d1) launches, or None when the pair does not chain."""
    buf = ctypes.create_string_buffer(256)
    rc = lib().ifx_conv_chain_kernel_name(ctypes.byref(d3), ctypes.byref(d1), buf, len(buf))
    if rc == 3:
        return None
    _check(rc, "ifx_conv_chain_kernel_name")
    return buf.value.decode()


def conv_proj_chain_fused(d3: ConvDesc, t_blk, w3_blk, bias3, mult3, shift3, dp: ConvDesc, x_blk, wp_blk, biasp,
                          multp, shiftp, y, d1: ConvDesc, w1_blk, bias1, mult1, shift1, t1, stream=None) -> None:
    """conv3 with its projection shortcut and the next block's conv1 as one launch
    (ifx_conv_proj_chain_fused)."""
    a = (t_blk, w3_blk, bias3, mult3, shift3)
    b = (x_blk, wp_blk, biasp, multp, shiftp, y)
    c = (w1_blk, bias1, mult1, shift1, t1)
    _dev(*a, *b, *c)
    _check(lib().ifx_conv_proj_chain_fused(ctypes.byref(d3), *[_ptr(t) for t in a], ctypes.byref(dp),
                                           *[_ptr(t) for t in b], ctypes.byref(d1), *[_ptr(t) for t in c],
                                           _stream(stream)), "ifx_conv_proj_chain_fused")


def conv_proj_chain_kernel_name(d3: ConvDesc, dp: ConvDesc, d1: ConvDesc):
    """The kernel ifx_conv_proj_chain_fused(d3, dp, d1) launches, or None when they do not chain."""
    buf = ctypes.create_string_buffer(256)
    rc = lib().ifx_conv_proj_chain_kernel_name(ctypes.byref(d3), ctypes.byref(dp), ctypes.byref(d1), buf, len(buf))
    if rc == 3:
        return None
    _check(rc, "ifx_conv_proj_chain_kernel_name")
    return buf.value.decode()


def conv_kernel_name(d: ConvDesc, proj: Optional[ConvDesc] = None) -> str:
    """The kernel instance ifx_conv_fused(d) (or ifx_conv_proj_fused(d, proj)) launches, as
    profilers print it (host-only query)."""
    buf = ctypes.create_string_buffer(256)
    if proj is None:
        _check(lib().ifx_conv_kernel_name(ctypes.byref(d), buf, len(buf)), "ifx_conv_kernel_name")
    else:
        _check(lib().ifx_conv_proj_kernel_name(ctypes.byref(d), ctypes.byref(proj), buf, len(buf)),
               "ifx_conv_proj_kernel_name")
    return buf.value.decode()


def probe_copy(src: torch.Tensor, dst: torch.Tensor, stream=None) -> None:
    """Streaming-copy ceiling probe (ifx_probe.h): dst = src, 16-byte non-temporal chunks."""
    _dev(src, dst)
    nbytes = src.numel() * src.element_size()
    assert dst.numel() * dst.element_size() >= nbytes
    _check(lib().ifx_probe_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream)), "ifx_probe_copy")


def probe_mfma_i8(out: torch.Tensor, blocks: int, iters: int, stream=None) -> int:
    """int8 MFMA ceiling probe (ifx_probe.h); returns the ops it performs."""
    _dev(out)
    assert out.dtype == torch.int32 and out.numel() >= 4 * blocks
    _check(lib().ifx_probe_mfma_i8(_ptr(out), blocks, iters, _stream(stream)), "ifx_probe_mfma_i8")
    return blocks * 4 * iters * 16 * 32768


def probe_mfma_i8_data(out: torch.Tensor, blocks: int, iters: int, stream=None) -> int:
    """int8 MFMA rate probe with operands that change every instruction (ifx_probe.h); returns its ops."""
    _dev(out)
    assert out.dtype == torch.int32 and out.numel() >= 4 * blocks
    _check(lib().ifx_probe_mfma_i8_data(_ptr(out), blocks, iters, _stream(stream)), "ifx_probe_mfma_i8_data")
    return blocks * 4 * iters * 4 * 16 * 32768


def probe_dma_lds(src: torch.Tensor, out: torch.Tensor, blocks: int, iters: int, stream=None) -> int:
    """Buffer->LDS DMA rate probe (ifx_probe.h) over the bytes of src; returns the bytes it moves."""
    _dev(src, out)
    nbytes = src.numel() * src.element_size()
    assert out.dtype == torch.int32 and out.numel() >= 4 * blocks
    _check(lib().ifx_probe_dma_lds(_ptr(src), nbytes, blocks, iters, _ptr(out), _stream(stream)),
           "ifx_probe_dma_lds")
    return blocks * 4 * iters * 8192


def probe_lds_read(offsets: torch.Tensor, out: torch.Tensor, blocks: int, iters: int, stream=None) -> int:
    """ds_read_b128 rate probe (ifx_probe.h) for the lane byte offsets (64 int32); returns the bytes it reads."""
    _dev(offsets, out)
    assert offsets.dtype == torch.int32 and offsets.numel() == 64
    assert out.dtype == torch.int32 and out.numel() >= blocks
    _check(lib().ifx_probe_lds_read(_ptr(offsets), blocks, iters, _ptr(out), _stream(stream)), "ifx_probe_lds_read")
    return blocks * 4 * iters * 8 * 1024


def probe_valu(kind: int, out: torch.Tensor, blocks: int, iters: int, stream=None) -> int:
    """VALU issue-rate probe (ifx_probe.h) of one operation pair (kind 0: requantisation core,
    1: integer add + xor, 2: the f64 form); returns the wave-level chain steps it runs."""
    _dev(out)
    assert out.dtype == torch.int32 and out.numel() >= blocks
    _check(lib().ifx_probe_valu(kind, _ptr(out), blocks, iters, _stream(stream)), "ifx_probe_valu")
    return blocks * 4 * iters * 8


# Bytes of the library-held scratch ifx_block_forward_noalloc uses (IFX_BLOCK_SCRATCH_BYTES).
BLOCK_SCRATCH_BYTES = 64 << 20


def block_forward_noalloc(p: BlockParams, x_blk, y_blk, stream=None) -> None:
    _dev(x_blk, y_blk)
    _check(lib().ifx_block_forward_noalloc(ctypes.byref(p), _ptr(x_blk), _ptr(y_blk), _stream(stream)),
           "ifx_block_forward_noalloc")


def net_workspace_bytes(p: NetParams, n: int) -> int:
    return lib().ifx_net_workspace_bytes(ctypes.byref(p), n)


def net_forward(p: NetParams, x_blk, logits, n: int, ws: torch.Tensor, stream=None) -> None:
    _dev(x_blk, logits, ws)
    _check(lib().ifx_net_forward(ctypes.byref(p), _ptr(x_blk), _ptr(logits), n, _ptr(ws),
                                 ws.numel() * ws.element_size(), _stream(stream)), "ifx_net_forward")


def fold_bn(x_scale: float, y_scale: float, eps: float, w_scale: torch.Tensor, gamma: torch.Tensor,
            beta: torch.Tensor, mean: torch.Tensor, var: torch.Tensor, conv_bias: Optional[torch.Tensor] = None,
            stream=None):
    """BN folding on the device (ifx_fold_bn): float32 device tensors [c_out] (w_scale
    may have one element) -> (bias, mult, shift, status) int32 device tensors."""
    _dev(w_scale, gamma, beta, mean, var, conv_bias)
    n = gamma.numel()
    f = BnFold(n, float(x_scale), float(y_scale), float(eps), 0 if w_scale.numel() == 1 else 1,
               w_scale.data_ptr(), conv_bias.data_ptr() if conv_bias is not None else None, gamma.data_ptr(),
               beta.data_ptr(), mean.data_ptr(), var.data_ptr())
    outs = [torch.empty(n, dtype=torch.int32, device=gamma.device) for _ in range(4)]
    _check(lib().ifx_fold_bn(ctypes.byref(f), *[_ptr(o) for o in outs], _stream(stream)), "ifx_fold_bn")
    return tuple(outs)


# ---------------------------------------------------------------------------
# Microscaled 4-bit tensors and group norm
# ---------------------------------------------------------------------------
_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

# The raw handle of a device's current stream, without a torch.cuda.Stream object around it, and the current
# device (these calls are a few microseconds long).
_current_index = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_current_raw = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _type(dtype: torch.dtype) -> int:
    t = _TYPES.get(dtype)
    if t is None:
        raise TypeError(f"float32, bfloat16 or float16 expected, not {dtype}")
    return t


def _fits(*values: int) -> None:
    """The library takes these as int32, and ctypes would pass a larger one modulo 2^32."""
    for v in values:
        if not -0x80000000 <= v <= 0x7fffffff:
            raise ValueError(f"{v} does not fit 32 bits")


def _on_device(*ts) -> int:
    """The device of the tensors given: one GPU, the current one (the library launches there)."""
    index = ts[0].get_device()
    for t in ts:
        if t is not None and t.get_device() != index:
            raise ValueError(f"tensors of one GPU expected, not {sorted({str(t.device) for t in ts if t is not None})}")
    if index < 0:
        raise ValueError("tensors of a GPU expected")
    if index != _current_index():
        raise ValueError(f"tensors on cuda:{index}, but the current device is cuda:{torch.cuda.current_device()}")
    return index


def _raw_stream(stream, index: int) -> int:
    if stream is None:
        return _current_raw(index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _pitch(t: torch.Tensor):
    """(rows, columns, elements from row to row) of a tensor whose last axis is contiguous and whose
    other axes step as one: a contiguous tensor, or a slice of the last axis of one."""
    shape = t.shape
    if not shape:
        raise ValueError("a tensor of one or more axes expected")
    k = shape[-1]
    if t.is_contiguous():
        return t.numel() // k if k else 0, k, k
    rows, ld = 1, None
    ok = k == 1 or t.stride(-1) == 1
    for size, stride in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if ld is None:
            ld = stride
        ok = ok and stride == ld * rows
        rows *= size
    ld = k if ld is None else ld
    if t.numel() and (not ok or ld < k):
        raise ValueError(f"rows of shape {tuple(shape)} and strides {t.stride()} do not lie at one pitch")
    return rows, k, max(ld, k)


def _alloc(like: torch.Tensor, stream, dtype, *shape) -> torch.Tensor:
    """Uninitialised memory on the device of `like` that belongs to the stream that will use it."""
    if stream is None:
        return torch.empty(*shape, dtype=dtype, device=like.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(*shape, dtype=dtype, device=like.device)


def _alloc_like(x: torch.Tensor, stream) -> torch.Tensor:
    """_alloc of x's type and shape, contiguous."""
    if stream is None and x.is_contiguous():
        return torch.empty_like(x)
    return _alloc(x, stream, x.dtype, *x.shape)


def _addr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _param(t: Optional[torch.Tensor], n: int, name: str) -> None:
    if t is not None and (t.dtype != torch.float32 or t.shape != (n,) or not t.is_contiguous()):
        raise ValueError(f"{name}: contiguous float32 of shape ({n},) expected")


class Mx4(NamedTuple):
    """A microscaled 4-bit tensor of codes.shape[1] rows and k columns (layout: include/ifx.h):
    codes uint8 [ceil(k / 128), rows, 64], scales uint8 [ceil(k / 128), rows, 4]."""
    codes: torch.Tensor
    scales: torch.Tensor
    k: int

    @property
    def rows(self) -> int:
        return self.codes.shape[1]


def _mx4_like(rows: int, k: int, like: torch.Tensor, stream) -> Mx4:
    k1 = (k + 127) // 128
    return Mx4(_alloc(like, stream, torch.uint8, k1, rows, 64), _alloc(like, stream, torch.uint8, k1, rows, 4), k)


def mx4_empty(rows: int, k: int, device="cuda") -> Mx4:
    """Uninitialised codes and scales, for the `out` of a call."""
    k1 = (k + 127) // 128
    return Mx4(torch.empty((k1, rows, 64), dtype=torch.uint8, device=device),
               torch.empty((k1, rows, 4), dtype=torch.uint8, device=device), k)


def _mx4_check(q: Mx4, name: str) -> int:
    """The rows of q."""
    codes, scales, k = q
    k1 = (k + 127) // 128
    rows = codes.shape[1] if codes.dim() == 3 else -1
    if (codes.shape != (k1, rows, 64) or scales.shape != (k1, rows, 4) or codes.dtype != torch.uint8
            or scales.dtype != torch.uint8 or not codes.is_contiguous() or not scales.is_contiguous()):
        raise ValueError(f"{name}: contiguous uint8 codes [{k1}, rows, 64] and scales [{k1}, rows, 4] expected for k = {k}")
    return rows


def mx4_quantize(x: torch.Tensor, out: Optional[Mx4] = None, stream=None) -> Mx4:
    """x [..., k] (float32, bfloat16 or float16) rounded to microscaled 4-bit codes, a row per leading
    index (ifx_mx4_quantize)."""
    rows, k, ld = _pitch(x)
    _fits(rows, k)
    if out is None:
        index = _on_device(x)
        out = _mx4_like(rows, k, x, stream)
    else:
        index = _on_device(x, out.codes, out.scales)
        if _mx4_check(out, "out") != rows or out.k != k:
            raise ValueError(f"out of {out.rows} x {out.k}, x of {rows} x {k}")
    _check(lib().ifx_mx4_quantize(x.data_ptr(), _type(x.dtype), ld, rows, k, out.codes.data_ptr(), out.scales.data_ptr(),
                                  _raw_stream(stream, index)), "ifx_mx4_quantize")
    return out


def mx4_dequantize(q: Mx4, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The values of a microscaled tensor, [rows, k] (ifx_mx4_dequantize)."""
    index = _on_device(q.codes, q.scales, out)
    rows, k = _mx4_check(q, "q"), q.k
    _fits(rows, k)
    ld = k
    if out is None:
        out = _alloc(q.codes, stream, dtype, rows, k)
    else:
        if out.shape != (rows, k):
            raise ValueError(f"out of shape {tuple(out.shape)}, q of {rows} x {k}")
        ld = _pitch(out)[2]
    _check(lib().ifx_mx4_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), rows, k, out.data_ptr(), _type(out.dtype),
                                    ld, _raw_stream(stream, index)), "ifx_mx4_dequantize")
    return out


def mx4_matmul(a: Mx4, w: Mx4, bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
               act: int = ACT_NONE, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """act(a @ w.T + bias + residual), [a.rows, w.rows] (ifx_mx4_matmul); bias float32 [w.rows],
    residual of the output's type and shape."""
    index = _on_device(a.codes, a.scales, w.codes, w.scales, bias, residual, out)
    m, n = _mx4_check(a, "a"), _mx4_check(w, "w")
    if a.k != w.k:
        raise ValueError(f"a of {a.k} columns, w of {w.k}")
    _fits(m, n, a.k, act)
    _param(bias, n, "bias")
    ld_y = ld_res = n
    if out is None:
        out = _alloc(a.codes, stream, dtype, m, n)
    else:
        if out.shape != (m, n):
            raise ValueError(f"out of shape ({m}, {n}) expected")
        ld_y = _pitch(out)[2]
    if residual is not None:
        if residual.shape != (m, n) or residual.dtype != out.dtype:
            raise ValueError(f"residual of shape ({m}, {n}) and {out.dtype} expected")
        ld_res = _pitch(residual)[2]
    d = Mx4Desc(m, n, a.k, _type(out.dtype), act, ld_y, ld_res)
    _check(lib().ifx_mx4_matmul(d, a.codes.data_ptr(), a.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(),
                                _addr(bias), _addr(residual), out.data_ptr(), _raw_stream(stream, index)),
           "ifx_mx4_matmul")
    return out


def _gn_desc(x: torch.Tensor, groups: int, act: int, eps: float) -> GnDesc:
    if x.dim() < 2:
        raise ValueError("x of shape [n, ..., c] expected")
    ld = _pitch(x)[2]
    hw = 1
    for size in x.shape[1:-1]:
        hw *= size
    _fits(x.shape[0], hw, x.shape[-1], groups, act)
    return GnDesc(x.shape[0], hw, x.shape[-1], groups, _type(x.dtype), act, eps, ld, ld, ld)


def _gn_ws(d: GnDesc, backward: int, like: torch.Tensor, stream):
    """The workspace (None where none is needed) and its bytes."""
    nbytes = lib().ifx_group_norm_workspace_bytes(d, backward)
    return (_alloc(like, stream, torch.uint8, nbytes) if nbytes else None), nbytes


def _like(t: torch.Tensor, x: torch.Tensor, name: str) -> int:
    if t.shape != x.shape or t.dtype != x.dtype:
        raise ValueError(f"{name}: shape {tuple(x.shape)} and {x.dtype} expected")
    return _pitch(t)[2]


def _shares(a: torch.Tensor, b: torch.Tensor, rows: int, c: int, ld_a: int, ld_b: int) -> bool:
    """Whether two tensors of one type, each of `rows` rows of c elements at its pitch, have an element in common."""
    d = (b.data_ptr() - a.data_ptr()) // a.element_size()
    if rows == 0 or d >= (rows - 1) * ld_a + c or -d >= (rows - 1) * ld_b + c:
        return False
    # side by side in the rows of a wider tensor, or not
    return ld_a != ld_b or d % ld_a < c or ld_a - d % ld_a < c


def group_norm_kernel_name(d: GnDesc, form: int = 0) -> str:
    """The (first) kernel instance that ifx_group_norm (form 0), its gradient (1) or its 4-bit form (2) launches
    for d, as profilers print it (host-only query)."""
    buf = ctypes.create_string_buffer(256)
    _check(lib().ifx_group_norm_kernel_name(ctypes.byref(d), form, buf, len(buf)), "ifx_group_norm_kernel_name")
    return buf.value.decode()


def group_norm(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
               bias: Optional[torch.Tensor] = None, eps: float = 1e-5, act: int = ACT_NONE,
               out: Optional[torch.Tensor] = None, stream=None):
    """Group norm of channels-last x [n, ..., c] with an activation (ifx_group_norm) ->
    (y, mean [n, groups], rstd [n, groups]).  As every call here it records nothing for autograd: the results
    require no gradient, group_norm_backward gives it."""
    index = _on_device(x, weight, bias, out)
    d = _gn_desc(x, groups, act, eps)
    _param(weight, d.c, "weight")
    _param(bias, d.c, "bias")
    if out is None:
        out = _alloc_like(x, stream)
        d.ld_y = d.c
    else:
        d.ld_y = _like(out, x, "out")
    count = max(groups, 0)  # refused below
    mean, rstd = _alloc(x, stream, torch.float32, d.n, count), _alloc(x, stream, torch.float32, d.n, count)
    ws, nbytes = _gn_ws(d, 0, x, stream)
    _check(lib().ifx_group_norm(d, x.data_ptr(), _addr(weight), _addr(bias), out.data_ptr(), mean.data_ptr(),
                                rstd.data_ptr(), _addr(ws), nbytes, _raw_stream(stream, index)), "ifx_group_norm")
    return out, mean, rstd


def group_norm_mx4(x: torch.Tensor, groups: int, weight: Optional[torch.Tensor] = None,
                   bias: Optional[torch.Tensor] = None, eps: float = 1e-5, act: int = ACT_NONE,
                   out: Optional[Mx4] = None, stream=None) -> Mx4:
    """group_norm whose result is rounded to microscaled 4-bit codes instead of being stored, a row per
    pixel (ifx_group_norm_mx4)."""
    index = _on_device(x, weight, bias, *(out[:2] if out is not None else ()))
    d = _gn_desc(x, groups, act, eps)
    _param(weight, d.c, "weight")
    _param(bias, d.c, "bias")
    rows = d.n * d.hw
    if out is None:
        out = _mx4_like(rows, d.c, x, stream)
    elif _mx4_check(out, "out") != rows or out.k != d.c:
        raise ValueError(f"out of {out.rows} x {out.k}, x of {rows} pixels of {d.c} channels")
    ws, nbytes = _gn_ws(d, 0, x, stream)
    _check(lib().ifx_group_norm_mx4(d, x.data_ptr(), _addr(weight), _addr(bias), out.codes.data_ptr(),
                                    out.scales.data_ptr(), None, None, _addr(ws), nbytes, _raw_stream(stream, index)),
           "ifx_group_norm_mx4")
    return out


def group_norm_backward(dy: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor, groups: int,
                        weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                        act: int = ACT_NONE, out: Optional[torch.Tensor] = None, stream=None):
    """Gradient of group_norm (ifx_group_norm_backward) -> (dx, dweight [c], dbias [c]); mean and rstd are
    the forward pass's.  dweight and dbias are float32, also where weight or bias is None (1 and 0)."""
    index = _on_device(dy, x, mean, rstd, weight, bias, out)
    d = _gn_desc(x, groups, act, 0.0)
    _param(weight, d.c, "weight")
    _param(bias, d.c, "bias")
    for t, name in ((mean, "mean"), (rstd, "rstd")):
        if t.dtype != torch.float32 or t.shape != (d.n, groups) or not t.is_contiguous():
            raise ValueError(f"{name}: contiguous float32 of shape ({d.n}, {groups}) expected")
    d.ld_dy = _like(dy, x, "dy")
    if out is None:
        out = _alloc_like(x, stream)
        d.ld_y = d.c
    else:
        d.ld_y = _like(out, x, "out")
    dweight, dbias = _alloc(x, stream, torch.float32, d.c), _alloc(x, stream, torch.float32, d.c)
    ws, nbytes = _gn_ws(d, 1, x, stream)
    _check(lib().ifx_group_norm_backward(d, dy.data_ptr(), x.data_ptr(), mean.data_ptr(), rstd.data_ptr(), _addr(weight),
                                         _addr(bias), out.data_ptr(), dweight.data_ptr(), dbias.data_ptr(), _addr(ws),
                                         nbytes, _raw_stream(stream, index)), "ifx_group_norm_backward")
    return out, dweight, dbias


# ---------------------------------------------------------------------------
# 8-bit floating point tensors, the gated projections and root mean square norm
# ---------------------------------------------------------------------------
#: The 8-bit formats: four exponent and three mantissa bits (up to 448), five and two (up to 57344).
FP8_E4M3, FP8_E5M2 = 0, 1


class Fp8(NamedTuple):
    """An 8-bit floating point tensor of codes.shape[1] rows and k columns (layout: include/ifx.h):
    codes uint8 [ceil(k / 128), rows, 128], scales uint8 [ceil(k / 512), rows, 4]."""
    codes: torch.Tensor
    scales: torch.Tensor
    k: int
    format: int = FP8_E4M3

    @property
    def rows(self) -> int:
        return self.codes.shape[1]


def _fp8_like(rows: int, k: int, format: int, like: torch.Tensor, stream) -> Fp8:
    return Fp8(_alloc(like, stream, torch.uint8, (k + 127) // 128, rows, 128),
               _alloc(like, stream, torch.uint8, (k + 511) // 512, rows, 4), k, format)


def fp8_empty(rows: int, k: int, format: int = FP8_E4M3, device="cuda") -> Fp8:
    """Uninitialised codes and scales, for the `out` of a call."""
    return Fp8(torch.empty(((k + 127) // 128, rows, 128), dtype=torch.uint8, device=device),
               torch.empty(((k + 511) // 512, rows, 4), dtype=torch.uint8, device=device), k, format)


def _fp8_check(q: Fp8, name: str) -> int:
    """The rows of q."""
    codes, scales, k, _ = q
    k1, k4 = (k + 127) >> 7, (k + 511) >> 9
    try:
        panels, rows, width = codes.shape
        words, same, four = scales.shape
    except ValueError:
        panels = rows = width = words = same = four = -1
    if (panels != k1 or width != 128 or words != k4 or same != rows or four != 4 or codes.dtype is not torch.uint8
            or scales.dtype is not torch.uint8 or not codes.is_contiguous() or not scales.is_contiguous()):
        raise ValueError(f"{name}: contiguous uint8 codes [{k1}, rows, 128] and scales [{k4}, rows, 4] expected for k = {k}")
    return rows


def _fp8_out(out: Optional[Fp8], rows: int, k: int, format: int, like: torch.Tensor, stream) -> Fp8:
    """`out`, which has to be of these sizes and this format, or a new tensor."""
    if out is None:
        return _fp8_like(rows, k, format, like, stream)
    if _fp8_check(out, "out") != rows or out.k != k or out.format != format:
        raise ValueError(f"out of {out.rows} x {out.k} in format {out.format}, {rows} x {k} in format {format} expected")
    return out


def _e4m3(format: int, name: str) -> None:
    if format != FP8_E4M3:
        raise ValueError(f"{name}: format FP8_E4M3 expected")


def _out_parts(out: Optional[Fp8]):
    return out[:2] if out is not None else ()


def fp8_quantize(x: torch.Tensor, format: int = FP8_E4M3, out: Optional[Fp8] = None, stream=None) -> Fp8:
    """x [..., k] (float32, bfloat16 or float16) rounded to 8 bits with a power of two per block of 128 columns, a row
    per leading index (ifx_fp8_quantize)."""
    rows, k, ld = _pitch(x)
    _fits(rows, k, format)
    index = _on_device(x, *_out_parts(out))
    out = _fp8_out(out, rows, k, format, x, stream)
    _check(lib().ifx_fp8_quantize(x.data_ptr(), _type(x.dtype), ld, rows, k, format, out.codes.data_ptr(),
                                  out.scales.data_ptr(), _raw_stream(stream, index)), "ifx_fp8_quantize")
    return out


def fp8_quantize_t(x: torch.Tensor, format: int = FP8_E4M3, out: Optional[Fp8] = None, stream=None) -> Fp8:
    """The transpose of x [..., n], a row per column of x, blocks of 128 consecutive leading indices
    (ifx_fp8_quantize_t)."""
    k, rows, ld = _pitch(x)
    if rows == 0:  # an empty tensor has no rows to _pitch
        k = 1
        for size in x.shape[:-1]:
            k *= size
    _fits(rows, k, format)
    index = _on_device(x, *_out_parts(out))
    out = _fp8_out(out, rows, k, format, x, stream)
    _check(lib().ifx_fp8_quantize_t(x.data_ptr(), _type(x.dtype), ld, rows, k, format, out.codes.data_ptr(),
                                    out.scales.data_ptr(), _raw_stream(stream, index)), "ifx_fp8_quantize_t")
    return out


def fp8_dequantize(q: Fp8, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """The values of an 8-bit tensor, [rows, k] (ifx_fp8_dequantize)."""
    index = _on_device(q.codes, q.scales, out)
    rows, k = _fp8_check(q, "q"), q.k
    _fits(rows, k, q.format)
    ld = k
    if out is None:
        out = _alloc(q.codes, stream, dtype, rows, k)
    else:
        if out.shape != (rows, k):
            raise ValueError(f"out of shape {tuple(out.shape)}, q of {rows} x {k}")
        ld = _pitch(out)[2]
    _check(lib().ifx_fp8_dequantize(q.codes.data_ptr(), q.scales.data_ptr(), q.format, rows, k, out.data_ptr(),
                                    _type(out.dtype), ld, _raw_stream(stream, index)), "ifx_fp8_dequantize")
    return out


def fp8_matmul(a: Fp8, w: Fp8, bias: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
               act: int = ACT_NONE, dtype: torch.dtype = torch.bfloat16, out: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """act(a @ w.T + bias + residual), [a.rows, w.rows] (ifx_fp8_matmul); a in either format, w in FP8_E4M3; bias
    float32 [w.rows], residual of the output's type and shape."""
    index = _on_device(a.codes, a.scales, w.codes, w.scales, bias, residual, out)
    m, n = _fp8_check(a, "a"), _fp8_check(w, "w")
    if a.k != w.k:
        raise ValueError(f"a of {a.k} columns, w of {w.k}")
    _e4m3(w.format, "w")
    _fits(m, n, a.k, act, a.format)
    _param(bias, n, "bias")
    ld_y = ld_res = n
    if out is None:
        out = _alloc(a.codes, stream, dtype, m, n)
    else:
        if out.shape != (m, n):
            raise ValueError(f"out of shape ({m}, {n}) expected")
        ld_y = _pitch(out)[2]
    if residual is not None:
        if residual.shape != (m, n) or residual.dtype != out.dtype:
            raise ValueError(f"residual of shape ({m}, {n}) and {out.dtype} expected")
        ld_res = _pitch(residual)[2]
    d = Fp8Desc(m, n, a.k, a.format, _type(out.dtype), act, ld_y, ld_res)
    _check(lib().ifx_fp8_matmul(d, a.codes.data_ptr(), a.scales.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(),
                                _addr(bias), _addr(residual), out.data_ptr(), _raw_stream(stream, index)),
           "ifx_fp8_matmul")
    return out


def _gated_desc(x: Fp8, w_gate: Fp8, w_up: Fp8, act: int, dtype: torch.dtype) -> GatedDesc:
    m, n = _fp8_check(x, "x"), _fp8_check(w_gate, "w_gate")
    if _fp8_check(w_up, "w_up") != n or not x.k == w_gate.k == w_up.k:
        raise ValueError(f"x of {x.k} columns, w_gate of {n} x {w_gate.k}, w_up of {w_up.rows} x {w_up.k}")
    _e4m3(x.format or w_gate.format or w_up.format, "x, w_gate and w_up")
    _fits(m, n, x.k, act)
    return GatedDesc(m, n, x.k, _type(dtype), act, n, n, n)


def _gated_addrs(x: Fp8, w_gate: Fp8, w_up: Fp8):
    return (x.codes.data_ptr(), x.scales.data_ptr(), w_gate.codes.data_ptr(), w_gate.scales.data_ptr(),
            w_up.codes.data_ptr(), w_up.scales.data_ptr())


def gated(x: Fp8, w_gate: Fp8, w_up: Fp8, act: int = ACT_SILU, dtype: torch.dtype = torch.bfloat16,
          out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """act(x @ w_gate.T) * (x @ w_up.T), [x.rows, w_gate.rows], in one kernel (ifx_gated); all in FP8_E4M3."""
    index = _on_device(*x[:2], *w_gate[:2], *w_up[:2], out)
    d = _gated_desc(x, w_gate, w_up, act, dtype if out is None else out.dtype)
    if out is None:
        out = _alloc(x.codes, stream, dtype, d.m, d.n)
    else:
        if out.shape != (d.m, d.n):
            raise ValueError(f"out of shape ({d.m}, {d.n}) expected")
        d.ld_y = _pitch(out)[2]
    _check(lib().ifx_gated(d, *_gated_addrs(x, w_gate, w_up), out.data_ptr(), _raw_stream(stream, index)), "ifx_gated")
    return out


def gated_fp8(x: Fp8, w_gate: Fp8, w_up: Fp8, act: int = ACT_SILU, out: Optional[Fp8] = None, stream=None) -> Fp8:
    """gated whose result is rounded to 8 bits (FP8_E4M3) instead of being stored (ifx_gated_fp8): the operand of the
    projection back."""
    index = _on_device(*x[:2], *w_gate[:2], *w_up[:2], *_out_parts(out))
    d = _gated_desc(x, w_gate, w_up, act, torch.float32)
    out = _fp8_out(out, d.m, d.n, FP8_E4M3, x.codes, stream)
    nbytes = lib().ifx_gated_workspace_bytes(d)
    ws = _alloc(x.codes, stream, torch.uint8, nbytes) if nbytes else None
    _check(lib().ifx_gated_fp8(d, *_gated_addrs(x, w_gate, w_up), out.codes.data_ptr(), out.scales.data_ptr(), _addr(ws),
                               nbytes, _raw_stream(stream, index)), "ifx_gated_fp8")
    return out


def gated_backward(dy: torch.Tensor, x: Fp8, w_gate: Fp8, w_up: Fp8, act: int = ACT_SILU, out=None, stream=None):
    """Gradient of gated at its two projections, which are computed anew (ifx_gated_backward) ->
    (dgate, dup) of dy's type and shape; out: a pair of such tensors, one of which may be dy.  The gradients of x and of
    the weights are products of these (fp8_quantize, fp8_quantize_t, fp8_matmul)."""
    index = _on_device(dy, *x[:2], *w_gate[:2], *w_up[:2], *(out if out is not None else ()))
    d = _gated_desc(x, w_gate, w_up, act, dy.dtype)
    if dy.shape != (d.m, d.n):
        raise ValueError(f"dy of shape ({d.m}, {d.n}) expected")
    d.ld_dy = _pitch(dy)[2]
    if out is None:
        out = (_alloc(dy, stream, dy.dtype, d.m, d.n), _alloc(dy, stream, dy.dtype, d.m, d.n))
    else:
        d.ld_y, d.ld_up = _like(out[0], dy, "out[0]"), _like(out[1], dy, "out[1]")
        if _shares(*out, d.m, d.n, d.ld_y, d.ld_up):
            raise ValueError("out: the two gradients share memory")
    _check(lib().ifx_gated_backward(d, dy.data_ptr(), *_gated_addrs(x, w_gate, w_up), out[0].data_ptr(), out[1].data_ptr(),
                                    _raw_stream(stream, index)), "ifx_gated_backward")
    return out


def _rms_desc(x: torch.Tensor, eps: float) -> RmsDesc:
    rows, c, ld = _pitch(x)
    _fits(rows, c)
    return RmsDesc(rows, c, _type(x.dtype), eps, ld, c, c, c, c, c)


def _rms_forward(x, weight, residual, eps, sum_out, stream, out=None):
    """The descriptor, the sum (x itself without a residual, unless sum_out is given or `out` takes x's place) and
    whether it is written."""
    d = _rms_desc(x, eps)
    _param(weight, d.c, "weight")
    if residual is not None:
        d.ld_res = _like(residual, x, "residual")
    if out is not None:
        d.ld_y = _like(out, x, "out")
    if sum_out is not None:
        d.ld_h = _like(sum_out, x, "sum_out")
        if out is not None and _shares(out, sum_out, d.rows, d.c, d.ld_y, d.ld_h):
            raise ValueError("out and sum_out share memory")
        return d, sum_out, True
    if residual is None and (out is None or not _shares(out, x, d.rows, d.c, d.ld_y, d.ld_x)):
        return d, x, False
    return d, _alloc(x, stream, x.dtype, *x.shape), True


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
             eps: float = 1e-5, out: Optional[torch.Tensor] = None, sum_out: Optional[torch.Tensor] = None, stream=None):
    """Root mean square norm of h = x + residual over the last axis (ifx_rms_norm) -> (y, h, rstd): y and h of x's
    shape and type, rstd float32 [rows].  Without a residual h is x itself, unless out takes its place.  sum_out may be x
    or the residual, out may be either too, but not sum_out.  Records nothing for autograd: rms_norm_backward gives the
    gradient."""
    index = _on_device(x, weight, residual, out, sum_out)
    d, h, written = _rms_forward(x, weight, residual, eps, sum_out, stream, out)
    if out is None:
        out = _alloc(x, stream, x.dtype, *x.shape)
    rstd = _alloc(x, stream, torch.float32, d.rows)
    _check(lib().ifx_rms_norm(d, x.data_ptr(), _addr(residual), _addr(weight), h.data_ptr() if written else None,
                              out.data_ptr(), rstd.data_ptr(), _raw_stream(stream, index)), "ifx_rms_norm")
    return out, h, rstd


def rms_norm_fp8(x: torch.Tensor, weight: Optional[torch.Tensor] = None, residual: Optional[torch.Tensor] = None,
                 eps: float = 1e-5, out: Optional[Fp8] = None, sum_out: Optional[torch.Tensor] = None, stream=None):
    """rms_norm whose result is rounded to 8 bits (FP8_E4M3) instead of being stored, a row per leading index
    (ifx_rms_norm_fp8) -> (q, h, rstd)."""
    index = _on_device(x, weight, residual, sum_out, *_out_parts(out))
    d, h, written = _rms_forward(x, weight, residual, eps, sum_out, stream)
    out = _fp8_out(out, d.rows, d.c, FP8_E4M3, x, stream)
    rstd = _alloc(x, stream, torch.float32, d.rows)
    _check(lib().ifx_rms_norm_fp8(d, x.data_ptr(), _addr(residual), _addr(weight), h.data_ptr() if written else None,
                                  out.codes.data_ptr(), out.scales.data_ptr(), rstd.data_ptr(),
                                  _raw_stream(stream, index)), "ifx_rms_norm_fp8")
    return out, h, rstd


def rms_norm_backward(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, weight: Optional[torch.Tensor] = None,
                      dh: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, stream=None):
    """Gradient of rms_norm (ifx_rms_norm_backward) -> (dx, dweight [c]) from the forward pass's h and rstd; dh is
    what reaches h past the norm.  dx is x's and the residual's; dweight is float32, also where weight is None (1)."""
    index = _on_device(dy, h, rstd, weight, dh, out)
    d = _rms_desc(h, 0.0)
    _param(weight, d.c, "weight")
    _param(rstd, d.rows, "rstd")
    d.ld_dy = _like(dy, h, "dy")
    if dh is not None:
        d.ld_dh = _like(dh, h, "dh")
    if out is None:
        out = _alloc(h, stream, h.dtype, *h.shape)
    else:
        d.ld_y = _like(out, h, "out")
    dweight = _alloc(h, stream, torch.float32, d.c)
    nbytes = lib().ifx_rms_norm_workspace_bytes(d)
    ws = _alloc(h, stream, torch.uint8, nbytes) if nbytes else None
    _check(lib().ifx_rms_norm_backward(d, dy.data_ptr(), h.data_ptr(), rstd.data_ptr(), _addr(weight), _addr(dh),
                                       out.data_ptr(), dweight.data_ptr(), _addr(ws), nbytes, _raw_stream(stream, index)),
           "ifx_rms_norm_backward")
    return out, dweight


class NetGraph:
    """ifx_net_forward for fixed buffers recorded once as a HIP graph (ifx_net_graph_create);
    launch() enqueues the whole network with one call.  Keeps the buffers alive."""

    def __init__(self, p: NetParams, x, logits, n: int, ws: torch.Tensor, keep=()):
        _dev(x, logits, ws)
        self._keep = (p, x, logits, ws, *keep)
        h = ctypes.c_void_p()
        _check(lib().ifx_net_graph_create(ctypes.byref(p), _ptr(x), _ptr(logits), n, _ptr(ws),
                                          ws.numel() * ws.element_size(), ctypes.byref(h)), "ifx_net_graph_create")
        self._h = h

    def launch(self, stream=None) -> None:
        if self._h is None:
            raise RuntimeError("graph destroyed")
        _check(lib().ifx_graph_launch(self._h, _stream(stream)), "ifx_graph_launch")

    def close(self) -> None:
        if self._h is not None:
            _check(lib().ifx_graph_destroy(self._h), "ifx_graph_destroy")
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def status_string(s: int) -> str:
    return lib().ifx_status_string(s).decode()


def last_hip_error() -> int:
    return lib().ifx_last_hip_error()


def version() -> int:
    return lib().ifx_version()


def exported_symbols() -> Sequence[str]:
    return [n for n in dir(lib()) if n.startswith("ifx_")]
