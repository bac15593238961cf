"""Thin Python binding of libconvrot.so, the gfx950 ConvRot low-bit linear.

Argument marshalling only: every step of the path runs in the HIP kernels
behind the C ABI declared in include/convrot.h. PyTorch provides device
memory and the current stream. There is no fallback: if the library is
missing this module raises at import, and every non-OK status raises
ConvRotError with the library's status text.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch

__all__ = [
    "ConvRotError", "lib", "Q", "GRAN", "OUT", "LAYOUT",
    "convrot_rotate_quantize", "convrot_rotate_quantize_dual", "convrot_dequantize_weights", "w4_pack_weights",
    "w4_pack_weights_f6", "w4_packed_f6_bytes", "w4_expand_weights_f6", "w4_pack_lora_up",
    "w4a4_gemm", "w4a4_gemm_workspace_size", "w4a8_gemm",
    "int8_tensorwise_gemm", "convrot_rq_workspace_size", "w4_packed_bytes",
    "ACT", "convrot_lora_forward", "convrot_lora_backward", "convrot_lora_backward_workspace_size",
    "convrot_act_checkpoint", "convrot_act_backward",
    "get_counters", "reset_counters", "device_check", "status_string",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libconvrot.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run __graft_entry__.build() "
        "(hipcc --offload-arch=gfx950). There is no non-HIP fallback.")

lib = ctypes.CDLL(LIB_PATH)


class Q:
    SYM_INT4 = 0
    SYM_INT8 = 1
    UNSIGNED_INT4_SHIFT = 2
    ASYM_UINT4 = 3


class GRAN:
    TENSOR = 0
    ROW = 1
    ROW_GROUP = 2


class OUT:
    BF16 = 0
    F32 = 1
    I32_RAW = 2


class LAYOUT:
    NATURAL = 0
    TILED = 1
    INT8 = 2
    F6 = 3
    F16 = 4


class ACT:
    GELU = 0
    GELU_TANH = 1
    SWIGLU = 2


class _Counters(ctypes.Structure):
    _fields_ = [("launches", ctypes.c_uint64 * 8), ("fallbacks", ctypes.c_uint64)]


_vp, _i64, _i, _f, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_SIGS = {
    "convrot_status_string": (ctypes.c_char_p, [_i]),
    "convrot_last_hip_error": (_i, []),
    "convrot_device_check": (_i, []),
    "convrot_get_counters": (None, [ctypes.POINTER(_Counters)]),
    "convrot_reset_counters": (None, []),
    "convrot_rq_workspace_size": (_sz, [_i64, _i64, _i, _i, _i, _i]),
    "convrot_rotate_quantize": (_i, [_vp, _i64, _i64, _i64, _i, _i, _i, _i, _f, _vp, _vp, _i, _vp, _i,
                                     _vp, _i, _vp, _vp, _vp, _sz, _vp]),
    "convrot_rotate_quantize_noalloc": (_i, [_vp, _i64, _i64, _i64, _i, _i, _i, _i, _f, _vp, _vp, _i, _vp, _i,
                                             _vp, _i, _vp, _vp, _vp]),
    "convrot_rotate_quantize_dual": (_i, [_vp, _i64, _i64, _i64, _i, _vp, _i, _vp, _vp, _vp, _vp, _sz, _vp]),
    "convrot_dequantize_weights": (_i, [_vp, _vp, _vp, _i64, _i64, _i, _i, _i, _i, _vp, _vp, _i, _vp, _vp]),
    "w4_packed_bytes": (_sz, [_i64, _i64, _i, _i, _i, _i]),
    "w4_pack_weights": (_i, [_vp, _vp, _vp, _i64, _i64, _i, _i, _i, _vp, _vp, _vp, _vp, _vp]),
    "w4_packed_f6_bytes": (_sz, [_i64, _i64]),
    "w4_pack_weights_f6": (_i, [_vp, _i64, _i64, _vp, _vp]),
    "w4_expand_weights_f6": (_i, [_vp, _i64, _i64, _vp, _vp]),
    "w4_pack_lora_up": (_i, [_vp, _i64, _i, _vp, _vp]),
    "w4a4_gemm_workspace_size": (_sz, [_i64, _i64, _i, _i]),
    "w4a4_gemm": (_i, [_vp, _i, _vp, _i, _i, _f, _vp, _i, _vp, _i, _vp, _vp, _i, _vp, _i, _vp,
                       _vp, _i, _i64, _i64, _i64, _i64, _vp, _sz, _vp]),
    "w4a8_gemm": (_i, [_vp, _i, _vp, _i, _vp, _vp, _vp, _i, _vp, _i, _vp, _i, _vp, _vp, _i, _i64, _i64, _i64, _i64,
                       _vp, _sz, _vp]),
    "int8_tensorwise_gemm": (_i, [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i64, _i64, _i64, _i64,
                                  _vp, _sz, _vp]),
    "convrot_lora_forward": (_i, [_vp, _i64, _vp, _vp, _i, _i, _vp, _vp, _i, _vp, _vp, _i64, _vp, _i, _i64, _vp,
                                  _i64, _i64, _i64, _vp]),
    "convrot_lora_backward_workspace_size": (_sz, [_i64, _i64, _i64, _i, _i]),
    "convrot_lora_backward": (_i, [_vp, _i64, _vp, _vp, _i64, _vp, _i, _i, _vp, _vp, _i, _i, _vp, _vp, _i, _vp,
                                   _vp, _i64, _vp, _i, _i64, _vp, _vp, _i, _i64, _i64, _i64, _vp, _sz, _vp]),
    "convrot_act_checkpoint": (_i, [_vp, _i64, _i64, _i64, _i, _vp, _i64, _vp, _vp, _vp]),
    "convrot_act_backward": (_i, [_vp, _i64, _vp, _vp, _i64, _i64, _i, _vp, _i64, _vp]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


class ConvRotError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = lib.convrot_status_string(status).decode()
        if status == 7:
            msg += f" (hipError {lib.convrot_last_hip_error()})"
        super().__init__(f"{where}: {msg}")


def status_string(status: int) -> str:
    return lib.convrot_status_string(status).decode()


def _check(status: int, where: str):
    if status != 0:
        raise ConvRotError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def device_check() -> int:
    return lib.convrot_device_check()


def get_counters():
    c = _Counters()
    lib.convrot_get_counters(ctypes.byref(c))
    return {"rotate_quantize": c.launches[0], "pack": c.launches[1], "w4a4": c.launches[2],
            "w4a8": c.launches[3], "int8": c.launches[4], "lora": c.launches[5], "act": c.launches[6],
            "fallbacks": c.fallbacks}


def reset_counters():
    lib.convrot_reset_counters()


def convrot_rq_workspace_size(rows, K, rot_group, qtype, gran, q_group=0) -> int:
    return lib.convrot_rq_workspace_size(rows, K, rot_group, qtype, gran, q_group)


def w4_packed_bytes(N, K, qtype, gran, q_group, which) -> int:
    return lib.w4_packed_bytes(N, K, qtype, gran, q_group, which)


def _scale_numel(rows, K, qtype, gran, q_group):
    if gran == GRAN.TENSOR:
        return (1,)
    if gran == GRAN.ROW:
        return (rows,)
    return (rows, K // q_group)


def convrot_rotate_quantize(x, rot_group=256, qtype=Q.SYM_INT4, gran=GRAN.TENSOR, q_group=0,
                            shift=0.0, lora_down=None, lora_act_f32=False, layout=LAYOUT.NATURAL,
                            codes=None, scales=None, zeros=None, lora_act=None, workspace=None,
                            stream=None, smooth=None):
    """x: bf16 [rows, K] (row stride may exceed K). Returns
    (codes, scales, zeros, lora_act); outputs are allocated when not given.
    Tiled int4 codes come back as uint8 [ceil(rows/16), K/64, 512], fp6
    fragments (layout F6) as uint8 [ceil(rows/32), K/64, 1536]."""
    rows, K = x.shape
    ldx = x.stride(0)
    dev = x.device
    if codes is None:
        if qtype == Q.SYM_INT8:
            codes = torch.empty((rows, K), dtype=torch.float16 if layout == LAYOUT.F16 else torch.int8, device=dev)
        elif layout == LAYOUT.TILED:
            codes = torch.empty(((rows + 15) // 16, K // 64, 512), dtype=torch.uint8, device=dev)
        elif layout == LAYOUT.F6:
            codes = torch.empty(((rows + 31) // 32, K // 64, 1536), dtype=torch.uint8, device=dev)
        else:
            codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=dev)
    if scales is None:
        sdt = torch.float16 if qtype == Q.ASYM_UINT4 else torch.float32
        scales = torch.empty(_scale_numel(rows, K, qtype, gran, q_group), dtype=sdt, device=dev)
    if zeros is None and qtype == Q.ASYM_UINT4:
        zeros = torch.empty((rows, K // 32), dtype=torch.uint8, device=dev)
    R = 0
    if lora_down is not None:
        R = lora_down.shape[0]
        if lora_act is None:
            lora_act = torch.empty((rows, R), dtype=torch.float32 if lora_act_f32 else torch.bfloat16,
                                   device=dev)
    need = convrot_rq_workspace_size(rows, K, rot_group, qtype, gran, q_group)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    st = lib.convrot_rotate_quantize(_ptr(x), rows, K, ldx, rot_group, qtype, gran, q_group,
                                     float(shift), _ptr(smooth), _ptr(lora_down), R, _ptr(lora_act),
                                     int(bool(lora_act_f32)), _ptr(codes), int(layout), _ptr(scales), _ptr(zeros),
                                     _ptr(workspace), wsb, _stream(stream))
    _check(st, "convrot_rotate_quantize")
    return codes, scales, zeros, lora_act


def convrot_rotate_quantize_dual(x, rot_group=256, layout4=LAYOUT.NATURAL, codes4=None, scale4=None,
                                 codes8=None, scale8=None, workspace=None, stream=None):
    """Per-tensor INT4 and INT8 codes of one rotation of x (bf16 [rows, K]).
    Returns (codes4, scale4, codes8, scale8)."""
    rows, K = x.shape
    dev = x.device
    if codes4 is None:
        shape = {LAYOUT.TILED: ((rows + 15) // 16, K // 64, 512),
                 LAYOUT.F6: ((rows + 31) // 32, K // 64, 1536)}.get(layout4, (rows, K // 2))
        codes4 = torch.empty(shape, dtype=torch.uint8, device=dev)
    if scale4 is None:
        scale4 = torch.empty(1, dtype=torch.float32, device=dev)
    if codes8 is None:
        codes8 = torch.empty((rows, K), dtype=torch.int8, device=dev)
    if scale8 is None:
        scale8 = torch.empty(1, dtype=torch.float32, device=dev)
    if workspace is None:
        need = convrot_rq_workspace_size(rows, K, rot_group, Q.SYM_INT4, GRAN.TENSOR, 0)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    wsb = workspace.numel() * workspace.element_size()
    st = lib.convrot_rotate_quantize_dual(_ptr(x), rows, K, x.stride(0), rot_group, _ptr(codes4), int(layout4),
                                          _ptr(scale4), _ptr(codes8), _ptr(scale8), _ptr(workspace), wsb,
                                          _stream(stream))
    _check(st, "convrot_rotate_quantize_dual")
    return codes4, scale4, codes8, scale8


def convrot_dequantize_weights(codes, scales, N, K, qtype=Q.SYM_INT4, gran=GRAN.TENSOR, q_group=0, rot_group=256,
                               zeros=None, delta_up=None, delta_down=None, out=None, stream=None):
    """Quantized weights (natural codes) -> bf16 [N, K] in the unrotated basis,
    plus delta_up [N, R] @ delta_down [R, K] when given (the LoRA merge)."""
    if out is None:
        out = torch.empty((N, K), dtype=torch.bfloat16, device=codes.device)
    R = 0 if delta_up is None else delta_up.shape[1]
    st = lib.convrot_dequantize_weights(_ptr(codes), _ptr(scales), _ptr(zeros), N, K, qtype, gran, q_group,
                                        rot_group, _ptr(delta_up), _ptr(delta_down), R, _ptr(out), _stream(stream))
    _check(st, "convrot_dequantize_weights")
    return out


def w4_pack_weights(codes, scales, N, K, qtype=Q.SYM_INT4, gran=GRAN.TENSOR, q_group=0, zeros=None,
                    want_wsum=False, stream=None):
    """Returns (packed, packed_scales, packed_zeros, w_sum)."""
    dev = codes.device
    packed = torch.empty(w4_packed_bytes(N, K, qtype, gran, q_group, 0), dtype=torch.uint8, device=dev)
    nsc = w4_packed_bytes(N, K, qtype, gran, q_group, 1)
    packed_scales = None
    if nsc:
        packed_scales = torch.empty(nsc, dtype=torch.uint8, device=dev)
    nz = w4_packed_bytes(N, K, qtype, gran, q_group, 2)
    packed_zeros = torch.empty(nz, dtype=torch.uint8, device=dev) if nz else None
    w_sum = torch.empty(N, dtype=torch.float32, device=dev) if want_wsum else None
    st = lib.w4_pack_weights(_ptr(codes), _ptr(scales), _ptr(zeros), N, K, qtype, gran, q_group,
                             _ptr(packed), _ptr(packed_scales), _ptr(packed_zeros), _ptr(w_sum),
                             _stream(stream))
    _check(st, "w4_pack_weights")
    if packed_scales is not None:
        packed_scales = packed_scales.view(torch.float16 if qtype == Q.ASYM_UINT4 else torch.float32)
    return packed, packed_scales, packed_zeros, w_sum


def w4_packed_f6_bytes(N, K) -> int:
    return lib.w4_packed_f6_bytes(N, K)


def w4_pack_weights_f6(codes, N, K, packed=None, stream=None):
    """Natural signed int4 codes [N, K/2] -> fp6 E2M3 fragments
    uint8 [N/32, K/64, 1536], the weight operand of the fp6 W4A4 GEMM."""
    if packed is None:
        packed = torch.empty((N // 32, K // 64, 1536), dtype=torch.uint8, device=codes.device)
    st = lib.w4_pack_weights_f6(_ptr(codes), N, K, _ptr(packed), _stream(stream))
    _check(st, "w4_pack_weights_f6")
    return packed


def w4_pack_lora_up(up, packed=None, stream=None):
    """Low-rank up-projection L1 bf16 [N, R] -> tiled bf16 [N/128, R, 128]
    (the lora_up operand of w4a4_gemm and w4a8_gemm)."""
    N, R = up.shape
    if packed is None:
        packed = torch.empty((N // 128, R, 128), dtype=torch.bfloat16, device=up.device)
    st = lib.w4_pack_lora_up(_ptr(up), N, R, _ptr(packed), _stream(stream))
    _check(st, "w4_pack_lora_up")
    return packed


def w4_expand_weights_f6(tiles, N, K, f6=None, stream=None):
    """Tile-packed INT4 weights (w4_pack_weights) -> fp6 E2M3 fragments
    uint8 [N/32, K/64, 1536] (w_layout F6 of w4a4_gemm)."""
    if f6 is None:
        f6 = torch.empty((N // 32, K // 64, 1536), dtype=torch.uint8, device=tiles.device)
    st = lib.w4_expand_weights_f6(_ptr(tiles), N, K, _ptr(f6), _stream(stream))
    _check(st, "w4_expand_weights_f6")
    return f6


def _out(M, N, out_type, dev, out):
    if out is not None:
        return out
    dt = {OUT.BF16: torch.bfloat16, OUT.F32: torch.float32, OUT.I32_RAW: torch.int32}[out_type]
    return torch.empty((M, N), dtype=dt, device=dev)


def _lora_rank(lora_up, N):
    """R of the tiled low-rank up-projection [N/128, R, 128] (0 without one)"""
    if lora_up is None:
        return 0
    if lora_up.dim() != 3 or lora_up.shape[0] * 128 != N or lora_up.shape[2] != 128:
        raise ValueError("lora_up must be tiled [N/128, R, 128] (w4_pack_lora_up)")
    return lora_up.shape[1]


def w4a4_gemm_workspace_size(N, K, a_layout, w_layout) -> int:
    return lib.w4a4_gemm_workspace_size(N, K, int(a_layout), int(w_layout))


def w4a4_gemm(a_codes, a_scales, a_gran, w_packed, w_scales, w_gran, M, N, K,
              a_unsigned=False, a_shift=0.0, w_sum=None, lora_act=None, lora_up=None,
              bias=None, out_type=OUT.BF16, out=None, a_layout=None, w_layout=None, workspace=None, stream=None):
    """a_layout defaults to F6 for [M/32, K/64, 1536] codes, TILED for
    [M/16, K/64, 512], else NATURAL. w_layout defaults to F6 for
    [N/32, K/64, 1536] weights (w4_pack_weights_f6), else TILED
    (w4_pack_weights). With F6 codes and TILED weights the call needs a
    workspace of w4a4_gemm_workspace_size bytes (allocated here when not
    given) into which it expands the weights before the fp6 GEMM.
    lora_up is L1 tiled by w4_pack_lora_up [N/128, R, 128]."""
    if a_layout is None:
        if a_codes.dim() == 3:
            a_layout = LAYOUT.F6 if a_codes.shape[-1] == 1536 else LAYOUT.TILED
        else:
            a_layout = LAYOUT.NATURAL
    if w_layout is None:
        w_layout = LAYOUT.F6 if (w_packed.dim() == 3 and w_packed.shape[-1] == 1536) else LAYOUT.TILED
    need = w4a4_gemm_workspace_size(N, K, a_layout, w_layout)
    if workspace is None and need:
        workspace = torch.empty(need, dtype=torch.uint8, device=a_codes.device)
    wsb = 0 if workspace is None else workspace.numel() * workspace.element_size()
    out = _out(M, N, out_type, a_codes.device, out)
    lora_f32 = int(lora_act is not None and lora_act.dtype == torch.float32)
    R = _lora_rank(lora_up, N)
    st = lib.w4a4_gemm(_ptr(a_codes), int(a_layout), _ptr(a_scales), a_gran, int(bool(a_unsigned)), float(a_shift),
                       _ptr(w_packed), int(w_layout), _ptr(w_scales), w_gran, _ptr(w_sum),
                       _ptr(lora_act), lora_f32, _ptr(lora_up), R, _ptr(bias),
                       _ptr(out), out_type, out.stride(0), M, N, K, _ptr(workspace), wsb, _stream(stream))
    _check(st, "w4a4_gemm")
    return out


def w4a8_gemm(a_codes, a_scales, a_gran, w_packed, w_scales, w_zeros, M, N, K, group=16,
              bias=None, out_type=OUT.BF16, out=None, stream=None, lora_act=None, lora_up=None, a_layout=None):
    """a_codes: int8 [M, K] (NATURAL) or float16 [M, K] (F16, the quantizer's
    fp16-carried codes); a_layout defaults from the dtype. lora_act [M, R]
    (bf16 or float32) with L1 bf16 (R = 32 or 64) adds the
    low-rank bypass; lora_up is L1 tiled by w4_pack_lora_up [N/128, R, 128]."""
    if a_layout is None:
        a_layout = LAYOUT.F16 if a_codes.dtype == torch.float16 else LAYOUT.NATURAL
    out = _out(M, N, out_type, a_codes.device, out)
    R = _lora_rank(lora_up, N)
    lora_f32 = int(lora_act is not None and lora_act.dtype == torch.float32)
    st = lib.w4a8_gemm(_ptr(a_codes), int(a_layout), _ptr(a_scales), a_gran, _ptr(w_packed), _ptr(w_scales),
                       _ptr(w_zeros), group, _ptr(lora_act), lora_f32, _ptr(lora_up), R, _ptr(bias),
                       _ptr(out), out_type, out.stride(0),
                       M, N, K, None, 0, _stream(stream))
    _check(st, "w4a8_gemm")
    return out


def int8_tensorwise_gemm(a_codes, a_scale, w, w_scale, M, N, K, bias=None, out_type=OUT.BF16,
                         out=None, stream=None):
    out = _out(M, N, out_type, a_codes.device, out)
    st = lib.int8_tensorwise_gemm(_ptr(a_codes), _ptr(a_scale), _ptr(w), _ptr(w_scale), _ptr(bias),
                                  _ptr(out), out_type, out.stride(0), M, N, K, None, 0,
                                  _stream(stream))
    _check(st, "int8_tensorwise_gemm")
    return out


# ---------------------------------------------------------------------------
# batched low-rank adapters and 8-bit activation checkpoints
#
# As everywhere in this binding, autograd records nothing: outputs require no
# gradient whatever the inputs do. The backward calls give the gradients.
# ---------------------------------------------------------------------------
_OUT_DTYPE = {OUT.BF16: torch.bfloat16, OUT.F32: torch.float32}
_BF16, _F32, _I32, _I8 = torch.bfloat16, torch.float32, torch.int32, torch.int8
_HERE_ALREADY = contextlib.nullcontext()


def _gpu(t, what):
    """Index of the GPU that the call runs on: that of its first tensor."""
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{what} must be on the GPU")
    return index


def _tensor(t, what, dtype, index, shape):
    """Address of a dense tensor argument; dtype, GPU, shape and contiguity checked."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {tuple(shape)} on GPU {index}")
    return t.data_ptr()


def _rows(t, what, dtype, index, rows, cols):
    """A [rows, cols] argument whose rows may lie further apart: (address, leading dimension)."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != (rows, cols):
        raise ValueError(f"{what} must be a {dtype} [{rows}, {cols}] tensor on GPU {index}")
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{what} must have contiguous rows")
    return t.data_ptr(), (ld if rows > 1 else cols)


def _on(index, stream):
    """The context in which a call allocates and launches: the tensors' GPU and
    the given stream (default: that GPU's current one)."""
    if stream is None:
        return _HERE_ALREADY if index == torch.cuda.current_device() else torch.cuda.device(index)
    if stream.device.index != index:
        raise ValueError("stream belongs to another GPU than the tensors")
    return torch.cuda.stream(stream)


def _hold(stream, *tensors):
    """Tensors of a call on a given stream: memory of theirs that is freed while
    the call still runs is not given out again before it has ended."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


# handle of a GPU's current stream, without the stream object around it
_current_stream_handle = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _refused(status, where, **tensors):
    """Raises for a call that was not accepted, naming addresses that the library does not take."""
    off = [k for k, t in tensors.items() if t is not None and t.data_ptr() % 16]
    _check(status, f"{where} ({', '.join(off)}: not at a multiple of 16 bytes)" if off else where)


def _out_dtype(out_type):
    if out_type not in _OUT_DTYPE:
        raise ValueError("the output type is OUT.BF16 or OUT.F32")
    return _OUT_DTYPE[out_type]


def _adapters(index, rows, down, up, seg_offsets, seg_adapter, scale):
    """Checks what both adapter calls share: (A, R, N, K, S) and the addresses
    of (down, up, seg_offsets, seg_adapter, scale)."""
    if rows.dim() != 2 or down.dim() != 3 or up.dim() != 3 or seg_adapter.dim() != 1:
        raise ValueError("x is [M, K], dy [M, N], down [A, R, K], up [A, N, R], seg_adapter [S]")
    A, R, K = down.shape
    N, S = up.shape[1], seg_adapter.shape[0]
    return A, R, N, K, S, (_tensor(down, "down", _BF16, index, (A, R, K)), _tensor(up, "up", _BF16, index, (A, N, R)),
                           _tensor(seg_offsets, "seg_offsets", _I32, index, (S + 1,)),
                           _tensor(seg_adapter, "seg_adapter", _I32, index, (S,)),
                           None if scale is None else _tensor(scale, "scale", _F32, index, (A,)))


def convrot_lora_forward(x, down, up, seg_offsets, seg_adapter, scale=None, base=None, out_type=OUT.BF16, out=None,
                         lora_act=None, stream=None):
    """Low-rank adapters of many requests beside one projection:
    out = base + scale[a] (x . down[a]^T) . up[a]^T for the rows
    seg_offsets[s] .. seg_offsets[s+1] of each segment s with adapter
    a = seg_adapter[s] (outside 0..A-1: none, out = base).

    x: bf16 [M, K]; down: bf16 [A, R, K]; up: bf16 [A, N, R]; seg_offsets:
    int32 [S+1]; seg_adapter: int32 [S]; scale: float32 [A]; base: [M, N] of
    the output's type (None: zero), which may be `out` itself. Rows of x, base
    and out may lie further apart than their length. Returns (out, lora_act):
    lora_act float32 [M, R] is what convrot_lora_backward reads. Outputs are
    allocated when not given. Not recorded by autograd: the gradients come from
    convrot_lora_backward."""
    index = _gpu(x, "x")
    A, R, N, K, S, (pd, pu, po, pa, ps) = _adapters(index, x, down, up, seg_offsets, seg_adapter, scale)
    M, dt = x.shape[0], _out_dtype(out_type)
    px, ldx = _rows(x, "x", _BF16, index, M, K)
    pb, ldb = (None, N) if base is None else _rows(base, "base", dt, index, M, N)
    with _on(index, stream):
        if out is None:
            out, ldo = torch.empty((M, N), dtype=dt, device=x.device), N
            py = out.data_ptr()
        else:
            py, ldo = _rows(out, "out", dt, index, M, N)
        if lora_act is None:
            lora_act = torch.empty((M, R), dtype=_F32, device=x.device)
            pl = lora_act.data_ptr()
        else:
            pl = _tensor(lora_act, "lora_act", _F32, index, (M, R))
        _hold(stream, x, down, up, seg_offsets, seg_adapter, scale, base, out, lora_act)
        st = lib.convrot_lora_forward(px, ldx, pd, pu, R, A, po, pa, S, ps, pb, ldb, py, out_type, ldo, pl, M, N, K,
                                      _current_stream_handle(index))
    if st:
        _refused(st, "convrot_lora_forward", x=x, down=down, up=up, seg_offsets=seg_offsets, seg_adapter=seg_adapter,
                 scale=scale, base=base, out=out, lora_act=lora_act)
    return out, lora_act


def convrot_lora_backward_workspace_size(M, N, K, R, n_adapters) -> int:
    return lib.convrot_lora_backward_workspace_size(M, N, K, R, n_adapters)


def convrot_lora_backward(dy, lora_act, x, down, up, seg_offsets, seg_adapter, scale=None, x_scales=None,
                          rot_group=256, dx_base=None, dx_type=OUT.BF16, dx=None, d_down=None, d_up=None,
                          want_dx=True, want_weights=True, accumulate=False, workspace=None, stream=None):
    """Gradients of convrot_lora_forward for dy bf16 [M, N]. Returns
    (dx, d_down, d_up): dx = dx_base + scale[a] (dy . up[a]) . down[a] in
    dx_type (None with want_dx=False), d_down float32 [A, R, K] and d_up
    float32 [A, N, R] (None with want_weights=False; accumulate=True adds to
    the given ones).

    x is the forward's input: bf16 [M, K], or as an 8-bit checkpoint the int8
    codes [M, K] that convrot_rotate_quantize (SYM_INT8, per row or per tensor,
    rot_group) made of it, with x_scales float32 [M] or [1]. Codes made with
    smooth stand for x * smooth: divide d_down by smooth then (and do not
    accumulate into it). x and lora_act are not read with want_weights=False
    and may be None then."""
    index = _gpu(dy, "dy")
    A, R, N, K, S, (pd, pu, po, pa, ps) = _adapters(index, dy, down, up, seg_offsets, seg_adapter, scale)
    M, dt, dev = dy.shape[0], _out_dtype(dx_type), dy.device
    pdy, lddy = _rows(dy, "dy", _BF16, index, M, N)
    pl = px = pxs = pb = pdx = pgd = pgu = None
    ldx = ldb = lddx = K
    gran = GRAN.ROW
    if want_weights:
        if accumulate and (d_down is None or d_up is None):
            raise ValueError("accumulate adds to given d_down and d_up")
        if lora_act is None or x is None:
            raise ValueError("the weight gradients need x and lora_act")
        pl = _tensor(lora_act, "lora_act", _F32, index, (M, R))
        px, ldx = _rows(x, "x", _BF16 if x_scales is None else _I8, index, M, K)
        if x_scales is not None:
            gran = GRAN.ROW if x_scales.numel() == M else GRAN.TENSOR
            pxs = _tensor(x_scales, "x_scales", _F32, index, (M if gran == GRAN.ROW else 1,))
    elif not want_dx:
        raise ValueError("nothing is wanted")
    if want_dx and dx_base is not None:
        pb, ldb = _rows(dx_base, "dx_base", dt, index, M, K)
    with _on(index, stream):
        if want_dx and dx is None:
            dx = torch.empty((M, K), dtype=dt, device=dev)
            pdx = dx.data_ptr()
        elif want_dx:
            pdx, lddx = _rows(dx, "dx", dt, index, M, K)
        if want_weights:
            if d_down is None:
                d_down = torch.empty((A, R, K), dtype=_F32, device=dev)
                pgd = d_down.data_ptr()
            else:
                pgd = _tensor(d_down, "d_down", _F32, index, (A, R, K))
            if d_up is None:
                d_up = torch.empty((A, N, R), dtype=_F32, device=dev)
                pgu = d_up.data_ptr()
            else:
                pgu = _tensor(d_up, "d_up", _F32, index, (A, N, R))
        if workspace is None:
            need = lib.convrot_lora_backward_workspace_size(M, N, K, R, A)
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        elif workspace.get_device() != index or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous on GPU {index}")
        _hold(stream, dy, down, up, seg_offsets, seg_adapter, scale, workspace)
        if want_weights:
            _hold(stream, lora_act, x, x_scales, d_down, d_up)
        if want_dx:
            _hold(stream, dx_base, dx)
        st = lib.convrot_lora_backward(pdy, lddy, pl, px, ldx, pxs, gran, rot_group, pd, pu, R, A, po, pa, S, ps,
                                       pb, ldb, pdx, dx_type, lddx, pgd, pgu, int(bool(accumulate)), M, N, K,
                                       workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                       _current_stream_handle(index))
    if st:
        read = dict(dy=dy, down=down, up=up, seg_offsets=seg_offsets, seg_adapter=seg_adapter, scale=scale, workspace=workspace)
        if want_weights:
            read.update(x=x, x_scales=x_scales, lora_act=lora_act, d_down=d_down, d_up=d_up)
        if want_dx:
            read.update(dx_base=dx_base, dx=dx)
        _refused(st, "convrot_lora_backward", **read)
    return (dx if want_dx else None), (d_down if want_weights else None), (d_up if want_weights else None)


def _act_width(t, act, what):
    if t.dim() != 2 or act not in (0, 1, 2):
        raise ValueError(f"{what} has two dimensions and act is one of ACT")
    return t.shape


def convrot_act_checkpoint(z, act, y=None, codes=None, scales=None, stream=None):
    """y = act(z) (ACT.GELU, ACT.GELU_TANH: z bf16 [rows, C]; ACT.SWIGLU: z
    bf16 [rows, 2C], gate then linear half), with z kept as int8 codes and one
    float32 scale per row and 64 columns. Returns (y, codes, scales). Not
    recorded by autograd: the gradient comes from convrot_act_backward."""
    index = _gpu(z, "z")
    rows, W = _act_width(z, act, "z")
    C = W // 2 if act == ACT.SWIGLU else W
    if C % 64 or W % 64:
        raise ValueError("C must be a multiple of 64")
    pz, ldz = _rows(z, "z", _BF16, index, rows, W)
    with _on(index, stream):
        if y is None:
            y, ldy = torch.empty((rows, C), dtype=_BF16, device=z.device), C
            py = y.data_ptr()
        else:
            py, ldy = _rows(y, "y", _BF16, index, rows, C)
        if codes is None:
            codes = torch.empty((rows, W), dtype=_I8, device=z.device)
            pc = codes.data_ptr()
        else:
            pc = _tensor(codes, "codes", _I8, index, (rows, W))
        if scales is None:
            scales = torch.empty((rows, W // 64), dtype=_F32, device=z.device)
            ps = scales.data_ptr()
        else:
            ps = _tensor(scales, "scales", _F32, index, (rows, W // 64))
        _hold(stream, z, y, codes, scales)
        st = lib.convrot_act_checkpoint(pz, ldz, rows, C, act, py, ldy, pc, ps, _current_stream_handle(index))
    if st:
        _refused(st, "convrot_act_checkpoint", z=z, y=y, codes=codes, scales=scales)
    return y, codes, scales


def convrot_act_backward(dy, codes, scales, act, dz=None, stream=None):
    """dz = dy act'(z) with z read back from the codes and scales of
    convrot_act_checkpoint; dy bf16 [rows, C], dz bf16 shaped like codes."""
    index = _gpu(dy, "dy")
    rows, C = _act_width(dy, act, "dy")
    if C % 64:
        raise ValueError("C must be a multiple of 64")
    W = 2 * C if act == ACT.SWIGLU else C
    pdy, lddy = _rows(dy, "dy", _BF16, index, rows, C)
    pc = _tensor(codes, "codes", _I8, index, (rows, W))
    ps = _tensor(scales, "scales", _F32, index, (rows, W // 64))
    with _on(index, stream):
        if dz is None:
            dz, lddz = torch.empty((rows, W), dtype=_BF16, device=dy.device), W
            pz = dz.data_ptr()
        else:
            pz, lddz = _rows(dz, "dz", _BF16, index, rows, W)
        _hold(stream, dy, codes, scales, dz)
        st = lib.convrot_act_backward(pdy, lddy, pc, ps, rows, C, act, pz, lddz, _current_stream_handle(index))
    if st:
        _refused(st, "convrot_act_backward", dy=dy, codes=codes, scales=scales, dz=dz)
    return dz
