"""W4A4 ConvRot linear for AMD MI355X (gfx950): Python binding of libck4.so.

Argument marshalling only. Every step of the layer runs in the HIP kernels
behind the C ABI declared in ``include/ck4.h``; PyTorch provides device
memory and the current stream. If ``libck4.so`` has not been built, every call
raises: there is no CPU fallback.

The layer ("[PR #63] int4_tensorwise: W4A4 layout (+ConvRot) with fused CUDA
kernels", Description): rotate the activation rows with a block Hadamard
transform, quantise each row to int4 (absmax / 7) and pack it low nibble
first, multiply against int4 weights prepared the same way with an int32
GEMM, apply the row and column scales once in the epilogue, write bf16.
"""
from __future__ import annotations

import ctypes
import functools
import operator
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libck4.so")

CK4_OK, CK4_ERR_INVALID, CK4_ERR_UNSUPPORTED, CK4_ERR_DEVICE = 0, 1, 2, 3


class Ck4Error(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str):
        super().__init__(f"{fn} failed with status {status}: {detail}")
        self.status = status
        self.detail = detail


_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_F = ctypes.c_float
_PF = ctypes.POINTER(ctypes.c_float)  # host float array
_PI = ctypes.POINTER(ctypes.c_int)  # host int array
_HEADS = [_P, _I64, _I64]  # a [tokens, heads, d] tensor: pointer, token stride, head stride

SIGNATURES = {
    "ck4_version": ([], ctypes.c_char_p),
    "ck4_status_string": ([_I], ctypes.c_char_p),
    "ck4_last_error": ([], ctypes.c_char_p),
    "ck4_quantize_weight_convrot": ([_P, _I64, _I64, _I64, _I, _I, _P, _P, _P], _I),
    "ck4_quantize_weight_convrot_int8": ([_P, _I64, _I64, _I64, _I, _P, _P, _P], _I),
    "ck4_quantize_weight_convrot_sr": ([_P, _I64, _I64, _I64, _I, _I, _P, _I64, _P, _P, _P], _I),
    "ck4_rotate_quantize_act": ([_P, _I64, _I64, _I64, _I, _I, _P, _P, _P], _I),
    "ck4_rotate_act_f32": ([_P, _I64, _I64, _I64, _I, _P, _P], _I),
    "ck4_linear_w4a4": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck4_linear_w4a4_bf16": ([_P, _I64, _I64, _I64, _I, _P, _P, _P, _I64, _P, _P, _P, _I64, _P], _I),
    "ck4_gemm_w4a4_acc_i32": ([_P, _P, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck4_dequant_w4a8_grouped": ([_P, _P, _I64, _I64, _I, _I64, _I64, _P, _P, _P], _I),
    "ck4_linear_w8a8": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck4_w4a8_workspace_bytes": ([_I64, _I64, _I64, _I64], ctypes.c_size_t),
    "ck4_linear_w4a8_grouped": ([_P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _I64, _I64, _P, ctypes.c_size_t, _P], _I),
    "ck4_linear_w4a8_grouped_noalloc": ([_P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _I64, _I64, _P], _I),
    "ck4_linear_w4a8_grouped_bf16": ([_P, _I64, _I64, _I64, _I, _P, _P, _I, _I64, _I, _P, _P, _P, _I64, _P,
                                      ctypes.c_size_t, _P], _I),
    "ck4_quantize_weight_convrot_e4m3": ([_P, _I64, _I64, _I64, _I, _I, _P, _P, _P], _I),
    "ck4_dequant_w4a8_grouped_e4m3": ([_P, _P, _I64, _I64, _I, _I64, _I64, _P, _P, _P], _I),
    "ck4_linear_w4a8_grouped_e4m3": ([_P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _I64, _I64, _P, ctypes.c_size_t,
                                      _P], _I),
    "ck4_quantize_weight_convrot_codebook": ([_P, _I64, _I64, _I64, _I, _I, _PF, _I, _P, _P, _P], _I),
    "ck4_dequant_w4a8_codebook": ([_P, _P, _I, _PF, _I64, _I64, _I, _I64, _I64, _P, _P, _P], _I),
    "ck4_linear_w4a8_codebook": ([_P, _P, _P, _P, _I, _PF, _I64, _I64, _I64, _I, _P, _I64, _I64, _P,
                                  ctypes.c_size_t, _P], _I),
    "ck4_fp6_bytes": ([_I64, _I64], ctypes.c_size_t),
    "ck4_rotate_quantize_act_fp6": ([_P, _I64, _I64, _I64, _I, _P, _P, _P], _I),
    "ck4_quantize_weight_convrot_fp6": ([_P, _I64, _I64, _I64, _I, _P, _P, _P], _I),
    "ck4_linear_w4a4_fp6": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck4_gemm_w4a4_fp6_acc_i32": ([_P, _P, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck4_gemm_fp6_tile": ([_I64, _I64, _I64, ctypes.POINTER(_I), ctypes.POINTER(_I)], _I),
    "ck4_fp6c_bytes": ([_I64, _I64], ctypes.c_size_t),
    "ck4_rotate_quantize_act_fp6c": ([_P, _I64, _I64, _I64, _I, _P, _P, _P], _I),
    "ck4_quantize_weight_convrot_fp6c": ([_P, _I64, _I64, _I64, _I, _P, _P, _P], _I),
    "ck4_linear_w4a4_fp6c": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck4_gemm_w4a4_fp6c_acc_i32": ([_P, _P, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck4_linear_w4a4_fp6_lora": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck4_linear_w4a4_fp6c_lora": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck4_lora_prepare_down": ([_P, _I64, _I64, _I64, _I, _P, _P], _I),
    "ck4_lora_prepare_up": ([_P, _I64, _I64, _I64, _P, _P], _I),
    "ck4_lora_down": ([_P, _I64, _I64, _I64, _I, _P, _I64, ctypes.c_float, _P, _P], _I),
    "ck4_linear_w4a4_lora": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _I64, _P], _I),
    "ck4_qk_norm_rope": ([*_HEADS * 2, _I64, _I, _I, _I, _P, _P, _P, _I, _I, _PI, _P, _I, _F, *_HEADS * 2, _P], _I),
    "ck4_qk_norm_rope_workspace_bytes": ([_I64, _I], ctypes.c_size_t),
    "ck4_qk_norm_rope_backward": ([*_HEADS * 4, _I64, _I, _I, _I, _P, _P, _P, _I, _I, _PI, _P, _I, _F, *_HEADS * 2, _P, _P,
                                   _P, ctypes.c_size_t, _P], _I),
    "ck4_attention_workspace_bytes": ([_I64, _I64, _I64, _I, _I, _I], ctypes.c_size_t),
    "ck4_attention": ([*_HEADS * 3, _P, _P, _I64, _I64, _I64, _I, _I, _I, _I, _F, *_HEADS, _P, _P, ctypes.c_size_t, _P],
                      _I),
    "ck4_attention_backward_workspace_bytes": ([_I64, _I64, _I64, _I, _I, _I], ctypes.c_size_t),
    "ck4_attention_backward": ([*_HEADS * 5, _P, _P, _P, _I64, _I64, _I64, _I, _I, _I, _I, _F, *_HEADS * 3, _P,
                                ctypes.c_size_t, _P], _I),
    "ck4_attention_decode_workspace_bytes": ([_I64, _I64, _I, _I, _I], ctypes.c_size_t),
    "ck4_attention_decode": ([*_HEADS, _P, _I64, _I64, _I64, _P, _I64, _I64, _I64, _P, _I64, _I64, _I, _I, _I, _F, *_HEADS,
                              _P, _P, ctypes.c_size_t, _P], _I),
}


def lib():
    """The loaded libck4.so (ctypes). Raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"libck4.so not found at {LIB_PATH}: build it with "
                "`python -m int4_w4a4_quantized_amd._build` (there is no fallback path)")
        L = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def version() -> str:
    return lib().ck4_version().decode()


def _check(fn: str, status: int) -> None:
    if status != CK4_OK:
        raise Ck4Error(fn, status, lib().ck4_last_error().decode())


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


# Argument checks. Every wrapper checks types, dtypes, shapes, lengths and
# layouts of all its tensors first and their device last, before it calls the
# library: the kernels derive every buffer extent from m, n and k, so a short or
# mismatched tensor must be refused here rather than read out of bounds.

def _typed(t, dtype, name: str, dims: int | None = None) -> None:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    dtypes = dtype if isinstance(dtype, tuple) else (dtype,)
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims, got shape {tuple(t.shape)}")
    if t.dim() > 0 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have unit stride in its last dim")


def _dense(t, dtype, name: str, dims: int | None = None) -> None:
    """A contiguous tensor (the kernels take its rows back to back)."""
    _typed(t, dtype, name, dims)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _vec(t, dtype, name: str, count: int) -> None:
    """A contiguous vector holding at least `count` elements."""
    _dense(t, dtype, name)
    if t.numel() < count:
        raise ValueError(f"{name} holds {t.numel()} elements, needs at least {count}")


def _on_gpu(**tensors) -> None:
    dev = None
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA (HIP) tensor")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other operands on {dev}")


def _need(t: torch.Tensor, dtype: torch.dtype, name: str, dims: int | None = None) -> None:
    _typed(t, dtype, name, dims)
    _on_gpu(**{name: t})


def _out_checked(out, m: int, n: int, dtype=torch.bfloat16, name: str = "out") -> None:
    _typed(out, dtype, name, 2)
    if tuple(out.shape) != (m, n):
        raise ValueError(f"{name} must have shape {(m, n)}, got {tuple(out.shape)}")


def _fp6_nbytes(rows: int, k: int, compact: bool = False) -> int:
    return (rows + 15) // 16 * 16 * (k // 128) * (64 if compact else 96)


def _fp6_k(q6, name: str, compact: bool = False) -> int:
    """k of an FP6 operand [rows16, 3k/4], or of a compact one [rows16, k/2] (k a multiple of 128)."""
    _dense(q6, torch.uint8, name, 2)
    per = 64 if compact else 96
    if q6.shape[1] % per != 0:
        form = "k/2" if compact else "3k/4"
        raise ValueError(f"{name} has {q6.shape[1]} bytes per row: not {form} for k a multiple of 128")
    return q6.shape[1] * 128 // per


def _out_bf16(m: int, n: int, device) -> torch.Tensor:
    # the kernels store 4 columns per lane: keep the row stride a multiple of 4
    ld = (n + 3) // 4 * 4
    return torch.empty((m, ld), dtype=torch.bfloat16, device=device)[:, :n]


def quantize_weight_convrot(w: torch.Tensor, rot_block: int = 128, group: int = 0):
    """Offline ConvRot weight prep: fp32 [n, k] -> (int8 [n, k/2], fp32 [n] or [n, k/group])."""
    _need(w, torch.float32, "w", 2)
    n, k = w.shape
    wp = torch.empty((n, k // 2), dtype=torch.int8, device=w.device)
    ws = torch.empty((n,) if group == 0 else (n, k // group), dtype=torch.float32, device=w.device)
    _check("ck4_quantize_weight_convrot",
           lib().ck4_quantize_weight_convrot(_ptr(w), n, k, w.stride(0), rot_block, group, _ptr(wp), _ptr(ws),
                                             _stream(w.device)))
    return wp, ws


def quantize_weight_convrot_sr(w: torch.Tensor, u: torch.Tensor, rot_block: int = 128, group: int = 0):
    """Weight prep with stochastic rounding; u fp32 [n, k] holds one draw in [0, 1) per element."""
    _need(w, torch.float32, "w", 2)
    _need(u, torch.float32, "u", 2)
    n, k = w.shape
    wp = torch.empty((n, k // 2), dtype=torch.int8, device=w.device)
    ws = torch.empty((n,) if group == 0 else (n, k // group), dtype=torch.float32, device=w.device)
    _check("ck4_quantize_weight_convrot_sr",
           lib().ck4_quantize_weight_convrot_sr(_ptr(w), n, k, w.stride(0), rot_block, group, _ptr(u), u.stride(0),
                                                _ptr(wp), _ptr(ws), _stream(w.device)))
    return wp, ws


def quantize_weight_convrot_e4m3(w: torch.Tensor, rot_block: int = 128, group: int = 128):
    """Grouped weight prep with E4M3 group scales -> (int8 [n, k/2], uint8 E4M3 bytes [n, k/group])."""
    _need(w, torch.float32, "w", 2)
    n, k = w.shape
    wp = torch.empty((n, k // 2), dtype=torch.int8, device=w.device)
    gs = torch.empty((n, k // group), dtype=torch.uint8, device=w.device)
    _check("ck4_quantize_weight_convrot_e4m3",
           lib().ck4_quantize_weight_convrot_e4m3(_ptr(w), n, k, w.stride(0), rot_block, group, _ptr(wp), _ptr(gs),
                                                  _stream(w.device)))
    return wp, gs


def _codebook(codebook):
    """16 codebook entries (list, numpy array or CPU tensor) -> a host float[16]."""
    if isinstance(codebook, torch.Tensor):
        if codebook.device.type != "cpu":
            raise ValueError("the codebook is a host array of 16 floats")
        codebook = codebook.tolist()
    vals = [float(v) for v in (codebook.tolist() if hasattr(codebook, "tolist") else codebook)]
    if len(vals) != 16:
        raise ValueError(f"the codebook has 16 entries, got {len(vals)}")
    return (ctypes.c_float * 16)(*vals)


def quantize_weight_convrot_codebook(w: torch.Tensor, codebook, rot_block: int = 128, group: int = 128,
                                     scale_e4m3: bool = False):
    """Grouped weight prep against a frozen 16-entry codebook -> (int8 [n, k/2]
    packed indices, group scales fp32 [n, k/group] or uint8 E4M3 bytes)."""
    _need(w, torch.float32, "w", 2)
    n, k = w.shape
    wp = torch.empty((n, k // 2), dtype=torch.int8, device=w.device)
    gs = torch.empty((n, k // group), dtype=torch.uint8 if scale_e4m3 else torch.float32, device=w.device)
    _check("ck4_quantize_weight_convrot_codebook",
           lib().ck4_quantize_weight_convrot_codebook(_ptr(w), n, k, w.stride(0), rot_block, group,
                                                      _codebook(codebook), int(bool(scale_e4m3)), _ptr(wp), _ptr(gs),
                                                      _stream(w.device)))
    return wp, gs


def quantize_weight_convrot_int8(w: torch.Tensor, rot_block: int = 128):
    """Offline W8A8 weight prep: fp32 [n, k] -> (int8 codes [n, k], fp32 row scales [n])."""
    _need(w, torch.float32, "w", 2)
    n, k = w.shape
    wq = torch.empty((n, k), dtype=torch.int8, device=w.device)
    ws = torch.empty((n,), dtype=torch.float32, device=w.device)
    _check("ck4_quantize_weight_convrot_int8",
           lib().ck4_quantize_weight_convrot_int8(_ptr(w), n, k, w.stride(0), rot_block, _ptr(wq), _ptr(ws),
                                                  _stream(w.device)))
    return wq, ws


def rotate_quantize_act(x: torch.Tensor, rot_block: int = 128, bits: int = 4, out=None, scales=None):
    """Dynamic rotate + quantise: bf16 [m, k] -> (int8 [m, k/2] (bits 4) or [m, k] (bits 8), fp32 [m])."""
    _typed(x, torch.bfloat16, "x", 2)
    m, k = x.shape
    if out is not None:
        _dense(out, torch.int8, "out", 2)
        if tuple(out.shape) != (m, k // 2 if bits == 4 else k):
            raise ValueError(f"out must have shape {(m, k // 2 if bits == 4 else k)}, got {tuple(out.shape)}")
    if scales is not None:
        _vec(scales, torch.float32, "scales", m)
    _on_gpu(x=x, out=out, scales=scales)
    if out is None:
        out = torch.empty((m, k // 2 if bits == 4 else k), dtype=torch.int8, device=x.device)
    if scales is None:
        scales = torch.empty((m,), dtype=torch.float32, device=x.device)
    _check("ck4_rotate_quantize_act",
           lib().ck4_rotate_quantize_act(_ptr(x), m, k, x.stride(0), rot_block, bits, _ptr(out), _ptr(scales),
                                         _stream(x.device)))
    return out, scales


def rotate_act_f32(x: torch.Tensor, rot_block: int = 128):
    """fp32 block-Hadamard rotation of bf16 rows: [m, k] -> fp32 [m, k]."""
    _need(x, torch.bfloat16, "x", 2)
    m, k = x.shape
    r = torch.empty((m, k), dtype=torch.float32, device=x.device)
    _check("ck4_rotate_act_f32",
           lib().ck4_rotate_act_f32(_ptr(x), m, k, x.stride(0), rot_block, _ptr(r), _stream(x.device)))
    return r


def _check_gemm(x, w, x_scales, w_scales, bias, out, dtype, what: str):
    """Operands of a GEMM wrapper: x [m, c] and w [n, c] of `dtype`, contiguous,
    with the same row width c; scales and bias long enough; out [m, n] bf16."""
    _dense(x, dtype, "x_" + what, 2)
    _dense(w, dtype, "w_" + what, 2)
    if w.shape[1] != x.shape[1]:
        raise ValueError(f"the weight rows hold {w.shape[1]} bytes, the activation rows {x.shape[1]}: k differs")
    m, n = x.shape[0], w.shape[0]
    if x_scales is not None:
        _vec(x_scales, torch.float32, "x_scales", m)
    if w_scales is not None:
        _vec(w_scales, torch.float32, "w_scales", n)
    if bias is not None:
        _vec(bias, torch.float32, "bias", n)
    if out is not None:
        _out_checked(out, m, n)
    _on_gpu(x=x, w=w, x_scales=x_scales, w_scales=w_scales, bias=bias, out=out)
    return m, n


def linear_w4a4(x_q: torch.Tensor, x_scales: torch.Tensor, w_packed: torch.Tensor, w_scales: torch.Tensor,
                bias: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """y bf16 [m, n] from a quantised activation and a prepared weight."""
    m, n = _check_gemm(x_q, w_packed, x_scales, w_scales, bias, out, torch.int8, "q")
    k = x_q.shape[1] * 2
    if out is None:
        out = _out_bf16(m, n, x_q.device)
    _check("ck4_linear_w4a4",
           lib().ck4_linear_w4a4(_ptr(x_q), _ptr(x_scales), _ptr(w_packed), _ptr(w_scales), _ptr(bias), m, n, k,
                                 _ptr(out), out.stride(0), _stream(x_q.device)))
    return out


def gemm_w4a4_acc_i32(x_q: torch.Tensor, w_packed: torch.Tensor):
    """Exact int32 accumulators [m, n] of the W4A4 GEMM (same kernel, int32 store)."""
    m, n = _check_gemm(x_q, w_packed, None, None, None, None, torch.int8, "q")
    k = x_q.shape[1] * 2
    ldacc = (n + 3) // 4 * 4
    acc = torch.empty((m, ldacc), dtype=torch.int32, device=x_q.device)
    _check("ck4_gemm_w4a4_acc_i32",
           lib().ck4_gemm_w4a4_acc_i32(_ptr(x_q), _ptr(w_packed), m, n, k, _ptr(acc), ldacc, _stream(x_q.device)))
    return acc[:, :n]


def linear_w4a4_bf16(x: torch.Tensor, w_packed: torch.Tensor, w_scales: torch.Tensor, bias=None,
                     rot_block: int = 128, x_q=None, x_scales=None, out=None):
    """The whole layer in one library call: bf16 x [m, k] -> (y bf16 [m, n], x_q int8 [m, k/2], x_scales fp32 [m]).

    Bitwise rotate_quantize_act(x, rot_block, 4) followed by linear_w4a4; for
    m <= 2 (rot_block 128) one kernel does both."""
    _typed(x, torch.bfloat16, "x", 2)
    m, k = x.shape
    _dense(w_packed, torch.int8, "w_packed", 2)
    if w_packed.shape[1] * 2 != k:
        raise ValueError(f"the weight rows hold {w_packed.shape[1]} bytes, not k/2 = {k // 2}")
    n = w_packed.shape[0]
    _vec(w_scales, torch.float32, "w_scales", n)
    if bias is not None:
        _vec(bias, torch.float32, "bias", n)
    if x_q is not None:
        _dense(x_q, torch.int8, "x_q", 2)
        if tuple(x_q.shape) != (m, k // 2):
            raise ValueError(f"x_q must have shape {(m, k // 2)}, got {tuple(x_q.shape)}")
    if x_scales is not None:
        _vec(x_scales, torch.float32, "x_scales", m)
    if out is not None:
        _out_checked(out, m, n)
    _on_gpu(x=x, w_packed=w_packed, w_scales=w_scales, bias=bias, x_q=x_q, x_scales=x_scales, out=out)
    if x_q is None:
        x_q = torch.empty((m, k // 2), dtype=torch.int8, device=x.device)
    if x_scales is None:
        x_scales = torch.empty((m,), dtype=torch.float32, device=x.device)
    if out is None:
        out = _out_bf16(m, n, x.device)
    _check("ck4_linear_w4a4_bf16",
           lib().ck4_linear_w4a4_bf16(_ptr(x), m, k, x.stride(0), rot_block, _ptr(w_packed), _ptr(w_scales),
                                      _ptr(bias), n, _ptr(x_q), _ptr(x_scales), _ptr(out), out.stride(0),
                                      _stream(x.device)))
    return out, x_q, x_scales


def w4a4_linear(x: torch.Tensor, w_packed: torch.Tensor, w_scales: torch.Tensor, bias=None, rot_block: int = 128):
    """The whole layer: rotate + quantise x, then the W4A4 GEMM + epilogue (one library call)."""
    return linear_w4a4_bf16(x, w_packed, w_scales, bias, rot_block)[0]


def dequant_w4a8_grouped(w_packed: torch.Tensor, group_scales: torch.Tensor, group: int = 128, n0: int = 0,
                         nc: int | None = None, codebook=None):
    """Grouped int4 -> int8 decode of weight rows [n0, n0+nc) -> (int8 [nc, k], fp32 [nc]).

    group_scales: fp32, or uint8 holding E4M3 bytes. codebook: the 16 host
    entries the weight was prepared with, or None for plain int4 codes.
    """
    _dense(w_packed, torch.int8, "w_packed", 2)
    n, k = w_packed.shape[0], w_packed.shape[1] * 2
    if nc is None:
        nc = n - n0
    if group <= 0 or k % group != 0:
        raise ValueError(f"group={group} must divide k={k}")
    _vec(group_scales, (torch.float32, torch.uint8), "group_scales", n * (k // group))
    if not (0 <= n0 and 0 < nc and n0 + nc <= n):
        raise ValueError(f"rows [{n0}, {n0 + nc}) are not inside [0, {n})")
    _on_gpu(w_packed=w_packed, group_scales=group_scales)
    w8 = torch.empty((nc, k), dtype=torch.int8, device=w_packed.device)
    sr = torch.empty((nc,), dtype=torch.float32, device=w_packed.device)
    e4m3 = group_scales.dtype == torch.uint8
    if codebook is not None:
        _check("ck4_dequant_w4a8_codebook",
               lib().ck4_dequant_w4a8_codebook(_ptr(w_packed), _ptr(group_scales), int(e4m3), _codebook(codebook), n,
                                               k, group, n0, nc, _ptr(w8), _ptr(sr), _stream(w_packed.device)))
        return w8, sr
    name = "ck4_dequant_w4a8_grouped_e4m3" if e4m3 else "ck4_dequant_w4a8_grouped"
    _check(name, getattr(lib(), name)(_ptr(w_packed), _ptr(group_scales), n, k, group, n0, nc, _ptr(w8), _ptr(sr),
                                      _stream(w_packed.device)))
    return w8, sr


def linear_w8a8(x_q8, x_scales, w8, w_scales, bias=None, out=None):
    """Rowwise int8 linear from int8 activations and int8 weights -> bf16 [m, n]."""
    m, n = _check_gemm(x_q8, w8, x_scales, w_scales, bias, out, torch.int8, "q8")
    k = x_q8.shape[1]
    if out is None:
        out = _out_bf16(m, n, x_q8.device)
    _check("ck4_linear_w8a8",
           lib().ck4_linear_w8a8(_ptr(x_q8), _ptr(x_scales), _ptr(w8), _ptr(w_scales), _ptr(bias), m, n, k,
                                 _ptr(out), out.stride(0), _stream(x_q8.device)))
    return out


def w8a8_linear(x: torch.Tensor, w8: torch.Tensor, w_scales: torch.Tensor, bias=None, rot_block: int = 128):
    """The whole W8A8 ConvRot layer: rotate + int8-quantise x, then the int8 GEMM + epilogue."""
    x_q8, sx = rotate_quantize_act(x, rot_block, 8)
    return linear_w8a8(x_q8, sx, w8, w_scales, bias)


def w4a8_workspace_bytes(m: int, n: int, k: int, chunk_cols: int = 0) -> int:
    return int(lib().ck4_w4a8_workspace_bytes(m, n, k, chunk_cols))


def linear_w4a8_grouped(x_q8, x_scales, w_packed, group_scales, group: int = 128, chunk_cols: int = 0,
                        out=None, workspace=None, codebook=None):
    """Grouped W4A8 linear -> bf16 [m, n].

    chunk_cols > 0: decode per column chunk + int8 GEMM; < 0: one decode pass
    + one GEMM; 0: the library's policy (the fused kernel for m <= 64).
    group_scales: fp32, or uint8 holding E4M3 bytes. codebook: the 16 host
    entries the weight was prepared with, or None.
    """
    _dense(x_q8, torch.int8, "x_q8", 2)
    _dense(w_packed, torch.int8, "w_packed", 2)
    m, k = x_q8.shape
    n = w_packed.shape[0]
    if w_packed.shape[1] * 2 != k:
        raise ValueError(f"w_packed rows hold {w_packed.shape[1]} bytes, the int8 activation has k={k}")
    if group <= 0 or k % group != 0:
        raise ValueError(f"group={group} must divide k={k}")
    _vec(x_scales, torch.float32, "x_scales", m)
    _vec(group_scales, (torch.float32, torch.uint8), "group_scales", n * (k // group))
    if out is not None:
        _out_checked(out, m, n)
    if workspace is not None:
        _dense(workspace, torch.uint8, "workspace")
    _on_gpu(x_q8=x_q8, x_scales=x_scales, w_packed=w_packed, group_scales=group_scales, out=out,
            workspace=workspace)
    if out is None:
        out = _out_bf16(m, n, x_q8.device)
    need = w4a8_workspace_bytes(m, n, k, chunk_cols)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=x_q8.device)
    e4m3 = group_scales.dtype == torch.uint8
    if codebook is not None:
        _check("ck4_linear_w4a8_codebook",
               lib().ck4_linear_w4a8_codebook(_ptr(x_q8), _ptr(x_scales), _ptr(w_packed), _ptr(group_scales),
                                              int(e4m3), _codebook(codebook), m, n, k, group, _ptr(out),
                                              out.stride(0), chunk_cols, _ptr(workspace),
                                              0 if workspace is None else workspace.numel(), _stream(x_q8.device)))
        return out
    name = "ck4_linear_w4a8_grouped_e4m3" if e4m3 else "ck4_linear_w4a8_grouped"
    _check(name, getattr(lib(), name)(_ptr(x_q8), _ptr(x_scales), _ptr(w_packed), _ptr(group_scales), m, n, k,
                                      group, _ptr(out), out.stride(0), chunk_cols, _ptr(workspace),
                                      0 if workspace is None else workspace.numel(), _stream(x_q8.device)))
    return out


def linear_w4a8_grouped_bf16(x: torch.Tensor, w_packed: torch.Tensor, group_scales: torch.Tensor, group: int = 128,
                             rot_block: int = 128, x_q8=None, x_scales=None, out=None, workspace=None):
    """The whole grouped W4A8 layer in one library call: bf16 x [m, k] -> (y bf16 [m, n], x_q8 int8 [m, k],
    x_scales fp32 [m]).

    Bitwise rotate_quantize_act(x, rot_block, 8) followed by linear_w4a8_grouped(..., chunk_cols=0);
    for m = 1 (n <= 8192, rot_block 128, k <= 8192, groups of 32 or more) one kernel does both. group_scales:
    fp32, or uint8 holding E4M3 bytes."""
    _typed(x, torch.bfloat16, "x", 2)
    m, k = x.shape
    _dense(w_packed, torch.int8, "w_packed", 2)
    if w_packed.shape[1] * 2 != k:
        raise ValueError(f"the weight rows hold {w_packed.shape[1]} bytes, not k/2 = {k // 2}")
    n = w_packed.shape[0]
    if group <= 0 or k % group != 0:
        raise ValueError(f"group={group} must divide k={k}")
    _vec(group_scales, (torch.float32, torch.uint8), "group_scales", n * (k // group))
    if x_q8 is not None:
        _dense(x_q8, torch.int8, "x_q8", 2)
        if tuple(x_q8.shape) != (m, k):
            raise ValueError(f"x_q8 must have shape {(m, k)}, got {tuple(x_q8.shape)}")
    if x_scales is not None:
        _vec(x_scales, torch.float32, "x_scales", m)
    if out is not None:
        _out_checked(out, m, n)
    if workspace is not None:
        _dense(workspace, torch.uint8, "workspace")
    _on_gpu(x=x, w_packed=w_packed, group_scales=group_scales, x_q8=x_q8, x_scales=x_scales, out=out,
            workspace=workspace)
    if x_q8 is None:
        x_q8 = torch.empty((m, k), dtype=torch.int8, device=x.device)
    if x_scales is None:
        x_scales = torch.empty((m,), dtype=torch.float32, device=x.device)
    if out is None:
        out = _out_bf16(m, n, x.device)
    need = w4a8_workspace_bytes(m, n, k, 0)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=x.device)
    e4m3 = group_scales.dtype == torch.uint8
    _check("ck4_linear_w4a8_grouped_bf16",
           lib().ck4_linear_w4a8_grouped_bf16(_ptr(x), m, k, x.stride(0), rot_block, _ptr(w_packed),
                                              _ptr(group_scales), int(e4m3), n, group, _ptr(x_q8), _ptr(x_scales),
                                              _ptr(out), out.stride(0), _ptr(workspace),
                                              0 if workspace is None else workspace.numel(), _stream(x.device)))
    return out, x_q8, x_scales


def linear_w4a8_grouped_noalloc(x_q8, x_scales, w_packed, group_scales, group: int = 128, chunk_cols: int = 0,
                                out=None):
    """linear_w4a8_grouped (fp32 group scales) without a workspace: the decode paths use the library's fixed
    device buffer (ck4.h: CK4_NOALLOC_SCRATCH_BYTES per GPU), so the call allocates nothing beyond `out` when
    one is given. Calls that overlap on one GPU race on that buffer."""
    _dense(x_q8, torch.int8, "x_q8", 2)
    _dense(w_packed, torch.int8, "w_packed", 2)
    m, k = x_q8.shape
    n = w_packed.shape[0]
    if w_packed.shape[1] * 2 != k:
        raise ValueError(f"w_packed rows hold {w_packed.shape[1]} bytes, the int8 activation has k={k}")
    if group <= 0 or k % group != 0:
        raise ValueError(f"group={group} must divide k={k}")
    _vec(x_scales, torch.float32, "x_scales", m)
    _vec(group_scales, torch.float32, "group_scales", n * (k // group))
    if out is not None:
        _out_checked(out, m, n)
    _on_gpu(x_q8=x_q8, x_scales=x_scales, w_packed=w_packed, group_scales=group_scales, out=out)
    if out is None:
        out = _out_bf16(m, n, x_q8.device)
    _check("ck4_linear_w4a8_grouped_noalloc",
           lib().ck4_linear_w4a8_grouped_noalloc(_ptr(x_q8), _ptr(x_scales), _ptr(w_packed), _ptr(group_scales), m,
                                                 n, k, group, _ptr(out), out.stride(0), chunk_cols,
                                                 _stream(x_q8.device)))
    return out


def _rows16(n: int) -> int:
    return (n + 15) // 16 * 16


# FP6 operand path (large m): int4 codes held as FP6 E2M3 q / 8 in the MFMA
# operand layout, uint8 [rows16, k * 3 / 4]; bit-identical results to the
# int4 path at twice the matrix rate.

def fp6_bytes(rows: int, k: int) -> int:
    return int(lib().ck4_fp6_bytes(rows, k))


def gemm_fp6_tile(m: int, n: int, k: int):
    """(tile_m, tile_n): the output tile the FP6 GEMM launches for an m x n x k product."""
    tm, tn = ctypes.c_int(0), ctypes.c_int(0)
    _check("ck4_gemm_fp6_tile", lib().ck4_gemm_fp6_tile(m, n, k, ctypes.byref(tm), ctypes.byref(tn)))
    return tm.value, tn.value


def rotate_quantize_act_fp6(x: torch.Tensor, rot_block: int = 128, out=None, scales=None):
    """bf16 [m, k] -> (uint8 [rows16(m), 3k/4] FP6 codes, fp32 [m] scales)."""
    _typed(x, torch.bfloat16, "x", 2)
    m, k = x.shape
    if out is not None:
        _vec(out, torch.uint8, "out", _fp6_nbytes(m, k))
    if scales is not None:
        _vec(scales, torch.float32, "scales", m)
    _on_gpu(x=x, out=out, scales=scales)
    if out is None:
        out = torch.empty((_rows16(m), k * 3 // 4), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((m,), dtype=torch.float32, device=x.device)
    _check("ck4_rotate_quantize_act_fp6",
           lib().ck4_rotate_quantize_act_fp6(_ptr(x), m, k, x.stride(0), rot_block, _ptr(out), _ptr(scales),
                                             _stream(x.device)))
    return out, scales


def quantize_weight_convrot_fp6(w: torch.Tensor, rot_block: int = 128):
    """fp32 [n, k] -> (uint8 [rows16(n), 3k/4] FP6 codes, fp32 [n] row scales)."""
    _need(w, torch.float32, "w", 2)
    n, k = w.shape
    wq = torch.empty((_rows16(n), k * 3 // 4), dtype=torch.uint8, device=w.device)
    ws = torch.empty((n,), dtype=torch.float32, device=w.device)
    _check("ck4_quantize_weight_convrot_fp6",
           lib().ck4_quantize_weight_convrot_fp6(_ptr(w), n, k, w.stride(0), rot_block, _ptr(wq), _ptr(ws),
                                                 _stream(w.device)))
    return wq, ws


def linear_w4a4_fp6(x_q6, x_scales, w_q6, w_scales, bias=None, out=None, m: int | None = None,
                    n: int | None = None):
    """W4A4 GEMM + epilogue from FP6 operands -> bf16 [m, n] (m, n default to the scale lengths)."""
    _typed(x_scales, torch.float32, "x_scales")
    _typed(w_scales, torch.float32, "w_scales")
    m = x_scales.numel() if m is None else m
    n = w_scales.numel() if n is None else n
    k = _check_fp6_gemm(x_q6, w_q6, m, n, x_scales, w_scales, bias, out)
    if out is None:
        out = _out_bf16(m, n, x_q6.device)
    _check("ck4_linear_w4a4_fp6",
           lib().ck4_linear_w4a4_fp6(_ptr(x_q6), _ptr(x_scales), _ptr(w_q6), _ptr(w_scales), _ptr(bias), m, n, k,
                                     _ptr(out), out.stride(0), _stream(x_q6.device)))
    return out


def _check_fp6_gemm(x_q6, w_q6, m: int, n: int, x_scales, w_scales, bias, out, compact: bool = False) -> int:
    """Operands of an FP6 (or compact FP6) GEMM wrapper; returns k."""
    k = _fp6_k(x_q6, "x_q6", compact)
    if _fp6_k(w_q6, "w_q6", compact) != k:
        raise ValueError(f"w_q6 rows hold {w_q6.shape[1]} bytes, x_q6 rows {x_q6.shape[1]}: k differs")
    if m <= 0 or n <= 0:
        raise ValueError("m and n must be positive")
    if x_q6.numel() < _fp6_nbytes(m, k, compact):
        raise ValueError(f"x_q6 holds {x_q6.numel()} bytes, {m} rows need {_fp6_nbytes(m, k, compact)}")
    if w_q6.numel() < _fp6_nbytes(n, k, compact):
        raise ValueError(f"w_q6 holds {w_q6.numel()} bytes, {n} rows need {_fp6_nbytes(n, k, compact)}")
    if x_scales is not None:
        _vec(x_scales, torch.float32, "x_scales", m)
    if w_scales is not None:
        _vec(w_scales, torch.float32, "w_scales", n)
    if bias is not None:
        _vec(bias, torch.float32, "bias", n)
    if out is not None:
        _out_checked(out, m, n)
    _on_gpu(x_q6=x_q6, w_q6=w_q6, x_scales=x_scales, w_scales=w_scales, bias=bias, out=out)
    return k


def gemm_w4a4_fp6_acc_i32(x_q6, w_q6, m: int, n: int):
    """Integer accumulators of the FP6 GEMM -> int32 [m, n]."""
    k = _check_fp6_gemm(x_q6, w_q6, m, n, None, None, None, None)
    acc = torch.empty((m, (n + 3) // 4 * 4), dtype=torch.int32, device=x_q6.device)
    _check("ck4_gemm_w4a4_fp6_acc_i32",
           lib().ck4_gemm_w4a4_fp6_acc_i32(_ptr(x_q6), _ptr(w_q6), m, n, k, _ptr(acc), acc.stride(0),
                                           _stream(x_q6.device)))
    return acc[:, :n]


def w4a4_linear_fp6(x: torch.Tensor, w_q6: torch.Tensor, w_scales: torch.Tensor, bias=None, rot_block: int = 128):
    """The whole layer on the FP6 path: rotate + quantise x to FP6 codes, then the GEMM + epilogue."""
    x_q6, sx = rotate_quantize_act_fp6(x, rot_block)
    return linear_w4a4_fp6(x_q6, sx, w_q6, w_scales, bias)


# Compact FP6 operands: the same images without the two zero exponent bits
# of each code, uint8 [rows16, k / 2] (ck4_fp6c_bytes); expanded in registers
# before the MFMAs, with the FP6 path's results bit for bit.

def fp6c_bytes(rows: int, k: int) -> int:
    return int(lib().ck4_fp6c_bytes(rows, k))


def rotate_quantize_act_fp6c(x: torch.Tensor, rot_block: int = 128, out=None, scales=None):
    """bf16 [m, k] -> (uint8 [rows16(m), k/2] compact FP6 codes, fp32 [m] scales)."""
    _typed(x, torch.bfloat16, "x", 2)
    m, k = x.shape
    if out is not None:
        _vec(out, torch.uint8, "out", _fp6_nbytes(m, k, True))
    if scales is not None:
        _vec(scales, torch.float32, "scales", m)
    _on_gpu(x=x, out=out, scales=scales)
    if out is None:
        out = torch.empty((_rows16(m), k // 2), dtype=torch.uint8, device=x.device)
    if scales is None:
        scales = torch.empty((m,), dtype=torch.float32, device=x.device)
    _check("ck4_rotate_quantize_act_fp6c",
           lib().ck4_rotate_quantize_act_fp6c(_ptr(x), m, k, x.stride(0), rot_block, _ptr(out), _ptr(scales),
                                              _stream(x.device)))
    return out, scales


def quantize_weight_convrot_fp6c(w: torch.Tensor, rot_block: int = 128):
    """fp32 [n, k] -> (uint8 [rows16(n), k/2] compact FP6 codes, fp32 [n] row scales)."""
    _need(w, torch.float32, "w", 2)
    n, k = w.shape
    wq = torch.empty((_rows16(n), k // 2), dtype=torch.uint8, device=w.device)
    ws = torch.empty((n,), dtype=torch.float32, device=w.device)
    _check("ck4_quantize_weight_convrot_fp6c",
           lib().ck4_quantize_weight_convrot_fp6c(_ptr(w), n, k, w.stride(0), rot_block, _ptr(wq), _ptr(ws),
                                                  _stream(w.device)))
    return wq, ws


def linear_w4a4_fp6c(x_q6c, x_scales, w_q6c, w_scales, bias=None, out=None, m: int | None = None,
                     n: int | None = None):
    """W4A4 GEMM + epilogue from compact FP6 operands -> bf16 [m, n]."""
    _typed(x_scales, torch.float32, "x_scales")
    _typed(w_scales, torch.float32, "w_scales")
    m = x_scales.numel() if m is None else m
    n = w_scales.numel() if n is None else n
    k = _check_fp6_gemm(x_q6c, w_q6c, m, n, x_scales, w_scales, bias, out, compact=True)
    if out is None:
        out = _out_bf16(m, n, x_q6c.device)
    _check("ck4_linear_w4a4_fp6c",
           lib().ck4_linear_w4a4_fp6c(_ptr(x_q6c), _ptr(x_scales), _ptr(w_q6c), _ptr(w_scales), _ptr(bias), m, n, k,
                                      _ptr(out), out.stride(0), _stream(x_q6c.device)))
    return out


def gemm_w4a4_fp6c_acc_i32(x_q6c, w_q6c, m: int, n: int):
    """Integer accumulators of the compact FP6 GEMM -> int32 [m, n]."""
    k = _check_fp6_gemm(x_q6c, w_q6c, m, n, None, None, None, None, compact=True)
    acc = torch.empty((m, (n + 3) // 4 * 4), dtype=torch.int32, device=x_q6c.device)
    _check("ck4_gemm_w4a4_fp6c_acc_i32",
           lib().ck4_gemm_w4a4_fp6c_acc_i32(_ptr(x_q6c), _ptr(w_q6c), m, n, k, _ptr(acc), acc.stride(0),
                                            _stream(x_q6c.device)))
    return acc[:, :n]


def w4a4_linear_fp6c(x: torch.Tensor, w_q6c: torch.Tensor, w_scales: torch.Tensor, bias=None, rot_block: int = 128):
    """The whole layer on compact FP6 operands: rotate + quantise, then the GEMM + epilogue."""
    x_q6c, sx = rotate_quantize_act_fp6c(x, rot_block)
    return linear_w4a4_fp6c(x_q6c, sx, w_q6c, w_scales, bias)


def lora_prepare_down(a: torch.Tensor, rot_block: int = 128):
    """Rotated LoRA down projection: fp32 A [rank, k] -> bf16 A R [rank, k] in MFMA fragment order."""
    _need(a, torch.float32, "a", 2)
    rank, k = a.shape
    a_pack = torch.empty((rank, k), dtype=torch.bfloat16, device=a.device)
    _check("ck4_lora_prepare_down",
           lib().ck4_lora_prepare_down(_ptr(a), rank, k, a.stride(0), rot_block, _ptr(a_pack), _stream(a.device)))
    return a_pack


def lora_prepare_up(b: torch.Tensor):
    """LoRA up projection: bf16 B [n, rank] -> fragment order [16 * ceil(n / 16), rank] (zero padding rows)."""
    _need(b, torch.bfloat16, "b", 2)
    n, rank = b.shape
    b_pack = torch.empty((_rows16(n), rank), dtype=torch.bfloat16, device=b.device)
    _check("ck4_lora_prepare_up",
           lib().ck4_lora_prepare_up(_ptr(b), n, rank, b.stride(0), _ptr(b_pack), _stream(b.device)))
    return b_pack


def lora_down(x: torch.Tensor, a_pack: torch.Tensor, alpha: float = 1.0, rot_block: int = 128, out=None):
    """t = bf16(alpha * bf16(x R) (A R)^T) in fragment order [16 * ceil(m / 16), rank], from bf16 x [m, k]."""
    _need(x, torch.bfloat16, "x", 2)
    _need(a_pack, torch.bfloat16, "a_pack", 2)
    m, k = x.shape
    rank = a_pack.shape[0]
    if a_pack.shape[1] != k or not a_pack.is_contiguous():
        raise ValueError("a_pack must be a contiguous [rank, k] tensor")
    if out is None:
        out = torch.empty((_rows16(m), rank), dtype=torch.bfloat16, device=x.device)
    _need(out, torch.bfloat16, "out", 2)
    if tuple(out.shape) != (_rows16(m), rank) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [16 * ceil(m / 16), rank] tensor")
    _check("ck4_lora_down",
           lib().ck4_lora_down(_ptr(x), m, k, x.stride(0), rot_block, _ptr(a_pack), rank, float(alpha), _ptr(out),
                               _stream(x.device)))
    return out


def linear_w4a4_lora(x_q: torch.Tensor, x_scales: torch.Tensor, w_packed: torch.Tensor, w_scales: torch.Tensor,
                     t_pack: torch.Tensor, b_pack: torch.Tensor, bias: torch.Tensor | None = None,
                     out: torch.Tensor | None = None):
    """W4A4 linear with the LoRA up projection in its epilogue: y = base + t B^T, bf16 [m, n].

    t_pack from lora_down, b_pack from lora_prepare_up (both in fragment order)."""
    m, n = _check_gemm(x_q, w_packed, x_scales, w_scales, bias, out, torch.int8, "q")
    k = x_q.shape[1] * 2
    _need(t_pack, torch.bfloat16, "t_pack", 2)
    _need(b_pack, torch.bfloat16, "b_pack", 2)
    rank = t_pack.shape[1]
    if tuple(t_pack.shape) != (_rows16(m), rank) or not t_pack.is_contiguous():
        raise ValueError("t_pack must be a contiguous [16 * ceil(m / 16), rank] tensor")
    if tuple(b_pack.shape) != (_rows16(n), rank) or not b_pack.is_contiguous():
        raise ValueError("b_pack must be a contiguous [16 * ceil(n / 16), rank] tensor")
    if out is None:
        out = _out_bf16(m, n, x_q.device)
    _need(out, torch.bfloat16, "out", 2)
    _check("ck4_linear_w4a4_lora",
           lib().ck4_linear_w4a4_lora(_ptr(x_q), _ptr(x_scales), _ptr(w_packed), _ptr(w_scales), _ptr(bias),
                                      _ptr(t_pack), _ptr(b_pack), rank, m, n, k, _ptr(out), out.stride(0),
                                      _stream(x_q.device)))
    return out


def linear_w4a4_fp6_lora(x_q6: torch.Tensor, x_scales: torch.Tensor, w_q6: torch.Tensor, w_scales: torch.Tensor,
                         t_pack: torch.Tensor, b_pack: torch.Tensor, bias: torch.Tensor | None = None,
                         out: torch.Tensor | None = None):
    """linear_w4a4_lora on the FP6 operand path (same bits): y = base + t B^T, bf16 [m, n]."""
    return _fp6_lora(x_q6, x_scales, w_q6, w_scales, t_pack, b_pack, bias, out, False)


def linear_w4a4_fp6c_lora(x_q6c: torch.Tensor, x_scales: torch.Tensor, w_q6c: torch.Tensor,
                          w_scales: torch.Tensor, t_pack: torch.Tensor, b_pack: torch.Tensor,
                          bias: torch.Tensor | None = None, out: torch.Tensor | None = None):
    """linear_w4a4_lora on compact FP6 operands (same bits): y = base + t B^T, bf16 [m, n]."""
    return _fp6_lora(x_q6c, x_scales, w_q6c, w_scales, t_pack, b_pack, bias, out, True)


def _fp6_lora(x_q6, x_scales, w_q6, w_scales, t_pack, b_pack, bias, out, compact: bool):
    _typed(x_scales, torch.float32, "x_scales")
    _typed(w_scales, torch.float32, "w_scales")
    m, n = x_scales.numel(), w_scales.numel()
    k = _check_fp6_gemm(x_q6, w_q6, m, n, x_scales, w_scales, bias, out, compact=compact)
    _need(t_pack, torch.bfloat16, "t_pack", 2)
    _need(b_pack, torch.bfloat16, "b_pack", 2)
    rank = t_pack.shape[1]
    if tuple(t_pack.shape) != (_rows16(m), rank) or not t_pack.is_contiguous():
        raise ValueError("t_pack must be a contiguous [16 * ceil(m / 16), rank] tensor")
    if tuple(b_pack.shape) != (_rows16(n), rank) or not b_pack.is_contiguous():
        raise ValueError("b_pack must be a contiguous [16 * ceil(n / 16), rank] tensor")
    if out is None:
        out = _out_bf16(m, n, x_q6.device)
    _need(out, torch.bfloat16, "out", 2)
    name = "ck4_linear_w4a4_fp6c_lora" if compact else "ck4_linear_w4a4_fp6_lora"
    _check(name, getattr(lib(), name)(_ptr(x_q6), _ptr(x_scales), _ptr(w_q6), _ptr(w_scales), _ptr(bias),
                                      _ptr(t_pack), _ptr(b_pack), rank, m, n, k, _ptr(out), out.stride(0),
                                      _stream(x_q6.device)))
    return out


def w4a4_lora_linear(x: torch.Tensor, w_packed: torch.Tensor, w_scales: torch.Tensor, a_pack: torch.Tensor,
                     b_pack: torch.Tensor, alpha: float = 1.0, bias=None, rot_block: int = 128):
    """The whole layer with a dynamic LoRA: quantise x, down-project its rotation, GEMM + fused up projection."""
    x_q, sx = rotate_quantize_act(x, rot_block, 4)
    t = lora_down(x, a_pack, alpha, rot_block)
    return linear_w4a4_lora(x_q, sx, w_packed, w_scales, t, b_pack, bias)


def w4a4_lora_linear_fp6(x: torch.Tensor, w_q6: torch.Tensor, w_scales: torch.Tensor, a_pack: torch.Tensor,
                         b_pack: torch.Tensor, alpha: float = 1.0, bias=None, rot_block: int = 128):
    """w4a4_lora_linear on the FP6 operand path (same bits): FP6 codes of x, LoRA down projection, FP6 GEMM with
    the fused up projection."""
    x_q6, sx = rotate_quantize_act_fp6(x, rot_block)
    t = lora_down(x, a_pack, alpha, rot_block)
    return linear_w4a4_fp6_lora(x_q6, sx, w_q6, w_scales, t, b_pack, bias)


def w4a4_lora_linear_fp6c(x: torch.Tensor, w_q6c: torch.Tensor, w_scales: torch.Tensor, a_pack: torch.Tensor,
                          b_pack: torch.Tensor, alpha: float = 1.0, bias=None, rot_block: int = 128):
    """w4a4_lora_linear on compact FP6 operands (same bits): compact codes of x, LoRA down projection, GEMM with
    the fused up projection."""
    x_q6c, sx = rotate_quantize_act_fp6c(x, rot_block)
    t = lora_down(x, a_pack, alpha, rot_block)
    return linear_w4a4_fp6c_lora(x_q6c, sx, w_q6c, w_scales, t, b_pack, bias)


# The attention half of a transformer block, around the projections above.
# Heads are bf16 [tokens, heads, d] tensors with unit stride in d; tokens and
# heads may be strided (views of a fused projection's rows, slices of a joint
# buffer), in multiples of 8 elements from a 16-byte aligned start.
#
# As all calls of this library, these record no autograd history: a result has
# none, whether or not an argument requires a gradient. Gradients are what the
# _backward calls return, from these operators' outputs to their inputs; the
# quantised projections have no gradients.

# These calls run between small kernels at decode sizes, so their checks stay
# at a few attribute reads a tensor.

_BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32


def _heads(t, name: str, shape=None):
    """(pointer, token stride, head stride) of a [tokens, heads, d] tensor of the given shape."""
    if isinstance(t, torch.Tensor) and t.dtype is _BF16 and t.dim() == 3 and (shape is None or t.shape == shape):
        st, sh, sd = t.stride()
        if sd == 1:
            return t.data_ptr(), st, sh
    _typed(t, _BF16, name)
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be [tokens, heads, d] with unit stride in its last dim, got shape {tuple(t.shape)}")


def _given(t, name: str, shape):
    """_heads of an output that the caller gives; None of one that is to be made."""
    return None if t is None else _heads(t, name, shape)


def _new(like):
    """A new tensor like a checked one, and its (pointer, token stride, head stride)."""
    t = torch.empty_like(like)
    st, sh, _ = t.stride()
    return t, (t.data_ptr(), st, sh)


def _exact(t, dtype, name: str, shape) -> int:
    """The pointer of a contiguous tensor of exactly this type and shape."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        _dense(t, dtype, name)
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t.data_ptr()


def _gpu_stream(names: str, *tensors):
    """The current stream of the device that all tensors are on; names: theirs, for what is raised if they are not."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev or dev < 0:
            _on_gpu(**dict(zip(names.split(), tensors)))  # names the one that is not
    return torch._C._cuda_getCurrentRawStream(dev)


@functools.lru_cache(maxsize=64)
def _host_ints(values: tuple):
    """A host array of ints, and their sum."""
    if any(v != ctypes.c_int(v).value for v in values):
        raise ValueError(f"sections must be 32-bit whole numbers, got {values}")
    return (ctypes.c_int * len(values))(*values), sum(values)


def _rope_args(tokens: int, d: int, q_weight, k_weight, positions, freqs, sections):
    """(q_weight, k_weight, positions) pointers, fp32 positions?, axes, the sections as a host array, freqs' pointer."""
    qw = None if q_weight is None else _exact(q_weight, _F32, "q_weight", (d,))
    kw = None if k_weight is None else _exact(k_weight, _F32, "k_weight", (d,))
    if not isinstance(positions, torch.Tensor) or positions.dtype is not _I32 or not positions.is_contiguous():
        _dense(positions, (_I32, _F32), "positions")
    if not isinstance(freqs, torch.Tensor) or freqs.dtype is not _F32 or freqs.dim() != 1 or not freqs.is_contiguous():
        _dense(freqs, _F32, "freqs", 1)
    pairs = freqs.shape[0]
    try:
        secs, total = _host_ints((pairs,) if sections is None else tuple(map(operator.index, sections)))
    except TypeError:
        raise ValueError(f"sections must be whole numbers, one an axis, got {sections!r}") from None
    axes = len(secs)
    if positions.shape != (tokens, axes) and not (axes == 1 and positions.shape == (tokens,)):
        raise ValueError(f"positions must have shape {(tokens, axes)}, got {tuple(positions.shape)}")
    if total != pairs:
        raise ValueError(f"the sections hold {total} pairs, freqs {pairs}")
    if 2 * pairs > d:
        raise ValueError(f"{pairs} rotated pairs do not fit a head of {d}")
    return qw, kw, positions.data_ptr(), positions.dtype is _F32, axes, secs, freqs.data_ptr()


def _qk_shapes(q, k):
    """tokens, hq, hk, d of a norm call, and (pointer, strides) of both tensors."""
    qa, ka = _heads(q, "q"), _heads(k, "k")
    t, hq, d = q.shape
    tk, hk, dk = k.shape
    if tk != t:
        raise ValueError(f"k must have shape {(t, hk, d)}, got {tuple(k.shape)}")
    if dk != d:
        raise ValueError(f"k has heads of {dk}, q of {d}")
    return t, hq, hk, d, qa, ka


def _opt(t):
    return None if t is None else t.data_ptr()


def qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight, k_weight, positions: torch.Tensor, freqs: torch.Tensor,
                 sections=None, interleaved: bool = True, eps: float = 1e-6, q_out=None, k_out=None):
    """RMS norm of every query and key head with the rotary rotation, in one pass.

    q [tokens, hq, d], k [tokens, hk, d] bf16; q_weight, k_weight fp32 [d] or
    None (ones); positions int32 or fp32 [tokens, axes] (or [tokens]); freqs
    fp32 [pairs], the angle per position step of every rotated pair; sections:
    how many pairs follow each axis, in order (default: all follow one).
    interleaved: pairs (2j, 2j + 1), else (j, j + pairs); elements past the
    pairs are normalised only. Returns (q_out, k_out), bf16; q_out and k_out
    may be given, also as q and k themselves. No autograd history is recorded:
    gradients are qk_norm_rope_backward's.
    """
    t, hq, hk, d, qa, ka = _qk_shapes(q, k)
    qw, kw, pos, pos_f32, axes, secs, fr = _rope_args(t, d, q_weight, k_weight, positions, freqs, sections)
    qo, ko = _given(q_out, "q_out", q.shape), _given(k_out, "k_out", k.shape)
    stream = _gpu_stream("q k q_weight k_weight positions freqs q_out k_out", q, k, q_weight, k_weight, positions, freqs,
                         q_out, k_out)
    if qo is None:
        q_out, qo = _new(q)
    if ko is None:
        k_out, ko = _new(k)
    _check("ck4_qk_norm_rope",
           lib().ck4_qk_norm_rope(*qa, *ka, t, hq, hk, d, qw, kw, pos, pos_f32, axes, secs, fr, bool(interleaved), eps,
                                  *qo, *ko, stream))
    return q_out, k_out


def _workspace(workspace, need: int, like):
    """The caller's workspace, or a new one (None where none is needed)."""
    return like.new_empty(need, dtype=torch.uint8) if workspace is None and need else workspace


def _extent(workspace):
    """(pointer, bytes) of a workspace; none for sizes that need none, or that the library refuses."""
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())


def qk_norm_rope_backward(dq_out: torch.Tensor, dk_out: torch.Tensor, q: torch.Tensor, k: torch.Tensor, q_weight, k_weight,
                          positions: torch.Tensor, freqs: torch.Tensor, sections=None, interleaved: bool = True,
                          eps: float = 1e-6, dq=None, dk=None, workspace=None):
    """Gradients of qk_norm_rope: its arguments, and the gradients of its
    outputs. Returns (dq, dk, dq_weight, dk_weight), bf16 heads and fp32 [d]
    (None for a weight that is None). dq may be dq_out or q, dk likewise.
    workspace: uint8, ck4_qk_norm_rope_workspace_bytes (default: allocated here)."""
    t, hq, hk, d, qa, ka = _qk_shapes(q, k)
    dqo, dko = _heads(dq_out, "dq_out", q.shape), _heads(dk_out, "dk_out", k.shape)
    qw, kw, pos, pos_f32, axes, secs, fr = _rope_args(t, d, q_weight, k_weight, positions, freqs, sections)
    dqa, dka = _given(dq, "dq", q.shape), _given(dk, "dk", k.shape)
    if workspace is not None:
        _dense(workspace, torch.uint8, "workspace")
    stream = _gpu_stream("dq_out dk_out q k q_weight k_weight positions freqs dq dk workspace", dq_out, dk_out, q, k,
                         q_weight, k_weight, positions, freqs, dq, dk, workspace)
    if dqa is None:
        dq, dqa = _new(q)
    if dka is None:
        dk, dka = _new(k)
    L = lib()
    workspace = _workspace(workspace, L.ck4_qk_norm_rope_workspace_bytes(t, d), q)
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    _check("ck4_qk_norm_rope_backward",
           L.ck4_qk_norm_rope_backward(*dqo, *dko, *qa, *ka, t, hq, hk, d, qw, kw, pos, pos_f32, axes, secs, fr,
                                       bool(interleaved), eps, *dqa, *dka, _opt(dqw), _opt(dkw), *_extent(workspace),
                                       stream))
    return dq, dk, dqw, dkw


def _qkv(q, k, v):
    """(pointer, strides) of the three operands of an attention call."""
    qa, ka = _heads(q, "q"), _heads(k, "k")
    va = _heads(v, "v", k.shape)
    if k.shape[2] != q.shape[2]:
        raise ValueError(f"k has heads of {k.shape[2]}, q of {q.shape[2]}")
    return qa, ka, va


def _cu(cu_q, cu_k):
    """The number of packed sequences."""
    if cu_q is None and cu_k is None:
        return 1
    for name, cu in (("cu_q", cu_q), ("cu_k", cu_k)):
        if not isinstance(cu, torch.Tensor) or cu.dtype is not _I32 or cu.dim() != 1 or not cu.is_contiguous():
            _dense(cu, _I32, name, 1)
    if cu_q.shape != cu_k.shape or cu_q.shape[0] < 2:
        raise ValueError(f"cu_q and cu_k must hold one start more than there are sequences, got {cu_q.shape[0]} and "
                         f"{cu_k.shape[0]}")
    return cu_q.shape[0] - 1


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q=None, cu_k=None, causal: bool = False, scale=None,
              out=None, lse=None, workspace=None):
    """Softmax attention over packed sequences, with grouped heads.

    q [tq, hq, d], k and v [tk, hk, d] bf16, hq a multiple of hk, d a multiple
    of 8 up to 128. cu_q, cu_k int32 [sequences + 1] on the GPU: sequence i
    owns the rows [cu_q[i], cu_q[i + 1]) of q and [cu_k[i], cu_k[i + 1]) of k
    and v, from 0 to tq and tk (default: one sequence of all rows). Causal: row i of a
    sequence with nq queries and nk keys sees the keys j <= i + nk - nq.
    scale: default 1 / sqrt(d). Returns (out bf16 [tq, hq, d], lse fp32
    [hq, tq]): lse is the log-sum-exp of a row's scaled scores, which the
    backward pass takes. A row that sees nothing has out 0 and lse -inf. No
    autograd history is recorded: gradients are attention_backward's.
    workspace: uint8, ck4_attention_workspace_bytes (default: allocated here
    where that is not 0).
    """
    qa, ka, va = _qkv(q, k, v)
    tq, hq, d = q.shape
    seqs = _cu(cu_q, cu_k)
    tk, hk, _ = k.shape
    L = lib()
    oa = _given(out, "out", q.shape)
    if lse is not None:
        _exact(lse, _F32, "lse", (hq, tq))
    if workspace is not None:
        _dense(workspace, torch.uint8, "workspace")
    stream = _gpu_stream("q k v cu_q cu_k out lse workspace", q, k, v, cu_q, cu_k, out, lse, workspace)
    if oa is None:
        out, oa = _new(q)
    if lse is None:
        lse = q.new_empty((hq, tq), dtype=_F32)
    workspace = _workspace(workspace, L.ck4_attention_workspace_bytes(seqs, tq, tk, hq, hk, d), q)
    _check("ck4_attention",
           L.ck4_attention(*qa, *ka, *va, _opt(cu_q), _opt(cu_k), seqs, tq, tk, hq, hk, d, bool(causal),
                           d ** -0.5 if scale is None else scale, *oa, lse.data_ptr(), *_extent(workspace),
                           stream))
    return out, lse


def attention_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, out: torch.Tensor,
                       lse: torch.Tensor, cu_q=None, cu_k=None, causal: bool = False, scale=None, dq=None, dk=None,
                       dv=None, workspace=None):
    """Gradients of attention: its arguments, its results out and lse, and the
    gradient of out. Returns (dq, dk, dv) bf16; the gradients of query heads
    that share a key head are summed in fp32. The same inputs give the same
    bits. workspace: uint8, ck4_attention_backward_workspace_bytes (default:
    allocated here)."""
    qa, ka, va = _qkv(q, k, v)
    tq, hq, d = q.shape
    seqs = _cu(cu_q, cu_k)
    ga, oa, la = _heads(dout, "dout", q.shape), _heads(out, "out", q.shape), _exact(lse, _F32, "lse", (hq, tq))
    dqa, dka, dva = _given(dq, "dq", q.shape), _given(dk, "dk", k.shape), _given(dv, "dv", k.shape)
    if workspace is not None:
        _dense(workspace, torch.uint8, "workspace")
    stream = _gpu_stream("dout q k v out lse cu_q cu_k dq dk dv workspace", dout, q, k, v, out, lse, cu_q, cu_k, dq, dk, dv,
                         workspace)
    if dqa is None:
        dq, dqa = _new(q)
    if dka is None:
        dk, dka = _new(k)
    if dva is None:
        dv, dva = _new(v)
    L = lib()
    tk, hk, _ = k.shape
    workspace = _workspace(workspace, L.ck4_attention_backward_workspace_bytes(seqs, tq, tk, hq, hk, d), q)
    _check("ck4_attention_backward",
           L.ck4_attention_backward(*ga, *qa, *ka, *va, *oa, la, _opt(cu_q), _opt(cu_k), seqs, tq, tk, hq, hk, d,
                                    bool(causal), d ** -0.5 if scale is None else scale, *dqa, *dka, *dva,
                                    *_extent(workspace), stream))
    return dq, dk, dv


def attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, lengths: torch.Tensor, scale=None,
                     out=None, lse=None, workspace=None):
    """Attention of one new token per sequence over a key/value cache.

    q [batch, hq, d] bf16; k_cache, v_cache [batch, slots, hk, d] bf16 with
    unit stride in d, otherwise strided in multiples of 8; lengths int32
    [batch] on the GPU: the filled slots of each sequence, from slot 0 on
    (what the other slots hold, NaN included, does not matter). Returns (out
    bf16 [batch, hq, d], lse fp32 [hq, batch]); a sequence of length 0 has out
    0 and lse -inf. No autograd history is recorded, and there are no gradients.
    workspace: uint8, ck4_attention_decode_workspace_bytes (default: allocated
    here where that is not 0).
    """
    qa = _heads(q, "q")
    b, hq, d = q.shape
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        _typed(c, _BF16, name, 4)
    _, slots, hk, _ = k_cache.shape
    if k_cache.shape != (b, slots, hk, d) or v_cache.shape != k_cache.shape:
        raise ValueError(f"k_cache and v_cache must be [{b}, slots, hk, {d}], got {tuple(k_cache.shape)} and "
                         f"{tuple(v_cache.shape)}")
    na = _exact(lengths, _I32, "lengths", (b,))
    oa = _given(out, "out", q.shape)
    if lse is not None:
        _exact(lse, _F32, "lse", (hq, b))
    if workspace is not None:
        _dense(workspace, torch.uint8, "workspace")
    stream = _gpu_stream("q k_cache v_cache lengths out lse workspace", q, k_cache, v_cache, lengths, out, lse, workspace)
    if oa is None:
        out, oa = _new(q)
    if lse is None:
        lse = q.new_empty((hq, b), dtype=_F32)
    L = lib()
    workspace = _workspace(workspace, L.ck4_attention_decode_workspace_bytes(b, slots, hq, hk, d), q)
    ks, vs = k_cache.stride(), v_cache.stride()
    _check("ck4_attention_decode",
           L.ck4_attention_decode(*qa, k_cache.data_ptr(), ks[0], ks[1], ks[2], v_cache.data_ptr(), vs[0], vs[1], vs[2], na,
                                  b, slots, hq, hk, d, d ** -0.5 if scale is None else scale, *oa, lse.data_ptr(),
                                  *_extent(workspace), stream))
    return out, lse
