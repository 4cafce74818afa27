"""Fused randomized Hadamard rotation + 4-bit quantization of activations (B200).

Thin ctypes binding over the C ABI in include/kq.h (libkq.so, built in-tree by
`python -m hadamard_rotated_activation_b200.build`).  Functions carry the C
names and only marshal arguments: torch CUDA tensors become device pointers and
the current torch stream becomes the kq stream.  Every step of the path runs in
the library's CUDA kernels; there is no other implementation here, and a
missing library is an error.  The decode-step calls, which are short, are
marshalled by a small extension module (csrc/kq_call.c) when nothing is wrong
with their arguments, and by the functions below otherwise.

PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libkq.so")

KQ_OK = 0
KQ_ERR_INVALID_ARG = -1
KQ_ERR_UNSUPPORTED = -2
KQ_ERR_MISALIGNED = -3
KQ_ERR_CUDA = -4

KQ_F32 = 0
KQ_BF16 = 1

KQ_INVERSE = 1
KQ_SCALE_STATIC = 2
KQ_SCALE_DYNAMIC = 4
KQ_SCALES_MMA = 8
KQ_DYN_STATS = 16
KQ_DYN_EXACT = 32
KQ_DYN_QUANT = 64

KQ_FMT_INT4_SYM = 0
KQ_FMT_INT4_ASYM = 1
KQ_FMT_NVFP4 = 2
KQ_FMT_MXFP4 = 3

C_SYMBOLS = (
    "kq_rht", "kq_rht_quant_int4", "kq_rht_quant_nvfp4", "kq_dequant",
    "kq_dequant_rht_inverse", "kq_rht_quant_mxfp4", "kq_rht_quant_int4_kv",
    "kq_device_errors", "kq_diag_wait_timeout",
    "kq_workspace_size", "kq_status_str", "kq_last_cuda_error", "kq_version",
    "kq_rht_quant_nvfp4_dynamic_noalloc", "kq_diag_tc_steps", "kq_diag_fail_next_launch",
    "kq_gemm_nvfp4", "kq_diag_tc_steps_f16",
    "kq_gemv", "kq_attn_decode_int4_kv", "kq_attn_workspace_size", "kq_kv_copy_pages",
)

# Fixed device scratch of kq_rht_quant_nvfp4_dynamic_noalloc (see include/kq.h).
KQ_NOALLOC_SCRATCH_BYTES = 1 << 20
KQ_NOALLOC_MAX_TOKENS = (KQ_NOALLOC_SCRATCH_BYTES - 16) // 8

# Limits of kq_gemv (see include/kq.h).
KQ_GEMV_MAX_TOKENS = 16
KQ_GEMV_MAX_K = 131072

_lib = None


class KQError(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = f"{where}: {status_str(status)} ({status})"
        if status == KQ_ERR_CUDA:
            msg += f", cuda error {lib().kq_last_cuda_error()}"
        super().__init__(msg)
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libkq.so (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m hadamard_rotated_activation_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    L.kq_rht.argtypes = [vp, i32, i64, i32, i32, vp, vp, i32, vp]
    L.kq_rht.restype = i32
    L.kq_rht_quant_int4.argtypes = [vp, i32, i64, i32, i32, vp, i32, i32, vp, vp, vp, vp]
    L.kq_rht_quant_int4.restype = i32
    L.kq_rht_quant_nvfp4.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, vp, vp, sz, i32, vp]
    L.kq_rht_quant_nvfp4.restype = i32
    L.kq_dequant.argtypes = [i32, vp, vp, vp, vp, i64, i32, i32, vp, vp]
    L.kq_dequant.restype = i32
    L.kq_rht_quant_mxfp4.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp, vp]
    L.kq_rht_quant_mxfp4.restype = i32
    L.kq_rht_quant_int4_kv.argtypes = [vp, i32, i64, i32, i32, vp, i32, vp, i64, vp, vp, vp, vp]
    L.kq_rht_quant_int4_kv.restype = i32
    L.kq_device_errors.argtypes = [vp]
    L.kq_device_errors.restype = i32
    L.kq_diag_wait_timeout.argtypes = [ctypes.c_longlong, vp]
    L.kq_diag_wait_timeout.restype = i32
    L.kq_dequant_rht_inverse.argtypes = [i32, vp, vp, vp, vp, i64, i32, i32, i32, vp, vp, i32,
                                         vp]
    L.kq_dequant_rht_inverse.restype = i32
    L.kq_rht_quant_nvfp4_dynamic_noalloc.argtypes = [vp, i32, i64, i32, i32, vp, vp, vp,
                                                     vp, vp]
    L.kq_rht_quant_nvfp4_dynamic_noalloc.restype = i32
    L.kq_workspace_size.argtypes = [i64, i32, i32]
    L.kq_workspace_size.restype = sz
    L.kq_status_str.argtypes = [i32]
    L.kq_status_str.restype = ctypes.c_char_p
    L.kq_last_cuda_error.argtypes = []
    L.kq_last_cuda_error.restype = i32
    L.kq_version.argtypes = []
    L.kq_version.restype = i32
    L.kq_diag_tc_steps.argtypes = [vp, vp, vp, vp, vp, vp]
    L.kq_diag_tc_steps.restype = i32
    L.kq_diag_fail_next_launch.argtypes = [i32]
    L.kq_diag_fail_next_launch.restype = None
    L.kq_diag_tc_steps_f16.argtypes = [vp, vp, vp, vp, vp, vp]
    L.kq_diag_tc_steps_f16.restype = i32
    L.kq_gemm_nvfp4.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, vp, i32, vp]
    L.kq_gemm_nvfp4.restype = i32
    L.kq_gemv.argtypes = [i32, vp, i32, i64, vp, vp, vp, vp, i64, i32, i32, vp, i32, vp]
    L.kq_gemv.restype = i32
    L.kq_attn_decode_int4_kv.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp, vp, i64,
                                         vp, i64, i32, vp, i32, i32, ctypes.c_float, vp, vp, sz,
                                         vp]
    L.kq_attn_decode_int4_kv.restype = i32
    L.kq_attn_workspace_size.argtypes = [i64, i32, i32]
    L.kq_attn_workspace_size.restype = sz
    L.kq_kv_copy_pages.argtypes = [vp, i64, i32, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    L.kq_kv_copy_pages.restype = i32
    _lib = L
    return L


def status_str(status: int) -> str:
    return lib().kq_status_str(int(status)).decode()


# ------------------------------------------------------------ marshalling
def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("kq functions take CUDA tensors (device pointers)")
    if not t.is_contiguous():
        raise ValueError("kq functions take contiguous tensors")
    return t.data_ptr()


def _stream(stream) -> Optional[int]:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _dtype_code(x) -> int:
    import torch
    if x.dtype == torch.bfloat16:
        return KQ_BF16
    if x.dtype == torch.float32:
        return KQ_F32
    raise ValueError(f"unsupported input dtype {x.dtype}")


def _check(status: int, where: str) -> None:
    if status != KQ_OK:
        raise KQError(status, where)


# -------------------------------------------------------------- C names
def kq_rht(x, block: int, signs, out, inverse: bool = False, stream=None) -> None:
    """Rotation only (fp32 out): forward y = x D H^T / sqrt(b), or the inverse."""
    t, n = x.shape
    _check(lib().kq_rht(_ptr(x), _dtype_code(x), t, n, block, _ptr(signs), _ptr(out),
                        KQ_INVERSE if inverse else 0, _stream(stream)), "kq_rht")


def kq_rht_quant_int4(x, block: int, signs, group: int, asym: bool, codes, scales,
                      zeros=None, stream=None) -> None:
    """Rotation + INT4: symmetric per token (group 0, fp32 scales) or
    asymmetric per group of 128 (fp16 scales and zero-points)."""
    t, n = x.shape
    _check(lib().kq_rht_quant_int4(_ptr(x), _dtype_code(x), t, n, block, _ptr(signs),
                                   group, 1 if asym else 0, _ptr(codes), _ptr(scales),
                                   _ptr(zeros), _stream(stream)), "kq_rht_quant_int4")


def kq_rht_quant_nvfp4(x, block: int, signs, codes, block_scales, tensor_scale,
                       workspace=None, dynamic: bool = True, stream=None,
                       mma_layout: bool = False, phases: int = 0) -> None:
    """Rotation + NVFP4 (E2M1 codes, E4M3 scale per 16, fp32 tensor scale).
    dynamic=True computes and writes the tensor scale (needs `workspace` of
    kq_workspace_size bytes); dynamic=False reads it.  mma_layout=True writes
    the block scales in the tensor-core layout kq_gemm_nvfp4 reads (a buffer
    of sf_mma_bytes(tokens, dim) bytes)."""
    t, n = x.shape
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    flags = ((KQ_SCALE_DYNAMIC if dynamic else KQ_SCALE_STATIC) |
             (KQ_SCALES_MMA if mma_layout else 0) | phases)
    _check(lib().kq_rht_quant_nvfp4(_ptr(x), _dtype_code(x), t, n, block, _ptr(signs),
                                    _ptr(codes), _ptr(block_scales), _ptr(tensor_scale),
                                    _ptr(workspace), ws_bytes, flags, _stream(stream)),
           "kq_rht_quant_nvfp4")


def kq_rht_quant_int4_kv(x, signs, slot_mapping, codes_cache, scales_cache, zeros_cache,
                         stream=None) -> None:
    """Rotation (per-head H_128) + asymmetric INT4 g128 into KV-cache rows:
    token t lands in row slot_mapping[t] (int64; negative = skip)."""
    t, n = x.shape
    _check(lib().kq_rht_quant_int4_kv(_ptr(x), _dtype_code(x), t, n, 128, _ptr(signs), 128,
                                      _ptr(slot_mapping), codes_cache.shape[0],
                                      _ptr(codes_cache), _ptr(scales_cache), _ptr(zeros_cache),
                                      _stream(stream)),
           "kq_rht_quant_int4_kv")


def kq_rht_quant_mxfp4(x, block: int, signs, codes, scales, stream=None) -> None:
    """Rotation + MXFP4 (E2M1 codes, one E8M0 scale byte per 32 elements)."""
    t, n = x.shape
    _check(lib().kq_rht_quant_mxfp4(_ptr(x), _dtype_code(x), t, n, block, _ptr(signs),
                                    _ptr(codes), _ptr(scales), _stream(stream)),
           "kq_rht_quant_mxfp4")


def kq_rht_quant_nvfp4_dynamic_noalloc(x, block: int, signs, codes, block_scales,
                                       tensor_scale, stream=None) -> None:
    """Dynamic-scale NVFP4 for callers that cannot allocate device memory: the
    workspace is the library's own fixed device array (at most
    KQ_NOALLOC_MAX_TOKENS rows).  Calls that overlap on the GPU race."""
    t, n = x.shape
    _check(lib().kq_rht_quant_nvfp4_dynamic_noalloc(
        _ptr(x), _dtype_code(x), t, n, block, _ptr(signs), _ptr(codes), _ptr(block_scales),
        _ptr(tensor_scale), _stream(stream)), "kq_rht_quant_nvfp4_dynamic_noalloc")


def sharded_dynamic_protocol(run_phase, lower, gmax, all_reduce_max, empty: bool) -> None:
    """The order of a sharded dynamic NVFP4 call on one rank: phase 1, MAX
    over the ranks of the lower bound (`lower`, the workspace's bytes 0-3 as
    int32), phase 2, MAX of the exact maximum (`gmax`, bytes 8-15 as int64),
    phase 3.  Every rank takes both collectives, a rank with no rows too (it
    contributes zeros).  run_phase(flag) runs one phase of the library."""
    if empty:
        lower.zero_()
        gmax.zero_()
    else:
        run_phase(KQ_DYN_STATS)
    all_reduce_max(lower)
    if not empty:
        run_phase(KQ_DYN_EXACT)
    all_reduce_max(gmax)
    if not empty:
        run_phase(KQ_DYN_QUANT)


def nvfp4_dynamic_sharded(x, block: int, signs, codes, block_scales, tensor_scale, workspace,
                          all_reduce_max, stream=None, mma_layout: bool = False) -> None:
    """Dynamic NVFP4 of a tensor whose rows are split over ranks: every rank
    gets the tensor scale of the whole tensor (the single-call result).
    all_reduce_max(t) reduces a one-element int32 or int64 device tensor in
    place with MAX over the ranks (torch.distributed.all_reduce with
    ReduceOp.MAX, say).  See kq_rht_quant_nvfp4 in include/kq.h."""
    torch = _torch()
    ws8 = workspace.view(-1)

    def run(flag):
        kq_rht_quant_nvfp4(x, block, signs, codes, block_scales, tensor_scale, workspace, True,
                           stream=stream, mma_layout=mma_layout, phases=flag)
    sharded_dynamic_protocol(run, ws8[0:4].view(torch.int32), ws8[8:16].view(torch.int64),
                             all_reduce_max, x.shape[0] == 0)


_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def kq_gemm_nvfp4(a_codes, a_scales, a_tensor_scale, b_codes, b_scales, b_tensor_scale, c,
                  stream=None) -> None:
    """C = ta tb A_q B_q^T on the block-scaled tensor cores: A [m, k/2] and B
    [n, k/2] packed E2M1 codes with block scales in the tensor-core layout
    (kq_rht_quant_nvfp4(..., mma_layout=True)); C [m, n] fp32 or bf16."""
    m, kb = a_codes.shape
    n = b_codes.shape[0]
    _check(lib().kq_gemm_nvfp4(_ptr(a_codes), _ptr(a_scales), _ptr(a_tensor_scale),
                               _ptr(b_codes), _ptr(b_scales), _ptr(b_tensor_scale), m, n,
                               2 * kb, _ptr(c), _dtype_code(c), _stream(stream)),
           "kq_gemm_nvfp4")


# ------------------------------------------------- decode-step operators
# These calls are short (a few microseconds of GPU work), so their marshalling
# asks each tensor only what the kernels rely on, and a native module does it
# for calls that are right: it returns the status, or None, having called
# nothing, for all others (and for all calls where it was not built).
_call = None


class _PythonOnly:
    """In place of the module where it was not built: every call is left to Python."""

    @staticmethod
    def gemv(*args):
        return None

    attn = copy = gemv


def _native():
    """The marshalling module, loaded and told of the library (once)."""
    global _call
    if _call is None:
        import importlib
        L, torch = lib(), _torch()
        try:
            mod = importlib.import_module("._kq_call", __name__)
        except ImportError as e:
            import warnings
            warnings.warn(f"the _kq_call extension module is missing ({e}): decode-step calls take "
                          "a few microseconds more; build it with "
                          "`python -m hadamard_rotated_activation_b200.build`", RuntimeWarning)
            _call = _PythonOnly
            return _call
        mod.init(torch.bfloat16, torch.float32, torch.float16, torch.uint8, torch.int8,
                 torch.int32, torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice,
                 *[ctypes.cast(f, ctypes.c_void_p).value
                   for f in (L.kq_gemv, L.kq_attn_decode_int4_kv, L.kq_kv_copy_pages)])
        _call = mod
    return _call


def _want(t, what: str, dtype, shape, index: int) -> int:
    """Device pointer of a contiguous tensor of this type and shape on device
    `index`; ValueError for anything else.  The kernels take sizes from the
    shapes, so a wrong one would read or write out of bounds."""
    if t is None:
        raise ValueError(f"{what}: missing")
    if t.dtype is dtype and t.shape == shape and t.get_device() == index >= 0 \
            and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda:
        raise ValueError(f"{what}: kq functions take CUDA tensors (device pointers)")
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{what}: expected {dtype} {list(shape)}, "
                         f"got {t.dtype} {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: kq functions take contiguous tensors")
    raise ValueError(f"{what}: on cuda:{t.get_device()}, the call's tensors are on cuda:{index}")


def _there(**arguments) -> None:
    """ValueError for a missing tensor or cache."""
    for name, a in arguments.items():
        if a is None:
            raise ValueError(f"{name}: missing")


def _int32(**sizes) -> None:
    """ValueError for a size that the C entry's 32 bits would cut."""
    for name, v in sizes.items():
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{name}: {v} does not fit 32 bits")


def _launch(fn, where: str, index: int, stream, *args) -> None:
    """fn(*args, stream) with device `index` current; its current stream when
    none is given."""
    torch = _torch()
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(index)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != KQ_OK:
        raise KQError(status, where)


def kq_gemv(fmt: int, x, codes, scales, zeros, tensor_scale, group: int, y,
            stream=None) -> None:
    """y = x W^T for a few tokens: x [m, k] (m <= KQ_GEMV_MAX_TOKENS), W [n, k]
    in a 4-bit format as kq_dequant takes it, y [m, n]; x and y fp32 or bf16."""
    status = (_call or _native()).gemv(fmt, x, codes, scales, zeros, tensor_scale, group, y,
                                       stream)
    if status is None:
        _gemv_checked(fmt, x, codes, scales, zeros, tensor_scale, group, y, stream)
    elif status != KQ_OK:
        raise KQError(status, "kq_gemv")


def _gemv_checked(fmt, x, codes, scales, zeros, tensor_scale, group, y, stream) -> None:
    torch = _torch()
    _there(x=x, codes=codes, y=y)
    if x.dim() != 2 or codes.dim() != 2:
        raise ValueError("x is [m, k] and codes are [n, k/2]")
    (m, k), n, at = x.shape, codes.shape[0], x.get_device()
    if (k | group | fmt) >> 31:
        _int32(k=k, group=group, fmt=fmt)
    z = t = None
    if fmt == KQ_FMT_INT4_ASYM:
        s = _want(scales, "scales", torch.float16, (n, k // 128), at)
        z = _want(zeros, "zeros", torch.float16, (n, k // 128), at)
    elif fmt == KQ_FMT_INT4_SYM:
        s = _want(scales, "scales", torch.float32, (n,), at)
    elif fmt == KQ_FMT_NVFP4:
        s = _want(scales, "scales", torch.uint8, (n, k // 16), at)
        t = _want(tensor_scale, "tensor_scale", torch.float32, (1,), at)
    else:
        s = _want(scales, "scales", torch.uint8, (n, k // 32), at)
    _launch((_lib or lib()).kq_gemv, "kq_gemv", at, stream, fmt,
            _want(x, "x", x.dtype, (m, k), at), _dtype_code(x), m,
            _want(codes, "codes", torch.uint8, (n, k // 2), at), s, z, t, n, k, group,
            _want(y, "y", y.dtype, (m, n), at), _dtype_code(y))


class KVCacheInt4:
    """The three arrays of a paged INT4 cache (keys or values) as
    kq_rht_quant_int4_kv writes them: codes uint8 [num_slots, dim/2], scales
    and zeros fp16 [num_slots, dim/128]; with one more leading dimension a
    cache of several layers.  A view of the caller's tensors, which have to stay
    what they are: a call with a cache whose arrays were resized, or given other
    memory of another shape, type or place since, is refused with ValueError."""

    __slots__ = ("_view",)
    codes = property(lambda self: self._view[0])
    scales = property(lambda self: self._view[1])
    zeros = property(lambda self: self._view[2])
    layers = property(lambda self: self._view[3])
    num_slots = property(lambda self: self._view[4])
    dim = property(lambda self: self._view[5])
    index = property(lambda self: self._view[6])
    layered = property(lambda self: self._view[7])

    def __init__(self, codes, scales, zeros):
        torch = _torch()
        _there(codes=codes)
        if codes.dim() not in (2, 3):
            raise ValueError("codes are [num_slots, dim/2] or [layers, num_slots, dim/2]")
        lead, half, at = tuple(codes.shape[:-1]), codes.shape[-1], codes.get_device()
        if half % 64 != 0 or half == 0:
            raise ValueError(f"codes: {half} bytes a row are not whole 128-wide heads")
        _want(codes, "codes", torch.uint8, lead + (half,), at)
        _want(scales, "scales", torch.float16, lead + (half // 64,), at)
        _want(zeros, "zeros", torch.float16, lead + (half // 64,), at)
        layered = len(lead) == 2
        self._view = (codes, scales, zeros, lead[0] if layered else 1, lead[-1], 2 * half, at,
                      layered)

    def _addresses(self) -> list:
        """Of the arrays; ValueError where one is not what the cache was made of."""
        torch = _torch()
        lead = (self.layers, self.num_slots) if self.layered else (self.num_slots,)
        return [_want(self.codes, "codes", torch.uint8, lead + (self.dim // 2,), self.index),
                _want(self.scales, "scales", torch.float16, lead + (self.dim // 128,), self.index),
                _want(self.zeros, "zeros", torch.float16, lead + (self.dim // 128,), self.index)]

    def layer(self, i: int) -> "KVCacheInt4":
        """Layer i as a cache of its own (views of the same memory) for the writing call
        and the attention; page copies take the whole cache."""
        if not self.layered:
            raise ValueError("the cache has no layers")
        return KVCacheInt4(self.codes[i], self.scales[i], self.zeros[i])


def kq_attn_decode_int4_kv(q, k_cache: KVCacheInt4, v_cache: KVCacheInt4, k_signs, v_signs,
                           block_table, page_size: int, seq_lens, softmax_scale: float, out,
                           workspace, window: int = 0, sinks: int = 0, stream=None) -> None:
    """Attention of one new token per sequence over the paged INT4 caches: q and
    out bf16 [batch, q_heads, 128], block_table int32 [batch, width], seq_lens
    int32 [batch]; window > 0 keeps the last `window` tokens and the first
    `sinks` ones visible.  workspace: empty_attn_workspace(...)."""
    status = (_call or _native()).attn(q, k_cache, v_cache, k_signs, v_signs, block_table,
                                       page_size, seq_lens, softmax_scale, out, workspace, window,
                                       sinks, stream)
    if status is None:
        _attn_checked(q, k_cache, v_cache, k_signs, v_signs, block_table, page_size, seq_lens,
                      softmax_scale, out, workspace, window, sinks, stream)
    elif status != KQ_OK:
        raise KQError(status, "kq_attn_decode_int4_kv")


def _attn_checked(q, k_cache, v_cache, k_signs, v_signs, block_table, page_size, seq_lens,
                  softmax_scale, out, workspace, window, sinks, stream) -> None:
    torch = _torch()
    _there(q=q, k_cache=k_cache, v_cache=v_cache, block_table=block_table, workspace=workspace)
    if q.dim() != 3 or block_table.dim() != 2:
        raise ValueError("q is [batch, q_heads, 128] and block_table [batch, width]")
    batch, q_heads, _ = q.shape
    at, dim, width = q.get_device(), k_cache.dim, block_table.shape[1]
    if (page_size | window | sinks) >> 31:
        _int32(page_size=page_size, window=window, sinks=sinks)
    if k_cache.layered or v_cache.layered:
        raise ValueError("the attention reads one layer: pass cache.layer(i)")
    if v_cache.dim != dim or v_cache.num_slots != k_cache.num_slots:
        raise ValueError("the key and value caches differ in shape")
    if k_cache.index != at or v_cache.index != at:
        raise ValueError(f"the caches are not on cuda:{at}")
    shape = (batch, q_heads, 128)
    _launch((_lib or lib()).kq_attn_decode_int4_kv, "kq_attn_decode_int4_kv", at, stream,
            _want(q, "q", torch.bfloat16, shape, at), batch, q_heads, dim // 128,
            None if k_signs is None else _want(k_signs, "k_signs", torch.int8, (dim,), at),
            None if v_signs is None else _want(v_signs, "v_signs", torch.int8, (dim,), at),
            *k_cache._addresses(), *v_cache._addresses(),
            k_cache.num_slots, _want(block_table, "block_table", torch.int32, (batch, width), at),
            width, page_size, _want(seq_lens, "seq_lens", torch.int32, (batch,), at), window,
            sinks, softmax_scale, _want(out, "out", torch.bfloat16, shape, at),
            _want(workspace, "workspace", torch.uint8, workspace.shape, at), workspace.numel())


def kq_kv_copy_pages(pairs, page_size: int, k_cache: KVCacheInt4,
                     v_cache: Optional[KVCacheInt4] = None, stream=None) -> None:
    """Copies pages of the cache(s): pairs int32 [n, 2] of (source, destination)
    page; pairs with a page outside the cache are skipped."""
    status = (_call or _native()).copy(pairs, page_size, k_cache, v_cache, stream)
    if status is None:
        _copy_checked(pairs, page_size, k_cache, v_cache, stream)
    elif status != KQ_OK:
        raise KQError(status, "kq_kv_copy_pages")


def _copy_checked(pairs, page_size, k_cache, v_cache, stream) -> None:
    _there(pairs=pairs, k_cache=k_cache)
    if pairs.dim() != 2:
        raise ValueError("pairs are [n, 2]")
    at, n = k_cache.index, pairs.shape[0]
    if page_size >> 31:
        _int32(page_size=page_size)
    values = (None, None, None)
    if v_cache is not None:
        if v_cache.dim != k_cache.dim or v_cache.num_slots != k_cache.num_slots or \
                v_cache.layers != k_cache.layers:
            raise ValueError("the key and value caches differ in shape")
        if v_cache.index != at:
            raise ValueError(f"the caches are not both on cuda:{at}")
        values = v_cache._addresses()
    _launch((_lib or lib()).kq_kv_copy_pages, "kq_kv_copy_pages", at, stream,
            _want(pairs, "pairs", _torch().int32, (n, 2), at), n, page_size, k_cache.num_slots,
            k_cache.layers, k_cache.dim, *k_cache._addresses(), *values)


def kq_dequant(fmt: int, codes, scales, zeros, tensor_scale, tokens: int, dim: int,
               group: int, out, stream=None) -> None:
    """Codes and scales back to fp32 (exact product, one rounding)."""
    _check(lib().kq_dequant(fmt, _ptr(codes), _ptr(scales), _ptr(zeros),
                            _ptr(tensor_scale), tokens, dim, group, _ptr(out),
                            _stream(stream)), "kq_dequant")


def kq_dequant_rht_inverse(fmt: int, codes, scales, zeros, tensor_scale, tokens: int,
                           dim: int, block: int, group: int, signs, out, stream=None) -> None:
    """Dequantize and undo the rotation in one call; `out` is fp32 or bf16."""
    _check(lib().kq_dequant_rht_inverse(fmt, _ptr(codes), _ptr(scales), _ptr(zeros),
                                        _ptr(tensor_scale), tokens, dim, block, group,
                                        _ptr(signs), _ptr(out), _dtype_code(out),
                                        _stream(stream)),
           "kq_dequant_rht_inverse")


def kq_diag_tc_steps(a, b, d1, d2, status, stream=None, fp16=False) -> None:
    """Two tensor-core accumulation steps on caller data (diagnostic; see
    include/kq.h): a bf16 (fp16 with fp16=True) [128, 32], b [32, 128], d1/d2
    fp32 [128, 128], status one int32 (0 = the waits completed)."""
    fn = lib().kq_diag_tc_steps_f16 if fp16 else lib().kq_diag_tc_steps
    _check(fn(_ptr(a), _ptr(b), _ptr(d1), _ptr(d2), _ptr(status), _stream(stream)),
           "kq_diag_tc_steps")


def kq_device_errors():
    """The six error words of the tensor-core kernel families (read and
    cleared): 4096-wide, 12288-wide, block-128 GEMM, fused inverse,
    diagnostic, NVFP4 GEMM.  All zero: no bounded wait ran out since the last
    call."""
    buf = (ctypes.c_uint * 6)()
    _check(lib().kq_device_errors(buf), "kq_device_errors")
    return list(buf)


def kq_diag_wait_timeout(limit_cycles: int, stream=None) -> None:
    """Diagnostic: a wait that nothing satisfies, bounded by limit_cycles."""
    _check(lib().kq_diag_wait_timeout(int(limit_cycles), _stream(stream)),
           "kq_diag_wait_timeout")


def kq_workspace_size(tokens: int, dim: int, block: int) -> int:
    return int(lib().kq_workspace_size(tokens, dim, block))


def kq_version() -> int:
    return int(lib().kq_version())


# ------------------------------------------------- output allocation helpers
def empty_int4_sym(tokens: int, dim: int, device="cuda"):
    import torch
    return (torch.empty((tokens, dim // 2), dtype=torch.uint8, device=device),
            torch.empty((tokens,), dtype=torch.float32, device=device))


def empty_int4_asym(tokens: int, dim: int, group: int = 128, device="cuda"):
    import torch
    g = dim // group
    return (torch.empty((tokens, dim // 2), dtype=torch.uint8, device=device),
            torch.empty((tokens, g), dtype=torch.float16, device=device),
            torch.empty((tokens, g), dtype=torch.float16, device=device))


def empty_mxfp4(tokens: int, dim: int, device="cuda"):
    """(codes, scales) for kq_rht_quant_mxfp4."""
    import torch
    return (torch.empty((tokens, dim // 2), dtype=torch.uint8, device=device),
            torch.empty((tokens, dim // 32), dtype=torch.uint8, device=device))


def sf_mma_bytes(rows: int, dim: int) -> int:
    """Bytes of NVFP4 block scales in the tensor-core layout: rows padded to a
    multiple of 128, dim / 16 scales a row (dim % 64 == 0)."""
    return -(-rows // 128) * 128 * (dim // 16)


def empty_nvfp4(tokens: int, dim: int, block: int = 0, device="cuda", mma_layout=False):
    """(codes, block_scales, tensor_scale, workspace) for kq_rht_quant_nvfp4;
    with mma_layout the block scales are a flat buffer of sf_mma_bytes."""
    import torch
    ws = kq_workspace_size(tokens, dim, block)
    scales = (torch.zeros((sf_mma_bytes(tokens, dim),), dtype=torch.uint8, device=device)
              if mma_layout else
              torch.empty((tokens, dim // 16), dtype=torch.uint8, device=device))
    return (torch.empty((tokens, dim // 2), dtype=torch.uint8, device=device),
            scales,
            torch.empty((1,), dtype=torch.float32, device=device),
            torch.empty((max(ws, 16),), dtype=torch.uint8, device=device))


def empty_kv_cache(num_slots: int, dim: int, layers: int = 0, device="cuda") -> KVCacheInt4:
    """A KVCacheInt4 of num_slots rows (of `layers` layers when layers > 0)."""
    import torch
    lead = (layers, num_slots) if layers else (num_slots,)
    return KVCacheInt4(torch.empty(lead + (dim // 2,), dtype=torch.uint8, device=device),
                       torch.empty(lead + (dim // 128,), dtype=torch.float16, device=device),
                       torch.empty(lead + (dim // 128,), dtype=torch.float16, device=device))


def kq_attn_workspace_size(batch: int, q_heads: int, kv_heads: int) -> int:
    return int(lib().kq_attn_workspace_size(batch, q_heads, kv_heads))


def empty_attn_workspace(batch: int, q_heads: int, kv_heads: int, device="cuda"):
    """Workspace of kq_attn_decode_int4_kv; one per call that may overlap."""
    import torch
    return torch.empty((max(kq_attn_workspace_size(batch, q_heads, kv_heads), 16),),
                       dtype=torch.uint8, device=device)
