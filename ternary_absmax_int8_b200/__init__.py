"""Python binding of libtq (include/tq.h): the same names, argument marshalling only.

Every function forwards to the C ABI of the in-tree ``libtq.so``; all work runs
in its CUDA kernels. Tensors are passed as raw pointers (``data_ptr()``), an
``int`` is taken as a raw pointer, ``None`` as NULL. ``stream`` defaults to
PyTorch's current CUDA stream. A non-OK status raises :class:`TQError`. The
rotary and cache calls refuse tensors that the kernel would misread: of another
type, on another device, or a view that is neither contiguous nor rows at the
distance given.

There is no fallback: if ``libtq.so`` is missing, every call raises (the
package itself still imports, so that its ``build`` module can run). Build it
with ``python -m ternary_absmax_int8_b200.build``.
"""
from __future__ import annotations

import ctypes
import os
import sys

__all__ = [
    "TQError", "TQ_STACK_OVERLAP_PREV", "TQ_STACK_QUANTIZE", "TQ_STACK_RMSNORM",
    "TQ_STACK_RELU2_MUL", "TqProj", "lib_path",
    "tq_pack_host", "tq_quantize_act", "tq_gemv", "tq_gemm_prefill",
    "tq_quantize_act_stack", "tq_gemv_stack", "tq_quantize_act_stack_batch",
    "tq_gemv_stack_batch", "tq_gemm_prefill_stack", "tq_device_error", "tq_gemv_noalloc",
    "tq_status_string", "tq_last_error", "make_proj", "tq_rmsnorm_quantize",
    "tq_relu2_mul_rmsnorm_quantize", "tq_absmean_pack", "tq_selftest_wait_timeout",
    "tq_hadamard_quantize_act", "tq_hadamard_quantize_act_stack", "TqBinaryProj",
    "tq_pack_binary_host", "tq_gemv_binary",
    "tq_gemv_binary_stack", "make_binary_proj",
    "TQ_ROPE_INTERLEAVED", "TqRopeRows", "make_rope_rows", "tq_rope",
    "TqKv4Cache", "TqKv4Query", "make_kv4_cache", "tq_kv4_page_bytes", "tq_kv4_append",
    "tq_kv4_decode_workspace", "tq_kv4_prefill_workspace", "tq_kv4_decode", "tq_kv4_prefill",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
lib_path = os.path.join(_HERE, "libtq.so")

TQ_STACK_OVERLAP_PREV = 1
TQ_STACK_QUANTIZE = 2
TQ_STACK_RMSNORM = 4
TQ_STACK_RELU2_MUL = 8
TQ_ROPE_INTERLEAVED = 1
_STATUS = {0: "TQ_OK", 1: "TQ_ERR_NULL", 2: "TQ_ERR_SHAPE", 3: "TQ_ERR_ALIGN",
           4: "TQ_ERR_VALUE", 5: "TQ_ERR_CUDA", 6: "TQ_ERR_UNSUPPORTED"}


class TQError(RuntimeError):
    def __init__(self, status: int, message: str):
        self.status = status
        self.name = _STATUS.get(status, f"status {status}")
        super().__init__(f"{self.name}: {message}")


_vp, _i, _f = ctypes.c_void_p, ctypes.c_int, ctypes.c_float


class TqProj(ctypes.Structure):
    """Mirror of ``struct tq_proj``."""
    _fields_ = [
        ("packed", ctypes.c_void_p),
        ("x", ctypes.c_void_p),
        ("xq", ctypes.c_void_p),
        ("x_scale", ctypes.c_void_p),
        ("x_sum", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("acc_out", ctypes.c_void_p),
        ("w_scale", ctypes.c_float),
        ("N", ctypes.c_int),
        ("K", ctypes.c_int),
        ("gain", ctypes.c_void_p),
        ("x_f32", ctypes.c_void_p),
        ("up", ctypes.c_void_p),
        ("eps", ctypes.c_float),
        ("reserved", ctypes.c_int),
    ]


class TqBinaryProj(ctypes.Structure):
    """Mirror of ``struct tq_binary_proj``."""
    _fields_ = [
        ("bits", ctypes.c_void_p),
        ("scales_packed", ctypes.c_void_p),
        ("xq", ctypes.c_void_p),
        ("x_scale", ctypes.c_void_p),
        ("y", ctypes.c_void_p),
        ("acc_out", ctypes.c_void_p),
        ("N", ctypes.c_int),
        ("K", ctypes.c_int),
    ]


class TqRopeRows(ctypes.Structure):
    """Mirror of ``struct tq_rope_rows``."""
    _fields_ = [
        ("x_bf16", ctypes.c_void_p),
        ("x_f32", ctypes.c_void_p),
        ("y_bf16", ctypes.c_void_p),
        ("y_f32", ctypes.c_void_p),
        ("x_stride", ctypes.c_int64),
        ("y_stride", ctypes.c_int64),
        ("heads", ctypes.c_int),
        ("reserved", ctypes.c_int),
    ]


class TqKv4Cache(ctypes.Structure):
    """Mirror of ``struct tq_kv4_cache``."""
    _fields_ = [
        ("pages", ctypes.c_void_p),
        ("page_table", ctypes.c_void_p),
        ("page_stride", ctypes.c_int64),
        ("num_pages", ctypes.c_int),
        ("page_size", ctypes.c_int),
        ("kv_heads", ctypes.c_int),
        ("head_dim", ctypes.c_int),
        ("batch", ctypes.c_int),
        ("max_pages", ctypes.c_int),
    ]


class TqKv4Query(ctypes.Structure):
    """Mirror of ``struct tq_kv4_query``."""
    _fields_ = [
        ("q", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("lse", ctypes.c_void_p),
        ("q_stride", ctypes.c_int64),
        ("out_stride", ctypes.c_int64),
        ("q_heads", ctypes.c_int),
        ("window", ctypes.c_int),
        ("scale", ctypes.c_float),
        ("reserved", ctypes.c_int),
    ]


_i64, _sz = ctypes.c_int64, ctypes.c_size_t
_SIGS = {
    "tq_pack_host": [_vp, _vp, _i, _i, _i, _vp],
    "tq_quantize_act": [_vp, _vp, _vp, _vp, _i, _i, _i, _vp],
    "tq_gemv": [_vp, _f, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp],
    "tq_gemm_prefill": [_vp, _f, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp],
    "tq_gemv_noalloc": [_vp, _f, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp],
    "tq_quantize_act_stack": [ctypes.POINTER(TqProj), _i, _vp],
    "tq_gemv_stack": [ctypes.POINTER(TqProj), _i, ctypes.c_uint, _vp],
    "tq_quantize_act_stack_batch": [ctypes.POINTER(TqProj), _i, _i, _vp],
    "tq_gemv_stack_batch": [ctypes.POINTER(TqProj), _i, _i, ctypes.c_uint, _vp],
    "tq_gemm_prefill_stack": [ctypes.POINTER(TqProj), _i, _i, _vp],
    "tq_device_error": [ctypes.POINTER(ctypes.c_uint32), _i],
    "tq_rmsnorm_quantize": [_vp, _vp, _vp, _f, _vp, _vp, _vp, _i, _i, _vp],
    "tq_relu2_mul_rmsnorm_quantize": [_vp, _vp, _vp, _f, _vp, _vp, _vp, _i, _i, _vp],
    "tq_absmean_pack": [_vp, _vp, _vp, _i, _i, _vp],
    "tq_selftest_wait_timeout": [ctypes.c_uint, _vp],
    "tq_hadamard_quantize_act": [_vp, _vp, _vp, _vp, _i, _i, _i, _vp],
    "tq_hadamard_quantize_act_stack": [ctypes.POINTER(TqProj), _i, _i, _i, _vp],
    "tq_pack_binary_host": [_vp, _vp, _vp, _vp, _i, _i],
    "tq_gemv_binary": [_vp, _vp, _vp, _vp, _vp, _vp, _i, _i, _i, _vp],
    "tq_gemv_binary_stack": [ctypes.POINTER(TqBinaryProj), _i, _i, _vp],
    "tq_rope": [ctypes.POINTER(TqRopeRows), _i, _vp, _i64, _vp, ctypes.POINTER(_i), _i, _i, _i,
                _i, ctypes.c_uint, _vp],
    "tq_kv4_append": [ctypes.POINTER(TqKv4Cache), _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _i,
                      _vp],
    "tq_kv4_decode": [ctypes.POINTER(TqKv4Cache), ctypes.POINTER(TqKv4Query), _vp, _vp, _sz, _vp],
    "tq_kv4_prefill": [ctypes.POINTER(TqKv4Cache), ctypes.POINTER(TqKv4Query), _vp, _vp, _i, _vp,
                       _sz, _vp],
    "tq_kv4_decode_workspace": [ctypes.POINTER(TqKv4Cache), _i, ctypes.POINTER(_sz)],
    "tq_kv4_prefill_workspace": [ctypes.POINTER(TqKv4Cache), _i, _i, ctypes.POINTER(_sz)],
}
_lib_handle = None


def _load():
    """Load libtq.so once; raise loudly if it has not been built."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(lib_path):
            raise RuntimeError(
                f"{lib_path} is missing: build it with `python -m ternary_absmax_int8_b200.build`"
                " (there is no CPU fallback)")
        lib = ctypes.CDLL(lib_path)
        for name, args in _SIGS.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int
        lib.tq_status_string.argtypes = [ctypes.c_int]
        lib.tq_status_string.restype = ctypes.c_char_p
        lib.tq_kv4_page_bytes.argtypes = [_i, _i, _i]
        lib.tq_kv4_page_bytes.restype = _sz
        lib.tq_last_error.argtypes = []
        lib.tq_last_error.restype = ctypes.c_char_p
        _lib_handle = lib
    return _lib_handle


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if hasattr(t, "data_ptr"):
        return t.data_ptr()
    if hasattr(t, "ctypes"):  # numpy array
        return t.ctypes.data
    raise TypeError(f"cannot pass {type(t).__name__} as a pointer")


def _stream(stream):
    if stream is None:
        import torch
        if not torch.cuda.is_available():
            return None
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(rc: int):
    if rc != 0:
        raise TQError(rc, _load().tq_last_error().decode())


def tq_status_string(status: int) -> str:
    return _load().tq_status_string(status).decode()


def tq_last_error() -> str:
    return _load().tq_last_error().decode()


def tq_pack_host(w, packed, M: int, N: int, K: int, stream=0) -> None:
    """Host packing: w int8 [N,K] (CPU tensor or numpy) -> packed uint8 [N/4,K]."""
    _check(_load().tq_pack_host(_ptr(w), _ptr(packed), M, N, K, None))


def tq_quantize_act(x, xq, x_scale, x_sum, M: int, N: int, K: int, stream=None) -> None:
    _check(_load().tq_quantize_act(_ptr(x), _ptr(xq), _ptr(x_scale), _ptr(x_sum), M, N, K,
                                _stream(stream)))


def tq_gemv(packed, w_scale: float, xq, x_scale, x_sum, y, acc_out, M: int, N: int, K: int,
            stream=None) -> None:
    _check(_load().tq_gemv(_ptr(packed), float(w_scale), _ptr(xq), _ptr(x_scale), _ptr(x_sum),
                        _ptr(y), _ptr(acc_out), M, N, K, _stream(stream)))


def tq_gemm_prefill(packed, w_scale: float, xq, x_scale, x_sum, y, acc_out, M: int, N: int,
                    K: int, stream=None) -> None:
    _check(_load().tq_gemm_prefill(_ptr(packed), float(w_scale), _ptr(xq), _ptr(x_scale),
                                _ptr(x_sum), _ptr(y), _ptr(acc_out), M, N, K, _stream(stream)))


def tq_gemv_noalloc(packed, w_scale: float, xq, x_scale, x_sum, y, acc_out, M: int, N: int,
                    K: int, stream=None) -> None:
    """tq_gemv for 5 <= M <= 32 on fixed library scratch (allocates nothing)."""
    _check(_load().tq_gemv_noalloc(_ptr(packed), float(w_scale), _ptr(xq), _ptr(x_scale),
                                _ptr(x_sum), _ptr(y), _ptr(acc_out), M, N, K, _stream(stream)))


def tq_rmsnorm_quantize(x_bf16, x_f32, gain, eps: float, xq, x_scale, x_sum, M: int, K: int,
                        stream=None) -> None:
    """RMSNorm (gain, eps) then the absmax quantiser; exactly one of x_bf16 / x_f32."""
    _check(_load().tq_rmsnorm_quantize(_ptr(x_bf16), _ptr(x_f32), _ptr(gain), float(eps),
                                    _ptr(xq), _ptr(x_scale), _ptr(x_sum), M, K,
                                    _stream(stream)))


def tq_relu2_mul_rmsnorm_quantize(gate, up, gain, eps: float, xq, x_scale, x_sum, M: int,
                                  K: int, stream=None) -> None:
    """relu(gate)^2 * up, RMSNorm (gain, eps), then the absmax quantiser."""
    _check(_load().tq_relu2_mul_rmsnorm_quantize(_ptr(gate), _ptr(up), _ptr(gain), float(eps),
                                              _ptr(xq), _ptr(x_scale), _ptr(x_sum), M, K,
                                              _stream(stream)))


def tq_absmean_pack(w_bf16, packed, w_scale, N: int, K: int, stream=None) -> None:
    """Absmean ternary quantisation of bf16 weights [N,K] -> packed [N/4,K], w_scale [1]."""
    _check(_load().tq_absmean_pack(_ptr(w_bf16), _ptr(packed), _ptr(w_scale), N, K,
                                _stream(stream)))


def tq_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    """A bounded wait that nothing satisfies: sets the device error word."""
    _check(_load().tq_selftest_wait_timeout(int(limit_us), _stream(stream)))


def tq_hadamard_quantize_act(x, xq, x_scale, x_sum, M: int, K: int, n: int,
                             stream=None) -> None:
    """Blockwise Hadamard rotation (block n) then 4-bit absmax codes (-7..7 in int8)."""
    _check(_load().tq_hadamard_quantize_act(_ptr(x), _ptr(xq), _ptr(x_scale), _ptr(x_sum), M, K,
                                         int(n), _stream(stream)))


def tq_hadamard_quantize_act_stack(projs, M: int, n: int, stream=None) -> None:
    arr, cnt = _proj_array(projs)
    _check(_load().tq_hadamard_quantize_act_stack(arr, cnt, int(M), int(n), _stream(stream)))


def tq_pack_binary_host(w, scales, bits, scales_packed, N: int, K: int) -> None:
    """Host packing of binary g128 weights: w int8 [N,K] in {-1,+1}, fp16 scales
    [N,K/128] -> bits uint8 [N/8,K], scales_packed fp16 [N/8,K/128,8]."""
    _check(_load().tq_pack_binary_host(_ptr(w), _ptr(scales), _ptr(bits), _ptr(scales_packed),
                                    int(N), int(K)))


def tq_gemv_binary(bits, scales_packed, xq, x_scale, y, acc_out, M: int, N: int, K: int,
                   stream=None) -> None:
    _check(_load().tq_gemv_binary(_ptr(bits), _ptr(scales_packed), _ptr(xq), _ptr(x_scale),
                               _ptr(y), _ptr(acc_out), M, N, K, _stream(stream)))


def make_binary_proj(bits=None, scales_packed=None, xq=None, x_scale=None, y=None, acc_out=None,
                     N: int = 0, K: int = 0) -> TqBinaryProj:
    return TqBinaryProj(_ptr(bits), _ptr(scales_packed), _ptr(xq), _ptr(x_scale), _ptr(y),
                        _ptr(acc_out), int(N), int(K))


def tq_gemv_binary_stack(projs, M: int, stream=None) -> None:
    arr = (TqBinaryProj * len(projs))(*projs)
    _check(_load().tq_gemv_binary_stack(arr, len(projs), int(M), _stream(stream)))


def make_proj(packed=None, x=None, xq=None, x_scale=None, x_sum=None, y=None, acc_out=None,
              w_scale: float = 0.0, N: int = 0, K: int = 0, gain=None, x_f32=None, up=None,
              eps: float = 0.0) -> TqProj:
    return TqProj(_ptr(packed), _ptr(x), _ptr(xq), _ptr(x_scale), _ptr(x_sum), _ptr(y),
                  _ptr(acc_out), float(w_scale), int(N), int(K), _ptr(gain), _ptr(x_f32),
                  _ptr(up), float(eps), 0)


def _proj_array(projs):
    arr = (TqProj * len(projs))(*projs)
    return arr, len(projs)


def tq_quantize_act_stack(projs, stream=None) -> None:
    arr, n = _proj_array(projs)
    _check(_load().tq_quantize_act_stack(arr, n, _stream(stream)))


def tq_gemv_stack(projs, flags: int = 0, stream=None) -> None:
    arr, n = _proj_array(projs)
    _check(_load().tq_gemv_stack(arr, n, int(flags), _stream(stream)))


def tq_quantize_act_stack_batch(projs, M: int, stream=None) -> None:
    arr, n = _proj_array(projs)
    _check(_load().tq_quantize_act_stack_batch(arr, n, int(M), _stream(stream)))


def tq_gemv_stack_batch(projs, M: int, flags: int = 0, stream=None) -> None:
    arr, n = _proj_array(projs)
    _check(_load().tq_gemv_stack_batch(arr, n, int(M), int(flags), _stream(stream)))


def tq_gemm_prefill_stack(projs, M: int, stream=None) -> None:
    arr, n = _proj_array(projs)
    _check(_load().tq_gemm_prefill_stack(arr, n, int(M), _stream(stream)))


def tq_device_error(reset: bool = False) -> int:
    code = ctypes.c_uint32(0)
    _check(_load().tq_device_error(ctypes.byref(code), 1 if reset else 0))
    return int(code.value)


def _device() -> int:
    """The current CUDA device, or -2 (no tensor's) where there is none."""
    import torch
    if torch.cuda.is_initialized() or torch.cuda.is_available():
        return torch.cuda.current_device()
    return -2


def _here(stream):
    """The current CUDA device and the handle of `stream` (of the current one if None): what a
    call needs to know, looked up once."""
    torch = sys.modules.get("torch")
    if torch is None or not torch.cuda.is_initialized():
        return _device(), _stream(stream)
    # (torch's own functions for these look up again whether CUDA is up, and build a Stream)
    device = torch._C._cuda_getDevice()
    if stream is None:
        return device, torch._C._cuda_getCurrentRawStream(device)
    return device, _stream(stream)


# Element types that a pointer of each kind may come from (also plain whole numbers of its size,
# where the bits are what counts); filled when the first tensor is met, as torch is imported late.
_BF16, _F32, _I32, _U8 = [], [], [], []


def _gpu_ptr(t, kinds, device: int, stride: int = 0):
    """Pointer of a tensor of one of the types `kinds` on CUDA device `device`, the current one (an
    int or None passes through); one of another type would be misread, one elsewhere not be found
    here. Its elements must follow one another, but for rows that are `stride` elements apart."""
    if t is None or isinstance(t, int):
        return t
    if t.dtype in kinds and t.get_device() == device and (t.is_contiguous() or _rows(t, stride)):
        return t.data_ptr()
    if not kinds:
        import torch
        _BF16[:] = torch.bfloat16, torch.int16, torch.uint16
        _F32[:] = torch.float32,
        _I32[:] = torch.int32, torch.uint32
        _U8[:] = torch.uint8, torch.int8
        return _gpu_ptr(t, kinds, device, stride)
    if t.dtype not in kinds:
        raise TQError(4, f"a tensor of {kinds[0]} is wanted, not {t.dtype}")
    if t.get_device() != device:
        raise TQError(4, f"a tensor on {t.device}: tensors must be on the current CUDA device")
    raise TQError(4, f"a view of shape {tuple(t.shape)}, strides {tuple(t.stride())}: it must be "
                     "contiguous" + (f" or of rows {stride} elements apart" if stride else ""))


def _rows(t, stride: int) -> bool:
    """Whether t is rows that lie `stride` elements apart, each contiguous, in as many leading
    and trailing dimensions as it may be."""
    if t.dim() < 2 or (t.shape[-1] != 1 and t.stride(-1) != 1):
        return False
    want, inner = 1, True
    for size, step in zip(reversed(t.shape), reversed(t.stride())):
        if size == 1:
            continue
        if step != want:
            if not inner or step != stride or stride == 0:
                return False
            want, inner = stride, False
        want *= size
    return True


def _on(device: int, described, tensors):
    """A description that names `tensors`, which are on `device`. (Of addresses that are given as
    whole numbers the device is the caller's business.)"""
    if any(hasattr(t, "data_ptr") for t in tensors):
        described.device = device
    return described


def _same_device(described, device: int):
    """Refuse a description whose tensors are on another device than the current one."""
    made = getattr(described, "device", device)
    if made != device:
        raise TQError(4, f"described on device {made}, called on {device}: tensors must be on the "
                         "current CUDA device")


def make_rope_rows(rows, head_dim: int):
    """A table of ``tq_rope_rows`` from dicts with the keys x_bf16 or x_f32, y_bf16 or y_f32,
    heads and, for rows that are not packed, x_stride and y_stride (values between tokens)."""
    arr = (TqRopeRows * len(rows))()
    dev = _device()
    for e, r in zip(arr, rows):
        e.heads = int(r["heads"])
        e.x_stride = int(r.get("x_stride", 0)) or e.heads * int(head_dim)
        e.y_stride = int(r.get("y_stride", 0)) or e.heads * int(head_dim)
        e.x_bf16 = _gpu_ptr(r.get("x_bf16"), _BF16, dev, e.x_stride)
        e.x_f32 = _gpu_ptr(r.get("x_f32"), _F32, dev, e.x_stride)
        e.y_bf16 = _gpu_ptr(r.get("y_bf16"), _BF16, dev, e.y_stride)
        e.y_f32 = _gpu_ptr(r.get("y_f32"), _F32, dev, e.y_stride)
    return _on(dev, arr, [t for r in rows for t in r.values()])


def tq_rope(rows, pos, inv_freq, sections, T: int, head_dim: int, rot_dim: int, flags: int = 0,
            pos_stride: int = 0, stream=None) -> None:
    """Rotary positions of the rows in a make_rope_rows table; pos int32 [len(sections), T]."""
    dev, stream = _here(stream)
    _same_device(rows, dev)
    n = len(sections)
    pos_stride = int(pos_stride) or int(T)
    _check(_load().tq_rope(rows, len(rows), _gpu_ptr(pos, _I32, dev, pos_stride), pos_stride,
                           _gpu_ptr(inv_freq, _F32, dev), (_i * n)(*sections), n, int(T),
                           int(head_dim), int(rot_dim), int(flags), stream))


def tq_kv4_page_bytes(page_size: int, kv_heads: int, head_dim: int) -> int:
    return _load().tq_kv4_page_bytes(int(page_size), int(kv_heads), int(head_dim))


def make_kv4_cache(pages=None, page_table=None, num_pages: int = 0, page_size: int = 64,
                   kv_heads: int = 1, head_dim: int = 128, batch: int = 0, max_pages: int = 0,
                   page_stride: int = 0) -> TqKv4Cache:
    """Describe a 4-bit key/value cache. It holds pointers only: keep the tensors."""
    dev = _device()
    return _on(dev, TqKv4Cache(
        _gpu_ptr(pages, _U8, dev, page_stride), _gpu_ptr(page_table, _I32, dev, max_pages),
        int(page_stride), int(num_pages), int(page_size), int(kv_heads), int(head_dim),
        int(batch), int(max_pages)), (pages, page_table))


def tq_kv4_append(cache, k_bf16, v_bf16, k_f32, v_f32, tok_start, lens, T: int, k_stride: int = 0,
                  v_stride: int = 0, stream=None) -> None:
    """Quantise new keys and values into the cache's pages (one of the two pairs)."""
    dev, stream = _here(stream)
    _same_device(cache, dev)
    _check(_load().tq_kv4_append(
        ctypes.byref(cache), _gpu_ptr(k_bf16, _BF16, dev, k_stride),
        _gpu_ptr(v_bf16, _BF16, dev, v_stride), _gpu_ptr(k_f32, _F32, dev, k_stride),
        _gpu_ptr(v_f32, _F32, dev, v_stride), int(k_stride), int(v_stride),
        _gpu_ptr(tok_start, _I32, dev), _gpu_ptr(lens, _I32, dev), int(T), stream))


def tq_kv4_decode_workspace(cache, q_heads: int) -> int:
    size = _sz(0)
    _check(_load().tq_kv4_decode_workspace(ctypes.byref(cache), int(q_heads), ctypes.byref(size)))
    return size.value


def tq_kv4_prefill_workspace(cache, q_heads: int, T: int) -> int:
    size = _sz(0)
    _check(_load().tq_kv4_prefill_workspace(ctypes.byref(cache), int(q_heads), int(T),
                                            ctypes.byref(size)))
    return size.value


def _kv4_query(dev, q, out, lse, q_heads, scale, window, q_stride, out_stride):
    return ctypes.byref(TqKv4Query(_gpu_ptr(q, _BF16, dev, q_stride),
                                   _gpu_ptr(out, _BF16, dev, out_stride),
                                   _gpu_ptr(lse, _F32, dev), int(q_stride), int(out_stride),
                                   int(q_heads), int(window), float(scale), 0))


def tq_kv4_decode(cache, q, lens, out, lse, q_heads: int, scale: float, window: int = 0,
                  workspace=None, workspace_bytes: int = 0, q_stride: int = 0,
                  out_stride: int = 0, stream=None) -> None:
    """Attention of one new token per sequence over the cache."""
    dev, stream = _here(stream)
    _same_device(cache, dev)
    query = _kv4_query(dev, q, out, lse, q_heads, scale, window, q_stride, out_stride)
    _check(_load().tq_kv4_decode(ctypes.byref(cache), query, _gpu_ptr(lens, _I32, dev),
                                 _gpu_ptr(workspace, _U8, dev), int(workspace_bytes), stream))


def tq_kv4_prefill(cache, q, tok_start, lens, out, lse, T: int, q_heads: int, scale: float,
                   window: int = 0, workspace=None, workspace_bytes: int = 0, q_stride: int = 0,
                   out_stride: int = 0, stream=None) -> None:
    """Attention of any number of new tokens per sequence over the cache."""
    dev, stream = _here(stream)
    _same_device(cache, dev)
    query = _kv4_query(dev, q, out, lse, q_heads, scale, window, q_stride, out_stride)
    _check(_load().tq_kv4_prefill(ctypes.byref(cache), query, _gpu_ptr(tok_start, _I32, dev),
                                  _gpu_ptr(lens, _I32, dev), int(T),
                                  _gpu_ptr(workspace, _U8, dev), int(workspace_bytes), stream))
