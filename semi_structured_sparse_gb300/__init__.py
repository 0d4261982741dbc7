"""semi_structured_sparse_gb300 -- Python binding of libsp24 (2:4 sparse FP8 GEMM on GB300).

Argument marshalling only: every step runs in the library's CUDA kernels.
torch supplies device memory and the current stream; the library itself never
allocates.  There is no CPU fallback: if the library is missing or the device
is not an sm_103 GPU, every call raises.

    values, meta, sw = compress(w_bf16, gN=1, gK=None)        # prune + e4m3 + pack
    xq, sx          = quantize_act(x_fp32, gK=None)            # per-token / 1x128 e4m3
    y               = gemm(xq, sx, values, meta, sw, gM=1, gN=1, gK=None, x2=None, w2=None)

Between a layer's QKV and output projections (attention over a paged cache):

    cache = KVCache(k, v)                                      # bf16, or e4m3 codes with scales
    q     = qk_norm_rope(qkv, heads, cache, positions, slots, cos_sin)
    y     = attention_decode(q, cache, page_table, seq_lens)   # one new token per sequence
    y     = attention_prompt(q, cu_q, cache, page_table, seq_lens)
"""
import contextlib
import ctypes
import os

import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None

SP24_STATUS = {
    0: "SP24_OK", 1: "SP24_ERR_INVALID_ARG", 2: "SP24_ERR_UNSUPPORTED", 3: "SP24_ERR_ALIGNMENT",
    4: "SP24_ERR_CUDA", 5: "SP24_ERR_ARCH", 6: "SP24_ERR_WORKSPACE", 7: "SP24_ERR_DEVICE_TIMEOUT",
    8: "SP24_ERR_DEVICE_INDEX",
}

# Every entry point the C header declares, with its ctypes signature.
_P, _I64, _I, _SZ, _F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t, ctypes.c_float
SIGNATURES = {
    "sp24_status_string": ([_I], ctypes.c_char_p),
    "sp24_meta_bytes": ([_I64, _I64], _SZ),
    "sp24_fp8_compress": ([_P, _I64, _I64, _I64, _I, _I, _P, _P, _P, _P], _I),
    "sp24_fp8_quantize_act": ([_P, _I64, _I64, _I64, _I, _P, _P, _P], _I),
    "sp24_fp8_quantize_act_bf16": ([_P, _I64, _I64, _I64, _I, _P, _P, _P], _I),
    "sp24_fp8_decompress": ([_P, _P, _P, _I64, _I64, _I, _I, _P, _I64, _P], _I),
    "sp24_fp8_gemm": ([_P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _I64, _I, _I, _P, _P, _I64, _P, _P, _I64,
                       _P, _SZ, _P], _I),
    "sp24_fp8_gemm_workspace_size": ([_I64, _I64, _I64, _I64], _SZ),
    "sp24_set_decomposition": ([_I], _I),
    "sp24_fp8_gemm_decomposition": ([_I64, _I64, _I64, _I64, _P], _I),
    "sp24_fp8_gemm_batched": ([_P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _I64, _I, _I, _P, _P, _I64, _I64,
                               _I64, _I64, _I64, _I64, _I64, _I64, _I64, _P, _SZ, _P], _I),
    "sp24_fp8_gemm_fixed_scratch": ([_P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _I64, _I, _I, _P, _P, _I64, _P, _P,
                                     _I64, _P], _I),
    "sp24_last_device_error": ([_P], _I),
    "sp24_int8_compress": ([_P, _I64, _I64, _I64, _P, _P, _P, _P], _I),
    "sp24_int8_quantize_act": ([_P, _I64, _I64, _I64, _P, _P, _P], _I),
    "sp24_int8_gemm": ([_P, _P, _I64, _I64, _I64, _P, _P, _P, _I64, _P, _P, _I64, _P], _I),
    "sp24_qk_norm_rope": ([_P, _I64, _I64, _I, _P, _P, _F, _P, _I64, _I, _I, _P, _P, _P, _I64, _P, _P], _I),
    "sp24_attention_decode": ([_P, _I64, _I64, _I, _P, _P, _I64, _I64, _P, _F, _I, _I, _P, _I64, _P, _SZ, _P], _I),
    "sp24_attention_decode_workspace_size": ([_I, _I, _I], _SZ),
    "sp24_attention_prompt": ([_P, _I64, _I64, _I, _P, _I64, _P, _P, _I64, _I64, _P, _F, _I, _I, _P, _I64, _P, _SZ, _P],
                              _I),
    "sp24_attention_prompt_workspace_size": ([_I64, _I64, _I, _P, _I64, _I, _I], _SZ),
}


class Sp24Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__("%s failed: %s" % (where, SP24_STATUS.get(status, "status %d" % status)))


def library_path() -> str:
    return _build.LIB


def load(build_if_missing: bool = True):
    """Load libsp24.so (building it first if asked and it is absent or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    path = _build.LIB
    if build_if_missing:
        path = _build.build()
    if not os.path.exists(path):
        raise RuntimeError("libsp24.so is not built (run semi_structured_sparse_gb300.build.build())")
    lib = ctypes.CDLL(path)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != 0:
        if status in (1, 2, 3):
            raise ValueError("%s: %s" % (where, SP24_STATUS.get(status, status)))
        raise Sp24Error(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The library launches on the calling thread's current GPU, which need not be the operands'.
_current_gpu = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _on(index, fn, *args):
    """fn(*args) with the GPU `index` as the current one."""
    if _current_gpu() == index:
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def _stream(stream=None, index=None):
    """The handle of `stream`, or of GPU `index`'s current stream; None: the current GPU's."""
    if stream is None:
        stream = torch.cuda.current_stream(index)
    elif index is not None and stream.device_index != index:
        raise ValueError("the stream is one of GPU %d, the operands are on GPU %d" % (stream.device_index, index))
    return ctypes.c_void_p(stream.cuda_stream)


def _new(shape, dtype, stream, device, zero=False):
    """Memory for a kernel on `stream`, from that stream's own pool."""
    make = torch.zeros if zero else torch.empty
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return make(shape, dtype=dtype, device=device)


def _dev_tensor(t, dtype, name, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.stride(-1) != 1:
        raise ValueError("%s must have unit stride in its last dimension" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, the operands on %s" % (name, t.device, device))
    return t


def _cdiv(a, b):
    return (a + b - 1) // b


def _scale_count(K, gK, rows, g):
    """Scales of a [rows, K] operand at granularity g x gK (0 if gK is invalid:
    the library then refuses the call itself)."""
    if not gK or K % gK != 0 or g <= 0:
        return 0
    return (K // gK) * _cdiv(rows, g)


def _at_least(t, n, name):
    """The kernels read or write n elements of t; the C ABI cannot see sizes."""
    if not t.is_contiguous() or t.numel() < n:
        raise ValueError("%s must be contiguous with at least %d elements (has %d)" % (name, n, t.numel()))


def _matrix(t, rows, cols, name):
    """A [rows, cols] matrix with unit column stride and row stride >= cols."""
    if t.dim() != 2 or tuple(t.shape) != (rows, cols) or t.stride(0) < cols:
        raise ValueError("%s must be [%d, %d], got %s" % (name, rows, cols, tuple(t.shape)))


def workspace_size(M: int, N: int, K: int, r: int = 0) -> int:
    """Device scratch bytes gemm() wants for this shape (0 = none)."""
    return int(load().sp24_fp8_gemm_workspace_size(M, N, K, r))


DECOMP_HEURISTIC, DECOMP_DATA_PARALLEL, DECOMP_STREAM_K, DECOMP_CLUSTER_SPLIT = 0, 1, 2, 3


def set_decomposition(mode: int) -> None:
    """How later GEMM calls deal out the tiles' K ranges: DECOMP_HEURISTIC
    (default), DECOMP_DATA_PARALLEL (whole tiles), DECOMP_STREAM_K or
    DECOMP_CLUSTER_SPLIT (process-wide; workspace_size() follows the mode)."""
    _check(load().sp24_set_decomposition(int(mode)), "sp24_set_decomposition")


@contextlib.contextmanager
def decomposition(mode: int):
    """Run a block of GEMM calls under one decomposition mode, then restore
    the heuristic."""
    set_decomposition(mode)
    try:
        yield
    finally:
        set_decomposition(DECOMP_HEURISTIC)


def decomposition_of(M: int, N: int, K: int, r: int = 0):
    """(mode, CTAs per tile) a per-tensor-K call of this shape would use now."""
    cs = ctypes.c_int(1)
    mode = int(load().sp24_fp8_gemm_decomposition(M, N, K, r, ctypes.addressof(cs)))
    if mode < 0:
        raise ValueError("invalid shape or no usable device")
    return mode, cs.value


def meta_bytes(N: int, K: int) -> int:
    return int(load().sp24_meta_bytes(N, K))


def compress(w: torch.Tensor, gN: int = 1, gK: int = None, out=None, stream=None):
    """Magnitude 2:4 prune + e4m3 + pack of a bf16 weight [N, K].

    Returns (values uint8 [N, K/2], meta uint8 [N, K/8], scales fp32 [K/gK, ceil(N/gN)]).
    values and meta hold the library's tiled storage (128 x 128 weight tiles,
    each contiguous; see include/sp24.h), which is what gemm() reads.
    ``out`` may supply those three tensors (no allocation then)."""
    lib = load()
    _dev_tensor(w, torch.bfloat16, "w")
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    N, K = w.shape
    gK = K if gK is None else gK
    if out is None:
        values = _new((N, K // 2), torch.uint8, stream, w.device)
        meta = _new((N, K // 8), torch.uint8, stream, w.device)
        scales = _new((K // gK, (N + gN - 1) // gN), torch.float32, stream, w.device)
    else:
        values, meta, scales = out
        _dev_tensor(values, torch.uint8, "values", w.device)
        _dev_tensor(meta, torch.uint8, "meta", w.device)
        _dev_tensor(scales, torch.float32, "scales", w.device)
        _at_least(values, N * (K // 2), "values")
        _at_least(meta, N * (K // 8), "meta")
        _at_least(scales, _scale_count(K, gK, N, gN), "scales")
    _check(_on(w.get_device(), lib.sp24_fp8_compress, _ptr(w), N, K, w.stride(0), gN, gK, _ptr(values), _ptr(meta),
               _ptr(scales), _stream(stream, w.get_device())), "sp24_fp8_compress")
    return values, meta, scales


def decompress(values, meta, scales, gN: int = 1, gK: int = None, out=None, stream=None):
    """The dense dequantized weight bf16 [N, K] from compress()'s output: at the
    kept positions bf16(scale * e4m3 value), 0 elsewhere."""
    lib = load()
    _dev_tensor(values, torch.uint8, "values")
    if values.dim() != 2:
        raise ValueError("values must be [N, K/2]")
    N, K = values.shape[0], values.shape[1] * 2
    gK = K if gK is None else gK
    _dev_tensor(meta, torch.uint8, "meta", values.device)
    _dev_tensor(scales, torch.float32, "scales", values.device)
    _at_least(values, N * (K // 2), "values")
    _at_least(meta, N * (K // 8), "meta")
    _at_least(scales, _scale_count(K, gK, N, gN), "scales")
    if out is None:
        W = _new((N, K), torch.bfloat16, stream, values.device)
    else:
        W = _dev_tensor(out, torch.bfloat16, "out", values.device)
        _matrix(W, N, K, "out")
    _check(_on(values.get_device(), lib.sp24_fp8_decompress, _ptr(values), _ptr(meta), _ptr(scales), N, K, gN, gK, _ptr(W),
               W.stride(0), _stream(stream, values.get_device())), "sp24_fp8_decompress")
    return W


def quantize_act(x: torch.Tensor, gK: int = None, out=None, stream=None):
    """Dynamic e4m3 quantization of fp32 or bf16 activations [M, K]: returns
    (xq uint8 [M, K], sx fp32 [K/gK, M])."""
    lib = load()
    bf16 = isinstance(x, torch.Tensor) and x.dtype == torch.bfloat16
    _dev_tensor(x, torch.bfloat16 if bf16 else torch.float32, "x")
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    gK = K if gK is None else gK
    if out is None:
        xq = _new((M, K), torch.uint8, stream, x.device)
        sx = _new((K // gK, M), torch.float32, stream, x.device)
    else:
        xq, sx = out
        _dev_tensor(xq, torch.uint8, "xq", x.device)
        _dev_tensor(sx, torch.float32, "sx", x.device)
        _at_least(xq, M * K, "xq")  # written densely, row stride K
        _at_least(sx, _scale_count(K, gK, M, 1), "sx")
    f, name = ((lib.sp24_fp8_quantize_act_bf16, "sp24_fp8_quantize_act_bf16") if bf16
               else (lib.sp24_fp8_quantize_act, "sp24_fp8_quantize_act"))
    _check(_on(x.get_device(), f, _ptr(x), M, K, x.stride(0), gK, _ptr(xq), _ptr(sx), _stream(stream, x.get_device())), name)
    return xq, sx


def gemm(xq, sx, values, meta, sw, gM: int = 1, gN: int = 1, gK: int = None, x2=None, w2=None,
         out=None, workspace=None, stream=None, bias=None):
    """Y[M, N] (bf16) = scaled 2:4 sparse e4m3 GEMM of xq [M, K] with the packed weight
    (values [N, K/2], meta [N, K/8]) plus x2 [M, r] . w2 [N, r]^T and a bf16 bias [N]
    when given.  `workspace` (uint8, at least workspace_size(M, N, K, r) bytes) must be
    zeroed before its first use and may then be reused by later calls of any shape on
    the same stream; without one, each call that needs scratch allocates a zeroed one."""
    lib = load()
    _dev_tensor(xq, torch.uint8, "xq")
    dev_ = xq.device
    _dev_tensor(values, torch.uint8, "values", dev_)
    if xq.dim() != 2 or values.dim() != 2:
        raise ValueError("xq must be [M, K] and values [N, K/2]")
    _dev_tensor(meta, torch.uint8, "meta", dev_)
    _dev_tensor(sx, torch.float32, "sx", dev_)
    _dev_tensor(sw, torch.float32, "sw", dev_)
    M, K = xq.shape
    N = values.shape[0]
    gK = K if gK is None else gK
    r = 0
    if x2 is not None:
        _dev_tensor(x2, torch.bfloat16, "x2", dev_)
        _dev_tensor(w2, torch.bfloat16, "w2", dev_)
        r = x2.shape[1]
        if not (x2.is_contiguous() and w2.is_contiguous()):
            raise ValueError("x2 and w2 must be contiguous")
        _matrix(x2, M, r, "x2")
        _matrix(w2, N, r, "w2")
    if not (sx.is_contiguous() and sw.is_contiguous() and values.is_contiguous() and meta.is_contiguous()):
        raise ValueError("scales, values and meta must be contiguous")
    _at_least(values, N * (K // 2), "values")
    _at_least(meta, N * (K // 8), "meta")
    _at_least(sx, _scale_count(K, gK, M, gM), "sx")
    _at_least(sw, _scale_count(K, gK, N, gN), "sw")
    if bias is not None:
        _dev_tensor(bias, torch.bfloat16, "bias", dev_)
        if not bias.is_contiguous() or bias.numel() != N:
            raise ValueError("bias must be a contiguous bf16 vector of N values")
    if out is None:
        y = _new((M, N), torch.bfloat16, stream, dev_)
    else:
        y = _dev_tensor(out, torch.bfloat16, "out", dev_)
        _matrix(y, M, N, "out")
    ws_bytes = int(_on(xq.get_device(), lib.sp24_fp8_gemm_workspace_size, M, N, K, r))
    if ws_bytes and workspace is None:
        workspace = _new(ws_bytes, torch.uint8, stream, dev_, zero=True)
    elif workspace is not None:
        _dev_tensor(workspace, torch.uint8, "workspace", dev_)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _check(_on(xq.get_device(), lib.sp24_fp8_gemm, _ptr(xq), _ptr(sx), M, K, xq.stride(0), gM, _ptr(values), _ptr(meta),
               _ptr(sw), N, gN, gK, _ptr(x2), _ptr(w2), r, _ptr(bias), _ptr(y), y.stride(0), _ptr(workspace),
               0 if workspace is None else workspace.numel() * workspace.element_size(),
               _stream(stream, xq.get_device())), "sp24_fp8_gemm")
    return y


def gemm_batched(xq, sx, values, meta, sw, gM: int = 1, gN: int = 1, gK: int = None, bias=None, out=None,
                 workspace=None, stream=None):
    """L independent problems of one shape: xq [L, M, K], sx [L, K/gK, ceil(M/gM)],
    values [L, N, K/2], meta [L, N, K/8], sw [L, K/gK, ceil(N/gN)], bias [L, N] or
    None -> Y [L, M, N] bf16, Y[l] = gemm(xq[l], ..., bias[l])."""
    lib = load()
    for t, dt, nm in ((xq, torch.uint8, "xq"), (values, torch.uint8, "values"), (meta, torch.uint8, "meta"),
                      (sx, torch.float32, "sx"), (sw, torch.float32, "sw")):
        _dev_tensor(t, dt, nm)
        if t.dim() != 3 or not t[0].is_contiguous():
            raise ValueError("%s must be [L, ...] with contiguous problems" % nm)
    L, M, K = xq.shape
    N = values.shape[1]
    gK = K if gK is None else gK
    dev_ = xq.device
    for t, nm in ((values, "values"), (meta, "meta"), (sx, "sx"), (sw, "sw")):
        if t.device != dev_ or t.shape[0] != L:
            raise ValueError("%s must hold the same L problems on %s" % (nm, dev_))
    _at_least(values[0], N * (K // 2), "values[l]")
    _at_least(meta[0], N * (K // 8), "meta[l]")
    _at_least(sx[0], _scale_count(K, gK, M, gM), "sx[l]")
    _at_least(sw[0], _scale_count(K, gK, N, gN), "sw[l]")
    if bias is not None:
        _dev_tensor(bias, torch.bfloat16, "bias", dev_)
        if bias.shape != (L, N):
            raise ValueError("bias must be [L, N]")
    if out is None:
        y = _new((L, M, N), torch.bfloat16, stream, dev_)
    else:
        y = _dev_tensor(out, torch.bfloat16, "out", dev_)
        if y.dim() != 3 or tuple(y.shape) != (L, M, N) or y.stride(1) < N:
            raise ValueError("out must be [L, M, N]")
    ws_bytes = L * int(_on(xq.get_device(), lib.sp24_fp8_gemm_workspace_size, M, N, K, 0))
    if ws_bytes and workspace is None:
        workspace = _new(ws_bytes, torch.uint8, stream, dev_, zero=True)
    elif workspace is not None:
        _dev_tensor(workspace, torch.uint8, "workspace", dev_)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    _check(_on(
        xq.get_device(), lib.sp24_fp8_gemm_batched, _ptr(xq), _ptr(sx), M, K, xq.stride(1), gM, _ptr(values), _ptr(meta), _ptr(sw), N, gN, gK, _ptr(bias),
        _ptr(y), y.stride(1), L, xq.stride(0), sx.stride(0), values.stride(0), meta.stride(0), sw.stride(0),
        0 if bias is None else bias.stride(0), y.stride(0), _ptr(workspace),
        0 if workspace is None else workspace.numel() * workspace.element_size(),
        _stream(stream, xq.get_device())), "sp24_fp8_gemm_batched")
    return y


# --------------------------------------------------------------- int8 sibling
def compress_int8(w: torch.Tensor, out=None, stream=None):
    """Magnitude 2:4 prune + int8 (one scale per output channel) + pack of a bf16
    weight [N, K]: (values int8 [N, K/2], meta uint8 [N, K/8], scales fp32 [N]),
    values and meta in the tiled storage gemm_int8() reads."""
    lib = load()
    _dev_tensor(w, torch.bfloat16, "w")
    if w.dim() != 2:
        raise ValueError("w must be [N, K]")
    N, K = w.shape
    if out is None:
        values = _new((N, K // 2), torch.int8, stream, w.device)
        meta = _new((N, K // 8), torch.uint8, stream, w.device)
        scales = _new(N, torch.float32, stream, w.device)
    else:
        values, meta, scales = out
        _dev_tensor(values, torch.int8, "values", w.device)
        _dev_tensor(meta, torch.uint8, "meta", w.device)
        _dev_tensor(scales, torch.float32, "scales", w.device)
        _at_least(values, N * (K // 2), "values")
        _at_least(meta, N * (K // 8), "meta")
        _at_least(scales, N, "scales")
    _check(_on(w.get_device(), lib.sp24_int8_compress, _ptr(w), N, K, w.stride(0), _ptr(values), _ptr(meta), _ptr(scales),
               _stream(stream, w.get_device())), "sp24_int8_compress")
    return values, meta, scales


def quantize_act_int8(x: torch.Tensor, out=None, stream=None):
    """Per-token int8 quantization of fp32 activations [M, K]: (xq int8 [M, K], sx fp32 [M])."""
    lib = load()
    _dev_tensor(x, torch.float32, "x")
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    if out is None:
        xq = _new((M, K), torch.int8, stream, x.device)
        sx = _new(M, torch.float32, stream, x.device)
    else:
        xq, sx = out
        _dev_tensor(xq, torch.int8, "xq", x.device)
        _dev_tensor(sx, torch.float32, "sx", x.device)
        _matrix(xq, M, K, "xq")
        if not xq.is_contiguous():
            raise ValueError("xq must be contiguous")
        _at_least(sx, M, "sx")
    _check(_on(x.get_device(), lib.sp24_int8_quantize_act, _ptr(x), M, K, x.stride(0), _ptr(xq), _ptr(sx),
               _stream(stream, x.get_device())), "sp24_int8_quantize_act")
    return xq, sx


def gemm_int8(xq, sx, values, meta, sw, bias=None, out=None, stream=None):
    """Y[M, N] bf16 = bf16((sx[m] sw[n]) * float(sum of the kept xq[m, k] wq[n, k]) + bias[n])
    for int8 activations xq [M, K] and compress_int8()'s packed weight."""
    lib = load()
    _dev_tensor(xq, torch.int8, "xq")
    dev_ = xq.device
    _dev_tensor(values, torch.int8, "values", dev_)
    if xq.dim() != 2 or values.dim() != 2:
        raise ValueError("xq must be [M, K] and values [N, K/2]")
    _dev_tensor(meta, torch.uint8, "meta", dev_)
    _dev_tensor(sx, torch.float32, "sx", dev_)
    _dev_tensor(sw, torch.float32, "sw", dev_)
    M, K = xq.shape
    N = values.shape[0]
    if not (sx.is_contiguous() and sw.is_contiguous() and values.is_contiguous() and meta.is_contiguous()):
        raise ValueError("scales, values and meta must be contiguous")
    _at_least(values, N * (K // 2), "values")
    _at_least(meta, N * (K // 8), "meta")
    _at_least(sx, M, "sx")
    _at_least(sw, N, "sw")
    if bias is not None:
        _dev_tensor(bias, torch.bfloat16, "bias", dev_)
        if not bias.is_contiguous() or bias.numel() != N:
            raise ValueError("bias must be a contiguous bf16 vector of N values")
    if out is None:
        y = _new((M, N), torch.bfloat16, stream, dev_)
    else:
        y = _dev_tensor(out, torch.bfloat16, "out", dev_)
        _matrix(y, M, N, "out")
    _check(_on(xq.get_device(), lib.sp24_int8_gemm, _ptr(xq), _ptr(sx), M, K, xq.stride(0), _ptr(values), _ptr(meta),
               _ptr(sw), N, _ptr(bias), _ptr(y), y.stride(0), _stream(stream, xq.get_device())), "sp24_int8_gemm")
    return y


# ------------------------------------------------------------------ attention
class _KVCacheStruct(ctypes.Structure):
    """sp24_kv_cache of the C header."""
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("num_pages", _I64), ("page_stride", _I64),
                ("head_stride", _I64), ("token_stride", _I64), ("heads", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class KVCache:
    """A paged cache of keys and values: k and v [pages, heads, page size, head dim]
    (the last dimension with unit stride, the others any, the same for both), as bf16,
    or as uint8 e4m3 codes with k_scale and v_scale fp32 [heads].  It holds on to the
    tensors and owns nothing else; their memory is read and written in place."""

    def __init__(self, k, v, k_scale=None, v_scale=None):
        e4m3 = isinstance(k, torch.Tensor) and k.dtype == torch.uint8
        _dev_tensor(k, torch.uint8 if e4m3 else torch.bfloat16, "k")
        _dev_tensor(v, k.dtype, "v", k.device)
        if k.dim() != 4 or k.shape != v.shape or any(
                a != b for n, a, b in zip(k.shape, k.stride(), v.stride()) if n > 1):
            raise ValueError("k and v must be [pages, heads, page size, head dim] of one shape and one set of strides")
        pages, heads, page_size, head_dim = k.shape
        if pages < 1 or heads < 1 or head_dim not in (64, 128) or page_size not in (16, 32, 64, 128):
            raise ValueError("a cache needs a page and a head, pages of 16, 32, 64 or 128 tokens and heads of 64 or "
                             "128, got %s" % (tuple(k.shape),))
        if e4m3 != (k_scale is not None) or e4m3 != (v_scale is not None):
            raise ValueError("k_scale and v_scale go with uint8 e4m3 codes, and only with them")
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is not None:
                _dev_tensor(t, torch.float32, name, k.device)
                _at_least(t, heads, name)
        # An axis of one entry is never stepped along, and its stride may be anything.
        token = k.stride(2)
        head = k.stride(1) if heads > 1 else page_size * token
        page = k.stride(0) if pages > 1 else max(heads * head, page_size * token)
        if min(page, head, token) < head_dim or (page | head | token) * k.element_size() % 16 or \
                (k.data_ptr() | v.data_ptr()) % 16:
            raise ValueError("the cache's rows must not overlap, and start on 16-byte boundaries")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.heads, self.page_size, self.head_dim, self.device = heads, page_size, head_dim, k.device
        self._index = k.get_device()
        self._scale = head_dim ** -0.5
        self._struct = _KVCacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr() if e4m3 else None,
                                      v_scale.data_ptr() if e4m3 else None, pages, page, head, token, heads,
                                      page_size, head_dim, 1 if e4m3 else 0)
        self._address = ctypes.addressof(self._struct)


# The calls below run on every step of a decode loop, where a call's time on the
# host is several times its kernel's.  So each first asks its tensors, in one
# expression, whether all is as it should be, and only a call that is not goes
# through the checks that say what is wrong.
_BF16, _F32, _I32, _INT64, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.uint8


def _rows_of(t, rows, cols, cache, name):
    """Checks a bf16 tensor of `rows` rows, [rows, cols] or [rows, heads, d] with contiguous rows."""
    _dev_tensor(t, torch.bfloat16, name, cache.device)
    shape = tuple(t.shape)
    if not (_row_stride(t, cols) and shape[0] == rows):
        raise ValueError("%s must be [%d, %d] or [%d, heads, head dim] with contiguous rows, got %s with strides %s"
                         % (name, rows, cols, rows, shape, t.stride()))


def _row_stride(t, cols):
    """The row stride of a tensor whose rows are `cols` contiguous values (0: they are not)."""
    shape, stride = t.shape, t.stride()
    if len(shape) == 3:
        if shape[1] * shape[2] != cols or stride[2] != 1 or (stride[1] != shape[2] and shape[1] != 1):
            return 0
    elif len(shape) != 2 or shape[1] != cols or stride[1] != 1:
        return 0
    return stride[0] if shape[0] > 1 else cols  # a lone row's stride is never stepped along


def _vector(t, dtype, n, cache, name):
    _dev_tensor(t, dtype, name, cache.device)
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector of %d values, got %s" % (name, n, tuple(t.shape)))


def _matrix_of(t, dtype, cache, name, what):
    _dev_tensor(t, dtype, name, cache.device)
    if t.dim() != 2:
        raise ValueError("%s must be %s, got %s" % (name, what, tuple(t.shape)))


# The current stream's handle without a Stream object around it, where torch has that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, cache):
    if stream is not None:
        if stream.device_index != cache._index:
            raise ValueError("the stream is one of GPU %d, the cache is on GPU %d" % (stream.device_index, cache._index))
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(cache._index)
    return torch.cuda.current_stream(cache.device).cuda_stream


_MOST = 2 ** 31 - 1


def _int32(n):
    """A count of tokens that may pass 32 bits: above them it is all there are, and below zero stays below."""
    return min(max(n, -1), _MOST)  # (ctypes would keep the low 32 bits)


def qk_norm_rope(qkv, heads: int, cache: KVCache, positions, slots, cos_sin, q_weight=None, k_weight=None,
                 eps: float = 1e-6, interleaved: bool = False, out=None, stream=None):
    """One pass over the QKV projection's rows: per-head RMS norm (with q_weight and
    k_weight bf16 [head dim]; neither: no norm) and rotation of queries and keys, keys
    and values appended to the cache.

    qkv bf16 [T, (heads + 2 cache heads) * head dim]: query heads, key heads, value
    heads.  positions int32 [T]: each token's row of cos_sin fp32 [max_pos, rot] (rot/2
    cosines, then rot/2 sines); rot of the head dim's values are rotated, as pairs
    (i, i + rot/2), or (2i, 2i + 1) if interleaved.  slots int64 [T]: page * page_size +
    place of each token, negative for one that is not stored.  Returns the queries bf16
    [T, heads, head dim] (in ``out`` if given)."""
    lib = _lib or load()
    d, at = cache.head_dim, cache._index
    ok = False
    try:
        T = slots.shape[0]
        ldqkv = _row_stride(qkv, (heads + 2 * cache.heads) * d)
        max_pos, rot = cos_sin.shape
        if out is None:
            out, ldq = _new((T, heads, d), _BF16, stream, cache.device), heads * d
        else:
            ldq = _row_stride(out, heads * d)
        qw = kw = None
        ok = (slots.dtype is _INT64 and slots.dim() == 1 and slots.is_contiguous() and slots.get_device() == at and
              positions.dtype is _I32 and positions.shape == slots.shape and positions.is_contiguous() and
              positions.get_device() == at and qkv.dtype is _BF16 and ldqkv and qkv.shape[0] == T and
              qkv.get_device() == at and out.dtype is _BF16 and ldq and out.shape[0] == T and
              out.get_device() == at and cos_sin.dtype is _F32 and cos_sin.is_contiguous() and
              cos_sin.get_device() == at)
        if q_weight is not None or k_weight is not None:
            ok = (ok and q_weight.dtype is _BF16 and q_weight.shape == (d,) and q_weight.is_contiguous() and
                  q_weight.get_device() == at and k_weight.dtype is _BF16 and k_weight.shape == (d,) and
                  k_weight.is_contiguous() and k_weight.get_device() == at)
            qw, kw = q_weight.data_ptr(), k_weight.data_ptr()
    except (AttributeError, IndexError, ValueError, TypeError):
        ok = False
    if not ok:
        _vector(slots, _INT64, slots.numel() if isinstance(slots, torch.Tensor) else 0, cache, "slots")
        T = slots.shape[0]
        _vector(positions, _I32, T, cache, "positions")
        _rows_of(qkv, T, (heads + 2 * cache.heads) * d, cache, "qkv")
        if out is not None:
            _rows_of(out, T, heads * d, cache, "out")
        _matrix_of(cos_sin, _F32, cache, "cos_sin", "[max_pos, rot]")
        if (q_weight is None) != (k_weight is None):
            raise ValueError("q_weight and k_weight go together")
        if q_weight is not None:
            _vector(q_weight, _BF16, d, cache, "q_weight")
            _vector(k_weight, _BF16, d, cache, "k_weight")
        raise ValueError("cos_sin must be contiguous")
    st = _on(at, lib.sp24_qk_norm_rope, qkv.data_ptr(), T, ldqkv, heads, qw, kw, eps, cos_sin.data_ptr() if rot else None,
             max_pos, rot, 1 if interleaved else 0, positions.data_ptr(), slots.data_ptr(), out.data_ptr(), ldq,
             cache._address, _stream_of(stream, cache))
    if st:
        _check(st, "sp24_qk_norm_rope")
    return out


def attention_decode_workspace_size(cache: KVCache, heads: int) -> int:
    """Device scratch bytes attention_decode() needs for `heads` query heads."""
    return int(_on(cache._index, load().sp24_attention_decode_workspace_size, heads, cache.heads, cache.head_dim))


def _attention_args(q, cache, page_table, seq_lens, scale, out, stream):
    """The checks and arguments that both attention calls have in common."""
    d, at = cache.head_dim, cache._index
    ok = False
    try:
        shape = q.shape
        cols = shape[1] * shape[2] if len(shape) == 3 else shape[1]
        rows, heads = shape[0], cols // d
        ldq = _row_stride(q, cols)
        B, width = page_table.shape
        if out is None:
            out, ldy = _new(shape, _BF16, stream, cache.device), cols
        else:
            ldy = _row_stride(out, cols)
        ok = (q.dtype is _BF16 and ldq and q.get_device() == at and shape[-1] % d == 0 and
              (len(shape) == 2 or shape[2] == d) and out.dtype is _BF16 and ldy and out.shape[0] == rows and
              out.get_device() == at and page_table.dtype is _I32 and (page_table.stride(1) == 1 or width == 1) and
              page_table.get_device() == at and seq_lens.dtype is _I32 and seq_lens.shape == (B,) and
              seq_lens.is_contiguous() and seq_lens.get_device() == at)
    except (AttributeError, IndexError, ValueError, TypeError):
        ok = False
    if not ok:
        if not isinstance(q, torch.Tensor) or q.dim() not in (2, 3) or q.shape[-1] % d or (
                q.dim() == 3 and q.shape[2] != d):
            raise ValueError("q must be [rows, heads, %d] or [rows, heads * %d]" % (d, d))
        cols = q.shape[1] * q.shape[2] if q.dim() == 3 else q.shape[1]
        _rows_of(q, q.shape[0], cols, cache, "q")
        _matrix_of(page_table, _I32, cache, "page_table", "[sequences, pages]")
        _vector(seq_lens, _I32, page_table.shape[0], cache, "seq_lens")
        _rows_of(out, q.shape[0], cols, cache, "out")
        raise ValueError("the arguments' layouts are not ones that the library takes")
    ld_table = page_table.stride(0) if B > 1 else width
    return rows, ldq, heads, B, width, ld_table, seq_lens.data_ptr(), cache._scale if scale is None else scale, out, ldy


def attention_decode(q, cache: KVCache, page_table, seq_lens, scale: float = None, window: int = 0, sinks: int = 0,
                     out=None, workspace=None, stream=None):
    """Attention of one new token per sequence over the cache, which already holds it:
    q bf16 [B, heads, head dim], page_table int32 [B, pages], seq_lens int32 [B] (the new
    token included) -> bf16 like q.  With a window only the latest `window` tokens and the
    first `sinks` are seen.  scale defaults to head_dim ** -0.5.  `workspace` (uint8,
    attention_decode_workspace_size() bytes, zeroed once) may be kept for all later calls
    on one stream; without one, each call allocates a zeroed one."""
    lib = _lib or load()
    rows, ldq, heads, B, width, ld_table, lens_p, scale, out, ldy = _attention_args(
        q, cache, page_table, seq_lens, scale, out, stream)
    if rows != B:
        raise ValueError("q has %d rows, page_table %d sequences" % (rows, B))
    if not (0 <= window <= _MOST and 0 <= sinks <= _MOST):
        window, sinks = _int32(window), _int32(sinks)
    if workspace is None:
        workspace = _new(attention_decode_workspace_size(cache, heads), torch.uint8, stream, cache.device, zero=True)
    elif not (isinstance(workspace, torch.Tensor) and workspace.dtype is _U8 and
              workspace.get_device() == cache._index and workspace.is_contiguous()):
        _dev_tensor(workspace, _U8, "workspace", cache.device)
        raise ValueError("workspace must be contiguous")
    st = _on(cache._index, lib.sp24_attention_decode, q.data_ptr(), B, ldq, heads, cache._address, page_table.data_ptr(),
             width, ld_table, lens_p, scale, window, sinks, out.data_ptr(), ldy, workspace.data_ptr(), workspace.numel(),
             _stream_of(stream, cache))
    if st:
        _check(st, "sp24_attention_decode")
    return out


def attention_prompt_workspace_size(cache: KVCache, heads: int, rows: int, sequences: int, pages: int, window: int = 0,
                                    sinks: int = 0) -> int:
    """Device scratch bytes attention_prompt() would use for `rows` query rows of `heads`
    heads in `sequences` sequences with page tables of `pages` entries (0: none)."""
    return int(_on(cache._index, load().sp24_attention_prompt_workspace_size, rows, sequences, heads, cache._address, pages,
                   _int32(window), _int32(sinks)))


def attention_prompt(q, cu_q, cache: KVCache, page_table, seq_lens, scale: float = None, window: int = 0,
                     sinks: int = 0, out=None, workspace=None, stream=None):
    """Causal attention of a ragged batch of new tokens over the cache, which already
    holds them: sequence b has the rows cu_q[b] .. cu_q[b + 1] - 1 of q bf16 [T, heads,
    head dim], the last of the seq_lens[b] tokens that the cache holds for it.  cu_q int32
    [B + 1]; the others as for attention_decode().  `workspace` (uint8, of any contents, at
    least attention_prompt_workspace_size() bytes) is what few rows over a long cache are
    split through; without one, a call that would use it allocates it."""
    lib = _lib or load()
    rows, ldq, heads, B, width, ld_table, lens_p, scale, out, ldy = _attention_args(
        q, cache, page_table, seq_lens, scale, out, stream)
    if not (isinstance(cu_q, torch.Tensor) and cu_q.dtype is _I32 and cu_q.shape == (B + 1,) and cu_q.is_contiguous() and
            cu_q.get_device() == cache._index):
        _vector(cu_q, _I32, B + 1, cache, "cu_q")
    if not (0 <= window <= _MOST and 0 <= sinks <= _MOST):
        window, sinks = _int32(window), _int32(sinks)
    if workspace is None:
        # (Page tables of fewer tokens are never cut: the library asks for 512 keys per part.)
        need = width * cache.page_size >= 1024 and _on(
            cache._index, lib.sp24_attention_prompt_workspace_size, rows, B, heads, cache._address, width, window, sinks)
        if need:
            workspace = _new(need, _U8, stream, cache.device)
    elif not (isinstance(workspace, torch.Tensor) and workspace.dtype is _U8 and
              workspace.get_device() == cache._index and workspace.is_contiguous()):
        _dev_tensor(workspace, _U8, "workspace", cache.device)
        raise ValueError("workspace must be contiguous")
    st = _on(cache._index, lib.sp24_attention_prompt, q.data_ptr(), rows, ldq, heads, cu_q.data_ptr(), B, cache._address,
             page_table.data_ptr(), width, ld_table, lens_p, scale, window, sinks, out.data_ptr(), ldy,
             None if workspace is None else workspace.data_ptr(), 0 if workspace is None else workspace.numel(),
             _stream_of(stream, cache))
    if st:
        _check(st, "sp24_attention_prompt")
    return out


def last_device_error(stream=None):
    """Synchronise and raise if any library kernel gave up on a bounded wait, or met an
    index out of range, on the stream's GPU (without a stream: on the current one)."""
    index = _current_gpu() if stream is None else stream.device_index
    _check(_on(index, load().sp24_last_device_error, _stream(stream)), "device")
