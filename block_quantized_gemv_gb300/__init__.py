"""Python binding of libbqgemv (block-quantized skinny GEMV for sm_103a).

A thin ctypes layer over the C ABI in include/bqgemv.h: every function here
has the name of its C entry point without the ``bqg_`` prefix, checks that
the torch tensors it is given match the C contract, and passes raw device
pointers plus the current CUDA stream.  Where the C contract allows host
memory (the output of a single-matrix GEMV, either side of copy_sm), a pinned
CPU tensor is passed as its device-side alias (bqg_host_alias).  All
arithmetic runs in the library's CUDA kernels; PyTorch only provides memory
and streams.  There is no fallback: if the shared library is missing, every
call raises.  Every CUDA tensor must be on the current device (ValueError
otherwise, before anything is launched).
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

BF16, Q8_0, Q4_0, Q8_1, F32 = 0, 1, 2, 3, 4
OP_GEMV_BF16, OP_GEMV_Q8_0, OP_GEMV_Q4_0, OP_GEMV_Q4_0_Q8_1 = 0, 1, 2, 3
OP_QKV_Q4_0_Q8_1, OP_GATE_UP_Q4_0_Q8_1, OP_GEMM_Q4_0_BF16 = 4, 5, 6
OP_GATE_UP_Q8_1_Q4_0_Q8_1, OP_GEMM_Q8_0_BF16, OP_DECODE_LAYER_Q4_0_Q8_1 = 7, 8, 9
BLOCK_BYTES = {Q8_0: 34, Q4_0: 18, Q8_1: 36}
QK = 32
TILE_BYTES = {Q8_0: 1088, Q4_0: 576}     # 32 blocks of one repacked row

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_build", "libbqgemv.so")

EXPORTS = {
    # name: (argtypes, restype)
    "bqg_repacked_size": (["i", "i64", "i64"], "size"),
    "bqg_quantize_weights": (["i", "p", "p", "i64", "i64", "p"], "i"),
    "bqg_repack_weights": (["i", "p", "p", "i64", "i64", "p"], "i"),
    "bqg_quantize_q8_1": (["p", "i", "p", "i", "i64", "p"], "i"),
    "bqg_rmsnorm_quantize_q8_1": (["p", "i", "p", "f", "p", "i", "i64", "p"], "i"),
    "bqg_gemv_bf16": (["p", "p", "p", "i", "i64", "i64", "p", "size", "p"], "i"),
    "bqg_gemv_q8_0": (["p", "p", "p", "i", "i64", "i64", "p", "size", "p"], "i"),
    "bqg_gemv_q4_0": (["p", "p", "p", "i", "i64", "i64", "p", "size", "p"], "i"),
    "bqg_gemv_q4_0_q8_1": (["p", "p", "p", "i", "i64", "i64", "p", "size", "p"], "i"),
    "bqg_gemv_q4_0_q8_1_qkv": (["p", "p", "p", "p", "p", "p", "p", "i", "i64", "i64", "i64", "p", "size", "p"], "i"),
    "bqg_gemv_q4_0_q8_1_gate_up_swiglu": (["p", "p", "p", "p", "i", "i64", "i64", "p", "size", "p"], "i"),
    "bqg_gemv_q4_0_q8_1_gate_up_swiglu_q8_1": (["p", "p", "p", "p", "i", "i64", "i64", "p", "size", "p"], "i"),
    "bqg_decode_layer_q4_0_q8_1": (["p", "p", "i", "p", "p", "p", "p", "p", "p", "p", "p", "p", "p", "i", "i64",
                                    "i64", "i64", "i64", "p", "size", "p"], "i"),
    "bqg_gemm_q4_0_bf16": (["p", "p", "p", "i", "i64", "i64", "p", "size", "p"], "i"),
    "bqg_gemm_q8_0_bf16": (["p", "p", "p", "i", "i64", "i64", "p", "size", "p"], "i"),
    "bqg_debug_q4_0_q8_1_block_dots": (["p", "p", "p", "i64", "i64", "p"], "i"),
    "bqg_debug_q4_0_q8_1_block_dots_kslice": (["p", "p", "p", "i64", "i64", "p"], "i"),
    "bqg_workspace_size": (["i", "i", "i64", "i64"], "size"),
    "bqg_gemv_route": (["i", "i", "i64", "i64", "p"], "i"),
    "bqg_last_device_error": (["p", "p"], "i"),
    "bqg_set_pdl": (["i"], "i"),
    "bqg_host_alias": (["p", "p"], "i"),
    "bqg_copy_sm": (["p", "p", "size", "p"], "i"),
    "bqg_status_string": (["i"], "str"),
    "bqg_version": ([], "str"),
    "bqg_last_cuda_error": ([], "str"),
    "bqg_qk_norm_rope": (["p", "p", "i", "i64", "i64", "i64", "i", "i", "i", "i", "p", "p", "f", "p", "p", "i64", "i",
                          "i", "p", "p", "p"], "i"),
    "bqg_qk_norm_rope_kv_write": (["p", "p", "p", "i", "i64", "i64", "i64", "i64", "i", "i", "p", "p", "f", "p", "p",
                                   "i64", "i", "i", "p", "p", "p", "p"], "i"),
    "bqg_kv_write": (["p", "p", "i", "i64", "i64", "i64", "p", "p", "p"], "i"),
    "bqg_kv_read": (["p", "p", "i64", "i", "p", "p", "p"], "i"),
    "bqg_tree_attention": (["p", "i64", "p", "p", "i64", "p", "p", "i", "i64", "i", "i", "p", "f", "p", "p", "size",
                            "p"], "i"),
    "bqg_tree_attention_workspace_size": (["p", "i", "i", "i"], "size"),
    "bqg_shared_prefix_attention": (["p", "i64", "p", "p", "i64", "p", "p", "i", "i64", "i", "i", "p", "p", "i", "i64", "p",
                                     "f", "p", "p", "size", "p"], "i"),
    "bqg_shared_prefix_attention_workspace_size": (["p", "i", "i", "i", "i64", "i", "i64"], "size"),
    "bqg_tree_verify": (["p", "p", "i", "i64", "i64", "i64", "p", "p", "p", "i", "i64", "i", "p", "p", "p", "p", "p"], "i"),
    "bqg_kv_compact": (["p", "p", "i64", "p", "p", "p", "i", "i", "p", "p"], "i"),
    "bqg_kv_fork": (["p", "p", "i64", "i", "p", "p", "p", "p", "i", "p"], "i"),
    "bqg_gemv_q4_0_q8_1_noalloc": (["p", "p", "p", "i", "i64", "i64", "p"], "i"),
    "bqg_noalloc_scratch_bytes": ([], "size"),
}
_CT = {"i": ctypes.c_int, "i64": ctypes.c_int64, "p": ctypes.c_void_p, "size": ctypes.c_size_t,
       "str": ctypes.c_char_p, "f": ctypes.c_float}

_lock = threading.Lock()
_lib = None


class BqgError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        detail = f" [{load().bqg_last_cuda_error().decode()}]" if status == 5 else ""
        super().__init__(f"{where}: {status_string(status)} (status {status}){detail}")


def load(path: str | None = None) -> ctypes.CDLL:
    """Load (once) and return the shared library; raises if it is not built."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"libbqgemv is not built ({p} missing); run "
                                   "block_quantized_gemv_gb300.build.build()")
            L = ctypes.CDLL(p)
            for name, (args, res) in EXPORTS.items():
                fn = getattr(L, name)
                fn.argtypes = [_CT[a] for a in args]
                fn.restype = _CT[res]
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return load().bqg_status_string(int(status)).decode()


def version() -> str:
    return load().bqg_version().decode()


def _check(status: int, where: str):
    if status != 0:
        raise BqgError(status, where)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_cur_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream(stream=None) -> int:
    """The stream handle to enqueue on: `stream`, else torch's current stream
    of the current device (read without building a Stream object)."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and _cur_device is not None:
        return _raw_stream(_cur_device())
    return torch.cuda.current_stream().cuda_stream


def _current_device() -> int:
    return _cur_device() if _cur_device is not None else torch.cuda.current_device()


def check_device(index: int, current: int, name: str) -> None:
    """A CUDA tensor must live on the current device: the library launches
    on the current device and would otherwise dereference another GPU's
    memory."""
    if index != current:
        raise ValueError(f"{name} is on cuda:{index} but the current device is cuda:{current}; "
                         f"call under torch.cuda.device({index})")


def _check_tensor(t: torch.Tensor, name: str, dtype=None, numel=None) -> None:
    """Layout, dtype and size checks shared by device and host operands:
    `numel` is the byte count the call will touch."""
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if numel is not None and t.nbytes < numel:
        raise ValueError(f"{name} holds {t.nbytes} bytes, needs {numel}")


def _dev(t: torch.Tensor, name: str, dtype=None, numel=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    check_device(t.device.index, _current_device(), name)
    _check_tensor(t, name, dtype, numel)
    return t.data_ptr()


def weight_bytes(fmt: int, N: int, K: int):
    """Bytes of N repacked weight rows of K values (the layout of
    include/bqgemv.h: bf16 row-major; q4_0 / q8_0 rows of ceil(K/32/32)
    tiles of 576 / 1088 bytes), or None for a shape the library refuses by
    itself (K not a positive multiple of 32, N < 1).  The C boundary takes
    the weights as a bare pointer, so the binding checks their size."""
    if N < 1 or K < 1 or K % QK:
        return None
    if fmt == BF16:
        return N * K * 2
    return N * ((K // QK + 31) // 32) * TILE_BYTES[fmt]


def host_alias(t: torch.Tensor) -> int:
    """Device-side address of a page-locked (pinned) CPU tensor's memory:
    kernels given it read or write host memory over the CPU-GPU link."""
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise TypeError("host_alias wants a pinned CPU tensor")
    if not t.is_contiguous():
        raise ValueError("the tensor must be contiguous")
    out = ctypes.c_void_p(0)
    _check(load().bqg_host_alias(t.data_ptr(), ctypes.addressof(out)), "bqg_host_alias")
    return out.value


def _dev_or_host(t: torch.Tensor, name: str, dtype=None, numel=None):
    """_dev for a CUDA tensor; the host alias for a pinned CPU tensor."""
    if isinstance(t, torch.Tensor) and not t.is_cuda and t.is_pinned():
        _check_tensor(t, name, dtype, numel)
        return host_alias(t)
    return _dev(t, name, dtype, numel)


def copy_sm(dst: torch.Tensor, src: torch.Tensor, stream=None) -> torch.Tensor:
    """Copy src's bytes into dst with a kernel instead of a copy engine; each
    of the two may be a CUDA tensor or a pinned CPU tensor."""
    n = src.nbytes
    _check(load().bqg_copy_sm(_dev_or_host(dst, "dst", numel=n), _dev_or_host(src, "src"), n, _stream(stream)),
           "bqg_copy_sm")
    return dst


def _ws(ws):
    if ws is None:
        return None, 0
    return _dev(ws, "ws"), ws.nbytes


def row_bytes(fmt: int, K: int) -> int:
    """Bytes of one canonical row (bf16: 2K; block formats: K/32 blocks)."""
    return 2 * K if fmt == BF16 else (K // QK) * BLOCK_BYTES[fmt]


# --- load time -----------------------------------------------------------------
def repacked_size(fmt: int, N: int, K: int) -> int:
    return int(load().bqg_repacked_size(fmt, N, K))


def quantize_weights(fmt: int, W: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """fp32 N x K -> canonical q8_0/q4_0 blocks (uint8, N x row_bytes)."""
    N, K = W.shape
    if out is None:
        out = torch.empty((N, row_bytes(fmt, K)), dtype=torch.uint8, device=W.device)
    _check(load().bqg_quantize_weights(fmt, _dev(W, "W", torch.float32),
                                       _dev(out, "out", numel=N * row_bytes(fmt, K)), N, K, _stream(stream)),
           "bqg_quantize_weights")
    return out


def repack_weights(fmt: int, src: torch.Tensor, N: int, K: int, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    size = repacked_size(fmt, N, K)
    if out is None:
        out = torch.empty(size, dtype=torch.uint8, device=src.device)
    _check(load().bqg_repack_weights(fmt, _dev(src, "src", numel=N * row_bytes(fmt, K)),
                                     _dev(out, "out", numel=size), N, K, _stream(stream)),
           "bqg_repack_weights")
    return out


# --- per token -----------------------------------------------------------------
def quantize_q8_1(x: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """bf16 or fp32 M x K -> q8_1 blocks (uint8, M x K/32*36)."""
    M, K = x.shape
    dt = {torch.bfloat16: BF16, torch.float32: F32}.get(x.dtype)
    if dt is None:
        raise TypeError("x must be bf16 or fp32")
    if out is None:
        out = torch.empty((M, row_bytes(Q8_1, K)), dtype=torch.uint8, device=x.device)
    _check(load().bqg_quantize_q8_1(_dev(x, "x"), dt, _dev(out, "out", numel=M * row_bytes(Q8_1, K)), M, K,
                                    _stream(stream)), "bqg_quantize_q8_1")
    return out


def rmsnorm_quantize_q8_1(x: torch.Tensor, gamma: torch.Tensor | None = None, eps: float = 1e-5,
                          out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Fused RMSNorm (optional fp32 gain `gamma`) + q8_1 quantization:
    bf16 or fp32 M x K -> q8_1 blocks (uint8, M x K/32*36)."""
    M, K = x.shape
    dt = {torch.bfloat16: BF16, torch.float32: F32}.get(x.dtype)
    if dt is None:
        raise TypeError("x must be bf16 or fp32")
    if out is None:
        out = torch.empty((M, row_bytes(Q8_1, K)), dtype=torch.uint8, device=x.device)
    g = None if gamma is None else _dev(gamma, "gamma", torch.float32, K * 4)
    _check(load().bqg_rmsnorm_quantize_q8_1(_dev(x, "x"), dt, g, float(eps),
                                            _dev(out, "out", numel=M * row_bytes(Q8_1, K)), M, K, _stream(stream)),
           "bqg_rmsnorm_quantize_q8_1")
    return out


def _gemv(fn: str, wfmt: int, Wp, X, N: int, K: int, M: int, out, ws, stream, xbytes):
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=X.device)
    wsp, wsb = _ws(ws)
    _check(getattr(load(), fn)(_dev(Wp, "Wp", numel=weight_bytes(wfmt, N, K)), _dev(X, "X", numel=xbytes),
                               _dev_or_host(out, "Y", torch.float32, M * N * 4), M, N, K, wsp, wsb, _stream(stream)),
           fn)
    return out


def gemv_bf16(Wp, X, N, K, out=None, ws=None, stream=None):
    return _gemv("bqg_gemv_bf16", BF16, Wp, X, N, K, X.shape[0], out, ws, stream, X.shape[0] * K * 2)


def gemv_q8_0(Wp, X, N, K, out=None, ws=None, stream=None):
    return _gemv("bqg_gemv_q8_0", Q8_0, Wp, X, N, K, X.shape[0], out, ws, stream, X.shape[0] * K * 2)


def gemv_q4_0(Wp, X, N, K, out=None, ws=None, stream=None):
    return _gemv("bqg_gemv_q4_0", Q4_0, Wp, X, N, K, X.shape[0], out, ws, stream, X.shape[0] * K * 2)


def gemv_q4_0_q8_1(Wp, Xq, N, K, out=None, ws=None, stream=None):
    M = Xq.shape[0]
    return _gemv("bqg_gemv_q4_0_q8_1", Q4_0, Wp, Xq, N, K, M, out, ws, stream, M * row_bytes(Q8_1, K))


def gemv_q4_0_q8_1_noalloc(Wp, Xq, N, K, out=None, stream=None):
    """bqg_gemv_q4_0_q8_1 without a workspace argument: split-K scratch comes
    from a fixed array inside the library (for callers that cannot allocate)."""
    M = Xq.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=Xq.device)
    _check(load().bqg_gemv_q4_0_q8_1_noalloc(_dev(Wp, "Wp", numel=weight_bytes(Q4_0, N, K)), _dev(Xq, "Xq", numel=M * row_bytes(Q8_1, K)),
                                             _dev_or_host(out, "Y", torch.float32, M * N * 4), M, N, K,
                                             _stream(stream)), "bqg_gemv_q4_0_q8_1_noalloc")
    return out


def gemv_q4_0_q8_1_qkv(Wq, Wk, Wv, Xq, Nq, Nkv, K, out=None, ws=None, stream=None):
    M = Xq.shape[0]
    dev = Xq.device
    if out is None:
        out = (torch.empty((M, Nq), dtype=torch.float32, device=dev),
               torch.empty((M, Nkv), dtype=torch.float32, device=dev),
               torch.empty((M, Nkv), dtype=torch.float32, device=dev))
    Yq, Yk, Yv = out
    wsp, wsb = _ws(ws)
    _check(load().bqg_gemv_q4_0_q8_1_qkv(_dev(Wq, "Wq", numel=weight_bytes(Q4_0, Nq, K)),
                                         _dev(Wk, "Wk", numel=weight_bytes(Q4_0, Nkv, K)),
                                         _dev(Wv, "Wv", numel=weight_bytes(Q4_0, Nkv, K)),
                                         _dev(Xq, "Xq", numel=M * row_bytes(Q8_1, K)),
                                         _dev(Yq, "Yq", torch.float32, M * Nq * 4),
                                         _dev(Yk, "Yk", torch.float32, M * Nkv * 4),
                                         _dev(Yv, "Yv", torch.float32, M * Nkv * 4),
                                         M, Nq, Nkv, K, wsp, wsb, _stream(stream)), "bqg_gemv_q4_0_q8_1_qkv")
    return out


def gemv_q4_0_q8_1_gate_up_swiglu(Wg, Wu, Xq, N, K, out=None, ws=None, stream=None):
    M = Xq.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=Xq.device)
    wsp, wsb = _ws(ws)
    _check(load().bqg_gemv_q4_0_q8_1_gate_up_swiglu(_dev(Wg, "Wg", numel=weight_bytes(Q4_0, N, K)),
                                                    _dev(Wu, "Wu", numel=weight_bytes(Q4_0, N, K)),
                                                    _dev(Xq, "Xq", numel=M * row_bytes(Q8_1, K)),
                                                    _dev(out, "H", torch.float32, M * N * 4), M, N, K, wsp, wsb,
                                                    _stream(stream)), "bqg_gemv_q4_0_q8_1_gate_up_swiglu")
    return out


def gemv_q4_0_q8_1_gate_up_swiglu_q8_1(Wg, Wu, Xq, N, K, out=None, ws=None, stream=None):
    """gate+up+SwiGLU writing h as q8_1 blocks (uint8, M x N/32*36).  `ws`
    (workspace(OP_GATE_UP_Q8_1_Q4_0_Q8_1, ...)) must start zero-filled."""
    M = Xq.shape[0]
    if out is None:
        out = torch.empty((M, row_bytes(Q8_1, N)), dtype=torch.uint8, device=Xq.device)
    wsp, wsb = _ws(ws)
    _check(load().bqg_gemv_q4_0_q8_1_gate_up_swiglu_q8_1(_dev(Wg, "Wg", numel=weight_bytes(Q4_0, N, K)),
                                                         _dev(Wu, "Wu", numel=weight_bytes(Q4_0, N, K)),
                                                         _dev(Xq, "Xq", numel=M * row_bytes(Q8_1, K)),
                                                         _dev(out, "Hq", numel=M * row_bytes(Q8_1, N)), M, N, K,
                                                         wsp, wsb, _stream(stream)),
           "bqg_gemv_q4_0_q8_1_gate_up_swiglu_q8_1")
    return out


def decode_layer_q4_0_q8_1(xa, xb, Wq, Wk, Wv, Wg, Wu, Wd, Nq, Nkv, Nff, K, out=None, ws=None, stream=None):
    """One decode layer (M = 1) in one persistent launch: q8_1 of xa and xb,
    QKV from xa, gate+up+SwiGLU (h as q8_1) from xb, down projection of h.
    xa, xb: (1, K) bf16 or fp32.  Returns (Yq, Yk, Yv, Y).  `ws`
    (workspace(OP_DECODE_LAYER_Q4_0_Q8_1, 1, Nff, K)) must start zero-filled;
    it also holds h's q8_1 blocks (see `layer_hq`)."""
    if xa.dtype not in (torch.bfloat16, torch.float32) or xb.dtype != xa.dtype:
        raise TypeError("xa and xb must both be bfloat16 or both float32")
    dt = F32 if xa.dtype == torch.float32 else BF16
    nx = K * xa.element_size()
    if out is None:
        dev = xa.device
        out = tuple(torch.empty(n, dtype=torch.float32, device=dev) for n in (Nq, Nkv, Nkv, K))
    Yq, Yk, Yv, Y = out
    wsp, wsb = _ws(ws)
    _check(load().bqg_decode_layer_q4_0_q8_1(_dev(xa, "xa", numel=nx), _dev(xb, "xb", numel=nx), dt,
                                             _dev(Wq, "Wq", numel=weight_bytes(Q4_0, Nq, K)),
                                             _dev(Wk, "Wk", numel=weight_bytes(Q4_0, Nkv, K)),
                                             _dev(Wv, "Wv", numel=weight_bytes(Q4_0, Nkv, K)),
                                             _dev(Wg, "Wg", numel=weight_bytes(Q4_0, Nff, K)),
                                             _dev(Wu, "Wu", numel=weight_bytes(Q4_0, Nff, K)),
                                             _dev(Wd, "Wd", numel=weight_bytes(Q4_0, K, Nff)),
                                             _dev(Yq, "Yq", torch.float32, Nq * 4), _dev(Yk, "Yk", torch.float32, Nkv * 4),
                                             _dev(Yv, "Yv", torch.float32, Nkv * 4), _dev(Y, "Y", torch.float32, K * 4),
                                             1, Nq, Nkv, Nff, K, wsp, wsb, _stream(stream)),
           "bqg_decode_layer_q4_0_q8_1")
    return out


def layer_hq(ws, Nff):
    """The q8_1 blocks of h (uint8, Nff/32 * 36) inside a decode-layer workspace."""
    up16 = lambda b: (b + 15) // 16 * 16
    off = up16(Nff * 4) + up16(Nff // QK * 4)
    return ws[off:off + Nff // QK * BLOCK_BYTES[Q8_1]]


def gemm_q4_0_bf16(Wp, X, N, K, out=None, ws=None, stream=None):
    M = X.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=X.device)
    wsp, wsb = _ws(ws)
    _check(load().bqg_gemm_q4_0_bf16(_dev(Wp, "Wp", numel=weight_bytes(Q4_0, N, K)), _dev(X, "X", torch.bfloat16, M * K * 2),
                                     _dev(out, "Y", torch.float32, M * N * 4), M, N, K, wsp, wsb, _stream(stream)),
           "bqg_gemm_q4_0_bf16")
    return out


def gemm_q8_0_bf16(Wp, X, N, K, out=None, ws=None, stream=None):
    M = X.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=X.device)
    wsp, wsb = _ws(ws)
    _check(load().bqg_gemm_q8_0_bf16(_dev(Wp, "Wp", numel=weight_bytes(Q8_0, N, K)), _dev(X, "X", torch.bfloat16, M * K * 2),
                                     _dev(out, "Y", torch.float32, M * N * 4), M, N, K, wsp, wsb, _stream(stream)),
           "bqg_gemm_q8_0_bf16")
    return out


def _block_dots(fn, Wp, Xq, N, K, out, stream):
    if out is None:
        out = torch.empty((N, K // QK), dtype=torch.int32, device=Xq.device)
    _check(getattr(load(), fn)(_dev(Wp, "Wp", numel=weight_bytes(Q4_0, N, K)), _dev(Xq, "Xq", numel=row_bytes(Q8_1, K)),
                               _dev(out, "dots", torch.int32, N * (K // QK) * 4), N, K, _stream(stream)), fn)
    return out


def debug_q4_0_q8_1_block_dots(Wp, Xq, N, K, out=None, stream=None):
    """The integer block dots as gemv_q4_0_q8_1 computes them at M = 1 (its
    own kernel and plan), N x K/32 int32."""
    return _block_dots("bqg_debug_q4_0_q8_1_block_dots", Wp, Xq, N, K, out, stream)


def debug_q4_0_q8_1_block_dots_kslice(Wp, Xq, N, K, out=None, stream=None):
    """The same dots from the K-slice kernel's routine."""
    return _block_dots("bqg_debug_q4_0_q8_1_block_dots_kslice", Wp, Xq, N, K, out, stream)


# --- attention over a paged cache ------------------------------------------------
DEVERR_SLOT, DEVERR_POSITION, DEVERR_PAGE, DEVERR_LENGTH, DEVERR_ROW, DEVERR_DRAFT = 16, 32, 64, 128, 256, 512
_KV_DTYPE = {BF16: torch.bfloat16, Q8_0: torch.int8, Q4_0: torch.uint8}


class _KVCacheStruct(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int), ("page_size", ctypes.c_int), ("n_kv", ctypes.c_int), ("head_dim", ctypes.c_int),
                ("n_pages", ctypes.c_int64), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class KVCache:
    """A paged cache of keys and values over tensors of the caller
    (include/bqgemv.h, bqg_kv_cache): k, v [n_pages, n_kv, page_size, row]
    with rows of head_dim bf16 values (BF16), head_dim int8 codes (Q8_0) or
    head_dim / 2 uint8 code pairs (Q4_0); k_scale, v_scale
    [n_pages, n_kv, page_size, head_dim / 32] fp16 for the quantized formats.
    Keeps the tensors alive; the shapes are checked and the addresses taken
    once, here, so tensors and sizes cannot be set: other ones, another cache."""

    _FIXED = frozenset(("fmt", "n_pages", "n_kv", "page_size", "head_dim", "k", "v", "k_scale", "v_scale", "device_index",
                        "_struct", "_ptr"))

    def __setattr__(self, name, value):
        if name in self._FIXED and name in self.__dict__:
            raise AttributeError(f"a KVCache's {name} is fixed: its calls use what it was made with")
        object.__setattr__(self, name, value)

    def __init__(self, fmt: int, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor | None = None,
                 v_scale: torch.Tensor | None = None):
        if fmt not in _KV_DTYPE:
            raise ValueError("fmt must be BF16, Q8_0 or Q4_0")
        if k.dim() != 4 or v.shape != k.shape:
            raise ValueError("k and v must both be [n_pages, n_kv, page_size, row]")
        n_pages, n_kv, page, row = k.shape
        self.fmt, self.n_pages, self.n_kv, self.page_size = fmt, n_pages, n_kv, page
        self.head_dim = 2 * row if fmt == Q4_0 else row
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        ptrs = [_dev(k, "k", _KV_DTYPE[fmt]), _dev(v, "v", _KV_DTYPE[fmt])]
        if fmt != BF16:
            shape = (n_pages, n_kv, page, self.head_dim // QK)
            for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
                if t is None or tuple(t.shape) != shape:
                    raise ValueError(f"{name} must be {list(shape)}")
                ptrs.append(_dev(t, name, torch.float16))
        elif k_scale is not None or v_scale is not None:
            raise ValueError("a BF16 cache has no scales")
        self._struct = _KVCacheStruct(fmt, page, n_kv, self.head_dim, n_pages, *ptrs)
        self._ptr = ctypes.addressof(self._struct)
        self.device_index = k.device.index

    def _handle(self, cur: int) -> int:
        if self.device_index != cur:
            check_device(self.device_index, cur, "cache")
        return self._ptr


def kv_cache(fmt: int, n_pages: int, n_kv: int, page_size: int, head_dim: int, device="cuda") -> KVCache:
    """A zero-filled cache of n_pages pages."""
    if fmt not in _KV_DTYPE:
        raise ValueError("fmt must be BF16, Q8_0 or Q4_0")
    row = head_dim // 2 if fmt == Q4_0 else head_dim
    t = [torch.zeros((n_pages, n_kv, page_size, row), dtype=_KV_DTYPE[fmt], device=device) for _ in range(2)]
    if fmt != BF16:
        t += [torch.zeros((n_pages, n_kv, page_size, head_dim // QK), dtype=torch.float16, device=device)
              for _ in range(2)]
    return KVCache(fmt, *t)


_X_DTYPE = {torch.bfloat16: BF16, torch.float32: F32}


# These calls take up to nine tensors and their kernels a few microseconds, so the
# checks that hold are made inline; what does not pass goes through the full check,
# which raises with the reason.
def _ptr(t, cur: int, name: str, dtype, nbytes: int):
    """Pointer of a contiguous tensor on the current device `cur` with at least nbytes."""
    if type(t) is torch.Tensor and t.get_device() == cur and t.dtype is dtype and t.is_contiguous() and t.nbytes >= nbytes:
        return t.data_ptr()
    return _dev(t, name, dtype, nbytes)


def _vector(t, cur, name, dtype, n):
    """_ptr of exactly n values."""
    if type(t) is torch.Tensor and t.get_device() == cur and t.dtype is dtype and t.is_contiguous() and t.numel() == n:
        return t.data_ptr()
    p = _dev(t, name, dtype)
    if t.numel() != n:
        raise ValueError(f"{name} holds {t.numel()} values, needs {n}")
    return p


def _tokens(t, cur, name, shape, dtype):
    """(pointer, token stride) of [tokens, heads, head_dim] rows whose tokens
    may lie apart (a part of a fused projection's rows)."""
    if type(t) is torch.Tensor and t.get_device() == cur and t.dtype is dtype and t.shape == shape:
        s = t.stride()
        if s[2] == 1 and s[1] == shape[2]:
            return t.data_ptr(), s[0] if shape[0] > 1 else shape[1] * shape[2]
    return _tokens_checked(t, name, shape, dtype)


def _tokens_checked(t, name, shape, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    check_device(t.device.index, _current_device(), name)
    return t.data_ptr(), _token_stride(t, name, shape, dtype)


def _token_stride(t, name, shape, dtype):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} is {list(t.shape)}, needs {list(shape)}")
    n, h, d = shape
    s = t.stride()
    if t.numel() and ((d > 1 and s[2] != 1) or (h > 1 and s[1] != d)):
        raise ValueError(f"each token's heads of {name} must be contiguous")
    return s[0] if n > 1 else h * d


def _shape3(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 3:
        raise ValueError(f"{name} must be a [tokens, heads, head_dim] tensor")
    return t.shape


def _rotation(pos, table, T, cur):
    if table is None:
        if pos is not None:
            raise ValueError("pos without table")
        return None, None, 0, 0
    if table.dim() != 2:
        raise ValueError("table must be [n_pos, rot_dim]")
    n_pos, rot = table.shape
    return _vector(pos, cur, "pos", torch.int32, T), _ptr(table, cur, "table", torch.float32, 0), n_pos, rot


def _gains(gamma_q, gamma_k, eps, dim, cur):
    if eps is None:
        if gamma_q is not None or gamma_k is not None:
            raise ValueError("gamma without eps (no norm)")
        return 0, None, None, 0.0
    return (1, None if gamma_q is None else _vector(gamma_q, cur, "gamma_q", torch.float32, dim),
            None if gamma_k is None else _vector(gamma_k, cur, "gamma_k", torch.float32, dim), eps)


def _x_dtype(t, name):
    dt = _X_DTYPE.get(t.dtype)
    if dt is None:
        raise TypeError(f"{name} must be bf16 or fp32")
    return dt


def qk_norm_rope(q, k, pos=None, table=None, gamma_q=None, gamma_k=None, eps=None, interleaved=False, out=None,
                 stream=None):
    """Per-head RMSNorm (when eps is given) and rotation (when a table is) of
    queries [T, n_q, head_dim] and keys [T, n_kv, head_dim], bf16 or fp32,
    tokens possibly apart.  table: fp32 [n_pos, rot_dim], cos of the pair
    angles then their sines; pos: int32 [T].  Returns (q, k) in bf16."""
    cur = _current_device()
    shape = T, n_q, dim = _shape3(q, "q")
    n_kv = _shape3(k, "k")[1]
    dt = _x_dtype(q, "q")
    qp, qs = _tokens(q, cur, "q", shape, q.dtype)
    kp, ks = _tokens(k, cur, "k", (T, n_kv, dim), q.dtype)
    norm, gq, gk, eps = _gains(gamma_q, gamma_k, eps, dim, cur)
    pp, tp, n_pos, rot = _rotation(pos, table, T, cur)
    if out is None:
        out = (torch.empty((T, n_q, dim), dtype=torch.bfloat16, device=q.device),
               torch.empty((T, n_kv, dim), dtype=torch.bfloat16, device=q.device))
    _check(load().bqg_qk_norm_rope(qp, kp, dt, qs, ks, T, n_q, n_kv, dim, norm, gq, gk, eps, pp, tp, n_pos, rot,
                                   1 if interleaved else 0, _ptr(out[0], cur, "out[0]", torch.bfloat16, T * n_q * dim * 2),
                                   _ptr(out[1], cur, "out[1]", torch.bfloat16, T * n_kv * dim * 2), _stream(stream)),
           "bqg_qk_norm_rope")
    return out


def qk_norm_rope_kv_write(q, k, v, slots, cache: KVCache, pos=None, table=None, gamma_q=None, gamma_k=None, eps=None,
                          interleaved=False, out=None, stream=None):
    """qk_norm_rope with the keys, and the values v, going into `cache` at
    int64 `slots` (page * page_size + place; negative: not stored) in the same
    launch.  Returns the queries in bf16."""
    cur = _current_device()
    T, n_q, _ = _shape3(q, "q")
    dim, dtype = cache.head_dim, q.dtype
    dt = _x_dtype(q, "q")
    qp, qs = _tokens(q, cur, "q", (T, n_q, dim), dtype)
    kv = (T, cache.n_kv, dim)
    kp, ks = _tokens(k, cur, "k", kv, dtype)
    vp, vs = _tokens(v, cur, "v", kv, dtype)
    norm, gq, gk, eps = _gains(gamma_q, gamma_k, eps, dim, cur)
    pp, tp, n_pos, rot = _rotation(pos, table, T, cur)
    if out is None:
        out = torch.empty((T, n_q, dim), dtype=torch.bfloat16, device=q.device)
        op = out.data_ptr()
    else:
        op = _ptr(out, cur, "out", torch.bfloat16, T * n_q * dim * 2)
    _check(load().bqg_qk_norm_rope_kv_write(qp, kp, vp, dt, qs, ks, vs, T, n_q, norm, gq, gk, eps, pp, tp, n_pos, rot,
                                            1 if interleaved else 0, op,
                                            _vector(slots, cur, "slots", torch.int64, T), cache._handle(cur),
                                            _stream(stream)),
           "bqg_qk_norm_rope_kv_write")
    return out


def kv_write(k, v, slots, cache: KVCache, stream=None) -> None:
    """Keys and values [T, n_kv, head_dim] (bf16 or fp32) into `cache` at `slots`."""
    cur = _current_device()
    T = _shape3(k, "k")[0]
    dt = _x_dtype(k, "k")
    kv = (T, cache.n_kv, cache.head_dim)
    kp, ks = _tokens(k, cur, "k", kv, k.dtype)
    vp, vs = _tokens(v, cur, "v", kv, k.dtype)
    _check(load().bqg_kv_write(kp, vp, dt, ks, vs, T, _vector(slots, cur, "slots", torch.int64, T), cache._handle(cur),
                               _stream(stream)), "bqg_kv_write")


def kv_read(cache: KVCache, slots, dtype=torch.bfloat16, out=None, stream=None):
    """The cache's keys and values at `slots`, each [T, n_kv, head_dim] bf16
    or fp32; a negative slot reads as zeros."""
    cur = _current_device()
    T = slots.numel()
    dt = _X_DTYPE.get(dtype)
    if dt is None:
        raise TypeError("dtype must be bf16 or fp32")
    if out is None:
        shape, device = (T, cache.n_kv, cache.head_dim), slots.device
        out = torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device)
        kp, vp = out[0].data_ptr(), out[1].data_ptr()
    else:
        n = T * cache.n_kv * cache.head_dim * dtype.itemsize
        kp, vp = _ptr(out[0], cur, "out[0]", dtype, n), _ptr(out[1], cur, "out[1]", dtype, n)
    _check(load().bqg_kv_read(cache._handle(cur), _vector(slots, cur, "slots", torch.int64, T), T, dt, kp, vp,
                              _stream(stream)), "bqg_kv_read")
    return out


def tree_attention_workspace(cache: KVCache, n_q: int, n_seq: int, max_q: int) -> torch.Tensor:
    """A zero-filled workspace for tree_attention calls of these sizes."""
    n = int(load().bqg_tree_attention_workspace_size(cache._handle(_current_device()), n_q, n_seq, max_q))
    if n == 0:
        raise ValueError("not a tree_attention call on this device")
    return torch.zeros(n, dtype=torch.uint8, device=cache.k.device)


def tree_attention(q, cache: KVCache, block_table, ctx_len, q_start, max_q: int, mask=None, scale=None, out=None,
                   ws=None, stream=None) -> torch.Tensor:
    """Attention of each sequence's newest tokens (at most max_q <= 64 each)
    over its ctx_len context tokens and themselves, all already in `cache`.

    q: bf16 [n_tokens, n_q, head_dim], sequence after sequence, q_start int32
    [n_seq + 1] their first tokens; block_table int32 [n_seq, max_pages];
    ctx_len int32 [n_seq]; mask int64 [n_tokens], bit j set where new token j
    of the sequence is seen (a tree of drafted tokens), or None for causal;
    scale defaults to head_dim ** -0.5; ws: from tree_attention_workspace, and
    a call without one is refused.  Returns bf16 [n_tokens, n_q, head_dim]."""
    cur = _current_device()
    n, n_q, _ = _shape3(q, "q")
    dim = cache.head_dim
    qp, qs = _tokens(q, cur, "q", (n, n_q, dim), torch.bfloat16)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [n_seq, max_pages]")
    n_seq, max_pages = block_table.shape
    if out is None:
        out = torch.empty((n, n_q, dim), dtype=torch.bfloat16, device=q.device)
        op = out.data_ptr()
    else:
        op = _ptr(out, cur, "out", torch.bfloat16, n * n_q * dim * 2)
    if ws is None:
        wsp, wsb = None, 0
    else:
        wsb = ws.nbytes
        wsp = _ptr(ws, cur, "ws", ws.dtype, wsb)
    _check(load().bqg_tree_attention(qp, qs, cache._handle(cur), _ptr(block_table, cur, "block_table", torch.int32, 0),
                                     max_pages, _vector(ctx_len, cur, "ctx_len", torch.int32, n_seq),
                                     _vector(q_start, cur, "q_start", torch.int32, n_seq + 1), n_seq, n, max_q, n_q,
                                     None if mask is None else _vector(mask, cur, "mask", torch.int64, n),
                                     dim ** -0.5 if scale is None else scale,
                                     op, wsp, wsb, _stream(stream)),
           "bqg_tree_attention")
    return out


def shared_prefix_attention_workspace(cache: KVCache, n_q: int, n_seq: int, max_q: int, n_tokens: int, n_prefix: int = 1,
                                      max_shared: int | None = None) -> torch.Tensor:
    """A zero-filled workspace for shared_prefix_attention calls of at most these sizes."""
    n = int(load().bqg_shared_prefix_attention_workspace_size(cache._handle(_current_device()), n_q, n_seq, max_q, n_tokens,
                                                              n_prefix, n_tokens if max_shared is None else max_shared))
    if n == 0:
        raise ValueError("not a shared_prefix_attention call on this device")
    return torch.zeros(n, dtype=torch.uint8, device=cache.k.device)


def shared_prefix_attention(q, cache: KVCache, block_table, ctx_len, q_start, max_q: int, prefix_len, seq_start=None,
                            max_shared: int | None = None, mask=None, scale=None, out=None, ws=None,
                            stream=None) -> torch.Tensor:
    """tree_attention where sequences share their first tokens, which are read and multiplied once for all of them.

    Arguments and result as tree_attention's (ctx_len and block_table with the shared tokens), and: prefix_len int32
    [n_prefix], the tokens that sequences seq_start[g] .. seq_start[g + 1] - 1 share (at most the ctx_len of
    each; taken from the first one's pages); seq_start int32 [n_prefix + 1], or None for one prefix of all
    sequences; max_shared: query tokens behind one prefix at most (default: all of the call's, which with several
    prefixes may pick a slower kernel); ws: from
    shared_prefix_attention_workspace, and a call without one is refused."""
    cur = _current_device()
    n, n_q, _ = _shape3(q, "q")
    dim = cache.head_dim
    qp, qs = _tokens(q, cur, "q", (n, n_q, dim), torch.bfloat16)
    if block_table.dim() != 2:
        raise ValueError("block_table must be [n_seq, max_pages]")
    n_seq, max_pages = block_table.shape
    n_prefix = prefix_len.numel()
    if seq_start is None and n_prefix != 1:
        raise ValueError("several prefixes need seq_start")
    if out is None:
        out = torch.empty((n, n_q, dim), dtype=torch.bfloat16, device=q.device)
        op = out.data_ptr()
    else:
        op = _ptr(out, cur, "out", torch.bfloat16, n * n_q * dim * 2)
    if ws is None:
        wsp, wsb = None, 0
    else:
        wsb = ws.nbytes
        wsp = _ptr(ws, cur, "ws", ws.dtype, wsb)
    _check(load().bqg_shared_prefix_attention(
        qp, qs, cache._handle(cur), _ptr(block_table, cur, "block_table", torch.int32, 0), max_pages,
        _vector(ctx_len, cur, "ctx_len", torch.int32, n_seq), _vector(q_start, cur, "q_start", torch.int32, n_seq + 1), n_seq,
        n, max_q, n_q, _vector(prefix_len, cur, "prefix_len", torch.int32, n_prefix),
        None if seq_start is None else _vector(seq_start, cur, "seq_start", torch.int32, n_prefix + 1), n_prefix,
        n if max_shared is None else max_shared, None if mask is None else _vector(mask, cur, "mask", torch.int64, n),
        dim ** -0.5 if scale is None else scale, op, wsp, wsb, _stream(stream)),
        "bqg_shared_prefix_attention")
    return out


# --- verification of drafts, and what follows from it for the cache -------------
def _rows(t, cur, name, shape, dtype):
    """(pointer, row stride) of [rows, n] values, each row contiguous."""
    if type(t) is torch.Tensor and t.get_device() == cur and t.dtype is dtype and t.shape == shape:
        s = t.stride()
        if s[1] == 1:
            return t.data_ptr(), s[0] if shape[0] > 1 else shape[1]
    return _rows_checked(t, name, shape, dtype)


def _rows_checked(t, name, shape, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    check_device(t.device.index, _current_device(), name)
    return t.data_ptr(), _row_stride(t, name, shape, dtype)


def _row_stride(t, name, shape, dtype):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} is {list(t.shape)}, needs {list(shape)}")
    if t.numel() and shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"each row of {name} must be contiguous")
    return t.stride(0) if shape[0] > 1 else shape[1]


def tree_verify(target, tokens, q_start, max_q: int, u, parent=None, draft=None, out=None, stream=None):
    """Drafted tokens accepted or rejected against the target's probabilities, and the token that follows.

    target [n_tokens, vocab], bf16 or fp32 (rows may lie apart): the distribution behind each token; tokens int32
    [n_tokens], sequence after sequence (at most max_q <= 64 each), q_start int32 [n_seq + 1] their first ones, each
    one's token 0 the last given out; parent int32 [n_tokens], the token of its sequence that a draft stands
    behind, or None for chains; draft: as target, the distributions that the drafts were drawn from, or None for
    drafts that were chosen; u fp32 [n_tokens], numbers in [0, 1).  Returns int32 (n_accepted [n_seq], path
    [n_seq, max_q], next_token [n_seq]): how many tokens are kept, with token 0; their places, then -1; the next token."""
    cur = _current_device()
    if not isinstance(target, torch.Tensor) or target.dim() != 2:
        raise ValueError("target must be a [n_tokens, vocab] tensor")
    n, vocab = target.shape
    dt = _x_dtype(target, "target")
    tp, ts = _rows(target, cur, "target", (n, vocab), target.dtype)
    dp, ds = (None, 0) if draft is None else _rows(draft, cur, "draft", (n, vocab), target.dtype)
    n_seq = q_start.numel() - 1
    if n_seq < 0:
        raise ValueError("q_start must hold n_seq + 1 values")
    if out is None:
        i32 = dict(dtype=torch.int32, device=target.device)
        out = torch.empty(n_seq, **i32), torch.empty((n_seq, max(max_q, 0)), **i32), torch.empty(n_seq, **i32)
    _check(load().bqg_tree_verify(tp, dp, dt, ts, ds, vocab, _vector(tokens, cur, "tokens", torch.int32, n),
                                  None if parent is None else _vector(parent, cur, "parent", torch.int32, n),
                                  _vector(q_start, cur, "q_start", torch.int32, n_seq + 1), n_seq, n, max_q,
                                  _vector(u, cur, "u", torch.float32, n), _vector(out[0], cur, "out[0]", torch.int32, n_seq),
                                  _vector(out[1], cur, "out[1]", torch.int32, n_seq * max(max_q, 0)),
                                  _vector(out[2], cur, "out[2]", torch.int32, n_seq), _stream(stream)), "bqg_tree_verify")
    return out


def _table(t, cur):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("block_table must be [rows, max_pages]")
    return _ptr(t, cur, "block_table", torch.int32, 0), t.shape


def kv_compact(cache: KVCache, block_table, ctx_len, path, n_path, out=None, stream=None) -> torch.Tensor:
    """The accepted path's keys and values moved behind the context: new token path[b, k] of sequence b goes to place
    ctx_len[b] + k, for k < n_path[b] (path int32 [n_seq, max_q], ascending; as tree_verify gives them).  Returns the new
    lengths ctx_len + n_path, int32 [n_seq] (`out` may overlap none of ctx_len, path and n_path)."""
    cur = _current_device()
    bp, (n_seq, max_pages) = _table(block_table, cur)
    if not isinstance(path, torch.Tensor) or path.dim() != 2 or path.shape[0] != n_seq:
        raise ValueError("path must be [n_seq, max_q]")
    if out is None:
        out = torch.empty(n_seq, dtype=torch.int32, device=block_table.device)
    _check(load().bqg_kv_compact(cache._handle(cur), bp, max_pages, _vector(ctx_len, cur, "ctx_len", torch.int32, n_seq),
                                 _ptr(path, cur, "path", torch.int32, 0), _vector(n_path, cur, "n_path", torch.int32, n_seq),
                                 n_seq, path.shape[1], _vector(out, cur, "out", torch.int32, n_seq), _stream(stream)),
           "bqg_kv_compact")
    return out


def kv_fork(cache: KVCache, block_table, ctx_len, parent, child, fresh, stream=None) -> None:
    """Sequences branched: row child[i] of block_table int32 [rows, max_pages] gets row parent[i]'s full pages and, as the
    next one, page fresh[i] with a copy of the tokens in the parent's page in use; ctx_len int32 [rows] gets its length.
    parent, child, fresh: int32 [n]; children distinct and no parents, fresh pages distinct and in no row.  In place."""
    cur = _current_device()
    bp, (rows, max_pages) = _table(block_table, cur)
    n = parent.numel()
    _check(load().bqg_kv_fork(cache._handle(cur), bp, max_pages, rows, _vector(ctx_len, cur, "ctx_len", torch.int32, rows),
                              _vector(parent, cur, "parent", torch.int32, n), _vector(child, cur, "child", torch.int32, n),
                              _vector(fresh, cur, "fresh", torch.int32, n), n, _stream(stream)), "bqg_kv_fork")


# --- utilities -----------------------------------------------------------------
def workspace_size(op: int, M: int, N: int, K: int) -> int:
    return int(load().bqg_workspace_size(op, M, N, K))


def workspace(op: int, M: int, N: int, K: int, device="cuda") -> torch.Tensor | None:
    """A workspace for `op` (zero-filled, as the q8_1-output SwiGLU requires)."""
    n = workspace_size(op, M, N, K)
    return torch.zeros(n, dtype=torch.uint8, device=device) if n else None


ROUTE_K_SLICE, ROUTE_LANES_PER_ROW, ROUTE_LANES_PER_ROW_ROWS, ROUTE_TENSOR_CORE = 0, 1, 2, 3
ROUTE_NAMES = {0: "k_slice", 1: "lanes_per_row", 2: "lanes_per_row_rows", 3: "tensor_core"}


def gemv_route(op: int, M: int, N: int, K: int) -> int:
    """Which kernel serves a GEMV call of this shape on the current device
    (one of the ROUTE_* values)."""
    out = ctypes.c_int(-1)
    _check(load().bqg_gemv_route(op, M, N, K, ctypes.addressof(out)), "bqg_gemv_route")
    return out.value


def last_device_error(stream=None) -> int:
    out = ctypes.c_int(0)
    _check(load().bqg_last_device_error(_stream(stream), ctypes.addressof(out)), "bqg_last_device_error")
    return out.value


def set_pdl(enable: bool) -> bool:
    return bool(load().bqg_set_pdl(1 if enable else 0))
