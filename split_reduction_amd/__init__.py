"""Python binding of libskgemm.so, the split-K decode GEMM for MI355X (gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI declared in ``include/skgemm.h``. Functions carry the
C names and argument order; array arguments may be torch tensors on the GPU
(their storage address is passed) or plain integer device addresses. The
stream defaults to torch's current stream on the current device.

The library is loaded on first use. If it is missing or fails to load, every
call raises ``SkgemmError``: there is no fallback path.
"""

from __future__ import annotations

import ctypes
import json
import os

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libskgemm.so")

SKGEMM_OK = 0
SKGEMM_EINVAL = -1
SKGEMM_EALIGN = -2
SKGEMM_ESHAPE = -3
SKGEMM_ENOMEM = -4
SKGEMM_EHIP = -5
SKGEMM_ESCRATCH = -6

# skgemm_set_override knobs (include/skgemm.h, enum skgemm_knob)
KNOBS = {"kind": 0, "stream": 1, "shape": 2, "fold": 3, "cluster_c": 4, "wg_per_cu": 5,
         "pdefer": 6, "owner_wait": 7, "handoff": 8, "i8_shape": 9, "i8_split": 10}

# Element formats (include/skgemm.h, enum skgemm_format)
FORMATS = {"bf16": 0, "i8": 1, "e4m3": 2, "f32": 3}

_lib = None
_raw_stream = _device = None  # torch's functions, bound by the first call that asks for the stream
_torch_types = {}  # torch's element types that an operator's argument may have, filled by the first call


class SkgemmError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(what)


def _declare(lib):
    vp, i, sz, st = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    sig = {
        "skgemm_bf16": [vp, vp, vp, i, i, i, i, st],
        "skgemm_mxfp4": [vp, vp, vp, vp, i, i, i, i, st],
        "skgemm_mxfp8": [vp, vp, vp, vp, i, i, i, i, st],
        "skgemm_mxfp8_batched": [vp, vp, vp, vp, i, i, i, i, i, sz, sz, sz, sz, st],
        "skgemm_mxfp8_dequant": [vp, vp, vp, i, i, st],
        "skgemm_reserve": [i, i, i, st],
        "skgemm_reserve_batched": [i, i, i, i, st],
        "skgemm_bf16_batched": [vp, vp, vp, i, i, i, i, i, sz, sz, sz, st],
        "skgemm_mxfp4_batched": [vp, vp, vp, vp, i, i, i, i, i, sz, sz, sz, sz, st],
        "skgemm_release": [],
        "skgemm_mxfp4_dequant": [vp, vp, vp, i, i, st],
        "skgemm_pack_bf16": [vp, vp, sz, st],
        "skgemm_pack_e4m3": [vp, vp, sz, st],
        "skgemm_wave_sum": [vp, vp, sz, st],
        "skgemm_tactic_for": [i, i, i, i, i, ctypes.c_char_p, sz],
        "skgemm_last_hip_error": [],
        "skgemm_set_timeline": [vp, sz],
        "skgemm_read_probe": [vp, sz, vp, st],
        "skgemm_health": [vp, sz, st],
        "skgemm_set_override": [i, i],
        "skgemm_bf16_noalloc": [vp, vp, vp, i, i, i, i, st],
        "skgemm_bf16_e4m3": [vp, vp, vp, ctypes.c_float, i, i, i, i, st],
        "skgemm_bf16_chain": [vp, vp, vp, vp, i, i, i, st],
        "skgemm_i8": [vp, vp, vp, vp, vp, i, i, i, i, sz, sz, sz, st],
        "skgemm_logprobs": [vp, vp, vp, vp, vp, vp, vp, i, i, i, ctypes.c_float, i, sz, st],
        "skgemm_logprobs_grad": [vp, vp, vp, vp, vp, vp, vp, i, i, ctypes.c_float, i, sz, sz, st],
        "skgemm_reserve_ops": [st],
        "skgemm_rmsnorm": [vp, vp, vp, vp, vp, vp, i, i, ctypes.c_float, i, sz, sz, sz, sz, st],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.skgemm_strerror.argtypes = [ctypes.c_int]
    lib.skgemm_strerror.restype = ctypes.c_char_p


def lib():
    """The loaded libskgemm.so (raises SkgemmError if it is not built).

    torch is imported first: its wheel carries its own HIP runtime under the
    same soname (libamdhip64.so.7) but loads it by file name, so if this
    library pulled in the system runtime first, the process would hold two
    HIP runtimes and launches from here would fail (hipErrorNoDevice). With
    torch's runtime already loaded, this library binds to that one instance.
    """
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise SkgemmError(SKGEMM_EHIP, f"{LIB_PATH} is not built (run split_reduction_amd/build.py)")
        import torch  # noqa: F401  (one HIP runtime per process: torch's)

        try:
            handle = ctypes.CDLL(LIB_PATH)
        except OSError as e:
            raise SkgemmError(SKGEMM_EHIP, f"cannot load {LIB_PATH}: {e}") from e
        _declare(handle)
        _lib = handle
    return _lib


def strerror(code: int) -> str:
    return lib().skgemm_strerror(code).decode()


def _check(code: int, name: str) -> None:
    if code != SKGEMM_OK:
        extra = ""
        if code == SKGEMM_EHIP:
            extra = f" (hipError {lib().skgemm_last_hip_error()})"
        raise SkgemmError(code, f"{name}: {strerror(code)}{extra}")


def _types() -> dict:
    """The element types of the operators' tensors, with their size. A type of the
    same width would be read as the call's own: float16 logits as bf16, say."""
    if not _torch_types:
        import torch as t

        _torch_types.update(bf16=(2, (t.bfloat16,)), f32=(4, (t.float32,)), i64=(8, (t.int64,)), i8=(1, (t.int8,)),
                            i8_out=(1, (t.int8, t.uint8)), e4m3_out=(1, (t.uint8, t.float8_e4m3fn)))
    return _torch_types


def _wrong_type(a, types, what: str) -> SkgemmError:
    return SkgemmError(SKGEMM_EINVAL, f"{what}: elements of {a.dtype}, the call takes {' or '.join(map(str, types[1]))}")


def _ptr(a, nbytes: int = 0, what: str = "argument", types=None) -> int:
    """Device address of a tensor or of a plain integer address (None is 0).

    A tensor must live on the GPU, be contiguous and hold at least `nbytes`
    from its first element: the kernels read or write that dense block at the
    address, so a host tensor, a strided view or a short buffer would reach the
    device as a bad address. Such tensors raise SkgemmError(SKGEMM_EINVAL) here,
    before anything is launched, and so do elements of another type than `types`
    (one of _types; None: any). Integer addresses are passed through unchecked
    (the caller vouches for them)."""
    if a is None:
        return 0
    if isinstance(a, int):
        return a
    try:
        on_gpu = a.is_cuda  # a tenth of the time that a.device.type takes
    except AttributeError:
        on_gpu = a.device.type == "cuda"
    if not on_gpu:
        raise SkgemmError(SKGEMM_EINVAL, f"{what}: a tensor on {a.device}, not on the GPU")
    if types is None:
        size = a.element_size()
    elif a.dtype in types[1]:
        size = types[0]
    else:
        raise _wrong_type(a, types, what)
    if not a.is_contiguous():
        raise SkgemmError(SKGEMM_EINVAL, f"{what}: not contiguous")
    have = a.numel() * size
    if have < nbytes:
        raise SkgemmError(SKGEMM_EINVAL, f"{what}: holds {have} bytes, the call needs {nbytes}")
    return a.data_ptr()


def _rows(a, rows: int, row_bytes: int, stride, what: str, types):
    """(address, row stride in bytes) of a matrix whose rows are `row_bytes` long
    and contiguous, `stride` bytes apart (None: as the tensor's own rows are, or
    dense for an address). The tensor must be on the GPU, hold elements of
    `types` (one of _types) and reach to the end of the last row."""
    if stride is not None and stride < 0:
        raise SkgemmError(SKGEMM_EINVAL, f"{what}: a negative row stride")
    if a is None or isinstance(a, int):
        return a or 0, row_bytes if stride is None else stride
    if not a.is_cuda:
        raise SkgemmError(SKGEMM_EINVAL, f"{what}: a tensor on {a.device}, not on the GPU")
    if a.dtype not in types[1]:
        raise _wrong_type(a, types, what)
    size = types[0]
    n = a.numel() * size
    if stride is None and n == rows * row_bytes and a.is_contiguous():
        return a.data_ptr(), row_bytes  # dense
    if a.is_contiguous():
        if stride is None:
            stride = a.stride(0) * size if a.dim() == 2 and rows > 1 and a.stride(0) * size >= row_bytes else row_bytes
    elif a.dim() == 2 and (a.stride(1) == 1 or a.shape[1] == 1) and a.stride(0) >= 0:
        own = a.stride(0) * size
        if stride is None:
            stride = own
        elif stride != own and rows > 1:
            raise SkgemmError(SKGEMM_EINVAL, f"{what}: rows {own} bytes apart, not {stride}")
        if n:
            n = (a.shape[0] - 1) * own + a.shape[1] * size
        if a.shape[1] * size < row_bytes and rows > 0:
            raise SkgemmError(SKGEMM_EINVAL, f"{what}: rows of {a.shape[1] * size} bytes, the call needs {row_bytes}")
    else:
        raise SkgemmError(SKGEMM_EINVAL, f"{what}: rows are not contiguous")
    need = (rows - 1) * max(stride, 0) + row_bytes if rows > 0 and row_bytes > 0 else 0
    if n < need:
        raise SkgemmError(SKGEMM_EINVAL, f"{what}: holds {n} bytes, the call needs {need}")
    return a.data_ptr(), stride


def _format(name) -> int:
    if isinstance(name, str):
        if name not in FORMATS:
            raise SkgemmError(SKGEMM_EINVAL, f"unknown format {name!r}, one of {sorted(FORMATS)}")
        return FORMATS[name]
    return int(name)


def _n(*dims) -> int:
    """Product of the sizes, 0 if any is not positive (the library rejects or
    skips such calls itself, so they need no bytes)."""
    out = 1
    for d in dims:
        if d <= 0:
            return 0
        out *= d
    return out


def _batched(L: int, stride: int, one: int) -> int:
    """Bytes spanned by L problems `stride` bytes apart, each `one` bytes."""
    return 0 if L <= 0 or one == 0 else (L - 1) * max(stride, 0) + one


def _current_stream() -> int:
    """torch's current stream on the current device, without the Stream object
    that torch.cuda.current_stream() builds (2.7 us of a call's 11)."""
    global _raw_stream, _device
    if _device is None:
        import torch

        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if _raw_stream is None:
            return torch.cuda.current_stream().cuda_stream
        _device = torch.cuda.current_device
    return _raw_stream(_device())


def _stream(stream) -> int:
    if stream is None:
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def skgemm_bf16(W, X, C, T: int, N: int, K: int, split_k: int, stream=None) -> None:
    """C[T, N] = X[T, K] . W[N, K]^T (bf16 in and out, FP32 accumulation)."""
    code = lib().skgemm_bf16(_ptr(W, 2 * _n(N, K), "W"), _ptr(X, 2 * _n(T, K), "X"),
                             _ptr(C, 2 * _n(T, N), "C"), T, N, K, split_k, _stream(stream))
    _check(code, "skgemm_bf16")


def skgemm_bf16_e4m3(W, X, C8, c_scale: float, T: int, N: int, K: int, split_k: int, stream=None) -> None:
    """C8[T, N] (uint8 E4M3FN codes) of (X . W^T) * c_scale, saturated to +-448."""
    code = lib().skgemm_bf16_e4m3(_ptr(W, 2 * _n(N, K), "W"), _ptr(X, 2 * _n(T, K), "X"),
                                  _ptr(C8, _n(T, N), "C8"), float(c_scale), T, N, K, split_k, _stream(stream))
    _check(code, "skgemm_bf16_e4m3")


def skgemm_bf16_chain(Ws, X, Cs, dims, T: int, split_k: int, stream=None) -> None:
    """L GEMMs in one launch, C[i] = A_i . W[i]^T with A_0 = X, A_i = C[i-1];
    Ws and Cs are sequences of L tensors (or addresses), dims L + 1 sizes."""
    L = len(Ws)
    if len(Cs) != L or len(dims) != L + 1:
        raise SkgemmError(SKGEMM_EINVAL, "skgemm_bf16_chain: need L weights, L outputs and L + 1 dims")
    wp = (ctypes.c_void_p * max(L, 1))(*[_ptr(Ws[i], 2 * _n(dims[i + 1], dims[i]), f"W[{i}]") for i in range(L)])
    cp = (ctypes.c_void_p * max(L, 1))(*[_ptr(Cs[i], 2 * _n(T, dims[i + 1]), f"C[{i}]") for i in range(L)])
    dp = (ctypes.c_int * (L + 1))(*[int(d) for d in dims])
    code = lib().skgemm_bf16_chain(wp, _ptr(X, 2 * _n(T, dims[0]) if dims else 0, "X"), cp, dp, L, T, split_k,
                                   _stream(stream))
    _check(code, "skgemm_bf16_chain")


def skgemm_bf16_noalloc(W, X, C, T: int, N: int, K: int, split_k: int, stream=None) -> None:
    """skgemm_bf16 with the split-K workspace in the library's fixed per-GPU
    scratch: allocates nothing (SKGEMM_ESCRATCH when the call needs more)."""
    code = lib().skgemm_bf16_noalloc(_ptr(W, 2 * _n(N, K), "W"), _ptr(X, 2 * _n(T, K), "X"),
                                     _ptr(C, 2 * _n(T, N), "C"), T, N, K, split_k, _stream(stream))
    _check(code, "skgemm_bf16_noalloc")


def skgemm_mxfp4(Wq, Wscale, X, C, T: int, N: int, K: int, split_k: int, stream=None) -> None:
    """C = X . dequant(Wq, Wscale)^T with MXFP4 weights decoded in registers."""
    code = lib().skgemm_mxfp4(_ptr(Wq, _n(N, K) // 2, "Wq"), _ptr(Wscale, _n(N, K) // 32, "Wscale"),
                              _ptr(X, 2 * _n(T, K), "X"), _ptr(C, 2 * _n(T, N), "C"), T, N, K, split_k,
                              _stream(stream))
    _check(code, "skgemm_mxfp4")


def skgemm_bf16_batched(W, X, C, T: int, N: int, K: int, split_k: int, L: int, w_stride: int,
                        x_stride: int, c_stride: int, stream=None) -> None:
    """L problems of one shape in one launch; strides in bytes."""
    code = lib().skgemm_bf16_batched(_ptr(W, _batched(L, w_stride, 2 * _n(N, K)), "W"),
                                     _ptr(X, _batched(L, x_stride, 2 * _n(T, K)), "X"),
                                     _ptr(C, _batched(L, c_stride, 2 * _n(T, N)), "C"),
                                     T, N, K, split_k, L, w_stride, x_stride, c_stride, _stream(stream))
    _check(code, "skgemm_bf16_batched")


def skgemm_mxfp4_batched(Wq, Wscale, X, C, T: int, N: int, K: int, split_k: int, L: int, wq_stride: int,
                         wscale_stride: int, x_stride: int, c_stride: int, stream=None) -> None:
    """L MXFP4 problems of one shape in one launch; strides in bytes."""
    code = lib().skgemm_mxfp4_batched(_ptr(Wq, _batched(L, wq_stride, _n(N, K) // 2), "Wq"),
                                      _ptr(Wscale, _batched(L, wscale_stride, _n(N, K) // 32), "Wscale"),
                                      _ptr(X, _batched(L, x_stride, 2 * _n(T, K)), "X"),
                                      _ptr(C, _batched(L, c_stride, 2 * _n(T, N)), "C"),
                                      T, N, K, split_k, L, wq_stride, wscale_stride, x_stride, c_stride,
                                      _stream(stream))
    _check(code, "skgemm_mxfp4_batched")


def skgemm_mxfp8(Wq8, Wscale, X, C, T: int, N: int, K: int, split_k: int, stream=None) -> None:
    """C = X . dequant(Wq8, Wscale)^T with E4M3 weights and E8M0 block scales."""
    code = lib().skgemm_mxfp8(_ptr(Wq8, _n(N, K), "Wq8"), _ptr(Wscale, _n(N, K) // 32, "Wscale"),
                              _ptr(X, 2 * _n(T, K), "X"), _ptr(C, 2 * _n(T, N), "C"), T, N, K, split_k,
                              _stream(stream))
    _check(code, "skgemm_mxfp8")


def skgemm_mxfp8_batched(Wq8, Wscale, X, C, T: int, N: int, K: int, split_k: int, L: int, wq8_stride: int,
                         wscale_stride: int, x_stride: int, c_stride: int, stream=None) -> None:
    """L MXFP8 problems of one shape in one launch; strides in bytes."""
    code = lib().skgemm_mxfp8_batched(_ptr(Wq8, _batched(L, wq8_stride, _n(N, K)), "Wq8"),
                                      _ptr(Wscale, _batched(L, wscale_stride, _n(N, K) // 32), "Wscale"),
                                      _ptr(X, _batched(L, x_stride, 2 * _n(T, K)), "X"),
                                      _ptr(C, _batched(L, c_stride, 2 * _n(T, N)), "C"),
                                      T, N, K, split_k, L, wq8_stride, wscale_stride, x_stride, c_stride,
                                      _stream(stream))
    _check(code, "skgemm_mxfp8_batched")


def skgemm_rmsnorm(X, R, G, R_out, Y, y_scale, T: int, H: int, eps: float, out_format="bf16", x_stride=None,
                   r_stride=None, r_out_stride=None, y_stride=None, stream=None) -> None:
    """Y = (X + R) / rms(X + R) * G as bf16, or as "i8" / "e4m3" codes with a
    scale for each row; R_out = bf16(X + R). R, G and R_out may be None. X, R, G
    and R_out are bfloat16, y_scale float32, Y bfloat16, for "i8" int8 or uint8,
    for "e4m3" float8_e4m3fn or uint8."""
    f = _format(out_format)
    ty = _torch_types or _types()
    bf16 = ty["bf16"]
    ysize = 2 if f == 0 else 1
    x, xs = _rows(X, T, 2 * H, x_stride, "X", bf16)
    r, rs = _rows(R, T, 2 * H, r_stride, "R", bf16)
    ro, ros = _rows(R_out, T, 2 * H, r_out_stride, "R_out", bf16)
    y, ys = _rows(Y, T, ysize * H, y_stride, "Y", bf16 if f == 0 else ty["i8_out"] if f == 1 else ty["e4m3_out"])
    code = lib().skgemm_rmsnorm(x, r, _ptr(G, 2 * _n(H), "G", bf16), ro, y, _ptr(y_scale, 4 * _n(T), "y_scale", ty["f32"]),
                                T, H, eps, f, xs, rs, ros, ys, _stream(stream))
    _check(code, "skgemm_rmsnorm")


def skgemm_i8(Wq, w_scale, Xq, x_scale, C, T: int, N: int, K: int, out_format=None, w_stride=None, x_stride=None,
              c_stride=None, stream=None) -> None:
    """C[t, n] = x_scale[t] * w_scale[n] * (Xq . Wq^T)[t, n] with exact integer
    sums of int8 codes and float32 scales; C is bfloat16 or float32 (out_format
    "bf16" / "f32"; None: as C's elements are, bf16 for an address)."""
    if out_format is None:
        out_format = 3 if not isinstance(C, int) and C is not None and C.element_size() == 4 else 0
    f = _format(out_format)
    ty = _torch_types or _types()
    size = 4 if f == 3 else 2
    w, ws = _rows(Wq, N, K, w_stride, "Wq", ty["i8"])
    x, xs = _rows(Xq, T, K, x_stride, "Xq", ty["i8"])
    c, cs = _rows(C, T, size * N, c_stride, "C", ty["f32"] if f == 3 else ty["bf16"])
    code = lib().skgemm_i8(w, _ptr(w_scale, 4 * _n(N), "w_scale", ty["f32"]), x, _ptr(x_scale, 4 * _n(T), "x_scale", ty["f32"]),
                           c, T, N, K, f, ws, xs, cs, _stream(stream))
    _check(code, "skgemm_i8")


def _logits_format(logits, logits_format) -> int:
    if logits_format is None:
        return 3 if logits is not None and not isinstance(logits, int) and logits.element_size() == 4 else 0
    return _format(logits_format)


def skgemm_logprobs(logits, tokens, logprob, entropy, lse, top_logprob, top_ids, T: int, V: int, top_k: int = 0,
                    scale: float = 1.0, logits_format=None, stride=None, stream=None) -> None:
    """Of each row of scale * logits: the log probability of its token, the
    entropy, the log of the sum of exponentials, and the top_k best tokens with
    their log probabilities. Outputs may be None and are float32; tokens and ids
    are int64. logits are bfloat16 or float32 (logits_format "bf16" / "f32";
    None: as the elements are, bf16 for an address)."""
    f = _logits_format(logits, logits_format)
    ty = _torch_types or _types()
    f32, i64 = ty["f32"], ty["i64"]
    size = 4 if f == 3 else 2
    z, zs = _rows(logits, T, size * V, stride, "logits", f32 if f == 3 else ty["bf16"])
    code = lib().skgemm_logprobs(z, _ptr(tokens, 8 * _n(T), "tokens", i64), _ptr(logprob, 4 * _n(T), "logprob", f32),
                                 _ptr(entropy, 4 * _n(T), "entropy", f32), _ptr(lse, 4 * _n(T), "lse", f32),
                                 _ptr(top_logprob, 4 * _n(T, top_k), "top_logprob", f32),
                                 _ptr(top_ids, 8 * _n(T, top_k), "top_ids", i64), T, V, top_k, scale, f, zs,
                                 _stream(stream))
    _check(code, "skgemm_logprobs")


def skgemm_logprobs_grad(logits, tokens, lse, entropy, g_logprob, g_entropy, d_logits, T: int, V: int,
                         scale: float = 1.0, logits_format=None, stride=None, d_stride=None, stream=None) -> None:
    """The gradient of sum(g_logprob * logprob) + sum(g_entropy * entropy) to the
    logits, from the lse and entropy that skgemm_logprobs gave; d_logits has the
    logits' type and may be the logits themselves. g_logprob or g_entropy may be
    None (zeros); they, lse and entropy are float32, tokens int64."""
    f = _logits_format(logits, logits_format)
    ty = _torch_types or _types()
    f32 = ty["f32"]
    size = 4 if f == 3 else 2
    z, zs = _rows(logits, T, size * V, stride, "logits", f32 if f == 3 else ty["bf16"])
    d, ds = _rows(d_logits, T, size * V, d_stride, "d_logits", f32 if f == 3 else ty["bf16"])
    code = lib().skgemm_logprobs_grad(z, _ptr(tokens, 8 * _n(T), "tokens", ty["i64"]), _ptr(lse, 4 * _n(T), "lse", f32),
                                      _ptr(entropy, 4 * _n(T), "entropy", f32), _ptr(g_logprob, 4 * _n(T), "g_logprob", f32),
                                      _ptr(g_entropy, 4 * _n(T), "g_entropy", f32), d, T, V, scale, f, zs, ds,
                                      _stream(stream))
    _check(code, "skgemm_logprobs_grad")


def skgemm_mxfp8_dequant(Wq8, Wscale, W_out, N: int, K: int, stream=None) -> None:
    code = lib().skgemm_mxfp8_dequant(_ptr(Wq8, _n(N, K), "Wq8"), _ptr(Wscale, _n(N, K) // 32, "Wscale"),
                                      _ptr(W_out, 2 * _n(N, K), "W_out"), N, K, _stream(stream))
    _check(code, "skgemm_mxfp8_dequant")


def skgemm_reserve_batched(max_T: int, max_N: int, max_split_k: int, max_L: int, stream=None) -> None:
    _check(lib().skgemm_reserve_batched(max_T, max_N, max_split_k, max_L, _stream(stream)),
           "skgemm_reserve_batched")


def skgemm_reserve(max_T: int, max_N: int, max_split_k: int, stream=None) -> None:
    _check(lib().skgemm_reserve(max_T, max_N, max_split_k, _stream(stream)), "skgemm_reserve")


def skgemm_reserve_ops(stream=None) -> None:
    """Allocate the stream's workspace of skgemm_i8 and skgemm_logprobs now, as
    they cannot while the stream is captured."""
    _check(lib().skgemm_reserve_ops(_stream(stream)), "skgemm_reserve_ops")


def skgemm_release() -> None:
    _check(lib().skgemm_release(), "skgemm_release")


def skgemm_mxfp4_dequant(Wq, Wscale, W_out, N: int, K: int, stream=None) -> None:
    code = lib().skgemm_mxfp4_dequant(_ptr(Wq, _n(N, K) // 2, "Wq"), _ptr(Wscale, _n(N, K) // 32, "Wscale"),
                                      _ptr(W_out, 2 * _n(N, K), "W_out"), N, K, _stream(stream))
    _check(code, "skgemm_mxfp4_dequant")


def skgemm_pack_bf16(inp, out, n_pairs: int, stream=None) -> None:
    _check(lib().skgemm_pack_bf16(_ptr(inp, 8 * n_pairs, "in"), _ptr(out, 4 * n_pairs, "out"), n_pairs,
                                  _stream(stream)), "skgemm_pack_bf16")


def skgemm_pack_e4m3(inp, out, n_quads: int, stream=None) -> None:
    _check(lib().skgemm_pack_e4m3(_ptr(inp, 16 * n_quads, "in"), _ptr(out, 4 * n_quads, "out"), n_quads,
                                  _stream(stream)), "skgemm_pack_e4m3")


def skgemm_wave_sum(inp, out, n_waves: int, stream=None) -> None:
    _check(lib().skgemm_wave_sum(_ptr(inp, 256 * n_waves, "in"), _ptr(out, 256 * n_waves, "out"), n_waves,
                                 _stream(stream)), "skgemm_wave_sum")


def skgemm_tactic_for(T: int, N: int, K: int, split_k: int, weight_format: int = 0) -> dict:
    """The launch configuration a call with these sizes uses (host only).
    weight_format: 0 bf16, 1 MXFP4 (True also means MXFP4), 2 MXFP8."""
    buf = ctypes.create_string_buffer(512)
    code = lib().skgemm_tactic_for(T, N, K, split_k, int(weight_format), buf, len(buf))
    _check(code, "skgemm_tactic_for")
    return json.loads(buf.value.decode())


def skgemm_set_timeline(buf, capacity: int) -> None:
    """Opt-in per-workgroup phase stamps of the stream kernel (None turns them off)."""
    _check(lib().skgemm_set_timeline(_ptr(buf, 8 * capacity if buf is not None else 0, "buf"),
                                     capacity if buf is not None else 0), "skgemm_set_timeline")


def skgemm_read_probe(src, nbytes: int, sink, stream=None) -> None:
    """Plain coalesced read of nbytes at src (the streaming-read reference)."""
    _check(lib().skgemm_read_probe(_ptr(src, nbytes, "src"), nbytes, _ptr(sink, 4 * 512, "sink"),
                                   _stream(stream)), "skgemm_read_probe")


def skgemm_health(stream=None) -> dict:
    """Owner time-outs of the stream's split-K hand-off since the last call
    (read and cleared): {"timeouts": n, "records": [(group, rank, problem, ticks), ...]}."""
    words = (ctypes.c_uint32 * 128)()
    _check(lib().skgemm_health(words, 128, _stream(stream)), "skgemm_health")
    recs = [tuple(words[8 + 8 * r + i] for i in range(1, 5))
            for r in range(min(words[0], 15)) if words[8 + 8 * r] == 1]
    return {"timeouts": int(words[0]), "records": recs}


def skgemm_strerror(code: int) -> str:
    return strerror(code)


def skgemm_last_hip_error() -> int:
    return lib().skgemm_last_hip_error()


def skgemm_set_override(knob, value: int) -> None:
    """Pin a choice the library otherwise makes itself (tests and tuning runs);
    knob is a name of ``KNOBS`` or its number, value -1 restores the default."""
    k = KNOBS[knob] if isinstance(knob, str) else int(knob)
    _check(lib().skgemm_set_override(k, int(value)), "skgemm_set_override")


def clear_overrides() -> None:
    """Restore the library's own choice for every knob."""
    for k in KNOBS.values():
        _check(lib().skgemm_set_override(k, -1), "skgemm_set_override")
