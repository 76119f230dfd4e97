"""ctypes binding of libawq.so (declared in include/awq.h and awq_serving.h).

Argument marshalling only: every function here passes device pointers,
sizes and the current CUDA stream to the C ABI of the same name and raises
AwqError on a non-zero status; the serving calls also refuse tensors of another
device, type or layout than they read.  Every step of the search runs in the
library's sm_100a kernels; there is no fallback.  If the library is missing
the import of this module fails with a message saying how to build it.
"""

from __future__ import annotations

import ctypes
import os
import re
from ctypes import POINTER, c_char_p, c_double, c_float, c_int32, c_int64, c_size_t, c_uint8, c_void_p
from typing import Optional

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
# AWQ_LIB=debug loads the debug library (index checks in the kernels,
# awq_bounds_status); the default is the release library
LIB_PATH = os.path.join(PKG_DIR, "libawq_debug.so" if os.environ.get("AWQ_LIB") == "debug"
                        else "libawq.so")
HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "awq.h")
SERVING_HEADER_PATH = os.path.join(os.path.dirname(PKG_DIR), "include", "awq_serving.h")

STATUS = {
    0: "AWQ_OK",
    1: "AWQ_ERR_INVALID_ARG",
    2: "AWQ_ERR_UNSUPPORTED",
    3: "AWQ_ERR_WORKSPACE",
    4: "AWQ_ERR_CUDA",
    5: "AWQ_ERR_TIMEOUT",
    6: "AWQ_ERR_NONFINITE",
}


class AwqError(RuntimeError):
    def __init__(self, func: str, status: int, message: str):
        self.status = status
        self.status_name = STATUS.get(status, str(status))
        super().__init__(f"{func}: {self.status_name}: {message}")


SEARCH_DIRECT, SEARCH_GRAM, SEARCH_CACHED_Y, SEARCH_FUSED = 0, 1, 2, 3


class AwqConfig(ctypes.Structure):
    """awq_config: w_bit, group_size, zero_point ("05 — AWQ" §9 quant_config),
    n_alpha, n_clip, clip_min ("05 — AWQ" §4), search_form (0 direct scored
    GEMM, 1 Gram form, 2 cached fp16 output, 3 candidates made inside the
    GEMM)."""

    _fields_ = [
        ("w_bit", c_int32),
        ("group_size", c_int32),
        ("zero_point", c_int32),
        ("n_alpha", c_int32),
        ("n_clip", c_int32),
        ("clip_min", c_float),
        ("search_form", c_int32),
    ]

    @classmethod
    def make(cls, w_bit=4, group_size=128, zero_point=1, n_alpha=20, n_clip=0, clip_min=0.5,
             search_form=0):
        return cls(int(w_bit), int(group_size), int(zero_point), int(n_alpha), int(n_clip),
                   float(clip_min), int(search_form))


_SIGNATURES = {
    "awq_version": (c_char_p, []),
    "awq_last_error": (c_char_p, []),
    "awq_workspace_size": (c_size_t, [c_int64, c_int64, c_int64, POINTER(AwqConfig)]),
    "awq_workspace_size_min": (c_size_t, [c_int64, c_int64, c_int64, POINTER(AwqConfig)]),
    "awq_act_stats": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_void_p]),
    "awq_scale_grid": (c_int32, [c_void_p, c_int64, c_int32, c_void_p, c_void_p]),
    "awq_search_scale": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int64, c_void_p,
                                   POINTER(AwqConfig), c_void_p, c_size_t, c_void_p, c_void_p,
                                   c_void_p, c_void_p]),
    "awq_search_clip": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int64, c_void_p,
                                  POINTER(AwqConfig), c_void_p, c_size_t, c_void_p, c_void_p,
                                  c_void_p]),
    "awq_search_clip_noalloc": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int64,
                                          c_void_p, POINTER(AwqConfig), c_void_p, c_void_p,
                                          c_void_p]),
    "awq_candidate_codes": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, POINTER(AwqConfig),
                                      c_void_p, c_size_t, c_void_p, c_void_p, c_void_p, c_void_p]),
    "awq_clip_candidate_codes": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p,
                                           POINTER(AwqConfig), c_void_p, c_size_t, c_void_p,
                                           c_void_p, c_void_p, c_void_p, c_void_p]),
    "awq_quant_pack": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p, POINTER(AwqConfig),
                                 c_void_p, c_void_p, c_void_p, c_void_p]),
    "awq_fold_inv_scale": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p]),
    "awq_w4a16_gemm": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_void_p, c_void_p,
                                 c_int64, POINTER(AwqConfig), c_void_p, c_int64, c_void_p, c_size_t,
                                 c_void_p]),
    "awq_w4a16_workspace_size": (c_size_t, [c_int64, c_int64, c_int64, POINTER(AwqConfig)]),
    "awq_w4a16_lora_gemm": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_void_p, c_void_p,
                                      c_int64, POINTER(AwqConfig), c_void_p, c_void_p, c_void_p, c_int32,
                                      c_int32, c_void_p, c_void_p, c_int64, c_void_p, c_size_t, c_void_p]),
    "awq_w4a16_lora_workspace_size": (c_size_t, [c_int64, c_int64, c_int64, c_int32,
                                                 POINTER(AwqConfig)]),
    "awq_w4a16_moe": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_void_p, c_int32, c_int32,
                                c_int32, c_void_p, c_void_p, c_void_p, c_int64, c_void_p, c_void_p,
                                c_void_p, POINTER(AwqConfig), c_void_p, c_int64, c_void_p, c_void_p,
                                c_void_p, c_size_t, c_void_p]),
    "awq_w4a16_moe_workspace_size": (c_size_t, [c_int64, c_int64, c_int64, c_int32, c_int32,
                                                POINTER(AwqConfig)]),
    "awq_block_norm": (c_int32, [c_void_p, c_int64, c_void_p, c_int64, c_int64, c_int64, c_void_p, c_void_p,
                                 c_int64, c_float, c_void_p, c_float, c_void_p, c_int64, c_void_p, c_int64,
                                 c_void_p]),
    "awq_act_sums": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_void_p]),
    "awq_act_stats_finish": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p]),
    "awq_search_scale_sse": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, c_int64,
                                       c_void_p, POINTER(AwqConfig), c_void_p, c_size_t, c_void_p,
                                       c_void_p]),
    "awq_select_scale": (c_int32, [c_void_p, c_int64, c_int64, c_int64, c_void_p, POINTER(AwqConfig),
                                   c_void_p, c_size_t, c_void_p, c_void_p, c_void_p, c_void_p]),
    "awq_block_grams": (c_int32, [c_void_p, c_int64, c_int64, c_int64, POINTER(AwqConfig), c_void_p,
                                  c_size_t, c_void_p, c_void_p]),
    "awq_search_clip_grams": (c_int32, [c_void_p, c_int64, c_int64, c_void_p, c_void_p,
                                        POINTER(AwqConfig), c_void_p, c_size_t, c_void_p, c_void_p,
                                        c_void_p]),
    "awq_device_status": (c_int32, [c_void_p, c_void_p]),
    "awq_profile_enable": (c_int32, [c_int32]),
    "awq_profile_read": (c_int32, [c_char_p, POINTER(c_double), POINTER(c_int64)]),
    "awq_profile_reset": (c_int32, []),
    "awq_bounds_checks_enabled": (c_int32, []),
    "awq_bounds_status": (c_int32, []),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m post_weight_quantization_awq_b200.build` "
            "(nvcc, sm_100a); there is no fallback implementation")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGNATURES.items():
        try:
            fn = getattr(lib, name)
        except AttributeError as e:
            raise ImportError(f"{LIB_PATH} does not export {name}: rebuild it") from e
        fn.restype = res
        fn.argtypes = args
    return lib


class _Lib:
    """libawq.so, loaded on first use (so that the build module can be
    imported before the library exists); a missing or stale library raises
    ImportError at the first call."""

    _lib = None

    def _get(self) -> ctypes.CDLL:
        if _Lib._lib is None:
            _Lib._lib = _load()
        return _Lib._lib

    def __getattr__(self, name):
        fn = getattr(self._get(), name)
        setattr(self, name, fn)  # found without this call the next time
        return fn

    def __getitem__(self, name):
        return self._get()[name]


LIB = _Lib()


def header_functions(path: str = HEADER_PATH):
    """Names of the functions a header (include/awq.h) declares."""
    with open(path) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(awq_[a-z0-9_]+)\s*\(", text)))


def version() -> str:
    return LIB.awq_version().decode()


def last_error() -> str:
    return LIB.awq_last_error().decode()


def _check(func: str, status: int) -> None:
    if status != 0:
        raise AwqError(func, status, last_error())


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is not None:
        return int(stream)
    import torch
    # the current stream's handle without building a Stream object (0.1 against 3 us)
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def awq_workspace_size(T: int, inn: int, out: int, cfg: AwqConfig) -> int:
    n = LIB.awq_workspace_size(T, inn, out, ctypes.byref(cfg))
    if n == 0:
        raise AwqError("awq_workspace_size", 1, last_error())
    return int(n)


def awq_workspace_size_min(T: int, inn: int, out: int, cfg: AwqConfig) -> int:
    """The smallest workspace the search and clip calls accept (the alpha
    search then runs its candidates in chunks)."""
    n = LIB.awq_workspace_size_min(T, inn, out, ctypes.byref(cfg))
    if n == 0:
        raise AwqError("awq_workspace_size_min", 1, last_error())
    return int(n)


def awq_act_stats(X, abar, stream=None) -> None:
    """X: CUDA fp16 [T, in] (row stride X.stride(0)); abar: CUDA fp64 [in]."""
    _check("awq_act_stats", LIB.awq_act_stats(_ptr(X), X.shape[0], X.shape[1], X.stride(0),
                                              _ptr(abar), _stream(stream)))


def awq_scale_grid(abar, n_alpha: int, s, stream=None) -> None:
    _check("awq_scale_grid", LIB.awq_scale_grid(_ptr(abar), abar.shape[0], n_alpha, _ptr(s),
                                                _stream(stream)))


def awq_search_scale(X, W, abar, cfg: AwqConfig, ws, s_best, mse, best_idx, stream=None) -> None:
    _check("awq_search_scale", LIB.awq_search_scale(
        _ptr(X), X.shape[0], X.shape[1], X.stride(0), _ptr(W), W.shape[0], _ptr(abar),
        ctypes.byref(cfg), _ptr(ws), ws.numel() * ws.element_size(), _ptr(s_best), _ptr(mse),
        _ptr(best_idx), _stream(stream)))


def awq_search_clip(X, W, s, cfg: AwqConfig, ws, clip_idx, err=None, stream=None) -> None:
    _check("awq_search_clip", LIB.awq_search_clip(
        _ptr(X), X.shape[0], X.shape[1], X.stride(0), _ptr(W), W.shape[0], _ptr(s),
        ctypes.byref(cfg), _ptr(ws), ws.numel() * ws.element_size(), _ptr(clip_idx), _ptr(err),
        _stream(stream)))


def awq_search_clip_noalloc(X, W, s, cfg: AwqConfig, clip_idx, err=None, stream=None) -> None:
    """awq_search_clip without a workspace (scratch in the library's static
    device array; in <= 16384; overlapping calls race)."""
    _check("awq_search_clip_noalloc", LIB.awq_search_clip_noalloc(
        _ptr(X), X.shape[0], X.shape[1], X.stride(0), _ptr(W), W.shape[0], _ptr(s),
        ctypes.byref(cfg), _ptr(clip_idx), _ptr(err), _stream(stream)))


def awq_quant_pack(W, s, clip_idx, cfg: AwqConfig, qweight, qzeros, scales, stream=None) -> None:
    _check("awq_quant_pack", LIB.awq_quant_pack(
        _ptr(W), W.shape[0], W.shape[1], _ptr(s), _ptr(clip_idx), ctypes.byref(cfg),
        _ptr(qweight), _ptr(qzeros), _ptr(scales), _stream(stream)))


def awq_fold_inv_scale(v, s, stream=None) -> None:
    rows = v.shape[0]
    cols = v.numel() // rows
    _check("awq_fold_inv_scale", LIB.awq_fold_inv_scale(_ptr(v), rows, cols, _ptr(s),
                                                        _stream(stream)))


def awq_act_sums(X, sums, stream=None) -> None:
    """Exact sums of |X| over these tokens, int64 [in] in units of 2^-24."""
    _check("awq_act_sums", LIB.awq_act_sums(_ptr(X), X.shape[0], X.shape[1], X.stride(0),
                                            _ptr(sums), _stream(stream)))


def awq_act_stats_finish(sums, T_total: int, abar, stream=None) -> None:
    _check("awq_act_stats_finish", LIB.awq_act_stats_finish(_ptr(sums), int(T_total), sums.shape[0],
                                                            _ptr(abar), _stream(stream)))


def awq_search_scale_sse(X, W, abar, cfg: AwqConfig, ws, sse, stream=None) -> None:
    _check("awq_search_scale_sse", LIB.awq_search_scale_sse(
        _ptr(X), X.shape[0], X.shape[1], X.stride(0), _ptr(W), W.shape[0], _ptr(abar),
        ctypes.byref(cfg), _ptr(ws), ws.numel() * ws.element_size(), _ptr(sse), _stream(stream)))


def awq_select_scale(sse, T_total: int, out: int, abar, cfg: AwqConfig, ws, s_best, mse, best_idx,
                     stream=None) -> None:
    _check("awq_select_scale", LIB.awq_select_scale(
        _ptr(sse), int(T_total), abar.shape[0], int(out), _ptr(abar), ctypes.byref(cfg), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(s_best), _ptr(mse), _ptr(best_idx), _stream(stream)))


def awq_block_grams(X, cfg: AwqConfig, ws, G, stream=None) -> None:
    _check("awq_block_grams", LIB.awq_block_grams(
        _ptr(X), X.shape[0], X.shape[1], X.stride(0), ctypes.byref(cfg), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(G), _stream(stream)))


def awq_search_clip_grams(W, s, G, cfg: AwqConfig, ws, clip_idx, err=None, stream=None) -> None:
    _check("awq_search_clip_grams", LIB.awq_search_clip_grams(
        _ptr(W), W.shape[0], W.shape[1], _ptr(s), _ptr(G), ctypes.byref(cfg), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(clip_idx), _ptr(err), _stream(stream)))


def awq_candidate_codes(W, abar, cfg: AwqConfig, ws, q, z, delta, stream=None) -> None:
    """Codes q uint8 [n_alpha, out, in], zero points z uint8 and steps delta
    fp32 [n_alpha, out, in/g] of every candidate of the alpha search."""
    _check("awq_candidate_codes", LIB.awq_candidate_codes(
        _ptr(W), W.shape[0], W.shape[1], _ptr(abar), ctypes.byref(cfg), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(q), _ptr(z), _ptr(delta), _stream(stream)))


def awq_clip_candidate_codes(W, s, G, cfg: AwqConfig, ws, clip_idx, err, q, z, stream=None) -> None:
    """awq_search_clip_grams that also stores the clip candidates' codes q
    uint8 [out, n_clip, in] and zero points z uint8 [out, n_clip, in/128]."""
    _check("awq_clip_candidate_codes", LIB.awq_clip_candidate_codes(
        _ptr(W), W.shape[0], W.shape[1], _ptr(s), _ptr(G), ctypes.byref(cfg), _ptr(ws),
        ws.numel() * ws.element_size(), _ptr(clip_idx), _ptr(err), _ptr(q), _ptr(z),
        _stream(stream)))


def awq_w4a16_gemm(X, qweight, qzeros, scales, cfg: AwqConfig, Y, ws, stream=None) -> None:
    """Y [T, out] fp16 = X [T, in] times the packed weights, dequantised on the fly."""
    _check("awq_w4a16_gemm", LIB.awq_w4a16_gemm(
        _ptr(X), X.shape[0], X.shape[1], X.stride(0), _ptr(qweight), _ptr(qzeros), _ptr(scales),
        Y.shape[1], ctypes.byref(cfg), _ptr(Y), Y.stride(0), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))


def awq_w4a16_workspace_size(T: int, inn: int, out: int, cfg: AwqConfig) -> int:
    """Workspace bytes that let awq_w4a16_gemm split K for few tokens."""
    n = LIB.awq_w4a16_workspace_size(T, inn, out, ctypes.byref(cfg))
    if n == 0:
        raise AwqError("awq_w4a16_workspace_size", 1, last_error())
    return int(n)


_serving = None


def _current(stream):
    """(fp16, int32, fp32, uint8, the current device, the stream's handle), without the
    0.2 us of an import statement."""
    global _serving
    if _serving is None:
        import torch
        _serving = (torch.float16, torch.int32, torch.float32, torch.uint8, torch._C._cuda_getDevice,
                    torch._C._cuda_getCurrentRawStream)
    f16, i32, f32, u8, device, raw_stream = _serving
    dev = device()
    return f16, i32, f32, u8, dev, raw_stream(dev) if stream is None else int(stream)


def _refuse(func: str, dev: int, rows, dense) -> None:
    """Names the tensor for which a serving call was refused: rows and dense are
    (name, tensor or None, dtype, shape), the first with rows that may lie apart."""
    for name, t, dtype, shape in rows + dense:
        if t is None:
            continue
        if t.get_device() != dev:
            raise AwqError(func, 1, f"{name} is on {t.device}, the current device is cuda:{dev}")
        if t.dtype is not dtype:
            raise AwqError(func, 1, f"{name} is {t.dtype}, {dtype} is needed")
        if t.shape != shape:
            raise AwqError(func, 1, f"{name} is {tuple(t.shape)}, {tuple(shape)} is needed")
    for name, t, _, _ in rows:
        if t is not None and t.stride(-1) != 1:
            raise AwqError(func, 1, f"the values of a row of {name} must be contiguous")
    for name, t, _, _ in dense:
        if t is not None and not t.is_contiguous():
            raise AwqError(func, 1, f"{name} must be contiguous")


def awq_w4a16_lora_gemm(X, qweight, qzeros, scales, cfg: AwqConfig, A, B, c, adapter, Y, ws,
                        stream=None) -> None:
    """Y [T, out] fp16 = X times the packed weights, plus for each token its
    adapter's c_a (X A_a^T) B_a^T: A fp16 [n, rank, in], B fp16 [n, out, rank],
    c fp32 [n], adapter int32 [T] (-1: none)."""
    f16, i32, f32, _, dev, stream = _current(stream)
    T, inn = X.shape
    n, rank, _ = A.shape
    out, g = Y.shape[-1], cfg.group_size
    xs, ys = X.stride(), Y.stride()
    if not (dev == X.get_device() == qweight.get_device() == qzeros.get_device() == scales.get_device()
            == A.get_device() == B.get_device() == c.get_device() == adapter.get_device() == Y.get_device()
            == ws.get_device()
            and f16 is X.dtype is scales.dtype is A.dtype is B.dtype is Y.dtype
            and i32 is qweight.dtype is qzeros.dtype is adapter.dtype and c.dtype is f32
            and xs[1] == 1 and ys[1] == 1 and qweight.is_contiguous() and qzeros.is_contiguous()
            and scales.is_contiguous() and A.is_contiguous() and B.is_contiguous() and c.is_contiguous()
            and adapter.is_contiguous() and ws.is_contiguous() and A.shape[2] == inn and B.shape == (n, out, rank)
            and c.numel() == n and adapter.numel() == T and Y.shape == (T, out)
            and qweight.shape == (inn, out // 8) and scales.shape == (inn // g, out)
            and qzeros.shape == (inn // g, out // 8)):
        _refuse("awq_w4a16_lora_gemm", dev, (("X", X, f16, (T, inn)), ("Y", Y, f16, (T, out))), (
            ("qweight", qweight, i32, (inn, out // 8)), ("qzeros", qzeros, i32, (inn // g, out // 8)),
            ("scales", scales, f16, (inn // g, out)), ("A", A, f16, (n, rank, inn)), ("B", B, f16, (n, out, rank)),
            ("c", c, f32, (n,)), ("adapter", adapter, i32, (T,)), ("ws", ws, ws.dtype, ws.shape)))
    _check("awq_w4a16_lora_gemm", LIB.awq_w4a16_lora_gemm(
        X.data_ptr(), T, inn, xs[0], qweight.data_ptr(), qzeros.data_ptr(), scales.data_ptr(),
        out, ctypes.byref(cfg), A.data_ptr(), B.data_ptr(), c.data_ptr(), n, rank, adapter.data_ptr(),
        Y.data_ptr(), ys[0], ws.data_ptr(), ws.numel() * ws.element_size(), stream))


def awq_w4a16_lora_workspace_size(T: int, inn: int, out: int, rank: int, cfg: AwqConfig) -> int:
    n = LIB.awq_w4a16_lora_workspace_size(T, inn, out, rank, ctypes.byref(cfg))
    if n == 0:
        raise AwqError("awq_w4a16_lora_workspace_size", 1, last_error())
    return int(n)


def awq_w4a16_moe(X, router, gate_up, down, cfg: AwqConfig, renormalize: bool, mask, Y, ids, weights, ws,
                  stream=None) -> None:
    """A mixture-of-experts layer on packed experts: X fp16 [T, hidden], router
    fp16 [E, hidden], gate_up and down (qweight, qzeros, scales) with a leading
    expert axis, mask uint8 [T] or None; outputs Y [T, hidden] fp16, ids int32
    and weights fp32 [T, top_k]."""
    f16, i32, f32, u8, dev, stream = _current(stream)
    gq, gz, gs = gate_up
    dq, dz, ds = down
    T, hidden = X.shape
    E, inter, _ = dq.shape
    top_k, g = ids.shape[-1], cfg.group_size
    xs, ys = X.stride(), Y.stride()
    if not (dev == X.get_device() == router.get_device() == gq.get_device() == gz.get_device() == gs.get_device()
            == dq.get_device() == dz.get_device() == ds.get_device() == Y.get_device() == ids.get_device()
            == weights.get_device() == ws.get_device()
            and f16 is X.dtype is router.dtype is gs.dtype is ds.dtype is Y.dtype
            and i32 is gq.dtype is gz.dtype is dq.dtype is dz.dtype is ids.dtype and weights.dtype is f32
            and xs[1] == 1 and ys[1] == 1 and router.is_contiguous() and gq.is_contiguous() and gz.is_contiguous()
            and gs.is_contiguous() and dq.is_contiguous() and dz.is_contiguous() and ds.is_contiguous()
            and ids.is_contiguous() and weights.is_contiguous() and ws.is_contiguous()
            and router.shape == (E, hidden) and gq.shape == (E, hidden, inter // 4)
            and dq.shape == (E, inter, hidden // 8) and gs.shape == (E, hidden // g, 2 * inter)
            and gz.shape == (E, hidden // g, inter // 4) and ds.shape == (E, inter // g, hidden)
            and dz.shape == (E, inter // g, hidden // 8) and Y.shape == (T, hidden)
            and ids.shape == (T, top_k) and weights.shape == (T, top_k)
            and (mask is None or (mask.get_device() == dev and mask.dtype is u8 and mask.is_contiguous()
                                  and mask.numel() == T))):
        _refuse("awq_w4a16_moe", dev, (("X", X, f16, (T, hidden)), ("Y", Y, f16, (T, hidden))), (
            ("router", router, f16, (E, hidden)),
            ("gate_up qweight", gq, i32, (E, hidden, inter // 4)),
            ("gate_up qzeros", gz, i32, (E, hidden // g, inter // 4)),
            ("gate_up scales", gs, f16, (E, hidden // g, 2 * inter)),
            ("down qweight", dq, i32, (E, inter, hidden // 8)), ("down qzeros", dz, i32, (E, inter // g, hidden // 8)),
            ("down scales", ds, f16, (E, inter // g, hidden)), ("mask", mask, u8, (T,)),
            ("ids", ids, i32, (T, top_k)), ("weights", weights, f32, (T, top_k)), ("ws", ws, ws.dtype, ws.shape)))
    _check("awq_w4a16_moe", LIB.awq_w4a16_moe(
        X.data_ptr(), T, hidden, xs[0], None if mask is None else mask.data_ptr(), router.data_ptr(), E, top_k,
        1 if renormalize else 0, gq.data_ptr(), gz.data_ptr(), gs.data_ptr(), inter, dq.data_ptr(), dz.data_ptr(),
        ds.data_ptr(), ctypes.byref(cfg), Y.data_ptr(), ys[0], ids.data_ptr(), weights.data_ptr(), ws.data_ptr(),
        ws.numel() * ws.element_size(), stream))


def awq_w4a16_moe_workspace_size(T: int, hidden: int, inter: int, n_experts: int, top_k: int,
                                 cfg: AwqConfig) -> int:
    n = LIB.awq_w4a16_moe_workspace_size(T, hidden, inter, n_experts, top_k, ctypes.byref(cfg))
    if n == 0:
        raise AwqError("awq_w4a16_moe_workspace_size", 1, last_error())
    return int(n)


def awq_block_norm(R, V, post, gate, c: float, pre, eps: float, R_out, N_out, stream=None) -> None:
    """R_out = R + c gate rmsnorm(V) post and N_out = rmsnorm(R_out) pre over
    fp16 rows [T, d]; V, post, gate ([T, d] or [d]), pre and one of the outputs
    may be None."""
    f16, _, _, _, dev, stream = _current(stream)
    none = (0, 1)
    shape = T, d = R.shape
    by_token = gate is not None and gate.dim() == 2
    ldr, r1 = R.stride()
    ldv, v1 = none if V is None else V.stride()
    ldro, ro1 = none if R_out is None else R_out.stride()
    ldno, no1 = none if N_out is None else N_out.stride()
    ldg, g1 = gate.stride() if by_token else none
    if not (r1 == v1 == ro1 == no1 == g1 == 1 and R.dtype is f16 and R.get_device() == dev
            and (V is None or (V.dtype is f16 and V.get_device() == dev and V.shape == shape))
            and (R_out is None or (R_out.dtype is f16 and R_out.get_device() == dev and R_out.shape == shape))
            and (N_out is None or (N_out.dtype is f16 and N_out.get_device() == dev and N_out.shape == shape))
            and (pre is None or (pre.dtype is f16 and pre.get_device() == dev and pre.numel() == d
                                 and pre.is_contiguous()))
            and (post is None or (post.dtype is f16 and post.get_device() == dev and post.numel() == d
                                  and post.is_contiguous()))
            and (gate is None or (gate.dtype is f16 and gate.get_device() == dev
                                  and (gate.shape == shape if by_token else gate.numel() == d
                                       and gate.is_contiguous())))):
        rows = [("R", R, f16, shape), ("V", V, f16, shape), ("R_out", R_out, f16, shape), ("N_out", N_out, f16, shape)]
        dense = [("post", post, f16, (d,)), ("pre", pre, f16, (d,))]
        (rows if by_token else dense).append(("gate", gate, f16, shape if by_token else (d,)))
        _refuse("awq_block_norm", dev, rows, dense)
    _check("awq_block_norm", LIB.awq_block_norm(
        R.data_ptr(), ldr, None if V is None else V.data_ptr(), ldv, T, d, None if post is None else post.data_ptr(),
        None if gate is None else gate.data_ptr(), ldg, c, None if pre is None else pre.data_ptr(), eps,
        None if R_out is None else R_out.data_ptr(), ldro, None if N_out is None else N_out.data_ptr(), ldno,
        stream))


def awq_device_status(ws, stream=None) -> None:
    """Raises AwqError if the device status in workspace ``ws`` records a
    failure; ws=None reads the library's own status word (the calls that take
    no workspace: awq_quant_pack, awq_search_clip_noalloc)."""
    _check("awq_device_status", LIB.awq_device_status(_ptr(ws), _stream(stream)))


def awq_bounds_checks_enabled() -> bool:
    """True in the debug library (index checks compiled into the kernels)."""
    return bool(LIB.awq_bounds_checks_enabled())


def awq_bounds_status() -> None:
    """Raises AwqError if a kernel index check failed since the last call
    (debug library); clears the record.  A no-op in the release library."""
    _check("awq_bounds_status", LIB.awq_bounds_status())


def profile_enable(on: bool) -> None:
    _check("awq_profile_enable", LIB.awq_profile_enable(1 if on else 0))


def profile_read(name: str):
    ms, n = c_double(0.0), c_int64(0)
    _check("awq_profile_read", LIB.awq_profile_read(name.encode(), ctypes.byref(ms), ctypes.byref(n)))
    return ms.value, n.value


def profile_reset() -> None:
    _check("awq_profile_reset", LIB.awq_profile_reset())
