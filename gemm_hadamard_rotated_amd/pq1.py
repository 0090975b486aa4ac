"""Thin Python binding of libpq1 (include/pq1.h), same names as the C calls.

Argument marshalling only: every step of the computation runs in the HIP
kernels of libpq1.so.  PyTorch provides device memory and the stream (the
current torch stream of the tensors' device).  There is no CPU fallback:
if the library is missing or the tensors are not on a GPU, the calls raise.
"""
from __future__ import annotations

import ctypes
import math
import os
import threading
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("PQ1_LIBRARY") or os.path.join(_HERE, "libpq1.so")

PQ1_OK = 0
PQ1_F32, PQ1_BF16, PQ1_BF16_GEMM, PQ1_F16 = 0, 1, 2, 3
PQ1_ROPE_HALVES, PQ1_ROPE_ADJACENT = 0, 1
PQ1_X_ROW_MAJOR, PQ1_X_GEMM_ORDER = 0, 1
PQ1_GEMV_AUTO, PQ1_GEMV_LUT, PQ1_GEMV_EXPAND = 0, 1, 2
PQ1_GEMV_COUNTER_BYTES = 262144  # split-K bookkeeping at the start of a GEMV workspace
PQ1_GEMV_STATUS_OFFSET = 261888  # the status word inside it
PQ1_SPLITK_WAIT_GAVE_UP, PQ1_SPLITK_OUT_OF_STEP = 1, 2
PQ1_TEST_WITHHOLD_PUBLISH = 1
PQ1_ERR_SPLITK = 9
STATUS_NAMES = {0: "PQ1_OK", 1: "PQ1_ERR_NULL", 2: "PQ1_ERR_SHAPE", 3: "PQ1_ERR_ALIGN",
                4: "PQ1_ERR_PERM", 5: "PQ1_ERR_ALIAS", 6: "PQ1_ERR_DEVICE",
                7: "PQ1_ERR_LAUNCH", 8: "PQ1_ERR_ARG", 9: "PQ1_ERR_SPLITK"}

# every symbol include/pq1.h declares
EXPORTS = ("pq1_rotate", "pq1_gemv_workspace_bytes", "pq1_gemv", "pq1_gemv_ex",
           "pq1_rotate_gemv", "pq1_packed_bits_bytes", "pq1_packed_scales_bytes",
           "pq1_packed_scales_bytes_ex", "pq1_pack_weights", "pq1_pack_weights_rows",
           "pq1_pack_weights_ex", "pq1_embed", "pq1_gemv_packed", "pq1_rotate_gemv_packed",
           "pq1_gemv_packed_ex", "pq1_rotate_gemv_packed_ex", "pq1_gemm", "pq1_gemm_ex",
           "pq1_status_str", "pq1_abi_version", "pq1_last_hip_error", "pq1_set_test_flags",
           "pq1_rotate_gemv_packed_noalloc", "pq1_rope", "pq1_kv_append",
           "pq1_paged_attention", "pq1_paged_attention_workspace_bytes", "pq1_norm_rope",
           "pq1_norm_rope_grad", "pq1_norm_rope_grad_workspace_bytes", "pq1_kv_append_ex",
           "pq1_kv4_append", "pq1_kv4_read", "pq1_paged_attention_ex",
           "pq1_paged_attention_ex_workspace_bytes", "pq1_kv4_attention",
           "pq1_kv4_attention_workspace_bytes")


class Pq1Error(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(code, code)} ({msg})")
        self.code = code


class Pq1Perm(ctypes.Structure):
    _fields_ = [("hd", ctypes.c_int32), ("nk", ctypes.c_int32), ("rep", ctypes.c_int32)]


class Pq1Heads(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64)]


class Pq1RopeSpec(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_int32), ("axes", ctypes.c_int32),
                ("section", ctypes.c_int32 * 4), ("interleaved", ctypes.c_int32),
                ("pairing", ctypes.c_int32), ("inverse", ctypes.c_int32)]


class Pq1KvCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("pages", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


class Pq1HeadNorm(ctypes.Structure):
    _fields_ = [("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


class Pq1Kv4Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("page_size", ctypes.c_int32), ("pages", ctypes.c_int64),
                ("heads", ctypes.c_int32), ("dim", ctypes.c_int32)]


_lib = None
_lib_lock = threading.Lock()


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libpq1.so (raises if it has not been built)."""
    global _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m gemm_hadamard_rotated_amd.build`")
        lib = ctypes.CDLL(path)
        P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        PP = ctypes.POINTER(Pq1Perm)
        PH, PS, PC, PN, P4 = (ctypes.POINTER(c) for c in (Pq1Heads, Pq1RopeSpec, Pq1KvCache,
                                                          Pq1HeadNorm, Pq1Kv4Cache))
        F = ctypes.c_float
        sig = {
            "pq1_rotate": (I32, [P, P, PP, P, I32, I64, I64, P]),
            "pq1_gemv_workspace_bytes": (SZ, [I64, I64]),
            "pq1_gemv": (I32, [P, P, P, P, I64, I64, P, SZ, P]),
            "pq1_gemv_ex": (I32, [P, P, P, P, I64, I64, I32, P, SZ, P]),
            "pq1_rotate_gemv": (I32, [P, P, PP, P, P, P, I64, I64, P, SZ, P]),
            "pq1_packed_bits_bytes": (SZ, [I64, I64]),
            "pq1_packed_scales_bytes": (SZ, [I64, I64]),
            "pq1_packed_scales_bytes_ex": (SZ, [I64, I64, I32]),
            "pq1_pack_weights": (I32, [P, P, I64, I64, P, P, P]),
            "pq1_pack_weights_rows": (I32, [P, P, I64, I64, P, P, I64, I64, P]),
            "pq1_pack_weights_ex": (I32, [P, P, I64, I64, P, P, I32, I64, I64, P]),
            "pq1_embed": (I32, [P, I64, P, P, P, P, I64, I64, P]),
            "pq1_gemv_packed": (I32, [P, P, P, P, I64, I64, P, SZ, P]),
            "pq1_rotate_gemv_packed": (I32, [P, P, PP, P, P, P, I64, I64, P, SZ, P]),
            "pq1_gemv_packed_ex": (I32, [P, P, P, I32, P, I64, I64, P, SZ, P]),
            "pq1_rotate_gemv_packed_ex": (I32, [P, P, PP, P, P, I32, P, I64, I64, P, SZ, P]),
            "pq1_gemm": (I32, [P, P, P, P, I64, I64, I64, P]),
            "pq1_gemm_ex": (I32, [P, P, P, P, I64, I64, I64, I32, P]),
            "pq1_set_test_flags": (ctypes.c_uint32, [ctypes.c_uint32]),
            "pq1_rotate_gemv_packed_noalloc": (I32, [P, P, PP, P, P, I32, P, I64, I64, P]),
            "pq1_rope": (I32, [PH, PH, P, P, PS, I64, I32, I32, P]),
            "pq1_kv_append": (I32, [PH, PH, P, PH, PH, I32, P, P, PS, PC, I64, P]),
            "pq1_paged_attention": (I32, [PH, PH, PC, P, I64, P, P, I64, I64, I32, I64, I64,
                                          ctypes.c_float, I32, I32, P, SZ, P]),
            "pq1_paged_attention_workspace_bytes": (SZ, [I64, I64, I32, I32, I32, I64, I64]),
            "pq1_norm_rope": (I32, [PH, PH, P, F, P, P, PS, I64, I32, I32, P]),
            "pq1_norm_rope_grad": (I32, [PH, PH, PH, P, P, F, P, P, PS, I64, I32, I32, P, SZ, P]),
            "pq1_norm_rope_grad_workspace_bytes": (SZ, [I64, I32]),
            "pq1_kv_append_ex": (I32, [PH, PH, P, PH, PH, I32, P, P, PS, PN, PC, I64, P]),
            "pq1_kv4_append": (I32, [PH, PH, P, PH, PH, I32, P, P, PS, PN, P4, I64, P]),
            "pq1_kv4_read": (I32, [P4, P, PH, PH, I64, P]),
            "pq1_paged_attention_ex": (I32, [PH, PH, PC, P, I64, P, P, I64, I64, I32, I64, I64, F,
                                             I32, I32, I32, P, SZ, P]),
            "pq1_paged_attention_ex_workspace_bytes": (SZ, [I64, I64, I32, I32, I32, I64, I64, I32,
                                                            I32]),
            "pq1_kv4_attention": (I32, [PH, PH, P4, P, I64, P, P, I64, I64, I32, I64, I64, F, I32,
                                        I32, I32, P, SZ, P]),
            "pq1_kv4_attention_workspace_bytes": (SZ, [I64, I64, I32, I32, I32, I64, I64, I32, I32]),
            "pq1_status_str": (ctypes.c_char_p, [I32]),
            "pq1_abi_version": (I32, []),
            "pq1_last_hip_error": (I32, []),
        }
        for name, (res, args) in sig.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def _check(code: int, where: str):
    if code != PQ1_OK:
        lib = load_library()
        raise Pq1Error(code, where, lib.pq1_status_str(code).decode()
                       + f"; hip error {lib.pq1_last_hip_error()}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(dev).cuda_stream)


def _need(t: torch.Tensor, name: str, dtypes: Sequence[torch.dtype], dev=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU (no CPU path exists)")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# The library takes plain pointers and sizes, so it cannot see a tensor that
# is smaller than the sizes say; these checks keep a mismatched tensor from
# reaching a kernel that would read or write past its end.
def _need_numel(t: torch.Tensor, name: str, n: int):
    if t.numel() != n:
        raise ValueError(f"{name} has {t.numel()} elements, expected {n}")


def _need_weights(w_bits: torch.Tensor, scales: torch.Tensor, K: int, what: str) -> int:
    """w_bits [N][K/32] words and scales [N][K/128] for an activation of
    width K; returns N.  (A K the library rejects is left to it.)"""
    if w_bits.dim() != 2:
        raise ValueError(f"{what}: w_bits must be 2-D, [N][K/32] words")
    N = int(w_bits.shape[0])
    if w_bits.shape[1] * 32 != K:
        raise ValueError(f"{what}: w_bits has {w_bits.shape[1]} words per row, "
                         f"an activation of width {K} needs {K / 32:g}")
    if K % 128 == 0:
        _need_numel(scales, "scales", N * (K // 128))
    return N


def _perm(perm):
    if perm is None:
        return None
    hd, nk, rep = (int(v) for v in perm)
    return ctypes.byref(Pq1Perm(hd, nk, rep))


_WORD_DTYPES = (torch.int32, torch.uint32)

# ----------------------------------------------------------------------------
# GEMV workspace, one per (device, stream), grown on demand.  A new workspace
# is zero-filled; every call leaves its counter region in a state the next call
# accepts, so calls of any shapes ordered on the stream can share it
# (include/pq1.h).
# ----------------------------------------------------------------------------
_ws = {}
_ws_retired = []  # replaced workspaces, kept alive for graphs that captured them
_ws_lock = threading.Lock()


def check_gemv_workspace(device: Optional[torch.device] = None) -> None:
    """Raise Pq1Error(PQ1_ERR_SPLITK) if a packed-layout GEMV on the current
    stream's workspace reported trouble in the workspace's status word since
    the last check (a split-K wait that gave up, or bookkeeping found out of
    step; the affected outputs are NaN).  Waits for the stream.  On an error
    the counter region is zero-filled, so the next call starts in step."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    key = (device.index, torch.cuda.current_stream(device).cuda_stream)
    with _ws_lock:
        ws = _ws.get(key)
    if ws is None:
        return
    word = ws[PQ1_GEMV_STATUS_OFFSET:PQ1_GEMV_STATUS_OFFSET + 4].view(torch.int32)
    status = int(word.item())
    if status:
        ws[:PQ1_GEMV_COUNTER_BYTES].zero_()
        parts = []
        if status & PQ1_SPLITK_WAIT_GAVE_UP:
            parts.append("a split-K wait gave up")
        if status & PQ1_SPLITK_OUT_OF_STEP:
            parts.append("split-K bookkeeping was out of step")
        raise Pq1Error(PQ1_ERR_SPLITK, "GEMV workspace",
                       " and ".join(parts) + "; the affected outputs are NaN")


def pq1_set_test_flags(flags: int) -> int:
    """Failure-handling tests only (include/pq1.h); returns the previous flags."""
    return int(load_library().pq1_set_test_flags(int(flags)))


def gemv_workspace(N: int, K: int, device: torch.device) -> torch.Tensor:
    lib = load_library()
    need = int(lib.pq1_gemv_workspace_bytes(int(N), int(K)))
    if need == 0:
        raise Pq1Error(2, "pq1_gemv_workspace_bytes", "invalid shape")
    stream = torch.cuda.current_stream(device).cuda_stream
    key = (device.index, stream)
    with _ws_lock:
        ws = _ws.get(key)
        if ws is None or ws.numel() < need:
            if ws is not None:
                # a graph captured earlier may still hold the old buffer's address
                _ws_retired.append(ws)
            ws = torch.zeros(max(need, 1 << 20), dtype=torch.uint8, device=device)
            _ws[key] = ws
        return ws


# ----------------------------------------------------------------------------
# Calls
# ----------------------------------------------------------------------------
def pq1_rotate(x: torch.Tensor, signs: torch.Tensor, perm=None,
               out_dtype: torch.dtype = torch.float32,
               out: Optional[torch.Tensor] = None, gemm_order: bool = False) -> torch.Tensor:
    """x_rot = WHT_1024(signs * P x) / 32 per row of x ([K] or [M][K] fp32).

    With out_dtype=torch.bfloat16 and gemm_order=True the result is stored in
    the K order of pq1_gemm's operand (PQ1_BF16_GEMM)."""
    _need(x, "x", (torch.float32,))
    dev = x.device
    _need(signs, "signs", (torch.float32,), dev)
    K = x.shape[-1]
    M = x.numel() // K if K else 0
    _need_numel(signs, "signs", K)
    code = {torch.float32: PQ1_F32, torch.bfloat16: PQ1_BF16}.get(out_dtype)
    if code is None:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    if gemm_order:
        if code != PQ1_BF16:
            raise ValueError("gemm_order needs out_dtype=torch.bfloat16")
        code = PQ1_BF16_GEMM
    if out is None:
        out = torch.empty(x.shape, dtype=out_dtype, device=dev)
    else:
        _need(out, "out", (out_dtype,), dev)
        if out.shape != x.shape:
            raise ValueError("out must have the shape of x")
    lib = load_library()
    with torch.cuda.device(dev):
        _check(lib.pq1_rotate(_ptr(x), _ptr(signs), _perm(perm), _ptr(out), code, M, K,
                              _stream(dev)), "pq1_rotate")
    return out


def pq1_gemv_ex(x_rot: torch.Tensor, w_bits: torch.Tensor, scales: torch.Tensor,
                algo: int = PQ1_GEMV_AUTO, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = W x_rot for one [K] fp32 activation; W from packed bits and scales."""
    _need(x_rot, "x_rot", (torch.float32,))
    dev = x_rot.device
    _need(w_bits, "w_bits", _WORD_DTYPES, dev)
    _need(scales, "scales", (torch.float32,), dev)
    K = x_rot.numel()
    N = _need_weights(w_bits, scales, K, "pq1_gemv_ex")
    if out is None:
        out = torch.empty(N, dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), dev)
        _need_numel(out, "out", N)
    lib = load_library()
    with torch.cuda.device(dev):
        ws = gemv_workspace(N, K, dev) if K >= 128 and K % 128 == 0 and N >= 1 else None
        _check(lib.pq1_gemv_ex(_ptr(x_rot), _ptr(w_bits), _ptr(scales), _ptr(out), N, K,
                               int(algo), _ptr(ws), 0 if ws is None else ws.numel(),
                               _stream(dev)), "pq1_gemv_ex")
    return out


def pq1_gemv(x_rot, w_bits, scales, out=None) -> torch.Tensor:
    return pq1_gemv_ex(x_rot, w_bits, scales, PQ1_GEMV_AUTO, out)


def pq1_rotate_gemv(x: torch.Tensor, signs: torch.Tensor, w_bits: torch.Tensor,
                    scales: torch.Tensor, perm=None,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = W WHT_1024(signs * P x) / 32 in one launch, for one [K] activation."""
    _need(x, "x", (torch.float32,))
    dev = x.device
    _need(signs, "signs", (torch.float32,), dev)
    _need(w_bits, "w_bits", _WORD_DTYPES, dev)
    _need(scales, "scales", (torch.float32,), dev)
    K = x.numel()
    N = _need_weights(w_bits, scales, K, "pq1_rotate_gemv")
    _need_numel(signs, "signs", K)
    if out is None:
        out = torch.empty(N, dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), dev)
        _need_numel(out, "out", N)
    lib = load_library()
    with torch.cuda.device(dev):
        ws = gemv_workspace(N, K, dev) if K >= 128 and K % 128 == 0 and N >= 1 else None
        _check(lib.pq1_rotate_gemv(_ptr(x), _ptr(signs), _perm(perm), _ptr(w_bits),
                                   _ptr(scales), _ptr(out), N, K, _ptr(ws),
                                   0 if ws is None else ws.numel(), _stream(dev)),
               "pq1_rotate_gemv")
    return out


# pq1_scale_dtype: storage type of the packed scales
SCALE_DTYPES = {"f32": 0, "f16": 1}
_SCALE_TORCH = {"f32": torch.float32, "f16": torch.float16}


def _scale_code(scale_dtype: str) -> int:
    if scale_dtype not in SCALE_DTYPES:
        raise Pq1Error(8, "scale_dtype", f"unknown scale dtype {scale_dtype!r} (f32 or f16)")
    return SCALE_DTYPES[scale_dtype]


class PackedWeights:
    """Band-interleaved copy of a 1-bit weight matrix (see pq1_pack_weights);
    scale_dtype is the storage type of its scales ("f32" or "f16")."""

    def __init__(self, bits: torch.Tensor, scales: torch.Tensor, N: int, K: int,
                 scale_dtype: str = "f32"):
        self.bits, self.scales, self.N, self.K = bits, scales, int(N), int(K)
        self.scale_dtype = scale_dtype

    @property
    def device(self):
        return self.bits.device


def _need_packed(pw: PackedWeights, dev):
    """The packed arrays are on `dev` and as large as the library says a
    packed matrix of pw.N x pw.K is."""
    if not isinstance(pw, PackedWeights):
        raise TypeError("pw must be a PackedWeights (pq1_pack_weights)")
    lib = load_library()
    nb = int(lib.pq1_packed_bits_bytes(pw.N, pw.K))
    ns = int(lib.pq1_packed_scales_bytes_ex(pw.N, pw.K, _scale_code(pw.scale_dtype)))
    for t, name, need in ((pw.bits, "packed bits", nb), (pw.scales, "packed scales", ns)):
        if t.device != dev:
            raise ValueError(f"{name} are on {t.device}, expected {dev}")
        if not t.is_contiguous() or t.numel() * t.element_size() < need:
            raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, need {need}")


def _alloc_packed(N: int, K: int, scale_dtype: str, dev, what: str) -> PackedWeights:
    lib = load_library()
    nb = int(lib.pq1_packed_bits_bytes(N, K))
    ns = int(lib.pq1_packed_scales_bytes_ex(N, K, _scale_code(scale_dtype)))
    if nb == 0 or ns == 0:
        raise Pq1Error(2, what, "invalid shape")
    dt = _SCALE_TORCH[scale_dtype]
    pbits = torch.empty(nb // 4, dtype=torch.int32, device=dev)
    pscales = torch.empty(ns // dt.itemsize, dtype=dt, device=dev)
    return PackedWeights(pbits, pscales, N, K, scale_dtype)


def _check_parts(parts, dev, what):
    if not parts:
        raise Pq1Error(2, what, "no matrices")
    KW = parts[0][0].shape[1]
    for w_bits, scales in parts:
        _need(w_bits, "w_bits", _WORD_DTYPES, dev)
        _need(scales, "scales", (torch.float32,), dev)
        if w_bits.dim() != 2 or w_bits.shape[1] != KW:
            raise Pq1Error(2, what, "all matrices must have the same K")
        _need_weights(w_bits, scales, KW * 32, what)
    return KW * 32, sum(w.shape[0] for w, _ in parts)


def pq1_pack_weights(w_bits: torch.Tensor, scales: torch.Tensor,
                     scale_dtype: str = "f32") -> PackedWeights:
    """Repack [N][K/32] words + [N][K/128] scales into the packed layout
    (scales stored as fp32, or rounded to f16 through pq1_pack_weights_ex)."""
    if scale_dtype != "f32":
        return pq1_pack_weights_ex(w_bits, scales, scale_dtype)
    _need(w_bits, "w_bits", _WORD_DTYPES)
    dev = w_bits.device
    _need(scales, "scales", (torch.float32,), dev)
    N, KW = w_bits.shape
    K = KW * 32
    _need_weights(w_bits, scales, K, "pq1_pack_weights")
    pw = _alloc_packed(N, K, "f32", dev, "pq1_pack_weights")
    lib = load_library()
    with torch.cuda.device(dev):
        _check(lib.pq1_pack_weights(_ptr(w_bits), _ptr(scales), N, K, _ptr(pw.bits),
                                    _ptr(pw.scales), _stream(dev)), "pq1_pack_weights")
    return pw


def pq1_pack_weights_ex(w_bits: torch.Tensor, scales: torch.Tensor, scale_dtype: str = "f16",
                        into: Optional[PackedWeights] = None, row0: int = 0) -> PackedWeights:
    """Repack one matrix with the given scale storage.  Without `into` a new
    packed matrix of N rows is made; with it, the rows go to rows row0 ..
    row0+N-1 of `into` (same K and scale_dtype), which is returned."""
    _need(w_bits, "w_bits", _WORD_DTYPES)
    dev = w_bits.device
    _need(scales, "scales", (torch.float32,), dev)
    code = _scale_code(scale_dtype)
    N, KW = w_bits.shape
    K = KW * 32
    _need_weights(w_bits, scales, K, "pq1_pack_weights_ex")
    if into is None:
        into = _alloc_packed(N, K, scale_dtype, dev, "pq1_pack_weights_ex")
        row0 = 0
    elif into.K != K or into.scale_dtype != scale_dtype or into.device != dev:
        raise Pq1Error(2, "pq1_pack_weights_ex", "target has another K, scale dtype or device")
    lib = load_library()
    with torch.cuda.device(dev):
        _check(lib.pq1_pack_weights_ex(_ptr(w_bits), _ptr(scales), N, K, _ptr(into.bits),
                                       _ptr(into.scales), code, into.N, row0, _stream(dev)),
               "pq1_pack_weights_ex")
    return into


def pq1_pack_weights_rows(parts, dev=None, scale_dtype: str = "f32") -> PackedWeights:
    """Pack several matrices with the same K, given as [(w_bits, scales), ...],
    one after another into one packed matrix (pq1_pack_weights_rows per part,
    or pq1_pack_weights_ex for f16 scales): one GEMV launch then yields their
    outputs one after another."""
    parts = list(parts)
    dev = parts[0][0].device if (dev is None and parts) else dev
    K, n_total = _check_parts(parts, dev, "pq1_pack_weights_rows")
    pw = _alloc_packed(n_total, K, scale_dtype, dev, "pq1_pack_weights_rows")
    lib = load_library()
    row0 = 0
    with torch.cuda.device(dev):
        for w_bits, scales in parts:
            n = w_bits.shape[0]
            if scale_dtype == "f32":
                _check(lib.pq1_pack_weights_rows(_ptr(w_bits), _ptr(scales), n, K, _ptr(pw.bits),
                                                 _ptr(pw.scales), n_total, row0, _stream(dev)),
                       "pq1_pack_weights_rows")
            else:
                pq1_pack_weights_ex(w_bits, scales, scale_dtype, into=pw, row0=row0)
            row0 += n
    return pw


def pq1_embed(tokens: torch.Tensor, w_bits: torch.Tensor, scales: torch.Tensor,
              signs: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Rows tokens[m] of a 1-bit table, with the inverse rotation:
    out[m] = signs * WHT_1024(dequantized row) / 32 (fp32 [M][K])."""
    _need(tokens, "tokens", (torch.int32,))
    dev = tokens.device
    _need(w_bits, "w_bits", _WORD_DTYPES, dev)
    _need(scales, "scales", (torch.float32,), dev)
    _need(signs, "signs", (torch.float32,), dev)
    V, KW = w_bits.shape
    K = KW * 32
    M = tokens.numel()
    _need_weights(w_bits, scales, K, "pq1_embed")
    _need_numel(signs, "signs", K)
    if out is None:
        out = torch.empty((M, K), dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), dev)
        _need_numel(out, "out", M * K)
    lib = load_library()
    with torch.cuda.device(dev):
        _check(lib.pq1_embed(_ptr(tokens), M, _ptr(w_bits), _ptr(scales), _ptr(signs), _ptr(out),
                             V, K, _stream(dev)), "pq1_embed")
    return out


def pq1_gemv_packed(x_rot: torch.Tensor, pw: PackedWeights,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = W x_rot with W given as PackedWeights (f16 scales: pq1_gemv_packed_ex)."""
    if pw.scale_dtype != "f32":
        return pq1_gemv_packed_ex(x_rot, pw, out)
    _need(x_rot, "x_rot", (torch.float32,))
    dev = x_rot.device
    _need_packed(pw, dev)
    _need_numel(x_rot, "x_rot", pw.K)
    if out is None:
        out = torch.empty(pw.N, dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), dev)
        _need_numel(out, "out", pw.N)
    lib = load_library()
    with torch.cuda.device(dev):
        ws = gemv_workspace(pw.N, pw.K, dev)
        _check(lib.pq1_gemv_packed(_ptr(x_rot), _ptr(pw.bits), _ptr(pw.scales), _ptr(out),
                                   pw.N, x_rot.numel(), _ptr(ws), ws.numel(), _stream(dev)),
               "pq1_gemv_packed")
    return out


def pq1_rotate_gemv_packed(x: torch.Tensor, signs: torch.Tensor, pw: PackedWeights, perm=None,
                           out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y = W WHT_1024(signs * P x) / 32 in one launch, W given as PackedWeights
    (f16 scales: pq1_rotate_gemv_packed_ex)."""
    if pw.scale_dtype != "f32":
        return pq1_rotate_gemv_packed_ex(x, signs, pw, perm, out)
    _need(x, "x", (torch.float32,))
    dev = x.device
    _need(signs, "signs", (torch.float32,), dev)
    _need_packed(pw, dev)
    _need_numel(x, "x", pw.K)
    _need_numel(signs, "signs", pw.K)
    if out is None:
        out = torch.empty(pw.N, dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), dev)
        _need_numel(out, "out", pw.N)
    lib = load_library()
    with torch.cuda.device(dev):
        ws = gemv_workspace(pw.N, pw.K, dev)
        _check(lib.pq1_rotate_gemv_packed(_ptr(x), _ptr(signs), _perm(perm), _ptr(pw.bits),
                                          _ptr(pw.scales), _ptr(out), pw.N, x.numel(), _ptr(ws),
                                          ws.numel(), _stream(dev)), "pq1_rotate_gemv_packed")
    return out


def pq1_gemv_packed_ex(x_rot: torch.Tensor, pw: PackedWeights,
                       out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pq1_gemv_packed for packed weights of either scale storage type."""
    _need(x_rot, "x_rot", (torch.float32,))
    dev = x_rot.device
    _need_packed(pw, dev)
    _need_numel(x_rot, "x_rot", pw.K)
    if out is None:
        out = torch.empty(pw.N, dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), dev)
        _need_numel(out, "out", pw.N)
    lib = load_library()
    with torch.cuda.device(dev):
        ws = gemv_workspace(pw.N, pw.K, dev)
        _check(lib.pq1_gemv_packed_ex(_ptr(x_rot), _ptr(pw.bits), _ptr(pw.scales),
                                      _scale_code(pw.scale_dtype), _ptr(out), pw.N, x_rot.numel(),
                                      _ptr(ws), ws.numel(), _stream(dev)), "pq1_gemv_packed_ex")
    return out


def pq1_rotate_gemv_packed_ex(x: torch.Tensor, signs: torch.Tensor, pw: PackedWeights, perm=None,
                              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pq1_rotate_gemv_packed for packed weights of either scale storage type."""
    _need(x, "x", (torch.float32,))
    dev = x.device
    _need(signs, "signs", (torch.float32,), dev)
    _need_packed(pw, dev)
    _need_numel(x, "x", pw.K)
    _need_numel(signs, "signs", pw.K)
    if out is None:
        out = torch.empty(pw.N, dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), dev)
        _need_numel(out, "out", pw.N)
    lib = load_library()
    with torch.cuda.device(dev):
        ws = gemv_workspace(pw.N, pw.K, dev)
        _check(lib.pq1_rotate_gemv_packed_ex(_ptr(x), _ptr(signs), _perm(perm), _ptr(pw.bits),
                                             _ptr(pw.scales), _scale_code(pw.scale_dtype),
                                             _ptr(out), pw.N, x.numel(), _ptr(ws), ws.numel(),
                                             _stream(dev)), "pq1_rotate_gemv_packed_ex")
    return out


def pq1_rotate_gemv_packed_noalloc(x: torch.Tensor, signs: torch.Tensor, pw: PackedWeights,
                                   perm=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """pq1_rotate_gemv_packed_ex with the library's own counter region: no
    workspace.  With `out` given the call allocates nothing (include/pq1.h)."""
    _need(x, "x", (torch.float32,))
    dev = x.device
    _need(signs, "signs", (torch.float32,), dev)
    _need_packed(pw, dev)
    _need_numel(x, "x", pw.K)
    _need_numel(signs, "signs", pw.K)
    if out is None:
        out = torch.empty(pw.N, dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), dev)
        _need_numel(out, "out", pw.N)
    lib = load_library()
    with torch.cuda.device(dev):
        _check(lib.pq1_rotate_gemv_packed_noalloc(_ptr(x), _ptr(signs), _perm(perm), _ptr(pw.bits),
                                                  _ptr(pw.scales), _scale_code(pw.scale_dtype),
                                                  _ptr(out), pw.N, x.numel(), _stream(dev)),
               "pq1_rotate_gemv_packed_noalloc")
    return out


def pq1_gemm_ex(x_rot_bf16: torch.Tensor, w_bits: torch.Tensor, scales: torch.Tensor,
                out: Optional[torch.Tensor] = None, gemm_order: bool = False) -> torch.Tensor:
    """Y = X W^T for a [M][K] bf16 activation block; fp32 [M][N] result.

    gemm_order=True: X is in the GEMM K order (pq1_rotate(..., gemm_order=True),
    x_layout PQ1_X_GEMM_ORDER); else row-major (PQ1_X_ROW_MAJOR)."""
    _need(x_rot_bf16, "x_rot_bf16", (torch.bfloat16, torch.int16, torch.uint16))
    dev = x_rot_bf16.device
    _need(w_bits, "w_bits", _WORD_DTYPES, dev)
    _need(scales, "scales", (torch.float32,), dev)
    if x_rot_bf16.dim() != 2:
        raise ValueError("x_rot_bf16 must be 2-D, [M][K]")
    M, K = x_rot_bf16.shape
    N = _need_weights(w_bits, scales, K, "pq1_gemm")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float32, device=dev)
    else:
        _need(out, "out", (torch.float32,), dev)
        _need_numel(out, "out", M * N)
    lib = load_library()
    with torch.cuda.device(dev):
        if gemm_order:
            code = lib.pq1_gemm_ex(_ptr(x_rot_bf16), _ptr(w_bits), _ptr(scales), _ptr(out), M, N,
                                   K, PQ1_X_GEMM_ORDER, _stream(dev))
        else:
            code = lib.pq1_gemm(_ptr(x_rot_bf16), _ptr(w_bits), _ptr(scales), _ptr(out), M, N, K,
                                _stream(dev))
        _check(code, "pq1_gemm_ex" if gemm_order else "pq1_gemm")
    return out


def pq1_gemm(x_rot_bf16: torch.Tensor, w_bits: torch.Tensor, scales: torch.Tensor,
             out: Optional[torch.Tensor] = None, gemm_order: bool = False) -> torch.Tensor:
    """Y = X W^T for a row-major [M][K] bf16 activation block (pq1_gemm);
    gemm_order=True forwards to pq1_gemm_ex with X in the GEMM K order."""
    return pq1_gemm_ex(x_rot_bf16, w_bits, scales, out, gemm_order)


def pq1_status_str(code: int) -> str:
    return load_library().pq1_status_str(int(code)).decode()


def pq1_abi_version() -> int:
    return int(load_library().pq1_abi_version())


def pq1_gemv_workspace_bytes(N: int, K: int) -> int:
    return int(load_library().pq1_gemv_workspace_bytes(int(N), int(K)))


# ----------------------------------------------------------------------------
# Attention layer: rotation by positions, the paged cache, attention over it
# ----------------------------------------------------------------------------
_TYPE_CODE = {torch.float32: PQ1_F32, torch.bfloat16: PQ1_BF16, torch.float16: PQ1_F16}
_FLOATS = tuple(_TYPE_CODE)
_PAIRINGS = {"halves": PQ1_ROPE_HALVES, "adjacent": PQ1_ROPE_ADJACENT}


# These calls are small and frequent (one decoded token: three of them a
# layer), so their path through Python is kept short: addresses go as plain
# integers, the stream comes from torch's raw accessor (0.1 us; a Stream object
# takes 2), and what a Rope or a KVCache can check is checked when it is made.
# A result is made like its input, in plain order (1.3 us; by its sizes 2.1).
# A torch without GPU support has no such accessors; it has no tensors either
# that would get as far as their use.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None)
_capturing = getattr(torch._C, "_cuda_isCurrentStreamCapturing", None)
_plain = torch.contiguous_format


def _refuse(t, name: str, dtypes, dev, shape=None):
    """Raise what is wrong with an argument."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU (no CPU path exists)")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must have dtype in {dtypes}, got {t.dtype}")
    if shape is not None:
        if t.shape != shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
        raise ValueError(f"{name} must be contiguous")
    if t.dim() != 3:
        raise ValueError(f"{name} must be 3-D, [tokens][heads][dim]")
    raise ValueError(f"{name}: the elements of a head must be contiguous")


def _need_heads(t: torch.Tensor, name: str, dtypes, dev=None):
    """A [tokens][heads][dim] tensor with contiguous head vectors: the
    library's view of it, and its shape."""
    try:
        dt, size = t.dtype, t.shape
        ts, hs, ds = t.stride()
        if dt not in dtypes or (not t.is_cuda if dev is None else t.device != dev) or (
                ds != 1 and size[2] != 1):
            _refuse(t, name, dtypes, dev)
    except (AttributeError, ValueError):  # no tensor, or not of three axes
        _refuse(t, name, dtypes, dev)
    # the stride of an axis of length one says nothing
    return Pq1Heads(t.data_ptr(), _TYPE_CODE[dt], ts if size[0] > 1 else 0,
                    hs if size[1] > 1 else 0), size


def _need_vector(t: torch.Tensor, name: str, dtype: torch.dtype, dev, shape) -> int:
    """The address of a contiguous tensor of this type and shape on dev."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != dev \
            or t.shape != shape or not t.is_contiguous():
        _refuse(t, name, (dtype,), dev, shape)
    return t.data_ptr()


def _too_many(size, name: str):
    raise ValueError(f"{name} has shape {tuple(size)}: heads and dim are 32-bit numbers")


def _same(size, expected, name: str):
    if size != expected:
        raise ValueError(f"{name} has shape {tuple(size)}, expected {tuple(expected)}")


def _launch(dev: torch.device, where: str, fn, *args):
    """fn(*args, current stream of dev) with dev current."""
    index = dev.index
    if _current_device() == index:
        code = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            code = fn(*args, _raw_stream(index))
    if code != PQ1_OK:
        _check(code, where)


def rope_frequencies(rot: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """The [rot / 2] fp64 frequencies base^(-2i / rot), radians per position."""
    i = torch.arange(int(rot) // 2, dtype=torch.float64, device=device)
    return torch.exp(i * (-2.0 * math.log(base) / int(rot)))


class Rope:
    """A rotation by positions, made once and used by every call: the first
    `rot` elements of a head turn, `sections` gives the pairs that each
    position axis owns (include/pq1.h, pq1_rope_spec).

    freqs  [rot / 2] fp64 on the GPU, radians per position (rope_frequencies,
           or any scaled variant of them).
    """

    def __init__(self, rot: int, sections: Optional[Sequence[int]] = None, *,
                 freqs: torch.Tensor, pairing: str = "halves", interleaved: bool = False):
        _need(freqs, "freqs", (torch.float64,))
        rot = int(rot)
        if rot < 2 or rot % 2 != 0 or rot >> 31:
            raise Pq1Error(2, "Rope", f"rot must be even, at least 2 and below 2^31, got {rot}")
        _need_numel(freqs, "freqs", rot // 2)
        sections = [rot // 2] if sections is None else [int(s) for s in sections]
        if not 1 <= len(sections) <= 4 or min(sections) < 0 or sum(sections) != rot // 2:
            raise Pq1Error(2, "Rope", f"one to four sections of together {rot // 2} pairs, "
                                      f"got {sections}")
        if pairing not in _PAIRINGS:
            raise Pq1Error(8, "Rope", f"unknown pairing {pairing!r} (halves or adjacent)")
        self.rot, self.sections, self.axes = rot, sections, len(sections)
        self._freqs_tensor = freqs
        padded = (sections + [0, 0, 0])[:4]
        self._spec = tuple(
            Pq1RopeSpec(rot, len(sections), (ctypes.c_int32 * 4)(*padded), int(bool(interleaved)),
                        _PAIRINGS[pairing], inverse) for inverse in (0, 1))

        self._device, self._freqs = freqs.device, freqs.data_ptr()

    @property
    def freqs(self) -> torch.Tensor:
        """The tensor given; its address went into the rotation, so another one
        needs another Rope."""
        return self._freqs_tensor

    def _need_positions(self, positions: torch.Tensor, T: int, dev) -> int:
        if self._device != dev:
            raise ValueError(f"the rotation's freqs are on {self._device}, expected {dev}")
        if self.axes == 1 and isinstance(positions, torch.Tensor) and positions.dim() == 1:
            return _need_vector(positions, "positions", torch.int32, dev, (T,))
        return _need_vector(positions, "positions", torch.int32, dev, (self.axes, T))


def pq1_rope(x: torch.Tensor, positions: torch.Tensor, rope: Rope,
             out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
             inverse: bool = False) -> torch.Tensor:
    """x [T][H][D] rotated by positions ([axes][T] int32, or [T] for one axis).

    x may be a slice (contiguous heads); out may be x itself.  inverse=True
    turns back, which is also the gradient of the forward call (like all calls
    here it is not recorded by autograd: results do not require a gradient)."""
    xv, size = _need_heads(x, "x", _FLOATS)
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    dev = x.device
    T, H, D = size
    if H >> 31 or D >> 31:
        _too_many(size, "x")
    pos = rope._need_positions(positions, T, dev)
    if out is None:
        dt = x.dtype if out_dtype is None else out_dtype
        if dt not in _TYPE_CODE:
            raise TypeError(f"out_dtype must be in {_FLOATS}")
        out = torch.empty_like(x, dtype=dt, memory_format=_plain)
        yv = Pq1Heads(out.data_ptr(), _TYPE_CODE[dt], H * D, D)
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out has dtype {out.dtype}, out_dtype is {out_dtype}")
        yv, out_size = _need_heads(out, "out", _FLOATS, dev)
        _same(out_size, size, "out")
    _launch(dev, "pq1_rope", (_lib or load_library()).pq1_rope, xv, yv, pos, rope._freqs,
            rope._spec[1 if inverse else 0], T, H, D)
    return out


class KVCache:
    """A paged key/value cache over two tensors of the caller's,
    [pages][heads][page_size][dim], bf16 or f16 (include/pq1.h, pq1_kv_cache)."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        _need(k, "k", (torch.bfloat16, torch.float16))
        _need(v, "v", (k.dtype,), k.device)
        if k.dim() != 4:
            raise ValueError("k must be 4-D, [pages][heads][page_size][dim]")
        _same(v.shape, k.shape, "v")
        if max(k.shape[1:]) >> 31:
            raise ValueError(f"k has shape {tuple(k.shape)}: heads, page_size and dim are 32-bit "
                             f"numbers")
        self._k, self._v = k, v
        self.pages, self.heads, self.page_size, self.dim = (int(n) for n in k.shape)
        self.dtype, self.device = k.dtype, k.device
        self._inputs = (torch.float32, k.dtype)
        self._struct = Pq1KvCache(k.data_ptr(), v.data_ptr(), _TYPE_CODE[k.dtype],
                                  self.page_size, self.pages, self.heads, self.dim)

    # The tensors given; their addresses went into the struct, so other ones
    # need another KVCache.
    @property
    def k(self) -> torch.Tensor:
        return self._k

    @property
    def v(self) -> torch.Tensor:
        return self._v

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, dim: int,
              dtype: torch.dtype = torch.bfloat16, device=None) -> "KVCache":
        device = torch.device("cuda") if device is None else device
        shape = (int(pages), int(heads), int(page_size), int(dim))
        return cls(torch.empty(shape, dtype=dtype, device=device),
                   torch.empty(shape, dtype=dtype, device=device))


class HeadNorm:
    """The norms of an append's keys and queries: each head over the root of its
    mean square (plus eps) and times a weight, [dim] fp32 on the GPU.  A weight
    that is None leaves its heads as they are."""

    def __init__(self, k_weight: Optional[torch.Tensor], q_weight: Optional[torch.Tensor] = None, *,
                 eps: float = 1e-6):
        given = [w for w in (k_weight, q_weight) if w is not None]
        if not given:
            raise ValueError("a norm needs a weight")
        for w in given:
            _need(w, "weight", (torch.float32,), given[0].device)
            if w.shape != given[0].shape or w.dim() != 1:
                raise ValueError(f"weights must be 1-D, [dim], got {[tuple(w.shape) for w in given]}")
        _need_eps(eps, "HeadNorm")
        self._k_weight, self._q_weight, self._eps = k_weight, q_weight, float(eps)
        self._device, self._dim = given[0].device, given[0].numel()
        self._struct = Pq1HeadNorm(_ptr(q_weight), _ptr(k_weight), self._eps)

    # What was given; it went into the struct, the tensors as addresses, so other
    # ones need another HeadNorm.
    @property
    def eps(self) -> float:
        return self._eps

    @property
    def k_weight(self) -> Optional[torch.Tensor]:
        return self._k_weight

    @property
    def q_weight(self) -> Optional[torch.Tensor]:
        return self._q_weight

    def _need_fit(self, dim: int, dev):
        if self._device != dev:
            raise ValueError(f"the norm's weights are on {self._device}, expected {dev}")
        if self._dim != dim:
            raise ValueError(f"the norm's weights have {self._dim} elements, expected {dim}")
        return self._struct


def _need_eps(eps: float, where: str) -> float:
    eps = float(eps)
    # as the C call sees it
    if not 2.0 ** -150 < eps < 3.4028236e38:
        raise Pq1Error(8, where, f"eps must be above 0 and finite in fp32, got {eps}")
    return eps


def _append(where: str, fn, cache, k, v, slots, positions, rope, q, q_out, norm):
    """Both appends: a launch of fn with the views of their arguments."""
    dev, dt = cache.device, cache.dtype
    kv, size = _need_heads(k, "k", cache._inputs, dev)
    T = size[0]
    _same(size, (T, cache.heads, cache.dim), "k")
    kind = (k.dtype,)
    vv, v_size = _need_heads(v, "v", kind, dev)
    _same(v_size, size, "v")
    at = _need_vector(slots, "slots", torch.int64, dev, (T,))
    spec = pos = freqs = None
    if rope is not None:
        if not isinstance(rope, Rope):
            raise TypeError("rope must be a Rope")
        if positions is None:
            raise ValueError("a rotation needs positions")
        pos = rope._need_positions(positions, T, dev)
        spec, freqs = rope._spec[0], rope._freqs
    qv = ov = None
    Hq = 0
    if q is not None:
        qv, size = _need_heads(q, "q", kind, dev)
        Hq = size[1]
        _same(size, (T, Hq, cache.dim), "q")
        if Hq >> 31:
            _too_many(size, "q")
        if q_out is None:
            q_out = torch.empty_like(q, dtype=dt, memory_format=_plain)
            ov = Pq1Heads(q_out.data_ptr(), _TYPE_CODE[dt], Hq * cache.dim, cache.dim)
        else:
            ov, out_size = _need_heads(q_out, "q_out", (dt,), dev)
            _same(out_size, size, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if fn is None:  # the 16-bit append has a call of its own without norms
        _launch(dev, where, (_lib or load_library()).pq1_kv_append, kv, vv, at, qv, ov, Hq, pos,
                freqs, spec, cache._struct, T)
        return q_out
    ns = None
    if norm is not None:
        if not isinstance(norm, HeadNorm):
            raise TypeError("norm must be a HeadNorm")
        ns = norm._need_fit(cache.dim, dev)
    _launch(dev, where, fn, kv, vv, at, qv, ov, Hq, pos, freqs, spec, ns, cache._struct, T)
    return q_out


def pq1_kv_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                  positions: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
                  q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                  norm: Optional[HeadNorm] = None) -> Optional[torch.Tensor]:
    """Store k and v ([T][heads][dim], slices allowed, fp32 or the cache's
    type) at slots ([T] int64, page * page_size + row; -1 is padding), keys
    rotated by `rope`; with q, the rotated queries are returned in the cache's
    type.  `norm` (pq1_kv_append_ex) comes before the rotation.  One launch."""
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    fn = None if norm is None else (_lib or load_library()).pq1_kv_append_ex
    return _append("pq1_kv_append" if norm is None else "pq1_kv_append_ex", fn, cache, k, v, slots,
                   positions, rope, q, q_out, norm)


class KV4Cache:
    """A paged key/value cache of 4-bit numbers over four uint8 tensors of the
    caller's: codes [pages][heads][page_size][dim / 2] and scales
    [pages][heads][page_size][dim / 32] (include/pq1.h, pq1_kv4_cache).  dtype,
    bf16 or f16, is the type of the queries and the one values are read in."""

    def __init__(self, k: torch.Tensor, k_scale: torch.Tensor, v: torch.Tensor,
                 v_scale: torch.Tensor, dtype: torch.dtype = torch.bfloat16):
        if dtype not in (torch.bfloat16, torch.float16):
            raise TypeError(f"dtype must be torch.bfloat16 or torch.float16, got {dtype}")
        _need(k, "k", (torch.uint8,))
        for t, name in ((k_scale, "k_scale"), (v, "v"), (v_scale, "v_scale")):
            _need(t, name, (torch.uint8,), k.device)
        if k.dim() != 4:
            raise ValueError("k must be 4-D, [pages][heads][page_size][dim / 2]")
        if k.shape[3] % 16 != 0:
            raise ValueError(f"k has shape {tuple(k.shape)}: dim must be a multiple of 32")
        if max(k.shape[1:]) >> 30:
            raise ValueError(f"k has shape {tuple(k.shape)}: heads, page_size and dim are 32-bit "
                             f"numbers")
        _same(v.shape, k.shape, "v")
        scales = torch.Size((*k.shape[:3], k.shape[3] // 16))
        _same(k_scale.shape, scales, "k_scale")
        _same(v_scale.shape, scales, "v_scale")
        self._k, self._k_scale, self._v, self._v_scale = k, k_scale, v, v_scale
        self.pages, self.heads, self.page_size = (int(n) for n in k.shape[:3])
        self.dim = 2 * int(k.shape[3])
        self.dtype, self.device = dtype, k.device
        self._inputs = (torch.float32, dtype)
        self._struct = Pq1Kv4Cache(k.data_ptr(), k_scale.data_ptr(), v.data_ptr(),
                                   v_scale.data_ptr(), _TYPE_CODE[dtype], self.page_size,
                                   self.pages, self.heads, self.dim)

    # The tensors given; their addresses went into the struct, so other ones
    # need another KV4Cache.
    @property
    def k(self) -> torch.Tensor:
        return self._k

    @property
    def k_scale(self) -> torch.Tensor:
        return self._k_scale

    @property
    def v(self) -> torch.Tensor:
        return self._v

    @property
    def v_scale(self) -> torch.Tensor:
        return self._v_scale

    @classmethod
    def empty(cls, pages: int, page_size: int, heads: int, dim: int,
              dtype: torch.dtype = torch.bfloat16, device=None) -> "KV4Cache":
        device = torch.device("cuda") if device is None else device
        if int(dim) % 32 != 0:
            raise ValueError(f"dim must be a multiple of 32, got {dim}")
        shape = (int(pages), int(heads), int(page_size))
        make = lambda n: torch.empty((*shape, n), dtype=torch.uint8, device=device)
        return cls(make(int(dim) // 2), make(int(dim) // 32), make(int(dim) // 2),
                   make(int(dim) // 32), dtype)


def pq1_kv4_append(cache: KV4Cache, k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                   positions: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
                   q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None,
                   norm: Optional[HeadNorm] = None) -> Optional[torch.Tensor]:
    """pq1_kv_append into a 4-bit cache: keys (after norm and rotation) and values
    become codes and scales (include/pq1.h); queries are returned in the cache's
    dtype.  One launch."""
    if not isinstance(cache, KV4Cache):
        raise TypeError("cache must be a KV4Cache")
    return _append("pq1_kv4_append", (_lib or load_library()).pq1_kv4_append, cache, k, v, slots,
                   positions, rope, q, q_out, norm)


def pq1_kv4_read(cache: KV4Cache, slots: torch.Tensor, k_out: Optional[torch.Tensor] = None,
                 v_out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None):
    """(keys, values) of rows slots ([T] int64) of a 4-bit cache, [T][heads][dim]
    each, in out_dtype (the cache's unless given).  Tensors may be given for both
    or for one; then that one alone is read, and None is in the other's place.
    Slots may repeat; one outside the cache gives zeros."""
    if not isinstance(cache, KV4Cache):
        raise TypeError("cache must be a KV4Cache")
    dev = cache.device
    T = slots.shape[0] if isinstance(slots, torch.Tensor) and slots.dim() == 1 else -1
    at = _need_vector(slots, "slots", torch.int64, dev, (T,))
    shape = (T, cache.heads, cache.dim)
    if k_out is None and v_out is None:
        dt = cache.dtype if out_dtype is None else out_dtype
        if dt not in _TYPE_CODE:
            raise TypeError(f"out_dtype must be in {_FLOATS}")
        k_out = torch.empty(shape, dtype=dt, device=dev)
        v_out = torch.empty(shape, dtype=dt, device=dev)
        kv, vv = (Pq1Heads(t.data_ptr(), _TYPE_CODE[dt], shape[1] * shape[2], shape[2])
                  for t in (k_out, v_out))
    else:
        views, kinds = [], _FLOATS if out_dtype is None else (out_dtype,)
        for t, name in ((k_out, "k_out"), (v_out, "v_out")):
            if t is None:
                views.append(None)
                continue
            view, size = _need_heads(t, name, kinds, dev)
            _same(size, shape, name)
            views.append(view)
            kinds = (t.dtype,)
        kv, vv = views
    _launch(dev, "pq1_kv4_read", (_lib or load_library()).pq1_kv4_read, cache._struct, at, kv, vv, T)
    return k_out, v_out


def _norm_arguments(x, weight, positions, rope, eps, where):
    """What both norm calls check: view and shape of x, weight's address, eps, and
    the rotation's positions, frequencies and specs (None without one)."""
    xv, size = _need_heads(x, "x", _FLOATS)
    dev = x.device
    if size[1] >> 31 or size[2] >> 31:
        _too_many(size, "x")
    w = _need_vector(weight, "weight", torch.float32, dev, (size[2],))
    eps = _need_eps(eps, where)
    if rope is None:
        return xv, size, dev, w, eps, None, None, (None, None)
    if not isinstance(rope, Rope):
        raise TypeError("rope must be a Rope")
    if positions is None:
        raise ValueError("a rotation needs positions")
    return xv, size, dev, w, eps, rope._need_positions(positions, size[0], dev), rope._freqs, rope._spec


def _out_like(x, size, out, out_dtype, dev, name):
    """The result given, or one made like x: the tensor and its view."""
    if out is None:
        dt = x.dtype if out_dtype is None else out_dtype
        if dt not in _TYPE_CODE:
            raise TypeError(f"out_dtype must be in {_FLOATS}")
        out = torch.empty_like(x, dtype=dt, memory_format=_plain)
        return out, Pq1Heads(out.data_ptr(), _TYPE_CODE[dt], size[1] * size[2], size[2])
    if out_dtype is not None and out.dtype != out_dtype:
        raise TypeError(f"{name} has dtype {out.dtype}, out_dtype is {out_dtype}")
    view, out_size = _need_heads(out, name, _FLOATS, dev)
    _same(out_size, size, name)
    return out, view


def pq1_norm_rope(x: torch.Tensor, weight: torch.Tensor, positions: Optional[torch.Tensor] = None,
                  rope: Optional[Rope] = None, eps: float = 1e-6,
                  out: Optional[torch.Tensor] = None, out_dtype: Optional[torch.dtype] = None,
                  inverse: bool = False) -> torch.Tensor:
    """Each head of x [T][H][D] over the root of its mean square (plus eps), times
    weight ([D] fp32), then rotated as by pq1_rope (rope None: not).  x may be a
    slice (contiguous heads); out may be x itself.  Not recorded by autograd:
    pq1_norm_rope_grad is the gradient."""
    xv, size, dev, w, eps, pos, freqs, spec = _norm_arguments(x, weight, positions, rope, eps,
                                                              "pq1_norm_rope")
    out, yv = _out_like(x, size, out, out_dtype, dev, "out")
    _launch(dev, "pq1_norm_rope", (_lib or load_library()).pq1_norm_rope, xv, yv, w, eps, pos, freqs,
            spec[1 if inverse else 0], *size)
    return out


def pq1_norm_rope_grad(grad: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
                       positions: Optional[torch.Tensor] = None, rope: Optional[Rope] = None,
                       eps: float = 1e-6, dx: Optional[torch.Tensor] = None,
                       weight_grad: bool = True, inverse: bool = False):
    """(dx, dweight) of pq1_norm_rope called with the same arguments, for a
    gradient `grad` of its result: dx of x's type (new unless given; x or grad
    itself may be), dweight [D] fp32, or None with weight_grad False."""
    xv, size, dev, w, eps, pos, freqs, spec = _norm_arguments(x, weight, positions, rope, eps,
                                                              "pq1_norm_rope_grad")
    gv, g_size = _need_heads(grad, "grad", _FLOATS, dev)
    _same(g_size, size, "grad")
    dx, dv = _out_like(x, size, dx, x.dtype, dev, "dx")
    T, H, D = size
    lib = _lib or load_library()
    dw = torch.empty_like(weight) if weight_grad else None
    args = (gv, xv, dv, w, dw.data_ptr() if weight_grad else None, eps, pos, freqs,
            spec[1 if inverse else 0], T, H, D)
    call = (dev, "pq1_norm_rope_grad", lib.pq1_norm_rope_grad, args,
            lib.pq1_norm_rope_grad_workspace_bytes, (T if weight_grad else 0, D))
    if _current_device() == dev.index:
        _with_workspace(*call)
    else:
        with torch.cuda.device(dev):
            _with_workspace(*call)
    return dx, dw


# Attention workspaces, one per (device, stream) and grown on demand: (tensor,
# address, bytes).  Kept apart from the GEMV's, whose counter region must stay
# as its calls leave it.  A call captured into a graph takes its own from the
# graph's memory instead: graphs captured on one stream may be replayed on
# several, and beside calls that are not captured.
# A call may be two launches, parts and their join: _attn_lock keeps those of
# two threads on one stream from coming between one another.
_attn_ws = {}
_attn_lock = threading.Lock()
_NO_WS = (None, None, 0)


def _grow_attention_workspace(key, need: int, device: torch.device):
    with _ws_lock:
        old = _attn_ws.get(key, _NO_WS)
        if old[2] < need:
            if old[0] is not None:
                # a graph captured earlier may still hold the old buffer's address
                _ws_retired.append(old[0])
            t = torch.empty(max(need, 1 << 20), dtype=torch.uint8, device=device)
            old = _attn_ws[key] = (t, t.data_ptr(), t.numel())
        return old


def _hints_and_window(max_q: int, max_kv: int, window: int):
    """The three as numbers of the C call's widths (64, 64 and 32 bits), which
    would take any others by their low bits: past all lengths, or below zero,
    every number says the same."""
    hint = lambda n: max(-1, min(n, 1 << 62))
    return hint(max_q), hint(max_kv), max(-1, min(window, 0x7fffffff))


def _attention_arguments(q, cache, page_table, cu_q, kv_len, max_q, max_kv, scale, causal, window,
                         out, out_dtype):
    """What the attention calls check; their result and the C calls' arguments up to
    the window."""
    dev, dt = cache.device, cache.dtype
    qv, size = _need_heads(q, "q", (dt,), dev)
    T, Hq, D = size
    if D != cache.dim:
        raise ValueError(f"q has shape {tuple(size)}, expected {(T, Hq, cache.dim)}")
    if Hq >> 31:
        _too_many(size, "q")
    if not isinstance(page_table, torch.Tensor):
        raise TypeError("page_table must be a torch.Tensor")
    if page_table.dim() != 2:
        raise ValueError("page_table must be 2-D, [sequences][pages]")
    B, max_pages = page_table.shape
    table = _need_vector(page_table, "page_table", torch.int32, dev, (B, max_pages))
    cu = _need_vector(cu_q, "cu_q", torch.int32, dev, (B + 1,))
    lens = _need_vector(kv_len, "kv_len", torch.int32, dev, (B,))
    if out is None:
        if out_dtype is not None:
            if out_dtype != dt and out_dtype != torch.float32:
                raise TypeError(f"out_dtype must be {dt} or torch.float32")
            dt = out_dtype
        out = torch.empty_like(q, dtype=dt, memory_format=_plain)
        ov = Pq1Heads(out.data_ptr(), _TYPE_CODE[dt], Hq * D, D)
    else:
        if out_dtype is not None and out.dtype != out_dtype:
            raise TypeError(f"out has dtype {out.dtype}, out_dtype is {out_dtype}")
        ov, out_size = _need_heads(out, "out", (dt, torch.float32), dev)
        _same(out_size, size, "out")
    max_q, max_kv, window = int(max_q), int(max_kv), int(window)
    if max_q >> 62 or max_kv >> 62 or window >> 31:
        max_q, max_kv, window = _hints_and_window(max_q, max_kv, window)
    return out, (qv, ov, cache._struct, table, max_pages, cu, lens, B, T, Hq, max_q, max_kv,
                 D ** -0.5 if scale is None else float(scale), 1 if causal else 0, window)


def pq1_paged_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor,
                        cu_q: torch.Tensor, kv_len: torch.Tensor, max_q: int, max_kv: int,
                        scale: Optional[float] = None, causal: bool = True, window: int = 0,
                        out: Optional[torch.Tensor] = None,
                        out_dtype: Optional[torch.dtype] = None, sinks: int = 0) -> torch.Tensor:
    """Attention of the new tokens q [T][Hq][dim] of B sequences over the
    cache (include/pq1.h, pq1_paged_attention).

    page_table [B][max_pages], cu_q [B+1] and kv_len [B] are int32 on the GPU;
    max_q and max_kv are the longest chunk and kv_len, known on the host.
    scale defaults to dim^-0.5.  With a window the first `sinks` keys of a sequence
    stay visible (pq1_paged_attention_ex).  out (of q's type, or fp32) is new unless
    given; rows that no sequence owns keep what they held.  The workspace is the
    binding's: one for each stream, and one in each graph's own memory."""
    if not isinstance(cache, KVCache):
        raise TypeError("cache must be a KVCache")
    out, args = _attention_arguments(q, cache, page_table, cu_q, kv_len, max_q, max_kv, scale,
                                     causal, window, out, out_dtype)
    lib = _lib or load_library()
    dev = cache.device
    if sinks:
        _attend_window(dev, "pq1_paged_attention_ex", lib.pq1_paged_attention_ex,
                       lib.pq1_paged_attention_ex_workspace_bytes, cache, args, sinks)
    elif _current_device() == dev.index:
        _attend(lib, dev, cache.heads, args)
    else:
        with torch.cuda.device(dev):
            _attend(lib, dev, cache.heads, args)
    return out


def pq1_kv4_attention(q: torch.Tensor, cache: KV4Cache, page_table: torch.Tensor,
                      cu_q: torch.Tensor, kv_len: torch.Tensor, max_q: int, max_kv: int,
                      scale: Optional[float] = None, causal: bool = True, window: int = 0,
                      out: Optional[torch.Tensor] = None,
                      out_dtype: Optional[torch.dtype] = None, sinks: int = 0) -> torch.Tensor:
    """pq1_paged_attention over a 4-bit cache, q of its dtype: the same result as
    over a cache that holds the values of pq1_kv4_read."""
    if not isinstance(cache, KV4Cache):
        raise TypeError("cache must be a KV4Cache")
    out, args = _attention_arguments(q, cache, page_table, cu_q, kv_len, max_q, max_kv, scale,
                                     causal, window, out, out_dtype)
    lib = _lib or load_library()
    _attend_window(cache.device, "pq1_kv4_attention", lib.pq1_kv4_attention,
                   lib.pq1_kv4_attention_workspace_bytes, cache, args, sinks)
    return out


def _attend_window(dev, where: str, fn, need_of, cache, args, sinks: int) -> None:
    sinks = int(sinks)
    if sinks >> 31:  # past all lengths, or below zero, every number says the same
        sinks = max(-1, min(sinks, 0x7fffffff))
    args = (*args, sinks)
    B, T, Hq, max_q, max_kv = args[7:12]
    sizes = (B, T, Hq, cache.heads, cache.dim, max_q, max_kv, args[14], sinks)
    if _current_device() == dev.index:
        _with_workspace(dev, where, fn, args, need_of, sizes)
    else:
        with torch.cuda.device(dev):
            _with_workspace(dev, where, fn, args, need_of, sizes)


def _attend(lib, dev, heads: int, args) -> None:
    _with_workspace(dev, "pq1_paged_attention", lib.pq1_paged_attention, args,
                    _attention_workspace_bytes, (lib, heads, args))


def _with_workspace(dev, where: str, fn, args, need_of, sizes) -> None:
    """The call with the stream's present workspace; only if the library
    refuses that is the size asked for (0.5 us a call)."""
    stream = _raw_stream(dev.index)
    if stream and _capturing():  # (the default stream cannot be captured)
        need = need_of(*sizes)
        ws = torch.empty(need, dtype=torch.uint8, device=dev) if need else None
        code = fn(*args, ws.data_ptr() if need else None, need, stream)
        if code != PQ1_OK:
            _check(code, where)
        return
    key = (dev.index, stream)
    with _attn_lock:
        ws = _attn_ws.get(key, _NO_WS)
        code = fn(*args, ws[1], ws[2], stream)
        if code == PQ1_OK:
            return
        if code in (1, 8):  # PQ1_ERR_NULL, PQ1_ERR_ARG: perhaps no workspace yet, or too small a one
            need = need_of(*sizes)
            if need > ws[2]:
                ws = _grow_attention_workspace(key, need, dev)
                code = fn(*args, ws[1], ws[2], stream)
    if code != PQ1_OK:
        _check(code, where)


def _attention_workspace_bytes(lib, heads: int, args) -> int:
    B, T, Hq, max_q, max_kv = args[7:12]
    return lib.pq1_paged_attention_workspace_bytes(B, T, Hq, heads, args[2].dim, max_q, max_kv)
