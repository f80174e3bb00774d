"""Python binding of the shape-adaptive GEMM library (``libsam.so``).

Argument marshalling only: every step of C = A·B runs in the library's HIP
kernels. PyTorch supplies device memory and the current stream; nothing here
computes a product, and there is no CPU fallback — if the library is missing
or the device is not gfx950 the call raises.

The C ABI is declared in ``include/sam.h``; the names here follow it without
the ``sam_`` prefix.
"""
from __future__ import annotations

import ctypes
import functools
import re
from pathlib import Path

import os

PKG = Path(__file__).resolve().parent
# SAM_LIBRARY may point at another build of the same library (A/B timing).
LIB_PATH = Path(os.environ.get("SAM_LIBRARY", PKG / "libsam.so"))
HEADER = PKG.parent / "include" / "sam.h"

F32, BF16, F16, MXFP8, MXFP4 = 0, 1, 2, 3, 4
DTYPES = {"f32": F32, "bf16": BF16, "f16": F16, "mxfp8": MXFP8, "mxfp4": MXFP4}
FP8_FORMATS = {"e4m3": 0, "e5m2": 1}
DTYPE_NAMES = {v: k for k, v in DTYPES.items()}

STATUS = {
    0: "SAM_OK", -1: "SAM_ERR_INVALID_ARG", -2: "SAM_ERR_MISALIGNED",
    -3: "SAM_ERR_WORKSPACE", -4: "SAM_ERR_UNSUPPORTED",
    -5: "SAM_ERR_UNSUPPORTED_DEVICE", -6: "SAM_ERR_LAUNCH", -7: "SAM_ERR_INTERNAL",
}


class SamError(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        self.name = STATUS.get(status, str(status))
        super().__init__(f"{self.name}: {detail}")


class SamPlan(ctypes.Structure):
    _fields_ = [
        ("struct_size", ctypes.c_uint32), ("variant_id", ctypes.c_int32),
        ("name", ctypes.c_char * 64), ("dtype", ctypes.c_int32),
        ("tile_m", ctypes.c_int32), ("tile_n", ctypes.c_int32), ("tile_k", ctypes.c_int32),
        ("waves_m", ctypes.c_int32), ("waves_n", ctypes.c_int32), ("mfma_m", ctypes.c_int32),
        ("split_k", ctypes.c_int32), ("group_m", ctypes.c_int32), ("xcd_remap", ctypes.c_int32),
        ("a_vector", ctypes.c_int32), ("b_vector", ctypes.c_int32),
        ("grid_wgs", ctypes.c_int64), ("workspace_bytes", ctypes.c_uint64),
        ("est_us", ctypes.c_double), ("raster_n", ctypes.c_int32), ("operand_swap", ctypes.c_int32),
        ("sk_dp_tiles", ctypes.c_int64), ("tuned", ctypes.c_int32),
    ]

    def as_dict(self) -> dict:
        d = {f: getattr(self, f) for f, _ in self._fields_}
        d["name"] = self.name.decode()
        return d


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library. Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not LIB_PATH.exists():
        raise ImportError(f"{LIB_PATH} is missing: run `python -m shape_adaptive_matrix_amd.build`")
    # torch ships its own HIP runtime under the same soname as the system one
    # libsam.so links. Whichever is loaded first serves the whole process, and
    # torch cannot initialise the GPU on the other; so when torch is present
    # it is loaded first and the library binds to its runtime.
    try:
        import torch  # noqa: F401
    except ImportError:
        pass
    L = ctypes.CDLL(str(LIB_PATH))
    i64, u64, vp, i32 = ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p, ctypes.c_int32
    P = ctypes.POINTER(SamPlan)
    sig = {
        "sam_gemm_plan": ([i64, i64, i64, ctypes.c_int, P], ctypes.c_int),
        "sam_gemm_f32": ([vp, vp, vp, i64, i64, i64, vp, u64, vp], ctypes.c_int),
        "sam_gemm_bf16": ([vp, vp, vp, i64, i64, i64, vp, u64, vp], ctypes.c_int),
        "sam_gemm_f16": ([vp, vp, vp, i64, i64, i64, vp, u64, vp], ctypes.c_int),
        "sam_variant_count": ([], i32),
        "sam_variant_info": ([i32, P], ctypes.c_int),
        "sam_variant_plan": ([i32, i64, i64, i64, ctypes.c_int, i32, P], ctypes.c_int),
        "sam_gemm_variant": ([i32, ctypes.c_int, i32, vp, vp, vp, i64, i64, i64, vp, u64, vp], ctypes.c_int),
        "sam_variant_plan_r": ([i32, i64, i64, i64, ctypes.c_int, i32, i32, P], ctypes.c_int),
        "sam_gemm_variant_r": ([i32, ctypes.c_int, i32, i32, vp, vp, vp, i64, i64, i64, vp, u64, vp], ctypes.c_int),
        "sam_gemm_plan_model": ([i64, i64, i64, ctypes.c_int, P], ctypes.c_int),
        "sam_gemm_ex": ([ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, i64, i64, ctypes.c_float, vp, i64, vp, i64,
                         ctypes.c_float, vp, i64, vp, u64, vp], ctypes.c_int),
        "sam_gemm_ex_workspace": ([ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, i64, i64, i64, i64, i64,
                                   ctypes.c_float, ctypes.c_float, ctypes.POINTER(ctypes.c_uint64)], ctypes.c_int),
        "sam_gemm_ex_variant": ([i32, i32, i32, ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, i64, i64,
                                 ctypes.c_float, vp, i64, vp, i64, ctypes.c_float, vp, i64, vp, u64, vp],
                                ctypes.c_int),
        "sam_gemm_ex_variant_workspace": ([i32, i32, i32, ctypes.c_int, ctypes.c_int, ctypes.c_int, i64, i64, i64,
                                           i64, i64, i64, ctypes.c_float, ctypes.c_float,
                                           ctypes.POINTER(ctypes.c_uint64)], ctypes.c_int),
        "sam_gemm_mxfp8": ([ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp, i64, i64, i64, vp, u64, vp],
                           ctypes.c_int),
        "sam_gemm_mxfp8_variant": ([i32, i32, ctypes.c_int, ctypes.c_int, vp, vp, vp, vp, vp, i64, i64, i64, vp,
                                    u64, vp], ctypes.c_int),
        "sam_gemm_mxfp4": ([vp, vp, vp, vp, vp, i64, i64, i64, vp, u64, vp], ctypes.c_int),
        "sam_gemm_mxfp4_variant": ([i32, i32, vp, vp, vp, vp, vp, i64, i64, i64, vp, u64, vp], ctypes.c_int),
        "sam_gemm_noalloc": ([ctypes.c_int, vp, vp, vp, i64, i64, i64, vp], ctypes.c_int),
        "sam_adapter_gemm": ([ctypes.c_int, ctypes.c_int, i64, i64, i64, i64, i64, vp, i64, vp, i64, vp, vp, vp, vp,
                              ctypes.c_int, vp, i64, vp, u64, vp], ctypes.c_int),
        "sam_adapter_gemm_workspace": ([ctypes.c_int, ctypes.c_int, i64, i64, i64, i64, i64, i64, i64,
                                        ctypes.POINTER(u64)], ctypes.c_int),
        "sam_adapter_backward": ([ctypes.c_int, ctypes.c_int, i64, i64, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp,
                                  vp, vp, vp, ctypes.c_int, vp, i64, vp, vp, vp, u64, vp], ctypes.c_int),
        "sam_adapter_backward_workspace": ([ctypes.c_int, ctypes.c_int, i64, i64, i64, i64, i64, i64, i64, i64, i32,
                                            i32, ctypes.POINTER(u64)], ctypes.c_int),
        "sam_distill_loss": ([ctypes.c_int, i64, i64, i64, vp, i64, ctypes.c_int, vp, vp, vp, ctypes.c_float, vp, vp,
                              vp], ctypes.c_int),
        "sam_distill_grad": ([ctypes.c_int, i64, i64, i64, vp, i64, vp, ctypes.c_int, vp, vp, vp, ctypes.c_float, vp,
                              i64, vp], ctypes.c_int),
        "sam_distill": ([ctypes.c_int, i64, i64, i64, vp, i64, ctypes.c_int, vp, vp, vp, ctypes.c_float, vp, vp, i64,
                         vp], ctypes.c_int),
        "sam_quantize_mxfp4": ([ctypes.c_int, ctypes.c_int, i64, i64, vp, i64, vp, vp, vp], ctypes.c_int),
        "sam_dequantize_mxfp4": ([ctypes.c_int, i64, i64, vp, vp, vp, i64, vp], ctypes.c_int),
        "sam_linear_mxfp4": ([ctypes.c_int, i64, i64, i64, vp, i64, vp, vp, ctypes.c_int, vp, i64, vp, u64, vp],
                             ctypes.c_int),
        "sam_linear_mxfp4_workspace": ([ctypes.c_int, ctypes.c_int, i64, i64, i64, ctypes.POINTER(u64)], ctypes.c_int),
        "sam_linear_mxfp4_backward": ([ctypes.c_int, i64, i64, i64, vp, i64, vp, vp, ctypes.c_int, vp, i64, vp, u64, vp],
                                      ctypes.c_int),
        "sam_linear_mxfp4_backward_workspace": ([ctypes.c_int, ctypes.c_int, i64, i64, i64, ctypes.POINTER(u64)],
                                                ctypes.c_int),
        "sam_linear_mxfp4_backward_workspace_strided": ([ctypes.c_int, ctypes.c_int, i64, i64, i64, i64, i64,
                                                         ctypes.POINTER(u64)], ctypes.c_int),
        "sam_token_logprobs": ([ctypes.c_int, i64, i64, i64, vp, i64, vp, ctypes.c_float, vp, vp, vp, vp, vp, vp, u64, vp],
                               ctypes.c_int),
        "sam_token_logprobs_workspace": ([ctypes.c_int, i64, i64, i64, ctypes.POINTER(u64)], ctypes.c_int),
        "sam_token_logprobs_grad": ([ctypes.c_int, i64, i64, vp, i64, vp, ctypes.c_float, vp, vp, vp, vp, vp, i64, vp],
                                    ctypes.c_int),
        "sam_device_check": ([], ctypes.c_int),
        "sam_status_string": ([ctypes.c_int], ctypes.c_char_p),
        "sam_last_error": ([], ctypes.c_char_p),
        "sam_build_info": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sig.items():
        f = getattr(L, name)
        f.argtypes = args
        f.restype = res
    _lib = L
    return L


def header_symbols() -> list[str]:
    """Function names declared in include/sam.h."""
    text = HEADER.read_text()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(sam_\w+)\s*\(", text)))


def _check(status: int):
    if status != 0:
        raise SamError(status, lib().sam_last_error().decode())


def _dt(dtype) -> int:
    if isinstance(dtype, int):
        return dtype
    return DTYPES[dtype]


# -- host-only queries ---------------------------------------------------------
def plan(M: int, N: int, K: int, dtype="f32") -> dict:
    p = SamPlan()
    _check(lib().sam_gemm_plan(M, N, K, _dt(dtype), ctypes.byref(p)))
    return p.as_dict()


def variant_count() -> int:
    return lib().sam_variant_count()


def variant_info(vid: int) -> dict:
    p = SamPlan()
    _check(lib().sam_variant_info(vid, ctypes.byref(p)))
    return p.as_dict()


def variant_plan(vid: int, M: int, N: int, K: int, dtype="f32", split_k: int = 0, raster: int = -1) -> dict:
    """Plan of a forced variant and split (0: its own choice, -1: stream-K)
    and raster order (-1: the cost model's choice, 0 M-major, 1 N-major)."""
    p = SamPlan()
    _check(lib().sam_variant_plan_r(vid, M, N, K, _dt(dtype), split_k, raster, ctypes.byref(p)))
    return p.as_dict()


def plan_model(M: int, N: int, K: int, dtype="f32") -> dict:
    """The cost model's own plan, ignoring the frozen table (host only)."""
    p = SamPlan()
    _check(lib().sam_gemm_plan_model(M, N, K, _dt(dtype), ctypes.byref(p)))
    return p.as_dict()


def build_info() -> str:
    return lib().sam_build_info().decode()


def device_check() -> None:
    _check(lib().sam_device_check())


def last_error() -> str:
    return lib().sam_last_error().decode()


# -- device calls (torch tensors for memory and streams) ------------------------
def _torch_dtype_code(t, dtype):
    import torch
    if dtype is not None:
        return _dt(dtype)
    m = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
    if t.dtype not in m:
        raise TypeError(f"pass dtype= for operands of type {t.dtype}")
    return m[t.dtype]


def _stream_ptr(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() else None


def _on_device(tensors, names, device=None):
    """Every tensor lives on one GPU (the first one's unless `device` is
    given): the library is handed raw device pointers, and a host pointer or
    another GPU's memory must never reach a kernel."""
    dev = device
    for t, name in zip(tensors, names):
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a GPU tensor (got device {t.device})")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, the other operands on {dev}")
    return dev


def _operands(A, B, dtype):
    code = _torch_dtype_code(A, dtype)
    if A.dim() != 2 or B.dim() != 2 or A.shape[1] != B.shape[0]:
        raise ValueError(f"bad shapes {tuple(A.shape)} x {tuple(B.shape)}")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous row-major")
    want = 4 if code == F32 else 2
    if A.element_size() != want or B.element_size() != want:
        raise TypeError("operand element size does not match the dtype")
    return code


def _new(shape, dtype, device, stream):
    """A result of a call on `stream` (torch's current stream when None), from
    that stream's memory: another stream's work may still be using what the
    caching allocator would hand out on it."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _output(C, M, N, others, names, workspace=None, stream=None):
    """Checks, before anything reaches the library, that the caller's C is a
    compact float32 [M][N] matrix and that C, the workspace and the operands
    (`others`) all live on one GPU; returns C, or a new one on that GPU (_new)."""
    import torch
    if C is not None:
        if C.dtype != torch.float32:
            raise TypeError(f"C must be float32 (got {C.dtype})")
        if tuple(C.shape) != (M, N):
            raise ValueError(f"C must have shape ({M}, {N}) (got {tuple(C.shape)})")
        if not C.is_contiguous():
            raise ValueError("C must be contiguous row-major")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    dev = _on_device((*others, C, workspace), (*names, "C", "workspace"))
    if C is None:
        C = _new((M, N), torch.float32, dev, stream)
    return C


def _workspace_bytes(workspace) -> int:
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def workspace_for(plan_dict: dict, device, stream=None):
    """A workspace of the plan's size, allocated on `stream` (torch's current
    stream when None). The caching allocator hands freed memory only to later
    work on the stream it was allocated on, so a workspace that goes out of
    scope when the call returns is not reused while the call's kernels, queued
    on that stream, still use it."""
    import torch
    n = int(plan_dict["workspace_bytes"])
    if n == 0:
        return None
    if stream is None:
        return torch.empty((n + 3) // 4, dtype=torch.float32, device=device)
    with torch.cuda.stream(stream):
        return torch.empty((n + 3) // 4, dtype=torch.float32, device=device)


def gemm(A, B, C=None, dtype=None, workspace=None, stream=None):
    """C = A·B on the tensors' device through the dispatcher; returns C (FP32)."""
    code = _operands(A, B, dtype)
    M, K = A.shape
    N = B.shape[1]
    C = _output(C, M, N, (A, B), ("A", "B"), workspace, stream)
    p = plan(M, N, K, code)
    if workspace is None:
        workspace = workspace_for(p, A.device, stream)
    ws_bytes = _workspace_bytes(workspace)
    fn = {F32: lib().sam_gemm_f32, BF16: lib().sam_gemm_bf16, F16: lib().sam_gemm_f16}[code]
    _check(fn(_ptr(A), _ptr(B), _ptr(C), M, N, K, _ptr(workspace), ws_bytes, _stream_ptr(stream)))
    return C


def gemm_variant(vid: int, A, B, C=None, split_k: int = 0, dtype=None, workspace=None, stream=None,
                 raster: int = -1):
    """C = A·B with a forced variant (and split; 0 = the variant's own pick;
    raster -1 = the cost model's raster order, 0 M-major, 1 N-major)."""
    code = _operands(A, B, dtype)
    M, K = A.shape
    N = B.shape[1]
    C = _output(C, M, N, (A, B), ("A", "B"), workspace, stream)
    p = variant_plan(vid, M, N, K, code, split_k, raster)
    if workspace is None:
        workspace = workspace_for(p, A.device, stream)
    ws_bytes = _workspace_bytes(workspace)
    _check(lib().sam_gemm_variant_r(vid, code, p["split_k"], p["raster_n"], _ptr(A), _ptr(B), _ptr(C), M, N, K,
                                    _ptr(workspace), ws_bytes, _stream_ptr(stream)))
    return C


SCRATCH_BYTES = 64 << 20   # SAM_SCRATCH_BYTES of include/sam.h


def gemm_noalloc(A, B, C=None, dtype=None, stream=None):
    """C = A·B through sam_gemm_noalloc: the plan of gemm(), with its
    workspace in the library's per-GPU scratch array (no allocation in the
    library; C is allocated here only when not given)."""
    code = _operands(A, B, dtype)
    M, K = A.shape
    N = B.shape[1]
    C = _output(C, M, N, (A, B), ("A", "B"), stream=stream)
    _check(lib().sam_gemm_noalloc(code, _ptr(A), _ptr(B), _ptr(C), M, N, K, _stream_ptr(stream)))
    return C


def _rows(t, name):
    """Row stride of a 2-D tensor whose rows are contiguous (a compact matrix
    or a view of one with padded rows). Rows that share memory (an expanded
    tensor's) have no such stride."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}'s rows share memory (stride {t.stride(0)}, rows of {t.shape[1]}): pass a copy")
    return max(int(t.stride(0)), int(t.shape[1]), 1)


def ex_workspace_bytes(M, N, K, trans_a, trans_b, lda, ldb, ldc, alpha, beta, dtype="f32", variant=None,
                       split=0, raster=-1) -> int:
    n = ctypes.c_uint64()
    if variant is None:
        _check(lib().sam_gemm_ex_workspace(_dt(dtype), int(trans_a), int(trans_b), M, N, K, lda, ldb, ldc,
                                           float(alpha), float(beta), ctypes.byref(n)))
    else:
        _check(lib().sam_gemm_ex_variant_workspace(int(variant), int(split), int(raster), _dt(dtype), int(trans_a),
                                                   int(trans_b), M, N, K, lda, ldb, ldc, float(alpha), float(beta),
                                                   ctypes.byref(n)))
    return int(n.value)


def gemm_ex(A, B, C=None, trans_a=False, trans_b=False, alpha=1.0, beta=0.0, dtype=None, workspace=None,
            stream=None, variant=None, split=0, raster=-1):
    """C = alpha·op(A)·op(B) + beta·C (sam_gemm_ex); returns C. op(A) is A or
    A.T as stored (A is K x M when trans_a), likewise B; A, B and C may be
    views with padded rows (their row stride is the leading dimension).
    variant: a forced plan (sam_gemm_ex_variant, with split and raster)."""
    import torch
    code = _torch_dtype_code(A, dtype)
    want = 4 if code == F32 else 2
    if A.element_size() != want or B.element_size() != want:
        raise TypeError("operand element size does not match the dtype")
    lda, ldb = _rows(A, "A"), _rows(B, "B")
    M, K = (A.shape[1], A.shape[0]) if trans_a else (A.shape[0], A.shape[1])
    Kb, N = (B.shape[1], B.shape[0]) if trans_b else (B.shape[0], B.shape[1])
    if Kb != K:
        raise ValueError(f"op(A) is {M}x{K} but op(B) is {Kb}x{N}")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    dev = _on_device((A, B, C, workspace), ("A", "B", "C", "workspace"))
    if C is None:
        if beta != 0.0:
            raise ValueError("beta != 0 needs C")
        C = _new((M, N), torch.float32, dev, stream)
    if tuple(C.shape) != (M, N) or C.dtype != torch.float32:
        raise ValueError(f"C must be float32 [{M}, {N}]")
    ldc = _rows(C, "C")
    if workspace is None:
        n = ex_workspace_bytes(M, N, K, trans_a, trans_b, lda, ldb, ldc, alpha, beta, code, variant, split, raster)
        workspace = workspace_for({"workspace_bytes": n}, dev, stream)
    ws_bytes = _workspace_bytes(workspace)
    tail = (M, N, K, float(alpha), _ptr(A), lda, _ptr(B), ldb, float(beta), _ptr(C), ldc, _ptr(workspace), ws_bytes,
            _stream_ptr(stream))
    if variant is None:
        _check(lib().sam_gemm_ex(code, int(trans_a), int(trans_b), *tail))
    else:
        _check(lib().sam_gemm_ex_variant(int(variant), int(split), int(raster), code, int(trans_a), int(trans_b),
                                         *tail))
    return C



def _mx_operands(A, SA, Bt, SB, fmt_a, fmt_b):
    import torch
    for t, name in ((A, "A"), (SA, "scale_a"), (Bt, "Bt"), (SB, "scale_b")):
        if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous 2-D uint8 tensor")
    M, K = A.shape
    N = Bt.shape[0]
    if Bt.shape[1] != K or tuple(SA.shape) != (M, K // 32) or tuple(SB.shape) != (N, K // 32):
        raise ValueError(f"bad shapes A{tuple(A.shape)} scale_a{tuple(SA.shape)} Bt{tuple(Bt.shape)} "
                         f"scale_b{tuple(SB.shape)}")
    return M, N, K, FP8_FORMATS[fmt_a], FP8_FORMATS[fmt_b]


def gemm_mxfp8(A, SA, Bt, SB, fmt_a="e4m3", fmt_b="e4m3", C=None, workspace=None, stream=None):
    """Block-scaled 8-bit GEMM (sam_gemm_mxfp8): A [M][K] and Bt [N][K] element
    codes, SA [M][K/32] and SB [N][K/32] E8M0 scale codes, all uint8 on the
    device; returns C [M][N] FP32."""
    import torch
    M, N, K, fa, fb = _mx_operands(A, SA, Bt, SB, fmt_a, fmt_b)
    C = _output(C, M, N, (A, SA, Bt, SB), ("A", "scale_a", "Bt", "scale_b"), workspace, stream)
    if workspace is None:
        workspace = workspace_for(plan(M, N, K, MXFP8), A.device, stream)
    ws_bytes = _workspace_bytes(workspace)
    _check(lib().sam_gemm_mxfp8(fa, fb, _ptr(A), _ptr(SA), _ptr(Bt), _ptr(SB), _ptr(C), M, N, K, _ptr(workspace),
                                ws_bytes, _stream_ptr(stream)))
    return C


def gemm_mxfp8_variant(vid: int, A, SA, Bt, SB, fmt_a="e4m3", fmt_b="e4m3", C=None, split_k: int = 0,
                       workspace=None, stream=None):
    """gemm_mxfp8 with a forced variant and split (0 = the variant's pick)."""
    import torch
    M, N, K, fa, fb = _mx_operands(A, SA, Bt, SB, fmt_a, fmt_b)
    C = _output(C, M, N, (A, SA, Bt, SB), ("A", "scale_a", "Bt", "scale_b"), workspace, stream)
    p = variant_plan(vid, M, N, K, MXFP8, split_k)
    if workspace is None:
        workspace = workspace_for(p, A.device, stream)
    ws_bytes = _workspace_bytes(workspace)
    _check(lib().sam_gemm_mxfp8_variant(vid, p["split_k"], fa, fb, _ptr(A), _ptr(SA), _ptr(Bt), _ptr(SB), _ptr(C),
                                        M, N, K, _ptr(workspace), ws_bytes, _stream_ptr(stream)))
    return C


def _mx4_operands(A, SA, Bt, SB):
    import torch
    for t, name in ((A, "A"), (SA, "scale_a"), (Bt, "Bt"), (SB, "scale_b")):
        if t.dtype != torch.uint8 or t.dim() != 2 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous 2-D uint8 tensor")
    M, K = A.shape[0], 2 * A.shape[1]
    N = Bt.shape[0]
    if Bt.shape[1] != K // 2 or tuple(SA.shape) != (M, K // 32) or tuple(SB.shape) != (N, K // 32):
        raise ValueError(f"bad shapes A{tuple(A.shape)} scale_a{tuple(SA.shape)} Bt{tuple(Bt.shape)} "
                         f"scale_b{tuple(SB.shape)}")
    return M, N, K


def gemm_mxfp4(A, SA, Bt, SB, C=None, workspace=None, stream=None):
    """Block-scaled 4-bit GEMM (sam_gemm_mxfp4): A [M][K/2] and Bt [N][K/2]
    bytes of packed E2M1 codes (low nibble first), SA [M][K/32] and SB
    [N][K/32] E8M0 scale codes, all uint8 on the device; returns C [M][N] FP32."""
    import torch
    M, N, K = _mx4_operands(A, SA, Bt, SB)
    C = _output(C, M, N, (A, SA, Bt, SB), ("A", "scale_a", "Bt", "scale_b"), workspace, stream)
    if workspace is None:
        workspace = workspace_for(plan(M, N, K, MXFP4), A.device, stream)
    ws_bytes = _workspace_bytes(workspace)
    _check(lib().sam_gemm_mxfp4(_ptr(A), _ptr(SA), _ptr(Bt), _ptr(SB), _ptr(C), M, N, K, _ptr(workspace), ws_bytes,
                                _stream_ptr(stream)))
    return C


def gemm_mxfp4_variant(vid: int, A, SA, Bt, SB, C=None, split_k: int = 0, workspace=None, stream=None):
    """gemm_mxfp4 with a forced variant and split (0 = the variant's pick)."""
    import torch
    M, N, K = _mx4_operands(A, SA, Bt, SB)
    C = _output(C, M, N, (A, SA, Bt, SB), ("A", "scale_a", "Bt", "scale_b"), workspace, stream)
    p = variant_plan(vid, M, N, K, MXFP4, split_k)
    if workspace is None:
        workspace = workspace_for(p, A.device, stream)
    ws_bytes = _workspace_bytes(workspace)
    _check(lib().sam_gemm_mxfp4_variant(vid, p["split_k"], _ptr(A), _ptr(SA), _ptr(Bt), _ptr(SB), _ptr(C), M, N, K,
                                        _ptr(workspace), ws_bytes, _stream_ptr(stream)))
    return C


# -- low-rank adapters beside a shared projection --------------------------------
# A call of few rows takes as long on the host as on the GPU, so these checks
# read each property of a tensor once.
def _matrix(t, name):
    """(rows, columns, row stride) of a 2-D tensor with contiguous rows."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    (rows, cols), (ld, step) = t.shape, t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must be 2-D with contiguous rows")
    if rows > 1 and ld < cols:
        raise ValueError(f"{name}'s rows share memory (stride {ld}, rows of {cols}): pass a copy")
    return rows, cols, max(ld, cols, 1)


def _one_gpu(names, tensors):
    """_on_device, for tensors that are in order by comparing device numbers."""
    d = tensors[0].get_device()
    for t in tensors:
        if t is not None and (d < 0 or t.get_device() != d):
            _on_device(tensors, names)
    return d


def _address(t):
    return t.data_ptr() if t is not None else None


def _stream_address(stream):
    import torch
    if stream is not None:
        return stream.cuda_stream
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # without a Stream object around it
    return raw(torch.cuda.current_device()) if raw else torch.cuda.current_stream().cuda_stream


def _adapter_operands(X, W, A, B, ids, scale, trans_w):
    """Checks of the tensors that the adapter calls share; (code, M, N, K, n, rank, ldx, ldw)."""
    import torch
    dt = X.dtype
    if dt != torch.bfloat16 and dt != torch.float16:
        raise TypeError(f"X must be bfloat16 or float16 (got {dt})")
    for t, name in ((W, "W"), (A, "A"), (B, "B")):
        if t.dtype != dt:
            raise TypeError(f"{name} is {t.dtype}, X is {dt}")
    M, K, ldx = _matrix(X, "X")
    Kw, N, ldw = _matrix(W, "W")
    if trans_w:
        Kw, N = N, Kw
    if Kw != K:
        raise ValueError(f"X has rows of {K}, W {tuple(W.shape)} (trans_w={bool(trans_w)}) takes {Kw}")
    sa, sb = A.shape, B.shape
    if len(sa) != 3 or len(sb) != 3 or sa[:2] != sb[:2] or sa[2] != K or sb[2] != N:
        raise ValueError(f"A must be [n, rank, {K}] and B [n, rank, {N}] (got {tuple(sa)}, {tuple(sb)})")
    if not (A.is_contiguous() and B.is_contiguous()):
        raise ValueError("A and B must be contiguous")
    if ids.dtype != torch.int32 or ids.dim() != 1 or ids.numel() != M or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous int32 tensor of {M} (got {ids.dtype} {tuple(ids.shape)})")
    n, rank = sa[0], sa[1]
    if scale is not None and (scale.dtype != torch.float32 or scale.dim() != 1 or scale.numel() != n
                              or not scale.is_contiguous()):
        raise ValueError(f"scale must be a contiguous float32 tensor of {n}")
    return BF16 if dt == torch.bfloat16 else F16, M, N, K, n, rank, ldx, ldw


def _adapter_result(Y, rows, cols, out_dtype, like, code, name, stream):
    """The result tensor (given or new), its type code and row stride."""
    import torch
    if Y is not None:
        if out_dtype is not None and Y.dtype != out_dtype:
            raise TypeError(f"{name} is {Y.dtype}, out_dtype {out_dtype}")
        out_dtype = Y.dtype
    elif out_dtype is None:
        out_dtype = torch.float32
    if out_dtype != like.dtype and out_dtype != torch.float32:
        raise TypeError(f"{name} must be float32 or {like.dtype} (got {out_dtype})")
    out = F32 if out_dtype == torch.float32 else code
    if Y is None:
        shape = (rows, cols)
        Y = like.new_empty(shape) if out == code and stream is None else _new(shape, out_dtype, like.device, stream)
        return Y, out, max(cols, 1)
    r, c, ld = _matrix(Y, name)
    if r != rows or c != cols:
        raise ValueError(f"{name} must have shape ({rows}, {cols}) (got {tuple(Y.shape)})")
    return Y, out, ld


@functools.lru_cache(maxsize=4096)
def _adapter_workspace_bytes(name, *args):
    """Workspace bytes of a call: a function of its sizes and strides alone."""
    b = ctypes.c_uint64()
    _check(getattr(lib(), name)(*args, ctypes.byref(b)))
    return b.value


def _adapter_workspace(nbytes, like, stream):
    """nbytes of `like`'s GPU, allocated on `stream` (see workspace_for)."""
    if not nbytes:
        return None
    if stream is not None:
        return workspace_for({"workspace_bytes": nbytes}, like.device, stream)
    es = like.element_size()
    return like.new_empty((nbytes + es - 1) // es)


def adapter_gemm(X, W, A, B, ids, scale=None, Y=None, trans_w=False, out_dtype=None, workspace=None, stream=None):
    """Y[m] = X[m]·W + scale[a]·(X[m]·A[a]^T)·B[a] with a = ids[m]
    (sam_adapter_gemm); rows whose id is outside 0 .. n-1 get X[m]·W alone.

    X [M, K] and W [K, N] (trans_w: [N, K]), bfloat16 or float16, may be views
    with padded rows; A [n, rank, K], B [n, rank, N], ids int32 [M], scale
    float32 [n]. Returns Y [M, N], float32 unless out_dtype (or Y) is of the
    operands' type."""
    code, M, N, K, n, rank, ldx, ldw = _adapter_operands(X, W, A, B, ids, scale, trans_w)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _one_gpu(("X", "W", "A", "B", "ids", "scale", "Y", "workspace"), (X, W, A, B, ids, scale, Y, workspace))
    Y, out, ldy = _adapter_result(Y, M, N, out_dtype, X, code, "Y", stream)
    t = int(trans_w)
    if workspace is None:
        need = _adapter_workspace_bytes("sam_adapter_gemm_workspace", code, t, M, N, K, n, rank, ldx, ldw)
        workspace = _adapter_workspace(need, X, stream)
    else:
        need = _workspace_bytes(workspace)
    _check(lib().sam_adapter_gemm(code, t, M, N, K, n, rank, _address(X), ldx, _address(W), ldw, _address(A),
                                  _address(B), _address(ids), _address(scale), out, _address(Y), ldy,
                                  _address(workspace), need, _stream_address(stream)))
    return Y


def adapter_backward(dY, X, W, A, B, ids, scale=None, dX=None, dA=None, dB=None, trans_w=False, out_dtype=None,
                     need_dx=True, need_dab=True, workspace=None, stream=None):
    """Gradients of adapter_gemm for dY [M, N] (sam_adapter_backward): (dX, dA,
    dB), dX [M, K] float32 unless out_dtype (or dX) is of the operands' type,
    dA [n, rank, K] and dB [n, rank, N] float32. need_dx / need_dab False:
    that part is not computed and None is returned for it."""
    import torch
    code, M, N, K, n, rank, ldx, ldw = _adapter_operands(X, W, A, B, ids, scale, trans_w)
    if dY.dtype != X.dtype or tuple(dY.shape) != (M, N):
        raise ValueError(f"dY must be {X.dtype} [{M}, {N}] (got {dY.dtype} {tuple(dY.shape)})")
    lddy = _matrix(dY, "dY")[2]
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _one_gpu(("dY", "X", "W", "A", "B", "ids", "scale", "dX", "dA", "dB", "workspace"),
             (dY, X, W, A, B, ids, scale, dX, dA, dB, workspace))
    out, lddx = F32, max(K, 1)
    if need_dx:
        dX, out, lddx = _adapter_result(dX, M, K, out_dtype, X, code, "dX", stream)
    else:
        dX = None
    if need_dab:
        dA, dB = (_new(s, torch.float32, X.device, stream) if t is None else t
                  for t, s in ((dA, A.shape), (dB, B.shape)))
        for t, like, name in ((dA, A, "dA"), (dB, B, "dB")):
            if t.dtype != torch.float32 or t.shape != like.shape or not t.is_contiguous():
                raise ValueError(f"{name} must be contiguous float32 {tuple(like.shape)}")
    else:
        dA = dB = None
    t = int(trans_w)
    if workspace is None:
        need = _adapter_workspace_bytes("sam_adapter_backward_workspace", code, t, M, N, K, n, rank, lddy, ldx, ldw,
                                        int(need_dx), int(need_dab))
        workspace = _adapter_workspace(need, X, stream)
    else:
        need = _workspace_bytes(workspace)
    _check(lib().sam_adapter_backward(code, t, M, N, K, n, rank, _address(dY), lddy, _address(X), ldx, _address(W),
                                      ldw, _address(A), _address(B), _address(ids), _address(scale), out, _address(dX),
                                      lddx, _address(dA), _address(dB), _address(workspace), need,
                                      _stream_address(stream)))
    return dX, dA, dB


# -- distillation from a teacher's top logits --------------------------------------
def _distill_operands(logits, teacher, index, weight):
    """Checks of the tensors that the distillation calls share; (code, teacher's code, rows, V, top, ldz)."""
    import torch
    codes = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
    code, t_code = codes.get(logits.dtype), codes.get(teacher.dtype)
    if code is None:
        raise TypeError(f"logits must be float32, bfloat16 or float16 (got {logits.dtype})")
    if t_code is None:
        raise TypeError(f"teacher must be float32, bfloat16 or float16 (got {teacher.dtype})")
    rows, V, ldz = _matrix(logits, "logits")
    shape = teacher.shape
    if len(shape) != 2 or shape[0] != rows or not teacher.is_contiguous():
        raise ValueError(f"teacher must be a contiguous [{rows}, top] tensor (got {tuple(shape)})")
    if index.dtype != torch.int32 or index.shape != shape or not index.is_contiguous():
        raise ValueError(f"index must be a contiguous int32 {tuple(shape)} tensor")
    if weight is not None:
        _per_row(weight, rows, None, "weight")
    return code, t_code, rows, V, shape[1], ldz


def _per_row(t, rows, like, name, stream=None):
    """t, checked, or (None) a new float32 tensor of `rows` beside `like`."""
    import torch
    if t is None:
        if stream is None:
            return torch.empty(rows, dtype=torch.float32, device=like.device)
        return _new(rows, torch.float32, like.device, stream)
    if t.dtype != torch.float32 or t.dim() != 1 or t.numel() != rows or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor of {rows}")
    return t


def _distill_result(grad, logits, V, stream):
    """The gradient (given or new) and its row stride."""
    if grad is None:
        shape = logits.shape
        return logits.new_empty(shape) if stream is None else _new(shape, logits.dtype, logits.device, stream), max(V, 1)
    if grad.dtype != logits.dtype or grad.shape != logits.shape:
        raise ValueError(f"grad must be {logits.dtype} {tuple(logits.shape)}")
    return grad, _matrix(grad, "grad")[2]


def distill_loss(logits, teacher, index, weight=None, temperature=1.0, loss=None, lse=None, stream=None):
    """Distillation loss of every row, and log-sum-exp of logits / temperature
    (sam_distill_loss): (loss, lse), float32 [rows].

    logits [rows, V] float32, bfloat16 or float16 (a view with padded rows is
    fine), teacher [rows, top] logits of the same or another of these types
    at the vocabulary entries index (int32; outside 0 .. V-1: empty), weight
    float32 [rows]."""
    code, t_code, rows, V, top, ldz = _distill_operands(logits, teacher, index, weight)
    _one_gpu(("logits", "teacher", "index", "weight", "loss", "lse"), (logits, teacher, index, weight, loss, lse))
    loss, lse = _per_row(loss, rows, logits, "loss", stream), _per_row(lse, rows, logits, "lse", stream)
    _check(lib().sam_distill_loss(code, rows, V, top, _address(logits), ldz, t_code, _address(teacher),
                                  _address(index), _address(weight), float(temperature), _address(loss),
                                  _address(lse), _stream_address(stream)))
    return loss, lse


def distill_grad(logits, lse, teacher, index, weight=None, temperature=1.0, grad=None, stream=None):
    """Gradient of the distillation loss with respect to the logits, from the
    lse of distill_loss (sam_distill_grad). grad may be logits itself."""
    code, t_code, rows, V, top, ldz = _distill_operands(logits, teacher, index, weight)
    _one_gpu(("logits", "lse", "teacher", "index", "weight", "grad"), (logits, lse, teacher, index, weight, grad))
    if lse is None:
        raise ValueError("lse is what distill_loss returned; distill makes loss and gradient without it")
    lse = _per_row(lse, rows, logits, "lse")
    grad, ldg = _distill_result(grad, logits, V, stream)
    _check(lib().sam_distill_grad(code, rows, V, top, _address(logits), ldz, _address(lse), t_code, _address(teacher),
                                  _address(index), _address(weight), float(temperature), _address(grad), ldg,
                                  _stream_address(stream)))
    return grad


def distill(logits, teacher, index, weight=None, temperature=1.0, loss=None, grad=None, stream=None):
    """Distillation loss of every row and its gradient with respect to the
    logits, which are read once (sam_distill): (loss, grad). grad may be
    logits itself."""
    code, t_code, rows, V, top, ldz = _distill_operands(logits, teacher, index, weight)
    _one_gpu(("logits", "teacher", "index", "weight", "loss", "grad"), (logits, teacher, index, weight, loss, grad))
    loss = _per_row(loss, rows, logits, "loss", stream)
    grad, ldg = _distill_result(grad, logits, V, stream)
    _check(lib().sam_distill(code, rows, V, top, _address(logits), ldz, t_code, _address(teacher), _address(index),
                             _address(weight), float(temperature), _address(loss), _address(grad), ldg,
                             _stream_address(stream)))
    return loss, grad


# -- MXFP4 tensors and the 4-bit projection -----------------------------------------
_CODES = {}   # torch's types to type codes


def _value_code(t, name):
    code = _CODES.get(t.dtype)
    if code is None:
        import torch
        _CODES.update({torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16})
        code = _CODES.get(t.dtype)
        if code is None:
            raise TypeError(f"{name} must be float32, bfloat16 or float16 (got {t.dtype})")
    return code


def _elsewhere(d):
    """A context on GPU d, or None where it is the current one."""
    import torch
    current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)   # without the first call's set-up around it
    return None if d == current() else torch.cuda.device(d)


def _mxfp4_tensor(codes, scales):
    """(rows, blocks) of a tensor's codes and scales."""
    import torch
    u8, shape = torch.uint8, codes.shape
    if codes.dtype != u8 or len(shape) != 2 or shape[1] % 16 or not codes.is_contiguous():
        raise ValueError(f"codes must be a contiguous uint8 [rows, 16 blocks] tensor (got {codes.dtype} {tuple(shape)})")
    rows, blocks = shape[0], shape[1] // 16
    if scales.dtype != u8 or scales.shape != (rows, blocks) or not scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous uint8 [{rows}, {blocks}] tensor (got {scales.dtype} {tuple(scales.shape)})")
    return rows, blocks


def _columns(K, blocks, like=None):
    """K values a row (those of `like`, a given result, or whole blocks when
    None), which `blocks` blocks of 32 have to hold."""
    if K is None:
        if like is None or like.dim() != 2:
            return 32 * blocks
        K = like.shape[1]
    if (K + 31) // 32 != blocks:
        raise ValueError(f"rows of {K} values are {(K + 31) // 32} blocks, the codes have {blocks}")
    return K


def quantize_mxfp4(X, trans=False, codes=None, scales=None, stream=None):
    """MXFP4 codes and scales of X's rows (trans: of its columns, for a weight
    stored K x N): (codes, scales), uint8 [rows, 16 ceil(K / 32)] and [rows,
    ceil(K / 32)] (sam_quantize_mxfp4). X is 2-D float32, bfloat16 or float16
    and may be a view with padded rows."""
    import torch
    code = _value_code(X, "X")
    rows, K, ldx = _matrix(X, "X")
    if trans:
        rows, K = K, rows
    there = _elsewhere(_one_gpu(("X", "codes", "scales"), (X, codes, scales)))
    if there:
        with there:
            return quantize_mxfp4(X, trans, codes, scales, stream)
    blocks = (K + 31) // 32
    given = codes is not None or scales is not None
    if codes is None:
        codes = _new((rows, 16 * blocks), torch.uint8, X.device, stream)
    if scales is None:
        scales = _new((rows, blocks), torch.uint8, X.device, stream)
    if given and _mxfp4_tensor(codes, scales) != (rows, blocks):
        raise ValueError(f"codes and scales must be of {rows} rows and {blocks} blocks (got {tuple(scales.shape)})")
    _check(lib().sam_quantize_mxfp4(code, int(trans), rows, K, _address(X), ldx, _address(codes), _address(scales),
                                    _stream_address(stream)))
    return codes, scales


def dequantize_mxfp4(codes, scales, K=None, out_dtype=None, X=None, stream=None):
    """The values that codes and scales stand for (sam_dequantize_mxfp4): X
    [rows, K], bfloat16 unless out_dtype (or X) says otherwise. K: 32 a block
    unless given (or X is)."""
    import torch
    rows, blocks = _mxfp4_tensor(codes, scales)
    K = _columns(K, blocks, X)
    there = _elsewhere(_one_gpu(("codes", "scales", "X"), (codes, scales, X)))
    if there:
        with there:
            return dequantize_mxfp4(codes, scales, K, out_dtype, X, stream)
    if X is None:
        X = _new((rows, K), torch.bfloat16 if out_dtype is None else out_dtype, codes.device, stream)
    elif out_dtype is not None and X.dtype != out_dtype:
        raise TypeError(f"X is {X.dtype}, out_dtype {out_dtype}")
    code = _value_code(X, "X")
    r, c, ldx = _matrix(X, "X")
    if (r, c) != (rows, K):
        raise ValueError(f"X must have shape ({rows}, {K}) (got {tuple(X.shape)})")
    _check(lib().sam_dequantize_mxfp4(code, rows, K, _address(codes), _address(scales), _address(X), ldx,
                                      _stream_address(stream)))
    return X


def linear_mxfp4(X, codes, scales, Y=None, out_dtype=None, workspace=None, stream=None):
    """Y = q(X)·Wq^T: X's rows rounded to MXFP4 times a weight kept in it
    (sam_linear_mxfp4). X [M, K] float32, bfloat16 or float16, may be a view
    with padded rows; codes and scales of the weight's N rows as
    quantize_mxfp4 gives them. Returns Y [M, N], float32 unless out_dtype (or
    Y) is of X's type."""
    code = _value_code(X, "X")
    N, blocks = _mxfp4_tensor(codes, scales)
    M, K, ldx = _matrix(X, "X")
    _columns(K, blocks)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    there = _elsewhere(_one_gpu(("X", "codes", "scales", "Y", "workspace"), (X, codes, scales, Y, workspace)))
    if there:
        with there:
            return linear_mxfp4(X, codes, scales, Y, out_dtype, workspace, stream)
    Y, out, ldy = _adapter_result(Y, M, N, out_dtype, X, code, "Y", stream)
    if workspace is None:
        need = _adapter_workspace_bytes("sam_linear_mxfp4_workspace", code, out, M, N, K)
        workspace = _adapter_workspace(need, X, stream)
    else:
        need = _workspace_bytes(workspace)
    _check(lib().sam_linear_mxfp4(code, M, N, K, _address(X), ldx, _address(codes), _address(scales), out, _address(Y),
                                  ldy, _address(workspace), need, _stream_address(stream)))
    return Y


def linear_mxfp4_backward(dY, codes, scales, K=None, dX=None, out_dtype=None, workspace=None, stream=None):
    """Gradient of linear_mxfp4 with respect to X for dY [M, N], X's rounding
    passed through (sam_linear_mxfp4_backward): dX = dY·Wq [M, K], float32
    unless out_dtype (or dX) is of dY's type. K: 32 a block unless given (or dX is)."""
    code = _value_code(dY, "dY")
    N, blocks = _mxfp4_tensor(codes, scales)
    K = _columns(K, blocks, dX)
    M, n, lddy = _matrix(dY, "dY")
    if n != N:
        raise ValueError(f"dY has rows of {n}, the weight {N} rows")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    there = _elsewhere(_one_gpu(("dY", "codes", "scales", "dX", "workspace"), (dY, codes, scales, dX, workspace)))
    if there:
        with there:
            return linear_mxfp4_backward(dY, codes, scales, K, dX, out_dtype, workspace, stream)
    dX, out, lddx = _adapter_result(dX, M, K, out_dtype, dY, code, "dX", stream)
    if workspace is None:
        need = _adapter_workspace_bytes("sam_linear_mxfp4_backward_workspace_strided", code, out, M, N, K, lddy, lddx)
        workspace = _adapter_workspace(need, dY, stream)
    else:
        need = _workspace_bytes(workspace)
    _check(lib().sam_linear_mxfp4_backward(code, M, N, K, _address(dY), lddy, _address(codes), _address(scales), out,
                                           _address(dX), lddx, _address(workspace), need, _stream_address(stream)))
    return dX


# -- log probabilities of given tokens ----------------------------------------------
def _logits_and_tokens(logits, tokens):
    import torch
    code = _value_code(logits, "logits")
    rows, V, ldz = _matrix(logits, "logits")
    if tokens.dtype != torch.int32 or tokens.dim() != 1 or tokens.numel() != rows or not tokens.is_contiguous():
        raise ValueError(f"tokens must be a contiguous int32 tensor of {rows} (got {tokens.dtype} {tuple(tokens.shape)})")
    return code, rows, V, ldz


def _result(t, shape, dtype, like, name, stream):
    """t, checked, or (None) a new tensor of this shape beside `like`."""
    if t is None:
        return like.new_empty(shape, dtype=dtype) if stream is None else _new(shape, dtype, like.device, stream)
    if t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {shape} tensor (got {t.dtype} {tuple(t.shape)})")
    return t


def token_logprobs(logits, tokens, temperature=1.0, top=0, logprob=None, entropy=None, norm=None, top_logprob=None,
                   top_index=None, workspace=None, stream=None):
    """Log probability of every row's token, the row's entropy and its norm
    (largest logit, log of the sum of exp((z - largest) / temperature)), and
    with `top` its most likely entries (sam_token_logprobs): (logprob [rows],
    entropy [rows], norm [rows, 2]), and with top also top_logprob and
    top_index (int32) [rows, top], most likely first, the lowest index first
    among equals.

    logits [rows, V] float32, bfloat16 or float16 (a view with padded rows is
    fine), tokens int32 [rows] (outside 0 .. V-1: none, logprob 0). top_index
    with top_logprob is what the distillation calls take from a teacher."""
    import torch
    code, rows, V, ldz = _logits_and_tokens(logits, tokens)
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    there = _elsewhere(_one_gpu(("logits", "tokens", "logprob", "entropy", "norm", "top_logprob", "top_index", "workspace"),
                                (logits, tokens, logprob, entropy, norm, top_logprob, top_index, workspace)))
    if there:
        with there:
            return token_logprobs(logits, tokens, temperature, top, logprob, entropy, norm, top_logprob, top_index,
                                  workspace, stream)
    f32 = torch.float32
    if workspace is None:
        need = _adapter_workspace_bytes("sam_token_logprobs_workspace", code, rows, V, top)
        workspace = _adapter_workspace(need, logits, stream)
    else:
        need = _workspace_bytes(workspace)
    logprob = _result(logprob, (rows,), f32, logits, "logprob", stream)
    entropy = _result(entropy, (rows,), f32, logits, "entropy", stream)
    norm = _result(norm, (rows, 2), f32, logits, "norm", stream)
    if top:
        top_logprob = _result(top_logprob, (rows, top), f32, logits, "top_logprob", stream)
        top_index = _result(top_index, (rows, top), torch.int32, logits, "top_index", stream)
    _check(lib().sam_token_logprobs(code, rows, V, top, _address(logits), ldz, _address(tokens), float(temperature),
                                    _address(logprob), _address(entropy), _address(norm), _address(top_logprob),
                                    _address(top_index), _address(workspace), need, _stream_address(stream)))
    return (logprob, entropy, norm, top_logprob, top_index) if top else (logprob, entropy, norm)


def token_logprobs_grad(logits, tokens, norm, entropy=None, dlogprob=None, dentropy=None, temperature=1.0, grad=None,
                        stream=None):
    """Gradient with respect to the logits for the gradients dlogprob and
    dentropy (float32 [rows], None: 0) of token_logprobs' results, from its
    norm and entropy (sam_token_logprobs_grad). grad may be logits itself."""
    code, rows, V, ldz = _logits_and_tokens(logits, tokens)
    import torch
    there = _elsewhere(_one_gpu(("logits", "tokens", "norm", "entropy", "dlogprob", "dentropy", "grad"),
                                (logits, tokens, norm, entropy, dlogprob, dentropy, grad)))
    if there:
        with there:
            return token_logprobs_grad(logits, tokens, norm, entropy, dlogprob, dentropy, temperature, grad, stream)
    if norm is None or (dentropy is not None and entropy is None):
        raise ValueError("norm, and with dentropy entropy, are what token_logprobs returned")
    _result(norm, (rows, 2), torch.float32, logits, "norm", stream)
    for t, name in ((entropy, "entropy"), (dlogprob, "dlogprob"), (dentropy, "dentropy")):
        if t is not None:
            _result(t, (rows,), torch.float32, logits, name, stream)
    grad, ldg = _distill_result(grad, logits, V, stream)
    _check(lib().sam_token_logprobs_grad(code, rows, V, _address(logits), ldz, _address(tokens), float(temperature),
                                         _address(norm), _address(entropy), _address(dlogprob), _address(dentropy),
                                         _address(grad), ldg, _stream_address(stream)))
    return grad
