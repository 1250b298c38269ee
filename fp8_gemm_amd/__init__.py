"""Python binding of the gfx950 FP8 GEMM library (include/fp8_gemm.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels of ``libfp8gemm.so``.  PyTorch supplies device memory and the stream.
There is no fallback: if the library is missing, or the device is not gfx950,
calls raise.

Functions take torch tensors on the GPU:

* FP8 operands as ``torch.float8_e4m3fn``, ``torch.float8_e5m2`` or
  ``torch.uint8`` (raw codes; then pass ``a_dtype`` / ``b_dtype``);
* scales as float32 tensors on the device (one element, or one per expert);
* index vectors as int32 tensors on the device;
* outputs as ``torch.bfloat16`` tensors (allocated if not given).

Autograd does not follow these calls: their outputs are plain tensors, also
where an input requires a gradient.  The forms for training come with backward
functions, which the caller calls (from a ``torch.autograd.Function``, say).
"""
from __future__ import annotations

import ctypes
import os

E4M3 = 0
E5M2 = 1

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp8gemm.so")

_lib = None


class Fp8GemmError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[{status}] {message}")
        self.status = status


class Plan(ctypes.Structure):
    _fields_ = [("variant", ctypes.c_int), ("tile_m", ctypes.c_int), ("tile_n", ctypes.c_int),
                ("token_blocks", ctypes.c_int), ("workgroups", ctypes.c_int64), ("k_splits", ctypes.c_int)]


SYMBOLS = ("fp8_gemm_nt", "fp8_gemm_nt_noalloc", "fp8_gemm_nt_blockscaled", "fp8_gemm_nt_channelwise",
           "fp8_grouped_gemm_masked_blockscaled", "fp8_grouped_gemm_contig_blockscaled", "fp8_grouped_gemm_masked", "fp8_grouped_gemm_contig",
           "bf16_gemm_nt", "fp8_gemm_plan", "fp8_gemm_strerror", "fp8_gemm_abi_version",
           "fp8_gemm_nt_fused", "bf16_gemm_nt_fused", "bf16_gemm_nt_fused_backward",
           "bf16_gemm_nt_fused_backward_workspace", "fp8_gated_nt", "bf16_gated_nt", "bf16_gated_nt_backward",
           "bf16_gated_nt_backward_workspace", "fp8_gemm_fused_plan",
           "bf16_grouped_gemm_ragged", "bf16_grouped_gemm_ragged_backward", "int8_grouped_gemm_ragged",
           "int8_gemm_nt_fused", "int8_quantize_rows", "fp8_gemm_experts_plan")

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}


def load_library(path: str = LIB_PATH):
    """Load libfp8gemm.so (built by __graft_entry__.build() or fp8_gemm_amd._build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with `python -m fp8_gemm_amd._build`")
    lib = ctypes.CDLL(path)
    P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    lib.fp8_gemm_nt.argtypes = [P, I64, I, P, I64, I, P, P, P, I64, I, I, I, P]
    lib.fp8_gemm_nt.restype = I
    lib.fp8_gemm_nt_noalloc.argtypes = [P, I64, I, P, I64, I, P, P, P, I64, I, I, I, P]
    lib.fp8_gemm_nt_noalloc.restype = I
    lib.fp8_gemm_nt_blockscaled.argtypes = [P, I64, I, P, I64, I, P, I64, P, I64, P, I64, I, I, I, P]
    lib.fp8_gemm_nt_blockscaled.restype = I
    lib.fp8_gemm_nt_channelwise.argtypes = [P, I64, I, P, I64, I, P, P, P, P, I64, I, I, I, P]
    lib.fp8_gemm_nt_channelwise.restype = I
    lib.fp8_grouped_gemm_masked.argtypes = [P, I, P, I, P, P, P, P, I, I, I, I, I, P]
    lib.fp8_grouped_gemm_masked.restype = I
    lib.fp8_grouped_gemm_masked_blockscaled.argtypes = [P, I, P, I, P, I64, P, I64, P, P, I, I, I, I, I, P]
    lib.fp8_grouped_gemm_masked_blockscaled.restype = I
    lib.fp8_grouped_gemm_contig.argtypes = [P, I, P, I, P, P, P, P, I, I, I, I, P]
    lib.fp8_grouped_gemm_contig.restype = I
    lib.fp8_grouped_gemm_contig_blockscaled.argtypes = [P, I, P, I, P, I64, P, I64, P, P, I, I, I, I, P]
    lib.fp8_grouped_gemm_contig_blockscaled.restype = I
    lib.bf16_gemm_nt.argtypes = [P, I64, P, I64, P, I64, I, I, I, P]
    lib.bf16_gemm_nt.restype = I
    lib.fp8_gemm_plan.argtypes = [I, I, I, I, I, I, ctypes.POINTER(Plan)]
    lib.fp8_gemm_plan.restype = I
    lib.fp8_gemm_strerror.argtypes = [I]
    lib.fp8_gemm_strerror.restype = ctypes.c_char_p
    lib.fp8_gemm_nt_fused.argtypes = [P, I64, I, P, I64, I, P, I, P, I, P, I, P, I64, P, I64, I, I, I, P]
    lib.fp8_gemm_nt_fused.restype = I
    lib.bf16_gemm_nt_fused.argtypes = [P, I64, P, I64, P, I, P, I64, P, I64, P, I64, I, I, I, P]
    lib.bf16_gemm_nt_fused.restype = I
    lib.bf16_gemm_nt_fused_backward.argtypes = [P, I64, P, I64, P, I64, P, I64, I, P, I64, P, I64, P, P, I64, I, I, I, P]
    lib.bf16_gemm_nt_fused_backward.restype = I
    lib.bf16_gemm_nt_fused_backward_workspace.argtypes = [I, I, I]
    lib.bf16_gemm_nt_fused_backward_workspace.restype = I64
    lib.fp8_gated_nt.argtypes = [P, I64, I, P, I64, P, I64, I, P, I, P, P, I, I, P, I64, I, I, I, P]
    lib.fp8_gated_nt.restype = I
    lib.bf16_gated_nt.argtypes = [P, I64, P, I64, P, I64, I, P, I64, P, P, I64, I, I, I, P]
    lib.bf16_gated_nt.restype = I
    lib.bf16_gated_nt_backward.argtypes = [P, I64, P, I64, P, I64, P, I64, P, P, I64, I, P, I64, P, P, I64, P, I64,
                                           I, I, I, P]
    lib.bf16_gated_nt_backward.restype = I
    lib.bf16_gated_nt_backward_workspace.argtypes = [I, I, I]
    lib.bf16_gated_nt_backward_workspace.restype = I64
    lib.fp8_gemm_fused_plan.argtypes = [I, I, I, I, ctypes.POINTER(Plan)]
    lib.fp8_gemm_fused_plan.restype = I
    lib.bf16_grouped_gemm_ragged.argtypes = [P, I64, P, I64, I64, P, P, I64, I, I, I, I, P]
    lib.bf16_grouped_gemm_ragged.restype = I
    lib.bf16_grouped_gemm_ragged_backward.argtypes = [P, I64, P, I64, P, I64, I64, P, P, I64, P, I64, I64, I, I, I, I, P]
    lib.bf16_grouped_gemm_ragged_backward.restype = I
    lib.int8_grouped_gemm_ragged.argtypes = [P, I64, P, I64, I64, P, P, P, P, I64, I, I, I, I, P]
    lib.int8_grouped_gemm_ragged.restype = I
    lib.int8_gemm_nt_fused.argtypes = [P, I64, P, I64, P, I, P, I, P, I, P, I64, P, I64, I, I, I, P]
    lib.int8_gemm_nt_fused.restype = I
    lib.int8_quantize_rows.argtypes = [P, I64, P, I64, P, I, I, P]
    lib.int8_quantize_rows.restype = I
    lib.fp8_gemm_experts_plan.argtypes = [I, I, I, I, I, ctypes.POINTER(Plan)]
    lib.fp8_gemm_experts_plan.restype = I
    lib.fp8_gemm_abi_version.argtypes = []
    lib.fp8_gemm_abi_version.restype = I
    _lib = lib
    return lib


def _check(status: int):
    if status != 0:
        raise Fp8GemmError(status, load_library().fp8_gemm_strerror(status).decode())


def plan(op: int, m: int, n: int, k: int, groups: int = 1, expected_m: int = 0) -> Plan:
    """Kernel choice for a problem (no launch).  op: 0 dense, 1 masked, 2 contiguous,
    3 block-scaled dense, 4 BF16 dense (k in elements)."""
    out = Plan()
    _check(load_library().fp8_gemm_plan(op, m, n, k, groups, expected_m, ctypes.byref(out)))
    return out


# ---------------------------------------------------------------------------
# torch-facing wrappers
# ---------------------------------------------------------------------------

def _torch():
    import torch
    return torch


def _fp8_code(t, dtype_arg, name):
    torch = _torch()
    if t.dtype == torch.float8_e4m3fn:
        d = E4M3
    elif t.dtype == torch.float8_e5m2:
        d = E5M2
    elif t.dtype == torch.uint8:
        if dtype_arg is None:
            raise TypeError(f"{name} is uint8: pass its FP8 dtype (E4M3 or E5M2)")
        d = dtype_arg
    else:
        raise TypeError(f"{name} must be float8_e4m3fn, float8_e5m2 or uint8 codes, got {t.dtype}")
    if dtype_arg is not None and dtype_arg != d:
        raise TypeError(f"{name}: dtype argument {dtype_arg} contradicts tensor dtype {t.dtype}")
    return d


def _require_cuda(*ts):
    for t in ts:
        if not t.is_cuda:
            raise ValueError("all tensors must be on the GPU")


def _scale(t, n, name):
    torch = _torch()
    if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor with {n} element(s)")
    return t


def _stream():
    return ctypes.c_void_p(_torch().cuda.current_stream().cuda_stream)


def gemm_nt(a, b, scale_a, scale_b, out=None, a_dtype=None, b_dtype=None, no_alloc=False):
    """D[M, N] = bf16(scale_a * scale_b * a[M, K] . b[N, K]^T).  no_alloc:
    call fp8_gemm_nt_noalloc (the library's fixed scratch array instead of
    its workspace; `out` must then be given, so nothing is allocated here
    either)."""
    torch = _torch()
    if no_alloc and out is None:
        raise ValueError("no_alloc=True needs out")
    fa = _fp8_code(a, a_dtype, "a")
    fb = _fp8_code(b, b_dtype, "b")
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[1]:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)} are not [M, K] and [N, K]")
    if a.stride(1) != 1 or b.stride(1) != 1:
        raise ValueError("a and b must be K-contiguous (stride(1) == 1)")
    M, K = a.shape
    N = b.shape[0]
    _require_cuda(a, b, scale_a, scale_b)
    _scale(scale_a, 1, "scale_a")
    _scale(scale_b, 1, "scale_b")
    if out is None:
        # D's row stride must be a multiple of 8 elements: pad the allocation
        # and hand back the [M, N] view.
        n_pad = max(8, ((N + 7) // 8) * 8)
        out = torch.empty((M, n_pad), dtype=torch.bfloat16, device=a.device)[:, :N]
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (M, N) or (N > 1 and out.stride(1) != 1):
        raise ValueError("out must be a [M, N] bfloat16 tensor with unit column stride")
    _require_cuda(out)
    # Row strides of size-0 or single-row dimensions are arbitrary in torch;
    # the library only needs them to be valid, as they are never stepped over.
    lda = a.stride(0) if (M > 1 and K > 0) else max(16, ((K + 15) // 16) * 16)
    ldb = b.stride(0) if (N > 1 and K > 0) else max(16, ((K + 15) // 16) * 16)
    ldd = out.stride(0) if M > 1 else max(8, ((N + 7) // 8) * 8)
    lib = load_library()
    fn = lib.fp8_gemm_nt_noalloc if no_alloc else lib.fp8_gemm_nt
    _check(fn(a.data_ptr(), lda, fa, b.data_ptr(), ldb, fb, scale_a.data_ptr(), scale_b.data_ptr(), out.data_ptr(),
              ldd, M, N, K, _stream()))
    return out


def gemm_nt_bf16(a, b, out=None):
    """BF16 comparison path: D[M, N] = bf16(a[M, K] . b[N, K]^T), a and b
    bfloat16 (or int16 / uint16 bit patterns), K-contiguous."""
    torch = _torch()
    for t, name in ((a, "a"), (b, "b")):
        if t.dtype not in (torch.bfloat16, torch.int16, torch.uint16):
            raise TypeError(f"{name} must be bfloat16 (or 16-bit bit patterns), got {t.dtype}")
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[1]:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)} are not [M, K] and [N, K]")
    if a.stride(1) != 1 or b.stride(1) != 1:
        raise ValueError("a and b must be K-contiguous (stride(1) == 1)")
    M, K = a.shape
    N = b.shape[0]
    _require_cuda(a, b)
    if out is None:
        n_pad = max(8, ((N + 7) // 8) * 8)
        out = torch.empty((M, n_pad), dtype=torch.bfloat16, device=a.device)[:, :N]
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (M, N) or (N > 1 and out.stride(1) != 1):
        raise ValueError("out must be a [M, N] bfloat16 tensor with unit column stride")
    _require_cuda(out)
    lda = a.stride(0) if (M > 1 and K > 0) else max(8, ((K + 7) // 8) * 8)
    ldb = b.stride(0) if (N > 1 and K > 0) else max(8, ((K + 7) // 8) * 8)
    ldd = out.stride(0) if M > 1 else max(8, ((N + 7) // 8) * 8)
    _check(load_library().bf16_gemm_nt(a.data_ptr(), lda, b.data_ptr(), ldb, out.data_ptr(), ldd,
                                       M, N, K, _stream()))
    return out


def gemm_nt_blockscaled(a, b, scale_a, scale_b, out=None, a_dtype=None, b_dtype=None):
    """D[M, N] = bf16(sum_kb 2^(ea-127) 2^(eb-127) a[M, K-block] . b[N, K-block]^T).

    scale_a: uint8 E8M0 codes [ceil(K/128), M'] (M' >= M, M' % 4 == 0; element
    [kb, m] scales row m over K block kb); scale_b: uint8 E8M0 codes
    [ceil(N/128), KB'] (KB' >= ceil(K/128), KB' % 4 == 0; element [nb, kb]
    scales rows 128 nb .. 128 nb + 127 over K block kb).  Both on the GPU with
    unit stride along their second dimension.
    """
    torch = _torch()
    fa = _fp8_code(a, a_dtype, "a")
    fb = _fp8_code(b, b_dtype, "b")
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[1]:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)} are not [M, K] and [N, K]")
    if a.stride(1) != 1 or b.stride(1) != 1:
        raise ValueError("a and b must be K-contiguous (stride(1) == 1)")
    M, K = a.shape
    N = b.shape[0]
    kb, nb = (K + 127) // 128, (N + 127) // 128
    for t, name, rows in ((scale_a, "scale_a", kb), (scale_b, "scale_b", nb)):
        if t.dtype != torch.uint8 or t.dim() != 2 or t.shape[0] != rows or (t.shape[0] > 1 and t.stride(1) != 1):
            raise ValueError(f"{name} must be a uint8 [{rows}, *] tensor with unit column stride")
    if scale_a.shape[1] < M or scale_b.shape[1] < kb:
        raise ValueError("scale_a needs >= M columns and scale_b >= ceil(K/128) columns")
    _require_cuda(a, b, scale_a, scale_b)
    if out is None:
        n_pad = max(8, ((N + 7) // 8) * 8)
        out = torch.empty((M, n_pad), dtype=torch.bfloat16, device=a.device)[:, :N]
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (M, N) or (N > 1 and out.stride(1) != 1):
        raise ValueError("out must be a [M, N] bfloat16 tensor with unit column stride")
    _require_cuda(out)
    lda = a.stride(0) if (M > 1 and K > 0) else max(16, ((K + 15) // 16) * 16)
    ldb = b.stride(0) if (N > 1 and K > 0) else max(16, ((K + 15) // 16) * 16)
    ldd = out.stride(0) if M > 1 else max(8, ((N + 7) // 8) * 8)
    lds_a = scale_a.stride(0) if kb > 1 else max(4, ((scale_a.shape[1] + 3) // 4) * 4)
    lds_b = scale_b.stride(0) if nb > 1 else max(4, ((scale_b.shape[1] + 3) // 4) * 4)
    _check(load_library().fp8_gemm_nt_blockscaled(a.data_ptr(), lda, fa, b.data_ptr(), ldb, fb,
                                                  scale_a.data_ptr(), lds_a, scale_b.data_ptr(), lds_b,
                                                  out.data_ptr(), ldd, M, N, K, _stream()))
    return out


def gemm_nt_channelwise(a, b, scale_a=None, scale_b=None, bias=None, out=None, a_dtype=None, b_dtype=None):
    """D[M, N] = bf16(scale_a[m] * scale_b[n] * a[m] . b[n] + bias[n]).

    scale_a: float32 [M] or None (1); scale_b, bias: float32 [N] or None (1, 0),
    contiguous, on the GPU.
    """
    torch = _torch()
    fa = _fp8_code(a, a_dtype, "a")
    fb = _fp8_code(b, b_dtype, "b")
    if a.dim() != 2 or b.dim() != 2 or a.shape[1] != b.shape[1]:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)} are not [M, K] and [N, K]")
    if a.stride(1) != 1 or b.stride(1) != 1:
        raise ValueError("a and b must be K-contiguous (stride(1) == 1)")
    M, K = a.shape
    N = b.shape[0]
    ptrs = []
    for t, n, name in ((scale_a, M, "scale_a"), (scale_b, N, "scale_b"), (bias, N, "bias")):
        if t is None:
            ptrs.append(None)
            continue
        if t.dtype != torch.float32 or t.numel() != n or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor with {n} elements")
        _require_cuda(t)
        ptrs.append(t.data_ptr())
    _require_cuda(a, b)
    if out is None:
        n_pad = max(8, ((N + 7) // 8) * 8)
        out = torch.empty((M, n_pad), dtype=torch.bfloat16, device=a.device)[:, :N]
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (M, N) or (N > 1 and out.stride(1) != 1):
        raise ValueError("out must be a [M, N] bfloat16 tensor with unit column stride")
    _require_cuda(out)
    lda = a.stride(0) if (M > 1 and K > 0) else max(16, ((K + 15) // 16) * 16)
    ldb = b.stride(0) if (N > 1 and K > 0) else max(16, ((K + 15) // 16) * 16)
    ldd = out.stride(0) if M > 1 else max(8, ((N + 7) // 8) * 8)
    _check(load_library().fp8_gemm_nt_channelwise(a.data_ptr(), lda, fa, b.data_ptr(), ldb, fb, ptrs[0], ptrs[1],
                                                  ptrs[2], out.data_ptr(), ldd, M, N, K, _stream()))
    return out


def grouped_gemm_masked(a, b, scale_a, scale_b, masked_m, out=None, expected_m=0, a_dtype=None, b_dtype=None):
    """Masked grouped GEMM: a [G, cap, K], b [G, N, K], masked_m int32 [G],
    scale_b float32 [G]; out [G, cap, N] bf16 (rows >= masked_m[g] untouched)."""
    torch = _torch()
    fa = _fp8_code(a, a_dtype, "a")
    fb = _fp8_code(b, b_dtype, "b")
    if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[2] != b.shape[2]:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)} are not [G, cap, K] and [G, N, K]")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous")
    G, cap, K = a.shape
    N = b.shape[1]
    _require_cuda(a, b, scale_a, scale_b, masked_m)
    _scale(scale_a, 1, "scale_a")
    _scale(scale_b, G, "scale_b")
    if masked_m.dtype != torch.int32 or masked_m.numel() != G or not masked_m.is_contiguous():
        raise ValueError("masked_m must be a contiguous int32 tensor with G elements")
    if out is None:
        out = torch.empty((G, cap, N), dtype=torch.bfloat16, device=a.device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (G, cap, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [G, cap, N] bfloat16 tensor")
    _require_cuda(out)
    _check(load_library().fp8_grouped_gemm_masked(a.data_ptr(), fa, b.data_ptr(), fb, scale_a.data_ptr(),
                                                  scale_b.data_ptr(), masked_m.data_ptr(), out.data_ptr(),
                                                  G, cap, N, K, int(expected_m), _stream()))
    return out


def grouped_gemm_masked_blockscaled(a, b, scale_a, scale_b, masked_m, out=None, expected_m=0, a_dtype=None,
                                    b_dtype=None):
    """Block-scaled masked grouped GEMM: a [G, cap, K], b [G, N, K], masked_m int32
    [G]; scale_a uint8 E8M0 [G, ceil(K/128), lds_a >= cap], scale_b uint8 E8M0
    [G, ceil(N/128), lds_b >= ceil(K/128)], contiguous; out [G, cap, N] bf16
    (rows >= masked_m[g] untouched)."""
    torch = _torch()
    fa = _fp8_code(a, a_dtype, "a")
    fb = _fp8_code(b, b_dtype, "b")
    if a.dim() != 3 or b.dim() != 3 or a.shape[0] != b.shape[0] or a.shape[2] != b.shape[2]:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)} are not [G, cap, K] and [G, N, K]")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous")
    G, cap, K = a.shape
    N = b.shape[1]
    kb, nb = (K + 127) // 128, (N + 127) // 128
    for t, name, mid, least in ((scale_a, "scale_a", kb, cap), (scale_b, "scale_b", nb, kb)):
        if (t.dtype != torch.uint8 or t.dim() != 3 or tuple(t.shape[:2]) != (G, mid) or t.shape[2] < least
                or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous uint8 [{G}, {mid}, >= {least}] tensor")
    _require_cuda(a, b, scale_a, scale_b, masked_m)
    if masked_m.dtype != torch.int32 or masked_m.numel() != G or not masked_m.is_contiguous():
        raise ValueError("masked_m must be a contiguous int32 tensor with G elements")
    if out is None:
        out = torch.empty((G, cap, N), dtype=torch.bfloat16, device=a.device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (G, cap, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [G, cap, N] bfloat16 tensor")
    _require_cuda(out)
    _check(load_library().fp8_grouped_gemm_masked_blockscaled(
        a.data_ptr(), fa, b.data_ptr(), fb, scale_a.data_ptr(), scale_a.shape[2], scale_b.data_ptr(),
        scale_b.shape[2], masked_m.data_ptr(), out.data_ptr(), G, cap, N, K, int(expected_m), _stream()))
    return out


def grouped_gemm_contig(a, b, scale_a, scale_b, grp_idx, out=None, a_dtype=None, b_dtype=None):
    """Contiguous grouped GEMM: a [M_total, K], b [G, N, K], grp_idx int32
    [M_total] (-1 = padding row), scale_b float32 [G]; out [M_total, N] bf16."""
    torch = _torch()
    fa = _fp8_code(a, a_dtype, "a")
    fb = _fp8_code(b, b_dtype, "b")
    if a.dim() != 2 or b.dim() != 3 or a.shape[1] != b.shape[2]:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)} are not [M_total, K] and [G, N, K]")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous")
    M_total, K = a.shape
    G, N = b.shape[0], b.shape[1]
    _require_cuda(a, b, scale_a, scale_b, grp_idx)
    _scale(scale_a, 1, "scale_a")
    _scale(scale_b, G, "scale_b")
    if grp_idx.dtype != torch.int32 or grp_idx.numel() != M_total or not grp_idx.is_contiguous():
        raise ValueError("grp_idx must be a contiguous int32 tensor with M_total elements")
    if out is None:
        out = torch.empty((M_total, N), dtype=torch.bfloat16, device=a.device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (M_total, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [M_total, N] bfloat16 tensor")
    _require_cuda(out)
    _check(load_library().fp8_grouped_gemm_contig(a.data_ptr(), fa, b.data_ptr(), fb, scale_a.data_ptr(),
                                                  scale_b.data_ptr(), grp_idx.data_ptr(), out.data_ptr(),
                                                  M_total, G, N, K, _stream()))
    return out


def grouped_gemm_contig_blockscaled(a, b, scale_a, scale_b, grp_idx, out=None, a_dtype=None, b_dtype=None):
    """Block-scaled contiguous grouped GEMM: a [M_total, K], b [G, N, K], grp_idx
    int32 [M_total] (-1 = padding); scale_a uint8 E8M0 [ceil(K/128), lds_a >=
    M_total], scale_b uint8 E8M0 [G, ceil(N/128), lds_b >= ceil(K/128)],
    contiguous; out [M_total, N] bf16 (padding rows untouched)."""
    torch = _torch()
    fa = _fp8_code(a, a_dtype, "a")
    fb = _fp8_code(b, b_dtype, "b")
    if a.dim() != 2 or b.dim() != 3 or a.shape[1] != b.shape[2]:
        raise ValueError(f"shapes {tuple(a.shape)} and {tuple(b.shape)} are not [M_total, K] and [G, N, K]")
    if not (a.is_contiguous() and b.is_contiguous()):
        raise ValueError("a and b must be contiguous")
    M_total, K = a.shape
    G, N = b.shape[0], b.shape[1]
    kb, nb = (K + 127) // 128, (N + 127) // 128
    if scale_a.dtype != torch.uint8 or scale_a.dim() != 2 or scale_a.shape[0] != kb or scale_a.shape[1] < M_total \
            or not scale_a.is_contiguous():
        raise ValueError(f"scale_a must be a contiguous uint8 [{kb}, >= {M_total}] tensor")
    if scale_b.dtype != torch.uint8 or scale_b.dim() != 3 or tuple(scale_b.shape[:2]) != (G, nb) \
            or scale_b.shape[2] < kb or not scale_b.is_contiguous():
        raise ValueError(f"scale_b must be a contiguous uint8 [{G}, {nb}, >= {kb}] tensor")
    if grp_idx.dtype != torch.int32 or grp_idx.numel() != M_total or not grp_idx.is_contiguous():
        raise ValueError("grp_idx must be a contiguous int32 tensor with M_total elements")
    _require_cuda(a, b, scale_a, scale_b, grp_idx)
    if out is None:
        out = torch.empty((M_total, N), dtype=torch.bfloat16, device=a.device)
    if out.dtype != torch.bfloat16 or tuple(out.shape) != (M_total, N) or not out.is_contiguous():
        raise ValueError("out must be a contiguous [M_total, N] bfloat16 tensor")
    _require_cuda(out)
    _check(load_library().fp8_grouped_gemm_contig_blockscaled(
        a.data_ptr(), fa, b.data_ptr(), fb, scale_a.data_ptr(), scale_a.shape[1], scale_b.data_ptr(),
        scale_b.shape[2], grp_idx.data_ptr(), out.data_ptr(), M_total, G, N, K, _stream()))
    return out


# ---------------------------------------------------------------------------
# Products with a fused epilogue and the gated feed-forward product
# (include/fp8_gemm_fused.h).  They run on the current stream of the tensors'
# device, which need not be the current one.
# ---------------------------------------------------------------------------

PLAN_PAIR = 16


def fused_plan(op: int, m: int, n: int, k: int) -> Plan:
    """Kernel choice of a fused or gated form (no launch).  op: 0 gemm_nt_fused, 1 gated_nt,
    2 gemm_nt_bf16_fused, 3 gated_nt_bf16, 4 a BF16 backward product (m x n, reduced over k), 4 + PLAN_PAIR two of them
    in one launch (the weight gradients of gated_nt_bf16_backward: N x K, reduced over M)."""
    out = Plan()
    _check(load_library().fp8_gemm_fused_plan(op, m, n, k, ctypes.byref(out)))
    return out


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {', '.join(ACTIVATIONS)}, got {name!r}") from None


# What the wrappers below look up on every call, once: a few-token kernel takes less time than the
# argument checks did through `import torch`, torch.device objects and torch.cuda.Stream.
class _Torch:
    def __init__(self):
        import torch
        self.bf16, self.f32, self.empty = torch.bfloat16, torch.float32, torch.empty
        self.i8, self.i32 = torch.int8, torch.int32
        self.fp8 = {torch.float8_e4m3fn: E4M3, torch.float8_e5m2: E5M2}
        self.current_device, self.guard = torch.cuda.current_device, torch.cuda.device
        # the current stream's handle without a Stream object around it, where torch offers that
        self.stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda index: torch.cuda.current_stream(index).cuda_stream)


_cached = None


def _tt():
    global _cached
    if _cached is None:
        _cached = _Torch()
    return _cached


def _call(tt, index, fn, *args):
    """fn(*args, stream) on the current stream of device `index`."""
    if index == tt.current_device():
        status = fn(*args, tt.stream(index))
    else:
        with tt.guard(index):
            status = fn(*args, tt.stream(index))
    if status:
        _check(status)


def _device(a, *others):
    """The GPU of `a`, which the other tensors (or None) must share."""
    index = a.get_device()
    if index < 0:
        raise ValueError("all tensors must be on the GPU")
    for t in others:
        if t is not None and t.get_device() != index:
            raise ValueError(f"all tensors must be on one GPU: {t.device} and {a.device}")
    return index


def _matrices(a, b, bname):
    """M, N, K of a [M, K] and b [N, K]."""
    sa, sb = a.shape, b.shape
    if len(sa) != 2 or len(sb) != 2 or sa[1] != sb[1]:
        raise ValueError(f"shapes {tuple(sa)} and {tuple(sb)} of a and {bname} are not [M, K] and [N, K]")
    return sa[0], sb[0], sa[1]


def _fp8_of(tt, t, dtype_arg, name):
    code = tt.fp8.get(t.dtype)
    if code is None or (dtype_arg is not None and dtype_arg != code):
        return _fp8_code(t, dtype_arg, name)
    return code


def _operand(t, name, rows, K, grain):
    """The row stride in elements of a K-contiguous [rows, K] operand (one that satisfies the library where
    torch's is arbitrary: a single row or an empty matrix)."""
    ld, unit = t.stride()
    if unit != 1 and K > 1:
        raise ValueError(f"{name} must be K-contiguous (stride(1) == 1)")
    return ld if rows > 1 and K else (K + grain - 1) // grain * grain


def _rows(t, name, M, N, dtype):
    """The row stride of a [M, N] matrix with unit column stride whose rows do not overlap."""
    if t.dtype != dtype or t.dim() != 2 or tuple(t.shape) != (M, N):
        raise ValueError(f"{name} must be a [{M}, {N}] {dtype} tensor, got {list(t.shape)} {t.dtype}")
    ld, unit = t.stride()
    if unit != 1 and N > 1:
        raise ValueError(f"{name} must have unit column stride")
    if M <= 1 or N == 0:
        return N
    if ld < N:
        raise ValueError(f"{name}: row stride {ld} below {N}")
    return ld


def _new(tt, M, N, device):
    """A BF16 [M, N] output in rows padded to 8 elements, and its row stride."""
    ld = (N + 7) // 8 * 8
    out = tt.empty((M, ld), dtype=tt.bf16, device=device)
    return (out if ld == N else out[:, :N]), ld


def _output(tt, out, a, index, M, N):
    if out is None:
        return _new(tt, M, N, a.device)
    if out.get_device() != index:
        raise ValueError(f"out is on {out.device}, a on {a.device}")
    ld = _rows(out, "out", M, N, tt.bf16)
    return out, (ld if M > 1 else (N + 7) // 8 * 8)


def _floats(tt, t, name, n, one=True):
    """A contiguous float32 vector of n values (or, if `one`, of a single one): (pointer, values)."""
    if t is None:
        return None, 0
    count = t.numel()
    if t.dtype != tt.f32 or not (count == n or (one and count == 1)) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous float32 tensor with {n}{' or 1' if one else ''} element(s)")
    return t.data_ptr(), count


def _ptr(t):
    return None if t is None else t.data_ptr()


def _bf16_only(tt, **tensors):
    for name, t in tensors.items():
        if t.dtype != tt.bf16:
            raise TypeError(f"{name} must be bfloat16, got {t.dtype}")


def gemm_nt_fused(a, b, scale_a=None, scale_b=None, bias=None, activation="none", residual=None, out=None,
                  a_dtype=None, b_dtype=None):
    """FP8 product with bias, activation and residual in its epilogue:

        out[M, N] = bf16(act(scale_a[m] * scale_b[n] * a[m] . b[n] + bias[n]) + residual[m, n])

    scale_a: float32, M elements or 1, or None (1); scale_b: float32, N elements
    or 1, or None; bias: float32 [N] or None; activation: "none", "relu",
    "silu", "gelu" (erf) or "gelu_tanh"; residual: bfloat16 [M, N] with any row
    stride, or None; it may be `out` itself.  Otherwise `out` must not share
    memory with an operand (columns of one buffer that do not overlap may be
    both); the library refuses such calls.
    """
    tt = _tt()
    fa, fb = _fp8_of(tt, a, a_dtype, "a"), _fp8_of(tt, b, b_dtype, "b")
    M, N, K = _matrices(a, b, "b")
    index = _device(a, b, scale_a, scale_b, bias, residual)
    lda, ldb = _operand(a, "a", M, K, 16), _operand(b, "b", N, K, 16)
    sa, na = _floats(tt, scale_a, "scale_a", M)
    sb, nb = _floats(tt, scale_b, "scale_b", N)
    bp, _ = _floats(tt, bias, "bias", N, one=False)
    ldr = 0 if residual is None else _rows(residual, "residual", M, N, tt.bf16)
    act = _activation(activation)
    out, ldd = _output(tt, out, a, index, M, N)
    _call(tt, index, load_library().fp8_gemm_nt_fused, a.data_ptr(), lda, fa, b.data_ptr(), ldb, fb, sa, na, sb, nb,
          bp, act, _ptr(residual), ldr, out.data_ptr(), ldd, M, N, K)
    return out


def gemm_nt_bf16_fused(a, b, bias=None, activation="none", residual=None, out=None, preact=None):
    """BF16 product with bias, activation and residual in its epilogue:

        z = a[m] . b[n] + bias[n];  out[M, N] = bf16(act(z) + residual[m, n])

    Arguments as for gemm_nt_fused.  preact: a float32 [M, N] tensor that
    receives z, for gemm_nt_bf16_fused_backward, or None; it is an output, and
    must not share memory with another one or an operand.
    """
    tt = _tt()
    _bf16_only(tt, a=a, b=b)
    M, N, K = _matrices(a, b, "b")
    index = _device(a, b, bias, residual, preact)
    lda, ldb = _operand(a, "a", M, K, 8), _operand(b, "b", N, K, 8)
    bp, _ = _floats(tt, bias, "bias", N, one=False)
    ldr = 0 if residual is None else _rows(residual, "residual", M, N, tt.bf16)
    ldp = 0 if preact is None else _rows(preact, "preact", M, N, tt.f32)
    act = _activation(activation)
    out, ldd = _output(tt, out, a, index, M, N)
    _call(tt, index, load_library().bf16_gemm_nt_fused, a.data_ptr(), lda, b.data_ptr(), ldb, bp, act, _ptr(residual),
          ldr, out.data_ptr(), ldd, _ptr(preact), ldp, M, N, K)
    return out


def _workspace(tt, size, device):
    if size < 0:
        _check(size)
    import torch
    return tt.empty(size, dtype=torch.uint8, device=device) if size else None


def gemm_nt_bf16_fused_backward(grad_out, a, b, activation="none", preact=None, bias_grad=False, a_grad=True,
                                b_grad=True):
    """Backward pass of gemm_nt_bf16_fused: (grad_a, grad_b, grad_bias) for the
    gradient `grad_out` of its output (bfloat16 [M, N], any row stride), where

        dz = grad_out * act'(preact);  grad_a = bf16(dz . b);  grad_b = bf16(dz^T . a);  grad_bias = dz summed over m

    preact: the tensor that the forward call filled (None with activation
    "none").  grad_bias is float32 [N]; what a_grad, b_grad or bias_grad
    excludes is None.  The residual's gradient is grad_out itself.
    """
    tt = _tt()
    _bf16_only(tt, grad_out=grad_out, a=a, b=b)
    M, N, K = _matrices(a, b, "b")
    index = _device(a, b, grad_out, preact)
    act = _activation(activation)
    lda, ldb = _operand(a, "a", M, K, 8), _operand(b, "b", N, K, 8)
    ldg = _rows(grad_out, "grad_out", M, N, tt.bf16)
    if preact is None and act:
        raise ValueError(f"activation {activation!r} needs preact")
    ldp = 0 if preact is None else _rows(preact, "preact", M, N, tt.f32)
    dev = a.device
    ga, ldga = _new(tt, M, K, dev) if a_grad else (None, 0)
    gb, ldgb = _new(tt, N, K, dev) if b_grad else (None, 0)
    gbias = tt.empty(N, dtype=tt.f32, device=dev) if bias_grad else None
    lib = load_library()
    ws = _workspace(tt, lib.bf16_gemm_nt_fused_backward_workspace(M, N, K), dev)
    _call(tt, index, lib.bf16_gemm_nt_fused_backward, grad_out.data_ptr(), ldg, a.data_ptr(), lda, b.data_ptr(), ldb,
          _ptr(preact), ldp, act, _ptr(ga), ldga, _ptr(gb), ldgb, _ptr(gbias), _ptr(ws),
          0 if ws is None else ws.numel(), M, N, K)
    return ga, gb, gbias


def _same_shape(t, name, N, K):
    if tuple(t.shape) != (N, K):
        raise ValueError(f"{name} is {list(t.shape)}, w_gate {[N, K]}")


def gated_nt(a, w_gate, w_up, scale_a=None, scale_gate=None, scale_up=None, activation="silu", out=None,
             a_dtype=None, w_dtype=None):
    """FP8 gated feed-forward product, one kernel for both projections, the
    activation and the product:

        out[M, N] = bf16(act(scale_a[m] * scale_gate[n] * a[m] . w_gate[n]) * (scale_a[m] * scale_up[n] * a[m] . w_up[n]))

    w_gate, w_up: [N, K] of one FP8 dtype (for example the two halves of a
    merged [2 N, K] weight); scales as for gemm_nt_fused, scale_gate and
    scale_up of the same length.
    """
    tt = _tt()
    fa, fw = _fp8_of(tt, a, a_dtype, "a"), _fp8_of(tt, w_gate, w_dtype, "w_gate")
    if _fp8_of(tt, w_up, w_dtype, "w_up") != fw:
        raise TypeError("w_gate and w_up must have one FP8 dtype")
    M, N, K = _matrices(a, w_gate, "w_gate")
    _same_shape(w_up, "w_up", N, K)
    index = _device(a, w_gate, w_up, scale_a, scale_gate, scale_up)
    lda, ldg, ldu = _operand(a, "a", M, K, 16), _operand(w_gate, "w_gate", N, K, 16), _operand(w_up, "w_up", N, K, 16)
    sa, na = _floats(tt, scale_a, "scale_a", M)
    sg, ng = _floats(tt, scale_gate, "scale_gate", N)
    su, nu = _floats(tt, scale_up, "scale_up", N)
    if ng and nu and ng != nu:
        raise ValueError("scale_gate and scale_up must have one length")
    act = _activation(activation)
    out, ldd = _output(tt, out, a, index, M, N)
    _call(tt, index, load_library().fp8_gated_nt, a.data_ptr(), lda, fa, w_gate.data_ptr(), ldg, w_up.data_ptr(), ldu,
          fw, sa, na, sg, su, max(ng, nu), act, out.data_ptr(), ldd, M, N, K)
    return out


def _gated_preact(tt, preact, M, N):
    """(gate, up, row stride) pointers of a float32 [2, M, N] tensor, whose two matrices do not overlap (one
    behind the other, or their rows in turn)."""
    if preact.dim() != 3 or preact.shape[0] != 2:
        raise ValueError(f"preact must be a [2, {M}, {N}] tensor, got {list(preact.shape)}")
    gate = preact[0]
    ld = _rows(gate, "preact", M, N, tt.f32)
    step = preact.stride(0)
    if M and N and step < (M - 1) * ld + N and (step < N or ld < step + N):
        raise ValueError("preact: its two matrices overlap")
    pointer = gate.data_ptr()
    return pointer, pointer + 4 * step, ld


def gated_nt_bf16(a, w_gate, w_up, activation="silu", out=None, preact=None):
    """BF16 gated feed-forward product:

        g = a[m] . w_gate[n];  u = a[m] . w_up[n];  out[M, N] = bf16(act(g) * u)

    preact: a float32 [2, M, N] tensor that receives g and u, for
    gated_nt_bf16_backward, or None.
    """
    tt = _tt()
    _bf16_only(tt, a=a, w_gate=w_gate, w_up=w_up)
    M, N, K = _matrices(a, w_gate, "w_gate")
    _same_shape(w_up, "w_up", N, K)
    index = _device(a, w_gate, w_up, preact)
    lda, ldg, ldu = _operand(a, "a", M, K, 8), _operand(w_gate, "w_gate", N, K, 8), _operand(w_up, "w_up", N, K, 8)
    pg, pu, ldp = (None, None, 0) if preact is None else _gated_preact(tt, preact, M, N)
    act = _activation(activation)
    out, ldd = _output(tt, out, a, index, M, N)
    _call(tt, index, load_library().bf16_gated_nt, a.data_ptr(), lda, w_gate.data_ptr(), ldg, w_up.data_ptr(), ldu,
          act, out.data_ptr(), ldd, pg, pu, ldp, M, N, K)
    return out


def gated_nt_bf16_backward(grad_out, a, w_gate, w_up, preact, activation="silu", a_grad=True, w_grad=True):
    """Backward pass of gated_nt_bf16: (grad_a, grad_gate, grad_up) for the
    gradient `grad_out` of its output (bfloat16 [M, N], any row stride), where

        dg = grad_out * u * act'(g);  du = grad_out * act(g)
        grad_a = bf16(dg . w_gate + du . w_up);  grad_gate = bf16(dg^T . a);  grad_up = bf16(du^T . a)

    preact: the tensor that the forward call filled.  w_gate and w_up share one
    row stride.  What a_grad or w_grad excludes is None.
    """
    tt = _tt()
    _bf16_only(tt, grad_out=grad_out, a=a, w_gate=w_gate, w_up=w_up)
    M, N, K = _matrices(a, w_gate, "w_gate")
    _same_shape(w_up, "w_up", N, K)
    index = _device(a, w_gate, w_up, grad_out, preact)
    lda, ldg, ldu = _operand(a, "a", M, K, 8), _operand(w_gate, "w_gate", N, K, 8), _operand(w_up, "w_up", N, K, 8)
    ldgrad = _rows(grad_out, "grad_out", M, N, tt.bf16)
    pg, pu, ldp = _gated_preact(tt, preact, M, N)
    act = _activation(activation)
    dev = a.device
    ga, ldga = _new(tt, M, K, dev) if a_grad else (None, 0)
    gw, ldgw = _new(tt, N, K, dev) if w_grad else (None, 0)
    gu = _new(tt, N, K, dev)[0] if w_grad else None
    lib = load_library()
    ws = _workspace(tt, lib.bf16_gated_nt_backward_workspace(M, N, K), dev)
    _call(tt, index, lib.bf16_gated_nt_backward, grad_out.data_ptr(), ldgrad, a.data_ptr(), lda, w_gate.data_ptr(),
          ldg, w_up.data_ptr(), ldu, pg, pu, ldp, act, _ptr(ga), ldga, _ptr(gw), _ptr(gu), ldgw, _ptr(ws),
          0 if ws is None else ws.numel(), M, N, K)
    return ga, gw, gu


# ---------------------------------------------------------------------------
# Experts' products over ragged groups of rows, products in 8-bit integers and
# the quantisation of rows (include/fp8_gemm_experts.h).  As above they run on
# the current stream of the tensors' device.
# ---------------------------------------------------------------------------

def experts_plan(op: int, m: int, n: int, k: int, groups: int = 1) -> Plan:
    """Kernel choice of a ragged or integer form (no launch).  op: 0 grouped_gemm_ragged_bf16, 1 grouped_gemm_ragged_int8,
    2 and 3 the token and weight gradients of grouped_gemm_ragged_bf16_backward, 4 gemm_nt_int8 without activation and
    residual.  Variant 0: nothing is launched (nothing to compute, or sizes that the call refuses)."""
    out = Plan()
    _check(load_library().fp8_gemm_experts_plan(op, m, n, k, groups, ctypes.byref(out)))
    return out


def _int8_only(tt, a, b):
    if a.dtype is not tt.i8 or b.dtype is not tt.i8:
        raise TypeError(f"a and b must be int8, got {a.dtype} and {b.dtype}")


def _ragged(tt, a, b, offsets):
    """M, G, N, K of a [M, K] and b [G, N, K] with the int32 offsets [G + 1] of the experts' rows."""
    sa, sb = a.shape, b.shape
    if len(sa) != 2 or len(sb) != 3 or sa[1] != sb[2]:
        raise ValueError(f"shapes {tuple(sa)} and {tuple(sb)} of a and b are not [M, K] and [G, N, K]")
    G = sb[0]
    if offsets.dtype != tt.i32 or tuple(offsets.shape) != (G + 1,) or not offsets.is_contiguous():
        raise ValueError(f"offsets must be a contiguous int32 tensor with {G + 1} elements, got {list(offsets.shape)} {offsets.dtype}")
    return sa[0], G, sb[1], sa[1]


def _expert_weights(b, G, N, K, grain):
    """The row and expert strides in elements of a K-contiguous [G, N, K] operand."""
    step, ld, unit = b.stride()
    if unit != 1 and K > 1:
        raise ValueError("b must be K-contiguous (stride(2) == 1)")
    if N <= 1 or not K:
        ld = (K + grain - 1) // grain * grain
    return ld, step if G > 1 else N * ld


def grouped_gemm_ragged_bf16(a, b, offsets, out=None):
    """BF16 product of ragged groups of rows with their experts' weights:

        out[r, n] = bf16(a[r] . b[g, n])    for offsets[g] <= r < offsets[g + 1]

    a: bfloat16 [M, K], the rows sorted by expert; b: bfloat16 [G, N, K] with
    any row stride, one expert's matrix behind the other's at any distance that
    keeps them apart; offsets: int32 [G + 1] on the GPU, not
    decreasing, from 0 to M; an expert may have any number of rows.  Rows of no
    expert (before offsets[0], from offsets[G] on) are left as they were in
    `out`, unset where it is allocated here.  K % 8 == 0 and N % 8 == 0.
    """
    tt = _tt()
    _bf16_only(tt, a=a, b=b)
    M, G, N, K = _ragged(tt, a, b, offsets)
    index = _device(a, b, offsets)
    lda = _operand(a, "a", M, K, 8)
    ldb, step = _expert_weights(b, G, N, K, 8)
    out, ldd = _output(tt, out, a, index, M, N)
    _call(tt, index, load_library().bf16_grouped_gemm_ragged, a.data_ptr(), lda, b.data_ptr(), ldb, step,
          offsets.data_ptr(), out.data_ptr(), ldd, M, G, N, K)
    return out


def grouped_gemm_ragged_bf16_backward(grad_out, a, b, offsets, a_grad=True, b_grad=True):
    """Backward pass of grouped_gemm_ragged_bf16: (grad_a, grad_b) for the
    gradient `grad_out` of its output (bfloat16 [M, N], unit column stride,
    rows that start 16-byte aligned), where

        grad_a[r] = bf16(grad_out[r] . b[g])                       0 for the rows of no expert
        grad_b[g] = bf16(sum over g's rows of grad_out[r]^T . a[r])  0 for an expert without rows

    What a_grad or b_grad excludes is None.
    """
    tt = _tt()
    _bf16_only(tt, grad_out=grad_out, a=a, b=b)
    M, G, N, K = _ragged(tt, a, b, offsets)
    if tuple(grad_out.shape) != (M, N):
        raise ValueError(f"grad_out must be a [{M}, {N}] tensor, got {list(grad_out.shape)}")
    index = _device(a, b, offsets, grad_out)
    lda, ldg = _operand(a, "a", M, K, 8), _operand(grad_out, "grad_out", M, N, 8)
    ldb, step = _expert_weights(b, G, N, K, 8)
    ga, ldga = _new(tt, M, K, a.device) if a_grad else (None, 0)
    gb = tt.empty((G, N, K), dtype=tt.bf16, device=a.device) if b_grad else None
    _call(tt, index, load_library().bf16_grouped_gemm_ragged_backward, grad_out.data_ptr(), ldg, a.data_ptr(), lda,
          b.data_ptr(), ldb, step, offsets.data_ptr(), _ptr(ga), ldga, _ptr(gb), K, N * K, M, G, N, K)
    return ga, gb


def grouped_gemm_ragged_int8(a, b, offsets, scale_a=None, scale_b=None, out=None):
    """The product of grouped_gemm_ragged_bf16 in 8-bit integers, with a scale for
    each row and each expert's channel:

        out[r, n] = bf16(scale_a[r] * scale_b[g, n] * a[r] . b[g, n])

    a: int8 [M, K]; b: int8 [G, N, K]; scale_a: float32 [M] or None (1);
    scale_b: float32 [G, N], contiguous, or None.  The sums are exact.
    K % 16 == 0 and K <= 131056, N % 8 == 0.
    """
    tt = _tt()
    _int8_only(tt, a, b)
    M, G, N, K = _ragged(tt, a, b, offsets)
    # (as many elements in another order: a scale of each channel for each expert)
    if scale_b is not None and scale_b.dim() > 1 and G > 1 and scale_b.shape[0] == N != G:
        raise ValueError(f"scale_b must be a [{G}, {N}] tensor, got {list(scale_b.shape)}")
    index = _device(a, b, offsets, scale_a, scale_b)
    lda = _operand(a, "a", M, K, 16)
    ldb, step = _expert_weights(b, G, N, K, 16)
    sa, _ = _floats(tt, scale_a, "scale_a", M, one=False)
    sb, _ = _floats(tt, scale_b, "scale_b", G * N, one=False)
    out, ldd = _output(tt, out, a, index, M, N)
    _call(tt, index, load_library().int8_grouped_gemm_ragged, a.data_ptr(), lda, b.data_ptr(), ldb, step, sa, sb,
          offsets.data_ptr(), out.data_ptr(), ldd, M, G, N, K)
    return out


def gemm_nt_int8(a, b, scale_a=None, scale_b=None, bias=None, activation="none", residual=None, out=None):
    """Product in 8-bit integers with bias, activation and residual in its epilogue:

        out[M, N] = bf16(act(scale_a[m] * scale_b[n] * a[m] . b[n] + bias[n]) + residual[m, n])

    a: int8 [M, K]; b: int8 [N, K]; everything else as for gemm_nt_fused.  The
    sums are exact: K % 16 == 0 and K <= 131056.
    """
    tt = _tt()
    _int8_only(tt, a, b)
    M, N, K = _matrices(a, b, "b")
    index = _device(a, b, scale_a, scale_b, bias, residual)
    lda, ldb = _operand(a, "a", M, K, 16), _operand(b, "b", N, K, 16)
    sa, na = _floats(tt, scale_a, "scale_a", M)
    sb, nb = _floats(tt, scale_b, "scale_b", N)
    bp, _ = _floats(tt, bias, "bias", N, one=False)
    ldr = 0 if residual is None else _rows(residual, "residual", M, N, tt.bf16)
    act = _activation(activation)
    out, ldd = _output(tt, out, a, index, M, N)
    _call(tt, index, load_library().int8_gemm_nt_fused, a.data_ptr(), lda, b.data_ptr(), ldb, sa, na, sb, nb, bp, act,
          _ptr(residual), ldr, out.data_ptr(), ldd, M, N, K)
    return out


def quantize_rows_int8(x, codes=None, scales=None):
    """Rows of x (bfloat16 [M, K]) in 8-bit integers: (codes, scales) with

        scales[m] = max_k |x[m, k]| / 127;  codes[m, k] = round(127 x[m, k] / max_k |x[m, k]|)

    rounded to the nearest whole number, halves to even.  codes: int8 [M, K],
    scales: float32 [M], both allocated if not given.  A row of zeros has the
    scale 0; one with an infinity or a NaN the scale NaN and codes 0.
    K % 16 == 0.
    """
    tt = _tt()
    if x.dtype is not tt.bf16:
        raise TypeError(f"x must be bfloat16, got {x.dtype}")
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"x must be a [M, K] tensor, got {list(shape)}")
    M, K = shape
    index = _device(x, codes, scales)
    ldx = _operand(x, "x", M, K, 16)
    device = x.device
    if codes is None:
        ldq = (K + 15) // 16 * 16
        codes = tt.empty(shape, dtype=tt.i8, device=device)
    else:
        ldq = _rows(codes, "codes", M, K, tt.i8)
        if M == 1:
            ldq = (K + 15) // 16 * 16              # (never stepped over)
    if scales is None:
        scales = tt.empty(M, dtype=tt.f32, device=device)
    elif scales.dtype != tt.f32 or tuple(scales.shape) != (M,) or not scales.is_contiguous():
        raise ValueError(f"scales must be a contiguous float32 tensor with {M} elements")
    _call(tt, index, load_library().int8_quantize_rows, x.data_ptr(), ldx, codes.data_ptr(), ldq, scales.data_ptr(), M, K)
    return codes, scales
