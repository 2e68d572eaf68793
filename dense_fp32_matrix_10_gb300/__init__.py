"""Single-precision GEMM for one NVIDIA GB300 (sm_103a).

    C = alpha * op(A) * op(B) + beta * C       (row-major FP32, op = N or T)

The computation happens entirely in the hand-written CUDA kernels of
``libsgemm_gb300.so`` (built from ``csrc/`` by ``build.py``); this package only
marshals arguments to its C ABI (``include/sgemm.h``) through ctypes.  PyTorch is
used for device memory and streams only.  There is no CPU fallback: every entry
point raises if the CUDA library is missing or cannot run.

Low level (same names and arguments as the C ABI, pointers as ints, raising
``SgemmError`` on any status other than success):
    sgemm, sgemm_ex, sgemm_strided_batched, sgemm_transpose, sgemm_noalloc,
    sgemm_select_algo, sgemm_last_launch_count,
    sgemm_last_device_status, sgemm_set_scratch_limit, sgemm_get_scratch_limit,
    sgemm_set_wait_budget_ns,
    sgemm_selftest_wait_timeout, sgemm_status_string, sgemm_algo_name,
    sgemm_version
High level (torch tensors): ``gemm``, ``gemm_strided_batched``, ``transpose``.

The linear layer in 8-bit floating point (module ``fp8``, ``include/sgemm_fp8.h``):
``gemm_fp8``, ``quantize_fp8``, ``quantize_fp8_both``, ``rms_norm_fp8``,
``rms_norm_backward`` on torch tensors, and the ``sgemm_*`` functions they call.

Around a gated block's products (module ``fp8_block``, ``include/sgemm_fp8_block.h``):
``sandwich_norm_fp8``, ``sandwich_norm_backward``, ``swiglu_fp8``, ``swiglu_backward_fp8``,
``requantize_fp8``, and the ``sgemm_*`` functions they call.
"""
from ._binding import (  # noqa: F401
    ALGO_AUTO, ALGO_NAIVE, ALGO_REG_2X2, ALGO_REG_4X4, ALGO_SIMT_CPASYNC, ALGO_SIMT_TMA,
    ALGO_SMALL, ALGO_SMEM_TILED, ALGO_TC_3XTF32,
    ALGOS, OP_N, OP_T, SCRATCH_UNLIMITED, STATUS, SgemmError, gemm, library_path, load_library,
    sgemm, sgemm_get_scratch_limit, sgemm_set_scratch_limit,
    sgemm_algo_name, sgemm_ex, sgemm_last_device_status, sgemm_last_launch_count, sgemm_noalloc,
    sgemm_select_algo, sgemm_selftest_wait_timeout, sgemm_set_wait_budget_ns,
    sgemm_status_string, sgemm_strided_batched, sgemm_transpose, sgemm_version,
    gemm_strided_batched, transpose)

_FP8_NAMES = (
    "RmsNormFp8", "gemm_fp8", "quantize_fp8", "quantize_fp8_both", "rms_norm_backward", "rms_norm_fp8", "sgemm_fp8",
    "sgemm_fp8_quantize", "sgemm_fp8_quantize_both", "sgemm_fp8_select_form", "sgemm_rms_norm_backward",
    "sgemm_rms_norm_backward_workspace", "sgemm_rms_norm_fp8")
_FP8_BLOCK_NAMES = (
    "SandwichNormFp8", "SandwichNormGrad", "SwigluFp8", "SwigluGradFp8", "requantize_fp8", "sandwich_norm_backward",
    "sandwich_norm_fp8", "swiglu_backward_fp8", "swiglu_fp8", "sgemm_fp8_requantize", "sgemm_sandwich_norm_backward",
    "sgemm_sandwich_norm_backward_workspace", "sgemm_sandwich_norm_fp8", "sgemm_swiglu_backward_fp8", "sgemm_swiglu_fp8")


def __getattr__(name):
    """The names of modules fp8 and fp8_block, which import torch, on first use."""
    if name in _FP8_NAMES:
        from . import fp8
        globals().update((n, getattr(fp8, n)) for n in _FP8_NAMES)
        return globals()[name]
    if name in _FP8_BLOCK_NAMES:
        from . import fp8_block
        globals().update((n, getattr(fp8_block, n)) for n in _FP8_BLOCK_NAMES)
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted({*globals(), *_FP8_NAMES, *_FP8_BLOCK_NAMES})
