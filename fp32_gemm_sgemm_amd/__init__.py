"""MI355X-native single-precision GEMM (row-major) behind a C ABI.

The compute path is the HIP library libsgemm.so (built from csrc/ for gfx950):
C = alpha * op(A) x op(B) + beta * C with optional transposed operands, strided
batches and K split across workgroups.  This package holds its thin ctypes
binding (binding.py) with the operators around a product (ops.py: bias,
activation and residual in the epilogue with their gradients, RMS norms, 8-bit
quantisation and products), what else a model's layer and its training step
need (layers.py: gated feed-forward blocks, layer norms, their gradients, and
gradients clipped to a norm), the seeded input generators (inputs.py) and
host-side counting (metrics.py).  libsgemm_lds_poison.so is the same code built as an
LDS race check, for the tests; libsgemm_timeline.so is the same code with
clock readings inside the direct-load kernel, which timeline.py reports.  The
library is loaded on first use; if it is missing, every entry point raises.
"""
from .binding import (  # noqa: F401
    SgemmCfg, SgemmError, load, sgemm, sgemm_batched, sgemm_f32, sgemm_f32_cfg_geometry,
    sgemm_f32_ex, sgemm_f32_ex_noalloc, sgemm_f32_gemm, sgemm_f32_num_variants, sgemm_f32_plan, sgemm_f32_query,
    sgemm_f32_strided_batched, sgemm_f32_variant, sgemm_f32_variant_ops, sgemm_f32_version,
    sgemm_f32_workspace_size, library, LIB_PATH, POISON_LIB_PATH, TIMELINE_LIB_PATH,
    SGEMM_KERNEL_MFMA, SGEMM_KERNEL_VALU, SGEMM_OP_N, SGEMM_OP_T, SGEMM_SCRATCH_BYTES,
    ACTIVATIONS, GATED_AUTO, GATED_PRODUCTS, GATED_ROWS, GATED_TILES, SgemmEpilogue, SgemmGate, SgemmTensor,
)
from .ops import (  # noqa: F401
    E4M3_MAX, activation_grad, gemm_e4m3, quantize_e4m3, rmsnorm, rmsnorm_backward, rmsnorm_e4m3,
    sgemm_epilogue, sgemm_epilogue_backward,
)
from .layers import (  # noqa: F401
    clip_grad_norm, gated_grad, gemm_e4m3_gated, grad_norm, layernorm, layernorm_backward, layernorm_e4m3,
    sgemm_gated, sgemm_gated_backward,
)
