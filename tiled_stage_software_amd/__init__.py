"""libgemm for AMD MI355X (gfx950): tiled, software-pipelined GEMM with hand-written HIP
kernels behind a C ABI (include/libgemm.h).  This package holds the HIP sources
(csrc/), the in-tree build (build.py), the ctypes binding (libgemm.py), the torch forms of the
operators around the products (ops.py) and the seeded input generators (inputs.py)."""
from .libgemm import (GEMM_OK, GEMM_ERR_INVALID_ARG, GEMM_ERR_UNSUPPORTED, GEMM_ERR_HIP,  # noqa: F401
                      GEMM_ROW_MAJOR, GEMM_COL_MAJOR, GEMM_F32, GEMM_BF16, GEMM_F16, GEMM_F8E4M3,
                      GEMM_KERNEL_AUTO, GEMM_KERNEL_VALU_RING, GEMM_KERNEL_VALU_STAGED,
                      GEMM_KERNEL_MFMA_RING, GEMM_KERNEL_MFMA_STAGED, GEMM_KERNEL_SCALE,
                      GEMM_ACT_NONE, GEMM_ACT_RELU, GEMM_ACT_GELU, GEMM_ACT_GELU_TANH, GEMM_ACT_SILU,
                      GEMM_ROPE_HALVES, GEMM_ROPE_NEIGHBOURS,
                      GemmError, GemmHeads, GemmOpts, GemmPlan, GemmRope, matmul, load)
from . import ops  # noqa: F401
