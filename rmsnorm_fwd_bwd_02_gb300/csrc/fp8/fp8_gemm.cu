// The product of two 8-bit tensors with block scales (fp8_gemm.cuh).
#include "fp8_gemm.cuh"
#include "fp8_registry.h"

namespace rmsk {

#define RMSK_FP8_GEMM(BN, SWAP)                                                      \
    {(const void *)&rms_fp8_gemm<float, BN, SWAP>, (const void *)&rms_fp8_gemm<bf16, BN, SWAP>, \
     (const void *)&rms_fp8_gemm<f16, BN, SWAP>}

const Fp8GemmKernels fp8_gemm_kernels = {{RMSK_FP8_GEMM(16, true), RMSK_FP8_GEMM(32, true),
                                          RMSK_FP8_GEMM(64, true), RMSK_FP8_GEMM(128, false)}};

} // namespace rmsk
