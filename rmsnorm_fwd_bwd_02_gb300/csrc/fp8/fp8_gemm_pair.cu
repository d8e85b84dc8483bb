// The product of two 8-bit tensors by pairs of CTAs (fp8_gemm_pair.cuh).
#include "fp8_gemm_pair.cuh"
#include "fp8_registry.h"

namespace rmsk {

const Fp8PairKernels fp8_pair_kernels = {{(const void *)&rms_fp8_gemm_pair<float>,
                                          (const void *)&rms_fp8_gemm_pair<bf16>,
                                          (const void *)&rms_fp8_gemm_pair<f16>}};

} // namespace rmsk
