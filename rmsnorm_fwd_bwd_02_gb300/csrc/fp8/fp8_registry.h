// fp8_registry.h -- the product's instantiations, which the host code in
// fp8_api.cu picks from.
#pragma once

namespace rmsk {

// fn[columns: 16, 32, 64 tokens, 128 features][RMSNORM_F32, BF16, F16 output]
struct Fp8GemmKernels {
    const void *fn[4][3];
};
extern const Fp8GemmKernels fp8_gemm_kernels;

// fn[RMSNORM_F32, BF16, F16 output]
struct Fp8PairKernels {
    const void *fn[3];
};
extern const Fp8PairKernels fp8_pair_kernels;

} // namespace rmsk
