// Rotation kernels of fp32 heads (rope.cuh), and the sum of the partial dw.
#include "rope.cuh"
#include "rope_table.h"

namespace rmsk {

// Sums the partial rows of dw, blockIdx.y = 0 the q heads' (rows 0 to
// ctas_q - 1), 1 the k heads', in a fixed order: thread (tx, ty) adds rows ty,
// ty + 32, ... of column 32 blockIdx.x + tx, then the 32 sums in ty order.
__global__ void __launch_bounds__(1024) rope_dw_reduce(const float *partial, int ctas_q, int ctas, int D,
                                                       float *dwq, float *dwk)
{
    __shared__ float sm[32][33];
    griddep_wait();
    griddep_launch_dependents();
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5, col = blockIdx.x * 32 + tx;
    const int from = blockIdx.y ? ctas_q : 0, to = blockIdx.y ? ctas : ctas_q;
    float *dw = blockIdx.y ? dwk : dwq;
    if (dw == nullptr)
        return;
    float s = 0.f;
    if (col < D)
#pragma unroll 4
        for (int i = from + ty; i < to; i += 32)
            s += __ldcg(partial + (int64_t)i * D + col);
    sm[ty][tx] = s;
    __syncthreads();
    if (ty == 0 && col < D) {
        float t = 0.f;
#pragma unroll
        for (int q = 0; q < 32; ++q)
            t += sm[q][tx];
        dw[col] = t;
    }
}

const RopeSet rope_f32 = {2, {ROPE_KERNELS(float, 4), ROPE_KERNELS(float, 1)}};
const void *const rope_dw_kernel = (const void *)rope_dw_reduce;

} // namespace rmsk
