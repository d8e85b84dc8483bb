// Rotation kernels of bf16 heads (rope.cuh).
#include "rope.cuh"
#include "rope_table.h"

namespace rmsk {
const RopeSet rope_bf16 = {3,
                           {ROPE_KERNELS(bf16, 8), ROPE_KERNELS(bf16, 4), ROPE_KERNELS(bf16, 1)}};
} // namespace rmsk
