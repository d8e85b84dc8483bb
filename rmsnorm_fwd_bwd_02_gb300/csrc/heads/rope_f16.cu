// Rotation kernels of fp16 heads (rope.cuh).
#include "rope.cuh"
#include "rope_table.h"

namespace rmsk {
const RopeSet rope_f16 = {3,
                           {ROPE_KERNELS(f16, 8), ROPE_KERNELS(f16, 4), ROPE_KERNELS(f16, 1)}};
} // namespace rmsk
