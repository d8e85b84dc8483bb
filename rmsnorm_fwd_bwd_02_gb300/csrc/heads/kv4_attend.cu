// Attention over a 4-bit cache (kv4_attend.cuh): bf16 and fp16, 8 query rows a
// tile, with heads of 128 features 16 too.
#include "kv4_attend.cuh"

namespace rmsk {

#define KV4(F, T)                                                                                       \
    {                                                                                                   \
        {(const void *)F<T, 64, 1>, nullptr},                                                           \
        {(const void *)F<T, 128, 1>, (const void *)F<T, 128, 2>}                                        \
    }
const Kv4Kernels kv4_kernels = {{KV4(kv4_attend, bf16), KV4(kv4_attend, f16)},
                                {KV4(kv4_combine, bf16), KV4(kv4_combine, f16)}};

} // namespace rmsk
