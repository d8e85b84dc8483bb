// Attention over a 4-bit cache for pieces of prompts (kv4_prompt.cuh): bf16 and
// fp16, heads of 64 and 128 features.
#include "kv4_prompt.cuh"

namespace rmsk {

const Kv4PromptKernels kv4_prompt_kernels = {
    {{(const void *)kv4_prompt<bf16, 64>, (const void *)kv4_prompt<bf16, 128>},
     {(const void *)kv4_prompt<f16, 64>, (const void *)kv4_prompt<f16, 128>}},
    {(int)PromptLayout<64>::total, (int)PromptLayout<128>::total},
    kPromptRows,
    kPromptThreads};

} // namespace rmsk
