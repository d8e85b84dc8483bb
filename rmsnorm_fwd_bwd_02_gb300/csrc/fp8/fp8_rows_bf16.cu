// 8-bit rows and blocks (fp8_rows.cuh) of bf16 tensors.
#include "fp8_rows.cuh"

namespace rmsk {

const Fp8RowSet fp8_rows_bf16 = {
    {RMSK_FP8_ROWS(bf16, 16, 1, 8, 256, 4, true, true, false),
     RMSK_FP8_ROWS(bf16, 16, 1, 16, 256, 4, true, true, false),
     RMSK_FP8_ROWS(bf16, 16, 1, 32, 256, 4, true, true, false),
     RMSK_FP8_ROWS(bf16, 16, 1, 0, 1024, 1, false, true, false),
     RMSK_FP8_ROWS(bf16, 16, 2, 0, 256, 3, true, false, false),
     RMSK_FP8_ROWS(bf16, 16, 2, 0, 512, 1, true, false, false),
     RMSK_FP8_ROWS(bf16, 8, 2, 0, 1024, 1, true, false, false),
     RMSK_FP8_ROWS(bf16, 4, 4, 0, 1024, 1, false, false, true)},
    {(const void *)&rms_fp8_blocks<bf16, 16, false>, (const void *)&rms_fp8_blocks<bf16, 8, false>,
     (const void *)&rms_fp8_blocks<bf16, 4, true>},
    {16, 8, 4}};

} // namespace rmsk
