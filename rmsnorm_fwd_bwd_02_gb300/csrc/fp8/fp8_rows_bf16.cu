// 8-bit rows and blocks (fp8_rows.cuh) of bf16 tensors.
#include "fp8_rows.cuh"

namespace rmsk {

const Fp8RowSet fp8_rows_bf16 = {
    {RMSK_FP8_ROWS(bf16, 16, 1, 2, 8, 256, 2), RMSK_FP8_ROWS(bf16, 16, 1, 2, 16, 256, 2),
     RMSK_FP8_ROWS(bf16, 16, 1, 2, 32, 256, 2), RMSK_FP8_ROWS(bf16, 16, 1, 1, 0, 1024, 1),
     RMSK_FP8_ROWS(bf16, 16, 2, 1, 0, 512, 2), RMSK_FP8_ROWS(bf16, 16, 4, 2, 0, 256, 2),
     RMSK_FP8_ROWS(bf16, 8, 4, 1, 0, 512, 1), RMSK_FP8_ROWS(bf16, 1, 16, 1, 0, 1024, 1)},
    {(const void *)&rms_fp8_blocks<bf16, 16>, (const void *)&rms_fp8_blocks<bf16, 8>,
     (const void *)&rms_fp8_blocks<bf16, 1>},
    {16, 8, 1}};

} // namespace rmsk
