// 8-bit rows and blocks (fp8_rows.cuh) of fp32 tensors.
#include "fp8_rows.cuh"

namespace rmsk {

const Fp8RowSet fp8_rows_f32 = {
    {RMSK_FP8_ROWS(float, 8, 1, 2, 16, 256, 2), RMSK_FP8_ROWS(float, 8, 1, 2, 32, 256, 2),
     RMSK_FP8_ROWS(float, 8, 2, 1, 32, 256, 2), RMSK_FP8_ROWS(float, 8, 2, 1, 0, 1024, 1),
     RMSK_FP8_ROWS(float, 8, 2, 1, 0, 1024, 1), RMSK_FP8_ROWS(float, 8, 4, 1, 0, 512, 1),
     RMSK_FP8_ROWS(float, 4, 4, 1, 0, 1024, 1), RMSK_FP8_ROWS(float, 1, 16, 1, 0, 1024, 1)},
    {(const void *)&rms_fp8_blocks<float, 8>, (const void *)&rms_fp8_blocks<float, 4>,
     (const void *)&rms_fp8_blocks<float, 1>},
    {8, 4, 1}};

} // namespace rmsk
