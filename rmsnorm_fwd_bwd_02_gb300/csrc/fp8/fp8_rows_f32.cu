// 8-bit rows and blocks (fp8_rows.cuh) of fp32 tensors.
#include "fp8_rows.cuh"

namespace rmsk {

const Fp8RowSet fp8_rows_f32 = {
    {RMSK_FP8_ROWS(float, 8, 1, 16, 256, 4, true, true, false),
     RMSK_FP8_ROWS(float, 8, 1, 32, 256, 4, true, true, false),
     RMSK_FP8_ROWS(float, 8, 2, 32, 256, 3, true, true, false),
     RMSK_FP8_ROWS(float, 8, 2, 0, 1024, 1, false, true, false),
     RMSK_FP8_ROWS(float, 8, 2, 0, 512, 2, true, false, false),
     RMSK_FP8_ROWS(float, 8, 4, 0, 512, 1, true, false, false),
     RMSK_FP8_ROWS(float, 4, 4, 0, 1024, 1, false, false, false),
     RMSK_FP8_ROWS(float, 4, 4, 0, 1024, 1, false, false, true)},
    {(const void *)&rms_fp8_blocks<float, 8, false>, (const void *)&rms_fp8_blocks<float, 4, false>,
     (const void *)&rms_fp8_blocks<float, 4, true>},
    {8, 4, 4}};

} // namespace rmsk
