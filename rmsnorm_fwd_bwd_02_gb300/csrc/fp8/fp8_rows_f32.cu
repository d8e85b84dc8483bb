// 8-bit rows and blocks (fp8_rows.cuh) of fp32 tensors. Per mode: rows that
// share a warp, a CTA a row (few rows; rows of up to 5120 columns for 16-bit
// types; wider ones), 16-byte packs; loose packs with rows that
// share a warp and with a CTA a row.
#include "fp8_rows.cuh"

namespace rmsk {

const Fp8RowSet fp8_rows_f32 = {
    {
        {RMSK_FP8_ROWS(float, kFp8ModeQuant, 8, 1, 16, 256, 4, true, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeQuant, 8, 1, 32, 256, 4, true, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeQuant, 8, 2, 32, 256, 3, true, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeQuant, 8, 4, 32, 256, 2, false, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeQuant, 8, 2, 0, 1024, 1, false, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeQuant, 8, 2, 0, 512, 2, true, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeQuant, 8, 4, 0, 512, 1, true, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeQuant, 4, 4, 0, 1024, 1, false, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeQuant, 4, 1, 32, 256, 4, true, true, true),
         RMSK_FP8_ROWS(float, kFp8ModeQuant, 4, 4, 32, 256, 3, true, true, true),
         RMSK_FP8_ROWS(float, kFp8ModeQuant, 4, 4, 0, 1024, 1, true, false, true)},
        {RMSK_FP8_ROWS(float, kFp8ModeNorm, 8, 1, 16, 256, 4, true, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeNorm, 8, 1, 32, 256, 4, true, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeNorm, 8, 2, 32, 256, 3, true, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeNorm, 8, 4, 32, 256, 2, false, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeNorm, 8, 2, 0, 1024, 1, false, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeNorm, 8, 2, 0, 512, 2, true, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeNorm, 8, 4, 0, 512, 1, true, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeNorm, 4, 4, 0, 1024, 1, false, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeNorm, 4, 1, 32, 256, 4, true, true, true),
         RMSK_FP8_ROWS(float, kFp8ModeNorm, 4, 4, 32, 256, 3, true, true, true),
         RMSK_FP8_ROWS(float, kFp8ModeNorm, 4, 4, 0, 1024, 1, true, false, true)},
        {RMSK_FP8_ROWS(float, kFp8ModeResidual, 8, 1, 16, 256, 4, false, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeResidual, 8, 1, 32, 256, 4, false, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeResidual, 8, 2, 32, 256, 3, false, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeResidual, 8, 4, 32, 256, 2, false, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeResidual, 8, 2, 0, 1024, 1, false, true, false),
         RMSK_FP8_ROWS(float, kFp8ModeResidual, 8, 2, 0, 512, 2, false, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeResidual, 8, 4, 0, 512, 1, false, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeResidual, 4, 4, 0, 1024, 1, false, false, false),
         RMSK_FP8_ROWS(float, kFp8ModeResidual, 4, 1, 32, 256, 4, false, true, true),
         RMSK_FP8_ROWS(float, kFp8ModeResidual, 4, 4, 32, 256, 3, false, true, true),
         RMSK_FP8_ROWS(float, kFp8ModeResidual, 4, 4, 0, 1024, 1, false, false, true)},
    },
    {(const void *)&rms_fp8_blocks<float, 8, false>,
     (const void *)&rms_fp8_blocks<float, 4, false>,
     (const void *)&rms_fp8_blocks<float, 4, true>},
    {8, 4, 4}};

} // namespace rmsk
