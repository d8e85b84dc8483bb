// 8-bit rows and blocks (fp8_rows.cuh) of bf16 tensors. Per mode: rows that
// share a warp, a CTA a row (few rows; rows of up to 5120 columns for 16-bit
// types; wider ones), 16-byte packs; loose packs with rows that
// share a warp and with a CTA a row.
// The quantisation of 16-byte packs uses 512 threads at most; its bound of 576
// holds it to 56 registers, with which three CTAs of 352 threads share an SM
// (8548 x 10984 bf16 48 us, 51 with 57 registers and two).
#include "fp8_rows.cuh"

namespace rmsk {

const Fp8RowSet fp8_rows_bf16 = {
    {
        {RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 16, 1, 8, 256, 4, true, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 16, 1, 16, 256, 4, true, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 16, 1, 32, 256, 4, true, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 16, 2, 32, 256, 3, true, false, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 16, 1, 0, 1024, 1, false, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 16, 2, 0, 160, 4, true, false, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 16, 2, 0, 512, 1, true, false, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 8, 4, 0, 576, 2, true, false, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 8, 1, 16, 256, 4, true, true, true),
         RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 8, 2, 32, 256, 4, true, true, true),
         RMSK_FP8_ROWS(bf16, kFp8ModeQuant, 8, 2, 0, 1024, 1, true, true, true)},
        {RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 16, 1, 8, 256, 4, true, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 16, 1, 16, 256, 4, true, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 16, 1, 32, 256, 4, true, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 16, 2, 32, 256, 3, true, false, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 16, 1, 0, 1024, 1, false, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 16, 2, 0, 160, 4, true, false, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 16, 2, 0, 512, 2, true, false, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 8, 4, 0, 512, 1, true, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 8, 1, 16, 256, 4, true, true, true),
         RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 8, 2, 32, 256, 4, true, true, true),
         RMSK_FP8_ROWS(bf16, kFp8ModeNorm, 8, 2, 0, 1024, 1, true, true, true)},
        {RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 16, 1, 8, 256, 4, false, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 16, 1, 16, 256, 4, false, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 16, 1, 32, 256, 4, false, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 16, 2, 32, 256, 2, false, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 16, 1, 0, 1024, 1, false, true, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 16, 2, 0, 160, 4, false, false, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 16, 2, 0, 1024, 1, false, false, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 8, 4, 0, 512, 2, false, false, false),
         RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 8, 1, 16, 256, 4, false, true, true),
         RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 8, 2, 32, 256, 4, false, true, true),
         RMSK_FP8_ROWS(bf16, kFp8ModeResidual, 8, 2, 0, 1024, 1, false, true, true)},
    },
    {(const void *)&rms_fp8_blocks<bf16, 16, false>,
     (const void *)&rms_fp8_blocks<bf16, 8, false>,
     (const void *)&rms_fp8_blocks<bf16, 8, true>},
    {16, 8, 8}};

} // namespace rmsk
