// rope_table.h -- the entries of the rotation kernels' tables (heads.h). Packs
// of one element hold no pair, so their two forms are one kernel.
#pragma once

#define ROPE_ADJ(E) ((E) > 1)
#define ROPE_FORMS(T, E, F)                                                                             \
    {(const void *)rms_rope_fwd<T, E, false, F>, (const void *)rms_rope_fwd<T, E, ROPE_ADJ(E), F>}
#define ROPE_KERNELS(T, E)                                                                              \
    {                                                                                                   \
        E, {ROPE_FORMS(T, E, 0), ROPE_FORMS(T, E, 1), ROPE_FORMS(T, E, 2)},                             \
            {rope_fwd_smem<E>(0, sizeof(T)), rope_fwd_smem<E>(1, sizeof(T)), rope_fwd_smem<E>(2, sizeof(T))},  \
            {(const void *)rms_rope_bwd<T, E, false>, (const void *)rms_rope_bwd<T, E, ROPE_ADJ(E)>},   \
            rope_bwd_smem<E>(sizeof(T))                                                                 \
    }
