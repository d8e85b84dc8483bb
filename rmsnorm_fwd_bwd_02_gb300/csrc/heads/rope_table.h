// rope_table.h -- the entries of the rotation kernels' tables (heads.h). Packs
// of one element hold no pair, so their two forms are one kernel.
#pragma once

#define ROPE_ADJ(E) ((E) > 1)
#define ROPE_KERNELS(T, E)                                                                              \
    {                                                                                                   \
        E,                                                                                              \
            {(const void *)rms_rope_fwd<T, E, false, false>,                                            \
             (const void *)rms_rope_fwd<T, E, ROPE_ADJ(E), false>},                                     \
            {(const void *)rms_rope_fwd<T, E, false, true>,                                             \
             (const void *)rms_rope_fwd<T, E, ROPE_ADJ(E), true>},                                      \
            {(const void *)rms_rope_bwd<T, E, false>, (const void *)rms_rope_bwd<T, E, ROPE_ADJ(E)>}    \
    }
