// Rows of a 4-bit cache as 8-bit rows (kv4_read): the codes' values and the
// scales as e4m3, both exact.
#include "rope.cuh"

namespace rmsk {

// e2m1 code -> e4m3 byte: 0 .5 1 1.5 2 3 4 6 and their negatives.
__device__ __forceinline__ uint32_t e4m3_of(uint32_t code)
{
    // e4m3 bytes of the eight magnitudes, one table word per four codes
    const uint32_t t = code & 4u ? 0x4C484440u : 0x3C383000u;
    return ((t >> (8u * (code & 3u))) & 0xFFu) | ((code & 8u) << 4);
}

// A thread a group of 16: eight code bytes to sixteen values, keys or values.
__global__ void __launch_bounds__(256) kv4_read(Kv4ReadParams p)
{
    griddep_wait();
    griddep_launch_dependents();
    const int G = p.D / kKv4Group;
    const int64_t per = 2 * (int64_t)p.heads * G, total = p.n * per;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
        const int64_t row = i / per;
        int rest = (int)(i - row * per);
        const bool is_v = rest >= p.heads * G;
        rest -= is_v ? p.heads * G : 0;
        const int h = rest / G, g = rest - h * G;
        const int64_t slot = ld_index(p.slots, row, p.slot64);
        uint2 c = make_uint2(0, 0);
        uint8_t s = 0;
        if (slot >= 0 && slot < p.limit) {
            const int64_t page = slot / p.page_size;
            const int within = (int)(slot - page * p.page_size), t = within % kKv4Tile;
            const uint8_t *tile = p.cache + ((page * p.heads + h) * (p.page_size / kKv4Tile) + within / kKv4Tile) *
                                                kv4_tile_bytes(p.D);
            c = *reinterpret_cast<const uint2 *>(is_v ? tile + kv4_v(p.D) + g * 128 + t * 8
                                                      : tile + t * (p.D / 2) + g * 8);
            s = is_v ? tile[kv4_vscale(p.D) + g * 16 + t] : tile[kv4_kscale(p.D) + t * G + g];
        }
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t half = ((j & 2 ? c.y : c.x) >> (16 * (j & 1))) & 0xFFFFu;
            w[j] = e4m3_of(half & 15u) | e4m3_of((half >> 4) & 15u) << 8 | e4m3_of((half >> 8) & 15u) << 16 |
                   e4m3_of(half >> 12) << 24;
        }
        const int64_t at = (row * p.heads + h) * G + g;
        st_row_v4((is_v ? p.v : p.k) + at * 16, make_uint4(w[0], w[1], w[2], w[3]));
        (is_v ? p.vs : p.ks)[at] = s;
    }
}

const void *const kv4_read_kernel = (const void *)kv4_read;

} // namespace rmsk
