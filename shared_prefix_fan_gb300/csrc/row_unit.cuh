// row_unit.cuh -- a unit of a row plan (windowed or 4-bit attention) as attn_rows.cu
// reads it: the first keys it sweeps in front of its own range, where that range's
// tiles begin, and the check of a page id before it is read through.
#pragma once

#include "fanout_internal.h"

namespace fanout {

// Tiles of a unit's own range start at a page: key_begin itself may lie inside
// one (the oldest key a window leaves visible), and the keys of that page before
// it are loaded with it, masked, and zeroed.
__device__ __forceinline__ int range_begin(const Unit& u, int page_size) {
    return u.key_begin & ~(page_size - 1);
}
__device__ __forceinline__ int range_tiles(const Unit& u, int page_size) {
    return (u.key_end - range_begin(u, page_size) + kBN - 1) / kBN;
}
// First key of a unit's run of first keys: keys before split_at belong to the
// shared range, so a unit behind it starts there.
__device__ __forceinline__ int first_begin(const Unit& u, int split_at) {
    return u.key_begin >= split_at ? split_at : 0;
}
__device__ __forceinline__ int first_tiles(const Unit& u, int split_at) {
    return u.pos_base > 0 ? (u.pos_base - first_begin(u, split_at) + kBN - 1) / kBN : 0;
}

// A page id outside the pool is recorded and page 0 read in its place: the
// call's result is then unspecified, but nothing outside the pool is touched.
__device__ __forceinline__ int32_t checked_page(const SplitParams& p, int32_t page) {
    if (page >= 0 && page < p.num_pages) return page;
    atomicCAS(p.err, 0, 1);  // FANOUT_EINVAL
    return 0;
}

}  // namespace fanout
