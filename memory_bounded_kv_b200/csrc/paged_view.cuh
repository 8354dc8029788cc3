// The kernels' view of a paged cache (layout: paged.cuh).
#pragma once

#include "common.cuh"

namespace kvb {

constexpr int kPageSlots = 64;

struct PagedCache {
    uint16_t* k;       // [P, kPageSlots, d]
    uint16_t* v;
    float* lb;         // [P, kPageSlots] or null
    int* pos;          // [P, kPageSlots]
    int* table;        // [B, Hkv, max_pages]
    int* len;          // [B, Hkv]
    int* free_pages;   // [P]
    int* free_count;   // [1]
    int Hkv, d, max_pages, num_pages;
};

// The page holding logical page j of row bg, or -1 (recording KVB_DERR_RANGE) when the table
// names no page of the pool.
__device__ __forceinline__ int page_of(const PagedCache& c, size_t bg, int j) {
    const int pg = c.table[bg * c.max_pages + j];
    if (pg < 0 || pg >= c.num_pages) {
        raise_error(KVB_DERR_RANGE);
        return -1;
    }
    return pg;
}

}  // namespace kvb
