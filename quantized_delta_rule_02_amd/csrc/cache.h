// Launchers of the quantised row cache (cache.hip), called by the C ABI (mix_api.cpp).
#pragma once
#include "runs.h"

namespace sq {

constexpr int kCacheMaxGroup = 1024;

struct CacheParams {
    int32_t dtype, format, d, group;
    int64_t n_rows, n_slots, row_bytes;
    Rows x;                          // rows written, or read back
    const int32_t* slots;            // [n_rows] or NULL: row i has slot i
    uint8_t* codes;                  // [n_slots][row_bytes]
    float* scales;                   // [n_slots][d / group]
};

// `vec`: d and group are multiples of 8, rows allow 16-byte accesses (two for float32), codes 8-byte (4-bit codes: 4-byte) ones.
hipError_t launch_cache_write(const CacheParams& p, bool vec, hipStream_t s);
hipError_t launch_cache_read(const CacheParams& p, bool vec, hipStream_t s);

}  // namespace sq
