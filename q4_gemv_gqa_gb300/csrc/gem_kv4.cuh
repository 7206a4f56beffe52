// gem_kv4.cuh — layout of the paged 4-bit KV cache (see include/gem.h) and its host checks.
#pragma once

#include "gem_internal.h"

namespace gem {
namespace kv4 {

constexpr int kTileTokens = 16;
constexpr int kMaxRequests = 4096;

// A tile holds 16 tokens of one KV head: K codes, V codes, K scales, V scales (18 d bytes).
__host__ __device__ constexpr int tile_bytes(int d) { return 18 * d; }
__host__ __device__ constexpr int codes_off(int d, int which) { return which * 8 * d; }
__host__ __device__ constexpr int scales_off(int d, int which) { return 16 * d + which * d; }

inline bool page_ok(int page) { return page == 16 || page == 32 || page == 64 || page == 128 || page == 256; }
inline int log2_of(int v) {
    int l = 0;
    while ((1 << l) < v) ++l;
    return l;
}
inline bool head_dim_ok(int d) { return d == 64 || d == 128 || d == 256 || d == 512; }

// The checks that every call on a pool makes.
inline gem_status pool_check(const void* pool, int64_t n_pages, int page, int n_kv, int d) {
    if (n_kv < 0 || d <= 0 || n_pages < 0) return GEM_ERR_INVALID_ARG;
    if (!head_dim_ok(d) || !page_ok(page) || n_pages > (INT32_MAX - 255) / page || n_kv > 65535)
        return GEM_ERR_UNSUPPORTED_SHAPE;
    if (n_pages && n_kv && !pool) return GEM_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(pool) & 15) return GEM_ERR_MISALIGNED;
    return GEM_OK;
}

// status, or the library's flag word of the current device when the caller gave none
inline gem_status flag_word(int32_t** status) {
    if (*status) return GEM_OK;
    DeviceInfo di;
    const gem_status st = device_info(&di);
    if (st == GEM_OK) *status = di.status_word;
    return st;
}

}  // namespace kv4
}  // namespace gem
