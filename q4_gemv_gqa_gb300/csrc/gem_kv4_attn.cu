// gem_kv4_attn.cu — grouped-query attention over the paged 4-bit KV cache.
#include <cmath>

#include "gem_device.cuh"
#include "gem_kv4.cuh"

namespace gem {
namespace kv4 {
namespace {

constexpr int kMaxGroup = 8;

struct AttnParams {
    const float* q;
    int64_t ldq, T;
    const int32_t *cu, *kv_len;
    int B, n_q, n_kv, G;
    const int32_t* table;
    int64_t max_pages;
    const uint8_t* pool;
    int64_t n_pages;
    int page, lpage, window;
    float scale;
    float* out;
    int64_t ldo;
    int* status;
};

// One CTA per (query row, KV head), one cached position per warp at a time, the lanes across d.
template <int D>
__global__ void __launch_bounds__(128) kv4_attn_rows_kernel(const AttnParams P) {
    constexpr int kWarps = 4, E = D / 32;
    __shared__ float qs[kMaxGroup][D];
    __shared__ float acc_s[kMaxGroup][D];
    __shared__ float ml[kWarps][kMaxGroup][2];
    __shared__ int found;
    pdl_wait_trigger();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    const int h = blockIdx.y;
    if (threadIdx.x == 0) found = -1;
    __syncthreads();
    for (int b = threadIdx.x; b < P.B; b += blockDim.x) {
        const int64_t c0 = P.cu[b], c1 = P.cu[b + 1], L = P.kv_len[b];
        const bool ok = c0 >= 0 && c0 <= c1 && c1 <= P.T && L >= c1 - c0 && L <= P.max_pages * P.page;
        if (!ok) {
            if (t == 0 && h == 0) atomicOr(P.status, GEM_DEVFLAG_POS_RANGE);
        } else if (c0 <= t && t < c1) {
            atomicMax(&found, b);
        }
    }
    __syncthreads();
    const int b = found;
    if (b < 0) return;
    const int p = P.kv_len[b] - P.cu[b + 1] + static_cast<int>(t);
    const int first = P.window ? max(0, p - P.window + 1) : 0;
    for (int i = threadIdx.x; i < P.G * D; i += blockDim.x)
        qs[i / D][i % D] = P.q[t * P.ldq + static_cast<int64_t>(h) * P.G * D + i] * P.scale;
    __syncthreads();
    float m[kMaxGroup], l[kMaxGroup], acc[kMaxGroup][E];
#pragma unroll
    for (int g = 0; g < kMaxGroup; ++g) {
        m[g] = -INFINITY, l[g] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[g][e] = 0.f;
    }
    const int page_tiles = P.page / kTileTokens;
    for (int j = first + w; j <= p; j += kWarps) {
        const int32_t id = P.table[b * P.max_pages + (j >> P.lpage)];
        if (id < 0 || id >= P.n_pages) {
            if (lane == 0) atomicOr(P.status, GEM_DEVFLAG_PAGE_RANGE);
            continue;
        }
        const uint8_t* tile = P.pool + ((static_cast<int64_t>(id) * P.n_kv + h) * page_tiles +
                                        (j & (P.page - 1)) / kTileTokens) * tile_bytes(D);
        const int row = j % kTileTokens;
        float kv[2][E];
#pragma unroll
        for (int which = 0; which < 2; ++which)
#pragma unroll
            for (int e = 0; e < E; ++e) {   // element 32 e + lane
                const int at = e * kTileTokens + row;
                const uint32_t byte = tile[codes_off(D, which) + at * 16 + (lane & 15)];
                const float s = __half2float(reinterpret_cast<const __half*>(tile + scales_off(D, which))[at]);
                kv[which][e] = static_cast<float>(static_cast<int>(lane < 16 ? byte & 15 : byte >> 4) - 8) * s;
            }
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) {
            if (g >= P.G) break;
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(qs[g][e * 32 + lane], kv[0][e], s);
            s = warp_sum(s);
            const float mn = fmaxf(m[g], s);
            const float corr = m[g] == mn ? 1.f : expf(m[g] - mn), pr = s == -INFINITY ? 0.f : expf(s - mn);
            m[g] = mn;
            l[g] = l[g] * corr + pr;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[g][e] = fmaf(pr, kv[1][e], acc[g][e] * corr);
        }
    }
    for (int g = 0; g < P.G; ++g)
        for (int e = threadIdx.x; e < D; e += blockDim.x) acc_s[g][e] = 0.f;
    if (lane == 0) {
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) ml[w][g][0] = m[g], ml[w][g][1] = l[g];
    }
    __syncthreads();
    for (int k = 0; k < kWarps; ++k) {   // the warps add their share in order
#pragma unroll
        for (int g = 0; g < kMaxGroup; ++g) {
            if (w != k || g >= P.G) break;
            float mx = -INFINITY;
            for (int i = 0; i < kWarps; ++i) mx = fmaxf(mx, ml[i][g][0]);
            const float c = m[g] == mx ? 1.f : expf(m[g] - mx);
#pragma unroll
            for (int e = 0; e < E; ++e) acc_s[g][e * 32 + lane] += c * acc[g][e];
        }
        __syncthreads();
    }
    for (int i = threadIdx.x; i < P.G * D; i += blockDim.x) {
        const int g = i / D, e = i % D;
        float mx = -INFINITY, den = 0.f;
        for (int k = 0; k < kWarps; ++k) mx = fmaxf(mx, ml[k][g][0]);
        for (int k = 0; k < kWarps; ++k) den += (ml[k][g][0] == mx ? 1.f : expf(ml[k][g][0] - mx)) * ml[k][g][1];
        P.out[t * P.ldo + static_cast<int64_t>(h) * P.G * D + i] = den == 0.f ? 0.f : acc_s[g][e] / den;
    }
}

}  // namespace
}  // namespace kv4
}  // namespace gem

extern "C" {

size_t gem_kv4_attn_workspace(int64_t T, int B, int n_q, int n_kv, int d) {
    (void)T, (void)B, (void)n_q, (void)n_kv, (void)d;
    return 0;
}

gem_status gem_kv4_attn(const float* q, int64_t ldq, int64_t T, const int32_t* cu_tokens, const int32_t* kv_len,
                        int B, int n_q, int n_kv, int d, const int32_t* table, int64_t max_pages,
                        const void* pool, int64_t n_pages, int page, int window, float scale, float* out,
                        int64_t ldo, void* workspace, size_t ws_bytes, int32_t* status, void* stream) {
    using namespace gem;
    using namespace gem::kv4;
    gem_status st = pool_check(pool, n_pages, page, n_kv, d);
    if (st != GEM_OK) return st;
    if (T < 0 || B < 0 || n_q < 0 || max_pages < 0 || window < 0) return GEM_ERR_INVALID_ARG;
    if (n_kv == 0 ? n_q != 0 : n_q % n_kv != 0) return GEM_ERR_INVALID_ARG;
    if (B > kMaxRequests || T > INT32_MAX || max_pages > (INT32_MAX - 255) / page ||
        (n_kv && n_q / n_kv > kMaxGroup))
        return GEM_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || B == 0 || n_q == 0) return GEM_OK;
    if (!q || !out || !cu_tokens || !kv_len || (max_pages && !table)) return GEM_ERR_INVALID_ARG;
    if (ldq < static_cast<int64_t>(n_q) * d || ldo < static_cast<int64_t>(n_q) * d) return GEM_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) & 15) || ldq % 4) return GEM_ERR_MISALIGNED;
    (void)workspace, (void)ws_bytes;
    AttnParams P{};
    P.q = q, P.ldq = ldq, P.T = T, P.cu = cu_tokens, P.kv_len = kv_len;
    P.B = B, P.n_q = n_q, P.n_kv = n_kv, P.G = n_q / n_kv;
    P.table = table, P.max_pages = max_pages, P.pool = static_cast<const uint8_t*>(pool), P.n_pages = n_pages;
    P.page = page, P.lpage = log2_of(page), P.window = window, P.scale = scale;
    P.out = out, P.ldo = ldo, P.status = status;
    if ((st = flag_word(&P.status)) != GEM_OK) return st;
    const void* kernel = d == 64    ? reinterpret_cast<const void*>(kv4_attn_rows_kernel<64>)
                         : d == 128 ? reinterpret_cast<const void*>(kv4_attn_rows_kernel<128>)
                         : d == 256 ? reinterpret_cast<const void*>(kv4_attn_rows_kernel<256>)
                                    : reinterpret_cast<const void*>(kv4_attn_rows_kernel<512>);
    void* args[] = {&P};
    return launch_pdl(kernel, dim3(static_cast<unsigned>(T), static_cast<unsigned>(n_kv)), dim3(128), 0,
                      static_cast<cudaStream_t>(stream), args);
}

}  // extern "C"
