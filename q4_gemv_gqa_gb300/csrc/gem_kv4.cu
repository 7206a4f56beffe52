// gem_kv4.cu — rows into and out of the paged 4-bit KV cache: quantising append, gather.
#include "gem_device.cuh"
#include "gem_kv4.cuh"

namespace gem {
namespace kv4 {
namespace {

struct RowsParams {
    const float *k, *v;      // append: the rows
    float *ko, *vo;          // gather: the rows (nullable)
    int64_t ldk, ldv, T;
    const int32_t* slot;
    uint8_t* pool;
    int64_t n_slots;
    int n_kv, d, lnb;        // log2 of d / 32
    int lpage;               // log2 of the page size
    int vec_k, vec_v;        // rows may be read or written 16 bytes at a time
    int* status;
};

// Four threads hold one block of 32 values of K and of V: thread u elements 4u .. 4u + 3 and
// 16 + 4u .. 16 + 4u + 3, which are the low and the high nibbles of word u of the block's 16 bytes of
// codes.  The eight blocks of a warp are eight consecutive tokens of one (head, block), so that the codes
// and the scales of a prompt's tokens are written next to one another, and the warps of a CTA have
// consecutive ones, so that it reads whole 1 KB pieces of the rows.
constexpr int kRowThreads = 256;
struct Place {
    int64_t t;
    int u, col;            // column of the row: the block's first plus 4 u
    uint8_t *code, *scale; // K's; V's are 8 d and d bytes on
};

__device__ __forceinline__ bool place_of(const RowsParams& P, Place& o) {
    o.u = threadIdx.x & 3;
    o.t = blockIdx.x * 8ll + ((threadIdx.x >> 2) & 7);
    const int part = blockIdx.y * (kRowThreads / 32) + (threadIdx.x >> 5);
    if (o.t >= P.T || part >= P.n_kv << P.lnb) return false;
    const int head = part >> P.lnb, blk = part & ((1 << P.lnb) - 1);
    o.col = part * 32 + o.u * 4;
    const int32_t s = P.slot[o.t];
    if (s < 0 || s >= P.n_slots) {
        if (s != -1 && part == 0 && o.u == 0) atomicOr(P.status, GEM_DEVFLAG_PAGE_RANGE);
        return false;
    }
    const int lpt = P.lpage - 4;
    const int64_t tile = ((static_cast<int64_t>(s >> P.lpage) * P.n_kv + head) << lpt) + ((s >> 4) & ((1 << lpt) - 1));
    const int at = blk * kTileTokens + s % kTileTokens;
    uint8_t* base = P.pool + tile * tile_bytes(P.d);
    o.code = base + at * 16 + o.u * 4;
    o.scale = base + scales_off(P.d, 0) + at * 2;
    return true;
}

__device__ __forceinline__ void load4(const float* p, bool vec, float (&x)[4]) {
    if (vec) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = p[i];
    }
}

// 8 + rint(x / s), ties to even, clamped to 0..15, decided exactly: the first guess from a
// reciprocal is off by less than one step beyond the nearest code, and x - q s is exact in fp32
// (both are multiples of the smaller of their last places, and the difference is no larger than x).
__device__ __forceinline__ int code_of(float x, float s, float inv) {
    float q = fminf(fmaxf(rintf(x * inv), -9.f), 8.f);   // beyond: clamped to the same codes
    const float r = fmaf(-q, s, x), h = 0.5f * fabsf(s);
    const bool over = fabsf(r) > h, tie = fabsf(r) == h;
    if (over || (tie && (static_cast<int>(q) & 1))) q += (r < 0.f) == (s < 0.f) ? 1.f : -1.f;
    return min(max(static_cast<int>(q) + 8, 0), 15);
}

// NaN where either is
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float d;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// The four low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The codes of a thread's eight values for scale s (not 0), a word.  The common case rounds x / s + 8 by
// adding it to 1.5 * 2^23, whose low byte then is the code (16, a value opposite to the largest, becomes
// 15); it stands where every remainder is below half a step, that is, where no value is on a border or
// within the reciprocal's error of one, and where s is a normal number, so that no ratio is past 8.01.
__device__ __forceinline__ uint32_t word_of(const float (&x)[8], float s) {
    const float inv = 1.0f / s, base = 12582912.f + 8.f;
    float worst = 0.f;
    uint32_t t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float u = fmaf(x[i], inv, base);
        worst = fmaxf(worst, fabsf(fmaf(base - u, s, x[i])));
        t[i] = __float_as_uint(u);
    }
    if (worst < 0.5f * fabsf(s) && fabsf(s) >= 6.103515625e-5f && fabsf(s) < 65504.f) {
        const uint32_t lo = low_bytes(t[0], t[1], t[2], t[3]), hi = low_bytes(t[4], t[5], t[6], t[7]);
        return (lo - (lo >> 4 & 0x01010101u)) | ((hi - (hi >> 4 & 0x01010101u)) << 4);
    }
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w |= static_cast<uint32_t>(code_of(x[i], s, inv) | (code_of(x[4 + i], s, inv) << 4)) << (8 * i);
    return w;
}

// One block's eighth: the largest value of the block by its four threads, the scale, this thread's codes.
__device__ __forceinline__ void quantise(const float (&x)[8], bool live, int u, uint8_t* code, uint8_t* scale) {
    float top = x[0], low = x[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = max_nan(top, x[i]), low = min_nan(low, x[i]);
#pragma unroll
    for (int m = 1; m < 4; m <<= 1) {
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, m));
        low = min_nan(low, __shfl_xor_sync(0xffffffffu, low, m));
    }
    float m = top > -low ? top : low;            // the value of largest magnitude
    const bool both = top == -low && top != 0.f;
    if (__any_sync(0xffffffffu, both)) {         // of either sign: the first of them
        int first = 32;
#pragma unroll
        for (int i = 7; i >= 0; --i)
            if (fabsf(x[i]) == top) first = (i < 4 ? 0 : 16) + u * 4 + (i & 3);
        int at = first;
#pragma unroll
        for (int s = 1; s < 4; s <<= 1) at = min(at, __shfl_xor_sync(0xffffffffu, at, s));
        bool minus = false;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if ((i < 4 ? 0 : 16) + u * 4 + (i & 3) == at) minus = x[i] < 0.f;
        const uint32_t quad = 0xfu << (threadIdx.x & 28);
        const bool any_minus = (__ballot_sync(0xffffffffu, minus) & quad) != 0;
        if (both) m = any_minus ? low : top;
    }
    if (!live) return;
    __half s16;
    uint32_t word = 0x88888888u;
    if (!(fabsf(m) < INFINITY)) {
        s16 = __ushort_as_half(0x7fff);
    } else {
        s16 = __float2half_rn(fminf(fmaxf(m * -0.125f, -65504.f), 65504.f));
        const float s = __half2float(s16);
        if (s != 0.f) word = word_of(x, s);
    }
    *reinterpret_cast<uint32_t*>(code) = word;
    if (u == 0) *reinterpret_cast<__half*>(scale) = s16;
}

// 4095 rows of 2 x 16 x 256 are 134 MB read and 19 MB written in 34.5 us, 4.4 TB/s, 66 % of the measured copy rate:
// bound by the latency of the loads, 64 bytes a thread, and of the chain behind them (extremes, scale, codes), with
// instructions issued in 58 % of the cycles.  K and V of a block in one thread share the slot and the address (a thread for each
// took 36 us, one with two octets of tokens 38).
__global__ void __launch_bounds__(kRowThreads) kv4_append_kernel(const RowsParams P) {
    pdl_wait_trigger();
    Place o{};
    const bool live = place_of(P, o);
    float x[2][8];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        if (live) {
            const float* src = (w ? P.v + o.t * P.ldv : P.k + o.t * P.ldk) + o.col;
            const bool vec = w ? P.vec_v : P.vec_k;
            load4(src, vec, reinterpret_cast<float(&)[4]>(x[w][0]));
            load4(src + 16, vec, reinterpret_cast<float(&)[4]>(x[w][4]));
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[w][i] = 0.f;
        }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w)
        quantise(x[w], live, o.u, o.code + codes_off(P.d, w), o.scale + w * P.d);
}

// The same rows back: 19 MB read, 134 MB written in 25.7 us, 6.0 TB/s, 88 % of the measured copy rate.
__global__ void __launch_bounds__(kRowThreads) kv4_gather_kernel(const RowsParams P) {
    pdl_wait_trigger();
    Place o;
    if (!place_of(P, o)) return;
    uint32_t code[2];
    float s[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        code[w] = *reinterpret_cast<const uint32_t*>(o.code + codes_off(P.d, w));
        s[w] = __half2float(*reinterpret_cast<const __half*>(o.scale + w * P.d));
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
        float* dst = w ? P.vo : P.ko;
        if (!dst) continue;
        dst += o.t * (w ? P.ldv : P.ldk) + o.col;
        float lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            lo[i] = static_cast<float>(static_cast<int>((code[w] >> (8 * i)) & 15) - 8) * s[w];
            hi[i] = static_cast<float>(static_cast<int>((code[w] >> (8 * i + 4)) & 15) - 8) * s[w];
        }
        if (w ? P.vec_v : P.vec_k) {
            *reinterpret_cast<float4*>(dst) = make_float4(lo[0], lo[1], lo[2], lo[3]);
            *reinterpret_cast<float4*>(dst + 16) = make_float4(hi[0], hi[1], hi[2], hi[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) dst[i] = lo[i], dst[16 + i] = hi[i];
        }
    }
}

bool vec_ok(const float* p, int64_t ld) { return !(reinterpret_cast<uintptr_t>(p) & 15) && ld % 4 == 0; }

gem_status rows_launch(const void* kernel, RowsParams& P, cudaStream_t stream) {
    const gem_status st = flag_word(&P.status);
    if (st != GEM_OK) return st;
    const int64_t x = (P.T + 7) / 8, y = ((static_cast<int64_t>(P.n_kv) << P.lnb) + kRowThreads / 32 - 1) / (kRowThreads / 32);
    if (x > INT32_MAX || y > 65535) return GEM_ERR_UNSUPPORTED_SHAPE;
    void* args[] = {&P};
    return launch_pdl(kernel, dim3(static_cast<unsigned>(x), static_cast<unsigned>(y)), dim3(kRowThreads), 0, stream, args);
}

}  // namespace
}  // namespace kv4
}  // namespace gem

extern "C" {

size_t gem_kv4_page_bytes(int n_kv, int d, int page) {
    if (n_kv <= 0 || n_kv > 65535 || !gem::kv4::head_dim_ok(d) || !gem::kv4::page_ok(page)) return 0;
    return static_cast<size_t>(n_kv) * (page / gem::kv4::kTileTokens) * gem::kv4::tile_bytes(d);
}

gem_status gem_kv4_append(const float* k, int64_t ldk, const float* v, int64_t ldv, int64_t T, int n_kv, int d,
                          const int32_t* slot, void* pool, int64_t n_pages, int page, int32_t* status,
                          void* stream) {
    using namespace gem::kv4;
    const gem_status st = pool_check(pool, n_pages, page, n_kv, d);
    if (st != GEM_OK) return st;
    if (T < 0) return GEM_ERR_INVALID_ARG;
    if (T == 0 || n_kv == 0) return GEM_OK;
    if (!k || !v || !slot || ldk < static_cast<int64_t>(n_kv) * d || ldv < static_cast<int64_t>(n_kv) * d)
        return GEM_ERR_INVALID_ARG;
    RowsParams P{};
    P.k = k, P.v = v, P.ldk = ldk, P.ldv = ldv, P.T = T, P.slot = slot;
    P.pool = static_cast<uint8_t*>(pool);
    P.n_slots = n_pages * page;
    P.n_kv = n_kv, P.d = d, P.lnb = log2_of(d / 32), P.lpage = log2_of(page);
    P.vec_k = vec_ok(k, ldk), P.vec_v = vec_ok(v, ldv);
    P.status = status;
    return rows_launch(reinterpret_cast<const void*>(kv4_append_kernel), P, static_cast<cudaStream_t>(stream));
}

gem_status gem_kv4_gather(const void* pool, int64_t n_pages, int page, int n_kv, int d, const int32_t* slot,
                          int64_t T, float* k, int64_t ldk, float* v, int64_t ldv, int32_t* status,
                          void* stream) {
    using namespace gem::kv4;
    const gem_status st = pool_check(pool, n_pages, page, n_kv, d);
    if (st != GEM_OK) return st;
    if (T < 0) return GEM_ERR_INVALID_ARG;
    if (T == 0 || n_kv == 0 || (!k && !v)) return GEM_OK;
    if (!slot || (k && ldk < static_cast<int64_t>(n_kv) * d) || (v && ldv < static_cast<int64_t>(n_kv) * d))
        return GEM_ERR_INVALID_ARG;
    RowsParams P{};
    P.ko = k, P.vo = v, P.ldk = ldk, P.ldv = ldv, P.T = T, P.slot = slot;
    P.pool = static_cast<uint8_t*>(const_cast<void*>(pool));
    P.n_slots = n_pages * page;
    P.n_kv = n_kv, P.d = d, P.lnb = log2_of(d / 32), P.lpage = log2_of(page);
    P.vec_k = vec_ok(k, ldk), P.vec_v = vec_ok(v, ldv);
    P.status = status;
    return rows_launch(reinterpret_cast<const void*>(kv4_gather_kernel), P, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
