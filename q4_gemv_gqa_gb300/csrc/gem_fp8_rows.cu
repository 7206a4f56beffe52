// gem_fp8_rows.cu — rows in 8-bit floating point (e4m3) with a scale for each 128 values: RMSNorm with the
// residual's addition (gem_rmsnorm_fp8), and the gated activation or a plain row (gem_quant_fp8).
//
// A warp holds a block of 128 values, four consecutive ones a lane, so that a block's loads and its codes
// are one contiguous piece and its largest magnitude one warp reduction.  The scale is a power of two:
// y / scale rounds nothing, and the only question is on which side of a border between two codes y lies.
// y is computed in fp32 with a known relative error e; where the codes of y (1 - e) and y (1 + e) agree
// they are the code, else (about 1e-5 of the values) y is taken again in fp64 and compared with the border,
// which is exact.  The same holds for the scale's own border, 448 * 2^k.
//
// Floors are the rows' bytes; what they take besides is instructions (45 to 52 % of the issue slots) between loads
// that few registers can hold ahead.  GB300: RMSNorm with residual 4096 x 5376 69 us (286 MB, 61 % of the copy rate),
// 8192 x 2560 59 us (68 %); SiLU 4093 x 9728 70 us (358 MB, 75 %), GELU 72 us (73 %); a plain row 36 us (81 %); a decoding
// step's rows 2 to 3 us, of more than 32 blocks (8 x 5376) 4.7 us.  Summing in fp32 first and deciding a row again where that leaves a code open took 75 to 98 us
// (one row of ten) and a second barrier.
#include <cmath>

#include "gem_device.cuh"

namespace gem {
namespace {

constexpr float kMaxCode = 448.f;
constexpr float kTiny = 7.888609052210118e-31f;   // 2^-100: a block below it is zeros
constexpr uint32_t kInfBits = 0x7f800000u;

__device__ __forceinline__ float pow2f(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// the smallest k with m <= 448 * 2^k, for 2^-100 <= m < inf
__device__ __forceinline__ int scale_exp(float m) {
    const int b = __float_as_int(m);
    return (b >> 23) - 127 - 8 + ((b & 0x7fffff) > 0x600000);   // 448 is 1.75 * 2^8
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return static_cast<uint32_t>(lo) | static_cast<uint32_t>(hi) << 16;
}

// magnitude of a finite code's value
__device__ __forceinline__ float e4m3_abs(uint32_t code) {
    const int e = static_cast<int>(code >> 3 & 15), m = static_cast<int>(code & 7);
    return e ? static_cast<float>(8 + m) * pow2f(e - 10) : static_cast<float>(m) * pow2f(-9);
}

// The code of y * 2^-k, exactly, where its neighbours in magnitude are a and b = a + 1 (same sign).
__device__ __forceinline__ uint32_t decide(uint32_t a, uint32_t b, double y, int k) {
    const double mid = 0.5 * (static_cast<double>(e4m3_abs(a)) + static_cast<double>(e4m3_abs(b)));
    const double t = fabs(y) * static_cast<double>(pow2f(-k));
    return t > mid || (t == mid && (a & 1)) ? b : a;
}

__device__ __forceinline__ uint32_t decide_x4(uint32_t lo, uint32_t hi, const double (&y)[4], int k) {
    uint32_t out = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t a = lo >> 8 * j & 255, b = hi >> 8 * j & 255;
        out |= (a == b ? a : decide(a, b, y[j], k)) << 8 * j;
    }
    return out;
}

// Four values as two packed pairs: an instruction does two of them.
struct Four {
    float2 a, b;
};
__device__ __forceinline__ Four four(float4 v) { return {make_float2(v.x, v.y), make_float2(v.z, v.w)}; }
__device__ __forceinline__ Four four(float v) { return {make_float2(v, v), make_float2(v, v)}; }
__device__ __forceinline__ float4 flat(Four v) { return make_float4(v.a.x, v.a.y, v.b.x, v.b.y); }
__device__ __forceinline__ Four operator+(Four x, Four y) { return {fadd2(x.a, y.a), fadd2(x.b, y.b)}; }
__device__ __forceinline__ Four operator*(Four x, Four y) { return {fmul2(x.a, y.a), fmul2(x.b, y.b)}; }
__device__ __forceinline__ Four fma4(Four x, Four y, Four z) { return {ffma2(x.a, y.a, z.a), ffma2(x.b, y.b, z.b)}; }
__device__ __forceinline__ uint32_t e4m3x4(Four v) { return e4m3x4(v.a.x, v.a.y, v.b.x, v.b.y); }

// bits of the largest magnitude; a NaN is larger than any
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)));
    return r;
}
__device__ __forceinline__ uint32_t abs_bits(Four v) { return __float_as_uint(max_nan(max_nan(v.a.x, v.a.y), max_nan(v.b.x, v.b.y))); }

// ---- sums to twice the precision (Dekker's and Knuth's error-free sums and products) ----------
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {   // the low part is not kept small against the high one
    const Pair s = two_sum(a.hi, b.hi);
    return {s.hi, s.lo + (a.lo + b.lo)};
}
// four sums at once, of the squares of v
struct Pairs {
    Four hi, lo;
};
__device__ __forceinline__ void add_squares(Pairs& s, Four v) {
    const Four minus = four(-1.f), p = v * v, e = fma4(v, v, p * minus);   // v^2 = p + e
    const Four t = s.hi + p, u = fma4(s.hi, minus, t), w = fma4(u, minus, t);
    // the sum's error: (hi - (t - u)) + (p - u)
    s.lo = s.lo + (fma4(w, minus, s.hi) + fma4(u, minus, p)) + e;
    s.hi = t;
}

// 1 / sqrt(s / H + eps) to about 2^-43; 1 / H as a pair
__device__ __forceinline__ Pair inv_rms(Pair s, Pair one_h, float eps) {
    const float q0 = s.hi * one_h.hi, q1 = fmaf(s.hi, one_h.hi, -q0) + fmaf(s.hi, one_h.lo, s.lo * one_h.hi);
    Pair q = two_sum(q0, eps);
    q.lo += q1;
    // brought near 1 by a power of 4: the products below then neither overflow nor lose bits
    const float to = q.hi < 0x1p-60f ? 0x1p64f : q.hi > 0x1p60f ? 0x1p-64f : 1.f, back = q.hi < 0x1p-60f ? 0x1p32f : q.hi > 0x1p60f ? 0x1p-32f : 1.f;
    q.hi *= to, q.lo *= to;
    const float r = rsqrtf(q.hi), a = r * r, b = fmaf(r, r, -a);
    const float t = fmaf(q.hi, a, -1.f) + fmaf(q.hi, b, q.lo * a);   // q r^2 - 1
    const float c = -0.5f * r * t, hi = r + c;                        // one Newton step, kept as a pair
    return {hi * back, ((r - hi) + c) * back};
}

// ---- RMSNorm with the residual's addition ------------------------------------------------------
struct NormParams {
    const float* x; int64_t ldx;
    const float* res; int64_t ldr;
    float* out; int64_t ldo;
    int64_t T; int H;
    const float* gamma;
    float eps;
    Pair one_h;             // 1 / H
    int fold;               // half of the power of two that the warps of a row fit in
    uint8_t* codes; int64_t ldc;
    float* scales; int64_t lds;
};

constexpr float kNormErr = 4.8e-7f;   // of h * gamma * r: three roundings and r's own, 4 * 2^-24, doubled

__device__ __forceinline__ double norm64(float h, float g, Pair r) {
    return static_cast<double>(h) * static_cast<double>(g) * (static_cast<double>(r.hi) + static_cast<double>(r.lo));
}
__device__ __noinline__ double norm64_top(float4 h, float4 g, Pair r) {
    return fmax(fmax(fabs(norm64(h.x, g.x, r)), fabs(norm64(h.y, g.y, r))), fmax(fabs(norm64(h.z, g.z, r)), fabs(norm64(h.w, g.w, r))));
}
__device__ __noinline__ uint32_t norm64_codes(uint32_t lo, uint32_t hi, float4 h, float4 g, Pair r, int k) {
    const double y[4] = {norm64(h.x, g.x, r), norm64(h.y, g.y, r), norm64(h.z, g.z, r), norm64(h.w, g.w, r)};
    return decide_x4(lo, hi, y, k);
}

// One CTA of ceil(blocks / NB) warps a row; a lane holds NB pieces of four values.  What concerns a block and not its
// values (scale, bounds) is done for the warp's NB blocks at once, a lane each.
template <int NB, int THREADS, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS) rmsnorm_fp8_kernel(const NormParams p) {
    __shared__ Pair part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    auto col = [&](int i) { return (warp + i * nw) * 128 + lane * 4; };
    auto gamma = [&](int i) {
        return p.gamma && col(i) < p.H ? four(__ldg(reinterpret_cast<const float4*>(p.gamma + col(i)))) : four(1.f);
    };
    const int64_t t = blockIdx.x;
    pdl_wait_trigger();
    Four h[NB], res[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {   // all loads before their use
        h[i] = res[i] = four(0.f);
        if (col(i) < p.H) {
            h[i] = four(__ldcs(reinterpret_cast<const float4*>(p.x + t * p.ldx + col(i))));
            if (p.res) res[i] = four(__ldcs(reinterpret_cast<const float4*>(p.res + t * p.ldr + col(i))));
        }
    }
    Pairs sum{four(0.f), four(0.f)};
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        h[i] = h[i] + res[i];
        if (p.out && col(i) < p.H) *reinterpret_cast<float4*>(p.out + t * p.ldo + col(i)) = flat(h[i]);
        add_squares(sum, h[i]);
    }
    Pair s = add(add({sum.hi.a.x, sum.lo.a.x}, {sum.hi.a.y, sum.lo.a.y}), add({sum.hi.b.x, sum.lo.b.x}, {sum.hi.b.y, sum.lo.b.y}));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        s = add(s, {__shfl_xor_sync(~0u, s.hi, o), __shfl_xor_sync(~0u, s.lo, o)});
    if (nw > 1) {
        if (lane == 0) part[warp] = s;
        __syncthreads();
        s = lane < nw ? part[lane] : Pair{0.f, 0.f};
        for (int o = p.fold; o > 0; o >>= 1)
            s = add(s, {__shfl_xor_sync(~0u, s.hi, o), __shfl_xor_sync(~0u, s.lo, o)});
        s = {__shfl_sync(~0u, s.hi, 0), __shfl_sync(~0u, s.lo, 0)};
    }
    const Pair r = inv_rms(s, p.one_h, p.eps);
    const bool finite = s.hi < __int_as_float(kInfBits);   // false for NaN too

    // (gamma is read from the caches where it is used, twice a row: registers for more rows at once count for more)
    uint32_t mb = 0;   // lane i: the largest of block i
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const uint32_t most = __reduce_max_sync(~0u, col(i) < p.H ? abs_bits(h[i] * gamma(i)) : 0u);
        if (lane == i) mb = most;
    }
    const float m = __uint_as_float(mb) * r.hi, m0 = m * (1.f - kNormErr), m1 = m * (1.f + kNormErr);
    const bool bad = !finite || !(m1 < __int_as_float(kInfBits)), some = !bad && m1 >= kTiny;
    int k = some ? scale_exp(fmaxf(m0, kTiny)) : 0;
    float scale = bad ? __int_as_float(0x7fffffff) : some ? pow2f(k) : 0.f;
    unsigned near = __ballot_sync(~0u, some && (k != scale_exp(m1) || m0 < kTiny));   // blocks next to a border of the scale
    while (near) {
        const int b = __ffs(near) - 1;
        near &= near - 1;
        double top = 0.0;
#pragma unroll
        for (int i = 0; i < NB; ++i)
            if (i == b && col(i) < p.H) top = norm64_top(flat(h[i]), flat(gamma(i)), r);
        const int kb = __shfl_sync(~0u, k, b);
        const bool zero = !__any_sync(~0u, top >= static_cast<double>(kTiny));
        const bool over = __any_sync(~0u, top > static_cast<double>(kMaxCode) * static_cast<double>(pow2f(kb)));
        if (lane == b) k += over, scale = zero ? 0.f : pow2f(k);
    }
    const float f = scale > 0.f ? r.hi * pow2f(-k) : 0.f;   // 0: codes 0 (a NaN scale is not above 0)
#pragma unroll
    for (int i = 0; i < NB; ++i) {
        const int c = col(i);
        const float fi = __shfl_sync(~0u, f, i);
        const Four g = gamma(i), v = h[i] * g;
        const uint32_t lo = e4m3x4(v * four(fi * (1.f - kNormErr)));
        uint32_t code = e4m3x4(v * four(fi * (1.f + kNormErr)));
        if (__any_sync(~0u, lo != code)) {
            const int ki = __shfl_sync(~0u, k, i);
            if (lo != code) code = norm64_codes(lo, code, flat(h[i]), flat(g), r, ki);
        }
        if (c < p.H) *reinterpret_cast<uint32_t*>(p.codes + t * p.ldc + c) = fi > 0.f ? code : 0u;
    }
    const int block = warp + lane * nw;
    if (lane < NB && block * 128 < p.H) p.scales[t * p.lds + block] = scale;
}

// ---- the gated activation, or a plain row --------------------------------------------------------
struct QuantParams {
    const float* x; int64_t ldx;
    const float* up; int64_t ldu;
    int H;
    uint8_t* codes; int64_t ldc;
    float* scales; int64_t lds;
};

constexpr int kPlain = 2;            // ACT: 0 SiLU, 1 GELU-tanh, 2 the row itself
constexpr float kGateLow = -83.f;    // the gate is 0 for z below it (e^83 is still finite in fp32)
constexpr float kGeluLow = -9.809149f;   // the least x whose exact z for GELU is not: z in fp32 falls on the wrong side next to it
constexpr double kGelu1 = 1.5957691216057308;                  // 2 sqrt(2 / pi)
constexpr double kGelu3 = kGelu1 * 0.044715;

// act(x) * u of four values, and a bound of their relative error: 9.5e-7, and for GELU, whose z is itself off by 2^-22
// of it, 2.4e-7 max(-z, 1/2) more (above 0 the gate's own flatness holds z's error down).  e^-z is 2^(a + b), a + b = -z log2(e) as a pair, so that its error stays
// 2^-22 for any z; then a reciprocal and two products.  The gate meets up first: it is far from 1 only where x is between
// -83 and 17, so wherever y counts (above 2^-118, the lowest border of a code) the gate times up is a normal number, or up
// itself.  The gate times x is not, with a tiny x and a large up.
template <int ACT>
__device__ __forceinline__ Four gated(Four x, Four u, float& err) {
    Four z = x;
    if (ACT == 1) z = x * fma4(x * x, four(static_cast<float>(kGelu3)), four(static_cast<float>(kGelu1)));
    // beyond these the gate is 0 or 1 all the same (and so for a NaN, which the product with x keeps)
    auto held = [](float v, float x) { return x >= (ACT == 1 ? kGeluLow : kGateLow) ? fminf(v, 100.f) : -200.f; };
    z = {make_float2(held(z.a.x, x.a.x), held(z.a.y, x.a.y)), make_float2(held(z.b.x, x.b.x), held(z.b.y, x.b.y))};
    err = 9.5e-7f;
    if (ACT == 1) {
        auto depth = [](float v) { return v > -150.f ? -v : 0.f; };   // a gate of 0 is exact
        err = fmaf(fmaxf(fmaxf(fmaxf(depth(z.a.x), depth(z.a.y)), fmaxf(depth(z.b.x), depth(z.b.y))), 0.5f), 2.4e-7f, err);
    }
    const float l2e = 1.4426950408889634f;
    const Four a = z * four(-l2e);
    const Four b = fma4(z, four(-1.925963033500947e-8f), fma4(z, four(-l2e), a * four(-1.f)));
    auto exp2_of = [](float v) {
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v));
        return e;
    };
    auto inverse = [](float v) {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
        return r;
    };
    Four e{make_float2(exp2_of(a.a.x), exp2_of(a.a.y)), make_float2(exp2_of(a.b.x), exp2_of(a.b.y))};
    // e (1 + b ln 2) + 1; at z = -200 e is infinite and b tiny, and its inverse 0
    e = fma4(e, fma4(b, four(0.6931471805599453f), four(1.f)), four(1.f));
    const Four r{make_float2(inverse(e.a.x), inverse(e.a.y)), make_float2(inverse(e.b.x), inverse(e.b.y))};
    return x * (r * u);
}
template <int ACT>
__device__ __noinline__ double gated64(float x, float u) {
    const double d = x;
    const double z = ACT == 1 ? d * (kGelu1 + kGelu3 * d * d) : d;
    return z < static_cast<double>(kGateLow) ? 0.0 : d * static_cast<double>(u) / (1.0 + exp(-z));
}
template <int ACT>
__device__ __noinline__ double gated64_top(float4 x, float4 u) {
    return fmax(fmax(fabs(gated64<ACT>(x.x, u.x)), fabs(gated64<ACT>(x.y, u.y))), fmax(fabs(gated64<ACT>(x.z, u.z)), fabs(gated64<ACT>(x.w, u.w))));
}
template <int ACT>
__device__ __noinline__ uint32_t gated64_codes(uint32_t lo, uint32_t hi, float4 x, float4 u, int k) {
    const double y[4] = {gated64<ACT>(x.x, u.x), gated64<ACT>(x.y, u.y), gated64<ACT>(x.z, u.z), gated64<ACT>(x.w, u.w)};
    return decide_x4(lo, hi, y, k);
}

// U blocks of one row a warp, one after the other; their loads first.
template <int ACT, int U>
__global__ void __launch_bounds__(256) quant_fp8_kernel(const QuantParams p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = blockIdx.x;
    const int first = (blockIdx.y * (blockDim.x >> 5) + warp) * U * 128;
    pdl_wait_trigger();
    if (first >= p.H) return;
    Four x[U], u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int c = first + i * 128 + lane * 4;
        x[i] = u[i] = four(0.f);
        if (c < p.H) {
            x[i] = four(__ldcs(reinterpret_cast<const float4*>(p.x + t * p.ldx + c)));
            if (ACT != kPlain) u[i] = four(__ldcs(reinterpret_cast<const float4*>(p.up + t * p.ldu + c)));
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int c = first + i * 128 + lane * 4;
        if (first + i * 128 >= p.H) break;
        Four v = x[i];
        float err = 0.f;
        if (ACT != kPlain) v = gated<ACT>(x[i], u[i], err);
        const uint32_t mb = __reduce_max_sync(~0u, abs_bits(v));
        const float m = __uint_as_float(mb);
        uint32_t code = 0;
        float scale = 0.f;
        if (mb >= kInfBits) {
            scale = __int_as_float(0x7fffffff);
        } else if (ACT == kPlain) {
            if (m >= kTiny) {
                const int k = scale_exp(m);
                scale = pow2f(k);
                code = e4m3x4(v * four(pow2f(-k)));
            }
        } else if (m * 1.0001f >= kTiny) {
            const float worst = ACT == 1 ? __uint_as_float(__reduce_max_sync(~0u, __float_as_uint(err))) : err;   // for the block
            int k = scale_exp(fmaxf(m * (1.f - worst), kTiny));
            bool zero = false;
            if (k != scale_exp(fmaxf(m * (1.f + worst), kTiny)) || m * (1.f - worst) < kTiny) {
                const double top = gated64_top<ACT>(flat(x[i]), flat(u[i]));
                zero = !__any_sync(~0u, top >= static_cast<double>(kTiny));
                if (__any_sync(~0u, top > static_cast<double>(kMaxCode) * static_cast<double>(pow2f(k)))) ++k;
            }
            if (!zero) {
                scale = pow2f(k);
                const uint32_t lo = e4m3x4(v * four(pow2f(-k) * (1.f - err)));
                code = e4m3x4(v * four(pow2f(-k) * (1.f + err)));
                if (lo != code) code = gated64_codes<ACT>(lo, code, flat(x[i]), flat(u[i]), k);
            }
        }
        if (c < p.H) *reinterpret_cast<uint32_t*>(p.codes + t * p.ldc + c) = code;
        if (lane == 0) p.scales[t * p.lds + (c >> 7)] = scale;
    }
}

bool off16(const void* q, int64_t ld, int64_t unit) { return (reinterpret_cast<uintptr_t>(q) & 15) || (ld % unit); }

gem_status check_out(const uint8_t* codes, int64_t ldc, const float* scales, int64_t lds, int64_t H) {
    if (!codes || !scales || ldc < H || lds < (H + 127) / 128) return GEM_ERR_INVALID_ARG;
    if (off16(codes, ldc, 16) || (reinterpret_cast<uintptr_t>(scales) & 3)) return GEM_ERR_MISALIGNED;
    return GEM_OK;
}

template <int NB, int THREADS, int CTAS>
gem_status launch_norm(NormParams p, int blocks, cudaStream_t stream) {
    const int warps = (blocks + NB - 1) / NB;
    while (2 * p.fold < warps) p.fold = p.fold ? 2 * p.fold : 1;
    void* args[] = {&p};
    return launch_pdl(reinterpret_cast<const void*>(rmsnorm_fp8_kernel<NB, THREADS, CTAS>), dim3(static_cast<unsigned>(p.T)),
                      dim3(warps * 32), 0, stream, args);
}

}  // namespace
}  // namespace gem

extern "C" {

gem_status gem_rmsnorm_fp8(const float* x, int64_t ldx, const float* residual, int64_t ldr, float* out, int64_t ldo,
                           int64_t T, int64_t H, const float* gamma, float eps, uint8_t* codes, int64_t ldc,
                           float* scales, int64_t lds, void* stream) {
    using namespace gem;
    if (T < 0 || H < 0 || !(eps >= 0.f && eps <= 0x1p127f)) return GEM_ERR_INVALID_ARG;   // plus any mean square it is finite
    if (H % 16 || H > 32768 || T >= (int64_t(1) << 31)) return GEM_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || H == 0) return GEM_OK;
    if (!x || ldx < H || (residual && ldr < H) || (out && ldo < H)) return GEM_ERR_INVALID_ARG;
    if ((out == x && ldo != ldx) || (out && out == residual && ldo != ldr)) return GEM_ERR_INVALID_ARG;
    gem_status st = check_out(codes, ldc, scales, lds, H);
    if (st != GEM_OK) return st;
    if (off16(x, ldx, 4) || (residual && off16(residual, ldr, 4)) || (out && off16(out, ldo, 4)) || off16(gamma, 0, 4))
        return GEM_ERR_MISALIGNED;
    DeviceInfo di;
    if ((st = device_info(&di)) != GEM_OK) return st;
    const double one_h = 1.0 / static_cast<double>(H);
    const float one_h_hi = static_cast<float>(one_h);
    NormParams p{x, ldx, residual, ldr, out, ldo, T, static_cast<int>(H), gamma, eps,
                 {one_h_hi, static_cast<float>(one_h - static_cast<double>(one_h_hi))}, 0, codes, ldc, scales, lds};
    const int blocks = static_cast<int>((H + 127) / 128);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // few rows: a block a warp, the shortest chain, as far as a CTA's 32 warps go (8 x 2560: 2.6 us); else four, in so few
    // registers that three rows are in work on an SM (8 x 5376: 4.7 us; 4096 x 5376: 69; two rows 81; one, with the next
    // row's loads ahead in 122 registers, 76)
    if (blocks <= 32 && T <= di.num_sms) return launch_norm<1, 1024, 1>(p, blocks, s);
    if (blocks <= 48) return launch_norm<4, 384, 3>(p, blocks, s);
    if (blocks <= 128) return launch_norm<4, 1024, 1>(p, blocks, s);
    return launch_norm<8, 1024, 1>(p, blocks, s);
}

gem_status gem_quant_fp8(const float* x, int64_t ldx, const float* up, int64_t ldu, int64_t T, int64_t H, int act,
                         uint8_t* codes, int64_t ldc, float* scales, int64_t lds, void* stream) {
    using namespace gem;
    if (T < 0 || H < 0 || act < 0 || act > 1) return GEM_ERR_INVALID_ARG;
    if (H % 16 || H > (int64_t(1) << 24) || T >= (int64_t(1) << 31)) return GEM_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || H == 0) return GEM_OK;
    if (!x || ldx < H || (up && ldu < H)) return GEM_ERR_INVALID_ARG;
    gem_status st = check_out(codes, ldc, scales, lds, H);
    if (st != GEM_OK) return st;
    if (off16(x, ldx, 4) || (up && off16(up, ldu, 4))) return GEM_ERR_MISALIGNED;
    QuantParams p{x, ldx, up, ldu, static_cast<int>(H), codes, ldc, scales, lds};
    constexpr int U = 2;
    const int units = static_cast<int>(((H + 127) / 128 + U - 1) / U), warps = std::min(8, units);
    const void* fn = !up ? reinterpret_cast<const void*>(quant_fp8_kernel<kPlain, U>)
                     : act == 0 ? reinterpret_cast<const void*>(quant_fp8_kernel<0, U>)
                                : reinterpret_cast<const void*>(quant_fp8_kernel<1, U>);
    void* args[] = {&p};
    return launch_pdl(fn, dim3(static_cast<unsigned>(T), static_cast<unsigned>((units + warps - 1) / warps)),
                      dim3(warps * 32), 0, static_cast<cudaStream_t>(stream), args);
}

}  // extern "C"
