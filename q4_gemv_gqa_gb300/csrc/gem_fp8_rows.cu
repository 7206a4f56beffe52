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
// Both kernels are bound by the loads and stores of their rows.
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

__device__ __forceinline__ uint32_t abs_bits(float4 v) {
    return max(max(__float_as_uint(fabsf(v.x)), __float_as_uint(fabsf(v.y))),
               max(__float_as_uint(fabsf(v.z)), __float_as_uint(fabsf(v.w))));
}

// ---- sums to twice the precision (Dekker's and Knuth's error-free sums and products) ----------
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
    const Pair s = two_sum(a.hi, b.hi);
    const float lo = s.lo + (a.lo + b.lo), hi = s.hi + lo;
    return {hi, lo - (hi - s.hi)};
}
__device__ __forceinline__ void add_square(Pair& s, float v) {
    const float p = v * v;
    const Pair t = two_sum(s.hi, p);
    s.hi = t.hi;
    s.lo += t.lo + fmaf(v, v, -p);
}

// 1 / sqrt(s / H + eps) to about 2^-43
__device__ __forceinline__ Pair inv_rms(Pair s, float H, float eps) {
    const float q0 = __fdiv_rn(s.hi, H);
    const float q1 = __fdiv_rn(fmaf(-q0, H, s.hi) + s.lo, H);
    Pair q = two_sum(q0, eps);
    q.lo += q1;
    const float r = rsqrtf(q.hi), a = r * r, b = fmaf(r, r, -a);
    const float t = fmaf(q.hi, a, -1.f) + fmaf(q.hi, b, q.lo * a);   // q r^2 - 1
    const float c = -0.5f * r * t, hi = r + c;                        // one Newton step, kept as a pair
    return {hi, (r - hi) + c};
}

// ---- RMSNorm with the residual's addition ------------------------------------------------------
struct NormParams {
    const float* x; int64_t ldx;
    const float* res; int64_t ldr;
    float* out; int64_t ldo;
    int64_t T; int H;
    const float* gamma;
    float eps;
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

// One CTA of ceil(blocks / NB) warps a row, rows dealt out round robin; a lane holds NB pieces of four
// values.  PIPE: it also holds gamma for all rows, and the next row's loads are in flight while it sums
// this one's (rows too long for the registers of that are read when their turn comes).
template <int NB, bool PIPE, int THREADS>
__global__ void __launch_bounds__(THREADS) rmsnorm_fp8_kernel(const NormParams p) {
    __shared__ Pair part[2][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    auto col = [&](int i) { return (warp + i * nw) * 128 + lane * 4; };
    const float4 zero4 = make_float4(0.f, 0.f, 0.f, 0.f);
    auto gamma = [&](int i) {
        return p.gamma && col(i) < p.H ? __ldg(reinterpret_cast<const float4*>(p.gamma + col(i))) : make_float4(1.f, 1.f, 1.f, 1.f);
    };
    float4 gs[PIPE ? NB : 1], nx[NB], nr[NB];
    auto request = [&](int64_t t) {
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            nx[i] = nr[i] = zero4;
            if (col(i) < p.H) {
                nx[i] = __ldcs(reinterpret_cast<const float4*>(p.x + t * p.ldx + col(i)));
                if (p.res) nr[i] = __ldcs(reinterpret_cast<const float4*>(p.res + t * p.ldr + col(i)));
            }
        }
    };
    pdl_wait_trigger();
    if (PIPE) {
#pragma unroll
        for (int i = 0; i < NB; ++i) gs[i] = gamma(i);
        request(blockIdx.x);
    }
    int turn = 0;
    for (int64_t t = blockIdx.x; t < p.T; t += gridDim.x, turn ^= 1) {
        if (!PIPE) request(t);
        float4 h[NB];
        Pair s{0.f, 0.f};
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            h[i] = make_float4(nx[i].x + nr[i].x, nx[i].y + nr[i].y, nx[i].z + nr[i].z, nx[i].w + nr[i].w);
            if (p.out && col(i) < p.H) *reinterpret_cast<float4*>(p.out + t * p.ldo + col(i)) = h[i];
            add_square(s, h[i].x);
            add_square(s, h[i].y);
            add_square(s, h[i].z);
            add_square(s, h[i].w);
        }
        if (PIPE && t + gridDim.x < p.T) request(t + gridDim.x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            s = add(s, {__shfl_xor_sync(~0u, s.hi, o), __shfl_xor_sync(~0u, s.lo, o)});
        if (nw > 1) {
            // two buffers in turn: a warp writes one again only behind the next row's barrier
            if (lane == 0) part[turn][warp] = s;
            __syncthreads();
            s = lane < nw ? part[turn][lane] : Pair{0.f, 0.f};
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                s = add(s, {__shfl_xor_sync(~0u, s.hi, o), __shfl_xor_sync(~0u, s.lo, o)});
        }
        const Pair r = inv_rms(s, static_cast<float>(p.H), p.eps);
        const bool finite = s.hi < __int_as_float(kInfBits);   // false for NaN too
#pragma unroll
        for (int i = 0; i < NB; ++i) {
            const int c = col(i);
            if (c - lane * 4 >= p.H) break;   // no such block (the same for the warp)
            const float4 g = PIPE ? gs[i] : gamma(i);
            float4 v = make_float4(h[i].x * g.x, h[i].y * g.y, h[i].z * g.z, h[i].w * g.w);
            if (c >= p.H) v = zero4;
            const uint32_t mb = __reduce_max_sync(~0u, abs_bits(v));
            const float m = __uint_as_float(mb) * r.hi, m0 = m * (1.f - kNormErr), m1 = m * (1.f + kNormErr);
            uint32_t code = 0;
            float scale = 0.f;
            if (!finite || mb >= kInfBits || !(m1 < __int_as_float(kInfBits))) {
                scale = __int_as_float(0x7fffffff);
            } else if (m1 >= kTiny) {
                int k = scale_exp(fmaxf(m0, kTiny));
                bool zero = false;
                if (k != scale_exp(m1) || m0 < kTiny) {   // next to a border
                    const double top = c < p.H ? norm64_top(h[i], g, r) : 0.0;
                    zero = !__any_sync(~0u, top >= static_cast<double>(kTiny));
                    if (__any_sync(~0u, top > static_cast<double>(kMaxCode) * static_cast<double>(pow2f(k)))) ++k;
                }
                if (!zero) {
                    scale = pow2f(k);
                    const float f = r.hi * pow2f(-k), f0 = f * (1.f - kNormErr), f1 = f * (1.f + kNormErr);
                    const uint32_t lo = e4m3x4(v.x * f0, v.y * f0, v.z * f0, v.w * f0);
                    code = e4m3x4(v.x * f1, v.y * f1, v.z * f1, v.w * f1);
                    if (lo != code) code = norm64_codes(lo, code, h[i], g, r, k);
                }
            }
            if (c < p.H) *reinterpret_cast<uint32_t*>(p.codes + t * p.ldc + c) = code;
            if (lane == 0) p.scales[t * p.lds + (c >> 7)] = scale;
        }
    }
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
constexpr float kGateLow = -83.f;    // the gate is 0 below it (e^83 is still finite in fp32)
constexpr double kGelu1 = 1.5957691216057308;                  // 2 sqrt(2 / pi)
constexpr double kGelu3 = kGelu1 * 0.044715;

// act(x) * u and a bound of its relative error.  e^-z is 2^(a + b), a + b = -z log2(e) as a pair, so that
// its error stays 2^-22 for any z; then a reciprocal and two products.  GELU's z itself is off by 2^-22 |z|.
template <int ACT>
__device__ __forceinline__ float gated(float x, float u, float& err) {
    const float g = ACT == 1 ? x * fmaf(x * x, static_cast<float>(kGelu3), static_cast<float>(kGelu1)) : x;
    const float z = fminf(fmaxf(g, -100.f), 100.f);   // beyond them the gate is 0 or 1 all the same
    err = ACT == 1 ? fmaf(fabsf(z), 2.4e-7f, 9.5e-7f) : 9.5e-7f;
    const float l2e = 1.4426950408889634f, a = -z * l2e;
    const float b = fmaf(-z, l2e, -a) - z * 1.925963033500947e-8f;
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a));
    e = fmaf(e, b * 0.6931471805599453f, e);
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
    return x * (z < kGateLow ? 0.f : x == x ? r : x) * u;
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
    float4 x[U], u[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int c = first + i * 128 + lane * 4;
        x[i] = u[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c < p.H) {
            x[i] = __ldcs(reinterpret_cast<const float4*>(p.x + t * p.ldx + c));
            if (ACT != kPlain) u[i] = __ldcs(reinterpret_cast<const float4*>(p.up + t * p.ldu + c));
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int c = first + i * 128 + lane * 4;
        if (first + i * 128 >= p.H) break;
        float4 v = x[i], err = make_float4(0.f, 0.f, 0.f, 0.f);
        if (ACT != kPlain) {
            v.x = gated<ACT>(x[i].x, u[i].x, err.x);
            v.y = gated<ACT>(x[i].y, u[i].y, err.y);
            v.z = gated<ACT>(x[i].z, u[i].z, err.z);
            v.w = gated<ACT>(x[i].w, u[i].w, err.w);
        }
        const uint32_t mb = __reduce_max_sync(~0u, abs_bits(v));
        const float m = __uint_as_float(mb);
        uint32_t code = 0;
        float scale = 0.f;
        if (mb >= kInfBits) {
            scale = __int_as_float(0x7fffffff);
        } else if (ACT == kPlain) {
            if (m >= kTiny) {
                const int k = scale_exp(m);
                const float f = pow2f(-k);
                scale = pow2f(k);
                code = e4m3x4(v.x * f, v.y * f, v.z * f, v.w * f);
            }
        } else if (m * 1.0001f >= kTiny) {
            // the largest error of the lanes' bounds stands for the block's
            const float worst = __uint_as_float(__reduce_max_sync(
                ~0u, __float_as_uint(fmaxf(fmaxf(err.x, err.y), fmaxf(err.z, err.w)))));
            int k = scale_exp(fmaxf(m * (1.f - worst), kTiny));
            bool zero = false;
            if (k != scale_exp(fmaxf(m * (1.f + worst), kTiny)) || m * (1.f - worst) < kTiny) {
                const double top = gated64_top<ACT>(x[i], u[i]);
                zero = !__any_sync(~0u, top >= static_cast<double>(kTiny));
                if (__any_sync(~0u, top > static_cast<double>(kMaxCode) * static_cast<double>(pow2f(k)))) ++k;
            }
            if (!zero) {
                scale = pow2f(k);
                const float f = pow2f(-k);
                v.x *= f, v.y *= f, v.z *= f, v.w *= f;
                const uint32_t lo = e4m3x4(fmaf(-v.x, err.x, v.x), fmaf(-v.y, err.y, v.y), fmaf(-v.z, err.z, v.z), fmaf(-v.w, err.w, v.w));
                code = e4m3x4(fmaf(v.x, err.x, v.x), fmaf(v.y, err.y, v.y), fmaf(v.z, err.z, v.z), fmaf(v.w, err.w, v.w));
                if (lo != code) code = gated64_codes<ACT>(lo, code, x[i], u[i], k);
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

template <int NB, bool PIPE, int THREADS>
gem_status launch_norm(NormParams p, int blocks, int ctas, cudaStream_t stream) {
    const int warps = (blocks + NB - 1) / NB;
    void* args[] = {&p};
    return launch_pdl(reinterpret_cast<const void*>(rmsnorm_fp8_kernel<NB, PIPE, THREADS>),
                      dim3(static_cast<unsigned>(std::min<int64_t>(p.T, ctas))), dim3(warps * 32), 0, stream, args);
}

}  // namespace
}  // namespace gem

extern "C" {

gem_status gem_rmsnorm_fp8(const float* x, int64_t ldx, const float* residual, int64_t ldr, float* out, int64_t ldo,
                           int64_t T, int64_t H, const float* gamma, float eps, uint8_t* codes, int64_t ldc,
                           float* scales, int64_t lds, void* stream) {
    using namespace gem;
    if (T < 0 || H < 0 || !(eps >= 0.f)) return GEM_ERR_INVALID_ARG;
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
    NormParams p{x, ldx, residual, ldr, out, ldo, T, static_cast<int>(H), gamma, eps, codes, ldc, scales, lds};
    const int blocks = static_cast<int>((H + 127) / 128);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    // few rows: a block a warp, the shortest chain; else four, with as many CTAs as stay resident
    if (blocks <= 32 && T <= di.num_sms) return launch_norm<1, true, 1024>(p, blocks, di.num_sms, s);
    if (blocks <= 64) return launch_norm<4, true, 512>(p, blocks, di.num_sms * std::max(1, 20 / ((blocks + 3) / 4)), s);
    return launch_norm<8, false, 1024>(p, blocks, di.num_sms * 4, s);
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
