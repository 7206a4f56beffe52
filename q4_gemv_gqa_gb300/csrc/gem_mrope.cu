// gem_mrope.cu — per-head QK-norm and rotary positions with one or several axes, for T tokens.
#include <cmath>
#include <type_traits>

#include "gem_device.cuh"
#include "gem_kv4.cuh"

namespace gem {
namespace kv4 {
namespace {

constexpr int kMaxAxes = 4;

// theta^(-2i/R) / (2 pi) in turns, 64-bit fixed point; the two lowest bits hold the frequency's axis
// (they change an angle by less than 2^-29 turns at the largest position).
struct MropeFreq {
    uint64_t f[kMaxHeadDim / 2];
};

struct MropeParams {
    const float* x;
    int64_t ldx;
    float* out;
    int64_t ldo, T;
    int n_q, nheads, d, R;
    const float *gamma_q, *gamma_k;
    float eps;
    const int32_t* pos;
    int64_t ldpos;
    int n_axes;
    int* status;
};

// cos and sin of pos * frequency.  The product is taken modulo one turn in 64-bit integers, which
// is exact; what is left, 32 bits of a turn, goes through fp32.
__device__ __forceinline__ void turn_cos_sin(const MropeParams& P, int64_t t, uint64_t f, float& c, float& s) {
    const int axis = static_cast<int>(f & 3);
    const uint32_t p = static_cast<uint32_t>(P.pos[axis * P.ldpos + t]);
    const uint64_t turns = static_cast<uint64_t>(p) * f;
    const int32_t top = static_cast<int32_t>((turns + 0x80000000ull) >> 32);
    sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
}

// 0: rotate row t; 1: padding; 2: a position out of range
__device__ __forceinline__ int row_state(const MropeParams& P, int64_t t) {
    const int32_t p0 = P.pos[t];
    if (p0 == -1) return 1;
    bool bad = p0 < 0;
    for (int a = 1; a < P.n_axes; ++a) bad |= P.pos[a * P.ldpos + t] < 0;
    return bad ? 2 : 0;
}

// The head dims that the library's layers have, with rows that can be read 16 bytes at a time.  D / 8 lanes
// (32 for D = 512) hold a head: a lane four neighbouring pairs (i, i + R/2) (past the rotated dims, pairs of
// kept ones), the same for every head, so that the angles are taken once for all heads of a warp and a
// head is two 16-byte loads, one reduction and two stores a lane.  A warp takes `heads` heads of one
// token, the loads of the next under way while one is rotated.  167.7 MB (read once, written once) take
// 34.5 us, 4.9 TB/s, 72 % of the measured copy rate, bound by the loads in flight (one head a warp ahead, 4093
// warps in all); a plain contiguous copy of the same bytes takes 28.7 us here.
template <int D>
__global__ void __launch_bounds__(256, D < 512 ? 4 : 2) mrope_rows_kernel(const MropeParams P, const __grid_constant__ MropeFreq F, int heads,
                                                         int chunks) {
    constexpr int kLanes = D < 256 ? D / 8 : 32, kSide = 32 / kLanes, NC = D / 8 / kLanes, kAhead = 1;
    pdl_wait_trigger();
    const int lane = threadIdx.x & 31, sub = lane / kLanes, at = lane % kLanes;
    const uint32_t unit = blockIdx.x * 8u + (threadIdx.x >> 5);
    const uint32_t token = unit / static_cast<uint32_t>(chunks);
    const int64_t t = token;
    if (t >= P.T) return;
    const int chunk = static_cast<int>(unit - token * chunks);
    const int state = row_state(P, t);
    if (state) {
        if (state == 2 && chunk == 0 && lane == 0) atomicOr(P.status, GEM_DEVFLAG_POS_RANGE);
        return;
    }
    const int half = P.R / 2, h0 = chunk * heads, h1 = min(P.nheads, h0 + heads);
    int at0[NC], at1[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int j = (c * kLanes + at) * 4;
        at0[c] = j < half ? j : half + j;
        at1[c] = at0[c] + (j < half ? half : (D - P.R) / 2);
    }
    const float* x = P.x + t * P.ldx;
    float* out = P.out + t * P.ldo;
    auto load = [](const float* p, float (&to)[4]) { *reinterpret_cast<float4*>(to) = *reinterpret_cast<const float4*>(p); };
    alignas(16) float a[kAhead][NC][4], b[kAhead][NC][4], an[kAhead][NC][4], bn[kAhead][NC][4];
    auto fetch = [&](int h) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (h + k * kSide < h1)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    load(x + (h + k * kSide) * D + at0[c], an[k][c]);
                    load(x + (h + k * kSide) * D + at1[c], bn[k][c]);
                }
    };
    fetch(h0 + sub);
    float co[NC][4], si[NC][4];
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int j = (c * kLanes + at) * 4;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            co[c][v] = 1.f, si[c][v] = 0.f;
            if (j < half) turn_cos_sin(P, t, F.f[j + v], co[c][v], si[c][v]);
        }
    }
    for (int h = h0 + sub; h - sub < h1; h += kAhead * kSide) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int v = 0; v < 4; ++v) a[k][c][v] = an[k][c][v], b[k][c][v] = bn[k][c][v];
        fetch(h + kAhead * kSide);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int hk = h + k * kSide;
            if (hk - sub >= h1) break;
            const float* gamma = hk < P.n_q ? P.gamma_q : P.gamma_k;
            float ss = 0.f;
#pragma unroll
            for (int c = 0; c < NC; ++c)
#pragma unroll
                for (int v = 0; v < 4; ++v) ss = fmaf(a[k][c][v], a[k][c][v], fmaf(b[k][c][v], b[k][c][v], ss));
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (hk >= h1) continue;
            if (gamma) {
                const float r = rsqrtf(ss * (1.f / D) + P.eps);
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    alignas(16) float g0[4], g1[4];
                    load(gamma + at0[c], g0);
                    load(gamma + at1[c], g1);
#pragma unroll
                    for (int v = 0; v < 4; ++v) a[k][c][v] *= r * g0[v], b[k][c][v] *= r * g1[v];
                }
            }
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                alignas(16) float y0[4], y1[4];
                const bool kept = (c * kLanes + at) * 4 >= half;   // as they are: times 0 an infinity would be NaN
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    y0[v] = kept ? a[k][c][v] : fmaf(a[k][c][v], co[c][v], -b[k][c][v] * si[c][v]);
                    y1[v] = kept ? b[k][c][v] : fmaf(a[k][c][v], si[c][v], b[k][c][v] * co[c][v]);
                }
                *reinterpret_cast<float4*>(out + hk * D + at0[c]) = *reinterpret_cast<float4*>(y0);
                *reinterpret_cast<float4*>(out + hk * D + at1[c]) = *reinterpret_cast<float4*>(y1);
            }
        }
    }
}

// Any even d and R: one warp per (token, head), the head in shared memory and the angles taken for each head
// (96 us on the rows above: scalar loads, and as many sines as values).
__global__ void __launch_bounds__(128) mrope_kernel(const MropeParams P, const __grid_constant__ MropeFreq F) {
    __shared__ float buf[4][kMaxHeadDim];
    pdl_wait_trigger();
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int64_t unit = blockIdx.x * 4ll + w;
    const int64_t t = unit / P.nheads;
    if (t >= P.T) return;
    const int head = static_cast<int>(unit % P.nheads);
    const int state = row_state(P, t);
    if (state) {
        if (state == 2 && head == 0 && lane == 0) atomicOr(P.status, GEM_DEVFLAG_POS_RANGE);
        return;
    }
    const float* x = P.x + t * P.ldx + static_cast<int64_t>(head) * P.d;
    float* out = P.out + t * P.ldo + static_cast<int64_t>(head) * P.d;
    const float* gamma = head < P.n_q ? P.gamma_q : P.gamma_k;
    float* sb = buf[w];
    float ss = 0.f;
    for (int e = lane; e < P.d; e += 32) {
        const float v = x[e];
        sb[e] = v;
        ss = fmaf(v, v, ss);
    }
    __syncwarp();
    if (gamma) {
        const float r = rsqrtf(warp_sum(ss) / static_cast<float>(P.d) + P.eps);
        for (int e = lane; e < P.d; e += 32) sb[e] = sb[e] * r * gamma[e];
        __syncwarp();
    }
    const int half = P.R / 2;
    for (int i = lane; i < half; i += 32) {
        float c, s;
        turn_cos_sin(P, t, F.f[i], c, s);
        const float a = sb[i], b = sb[i + half];
        out[i] = fmaf(a, c, -b * s);
        out[i + half] = fmaf(a, s, b * c);
    }
    for (int e = P.R + lane; e < P.d; e += 32) out[e] = sb[e];
}

// The frequencies are a function of these alone; a thread keeps the last ones it computed, since their powers
// cost more than the launch and layers of one kind ask for the same.  (Between kinds of layers with bases or
// sections of their own they are computed again.)
struct FreqKey {
    float theta;
    int n_axes, interleaved;
    int32_t sections[kMaxAxes];
    bool operator==(const FreqKey& o) const {
        return theta == o.theta && n_axes == o.n_axes && interleaved == o.interleaved &&
               std::equal(sections, sections + kMaxAxes, o.sections);
    }
};

const MropeFreq& frequencies(const FreqKey& key, int R) {
    thread_local FreqKey last{};
    thread_local MropeFreq F;
    if (key == last) return F;
    for (int i = 0, a = 0, left = key.sections[0]; i < R / 2; ++i) {
        int axis;
        if (key.interleaved) {
            axis = i % key.n_axes;
            if (axis && i >= key.n_axes * static_cast<int64_t>(key.sections[axis])) axis = 0;
        } else {
            while (left == 0) left = key.sections[++a];
            --left;
            axis = a;
        }
        // theta < 1 gives more than a turn a position: the whole turns drop out
        const double turns = std::pow(static_cast<double>(key.theta), -2.0 * i / R) * 0.15915494309189535;
        const double part = turns - std::floor(turns);
        F.f[i] = ((static_cast<uint64_t>(std::ldexp(part, 63)) << 1) & ~3ull) | static_cast<uint64_t>(axis);
    }
    last = key;
    return F;
}

}  // namespace
}  // namespace kv4
}  // namespace gem

extern "C" gem_status gem_qknorm_mrope(const float* qkv, int64_t ldqkv, int64_t T, int n_q, int n_kv, int d,
                                       const float* gamma_q, const float* gamma_k, float eps,
                                       const int32_t* pos, int64_t ldpos, int n_axes, const int32_t* sections,
                                       int interleaved, float theta, float* out, int64_t ldo, int32_t* status,
                                       void* stream) {
    using namespace gem;
    using namespace gem::kv4;
    if (T < 0 || n_q < 0 || n_kv < 0 || d <= 0 || !(eps >= 0.f) || interleaved < 0 || interleaved > 1)
        return GEM_ERR_INVALID_ARG;
    if (d > kMaxHeadDim || (d & 1) || n_axes < 1 || n_axes > kMaxAxes || n_q > 65535 || n_kv > 65535)
        return GEM_ERR_UNSUPPORTED_SHAPE;
    if (!sections || !(theta > 0.f) || !std::isfinite(theta)) return GEM_ERR_INVALID_ARG;
    int64_t half = 0;
    for (int a = 0; a < n_axes; ++a) {
        if (sections[a] < 0) return GEM_ERR_INVALID_ARG;
        half += sections[a];
    }
    if (half < 1 || 2 * half > d) return GEM_ERR_INVALID_ARG;
    const int R = static_cast<int>(2 * half);
    for (int a = 1; interleaved && a < n_axes; ++a)
        if (sections[a] && a + static_cast<int64_t>(sections[a] - 1) * n_axes >= half) return GEM_ERR_INVALID_ARG;
    const int64_t cols = static_cast<int64_t>(n_q + n_kv) * d;
    if (T == 0 || cols == 0) return GEM_OK;
    if (!qkv || !out || !pos || ldqkv < cols || ldo < cols || ldpos < T) return GEM_ERR_INVALID_ARG;
    if (out == qkv && ldo != ldqkv) return GEM_ERR_INVALID_ARG;

    const FreqKey key{theta, n_axes, interleaved, {sections[0], n_axes > 1 ? sections[1] : 0, n_axes > 2 ? sections[2] : 0,
                                                   n_axes > 3 ? sections[3] : 0}};
    const MropeFreq& F = frequencies(key, R);
    MropeParams P{};
    P.x = qkv, P.ldx = ldqkv, P.out = out, P.ldo = ldo, P.T = T;
    P.n_q = n_q, P.nheads = n_q + n_kv, P.d = d, P.R = R;
    P.gamma_q = gamma_q, P.gamma_k = gamma_k, P.eps = eps;
    P.pos = pos, P.ldpos = ldpos, P.n_axes = n_axes, P.status = status;
    gem_status st = flag_word(&P.status);
    if (st != GEM_OK) return st;
    // the vectorised kernel where every piece of a row can be read 16 bytes at a time
    auto aligned = [](const float* p, int64_t ld) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 4 == 0; };
    if (head_dim_ok(d) && half % 4 == 0 && aligned(qkv, ldqkv) && aligned(out, ldo) && aligned(gamma_q, 0) &&
        aligned(gamma_k, 0)) {
        DeviceInfo di;
        if ((st = device_info(&di)) != GEM_OK) return st;
        // All heads of a token in one warp, once that leaves 24 warps an SM: the angles are taken once and the
        // loads of the next head run behind the last one (4093 x 40 heads of 128: 34.4 us, with 8 heads a
        // warp 38.1); fewer for fewer tokens, down to one head a group of lanes.
        const int64_t all = T * P.nheads, side = d < 256 ? 256 / d : 1;
        int64_t per = (all + 24ll * di.num_sms - 1) / (24ll * di.num_sms);
        per = (per + side - 1) / side * side;
        int heads = static_cast<int>(std::max<int64_t>(side, std::min<int64_t>(per, P.nheads)));
        int chunks = (P.nheads + heads - 1) / heads;
        const int64_t blocks = (T * chunks + 7) / 8;
        if (blocks <= INT32_MAX / 8) {
            const void* kernel = d == 64    ? reinterpret_cast<const void*>(mrope_rows_kernel<64>)
                                 : d == 128 ? reinterpret_cast<const void*>(mrope_rows_kernel<128>)
                                 : d == 256 ? reinterpret_cast<const void*>(mrope_rows_kernel<256>)
                                            : reinterpret_cast<const void*>(mrope_rows_kernel<512>);
            void* vargs[] = {&P, const_cast<MropeFreq*>(&F), &heads, &chunks};
            return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, static_cast<cudaStream_t>(stream),
                              vargs);
        }
    }
    const int64_t blocks = (T * P.nheads + 3) / 4;
    if (blocks > INT32_MAX) return GEM_ERR_UNSUPPORTED_SHAPE;
    void* args[] = {&P, const_cast<MropeFreq*>(&F)};
    return launch_pdl(reinterpret_cast<const void*>(mrope_kernel), dim3(static_cast<unsigned>(blocks)), dim3(128), 0,
                      static_cast<cudaStream_t>(stream), args);
}
