// gem_fp8_gemm.cu — product of rows in 8-bit floating point with weights scaled by blocks of 128 x 128.
#include <cuda_fp8.h>

#include "gem_device.cuh"

namespace gem {
namespace {

struct GemmParams {
    const uint8_t* W;
    const float* ws;
    int N, K, M, kb;
    const uint8_t* x; int64_t ldx;
    const float* xs; int64_t ldxs;
    float* y; int64_t ldy;
    const float* res;
    int* status;
};

__device__ __forceinline__ float e4m3(uint8_t c) {
    __nv_fp8_e4m3 v;
    v.__x = c;
    return static_cast<float>(v);
}

// 64 x 64 results a CTA, 4 x 4 a thread; 16 of K at a time through shared memory.
__global__ void __launch_bounds__(256) fp8_gemm_kernel(const GemmParams p) {
    __shared__ float a[16][65], b[16][65];
    pdl_wait_trigger();
    const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {}, part[4][4] = {};
    for (int k0 = 0; k0 < p.K; k0 += 16) {
        for (int i = threadIdx.x; i < 1024; i += 256) {
            const int r = i >> 4, k = i & 15;
            a[k][r] = m0 + r < p.M ? e4m3(p.x[(m0 + r) * p.ldx + k0 + k]) : 0.f;
            b[k][r] = n0 + r < p.N ? e4m3(p.W[static_cast<int64_t>(n0 + r) * p.K + k0 + k]) : 0.f;
        }
        __syncthreads();
        for (int k = 0; k < 16; ++k)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) part[i][j] = fmaf(a[k][ty + 16 * i], b[k][tx + 16 * j], part[i][j]);
        __syncthreads();
        if ((k0 + 16) % 128 == 0 || k0 + 16 == p.K)
            for (int i = 0; i < 4; ++i)
                for (int j = 0; j < 4; ++j) {
                    const int m = min(m0 + ty + 16 * i, p.M - 1), n = min(n0 + tx + 16 * j, p.N - 1);
                    acc[i][j] = fmaf(part[i][j], p.xs[m * p.ldxs + k0 / 128] * p.ws[static_cast<int64_t>(n / 128) * p.kb + k0 / 128], acc[i][j]);
                    part[i][j] = 0.f;
                }
    }
    for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < p.M && n < p.N) p.y[m * p.ldy + n] = acc[i][j] + (p.res ? p.res[m * p.ldy + n] : 0.f);
        }
}

}  // namespace
}  // namespace gem

extern "C" {

gem_status gem_fp8_gemm(const void* W, const float* ws, int64_t N, int64_t K, const void* x, int64_t ldx,
                        const float* xs, int64_t ldxs, int64_t M, float* y, int64_t ldy, const float* residual,
                        int32_t* status, void* stream) {
    using namespace gem;
    if (M < 0 || N < 0 || K < 0) return GEM_ERR_INVALID_ARG;
    constexpr int64_t lim = (int64_t(1) << 31) - 512;
    if (K % 16 || M > lim || N > lim || K > lim) return GEM_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return GEM_OK;
    if (K == 0 || !W || !ws || !x || !xs || !y) return GEM_ERR_INVALID_ARG;
    if (ldx < K || ldxs < (K + 127) / 128 || ldy < N) return GEM_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(W) & 15) || (reinterpret_cast<uintptr_t>(x) & 15) || (ldx & 15) ||
        ((reinterpret_cast<uintptr_t>(ws) | reinterpret_cast<uintptr_t>(xs) | reinterpret_cast<uintptr_t>(y) |
          reinterpret_cast<uintptr_t>(residual) | reinterpret_cast<uintptr_t>(status)) & 3))
        return GEM_ERR_MISALIGNED;
    DeviceInfo di;
    gem_status st;
    if ((st = device_info(&di)) != GEM_OK) return st;
    GemmParams p{};
    p.W = static_cast<const uint8_t*>(W);
    p.ws = ws;
    p.N = static_cast<int>(N);
    p.K = static_cast<int>(K);
    p.M = static_cast<int>(M);
    p.kb = static_cast<int>((K + 127) / 128);
    p.x = static_cast<const uint8_t*>(x);
    p.ldx = ldx;
    p.xs = xs;
    p.ldxs = ldxs;
    p.y = y;
    p.ldy = ldy;
    p.res = residual;
    p.status = status ? status : di.status_word;
    void* args[] = {&p};
    return launch_pdl(reinterpret_cast<const void*>(fp8_gemm_kernel),
                      dim3(static_cast<unsigned>((N + 63) / 64), static_cast<unsigned>((M + 63) / 64)), dim3(256), 0,
                      static_cast<cudaStream_t>(stream), args);
}

}  // extern "C"
