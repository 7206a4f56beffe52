// gem_logprobs.cu — log probabilities of given tokens, their ranks, the entropy and the top alternatives of
// logit rows.
#include "gem_device.cuh"

namespace gem {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxTop = 64;

struct ScoreParams {
    const float* y; int64_t ldy;
    int64_t N;
    float scale;
    const int32_t* tokens;
    float* logp;
    int32_t* rank;
    float* entropy;
    int k;
    int32_t* idx;
    float* val;
    int* status;
};

// 64-bit keys in the order of the list: larger values first (NaN after every number), then lower indices
__device__ __forceinline__ uint64_t key_of(float v, int64_t i) {
    v = v == 0.f ? 0.f : v;   // -0 and 0 are equal
    uint32_t u = __float_as_uint(v);
    u = v != v ? 0u : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
    return static_cast<uint64_t>(u) << 32 | static_cast<uint32_t>(~static_cast<uint32_t>(i));
}

template <class T, class F>
__device__ T cta_reduce(T v, T* red, F f) {
    for (int o = 16; o > 0; o >>= 1) v = f(v, __shfl_xor_sync(~0u, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
    for (int i = 1; i < kThreads / 32; ++i) v = f(v, red[i]);
    return v;
}

__global__ void __launch_bounds__(kThreads) logprobs_kernel(const ScoreParams p) {
    __shared__ unsigned long long red64[kThreads / 32];
    __shared__ float red32[kThreads / 32];
    pdl_wait_trigger();
    const int64_t t = blockIdx.x;
    const float* row = p.y + t * p.ldy;
    auto larger = [](float a, float b) { return a > b || a != a ? a : b; };   // keeps a NaN
    auto sum = [](float a, float b) { return a + b; };
    float m = -INFINITY;
    for (int64_t i = threadIdx.x; i < p.N; i += kThreads) m = larger(row[i], m);
    m = cta_reduce(m, red32, larger);
    float s = 0.f, e = 0.f;
    for (int64_t i = threadIdx.x; i < p.N; i += kThreads) {
        const float d = p.scale * (row[i] - m), w = expf(d);
        s += w;
        if (w != 0.f) e = fmaf(w, d, e);
    }
    s = cta_reduce(s, red32, sum);
    e = cta_reduce(e, red32, sum);
    const float log_s = logf(s);
    if (p.entropy && threadIdx.x == 0) p.entropy[t] = log_s - e / s;
    if (p.tokens) {
        const int tok = p.tokens[t];
        const bool given = tok >= 0 && tok < p.N;
        unsigned long long above = 0;
        if (given && p.rank) {
            const uint64_t mine = key_of(row[tok], tok);
            for (int64_t i = threadIdx.x; i < p.N; i += kThreads) above += key_of(row[i], i) > mine;
            above = cta_reduce(above, red64, [](unsigned long long a, unsigned long long b) { return a + b; });
        }
        if (threadIdx.x == 0) {
            if (!given && tok != -1) atomicOr(p.status, GEM_DEVFLAG_POS_RANGE);
            if (p.logp) p.logp[t] = given ? p.scale * (row[tok] - m) - log_s : tok == -1 ? 0.f : __int_as_float(0x7fffffff);
            if (p.rank) p.rank[t] = given ? static_cast<int>(above) + 1 : 0;
        }
    }
    unsigned long long last = ~0ull;
    for (int r = 0; r < p.k; ++r) {
        unsigned long long best = 0;
        for (int64_t i = threadIdx.x; i < p.N; i += kThreads) {
            const unsigned long long q = key_of(row[i], i);
            if (q < last && q > best) best = q;
        }
        last = cta_reduce(best, red64, [](unsigned long long a, unsigned long long b) { return a > b ? a : b; });
        if (threadIdx.x == 0) {
            const int i = static_cast<int>(~static_cast<uint32_t>(last));
            p.idx[t * p.k + r] = i;
            p.val[t * p.k + r] = p.scale * (row[i] - m) - log_s;
        }
    }
}

}  // namespace
}  // namespace gem

extern "C" {

size_t gem_logprobs_workspace(int64_t T, int64_t N, int k) {
    (void)T, (void)N, (void)k;
    return 0;
}

gem_status gem_logprobs(const float* y, int64_t ldy, int64_t T, int64_t N, float scale, const int32_t* tokens,
                        float* logp, int32_t* rank, float* entropy, int k, int32_t* idx, float* val, void* workspace,
                        size_t ws_bytes, int32_t* status, void* stream) {
    using namespace gem;
    if (T < 0 || N < 1 || k < 0 || k > N || !(scale > 0.f) || !(scale <= 3.402823466e38f)) return GEM_ERR_INVALID_ARG;
    if (k > kMaxTop || N >= (int64_t(1) << 31) || T > ((int64_t(1) << 31) - 1) / ((N + 2047) / 2048))
        return GEM_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return GEM_OK;
    if (!y || ldy < N || (k && (!idx || !val)) || ((logp || rank) && !tokens)) return GEM_ERR_INVALID_ARG;
    const size_t need = gem_logprobs_workspace(T, N, k);
    if (need && (!workspace || ws_bytes < need)) return GEM_ERR_WORKSPACE;
    if (need && (reinterpret_cast<uintptr_t>(workspace) & 255)) return GEM_ERR_MISALIGNED;
    if ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(logp) |
         reinterpret_cast<uintptr_t>(rank) | reinterpret_cast<uintptr_t>(entropy) | reinterpret_cast<uintptr_t>(idx) |
         reinterpret_cast<uintptr_t>(val) | reinterpret_cast<uintptr_t>(status)) & 3)
        return GEM_ERR_MISALIGNED;
    DeviceInfo di;
    gem_status st;
    if ((st = device_info(&di)) != GEM_OK) return st;
    ScoreParams p{y, ldy, N, scale, tokens, logp, rank, entropy, k, idx, val, status ? status : di.status_word};
    void* args[] = {&p};
    return launch_pdl(reinterpret_cast<const void*>(logprobs_kernel), dim3(static_cast<unsigned>(T)), dim3(kThreads), 0,
                      static_cast<cudaStream_t>(stream), args);
}

}  // extern "C"
