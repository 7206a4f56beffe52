// gem_logprobs.cu — log probabilities of given tokens, their ranks, the entropy and the top alternatives of
// logit rows (gem_logprobs), in one pass over the logits.
//
// A thread keeps the largest logit m that it has seen, s = sum e^(l - m) and e = sum (l - m) e^(l - m), brings
// them to a new m where one comes, and after the pass they are joined the same way:
//     lse = m + log s,   entropy = log s - e / s.
// Both terms of the entropy are positive, so nothing cancels; l - m is formed before it is scaled, so that its
// error is relative.  The list of the k largest needs no second pass either: what can be in it is at least as
// large as the k-th largest of the first piece's warp maxima, and after that as the k-th in the list so far, so
// that a piece of 16 values a thread is looked at again only where its maximum passes that (a few of 10^5
// values do).  Banned entries (-inf) take part only where fewer than k others are left, and then the first k entries
// hold enough of them; a row whose numbers run out before that (NaN) is listed again, slowly.  The rank counts values
// only in pieces whose maximum reaches the given token's logit.
//
// Bound by the read of the logits where there are many: 1021 x 262144 takes 200 us (1.07 GB, 79 % of the copy rate; 197
// without a list).  61 x 151669 with 20 alternatives takes 24 us, 14 of them without a list: ten pieces a CTA, so
// beginning, listing and joining count; 1 x 262144 9.8 us with 5 alternatives, 7.2 without a list and 48 with 64, whose
// 16 parts hand on up to 128 keys each.  A row is one CTA's, or a cluster's, whose CTAs join their sums and lists
// through shared memory: no workspace, no counters, and an order that depends on the sizes alone.
#include <cmath>
#include <mutex>
#include <set>

#include "gem_tcgen05.cuh"

namespace gem {
namespace {

constexpr int kMaxTop = 64;
constexpr int kVec = 4;              // 16-byte loads of a thread in a piece of 16 values
constexpr int kHeld = 2048;          // keys that may wait to be sorted
constexpr float kLowest = -3.402823466e38f;
// Of the scale.  c = scale * log2 e stays finite and normal, and a difference of logits that passes the largest number
// has no weight at any of them.
constexpr float kLeastScale = 7.888609052210118e-31f, kMostScale = 1.2676506002282294e30f;   // 2^-100, 2^100

struct ScoreParams {
    const float* y; int64_t ldy;
    int64_t N;
    float scale;
    const int32_t* tokens;
    float* logp;
    int32_t* rank;
    float* entropy;
    int k, split;
    int32_t* idx;
    float* val;
    int* status;
};

// Order of the list as an integer: larger values first (NaN after every number), then, in a key's low word, lower indices.
__device__ __forceinline__ uint32_t order_of(float v) {
    v = v == 0.f ? 0.f : v;   // -0 and 0 are equal
    const uint32_t u = __float_as_uint(v);
    return v != v ? 0u : (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return o == 0 ? __int_as_float(0x7fffffff) : __uint_as_float((o & 0x80000000u) ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t key_of(float v, int64_t i) {
    return static_cast<uint64_t>(order_of(v)) << 32 | static_cast<uint32_t>(~static_cast<uint32_t>(i));
}

// Off by up to 2^-22 of the result, and x by its own roundings; a full exponential, off by 2^-24, would be several instructions
// more for each logit.  For the sum of a row it comes to 1e-7, a third of the last rounding of what leaves the kernel
// (300 rows of 151669: log p off by 2.9e-7 in the mean square, 3.7e-7 with full exponentials and no pairs; entropy 4.7e-7 and
// 4.3e-7).
__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

struct Sums {
    float m, s, e;   // e in powers of two: sum of w * log2 w
};
// c = scale * log2 e: e^(scale (a - b)) = 2^(c (a - b))
__device__ __forceinline__ void raise(Sums& a, float m, float c) {
    const float d = fmaxf((a.m - m) * c, -1e28f), f = exp2_fast(d);   // a sum of 2^31 times d is finite: it meets an f of 0
    a.e = f * fmaf(a.s, d, a.e);
    a.s *= f;
    a.m = m;
}
__device__ __forceinline__ Sums join(Sums a, Sums b, float c) {
    const float m = fmaxf(a.m, b.m);
    raise(a, m, c);
    raise(b, m, c);
    return {m, a.s + b.s, a.e + b.e};
}
__device__ __forceinline__ Sums shfl_xor(Sums a, int o) {
    return {__shfl_xor_sync(~0u, a.m, o), __shfl_xor_sync(~0u, a.s, o), __shfl_xor_sync(~0u, a.e, o)};
}

// What leaves the kernel: differences of numbers of about 10, each of which would cost a rounding as large as the last one.
// They are kept as pairs (Knuth's error-free sum), so that little but the last rounding is added to the sums' own error.
struct Pair {
    float hi, lo;
};
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = a + b, t = s - a;
    return {s, (a - (s - t)) + (b - t)};
}
// log s, 1 <= s < 2^32: k log 2 + log f, of which log 2 to 9 bits times k is exact (Cody and Waite's split); else NaN
__device__ __forceinline__ Pair log_pair(float s) {
    if (!(s > 0.f)) return {__int_as_float(0x7fffffff), 0.f};
    const uint32_t b = __float_as_uint(s);
    const int up = (b & 0x7fffffu) > 0x3504f3u, k = static_cast<int>(b >> 23) - 127 + up;   // 1.41421356
    const float f = __uint_as_float((b & 0x7fffffu) | static_cast<uint32_t>(127 - up) << 23), n = static_cast<float>(k);
    return {n * 0.693359375f, fmaf(n, -2.1219444005469058e-4f, logf(f))};
}
// scale * (v - m) - log s.  By halves: the difference may pass the largest number where its product with the scale does not.
__device__ __forceinline__ float log_prob(float v, float m, float scale, Pair log_s) {
    const Pair d = two_sum(0.5f * v, -0.5f * m);
    const float a = 2.f * (scale * d.hi);
    if (!(fabsf(a) < INFINITY)) return a - log_s.hi;
    const Pair r = two_sum(a, -log_s.hi);
    return r.hi + (r.lo - log_s.lo + 2.f * fmaf(scale, d.lo, fmaf(scale, d.hi, -0.5f * a)));
}
// log s - log 2 * e / s
__device__ __forceinline__ float entropy_of(float s, float e, Pair log_s) {
    const float q = e / s, l2 = -0.6931471805599453f, p = l2 * q;
    const Pair r = two_sum(log_s.hi, p);
    // what q's division left, what log 2 has beyond 24 bits, what the product lost
    return r.hi + (r.lo + log_s.lo + fmaf(l2, fmaf(-q, s, e) / s, fmaf(1.904654323148236e-9f, q, fmaf(l2, q, -p))));
}

template <int THREADS>
struct ScoreShared {
    unsigned long long held[kHeld];
    unsigned long long top[kMaxTop];
    Sums sums[THREADS / 32], all;
    uint32_t largest[THREADS / 32];
    int above[THREADS / 32], total;
    int n;
};

// x[j], without a place in memory for x
__device__ __forceinline__ float pick(const float (&x)[16], int j) {
    float a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = j & 8 ? x[i + 8] : x[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = j & 4 ? a[i + 4] : a[i];
#pragma unroll
    for (int i = 0; i < 2; ++i) a[i] = j & 2 ? a[i + 2] : a[i];
    return j & 1 ? a[1] : a[0];
}

// The k largest of the first n held keys (all different), in order, into sh.top and to the front of sh.held; sh.n
// becomes their number.  A key's place is the number of larger ones, counted by 1 to 32 lanes.  The keys have been
// written before a barrier; the result may be used at once.
template <int THREADS>
__device__ void sort_held(ScoreShared<THREADS>& sh, int n, int k) {
    const int tid = threadIdx.x;
    int shift = 5;
    while (shift > 0 && (n << shift) > THREADS) --shift;
    const int lanes = 1 << shift, part = tid & (lanes - 1), end = ((n << shift) + 31) & ~31;
    for (int at = tid; at < end; at += THREADS) {
        const int i = at >> shift;
        const unsigned long long mine = i < n ? sh.held[i] : ~0ull;
        int place = 0;
        for (int j = part; j < n; j += lanes) place += sh.held[j] > mine;
        for (int o = lanes >> 1; o > 0; o >>= 1) place += __shfl_xor_sync(~0u, place, o);
        if (part == 0 && i < n && place < k) sh.top[place] = mine;
    }
    __syncthreads();
    if (tid < min(n, k)) sh.held[tid] = sh.top[tid];
    if (tid == 0) sh.n = min(n, k);
    __syncthreads();
}

// The list of entries v0 .. v1 (16-byte pieces behind `head`) and of `more` single ones, where more came together
// than can wait (rising values), or too few (NaN): one entry a thread at a time, sorted as often as need be.
template <int THREADS>
__device__ __noinline__ void list_slowly(ScoreShared<THREADS>& sh, const float* row, int head, int64_t v0, int64_t v1, int64_t nv, int more, int k) {
    const int tid = threadIdx.x;
    unsigned long long least_key = 0;
    int n = 0;
    for (int64_t at = 4 * v0 - (more + 3) / 4 * 4; at < 4 * v1; at += THREADS) {
        __syncthreads();
        if (n + THREADS > kHeld) {
            sort_held(sh, n, k);
            n = min(n, k);
            least_key = n == k ? sh.top[k - 1] : 0ull;
        }
        if (tid == 0) sh.n = n;
        __syncthreads();
        const int64_t j = at + tid;   // below 4 v0: the single entries
        const int single = static_cast<int>(4 * v0 - j) - 1;
        if (j < 4 * v1 && (j >= 4 * v0 || single < more)) {
            const int64_t i = j >= 4 * v0 ? head + j : single < head ? single : 4 * nv + single;
            const unsigned long long key = key_of(row[i], i);
            if (key > least_key) sh.held[atomicAdd(&sh.n, 1)] = key;
        }
        __syncthreads();
        n = sh.n;
    }
}

template <int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) logprobs_kernel(const ScoreParams p) {
    __shared__ ScoreShared<THREADS> sh;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int W = THREADS / 32;
    const int64_t t = blockIdx.x / p.split;
    const int part = static_cast<int>(blockIdx.x % p.split);
    const float* row = p.y + t * p.ldy;
    // 16-byte pieces from the first aligned entry on; the entries before and after them are the first CTA's
    const int head = static_cast<int>(min(static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(row) & 15)) / 4 & 3), p.N));
    const int64_t nv = (p.N - head) / 4;
    const int more = part == 0 ? head + static_cast<int>(p.N - head - 4 * nv) : 0;
    const int64_t per = (nv + p.split - 1) / p.split, v0 = min(nv, per * part), v1 = min(nv, v0 + per);
    const float c = p.scale * 1.4426950408889634f;
    const int k = p.k;
    pdl_wait_trigger();

    // This thread's 16-byte pieces are first, first + THREADS, .. of the CTA's `len`; the next ones are on their way
    // while it works on the last (through shared memory, two or three deep, they came no faster).
    const float4* from = reinterpret_cast<const float4*>(row + head) + v0 + tid;
    const int len = static_cast<int>(v1 - v0);
    float4 next[kVec];
    auto request = [&](int at) {
        if (at + THREADS * kVec <= len) {
#pragma unroll
            for (int u = 0; u < kVec; ++u) next[u] = __ldcs(from + at + u * THREADS);
        } else {
#pragma unroll
            for (int u = 0; u < kVec; ++u)
                next[u] = at + u * THREADS + tid < len ? __ldcs(from + at + u * THREADS) : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        }
    };
    request(0);
    const int tok = p.tokens ? p.tokens[t] : -1;
    const bool given = tok >= 0 && tok < p.N, count = given && p.rank;
    const float target = given ? row[tok] : 0.f;
    auto is_above = [&](float v, int64_t i) {
        if (target != target) return v == v || i < tok;
        return v > target || (v == target && i < tok);
    };

    Sums sum{kLowest, 0.f, 0.f};
    int above = 0;
    unsigned long long least_key = 0;   // the list's least key; what is not above it is not looked at
    float floor_v = kLowest;            // its value, or the least finite one
    if (tid == 0) sh.n = 0;
    __syncthreads();
    if (tid < more) {
        const int64_t i = tid < head ? tid : 4 * nv + tid;
        const float v = row[i], m = fmaxf(v, kLowest), d = (v - m) * c, w = exp2_fast(d);
        sum = {m, w, fmaxf(d, -200.f) * (d < -200.f ? 0.f : w)};
        above += count && is_above(v, i);
        if (k && (v > -INFINITY || (v == v && tid < head))) sh.held[atomicAdd(&sh.n, 1)] = key_of(v, i);
    }
    // of entries before the given token equal ones are above it too; behind it nothing is above +inf, and a NaN bars all
    const float bound_before = target, bound_after = target == INFINITY ? __int_as_float(0x7fffffff) : nextafterf(target, INFINITY);
    int turn = 0, look_at = k == 0 ? 1 << 30 : k > W ? 0 : 1;
    for (int at = 0; at < len; at += THREADS * kVec, ++turn) {
        float x[4 * kVec];
#pragma unroll
        for (int u = 0; u < kVec; ++u) x[4 * u] = next[u].x, x[4 * u + 1] = next[u].y, x[4 * u + 2] = next[u].z, x[4 * u + 3] = next[u].w;
        request(at + THREADS * kVec);
        float most = x[0];
#pragma unroll
        for (int j = 1; j < 4 * kVec; ++j) most = fmaxf(most, x[j]);
        if (most > sum.m) raise(sum, most, c);
        float2 s2 = make_float2(0.f, 0.f), e2 = s2;
        const float2 m2 = make_float2(-sum.m, -sum.m), c2 = make_float2(c, c);
#pragma unroll
        for (int j = 0; j < 4 * kVec; j += 2) {
            const float2 d = fmul2(fadd2(make_float2(x[j], x[j + 1]), m2), c2), w = make_float2(exp2_fast(d.x), exp2_fast(d.y));
            s2 = fadd2(s2, w);
            e2 = ffma2(make_float2(fmaxf(d.x, -200.f), fmaxf(d.y, -200.f)), w, e2);   // w is 0 there; a NaN is in s
        }
        sum.s += s2.x + s2.y;
        sum.e += e2.x + e2.y;
        // bit j: entry j is there
        const int left = len - at - tid;
        const uint32_t valid = left <= 0 ? 0u : left > (kVec - 1) * THREADS ? 0xffffu : (1u << 4 * ((left + THREADS - 1) / THREADS)) - 1;
        auto index = [&](int j) { return head + 4 * (v0 + at + (j >> 2) * THREADS + tid) + (j & 3); };
        auto at_least = [&](float bound) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 4 * kVec; ++j) m |= x[j] >= bound ? 1u << j : 0u;
            return m;
        };
        if (count) {
            const int64_t low = head + 4 * (v0 + at), high = low + 4 * THREADS * kVec;
            if (target != target || (tok >= low && tok < high)) {   // one by one: here an entry's place counts
                for (int j = 0; j < 4 * kVec; ++j) above += (valid >> j & 1) && is_above(pick(x, j), index(j));
            } else {
                const float bound = tok >= high ? bound_before : bound_after;
                if (most >= bound) above += __popc(at_least(bound) & valid);
            }
        }
        if (k == 0) continue;
        if (turn == 0) {
            // At least k entries of the piece reach the k-th largest of the warps' maxima, or, with a longer list than
            // warps, the least of the warps' q-th largest lane maxima, q = ceil(k / warps).
            uint32_t o = most > -INFINITY ? order_of(most) : 0u, w = 0;   // -inf may stand for a NaN, or for no entry
            for (int q = (k + W - 1) / W; q > 0; --q) {
                w = __reduce_max_sync(~0u, o);
                if (o == w) o = 0;
            }
            if (lane == 0) sh.largest[warp] = w;
            __syncthreads();
            const uint32_t b = lane < W ? sh.largest[lane] : 0u;
            uint32_t bar;
            if (k > W) {
                bar = __reduce_min_sync(~0u, lane < W ? b : ~0u);
            } else {
                int larger = 0;
                for (int q = 0; q < W; ++q) {
                    const uint32_t other = __shfl_sync(~0u, b, q);
                    larger += other > b || (other == b && q < lane);
                }
                bar = __reduce_max_sync(~0u, lane < W && larger == k - 1 ? b : 0u);
            }
            least_key = bar ? (static_cast<unsigned long long>(bar) << 32) - 1 : 0ull;
            floor_v = bar ? value_of(bar) : kLowest;
        }
        const bool banned = turn == 0 && 4 * tid < k;   // among the first k entries
        if (most >= floor_v || banned) {
            uint32_t mask = at_least(floor_v);
            if (banned)
#pragma unroll
                for (int j = 0; j < 4; ++j) mask |= x[j] == -INFINITY && 4 * tid + j < k ? 1u << j : 0u;
            for (mask &= valid; mask; mask &= mask - 1) {
                const int j = __ffs(mask) - 1;
                const unsigned long long key = key_of(pick(x, j), index(j));
                if (key > least_key) {
                    const int pos = atomicAdd(&sh.n, 1);
                    if (pos < kHeld) sh.held[pos] = key;   // else all is listed again, below
                }
            }
        }
        // The list so far raises the bar, after 1 (2), 4, 8, 16, .. pieces: then about k entries pass it in as many again.
        if (turn == look_at) {
            look_at = 2 * turn + 1;
            __syncthreads();
            const int n = sh.n;
            if (n <= kHeld && n > k) {
                sort_held(sh, n, k);
                least_key = sh.top[k - 1];
                floor_v = fmaxf(value_of(static_cast<uint32_t>(least_key >> 32)), kLowest);
            }
            __syncthreads();
        }
    }

    for (int o = 16; o > 0; o >>= 1) {
        sum = join(sum, shfl_xor(sum, o), c);
        above += __shfl_xor_sync(~0u, above, o);
    }
    if (lane == 0) sh.sums[warp] = sum, sh.above[warp] = above;
    __syncthreads();
    if (k) {
        if (sh.n > kHeld || sh.n < min(static_cast<int64_t>(k), 4 * (v1 - v0) + more)) list_slowly(sh, row, head, v0, v1, nv, more, k);
        // a part of a row hands on a short list as it is
        if (p.split == 1 || sh.n > max(2 * k, 16)) sort_held(sh, sh.n, k);
    }
    if (warp == 0) {
        sum = lane < W ? sh.sums[lane] : Sums{kLowest, 0.f, 0.f};
        above = lane < W ? sh.above[lane] : 0;
        for (int o = 16; o > 0; o >>= 1) {
            sum = join(sum, shfl_xor(sum, o), c);
            above += __shfl_xor_sync(~0u, above, o);
        }
        if (lane == 0) sh.all = sum, sh.total = above;
    }
    __syncthreads();
    if (p.split > 1) {
        int listed = 0;
        cluster_sync();
        if (part == 0) {
            if (warp == 0) {
                sum = {kLowest, 0.f, 0.f};
                above = 0;
                if (lane < p.split) {
                    const uint32_t a = peer_addr(&sh.all, lane);
                    sum = {ld_peer(a), ld_peer(a + 4), ld_peer(a + 8)};
                    above = __float_as_int(ld_peer(peer_addr(&sh.total, lane)));
                }
                for (int o = 16; o > 0; o >>= 1) {
                    sum = join(sum, shfl_xor(sum, o), c);
                    above += __shfl_xor_sync(~0u, above, o);
                }
            }
            // the parts' lists one behind the other (this one's is in its place); a warp fetches every W-th
            const int m = lane < p.split ? __float_as_int(ld_peer(peer_addr(&sh.n, lane))) : 0;
            int n = m;   // up to and with part `lane`
            for (int o = 1; o < 32; o <<= 1) {
                const int other = __shfl_up_sync(~0u, n, o);
                n += lane >= o ? other : 0;
            }
            for (int r = 1 + warp; r < p.split; r += W) {
                const int size = __shfl_sync(~0u, m, r), to = __shfl_sync(~0u, n, r - 1);
                for (int i = lane; i < size; i += 32) {
                    const uint32_t a = peer_addr(&sh.held[i], r);
                    sh.held[to + i] = static_cast<unsigned long long>(__float_as_uint(ld_peer(a + 4))) << 32 | __float_as_uint(ld_peer(a));
                }
            }
            n = __shfl_sync(~0u, n, 31);
            listed = n;
            __syncthreads();
            if (tid == 0) sh.all = sum, sh.total = above;
        }
        __syncwarp();
        cluster_sync();   // what the others hold has been read
        if (part != 0) return;
        if (k) sort_held(sh, listed, k);
    }
    sum = sh.all;
    // no finite logit, or one that is not a number
    const Pair log_s = log_pair(sum.s);
    if (tid == 0) {
        if (p.entropy) p.entropy[t] = entropy_of(sum.s, sum.e, log_s);
        if (p.tokens) {
            if (!given && tok != -1) atomicOr(p.status, GEM_DEVFLAG_POS_RANGE);
            if (p.logp) p.logp[t] = given ? log_prob(target, sum.m, p.scale, log_s) : tok == -1 ? 0.f : __int_as_float(0x7fffffff);
            if (p.rank) p.rank[t] = given ? sh.total + 1 : 0;
        }
    }
    if (tid < k) {
        const unsigned long long key = sh.top[tid];
        p.idx[t * k + tid] = static_cast<int>(~static_cast<uint32_t>(key));
        p.val[t * k + tid] = log_prob(value_of(static_cast<uint32_t>(key >> 32)), sum.m, p.scale, log_s);
    }
}

}  // namespace
}  // namespace gem

extern "C" {

gem_status gem_logprobs(const float* y, int64_t ldy, int64_t T, int64_t N, float scale, const int32_t* tokens,
                        float* logp, int32_t* rank, float* entropy, int k, int32_t* idx, float* val, int32_t* status,
                        void* stream) {
    using namespace gem;
    if (T < 0 || N < 1 || k < 0 || k > N || !(scale >= kLeastScale && scale <= kMostScale)) return GEM_ERR_INVALID_ARG;
    if (k > kMaxTop || N >= (int64_t(1) << 31) || T >= (int64_t(1) << 28)) return GEM_ERR_UNSUPPORTED_SHAPE;
    if (T == 0) return GEM_OK;
    if (!y || ldy < N || (k && (!idx || !val)) || ((logp || rank) && !tokens)) return GEM_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(y) | reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(logp) |
         reinterpret_cast<uintptr_t>(rank) | reinterpret_cast<uintptr_t>(entropy) | reinterpret_cast<uintptr_t>(idx) |
         reinterpret_cast<uintptr_t>(val) | reinterpret_cast<uintptr_t>(status)) & 3)
        return GEM_ERR_MISALIGNED;
    DeviceInfo di;
    gem_status st;
    if ((st = device_info(&di)) != GEM_OK) return st;
    ScoreParams p{y, ldy, N, scale, tokens, logp, rank, entropy, k, 1, idx, val, status ? status : di.status_word};
    // Few rows: 16 CTAs of 512 threads a row (a cluster of that size wants the kernel's consent).  Else 256 threads, and
    // as many CTAs a row as take the shortest time.  A piece takes 0.5 us where an SM has one or two CTAs and 1.1 us where
    // it has the four that it holds; beginning, listing and joining take as long as 32 pieces; of clusters fewer fit.
    // (61 x 151669, list of 20: 4 CTAs a row 23 us, 2 28, 8 25; 150 rows: 2 CTAs 27 us, 4 35.)
    const bool few = T <= 4;
    const int threads = few ? 512 : 256;
    const int64_t pieces = (N / 4 + threads * kVec - 1) / (threads * kVec);
    const void* fn = few ? reinterpret_cast<const void*>(logprobs_kernel<512>) : reinterpret_cast<const void*>(logprobs_kernel<256>);
    if (few) {
        while (p.split < 16 && p.split < pieces) p.split *= 2;
        static std::mutex mu;
        static std::set<int> done;
        std::lock_guard<std::mutex> lk(mu);
        if (done.insert(di.device).second) GEM_CUDA_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
    } else {
        double best = 1e30;
        for (int s : {1, 2, 4, 8}) {
            if (s > 1 && s > pieces) break;
            const int64_t ctas = T * s, an_sm = (ctas + di.num_sms - 1) / di.num_sms;
            const double slots = di.num_sms * (s > 1 ? 3.7 : 4.0), rounds = std::ceil(static_cast<double>(ctas) / slots);
            const double piece = an_sm <= 2 ? 1.0 : an_sm == 3 ? 1.5 : 2.2;
            const double cost = rounds * (static_cast<double>((pieces + s - 1) / s) * piece + 32.0);
            if (cost < best) {
                best = cost;
                p.split = s;
            }
        }
    }
    void* args[] = {&p};
    return launch_pdl_cluster(fn, dim3(static_cast<unsigned>(T * p.split)), dim3(threads), 0, static_cast<cudaStream_t>(stream), args, p.split);
}

}  // extern "C"
