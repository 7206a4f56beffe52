// gem_kv4_attn.cu — grouped-query attention over the paged 4-bit KV cache.
//
// Mathematics.  For a query row q (one token, one query head) and the cached rows of its KV head,
//   out = sum_j p_j V_j / sum_j p_j,   p_j = 2^(c q.K_j - m),  c = scale * log2(e),
// in one pass with a running maximum m.  K and V are (code - 8) * s with one scale s per position and
// 32 dims, so with blocks b of 32 dims
//   q.K_j  = sum_b sK[j][b] sum_{e in b} q_e (code_je - 8)
//   out_e ~  sum_j (p_j sV[j][b]) (code_je - 8),  e in b.
//
// Tensor cores.  mma.sync m16n8k16 with the codes as the 16-row operand.  A nibble put into the low
// mantissa bits of 1024 is the binary16 number 1024 + code (1024 + 16 code for the next nibble), and
// one packed add or fma leaves code - 8, exactly: 9 instructions for 8 codes, 4 of them not on the
// integer pipe.  (The codes could enter as they are, as subnormals code * 2^-24 in 5 instructions, with
// the 8 taken out of the sums; measured, that costs 7 bits: products are aligned by their operands'
// exponent fields before they are added, and a relative error of 1.2e-5 was left.)  q, and p times V's
// scale, are fp32 and enter as binary16 hi + lo pairs (about 22 bits) under powers of two that keep
// them in binary16's range; up to four query rows put both halves into the eight columns of one
// instruction, more rows take two.  Each row has a power for every block of 32 dims, of q once a unit, of p sV in
// each step: one for all blocks loses the bits of the small ones (blocks 2^24 apart were 1e-4 off for q, 2e-2
// for V).
// The wide tcgen05 path wants both operands in binary16 or fp8 tiles in shared memory.  In decoding one
// operand is 4-bit codes and would first be written out four times as large, for eight columns of output, so
// the unpacking, not the multiply rate, would bound it just the same.  (That does not hold for chunks: 32 new
// tokens of four heads are the 128 rows of a tile.  They run here too, in units of 16 rows.)
//
// Schedule.  The work is (request, KV head, group of query rows) units of steps of 32 positions.  Their
// number is known on the device only, so a fixed grid of warps takes equal contiguous shares of all
// steps.  A warp streams its tiles with cp.async.bulk through a ring of its own and keeps its own
// running maximum, sum and output; a unit inside one share is written out at once, the parts of one
// that crosses shares are joined first inside the CTA, then, in order, by a second kernel.
#include <algorithm>
#include <cmath>
#include <mutex>
#include <type_traits>

#include "gem_device.cuh"
#include "gem_kv4.cuh"

namespace gem {
namespace kv4 {
namespace {

constexpr int kMaxGroup = 8;
constexpr int kStepTiles = 2;
constexpr int kStepTokens = kStepTiles * kTileTokens;
constexpr int kStages = 2;
constexpr int kSlack = 6;                   // log2 of how far a score may pass the maximum in use
// A row of probabilities in shared memory, in floats.  8 modulo 32 keeps the rows in banks of their own; the 8 behind
// the probabilities hold what takes q's powers of two back, for a block of dims and eight query rows.
constexpr int kProbRow = kStepTokens + 8;

struct AttnParams {
    const float* q;
    int64_t ldq, T;
    const int32_t *cu, *kv_len;
    int B, n_q, n_kv, G, GT;      // GT: tokens of a unit (GT * G query rows)
    int inv_g;                    // 2^16 / G rounded up: a row's token is row * inv_g / 2^16
    const int32_t* table;
    int64_t max_pages;
    const uint8_t* pool;
    int64_t n_pages;
    int lpage, window;
    float scale;
    float* out;
    int64_t ldo;
    int4* tasks;                  // workspace: one a worker, see the joining kernel
    float* part;                  // workspace: 2 slots a worker
    int workers;
    int* status;
};

// ---- what a request asks for ---------------------------------------------------------------------

struct Request {
    int row0, n, L;       // first query row, query rows, cached positions
    int tile0, steps;     // first tile that any row attends, steps from there on
    int groups;           // units of one KV head
};

__device__ __forceinline__ bool request_of(const AttnParams& P, int b, Request& r) {
    const int64_t c0 = P.cu[b], c1 = P.cu[b + 1], L = P.kv_len[b];
    r.row0 = static_cast<int>(c0);
    r.n = 0, r.L = 0, r.tile0 = 0, r.steps = 0, r.groups = 0;
    if (c0 < 0 || c0 > c1 || c1 > P.T || L < c1 - c0 || L > (P.max_pages << P.lpage)) return false;
    r.n = static_cast<int>(c1 - c0);
    r.L = static_cast<int>(L);
    if (r.n == 0) return true;
    r.tile0 = P.window ? max(0, r.L - r.n + 1 - P.window) / kTileTokens : 0;
    r.steps = ((r.L - 1) / kTileTokens - r.tile0) / kStepTiles + 1;
    r.groups = P.GT == 1 ? r.n : (r.n + P.GT - 1) / P.GT;
    return true;
}

// a / b; the usual case in 32 bits
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The query rows of unit u of request b: tokens j0 .. j0 + tokens - 1 of the request, positions p0 on.
struct Unit {
    int row0, h, j0, tokens, p0;
    int lo_all, hi_all;    // first and last position that any row attends
    int lo_max;            // from here to p0 every row attends
    int L, tile0, steps;   // of the request
    int units;             // of the request
    __device__ __forceinline__ Unit(const AttnParams& P, const Request& r, int u) {
        h = r.groups == 1 ? u : u / r.groups;
        j0 = (u - h * r.groups) * P.GT;
        tokens = min(P.GT, r.n - j0);
        row0 = r.row0 + j0;
        p0 = r.L - r.n + j0;
        hi_all = p0 + tokens - 1;
        lo_all = P.window ? max(0, p0 - P.window + 1) : 0;
        lo_max = P.window ? max(0, hi_all - P.window + 1) : 0;
        L = r.L, tile0 = r.tile0, steps = r.steps, units = r.groups * P.n_kv;
    }
};

// The unit after unit u of request b, which has `units`; there is one.
__device__ __forceinline__ Unit next_unit(const AttnParams& P, int units, int& b, int& u) {
    Request r;
    if (++u == units) {
        u = 0;
        do request_of(P, ++b, r);
        while (r.n == 0 && b < P.B - 1);
    } else {
        request_of(P, b, r);
    }
    return Unit(P, r, u);
}

// ---- small pieces ----------------------------------------------------------------------------------

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// D = A B
__device__ __forceinline__ void mma_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// Word of 8 codes, nibbles n0 .. n7 from the low end -> (n0, n4), (n1, n5), (n2, n6), (n3, n7), less 8 each.  (Integers
// put into the mantissa of a power of two are an old way to convert them; for 4-bit weights and binary16 it is
// described by Kim, Henry, Fahim and Awadalla, "Who Says Elephants Can't Run", 2022.)
struct Codes {
    uint32_t v[4];
};
__device__ __forceinline__ Codes codes_of(uint32_t w) {
    constexpr uint32_t kMagic = 0x64006400u;   // 1024, 1024
    uint32_t x[4];
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(x[0]) : "r"(w), "r"(kMagic));   // (a & b) | c
    asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(x[1]) : "r"(w), "r"(kMagic));
    const uint32_t u = w >> 8;
    asm("lop3.b32 %0, %1, 0x000f000f, %2, 0xea;" : "=r"(x[2]) : "r"(u), "r"(kMagic));
    asm("lop3.b32 %0, %1, 0x00f000f0, %2, 0xea;" : "=r"(x[3]) : "r"(u), "r"(kMagic));
    Codes c;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(c.v[i]) : "r"(x[i]), "r"(0xe408e408u));                       // - 1032
        asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(c.v[i + 1]) : "r"(x[i + 1]), "r"(0x2c002c00u), "r"(0xd480d480u));   // / 16 - 72
    }
    return c;
}

// (lo, hi) halves of a register, rounded toward zero
__device__ __forceinline__ uint32_t pack_rz(float lo, float hi) {
    uint32_t r;
    asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_rn(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float2 fmul2(float2 a, float2 b) {
    uint64_t ra, rb, rd;
    asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
    return d;
}
// the 11 leading significant bits, negated where flip is the sign bit
__device__ __forceinline__ float lead(float x, uint32_t flip) {
    return __uint_as_float((__float_as_uint(x) & 0xffffe000u) ^ flip);
}
// The power of two that brings x >= 0 into [2^14, 2^15), and its inverse.  (Below 2^-112 the power stays; infinity
// stays infinity.)
struct Scale2 {
    float up, down;
};
__device__ __forceinline__ Scale2 scale_to_2_14(float x) {
    const uint32_t e = max(__float_as_uint(x) & 0x7f800000u, 15u << 23);
    return {__uint_as_float((268u << 23) - e), __uint_as_float(e - (14u << 23))};
}

// A partial result in memory: rows of D sums, then (maximum, sum) of each row.
template <int D, int ROWS>
struct Part {
    static constexpr int kFloats = ROWS * (D + 2);
};

template <int D, int NT, bool PACK, int DW, int WARPS>
struct Cfg {
    static constexpr int kWarps = WARPS, kThreads = 32 * WARPS;
    static constexpr int kRows = PACK ? 4 : 8 * NT;      // query rows of a unit
    static constexpr int kDims = DW;                     // dims of one warp
    static constexpr int kPair = D / kDims;              // warps of a worker
    static constexpr int kBlocks = kDims / 32;
    static constexpr int kTile = tile_bytes(kDims);      // a tile's bytes in one warp's ring
    static constexpr int kStage = kStepTiles * kTile;
    static constexpr int kPartBytes = Part<D, kRows>::kFloats * 4;
    static constexpr int kRingNeed = (kPartBytes / kPair + 127) / 128 * 128;   // the ring later holds a partial result
    static constexpr int kRing = kStages * kStage > kRingNeed ? kStages * kStage : kRingNeed;
    static constexpr int kScales = kStepTiles * kBlocks * 192;   // fp32: K's 16 twice, V's 16
    static constexpr int kProbs = kRows * kProbRow * 4;
    static constexpr int kSwap = kPair > 1 ? kStages * kStepTiles * NT * 32 * 16 : 0;   // a buffer for each stage
    static constexpr int kWarpBytes = kRing + kScales + kProbs + kSwap;
    static constexpr int kWorkers = kWarps / kPair;      // of a CTA
    static size_t smem(int B) {
        return kWarps * static_cast<size_t>(kWarpBytes) + kWarps * kStages * 8 + (B > 32 ? (B + 1) * 8 : 0);
    }
};

// ---- the kernel ------------------------------------------------------------------------------------
//
// What bounds it: the warp instructions, about 850 a step of 32 positions at d 128 and four rows, of
// which unpacking the codes is 290 and splitting p times V's scale, with its powers of two, 180, and their
// latency, with three warps a scheduler issuing in 57 % of the cycles.  8 requests of up to 32,768 positions
// (32 / 8 heads, d 128, 257 MB): 75 us, 3.4 TB/s, 50 % of the measured copy rate (68 us with one power of two for all
// blocks, which loses bits).  Short batches are latency: 1 x 4097 positions take 9.3 us.
// One CTA of 12 warps an SM has 168 registers a thread for the sums, q and the operands under way; two of
// 8 have 128, spill, and took 71 us there against 66.7 at that point, 15.1 against 12.9 for 8 requests of up
// to 2049 positions; 10 warps took 76 and 12.1.
// Steps of 32 positions: with 16 the per-step work (waits, maxima, requests) weighs twice (85 us against
// 71 with two CTAs), and longer ones do not fit shared memory twice for every warp.

template <int D, int NT, bool PACK, int DW, int WARPS, int CTAS>
__global__ void __launch_bounds__(32 * WARPS, CTAS) kv4_attn_kernel(const AttnParams P) {
    using C = Cfg<D, NT, PACK, DW, WARPS>;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
    constexpr int NB = C::kBlocks, ROWS = C::kRows, PAIR = C::kPair;
    constexpr int NH = PACK ? 1 : 2;                     // B operands of a product: (hi | lo) or hi, lo
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int64_t sums[kWarps];
    __shared__ int tail_unit[C::kWorkers];
    __shared__ float weight[C::kWorkers * ROWS];
    __shared__ volatile int gave_up[kWarps];             // a wait of this warp ran out

    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int member = warp % PAIR;                      // which dims of the head this warp has
    const int worker = blockIdx.x * C::kWorkers + warp / PAIR;
    uint8_t* ring = smem + warp * C::kWarpBytes;
    float* scales = reinterpret_cast<float*>(ring + C::kRing);
    float* probs = reinterpret_cast<float*>(ring + C::kRing + C::kScales);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWarps * C::kWarpBytes) + warp * kStages;
    int64_t* plan = reinterpret_cast<int64_t*>(smem + kWarps * C::kWarpBytes + kWarps * kStages * 8);

    if (lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&bars[i], 1);
        fence_mbar_init();
        gave_up[warp] = 0;
    }
    __syncwarp();
    pdl_wait_trigger();

    // this worker's share of all steps, and the request and unit that it begins in
    Request r0;
    int b0 = 0;
    int64_t total, in_b0 = 0;
    auto split = [&]() { return quotient(total + P.workers - 1, P.workers); };
    if (P.B <= 32) {           // every warp for itself, a request a lane
        Request r;
        r.steps = r.groups = r.n = r.L = r.row0 = r.tile0 = 0;
        if (lane < P.B && !request_of(P, lane, r) && worker == 0) atomicOr(P.status, GEM_DEVFLAG_POS_RANGE);
        const int64_t v = static_cast<int64_t>(r.steps) * r.groups * P.n_kv;
        int64_t upto = v;
        for (int o = 1; o < P.B; o <<= 1) {
            const int64_t x = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += x;
        }
        total = __shfl_sync(0xffffffffu, upto, P.B - 1);
        const int64_t from = worker * split();
        b0 = min(P.B - 1, __popc(__ballot_sync(0xffffffffu, lane < P.B && upto <= from)));
        in_b0 = from - __shfl_sync(0xffffffffu, upto - v, b0);
        r0.row0 = __shfl_sync(0xffffffffu, r.row0, b0), r0.n = __shfl_sync(0xffffffffu, r.n, b0);
        r0.L = __shfl_sync(0xffffffffu, r.L, b0), r0.tile0 = __shfl_sync(0xffffffffu, r.tile0, b0);
        r0.steps = __shfl_sync(0xffffffffu, r.steps, b0), r0.groups = __shfl_sync(0xffffffffu, r.groups, b0);
    } else {
        int64_t carry = 0;     // steps before each request, in shared memory
        if (threadIdx.x == 0) plan[0] = 0;
        for (int base = 0; base < P.B; base += kThreads) {
            const int b = base + threadIdx.x;
            Request r;
            int64_t v = 0;
            if (b < P.B) {
                if (!request_of(P, b, r) && blockIdx.x == 0) atomicOr(P.status, GEM_DEVFLAG_POS_RANGE);
                v = static_cast<int64_t>(r.steps) * r.groups * P.n_kv;
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t x = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += x;
            }
            if (lane == 31) sums[warp] = v;
            __syncthreads();
            int64_t before = 0, all = 0;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                before += i < warp ? sums[i] : 0;
                all += sums[i];
            }
            if (b < P.B) plan[b + 1] = carry + before + v;
            carry += all;
            __syncthreads();
        }
        total = plan[P.B];
        const int64_t from = worker * split();
        int hi = P.B - 1;      // the last request that begins at or before the share
        while (b0 < hi) {
            const int mid = (b0 + hi + 1) >> 1;
            if (plan[mid] <= from) b0 = mid;
            else hi = mid - 1;
        }
        in_b0 = from - plan[b0];
        request_of(P, b0, r0);
    }
    const int64_t share = split();
    const int64_t begin = min(total, worker * share), end = min(total, begin + share);

    // the step to request next: unit, steps left of it, first tile, and the tiles that its rows attend
    int put_b = 0, put_u = 0, put_left = 0, put_tile = 0, put_lo = 0, put_hi = 0, put_h = 0, put_last_page = 0, put_units = 1;
    int64_t put_step = begin;
    int pbase = 0, pid = -1;   // table entries pbase .. pbase + 31 of the request, one a lane
    uint32_t lost = 0;         // tiles of the ring's stages that hold nothing
    bool dead = false;
    const uint32_t short_by = worker == 0 && (test_inject() & GEM_INJECT_RING_SHORTFALL) ? 16 : 0;
    const int lpt = P.lpage - 4;
    constexpr uint32_t kMask = (1u << kStepTiles) - 1;

    auto put_unit = [&](const Unit& un, int i) {   // go on at step i of a unit
        put_left = un.steps - i;
        put_units = un.units;
        put_tile = un.tile0 + i * kStepTiles;
        put_lo = un.lo_all / kTileTokens, put_hi = un.hi_all / kTileTokens;
        put_h = un.h;
        put_last_page = (un.L - 1) >> P.lpage;
        pbase = -64;
    };
    auto request_step = [&](int stage) {
        const int tile = put_tile + lane;
        const bool want = lane < kStepTiles && tile >= put_lo && tile <= put_hi;
        const int first = put_tile >> lpt;
        if (first - pbase + kStepTiles - 1 > 31) {   // a step's tiles lie in at most as many pages
            pbase = first;
            const int64_t at = pbase + lane;
            pid = at < P.max_pages && at <= put_last_page ? P.table[put_b * P.max_pages + at] : -1;
        }
        const int32_t id = __shfl_sync(0xffffffffu, pid, ((tile >> lpt) - pbase) & 31);
        const bool in = want && id >= 0 && id < P.n_pages;
        const uint32_t have = __ballot_sync(0xffffffffu, in);
        lost = (lost & ~(kMask << (stage * kStepTiles))) | ((~have & kMask) << (stage * kStepTiles));
        if (lane == 0) {
            uint32_t bytes = __popc(have) * C::kTile;
            if (put_step == 0) bytes += short_by;
            mbar_arrive_expect_tx(&bars[stage], bytes);
        }
        __syncwarp();
        if (in) {
            const uint8_t* src = P.pool + (((static_cast<int64_t>(id) * P.n_kv + put_h) << lpt) +
                                           (tile & ((1 << lpt) - 1))) * tile_bytes(D);
            const uint32_t dst = smem_u32(ring + stage * C::kStage + lane * C::kTile);
            if (PAIR == 1) {
                bulk_load(dst, src, C::kTile, &bars[stage]);
            } else {
                constexpr int kCodes = 8 * C::kDims, kScale = C::kDims;
                bulk_load(dst, src + member * kCodes, kCodes, &bars[stage]);
                bulk_load(dst + kCodes, src + codes_off(D, 1) + member * kCodes, kCodes, &bars[stage]);
                bulk_load(dst + 2 * kCodes, src + scales_off(D, 0) + member * kScale, kScale, &bars[stage]);
                bulk_load(dst + 2 * kCodes + kScale, src + scales_off(D, 1) + member * kScale, kScale, &bars[stage]);
            }
        } else if (want) {
            atomicOr(P.status, GEM_DEVFLAG_PAGE_RANGE);
        }
        put_tile += kStepTiles;
        if (++put_step < end && --put_left == 0) put_unit(next_unit(P, put_units, put_b, put_u), 0);
    };

    // the warps of a worker; each step has one
    auto member_sync = [&]() {
        if (PAIR > 1) asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / PAIR), "n"(32 * PAIR) : "memory");
    };

    const float to_log2 = P.scale * 1.4426950408889634f;

    // whether a wait of one of this worker's warps has run out (each sets its word before a step's barrier): then
    // its units are not written
    auto failed = [&]() {
        bool any = dead;
        if (PAIR > 1)
#pragma unroll
            for (int of = 0; of < PAIR; ++of) any |= gave_up[warp - member + of] != 0;
        return PAIR > 1 ? __any_sync(0xffffffffu, any) != 0 : any;
    };

    // state of the unit at hand
    uint32_t bq[NB][2][NT][NH][2];        // q: [block][low or high byte pair][column tile][hi, lo][register]
    float acc[NB][2][NT][4];              // output sums
    float m[NT][2], l[NT][2];
    int prow[NT][2];                      // positions of this lane's two rows of each column tile

    // rows of the S and output fragments: columns 2t, 2t + 1
    auto col_row = [&](int nt, int e) { return PACK ? (2 * t + e) & 3 : nt * 8 + 2 * t + e; };

    // q's values that go into this lane's operands: issued apart from their use
    float4 qv[NT][NB][2];
    auto load_q = [&](const Unit& un) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int row = PACK ? g & 3 : nt * 8 + g;
            const int tok = (row * P.inv_g) >> 16;
            const bool live = tok < un.tokens;
            const float* src = P.q + (un.row0 + static_cast<int64_t>(tok)) * P.ldq +
                               (static_cast<int64_t>(un.h) * P.G + (row - tok * P.G)) * D + member * C::kDims + 4 * t;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    qv[nt][b][k] = live ? *reinterpret_cast<const float4*>(src + b * 32 + 16 * k) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    auto begin_unit = [&](const Unit& un) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                const float4 lo4 = qv[nt][b][0], hi4 = qv[nt][b][1];
                const float x[8] = {lo4.x, lo4.y, lo4.z, lo4.w, hi4.x, hi4.y, hi4.z, hi4.w};
                float top = 0.f;
#pragma unroll
                for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(x[k]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const Scale2 f = scale_to_2_14(top);   // a power of two for each row's block
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const float v0 = x[4 * k + j] * f.up, v1 = x[4 * k + j + 2] * f.up;
                        const uint32_t hi = pack_rn(v0, v1);
                        const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                        const uint32_t lo = pack_rn(v0 - h.x, v1 - h.y);
                        bq[b][j][nt][0][k] = !PACK || g < 4 ? hi : lo;
                        if (!PACK) bq[b][j][nt][NH - 1][k] = lo;
                    }
                if (t == 0) probs[(b * NT + nt) * kProbRow + kStepTokens + g] = f.down;
            }
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int tk = (col_row(nt, k) * P.inv_g) >> 16;
                prow[nt][k] = un.p0 + min(tk, un.tokens - 1);
                m[nt][k] = -INFINITY;
                l[nt][k] = 0.f;
            }
        }
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[b][0][nt][k] = acc[b][1][nt][k] = 0.f;
    };

    // The unit's sums so far: put_row(row, maximum, sum of p) for every row, and
    // put_pair(row, dim, values of dim and dim + 1, sum of p) for its dims.
    auto finish = [&](auto&& put_pair, auto&& put_row) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], o);
                if (PACK) l[nt][k] += __shfl_xor_sync(0xffffffffu, l[nt][k], 2);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
                if (g == 0 && (!PACK || t < 2)) put_row(col_row(nt, k), m[nt][k], l[nt][k]);
#pragma unroll
            for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float v[4];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float a0 = acc[b][j][nt][k], a1 = acc[b][j][nt][2 + k];
                        if (PACK) {
                            a0 += __shfl_xor_sync(0xffffffffu, a0, 2);
                            a1 += __shfl_xor_sync(0xffffffffu, a1, 2);
                        }
                        v[j] = a0;
                        v[2 + j] = a1;
                    }
                    if (!PACK || t < 2) {
                        const int dim = member * C::kDims + b * 32 + 2 * g;
                        put_pair(col_row(nt, k), dim, make_float2(v[0], v[1]), l[nt][k]);
                        put_pair(col_row(nt, k), dim + 16, make_float2(v[2], v[3]), l[nt][k]);
                    }
                }
            }
        }
    };

    // ---- one step: kStepTiles tiles in stage `stage` ----
    // (clean: every row of the unit attends every position of it)
    auto compute = [&](int stage, auto clean_c, int pos0, int lo_all, int hi_all) {
        constexpr bool clean = decltype(clean_c)::value;
        const uint8_t* st = ring + stage * C::kStage;
        const uint32_t gone = (lost >> (stage * kStepTiles)) & kMask;
        // scales in fp32: K's as (row g, row g, row g + 8, row g + 8), V's as (2t, 2t + 1, 2t + 8, 2t + 9); a lane
        // takes positions 2r, 2r + 1, 2r + 8 and 2r + 9 of a block of both
        const __half2 zero2 = __float2half2_rn(0.f);
#pragma unroll
        for (int it = 0; it < kStepTiles * NB * 4; it += 32) {
            const int at = it + lane, sb = at >> 2, r = at & 3, s = sb / NB, b = sb % NB;
            if (kStepTiles * NB * 4 % 32 == 0 || sb < kStepTiles * NB) {
                const __half2* ks = reinterpret_cast<const __half2*>(st + s * C::kTile + scales_off(C::kDims, 0)) + b * 8 + r;
                const __half2* vs = ks + C::kDims / 4;
                // an infinite scale of K becomes NaN (x + 0 x): times a negative sum it would hide its position
                const float2 k0 = __half22float2(__hfma2(ks[0], zero2, ks[0])), k1 = __half22float2(__hfma2(ks[4], zero2, ks[4]));
                float4* to = reinterpret_cast<float4*>(scales + sb * 48);
                to[2 * r] = make_float4(k0.x, k0.x, k1.x, k1.x);
                to[2 * r + 1] = make_float4(k0.y, k0.y, k1.y, k1.y);
                __half2 v0 = vs[0], v1 = vs[4];
                if (!clean) {   // what no row attends may be anything
                    const int pos = pos0 + s * kTileTokens + 2 * r;
                    auto in = [&](int p) { return p >= lo_all && p <= hi_all && !(gone >> s & 1); };
                    const __half zero = __float2half_rn(0.f);
                    v0 = __halves2half2(in(pos) ? __low2half(v0) : zero, in(pos + 1) ? __high2half(v0) : zero);
                    v1 = __halves2half2(in(pos + 8) ? __low2half(v1) : zero, in(pos + 9) ? __high2half(v1) : zero);
                }
                const float2 f0 = __half22float2(v0), f1 = __half22float2(v1);
                to[8 + r] = make_float4(f0.x, f0.y, f1.x, f1.y);
            }
        }
        __syncwarp();

        // scores
        uint32_t kw[kStepTiles][NB / 2][4];
#pragma unroll
        for (int s = 0; s < kStepTiles; ++s)
#pragma unroll
            for (int b2 = 0; b2 < NB; b2 += 2)
                ldmatrix_x4(kw[s][b2 / 2][0], kw[s][b2 / 2][1], kw[s][b2 / 2][2], kw[s][b2 / 2][3],
                            smem_u32(st + s * C::kTile) + lane * 16 + b2 * 256);
        float sc[kStepTiles][NT][4];
#pragma unroll
        for (int s = 0; s < kStepTiles; ++s) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int k = 0; k < 4; ++k) sc[s][nt][k] = 0.f;
#pragma unroll
            for (int b2 = 0; b2 < NB; b2 += 2) {
                const uint32_t (&w)[4] = kw[s][b2 / 2];
#pragma unroll
                for (int b = b2; b < b2 + 2; ++b) {
                    const uint32_t wa = w[2 * (b - b2)], wb = w[2 * (b - b2) + 1];
                    const float4 ks = reinterpret_cast<const float4*>(scales + (s * NB + b) * 48)[g];
                    const Codes ca = codes_of(wa), cb = codes_of(wb);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float d[4];
                        mma_first(d, ca.v[0], cb.v[0], ca.v[1], cb.v[1], bq[b][0][nt][0][0], bq[b][0][nt][0][1]);
                        mma_16816(d, ca.v[2], cb.v[2], ca.v[3], cb.v[3], bq[b][1][nt][0][0], bq[b][1][nt][0][1]);
                        if (!PACK) {
                            mma_16816(d, ca.v[0], cb.v[0], ca.v[1], cb.v[1], bq[b][0][nt][NH - 1][0], bq[b][0][nt][NH - 1][1]);
                            mma_16816(d, ca.v[2], cb.v[2], ca.v[3], cb.v[3], bq[b][1][nt][NH - 1][0], bq[b][1][nt][NH - 1][1]);
                        }
                        float2* to = reinterpret_cast<float2*>(sc[s][nt]);
                        const float2 down = *reinterpret_cast<const float2*>(probs + (b * NT + nt) * kProbRow + kStepTokens + 2 * t);
                        to[0] = ffma2(fmul2(make_float2(ks.x, ks.y), make_float2(d[0], d[1])), down, to[0]);
                        to[1] = ffma2(fmul2(make_float2(ks.z, ks.w), make_float2(d[2], d[3])), down, to[1]);
                    }
                }
            }
        }
        if (PAIR > 1) {   // the head's other dims are the other members'; the buffers alternate with the stage,
                          // and a member that writes one again has passed the barrier after its last reading
            constexpr int kBuf = kStepTiles * NT * 32;
            auto buffer = [&](int of) {
                return reinterpret_cast<float4*>(smem + (warp - member + of) * C::kWarpBytes + C::kRing + C::kScales + C::kProbs) +
                       stage * kBuf;
            };
#pragma unroll
            for (int s = 0; s < kStepTiles; ++s)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    buffer(member)[(s * NT + nt) * 32 + lane] = make_float4(sc[s][nt][0], sc[s][nt][1], sc[s][nt][2], sc[s][nt][3]);
            member_sync();
#pragma unroll
            for (int s = 0; s < kStepTiles; ++s)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    // in the members' order, so that all of them get the same sums
                    float4 v = buffer(0)[(s * NT + nt) * 32 + lane];
#pragma unroll
                    for (int of = 1; of < PAIR; ++of) {
                        const float4 o = buffer(of)[(s * NT + nt) * 32 + lane];
                        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
                    }
                    sc[s][nt][0] = v.x, sc[s][nt][1] = v.y, sc[s][nt][2] = v.z, sc[s][nt][3] = v.w;
                }
        }

        // p: in log2 units; PACK: the two halves' sums, lanes t < 2 keep row g, the others row g + 8
        constexpr int NV = PACK ? 2 : 4;
        float x[kStepTiles][NT][NV];
        uint32_t masked = 0;
        bool up = false;
#pragma unroll
        for (int s = 0; s < kStepTiles; ++s)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (PACK) {
                    const float g0 = t < 2 ? sc[s][nt][2] : sc[s][nt][0], g1 = t < 2 ? sc[s][nt][3] : sc[s][nt][1];
                    const float k0 = t < 2 ? sc[s][nt][0] : sc[s][nt][2], k1 = t < 2 ? sc[s][nt][1] : sc[s][nt][3];
                    x[s][nt][0] = (k0 + __shfl_xor_sync(0xffffffffu, g0, 2)) * to_log2;
                    x[s][nt][1] = (k1 + __shfl_xor_sync(0xffffffffu, g1, 2)) * to_log2;
                } else {
#pragma unroll
                    for (int k = 0; k < NV; ++k) x[s][nt][k] = sc[s][nt][k] * to_log2;
                }
                if (!clean) {
#pragma unroll
                    for (int k = 0; k < NV; ++k) {
                        const int pos = pos0 + s * kTileTokens + g + (PACK ? (t >> 1) : (k >> 1)) * 8;
                        const int p = prow[nt][k & 1];
                        const bool in = pos <= p && (P.window == 0 || pos > p - P.window) && !(gone >> s & 1);
                        if (!in) x[s][nt][k] = -INFINITY, masked |= 1u << ((s * NT + nt) * NV + k);
                    }
                }
#pragma unroll
                for (int k = 0; k < NV; ++k) up |= x[s][nt][k] > m[nt][k & 1] + kSlack;
            }
        // Scores well past the maxima so far: new maxima, and the sums are rescaled.  (Any maximum would make
        // it half of the steps; p may pass 1 by kSlack powers of two instead.)  The scores are the same for all
        // warps of a head, so that the maxima are too: parts are joined under one of them.
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float corr[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float mx = m[nt][k];
#pragma unroll
                    for (int s = 0; s < kStepTiles; ++s)
#pragma unroll
                        for (int v = k; v < NV; v += 2) mx = fmaxf(mx, x[s][nt][v]);
#pragma unroll
                    for (int o = PACK ? 2 : 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                    corr[k] = m[nt][k] == mx ? 1.f : ex2(m[nt][k] - mx);
                    m[nt][k] = mx;
                    l[nt][k] *= corr[k];
                }
#pragma unroll
                for (int b = 0; b < NB; ++b) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        acc[b][j][nt][0] *= corr[0], acc[b][j][nt][1] *= corr[1];
                        acc[b][j][nt][2] *= corr[0], acc[b][j][nt][3] *= corr[1];
                    }
                }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float mb[2] = {m[nt][0] == -INFINITY ? 0.f : m[nt][0], m[nt][1] == -INFINITY ? 0.f : m[nt][1]};
#pragma unroll
            for (int s = 0; s < kStepTiles; ++s)
#pragma unroll
                for (int k = 0; k < NV; ++k) {
                    float p = ex2(x[s][nt][k] - mb[k & 1]);
                    if (!clean && (masked >> ((s * NT + nt) * NV + k) & 1)) p = -0.f;   // unlike one that underflowed
                    l[nt][k & 1] += p;
                    probs[col_row(nt, k & 1) * kProbRow + s * kTileTokens + g + (PACK ? (t >> 1) : (k >> 1)) * 8] = p;
                }
        }
        __syncwarp();

        // values
        uint32_t vw[kStepTiles][NB / 2][4];
#pragma unroll
        for (int s = 0; s < kStepTiles; ++s)
#pragma unroll
            for (int b2 = 0; b2 < NB; b2 += 2)
                ldmatrix_x4_trans(vw[s][b2 / 2][0], vw[s][b2 / 2][1], vw[s][b2 / 2][2], vw[s][b2 / 2][3],
                                  smem_u32(st + s * C::kTile + codes_off(C::kDims, 1)) + lane * 16 + b2 * 256);
        const uint32_t flip = !PACK || g >= 4 ? 0x80000000u : 0u;
        const float2 keep = !PACK || g >= 4 ? make_float2(1.f, 1.f) : make_float2(0.f, 0.f);
        float2 pr[kStepTiles][NT][2];
#pragma unroll
        for (int s = 0; s < kStepTiles; ++s)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const float* row = probs + (PACK ? g & 3 : nt * 8 + g) * kProbRow + s * kTileTokens + 2 * t;
                pr[s][nt][0] = *reinterpret_cast<const float2*>(row);
                pr[s][nt][1] = *reinterpret_cast<const float2*>(row + 8);
            }
        // A block's products of the step go into fresh accumulators and from there into the sums: the tensor
        // cores cut what they accumulate off toward zero, and a sum kept there through a long sequence drifts
        // (after 450 products it was 6.5e-6 off).  So each row's block has a power of two of its own in each
        // step, that of its largest product p sV, under which hi and lo fill binary16 whatever the scales and the
        // probabilities of other blocks, rows and steps are.
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            float d[2][NT][4];
            float2 v[kStepTiles][NT][2], back[NT];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float top = 0.f;
#pragma unroll
                for (int s = 0; s < kStepTiles; ++s) {
                    const float4 vs = reinterpret_cast<const float4*>(scales + (s * NB + b) * 48 + 32)[t];
                    const float2 p0 = pr[s][nt][0], p1 = pr[s][nt][1];
                    float2 v0 = fmul2(p0, make_float2(vs.x, vs.y));
                    float2 v1 = fmul2(p1, make_float2(vs.z, vs.w));
                    if (!clean) {   // a row leaves out a position whatever V's scale is there
                        auto out = [](float p) { return __float_as_uint(p) == 0x80000000u; };
                        v0.x = out(p0.x) ? 0.f : v0.x, v0.y = out(p0.y) ? 0.f : v0.y;
                        v1.x = out(p1.x) ? 0.f : v1.x, v1.y = out(p1.y) ? 0.f : v1.y;
                    }
                    top = fmaxf(top, fmaxf(fmaxf(fabsf(v0.x), fabsf(v0.y)), fmaxf(fabsf(v1.x), fabsf(v1.y))));
                    v[s][nt][0] = v0, v[s][nt][1] = v1;
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const Scale2 f = scale_to_2_14(top);
#pragma unroll
                for (int s = 0; s < kStepTiles; ++s)
#pragma unroll
                    for (int k = 0; k < 2; ++k) v[s][nt][k] = fmul2(v[s][nt][k], make_float2(f.up, f.up));
                back[nt].x = __shfl_sync(0xffffffffu, f.down, 8 * t);
                back[nt].y = __shfl_sync(0xffffffffu, f.down, 8 * t + 4);
            }
#pragma unroll
            for (int s = 0; s < kStepTiles; ++s) {
                const uint32_t wa = vw[s][b / 2][2 * (b & 1)], wb = vw[s][b / 2][2 * (b & 1) + 1];
                const Codes ca = codes_of(wa), cb = codes_of(wb);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const float2 v0 = v[s][nt][0], v1 = v[s][nt][1];
                    // hi: the leading 11 bits; lo: what they leave.  PACK: this lane's column is one of the two
                    const float2 r0 = ffma2(v0, keep, make_float2(lead(v0.x, flip), lead(v0.y, flip)));
                    const float2 r1 = ffma2(v1, keep, make_float2(lead(v1.x, flip), lead(v1.y, flip)));
                    const uint32_t lo0 = pack_rn(r0.x, r0.y), lo1 = pack_rn(r1.x, r1.y);
                    if (s == 0) {
                        mma_first(d[0][nt], ca.v[0], ca.v[1], cb.v[0], cb.v[1], lo0, lo1);
                        mma_first(d[1][nt], ca.v[2], ca.v[3], cb.v[2], cb.v[3], lo0, lo1);
                    } else {
                        mma_16816(d[0][nt], ca.v[0], ca.v[1], cb.v[0], cb.v[1], lo0, lo1);
                        mma_16816(d[1][nt], ca.v[2], ca.v[3], cb.v[2], cb.v[3], lo0, lo1);
                    }
                    if (!PACK) {
                        const uint32_t hi0 = pack_rz(v0.x, v0.y), hi1 = pack_rz(v1.x, v1.y);
                        mma_16816(d[0][nt], ca.v[0], ca.v[1], cb.v[0], cb.v[1], hi0, hi1);
                        mma_16816(d[1][nt], ca.v[2], ca.v[3], cb.v[2], cb.v[3], hi0, hi1);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float2* to = reinterpret_cast<float2*>(acc[b][j][nt]);
                    to[0] = ffma2(make_float2(d[j][nt][0], d[j][nt][1]), back[nt], to[0]);
                    to[1] = ffma2(make_float2(d[j][nt][2], d[j][nt][3]), back[nt], to[1]);
                }
        }
        __syncwarp();
    };

    // ---- the share ----
    int64_t tail = -1;
    int4 task = make_int4(-1, 0, 0, 0);
    if (begin < end) {
        const int64_t q0 = quotient(in_b0, r0.steps);
        int b = b0, u = static_cast<int>(q0), i = static_cast<int>(in_b0 - q0 * r0.steps);
        Unit un(P, r0, u);
        load_q(un);
        put_b = b, put_u = u;
        put_unit(un, i);
        for (int k = 0; k < kStages && put_step < end; ++k) request_step(k);
        int stage = 0;
        uint32_t parity = 0;
        int64_t step = begin;
        while (true) {
            const int64_t unit_end = min(end, step + (un.steps - i));
            const bool starts = i == 0, ends = step + (un.steps - i) <= end;
            if (!ends) tail = step - i;
            begin_unit(un);
            int pos0 = (un.tile0 + i * kStepTiles) * kTileTokens;
            for (; step < unit_end; ++step, pos0 += kStepTokens) {
                if (!dead) {
                    dead = __any_sync(0xffffffffu, !mbar_wait(&bars[stage], parity, P.status));
                    if (dead && lane == 0) {   // a copy never landed: give those in flight a bounded chance to
                        gave_up[warp] = 1;
                        for (int k = 0; k < kStages; ++k)
                            (void)mbar_wait(&bars[(stage + k) % kStages], parity ^ (stage + k >= kStages ? 1u : 0u), nullptr);
                    }
                    __syncwarp();
                }
                if (!dead) {
                    if (((lost >> (stage * kStepTiles)) & kMask) == 0 && pos0 >= un.lo_max && pos0 + kStepTokens - 1 <= un.p0)
                        compute(stage, std::true_type{}, pos0, un.lo_all, un.hi_all);
                    else if (pos0 <= un.hi_all && pos0 + kStepTokens > un.lo_all)
                        compute(stage, std::false_type{}, pos0, un.lo_all, un.hi_all);
                    else
                        member_sync();
                    if (put_step < end) request_step(stage);
                } else {   // go through the steps without work
                    member_sync();
                }
                if (++stage == kStages) stage = 0, parity ^= 1;
            }
            if (ends && !failed()) {
                if (starts) {   // the whole unit
                    finish([&](int row, int dim, float2 v, float sum) {
                        const int tok = (row * P.inv_g) >> 16;
                        if (tok >= un.tokens) return;
                        float* o = P.out + (un.row0 + static_cast<int64_t>(tok)) * P.ldo +
                                   (static_cast<int64_t>(un.h) * P.G + (row - tok * P.G)) * D + dim;
                        const float inv = sum == 0.f ? 0.f : 1.f / sum;
                        o[0] = v.x * inv, o[1] = v.y * inv;
                    }, [](int, float, float) {});
                } else {
                    task = make_int4(static_cast<int>(quotient(step - un.steps, share)), un.row0, un.tokens, un.h);
                    float* slot = P.part + static_cast<int64_t>(worker) * Part<D, ROWS>::kFloats;
                    finish([&](int row, int dim, float2 v, float) { *reinterpret_cast<float2*>(slot + row * D + dim) = v; },
                           [&](int row, float mx, float sum) {
                               if (member == 0) slot[ROWS * D + 2 * row] = mx, slot[ROWS * D + 2 * row + 1] = sum;
                           });
                }
            }
            if (step == end) break;
            i = 0;
            un = next_unit(P, un.units, b, u);
            load_q(un);
        }
        if (failed()) tail = task.x = -1;
    }
    if (lane == 0 && member == 0) P.tasks[worker] = task;
    // units that go on in the next share: join the parts of this CTA's workers (the rings are empty now)
    constexpr int kLocal = C::kRing / 4;
    if (tail >= 0) {
        __syncwarp();
        float* mine = reinterpret_cast<float*>(ring);
        finish([&](int row, int dim, float2 v, float) {
                   *reinterpret_cast<float2*>(mine + row * C::kDims + (dim - member * C::kDims)) = v;
               },
               [&](int row, float mx, float sum) {
                   mine[ROWS * C::kDims + 2 * row] = mx, mine[ROWS * C::kDims + 2 * row + 1] = sum;
               });
    }
    static_assert(kStages >= 2, "the members' buffers alternate");
    static_assert(NB * NT <= ROWS, "a row of probabilities for each block and column tile");
    static_assert(ROWS * (C::kDims + 2) <= kLocal, "a partial result fits the ring");
    constexpr int kW = C::kWorkers;
    auto state_of = [&](int w) {   // a worker's (maximum, sum) rows
        return reinterpret_cast<const float2*>(smem + w * PAIR * C::kWarpBytes + ROWS * C::kDims * 4);
    };
    if (lane == 0 && member == 0) tail_unit[warp / PAIR] = tail < 0 ? -1 : static_cast<int>(tail & 0x7fffffff);
    const bool lost_one = __syncthreads_or(dead);
    auto slot_of = [&](int first) {
        return P.part + (static_cast<int64_t>(P.workers) + blockIdx.x * kW + first) * Part<D, ROWS>::kFloats;
    };
    if (lost_one) {   // parts of this CTA may be missing: a maximum that is NaN, which no sum has, marks all of its slots
        for (int at = threadIdx.x; at < kW * ROWS; at += kThreads) {
            const int64_t up = ROWS * D + 2 * (at % ROWS);
            slot_of(at / ROWS)[up] = NAN;
            slot_of(at / ROWS - P.workers)[up] = NAN;
        }
        return;
    }
    int ids[kW];
#pragma unroll
    for (int w = 0; w < kW; ++w) ids[w] = tail_unit[w];
    // each worker's weight in its unit's part, and the part's (maximum, sum)
    for (int at = threadIdx.x; at < kW * ROWS; at += kThreads) {
        const int w = at / ROWS, row = at % ROWS, id = tail_unit[w];
        if (id < 0) continue;
        float2 ml[kW];
        float top = -INFINITY, sum = 0.f;
        int first = kW;
#pragma unroll
        for (int k = kW - 1; k >= 0; --k) {
            ml[k] = ids[k] == id ? state_of(k)[row] : make_float2(-INFINITY, 0.f);
            top = fmaxf(top, ml[k].x);
            if (ids[k] == id) first = k;
        }
#pragma unroll
        for (int k = 0; k < kW; ++k) {
            const float c = ml[k].x == top ? 1.f : ex2(ml[k].x - top);
            sum = fmaf(c, ml[k].y, sum);
            if (k == w) weight[w * ROWS + row] = c;
        }
        if (w == first) *reinterpret_cast<float2*>(slot_of(first) + ROWS * D + 2 * row) = make_float2(top, sum);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < ROWS * D / 2; i += kThreads) {
        const int row = i / (D / 2), dim = i % (D / 2) * 2;
        float2 o[kW], v = make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < kW; ++w)
            if (ids[w] >= 0)
                o[w] = *reinterpret_cast<const float2*>(smem + (w * PAIR + dim / C::kDims) * C::kWarpBytes +
                                                        (row * C::kDims + dim % C::kDims) * 4);
        int first = 0;
#pragma unroll
        for (int w = 0; w < kW; ++w) {
            if (ids[w] < 0) continue;
            if (w == 0 || ids[w] != ids[w - 1]) first = w, v = make_float2(0.f, 0.f);
            const float c = weight[w * ROWS + row];
            v.x = fmaf(c, o[w].x, v.x), v.y = fmaf(c, o[w].y, v.y);
            if (w == kW - 1 || ids[w] != ids[w + 1 < kW ? w + 1 : w])
                *reinterpret_cast<float2*>(slot_of(first) + row * D + dim) = v;
        }
    }
}

// Joins the parts of units that cross shares: one CTA for each row of a unit and the workers of one CTA
// of the first kernel.  A worker whose share holds the end of a unit that began earlier left a task:
// the first worker of the unit, its first query row, its tokens, its KV head.  The parts lie in order:
// one for each CTA whose workers the unit goes on from, then the last worker's own.  D / 4 threads hold
// four dims each; the groups of so many threads take every kSlices-th part and are joined in order.
// Latency: tasks, then parts, from L2; some 2 us behind the first kernel.
constexpr int kMergeThreads = 256;
template <int D, int ROWS, int CW>
__global__ void __launch_bounds__(kMergeThreads) kv4_attn_merge_kernel(const AttnParams P) {
    constexpr int kCols = D / 4, kSlices = kMergeThreads / kCols, kAhead = 4;
    __shared__ float4 v_s[kSlices][kCols];
    __shared__ float2 ml_s[kSlices];
    const int row = blockIdx.y, tok = (row * P.inv_g) >> 16;
    constexpr int64_t kFloats = Part<D, ROWS>::kFloats;
    const int col = threadIdx.x % kCols, slice = threadIdx.x / kCols;
    const int lane = threadIdx.x & 31;
    int4 mine = make_int4(-1, 0, 0, 0);
    pdl_wait_trigger();
    if (lane < CW) mine = P.tasks[blockIdx.x * CW + lane];
    for (uint32_t todo = __ballot_sync(0xffffffffu, mine.x >= 0 && tok < mine.z); todo; todo &= todo - 1) {
        const int from = __ffs(todo) - 1, w1 = blockIdx.x * CW + from;
        int4 task;
        task.x = __shfl_sync(0xffffffffu, mine.x, from), task.y = __shfl_sync(0xffffffffu, mine.y, from);
        task.w = __shfl_sync(0xffffffffu, mine.w, from);
        const int w0 = task.x, c0 = w0 / CW, c1 = (w1 - 1) / CW, parts = c1 - c0 + 2;
        float mx = -INFINITY, sum = 0.f;
        bool whole = true;     // no part is marked as missing
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k0 = slice; k0 < parts; k0 += kSlices * kAhead) {
            float2 ml[kAhead], ol[kAhead], oh[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const int k = k0 + a * kSlices, c = c0 + k;
                ml[a] = make_float2(-INFINITY, 0.f), ol[a] = oh[a] = make_float2(0.f, 0.f);
                if (k < parts) {
                    const float* s = P.part + (c > c1 ? w1 : P.workers + max(w0, c * CW)) * kFloats;
                    ml[a] = *reinterpret_cast<const float2*>(s + ROWS * D + 2 * row);
                    ol[a] = *reinterpret_cast<const float2*>(s + row * D + 4 * col);
                    oh[a] = *reinterpret_cast<const float2*>(s + row * D + 4 * col + 2);
                }
            }
            float top = mx;
#pragma unroll
            for (int a = 0; a < kAhead; ++a) top = fmaxf(top, ml[a].x), whole &= ml[a].x == ml[a].x;
            const float c = mx == top ? 1.f : ex2(mx - top);
            mx = top;
            sum *= c, v.x *= c, v.y *= c, v.z *= c, v.w *= c;
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                const float f = ml[a].x == mx ? 1.f : ex2(ml[a].x - mx);
                sum = fmaf(f, ml[a].y, sum);
                v.x = fmaf(f, ol[a].x, v.x), v.y = fmaf(f, ol[a].y, v.y);
                v.z = fmaf(f, oh[a].x, v.z), v.w = fmaf(f, oh[a].y, v.w);
            }
        }
        v_s[slice][col] = v;
        if (col == 0) ml_s[slice] = make_float2(whole ? mx : NAN, sum);
        __syncthreads();
        if (slice == 0) {
            mx = ml_s[0].x, whole = mx == mx;
            for (int k = 1; k < kSlices; ++k) mx = fmaxf(mx, ml_s[k].x), whole &= ml_s[k].x == ml_s[k].x;
            sum = 0.f, v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int k = 0; k < kSlices; ++k) {
                const float f = ml_s[k].x == mx ? 1.f : ex2(ml_s[k].x - mx);
                sum = fmaf(f, ml_s[k].y, sum);
                const float4 o = v_s[k][col];
                v.x = fmaf(f, o.x, v.x), v.y = fmaf(f, o.y, v.y), v.z = fmaf(f, o.z, v.z), v.w = fmaf(f, o.w, v.w);
            }
            float* o = P.out + (task.y + static_cast<int64_t>(tok)) * P.ldo +
                       (static_cast<int64_t>(task.w) * P.G + (row - tok * P.G)) * D + 4 * col;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            if (whole) o[0] = v.x * inv, o[1] = v.y * inv, o[2] = v.z * inv, o[3] = v.w * inv;
        }
        __syncthreads();
    }
}

// ---- host ------------------------------------------------------------------------------------------

struct Variant {
    const void *kernel, *merge;
    int rows, threads, ctas, cta_workers, part_floats;
    size_t (*smem)(int);
};

template <int D, int NT, bool PACK, int DW, int WARPS, int CTAS>
Variant variant() {
    using C = Cfg<D, NT, PACK, DW, WARPS>;
    return {reinterpret_cast<const void*>(kv4_attn_kernel<D, NT, PACK, DW, WARPS, CTAS>),
            reinterpret_cast<const void*>(kv4_attn_merge_kernel<D, C::kRows, C::kWorkers>), C::kRows, C::kThreads, CTAS, C::kWorkers,
            Part<D, C::kRows>::kFloats, C::smem};
}

// Query rows a unit has: one token's heads, or as many tokens as the batch has rows for on average while
// the sums of a warp stay in registers.  (Any batch is right with any of them: a request's tokens are cut
// into units.)  The host knows the rows of q, not the tokens that are there: a decoding step with rows to spare
// is run like one with more tokens, and the largest request of a mixed batch does not count alone.  8 x 32,768
// positions, four heads to a KV head: 75 us with 8 rows, 149 with 170; 8 x 2049: 13.4 and 21.9; at d 256, 16 k: 168 and
// 172.  Measured when these were compared: 8 rows of d 128 take 8 warps of 255 registers (4 x 32 new tokens: 62 us
// with 16 rows, 73 now; 12 warps spill, 104; 32 rows in warps of 64 dims, 77); so do 8 rows at d 256 and 512, with
// 256 dims a warp (1 x 32,769, d 512: 36 us then, 42 now; 128 dims a warp: 37 with 12 warps, 52 with 16).  Up to four
// rows take 128 dims a warp.
Variant pick(int64_t T, int B, int G, int d) {
    const int64_t tokens = std::max<int64_t>(1, (T + B - 1) / std::max(B, 1));
    const int64_t want = tokens * G;
    switch (d) {
        case 64:
            return want <= 4   ? variant<64, 1, true, 64, 12, 1>()
                   : want <= 8 ? variant<64, 1, false, 64, 12, 1>()
                               : variant<64, 2, false, 64, 8, 1>();
        case 128:
            return want <= 4   ? variant<128, 1, true, 128, 12, 1>()
                   : want <= 8 ? variant<128, 1, false, 128, 8, 1>()
                               : variant<128, 2, false, 128, 8, 1>();
        case 256: return want <= 4 ? variant<256, 1, true, 128, 12, 1>() : variant<256, 1, false, 256, 8, 1>();
        default: return want <= 4 ? variant<512, 1, true, 128, 12, 1>() : variant<512, 1, false, 256, 8, 1>();
    }
}

// Once for each kernel and device: the dynamic shared memory of the largest batch.
gem_status allow_smem(const void* kernel, const DeviceInfo& di, size_t bytes) {
    struct Done {
        int device;
        const void* kernel;
    };
    static std::mutex mu;
    static Done done[256];     // (beyond these it is set at every call)
    static int n = 0;
    std::lock_guard<std::mutex> lk(mu);
    for (int i = 0; i < n; ++i)
        if (done[i].device == di.device && done[i].kernel == kernel) return GEM_OK;
    GEM_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(std::min(bytes, di.smem_optin))));
    if (n < 256) done[n++] = {di.device, kernel};
    return GEM_OK;
}

size_t task_bytes(int workers) { return align_up(workers * sizeof(int4), 256); }

}  // namespace
}  // namespace kv4
}  // namespace gem

extern "C" {

size_t gem_kv4_attn_workspace(int64_t T, int B, int n_q, int n_kv, int d) {
    using namespace gem;
    using namespace gem::kv4;
    if (T <= 0 || B <= 0 || B > kMaxRequests || n_q <= 0 || n_kv <= 0 || n_q % n_kv || n_q / n_kv > kMaxGroup ||
        !head_dim_ok(d))
        return 0;
    DeviceInfo di;
    if (device_info(&di) != GEM_OK) return 0;
    const Variant v = pick(T, B, n_q / n_kv, d);
    const int workers = di.num_sms * v.ctas * v.cta_workers;
    return task_bytes(workers) + align_up(2ull * workers * v.part_floats * sizeof(float), 256);
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
    if (B > kMaxRequests || T > INT32_MAX / std::max(n_kv, 1) || max_pages > (INT32_MAX - 255) / page ||
        (n_kv && n_q / n_kv > kMaxGroup))
        return GEM_ERR_UNSUPPORTED_SHAPE;
    if (T == 0 || B == 0 || n_q == 0) return GEM_OK;
    if (!q || !out || q == out || !cu_tokens || !kv_len || (max_pages && !table)) return GEM_ERR_INVALID_ARG;
    if (ldq < static_cast<int64_t>(n_q) * d || ldo < static_cast<int64_t>(n_q) * d) return GEM_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) & 15) || ldq % 4 || (reinterpret_cast<uintptr_t>(workspace) & 255))
        return GEM_ERR_MISALIGNED;
    DeviceInfo di;
    if ((st = device_info(&di)) != GEM_OK) return st;
    const Variant v = pick(T, B, n_q / n_kv, d);
    if (!workspace || ws_bytes < gem_kv4_attn_workspace(T, B, n_q, n_kv, d)) return GEM_ERR_WORKSPACE;
    AttnParams P{};
    P.q = q, P.ldq = ldq, P.T = T, P.cu = cu_tokens, P.kv_len = kv_len;
    P.B = B, P.n_q = n_q, P.n_kv = n_kv, P.G = n_q / n_kv, P.GT = v.rows / P.G, P.inv_g = (65536 + P.G - 1) / P.G;
    P.table = table, P.max_pages = max_pages, P.pool = static_cast<const uint8_t*>(pool), P.n_pages = n_pages;
    P.lpage = log2_of(page), P.window = window, P.scale = scale;
    P.out = out, P.ldo = ldo, P.status = status ? status : di.status_word;
    const int ctas = di.num_sms * v.ctas;
    P.workers = ctas * v.cta_workers;
    P.tasks = static_cast<int4*>(workspace);
    P.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + task_bytes(P.workers));
    const size_t smem = v.smem(B);
    if (smem > di.smem_optin) return GEM_ERR_UNSUPPORTED_SHAPE;
    if ((st = allow_smem(v.kernel, di, v.smem(kMaxRequests))) != GEM_OK) return st;
    void* args[] = {&P};
    if ((st = launch_pdl(v.kernel, dim3(ctas), dim3(v.threads), smem, static_cast<cudaStream_t>(stream), args)) != GEM_OK)
        return st;
    return launch_pdl(v.merge, dim3(static_cast<unsigned>(ctas), static_cast<unsigned>(v.rows)),
                      dim3(kMergeThreads), 0, static_cast<cudaStream_t>(stream), args);
}

}  // extern "C"
