// gem_fp8_gemm.cu — product of rows in 8-bit floating point with weights scaled by blocks of 128 x 128
// (gem_fp8_gemm), on tcgen05.
//
// y[m][n] = sum_b xs[m][b] ws[n / 128][b] d_b[m][n],  d_b = the product over the 128 values of block b.
// The tensor cores sum d_b in tensor memory (four instructions of 32 values, the first of which overwrites);
// other warps read it back, scale it and add it to sums in registers while the next block's product runs in
// another part of tensor memory.  So the scales may have any values and the long sums are plain fp32.
//
// fp8_rows_kernel (up to 128 rows of x): the weights are what the call reads, and the rows of W take the 128-row side
// of the product, the rows of x its 16..128 columns.  The tensor cores read W straight from shared memory, so nothing
// is unpacked, and a tile may have any multiple of 8 rows of W (the rest of the 128 is whatever lies there, and not
// used): height and CTAs a tile are chosen so that the busiest SM is done first.  8 x 5376 x 21504: 19.7 us, 5.9 TB/s
// of W, 87 % of the copy rate; 61 x 21504 x 5376: 23.4 us, of which 17 stream (three CTAs on 120 rows of W; loads,
// products and scales keep shared memory as busy as the copy keeps HBM); 1 x 2048 x 4096: 4.6 us.
//
// fp8_tile_kernel (more rows): pairs of CTAs, 256 rows of x by up to 256 of W.  4096 x 5376 x 21504: 393 us in a burst
// (2.41 PFLOP/s, tensor cores 52 % active), 416 to 422 in a long run under the power cap.  Without the adds it takes 321 us,
// without the products 340 to 354, without
// both 234: reading back and adding 128 x 256 sums for each 128 of K takes as long as their product, and two buffers of
// tensor memory do not hide all of one behind the other.  Tried and not kept: halves of 128 columns with four buffers
// (420 us: x is read twice from shared memory); 160 columns with three (407, bound by the L2); W on the 256-row side and
// 320 columns of x in three buffers (686, and 30 us against 27 for 300 rows of x: smaller buffers wait longer for one
// another); the next read-back on its way while one is added (no change); 16 adding warps (403); the scales made by
// warps of their own (445, registers spill); reads of 32 or 64 columns in one (450 to 530, likewise).
#include "gem_tcgen05.cuh"

#include <array>
#include <map>
#include <mutex>
#include <utility>

namespace gem {
namespace {

struct GemmParams {
    const float* ws;
    const float* xs;
    int64_t ldxs;
    const float* res;
    float* y;
    int64_t ldy;
    int N, M, kb;
    int rows, tiles;        // rows of W a tile, tiles
    int split;              // CTAs of a cluster that share a tile's blocks
    int stages;             // of the ring
    int whole;              // K is a multiple of 128: one copy brings a step's blocks
    int chunk;              // blocks whose x scales are held at a time
    int* status;
};

// ---- few rows of x -----------------------------------------------------------------------------
// The last two warps load and issue the products; the others scale and add.  Of these, four times kWarps<NT>,
// warp w has the rows of W of lane quarter w % 4 and columns w / 4 * NT / kWarps<NT> and on.
constexpr int kMaxStages = 24;
constexpr int kMaxSplit = 8;
constexpr int kScaleBytes = 24 << 10;

// Blocks a ring stage and a tensor-memory buffer hold, of kBuffers such buffers (kGroup * NT columns each, 512
// together at most): the waits and the read-back latency of a step are paid once for kGroup blocks.
template <int NT>
constexpr int kGroup = NT <= 64 ? 4 : 2;
template <int NT>
constexpr int kBuffers = NT >= 64 ? 2 : 4;
template <int NT>
constexpr int kColumns = kBuffers<NT> * kGroup<NT> * NT;
// A cluster's CTAs hold their columns until all of them are done, and an allocation waits for as long as it has to: were
// two clusters on the same SMs, each with the columns that the other's second CTA wants, both would wait for ever (two
// streams are enough).  So the CTAs of a cluster take at least so much shared memory, used or not, that those which fit
// an SM fit in tensor memory too: two of up to 16 rows of x (256 columns), or a wider one alone.  Other launches hold
// columns only while they work.
constexpr int kSmSmem = 228 << 10;
template <int NT>
constexpr int kClusterSmem = NT <= 16 ? 2 * kGroup<NT> * (64 + NT) * 128 : 149 << 10;
static_assert(2 * kColumns<16> <= 512 && 3 * kClusterSmem<16> > kSmSmem && kClusterSmem<16> + kClusterSmem<32> > kSmSmem);
template <int NT>
constexpr int kWarps = NT <= 32 ? 2 : 4;
template <int NT>
constexpr int kPitch = NT + 4;   // of the x scales of a block: spreads a column's stores over the banks

struct RowsBarriers {
    uint64_t full[kMaxStages], empty[kMaxStages], dfull[4], dempty[4];
    uint32_t tmem;
    int dead;
};

template <int NT>
__global__ void __launch_bounds__(kWarps<NT> * 128 + 64) fp8_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const GemmParams p) {
    constexpr int NB = kBuffers<NT>, J = kGroup<NT>, COLS = kColumns<NT>, Q = kWarps<NT>, CW = NT / Q, XP = kPitch<NT>;
    extern __shared__ uint8_t raw[];
    __shared__ RowsBarriers bar;
    // the ring, 1024-byte aligned: a stage's blocks of W, then those of x; behind it the x scales
    uint8_t* ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    const int wbytes = p.rows * 128, stage_bytes = J * (wbytes + NT * 128);
    // a product reads 128 rows of W, of which p.rows are its own: the ring is followed by what that may be past its end
    float* xs_sh = reinterpret_cast<float*>(ring + p.stages * stage_bytes + max(0, 16384 - wbytes - J * NT * 128));
    float* part = reinterpret_cast<float*>(ring);   // [row of x][128], when all products are done
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = static_cast<int>(blockIdx.x) % p.split, first = static_cast<int>(blockIdx.x) / p.split, step = static_cast<int>(gridDim.x) / p.split;
    const int groups = (p.kb + J - 1) / J;
    const int b0 = groups * rank / p.split * J, b1 = min(p.kb, groups * (rank + 1) / p.split * J);   // this CTA's blocks
    volatile int* dead = &bar.dead;

    if (tid == 0) {
        bar.dead = 0;
        for (int i = 0; i < p.stages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&bar.dfull[i], 1);
            mbar_init(&bar.dempty[i], Q * ((p.rows + 31) / 32));   // the warps whose rows the tile has
        }
        fence_mbar_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
    }
    if (warp == 4 * Q + 1) tmem_alloc<1>(&bar.tmem, COLS);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    // steps of up to J blocks of a tile, in the same order in all warps
    const int ntile = first < p.tiles ? (p.tiles - first + step - 1) / step : 0;
    const int total = ntile * ((b1 - b0 + J - 1) / J);
    int issued = 0;   // by the loading warp

    if (warp == 4 * Q) {
        const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
        const uint32_t extra = blockIdx.x == 0 && (test_inject() & GEM_INJECT_RING_SHORTFALL) ? 16u : 0u;
        const uint32_t base = smem_u32(ring);
        // stage, row of W and block of the next load, counted up (a division would cost more than the load)
        int ws = 0, wb = b0, wn = first * p.rows, xs = 0, xb = b0;
        uint32_t phase = 1;
        auto load_w = [&](uint32_t more) {
            const int nj = p.whole ? J : min(J, b1 - wb);
            const uint32_t to = base + ws * stage_bytes;
            warp_expect_tx(&bar.full[ws], static_cast<uint32_t>(nj * (p.rows + NT) * 128) + more);
            if (p.whole)
                warp_tma_3d(to, &tmW, 0, wn, wb, &bar.full[ws], once);
            else
                for (int j = 0; j < nj; ++j) warp_tma_2d(to + j * wbytes, &tmW, (wb + j) * 128, wn, &bar.full[ws], once);
            if (++ws == p.stages) ws = 0, phase ^= 1;
            if ((wb += J) >= b1) wb = b0, wn += step * p.rows;
        };
        auto load_x = [&]() {
            const int nj = min(J, b1 - xb);
            const uint32_t to = base + xs * stage_bytes + J * wbytes;
            if (p.whole)
                warp_tma_3d(to, &tmX, 0, 0, xb, &bar.full[xs], keep);
            else
                for (int j = 0; j < nj; ++j) warp_tma_2d(to + j * NT * 128, &tmX, (xb + j) * 128, 0, &bar.full[xs], keep);
            if (++xs == p.stages) xs = 0;
            if ((xb += J) >= b1) xb = b0;
        };
        // the first ring's weights before the wait (no launch writes weights), its rows of x behind it
        const int ahead = min(total, p.stages);
        for (int i = 0; i < ahead; ++i) load_w(i == 0 ? extra : 0u);
        pdl_wait_trigger();
        for (int i = 0; i < ahead; ++i) load_x();
        for (issued = ahead; issued < total; ++issued) {
            if (!warp_wait(&bar.empty[ws], phase, p.status, dead)) break;
            load_w(0u);
            load_x();
        }
        if (issued < total) *dead = 1;
    } else if (warp == 4 * Q + 1) {
        constexpr uint32_t idesc = umma_idesc_e4m3(128, NT);
        const uint64_t da0 = umma_desc(smem_u32(ring)), db0 = umma_desc(smem_u32(ring) + J * wbytes);
        uint64_t da = da0, db = db0;
        int i = 0, s = 0, b = b0;
        uint32_t phase = 0;
        pdl_wait();   // the rows of x come behind it: its time is none of the bounded waits'
        for (; i < total; ++i) {
            const int d = i % NB, nj = min(J, b1 - b);
            if (i >= NB && !warp_wait(&bar.dempty[d], static_cast<uint32_t>((i / NB - 1) & 1), p.status, dead)) break;
            if (!warp_wait(&bar.full[s], phase, p.status, dead)) break;
            tc_fence_after();
#pragma unroll
            for (int j = 0; j < J; ++j)
                if (j < nj) umma_e4m3<1>(tmem + (d * J + j) * NT, da + j * (wbytes >> 4), db + j * NT * 8, idesc);
            umma_commit<1>(&bar.empty[s]);
            umma_commit<1>(&bar.dfull[d]);
            da += stage_bytes >> 4, db += stage_bytes >> 4;
            if (++s == p.stages) s = 0, phase ^= 1, da = da0, db = db0;
            if ((b += J) >= b1) b = b0;
        }
        if (i < total) {
            *dead = 1;
            // what was issued ends before the tensor memory is given back
            if (i > 0) (void)mbar_wait(&bar.dfull[(i - 1) % NB], static_cast<uint32_t>(((i - 1) / NB) & 1), nullptr);
        }
    } else {
        const int row = (warp & 3) * 32 + lane, col = (warp >> 2) * CW;
        const uint32_t from = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + col;
        pdl_wait_trigger();
        int i = 0;
        bool ok = true;
        for (int t = first; t < p.tiles; t += step) {
            const int n = t * p.rows + row;
            const bool mine = row < p.rows && n < p.N;
            const float* wrow = p.ws + static_cast<int64_t>(min(n, p.N - 1) >> 7) * p.kb;
            float2 acc[CW / 2];
#pragma unroll
            for (int m = 0; m < CW / 2; ++m) acc[m] = make_float2(0.f, 0.f);
            float w_next[J];
#pragma unroll
            for (int j = 0; j < J; ++j) w_next[j] = __ldg(wrow + min(b0 + j, p.kb - 1));
            int c = p.chunk - J;
            for (int b = b0; b < b1; b += J, ++i) {
                if ((c += J) == p.chunk) c = 0;
                if (c == 0 && (b1 - b0 > p.chunk || t == first)) {   // the next blocks' x scales, turned to [block][row]
                    const int nblk = min(p.chunk, b1 - b);
                    asm volatile("bar.sync 1, %0;" ::"n"(Q * 128) : "memory");
                    for (int m = warp; m < NT; m += 4 * Q) {   // all on their way at once
                        const float* src = p.xs + m * p.ldxs + b;
                        for (int q = lane; q < nblk; q += 32) {
                            if (m < p.M) cp_async_4(smem_u32(xs_sh + q * XP + m), src + q);
                            else xs_sh[q * XP + m] = 0.f;
                        }
                    }
                    cp_async_commit();
                    cp_async_wait<0>();
                    asm volatile("bar.sync 1, %0;" ::"n"(Q * 128) : "memory");
                }
                if ((warp & 3) * 32 >= p.rows) continue;
                float w[J];
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    w[j] = w_next[j];
                    w_next[j] = __ldg(wrow + min(b + J + j, p.kb - 1));
                }
                const int d = i % NB, nj = min(J, b1 - b);
                if (ok && !warp_wait(&bar.dfull[d], static_cast<uint32_t>((i / NB) & 1), p.status, dead)) {
                    *dead = 1;
                    ok = false;
                }
                if (!ok) continue;   // keeps to the barriers above
                tc_fence_after();
                // JB blocks at a time (what the registers hold); columns of blocks that the step lacks are read and not used
                constexpr int JB = J * CW > 32 && NT > 32 ? 32 / CW : J;
#pragma unroll
                for (int g = 0; g < J; g += JB) {
                    float v[JB][CW];
#pragma unroll
                    for (int j = 0; j < JB; ++j) tmem_ld<CW>(v[j], from + (d * J + g + j) * NT);
                    tmem_wait_ld();
                    if (g + JB == J) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&bar.dempty[d]);
                    }
#pragma unroll
                    for (int j = 0; j < JB; ++j)
                        if (g + j < nj) {
                            const float4* sx = reinterpret_cast<const float4*>(xs_sh + (c + g + j) * XP + col);
                            const float2 w2 = make_float2(w[g + j], w[g + j]);
#pragma unroll
                            for (int q = 0; q < CW / 4; ++q) {
                                const float4 x4 = sx[q];
                                acc[2 * q] = ffma2(make_float2(v[j][4 * q], v[j][4 * q + 1]), fmul2(make_float2(x4.x, x4.y), w2), acc[2 * q]);
                                acc[2 * q + 1] = ffma2(make_float2(v[j][4 * q + 2], v[j][4 * q + 3]), fmul2(make_float2(x4.z, x4.w), w2), acc[2 * q + 1]);
                            }
                        }
                }
            }
            if (p.split > 1) {   // (a warp without rows has waited for nothing: the ring may still be in use)
#pragma unroll
                for (int m = 0; m < CW; ++m)
                    if (row < p.rows && col + m < p.M) part[(col + m) * 128 + row] = m & 1 ? acc[m / 2].y : acc[m / 2].x;
            } else if (mine && ok) {
#pragma unroll
                for (int m = 0; m < CW; ++m)
                    if (col + m < p.M) {
                        const int64_t at = (col + m) * p.ldy + n;
                        const float v = m & 1 ? acc[m / 2].y : acc[m / 2].x;
                        p.y[at] = p.res ? v + p.res[at] : v;
                    }
            }
        }
    }
    __syncwarp();
    if (p.split > 1) {
        // the cluster's CTAs hold one tile's sums; each adds up a share of the rows of x, in order of k
        cluster_sync();
        if (warp < 4 * Q) {
            const int row = (warp & 3) * 32 + lane, n = first * p.rows + row;
            if (row < p.rows && n < p.N)
                for (int m0 = rank + p.split * (warp >> 2); m0 < p.M; m0 += 4 * p.split * Q) {   // four rows' reads at once
                    float v[4][kMaxSplit], add[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = min(m0 + i * p.split * Q, p.M - 1);
#pragma unroll
                        for (int r = 0; r < kMaxSplit; ++r) v[i][r] = r < p.split ? ld_peer(peer_addr(&part[m * 128 + row], r)) : 0.f;
                        add[i] = p.res ? p.res[m * p.ldy + n] : 0.f;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int m = m0 + i * p.split * Q;
                        float sum = v[i][0];
#pragma unroll
                        for (int r = 1; r < kMaxSplit; ++r) sum = r < p.split ? sum + v[i][r] : sum;
                        if (m < p.M) p.y[m * p.ldy + n] = p.res ? sum + add[i] : sum;
                    }
                }
        }
        __syncwarp();
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (*dead && warp == 4 * Q && lane == 0) drain_stages(bar.full, p.stages, max(0, issued - p.stages), issued - 1);
    if (warp == 4 * Q + 1) {
        tc_fence_after();
        tmem_free<1>(tmem, COLS);
    }
}

// ---- many rows of x ------------------------------------------------------------------------------
// Two CTAs work on one tile of 256 rows of x (128 a CTA) and BN rows of W (half of them loaded by each; the
// tensor cores of both read all of them): a product of 256 x BN halves what an SM loads for its share of the
// results, which would otherwise bound it.  Warps 0..7 scale and add (warp w: lane quarter w % 4, columns
// w / 4 * BN / 2 and on; a thread has one row of x, so a block's scale is one number), warp 8 loads, warp 9 of
// the first CTA issues the products of both; the last warpgroup gives its registers to the first two.  SPLIT: the two to
// four pairs of a cluster share the blocks of its one tile (130 x 21504 x 5376: 39 us, 56 by single pairs;
// 500 x 9728 x 2560: 23 and 28); a kernel of its own, for the other's registers are all in use.
constexpr int kTileChunk = 8;             // blocks whose x scales a warp holds at a time, twice
constexpr int kTilePitch = 33;            // of a block's 32 scales: spreads the copies over the banks
constexpr int kTileScales = 2 * kTileChunk * kTilePitch * 4;
constexpr int kTileSplit = 4;             // pairs of a cluster at most
constexpr int kTileWarps = 8;             // that scale and add
constexpr int kTileThreads = (kTileWarps + 4) * 32;
constexpr int kTileRegs = 232, kTileRegsLeft = 40;   // 256 * 232 + 128 * 40 = 384 * 168, what the block starts with

struct TileParams {
    const float* ws;
    const float* xs;
    int64_t ldxs;
    const float* res;
    float* y;
    int64_t ldy;
    int N, M, kb;
    int mtiles, tiles;
    int split;              // pairs of a cluster that share a tile's blocks
    int wide;               // y's rows (and the residual's) start on 16 bytes
    int copy;               // results leave by asynchronous copies: such rows, and no residual
    int* status;
};

struct TileBarriers {
    uint64_t full[8], empty[8], dfull[4], dempty[4], done;
    uint32_t tmem;
    int dead;
};

template <int BN>
constexpr int kTileStage = 16384 + BN * 64;
// Ring stages: what shared memory holds.  Small tiles need them, or they wait for the memory's latency (with 5 instead
// of 8 a step of 64 columns takes 0.24 us).
template <int BN>
constexpr int kTileStages = BN > 128 ? 5 : BN > 64 ? 7 : 8;
template <int BN>
constexpr int kTileSmem = 1024 + kTileStages<BN> * kTileStage<BN> + kTileWarps * (4096 + kTileScales);

static_assert(kTileSmem<256> + kClusterSmem<16> > kSmSmem && kTileSmem<64> + kClusterSmem<16> > kSmSmem);   // (as above)

template <int BN, bool SPLIT>
__global__ void __launch_bounds__(kTileThreads, 1) fp8_tile_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmY, const TileParams p) {
    constexpr int CW = BN / (kTileWarps / 4), STAGE = kTileStage<BN>, STAGES = kTileStages<BN>, NB = BN > 128 ? 2 : 4;   // buffers of BN columns of tensor memory
    extern __shared__ uint8_t raw[];
    __shared__ TileBarriers bar;
    uint8_t* ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t crank = cluster_rank(), rank = SPLIT ? crank & 1 : crank, lead = SPLIT ? crank & ~1u : 0u;   // the pair's first
    const int split = SPLIT ? p.split : 1, part = SPLIT ? static_cast<int>(crank >> 1) : 0;
    const int b0 = SPLIT ? p.kb * part / split : 0, b1 = SPLIT ? p.kb * (part + 1) / split : p.kb;   // the pair's blocks
    const int pair = static_cast<int>(blockIdx.x) / (2 * split), pairs = static_cast<int>(gridDim.x) / (2 * split);
    volatile int* dead = &bar.dead;

    if (tid == 0) {
        bar.dead = 0;
        for (int i = 0; i < STAGES; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&bar.dfull[i], 1);
            mbar_init(&bar.dempty[i], 2 * kTileWarps);
        }
        mbar_init(&bar.done, 1);
        fence_mbar_init();
        prefetch_tensormap(&tmW);
        prefetch_tensormap(&tmX);
    }
    if (warp == kTileWarps + 1) tmem_alloc<2>(&bar.tmem, 512);
    tc_fence_before();
    __syncthreads();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;
    const int ntile = pair < p.tiles ? (p.tiles - pair + pairs - 1) / pairs : 0;
    int issued = 0;   // stages, by the loading warp

    if (warp >= kTileWarps) regs_give<kTileRegsLeft>();
    if (warp >= kTileWarps + 2) {
    } else if (warp == kTileWarps) {
        pdl_wait_trigger();
        const uint64_t keep = l2_policy_evict_last();
        const uint32_t extra = blockIdx.x == 0 && (test_inject() & GEM_INJECT_RING_SHORTFALL) ? 16u : 0u;
        const uint32_t base = smem_u32(ring), full0 = peer_addr(&bar.full[0], lead);
        int s = 0;
        uint32_t phase = 1;
        bool ok = true;
        for (int i = 0; i < ntile && ok; ++i) {
            const int t = pair + i * pairs, mt = t % p.mtiles, nt = t / p.mtiles;
            const int m0 = mt * 256 + static_cast<int>(rank) * 128, n0 = nt * BN + static_cast<int>(rank) * (BN / 2);
            for (int b = b0; b < b1; ++b) {
                if (issued >= STAGES && !warp_wait(&bar.empty[s], phase, p.status, dead)) {
                    ok = false;
                    break;
                }
                if (rank == 0) warp_expect_tx(&bar.full[s], 2 * STAGE + (issued == 0 ? extra : 0u));
                warp_tma_2d_pair(base + s * STAGE, &tmX, b * 128, m0, full0 + 8 * s, keep);
                warp_tma_2d_pair(base + s * STAGE + 16384, &tmW, b * 128, n0, full0 + 8 * s, keep);
                ++issued;
                if (++s == STAGES) s = 0, phase ^= 1;
            }
        }
        // the last products' arrivals come from the other CTA's side: this one stays until they are here
        for (int i = 0; i < STAGES && ok; ++i) {   // (a stage without any passes at once)
            ok = warp_wait(&bar.empty[s], phase, p.status, dead);
            if (++s == STAGES) s = 0, phase ^= 1;
        }
        if (!ok) *dead = 1;
    } else if (warp == kTileWarps + 1) {
        if (rank == 0) {
            constexpr uint32_t idesc = umma_idesc_e4m3(256, BN);
            const uint64_t da0 = umma_desc(smem_u32(ring)), db0 = umma_desc(smem_u32(ring) + 16384);
            const int total = ntile * (b1 - b0);
            uint64_t da = da0, db = db0;
            int i = 0, s = 0;
            uint32_t phase = 0;
            pdl_wait();   // (as above)
            for (; i < total; ++i) {
                const int d = i & (NB - 1);
                if (i >= NB && !warp_wait(&bar.dempty[d], static_cast<uint32_t>((i / NB - 1) & 1), p.status, dead)) break;
                if (!warp_wait(&bar.full[s], phase, p.status, dead)) break;
                tc_fence_after();
                umma_e4m3<2>(tmem + d * BN, da, db, idesc);
                umma_commit<2>(&bar.empty[s], 3u << lead);
                umma_commit<2>(&bar.dfull[d], 3u << lead);
                da += STAGE >> 4, db += STAGE >> 4;
                if (++s == STAGES) s = 0, phase ^= 1, da = da0, db = db0;
            }
            if (i < total) {
                *dead = 1;
                // what was issued ends before the tensor memory is given back
                umma_commit<2>(&bar.done, 3u << lead);
                (void)mbar_wait(&bar.done, 0, nullptr);
            }
        }
    } else {
        regs_take<kTileRegs>();
        const int col = (warp >> 2) * CW;
        const uint32_t from = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + col;
        const uint32_t empty0 = peer_addr(&bar.dempty[0], lead);
        float* stage = reinterpret_cast<float*>(ring + STAGES * STAGE + warp * 4096);
        float* xs_sh = reinterpret_cast<float*>(ring + STAGES * STAGE + kTileWarps * 4096 + warp * kTileScales);
        pdl_wait_trigger();
        int i = 0;
        bool ok = true;
        for (int it = 0; it < ntile && ok; ++it) {
            const int t = pair + it * pairs, mt = t % p.mtiles, nt = t / p.mtiles;
            const int mw = mt * 256 + static_cast<int>(rank) * 128 + (warp & 3) * 32, n0 = nt * BN + col;   // the warp's first row and column
            // x scales of the next blocks, 8 of a row side by side, into [block][row]
            auto request = [&](int b, int half) {
                const int q = b + (lane & 7);
                const uint32_t to = smem_u32(xs_sh) + ((half * kTileChunk + (lane & 7)) * kTilePitch + (lane >> 3)) * 4;
                if (q < p.kb) {
                    const float* src = p.xs + q;
#pragma unroll
                    for (int r = 0; r < 32; r += 4) cp_async_4(to + 4 * r, src + min(mw + r + (lane >> 3), p.M - 1) * p.ldxs);
                }
                cp_async_commit();
            };
            request(b0, 0);
            request(b0 + kTileChunk, 1);
            // the warp's columns lie in one block of 128 rows of W, whose scales are requested two blocks ahead
            static_assert(128 % CW == 0);
            const float* wrow = p.ws + static_cast<int64_t>(min(n0, p.N - 1) >> 7) * p.kb;
            uint64_t acc[CW / 2];
#pragma unroll
            for (int m = 0; m < CW / 2; ++m) acc[m] = 0;
            float w0 = __ldg(wrow + b0), w1 = __ldg(wrow + min(b0 + 1, p.kb - 1));
            for (int b = b0; b < b1; ++b, ++i) {
                const int c = (b - b0) & (2 * kTileChunk - 1);
                if ((c & (kTileChunk - 1)) == 0) {
                    if (b > b0) {   // the half that is behind takes the blocks after the next ones
                        __syncwarp();
                        request(b + kTileChunk, (c / kTileChunk) ^ 1);
                    }
                    cp_async_wait<1>();
                    __syncwarp();
                }
                const uint64_t s2 = pair_of(xs_sh[c * kTilePitch + lane] * w0);
                w0 = w1;
                w1 = __ldg(wrow + min(b + 2, p.kb - 1));
                const int d = i & (NB - 1);
                if (!warp_wait(&bar.dfull[d], static_cast<uint32_t>((i / NB) & 1), p.status, dead)) {
                    *dead = 1;
                    ok = false;
                    break;
                }
                tc_fence_after();
                // 32 columns at a time, as two reads of 16 (one of 32, which wants its registers in a row, spills)
                constexpr int G = CW < 32 ? 1 : 2;
#pragma unroll
                for (int u = 0; u < CW / 16; u += G) {
                    float v[G][16];
#pragma unroll
                    for (int g = 0; g < G; ++g) tmem_ld<16>(v[g], from + d * BN + 16 * (u + g));
                    tmem_wait_ld();
                    if (u + G == CW / 16) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive_peer(empty0 + 8 * d);
                    }
#pragma unroll
                    for (int g = 0; g < G; ++g)
#pragma unroll
                        for (int q = 0; q < 8; ++q) pair_fma(acc[8 * (u + g) + q], v[g][2 * q], v[g][2 * q + 1], s2);
                }
            }
            cp_async_wait<0>();
            if (!ok) break;
            if constexpr (SPLIT) {   // to where the ring was: all products are done.  [row][column], 16-byte pieces turned by the row
                const int row = (warp & 3) * 32 + lane;
#pragma unroll
                for (int q = 0; q < CW / 4; ++q) {
                    const float2 lo = pair_get(acc[2 * q]), hi = pair_get(acc[2 * q + 1]);
                    reinterpret_cast<float4*>(ring)[row * (BN / 4) + ((col / 4 + q) ^ (row & 7))] = make_float4(lo.x, lo.y, hi.x, hi.y);
                }
            }
            // out through the warp's piece of shared memory, 32 columns at a time: rows of 128 bytes, whose
            // 16-byte pieces are turned by the row, so that neither side meets itself in a bank
#pragma unroll
            for (int c0 = 0; c0 < (SPLIT ? 0 : CW); c0 += 32) {
                tma_store_wait_read<0>();   // the elected lane's copies of what stood here before
                __syncwarp();
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    {
                        const float2 lo = pair_get(acc[(c0 + 4 * q) / 2]), hi = pair_get(acc[(c0 + 4 * q) / 2 + 1]);
                        reinterpret_cast<float4*>(stage)[lane * 8 + (q ^ (lane & 7))] = make_float4(lo.x, lo.y, hi.x, hi.y);
                    }
                if (p.copy) {
                    // rows and columns past the end of y are left out by the copy
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (n0 + c0 < p.N && mw < p.M) warp_tma_store_2d(&tmY, n0 + c0, mw, smem_u32(stage));
                    continue;
                }
                __syncwarp();
                const int q = lane & 7;
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += 4) {
                    const int r = r0 + (lane >> 3), m = mw + r, n = n0 + c0 + 4 * q;
                    if (m < p.M && n < p.N) {
                        float4 v = reinterpret_cast<const float4*>(stage)[r * 8 + (q ^ (r & 7))];
                        float* to = p.y + m * p.ldy + n;
                        const float* add = p.res ? p.res + m * p.ldy + n : nullptr;
                        if (p.wide && n + 4 <= p.N) {
                            if (add) {
                                const float4 a = *reinterpret_cast<const float4*>(add);
                                v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
                            }
                            *reinterpret_cast<float4*>(to) = v;
                        } else {
                            const float e[4] = {v.x, v.y, v.z, v.w};
                            for (int j = 0; j < 4 && n + j < p.N; ++j) to[j] = add ? e[j] + add[j] : e[j];
                        }
                    }
                }
                __syncwarp();
            }
        }
        tma_store_wait_read<0>();
    }
    __syncwarp();
    if constexpr (SPLIT) {
        // the parts of the cluster's one tile: each CTA adds up a share of its half's rows, in order of k
        cluster_sync();
        const int mt = pair % p.mtiles, nt = pair / p.mtiles;
        if (warp < kTileWarps) {
            const int first = 128 * part / split, end = 128 * (part + 1) / split;
            for (int i = first * (BN / 4) + tid; i < end * (BN / 4); i += kTileWarps * 32) {
                const int row = i / (BN / 4), q = i % (BN / 4);
                const int m = mt * 256 + static_cast<int>(rank) * 128 + row, n = nt * BN + 4 * q;
                if (m >= p.M || n >= p.N) continue;
                const float4* at = reinterpret_cast<const float4*>(ring) + row * (BN / 4) + (q ^ (row & 7));
                float4 v[kTileSplit];
#pragma unroll
                for (int r = 0; r < kTileSplit; ++r)
                    v[r] = r < split ? ld_peer4(peer_addr(at, 2 * r + rank)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int r = 1; r < kTileSplit; ++r)
                    if (r < split) v[0].x += v[r].x, v[0].y += v[r].y, v[0].z += v[r].z, v[0].w += v[r].w;
                float* to = p.y + m * p.ldy + n;
                const float* add = p.res ? p.res + m * p.ldy + n : nullptr;
                if (p.wide && n + 4 <= p.N) {
                    if (add) {
                        const float4 a = *reinterpret_cast<const float4*>(add);
                        v[0].x += a.x, v[0].y += a.y, v[0].z += a.z, v[0].w += a.w;
                    }
                    *reinterpret_cast<float4*>(to) = v[0];
                } else {
                    const float e[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
                    for (int j = 0; j < 4 && n + j < p.N; ++j) to[j] = add ? e[j] + add[j] : e[j];
                }
            }
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    // the copies of both CTAs are counted on the first one's barriers
    if (*dead && rank == 0 && warp == kTileWarps && lane == 0) drain_stages(bar.full, STAGES, max(0, issued - STAGES), issued - 1);
    __syncwarp();
    cluster_sync();
    if (warp == kTileWarps + 1) {
        tc_fence_after();
        tmem_free<2>(tmem, 512);
    }
}

gem_status ensure_smem(const void* fn, int device, size_t bytes) {
    static std::mutex mu;
    static std::map<std::pair<int, const void*>, size_t> done;
    std::lock_guard<std::mutex> lk(mu);
    size_t& have = done[{device, fn}];
    if (have >= bytes) return GEM_OK;
    GEM_CUDA_TRY(cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes)));
    have = bytes;
    return GEM_OK;
}

// CTAs of clusters of s that run at once, one an SM (a cluster lies in one GPC, so not all SMs can be used).
int cluster_room(const void* fn, int threads, int s, int device) {
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim = {static_cast<unsigned>(s), 1, 1};
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(s);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = kSmSmem / 2;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (ensure_smem(fn, device, kSmSmem / 2) == GEM_OK && cudaOccupancyMaxActiveClusters(&n, fn, &cfg) == cudaSuccess) return n * s;
    (void)cudaGetLastError();   // none then
    return 0;
}

// For every size of cluster of a kernel; asked once a device.
template <auto* KERNEL>
std::array<int, kMaxSplit + 1> cluster_rooms(int threads, int device) {
    static std::mutex mu;
    static std::map<int, std::array<int, kMaxSplit + 1>> known;
    std::lock_guard<std::mutex> lk(mu);
    auto [it, fresh] = known.try_emplace(device);
    if (fresh)
        for (int s = 2; s <= kMaxSplit; ++s) it->second[s] = cluster_room(reinterpret_cast<const void*>(KERNEL), threads, s, device);
    return it->second;
}

// Rows of W a tile and CTAs that share a tile's blocks by their time (returned in us, without beginning and end): the
// blocks' products and adds, whatever the rows of W, or the read of W but for the first blocks, which are on their way
// before the call begins.  A cluster costs its joining; of clusters there is one round.  (61 x 21504 x 5376: 3 CTAs on 120 rows, which it takes, 23.4 us, 3 on 128 23.7, 2 on 72 24.9,
// 1 on 72 37.9; 16 x 9728 x 2560, three weights in turn: 5 on 96, which it takes, 7.0, 4 on 128 6.8, 3 on 64 8.1, 2 on 64 9.1,
// 1 on 64 12.6.)
template <int NT>
double plan_rows(GemmParams* g, const DeviceInfo& di) {
    GemmParams& p = *g;
    constexpr int J = kGroup<NT>;
    constexpr double block = NT <= 16 ? 0.12 : NT <= 32 ? 0.16 : NT <= 64 ? 0.27 : 0.42;
    const int groups = (p.kb + J - 1) / J;
    const auto rooms = cluster_rooms<fp8_rows_kernel<NT>>(kWarps<NT> * 128 + 64, di.device);
    double best = 1e30;
    for (int r = 128; r >= 8; r -= 8) {
        const int tiles = (p.N + r - 1) / r;
        for (int s = 1; s <= kMaxSplit && s <= groups; ++s) {
            if (s > 1 && int64_t(tiles) * s > rooms[s]) continue;
            const int blocks = std::min(p.kb, (groups + s - 1) / s * J), rounds = s > 1 ? 1 : (tiles + di.num_sms - 1) / di.num_sms;
            const double total = static_cast<double>(rounds) * blocks;   // of the busiest SM
            // its share of the read, which fewer SMs do not draw at the whole rate
            const double read = std::max(static_cast<double>(std::min<int64_t>(int64_t(tiles) * s, di.num_sms)), 140.0) * r * (128.0 / 5.9e6);
            const double us = std::max(total * block, std::max(0.0, total - 8.0) * read) + (s > 1 ? 1.2 + 0.04 * p.M : 0.0);
            if (us < best * 0.999) {
                best = us;
                p.rows = r;
                p.split = s;
            }
        }
    }
    p.tiles = (p.N + p.rows - 1) / p.rows;
    return best;
}

template <int NT>
gem_status launch_rows(GemmParams p, const void* W, int64_t K, const void* x, int64_t ldx, const DeviceInfo& di, cudaStream_t stream) {
    gem_status st;
    plan_rows<NT>(&p, di);
    constexpr int J = kGroup<NT>;
    const int groups = (p.kb + J - 1) / J, per = (groups + p.split - 1) / p.split;
    p.chunk = std::min(per * J, kScaleBytes / (kPitch<NT> * 4) / J * J);
    const int stage = J * (p.rows + NT) * 128, after = std::max(0, 16384 - p.rows * 128 - J * NT * 128);
    const int fixed = 1024 + after + p.chunk * kPitch<NT> * 4;
    const int64_t grid = p.split > 1 ? int64_t(p.tiles) * p.split : std::min<int64_t>(p.tiles, di.num_sms);
    const int64_t steps = per * ((int64_t(p.tiles) * p.split + grid - 1) / grid);   // of the busiest CTA
    p.stages = static_cast<int>(std::min(std::min<int64_t>(kMaxStages, steps),
                                         (static_cast<int64_t>(di.smem_optin) - fixed - static_cast<int>(sizeof(RowsBarriers)) - 512) / stage));
    // a cluster's sums lie where the ring was, and the x scales behind the ring are still read by then (one stage is
    // too short for 128 rows of x on fewer than 128 of W, two are not)
    if (p.split > 1) p.stages = std::max(p.stages, (NT * 512 + stage - 1) / stage);
    static_assert(1024 + 16384 + kScaleBytes + NT * 512 + kGroup<NT> * (128 + NT) * 128 + sizeof(RowsBarriers) + 512 <= 227 << 10);
    const size_t smem = std::max(static_cast<size_t>(fixed + p.stages * stage), static_cast<size_t>(p.split > 1 ? kClusterSmem<NT> : 0));
    p.whole = K % 128 == 0;
    CUtensorMap tmW, tmX;
    const auto u8 = CU_TENSOR_MAP_DATA_TYPE_UINT8;
    const auto swz = CU_TENSOR_MAP_SWIZZLE_128B;
    const uint64_t uK = K, uN = p.N, uM = p.M, blocks = p.kb;
    const uint32_t rows = p.rows;
    if (p.whole) {
        if ((st = make_tensor_map_3d(&tmW, u8, W, {128, uN, blocks}, uK, 128, {128, rows, J}, swz)) != GEM_OK) return st;
        if ((st = make_tensor_map_3d(&tmX, u8, x, {128, uM, blocks}, ldx, 128, {128, NT, J}, swz)) != GEM_OK) return st;
    } else {
        if ((st = make_tensor_map_2d(&tmW, u8, W, uK, uN, uK, 128, rows, swz)) != GEM_OK) return st;
        if ((st = make_tensor_map_2d(&tmX, u8, x, uK, uM, ldx, 128, NT, swz)) != GEM_OK) return st;
    }
    const void* fn = reinterpret_cast<const void*>(fp8_rows_kernel<NT>);
    if ((st = ensure_smem(fn, di.device, smem)) != GEM_OK) return st;
    void* args[] = {&tmW, &tmX, &p};
    return launch_pdl_cluster(fn, dim3(static_cast<unsigned>(grid)), dim3(kWarps<NT> * 128 + 64), smem, stream, args, p.split);
}

template <int BN, bool SPLIT>
gem_status launch_tile(const GemmParams& g, int split, const void* W, int64_t K, const void* x, int64_t ldx, const DeviceInfo& di, cudaStream_t stream) {
    TileParams p{};
    p.split = split;
    p.ws = g.ws, p.xs = g.xs, p.ldxs = g.ldxs, p.res = g.res, p.y = g.y, p.ldy = g.ldy, p.N = g.N, p.M = g.M, p.kb = g.kb, p.status = g.status;
    p.mtiles = (p.M + 255) / 256;
    p.tiles = p.mtiles * ((p.N + BN - 1) / BN);
    p.wide = !(((reinterpret_cast<uintptr_t>(p.y) | reinterpret_cast<uintptr_t>(p.res)) & 15) || p.ldy % 4);
    gem_status st;
    CUtensorMap tmW, tmX;
    if ((st = make_tensor_map_2d(&tmW, CU_TENSOR_MAP_DATA_TYPE_UINT8, W, K, p.N, K, 128, BN / 2, CU_TENSOR_MAP_SWIZZLE_128B)) != GEM_OK) return st;
    if ((st = make_tensor_map_2d(&tmX, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, K, p.M, ldx, 128, 128, CU_TENSOR_MAP_SWIZZLE_128B)) != GEM_OK) return st;
    CUtensorMap tmY = tmX;
    p.copy = p.wide && !p.res;
    if (p.copy && (st = make_tensor_map_2d(&tmY, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, p.y, p.N, p.M, p.ldy * 4, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B)) != GEM_OK) return st;
    const void* fn = reinterpret_cast<const void*>(fp8_tile_kernel<BN, SPLIT>);
    if ((st = ensure_smem(fn, di.device, kTileSmem<BN>)) != GEM_OK) return st;
    const int pairs = split > 1 ? p.tiles * split : std::min(p.tiles, di.num_sms / 2);
    void* args[] = {&tmW, &tmX, &tmY, &p};
    return launch_pdl_cluster(fn, dim3(static_cast<unsigned>(2 * pairs)), dim3(kTileThreads), kTileSmem<BN>, stream, args, 2 * split);
}

}  // namespace
}  // namespace gem

extern "C" {

gem_status gem_fp8_gemm(const void* W, const float* ws, int64_t N, int64_t K, const void* x, int64_t ldx,
                        const float* xs, int64_t ldxs, int64_t M, float* y, int64_t ldy, const float* residual,
                        int32_t* status, void* stream_v) {
    using namespace gem;
    if (M < 0 || N < 0 || K < 0) return GEM_ERR_INVALID_ARG;
    constexpr int64_t lim = (int64_t(1) << 31) - 512;   // tiles at the edge end in 32 bits
    if (K % 16 || M > lim || N > lim || K > lim || ((M + 255) / 256) * ((N + 127) / 128) > lim) return GEM_ERR_UNSUPPORTED_SHAPE;
    if (M == 0 || N == 0) return GEM_OK;
    if (K == 0 || !W || !ws || !x || !xs || !y) return GEM_ERR_INVALID_ARG;
    if (ldx < K || ldxs < (K + 127) / 128 || ldy < N) return GEM_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(W) & 15) || (reinterpret_cast<uintptr_t>(x) & 15) || (ldx & 15) ||
        ((reinterpret_cast<uintptr_t>(ws) | reinterpret_cast<uintptr_t>(xs) | reinterpret_cast<uintptr_t>(y) |
          reinterpret_cast<uintptr_t>(residual) | reinterpret_cast<uintptr_t>(status)) & 3))
        return GEM_ERR_MISALIGNED;
    if (M == 1) ldx = K;   // leads nowhere, and a tensor map takes no stride of 2^40 or more
    DeviceInfo di;
    gem_status st;
    if ((st = device_info(&di)) != GEM_OK) return st;
    GemmParams p{};
    p.ws = ws;
    p.N = static_cast<int>(N);
    p.kb = static_cast<int>((K + 127) / 128);
    p.ldxs = ldxs;
    p.ldy = ldy;
    p.status = status ? status : di.status_word;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    p.M = static_cast<int>(M);
    p.xs = xs;
    p.y = y;
    p.res = residual;
    if (M <= 16) return launch_rows<16>(p, W, K, x, ldx, di, stream);
    if (M <= 32) return launch_rows<32>(p, W, K, x, ldx, di, stream);
    if (M <= 64) return launch_rows<64>(p, W, K, x, ldx, di, stream);
    // More rows: tiles of 256, 128 or 64 columns by their time, rounds of 76 pairs x blocks x 0.5, 0.32 or 0.24 us (a
    // smaller tile costs more for its size and less where there are few); where few tiles have many blocks, clusters of two
    // to four pairs share them out, which costs 4 us for the join.  Up to 128 rows the kernel above where it takes less
    // (128 x 21504 x 5376: 31 us and 48, 128 x 5376 x 21504: 38 and 47; 128 x 2048 x 4096: 13 and 7.7).
    struct Choice { double us = 1e30; int bn = 256, split = 1; } best;
    const int64_t mt = (M + 255) / 256, pairs = di.num_sms / 2;
    const auto rooms = cluster_rooms<fp8_tile_kernel<256, true>>(kTileThreads, di.device);
    for (auto [bn, step] : {std::pair(256, 0.5), std::pair(128, 0.32), std::pair(64, 0.24)}) {
        const int64_t tiles = mt * ((N + bn - 1) / bn);
        for (int s = 1; s <= (bn > 64 ? kTileSplit : 1) && (s == 1 || s * 4 <= p.kb); ++s) {
            if (s > 1 && tiles * 2 * s > rooms[2 * s]) break;
            const double us = 4.0 + static_cast<double>(s > 1 ? 1 : (tiles + pairs - 1) / pairs) * ((p.kb + s - 1) / s) * step + (s > 1 ? 4.0 : 0.0);
            if (us < best.us) best = {us, bn, s};
        }
    }
    if (M <= 128 && plan_rows<128>(&p, di) + 4.5 <= best.us) return launch_rows<128>(p, W, K, x, ldx, di, stream);
    if (best.bn == 256) return best.split > 1 ? launch_tile<256, true>(p, best.split, W, K, x, ldx, di, stream) : launch_tile<256, false>(p, 1, W, K, x, ldx, di, stream);
    if (best.bn == 128) return best.split > 1 ? launch_tile<128, true>(p, best.split, W, K, x, ldx, di, stream) : launch_tile<128, false>(p, 1, W, K, x, ldx, di, stream);
    return launch_tile<64, false>(p, 1, W, K, x, ldx, di, stream);
}

}  // extern "C"
