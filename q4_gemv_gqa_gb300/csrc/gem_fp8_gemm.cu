// gem_fp8_gemm.cu — product of rows in 8-bit floating point with weights scaled by blocks of 128 x 128
// (gem_fp8_gemm), on tcgen05.
//
// y[m][n] = sum_b xs[m][b] ws[n / 128][b] d_b[m][n],  d_b = the product over the 128 values of block b.
// The tensor cores sum d_b in tensor memory (four instructions of 32 values, the first of which overwrites);
// other warps read it back, scale it and add it to sums in registers while the next block's product runs in
// another part of tensor memory.  So the scales may have any values and the long sums are plain fp32.
//
// fp8_rows_kernel (up to 128 rows of x): the weights are what the call reads, and the rows of W take the
// 128-row side of the product, the rows of x its 16..128 columns.
#include "gem_tcgen05.cuh"

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
constexpr int kScaleBytes = 24 << 10;

// Blocks a ring stage and a tensor-memory buffer hold, of four such buffers (kGroup * NT columns each, 512
// together at most): the waits and the read-back latency of a step are paid once for kGroup blocks.
template <int NT>
constexpr int kGroup = NT <= 32 ? 4 : NT == 64 ? 2 : 1;
template <int NT>
constexpr int kWarps = NT <= 32 ? 2 : 4;
constexpr int kBuffers = 4;
template <int NT>
constexpr int kPitch = NT + 4;   // of the x scales of a block: spreads a column's stores over the banks

struct RowsBarriers {
    uint64_t full[kMaxStages], empty[kMaxStages], dfull[4], dempty[4];
    uint32_t tmem;
    int dead;
};

template <int NT>
__global__ void __launch_bounds__(kWarps<NT> * 128 + 64) fp8_rows_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const GemmParams p) {
    constexpr int NB = kBuffers, J = kGroup<NT>, COLS = NB * J * NT, Q = kWarps<NT>, CW = NT / Q, XP = kPitch<NT>;
    extern __shared__ uint8_t raw[];
    __shared__ RowsBarriers bar;
    // the ring, 1024-byte aligned: a stage's blocks of W, then those of x; behind it the x scales and the cluster's sums
    uint8_t* ring = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    const int wbytes = p.rows * 128, stage_bytes = J * (wbytes + NT * 128);
    // a product reads 128 rows of W, of which p.rows are its own: the ring is followed by what that may be past its end
    float* xs_sh = reinterpret_cast<float*>(ring + p.stages * stage_bytes + max(0, 16384 - wbytes - J * NT * 128));
    float* part = xs_sh + p.chunk * XP;
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
            mbar_init(&bar.dempty[i], 4 * Q);
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
#pragma unroll
                    for (int u = 0; u < CW / 4; ++u) {   // a warp takes the rows warp, warp + 4 Q, ..
                        const int m = warp + 4 * Q * u;
                        const float* src = p.xs + m * p.ldxs + b;
                        for (int q = lane; q < nblk; q += 32) xs_sh[q * XP + m] = m < p.M ? __ldg(src + q) : 0.f;
                    }
                    asm volatile("bar.sync 1, %0;" ::"n"(Q * 128) : "memory");
                }
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
                // columns of blocks that the step does not have are read and not used
                float v[J][CW];
#pragma unroll
                for (int j = 0; j < J; ++j) tmem_ld<CW>(v[j], from + (d * J + j) * NT);
                tmem_wait_ld();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.dempty[d]);
#pragma unroll
                for (int j = 0; j < J; ++j)
                    if (j < nj) {
                        const float4* sx = reinterpret_cast<const float4*>(xs_sh + (c + j) * XP + col);
#pragma unroll
                        for (int q = 0; q < CW / 4; ++q) {
                            const float4 x4 = sx[q];
                            const float2 w2 = make_float2(w[j], w[j]);
                            acc[2 * q] = ffma2(make_float2(v[j][4 * q], v[j][4 * q + 1]), fmul2(make_float2(x4.x, x4.y), w2), acc[2 * q]);
                            acc[2 * q + 1] = ffma2(make_float2(v[j][4 * q + 2], v[j][4 * q + 3]), fmul2(make_float2(x4.z, x4.w), w2), acc[2 * q + 1]);
                        }
                    }
            }
            if (p.split > 1) {
#pragma unroll
                for (int m = 0; m < CW; ++m)
                    if (col + m < p.M) part[(col + m) * 128 + row] = m & 1 ? acc[m / 2].y : acc[m / 2].x;
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
                for (int m = rank + p.split * (warp >> 2); m < p.M; m += p.split * Q) {
                    float v = 0.f;
                    for (int r = 0; r < p.split; ++r) v += ld_peer(peer_addr(&part[m * 128 + row], r));
                    const int64_t at = m * p.ldy + n;
                    p.y[at] = p.res ? v + p.res[at] : v;
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

template <int NT>
gem_status launch_rows(GemmParams p, const void* W, int64_t K, const void* x, int64_t ldx, const DeviceInfo& di, cudaStream_t stream) {
    gem_status st;
    // Rows of W a tile and CTAs that share a tile's blocks: the shortest time of the busiest SM.  A block costs its
    // bytes, or its products where it has fewer than 64 rows (they take the same time for any number of rows);
    // a cluster costs its joining.  Clusters only where one round of them does it: 4 CTAs of one GPC fit 36 times.
    p.split = 1;
    p.rows = 128;
    double best = 1e30;
    for (int s : {1, 2, 4}) {
        const int room = s == 1 ? di.num_sms : s == 2 ? di.num_sms / 2 * 2 : di.num_sms / 4 * 4 - 8;
        if (s > 1 && p.kb < 8 * s) break;
        for (int r = 128; r >= 8; r -= 8) {
            const int64_t ctas = int64_t(s) * ((p.N + r - 1) / r);
            if (s > 1 && ctas > room) continue;
            const int64_t rounds = (ctas + di.num_sms - 1) / di.num_sms;
            const double cost = static_cast<double>(rounds) * ((p.kb + s - 1) / s) * std::max(r, 64) + (s > 1 ? 300.0 : 0.0);
            if (cost < best * 0.999) {
                best = cost;
                p.rows = r;
                p.split = s;
            }
        }
    }
    p.tiles = (p.N + p.rows - 1) / p.rows;
    constexpr int J = kGroup<NT>;
    const int groups = (p.kb + J - 1) / J, per = (groups + p.split - 1) / p.split;
    p.chunk = std::min(per * J, kScaleBytes / (kPitch<NT> * 4) / J * J);
    const int stage = J * (p.rows + NT) * 128, after = std::max(0, 16384 - p.rows * 128 - J * NT * 128);
    const int fixed = 1024 + after + p.chunk * kPitch<NT> * 4 + (p.split > 1 ? NT * 512 : 0);
    const int64_t grid = p.split > 1 ? int64_t(p.tiles) * p.split : std::min<int64_t>(p.tiles, di.num_sms);
    const int64_t steps = per * ((int64_t(p.tiles) * p.split + grid - 1) / grid);   // of the busiest CTA
    p.stages = static_cast<int>(std::min(std::min<int64_t>(kMaxStages, steps),
                                         (static_cast<int64_t>(di.smem_optin) - fixed - static_cast<int>(sizeof(RowsBarriers)) - 512) / stage));
    const size_t smem = static_cast<size_t>(fixed + p.stages * stage);
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

}  // namespace
}  // namespace gem

extern "C" {

gem_status gem_fp8_gemm(const void* W, const float* ws, int64_t N, int64_t K, const void* x, int64_t ldx,
                        const float* xs, int64_t ldxs, int64_t M, float* y, int64_t ldy, const float* residual,
                        int32_t* status, void* stream_v) {
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
    p.ws = ws;
    p.N = static_cast<int>(N);
    p.kb = static_cast<int>((K + 127) / 128);
    p.ldxs = ldxs;
    p.ldy = ldy;
    p.status = status ? status : di.status_word;
    cudaStream_t stream = static_cast<cudaStream_t>(stream_v);
    for (int64_t m = 0; m < M; m += 128) {
        p.M = static_cast<int>(std::min<int64_t>(128, M - m));
        p.xs = xs + m * ldxs;
        p.y = y + m * ldy;
        p.res = residual ? residual + m * ldy : nullptr;
        const uint8_t* xm = static_cast<const uint8_t*>(x) + m * ldx;
        if (p.M <= 16) st = launch_rows<16>(p, W, K, xm, ldx, di, stream);
        else if (p.M <= 32) st = launch_rows<32>(p, W, K, xm, ldx, di, stream);
        else if (p.M <= 64) st = launch_rows<64>(p, W, K, xm, ldx, di, stream);
        else st = launch_rows<128>(p, W, K, xm, ldx, di, stream);
        if (st != GEM_OK) return st;
    }
    return GEM_OK;
}

}  // extern "C"
