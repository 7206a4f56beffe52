// gem_kv_tables.cu — block tables and slot maps of a paged KV cache, from request lengths.
#include "gem_device.cuh"
#include "gem_kv4.cuh"

namespace gem {
namespace kv4 {
namespace {

constexpr int kTabThreads = 1024;

struct TableParams {
    const int32_t *cached, *fresh;
    int B, page, lpage;
    int32_t* table;
    int64_t max_pages;
    int32_t* ring;
    int64_t n_pages;
    const int64_t* ring_in;
    int64_t* ring_out;
    int32_t *kv_len, *cu, *slot, *pos, *seq;
    int64_t T_cap;
    int* status;
};

// Inclusive sums of two values over the CTA's threads (over the warp alone where `single`), and the sums
// of all of them.
__device__ __forceinline__ void scan2(bool single, int64_t (&v)[2], int64_t (&total)[2], int64_t (*warp_sums)[32]) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int64_t u = __shfl_up_sync(0xffffffffu, v[k], o);
            if (lane >= o) v[k] += u;
        }
    if (single) {
#pragma unroll
        for (int k = 0; k < 2; ++k) total[k] = __shfl_sync(0xffffffffu, v[k], 31);
        return;
    }
    __syncthreads();   // the last scan's sums have been read
    if (lane == 31) warp_sums[0][w] = v[0], warp_sums[1][w] = v[1];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        int64_t s = warp_sums[k][lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += u;
        }
        total[k] = __shfl_sync(0xffffffffu, s, 31);
        const int64_t before = __shfl_sync(0xffffffffu, s, w > 0 ? w - 1 : 0);
        v[k] += w > 0 ? before : 0;
    }
}

__device__ __forceinline__ int64_t ring_at(int64_t at, int64_t n) {
    if (((at | n) >> 32) == 0) return static_cast<uint32_t>(at) % static_cast<uint32_t>(n);
    return at % n;
}

// Three rounds of running sums over the requests, in chunks of the CTA's threads, then the pages and the
// tokens.  Every CTA goes through the requests (they are few, and a second launch or a grid barrier costs
// more than the sums); the requests' pages are dealt out to the CTAs, and so are the tokens, whose page
// comes from the table or, where this call hands it out, straight from the ring, so that no CTA waits for
// another's writes.  Up to 32 requests one warp does the sums without a barrier.
// 2.7 us for 8 requests with a token each, which is latency; 9 us for 1024 requests and 98 k tokens (1.3 MB): the sums,
// which every CTA repeats, with their barriers, and a search for each token, 3.9 M warp instructions in all.
__global__ void __launch_bounds__(kTabThreads) kv_tables_kernel(const TableParams P) {
    __shared__ int64_t warp_sums[2][32];
    __shared__ int32_t cu_s[kMaxRequests + 1];      // tokens before request b
    __shared__ int32_t first_s[kMaxRequests];       // pages handed out before request b
    pdl_wait_trigger();
    const int tid = threadIdx.x, lane = tid & 31;
    const int64_t head = P.ring_in[0], tail = P.ring_in[1];
    int64_t free_pages = tail - head;
    const bool bad_ring = head < 0 || free_pages < 0 || free_pages > P.n_pages;
    int64_t room = P.n_pages - free_pages;
    if (bad_ring) free_pages = room = 0;
    const int64_t page = P.page;
    int64_t c_wants = 0, c_asked = 0, c_need = 0, c_n = 0, c_given = 0, c_back = 0;
    bool refused = false;
    const bool single = P.B <= 32, chief = blockIdx.x == 0;
    for (int base = 0; base < P.B && (!single || tid < 32); base += blockDim.x) {
        const int b = base + tid;
        const bool in = b < P.B;
        const int64_t cached = in ? P.cached[b] : 0, fresh = in ? P.fresh[b] : 0;
        const int64_t held = (cached + page - 1) >> P.lpage;
        bool ok = in && cached >= 0 && fresh >= -1 && cached + max(fresh, int64_t(0)) <= P.max_pages * page;
        const bool ends = ok && fresh == -1;
        const int64_t wants = ok && !ends ? fresh : 0;
        int64_t back = ends ? held : 0;
        int64_t v[2] = {wants, back}, total[2];
        scan2(single, v, total, warp_sums);
        ok = ok && (wants == 0 || v[0] + c_wants <= P.T_cap) && (back == 0 || v[1] + c_asked <= room);
        c_wants += total[0], c_asked += total[1];
        int64_t need = ok && !ends ? ((cached + wants + page - 1) >> P.lpage) - held : 0;
        v[0] = need, v[1] = 0;
        scan2(single, v, total, warp_sums);
        ok = ok && (need == 0 || v[0] + c_need <= free_pages);
        c_need += total[0];
        if (!ok) need = back = 0;
        const int64_t n = ok ? wants : 0;
        // what is taken fits 32 bits: tokens, and pages given and put back
        v[0] = n, v[1] = need << 32 | back;
        scan2(single, v, total, warp_sums);
        const int64_t n_run = v[0] + c_n, given = (v[1] >> 32) - need + c_given, put = (v[1] & 0xffffffff) - back + c_back;
        c_n += total[0], c_given += total[1] >> 32, c_back += total[1] & 0xffffffff;
        if (in) {
            cu_s[b + 1] = static_cast<int32_t>(n_run);
            first_s[b] = static_cast<int32_t>(given);
            if (chief) {
                P.kv_len[b] = static_cast<int32_t>(ok && ends ? 0 : cached + n);
                P.cu[b + 1] = static_cast<int32_t>(n_run);
                refused |= !ok;
            }
        }
        // pages: each warp takes the requests of its lanes that have some, the lanes their pages
        for (uint32_t todo = __ballot_sync(0xffffffffu, need > 0 || back > 0); todo; todo &= todo - 1) {
            const int from = __ffs(todo) - 1, rb = b - lane + from;
            if ((rb % gridDim.x) != blockIdx.x) continue;
            const int64_t take = __shfl_sync(0xffffffffu, need, from), give = __shfl_sync(0xffffffffu, back, from);
            const int64_t h0 = __shfl_sync(0xffffffffu, held, from);
            const int64_t at = __shfl_sync(0xffffffffu, ends ? tail + put : head + given, from);
            int32_t* row = P.table + rb * P.max_pages;
            for (int64_t k = lane; k < take; k += 32) row[h0 + k] = P.ring[ring_at(at + k, P.n_pages)];
            for (int64_t k = lane; k < give; k += 32) P.ring[ring_at(at + k, P.n_pages)] = row[k];
        }
    }
    if (tid == 0) {
        cu_s[0] = 0;
        if (chief) {
            P.cu[0] = 0;
            P.ring_out[0] = head + c_given;
            P.ring_out[1] = tail + c_back;
            if (bad_ring) atomicOr(P.status, GEM_DEVFLAG_PAGE_RANGE);
        }
    }
    if (refused) atomicOr(P.status, GEM_DEVFLAG_NO_ROOM);
    __syncthreads();
    const int32_t taken = P.B ? cu_s[P.B] : 0;
    for (int64_t t = blockIdx.x * static_cast<int64_t>(blockDim.x) + tid; t < P.T_cap;
         t += static_cast<int64_t>(gridDim.x) * blockDim.x) {
        int32_t slot = -1, pos = -1, seq = -1;
        if (t < taken) {
            int lo = 0, hi = P.B - 1;   // the last request whose tokens begin at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu_s[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            const int64_t cached = P.cached[lo], held = (cached + page - 1) >> P.lpage;
            const int64_t p = cached + (t - cu_s[lo]), pi = p >> P.lpage;
            const int32_t id = pi < held ? P.table[lo * P.max_pages + pi]
                                         : P.ring[ring_at(head + first_s[lo] + (pi - held), P.n_pages)];
            if (id >= 0 && id < P.n_pages) {
                slot = static_cast<int32_t>(id * page + (p & (page - 1)));
            } else {   // not a page: a slot that every reader refuses
                slot = INT32_MIN;
                atomicOr(P.status, GEM_DEVFLAG_PAGE_RANGE);
            }
            pos = static_cast<int32_t>(p);
            seq = lo;
        }
        P.slot[t] = slot;
        P.pos[t] = pos;
        P.seq[t] = seq;
    }
}

}  // namespace
}  // namespace kv4
}  // namespace gem

extern "C" gem_status gem_kv_block_tables(const int32_t* cached, const int32_t* fresh, int B, int page,
                                          int32_t* table, int64_t max_pages, int32_t* ring, int64_t n_pages,
                                          const int64_t* ring_in, int64_t* ring_out, int32_t* kv_len,
                                          int32_t* cu_tokens, int32_t* slot, int32_t* pos, int32_t* seq,
                                          int64_t T_cap, int32_t* status, void* stream) {
    using namespace gem;
    using namespace gem::kv4;
    if (B < 0 || max_pages < 0 || n_pages < 0 || T_cap < 0) return GEM_ERR_INVALID_ARG;
    if (B > kMaxRequests || !page_ok(page) || n_pages > (INT32_MAX - 255) / page ||
        max_pages > (INT32_MAX - 255) / page || T_cap > INT32_MAX)
        return GEM_ERR_UNSUPPORTED_SHAPE;
    if (!ring_in || !ring_out || !cu_tokens || (n_pages && !ring)) return GEM_ERR_INVALID_ARG;
    if (B && (!cached || !fresh || !kv_len || (max_pages && !table))) return GEM_ERR_INVALID_ARG;
    if (T_cap && (!slot || !pos || !seq)) return GEM_ERR_INVALID_ARG;
    if (ring_out == ring_in || (B && (kv_len == cached || kv_len == fresh))) return GEM_ERR_INVALID_ARG;
    TableParams P{};
    P.cached = cached, P.fresh = fresh, P.B = B, P.page = page, P.lpage = log2_of(page);
    P.table = table, P.max_pages = max_pages, P.ring = ring, P.n_pages = n_pages;
    P.ring_in = ring_in, P.ring_out = ring_out, P.kv_len = kv_len, P.cu = cu_tokens;
    P.slot = slot, P.pos = pos, P.seq = seq, P.T_cap = T_cap, P.status = status;
    DeviceInfo di;
    const gem_status st = device_info(&di);
    if (st != GEM_OK) return st;
    if (!status) P.status = di.status_word;
    void* args[] = {&P};
    // a thread for each token of a large step; a decode step's tokens fit a CTA of few threads, which starts
    // sooner
    const int threads = B <= 32 && T_cap <= 256 ? 256 : kTabThreads;
    const int64_t ctas = std::max<int64_t>(1, std::min<int64_t>(di.num_sms, (T_cap + threads - 1) / threads));
    return launch_pdl(reinterpret_cast<const void*>(kv_tables_kernel), dim3(static_cast<unsigned>(ctas)), dim3(threads), 0,
                      static_cast<cudaStream_t>(stream), args);
}
