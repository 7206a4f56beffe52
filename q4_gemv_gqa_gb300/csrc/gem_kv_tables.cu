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

// Inclusive sum over the CTA's threads; *total receives the sum of all of them.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* warp_sums, int64_t* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    __syncthreads();   // the last scan's sums have been read
    if (lane == 31) warp_sums[w] = v;
    __syncthreads();
    int64_t s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
    }
    *total = __shfl_sync(0xffffffffu, s, 31);
    const int64_t before = __shfl_sync(0xffffffffu, s, w > 0 ? w - 1 : 0);
    return v + (w > 0 ? before : 0);
}

// One CTA: the running sums over the requests in chunks of 1024, then the pages and the tokens.
__global__ void __launch_bounds__(kTabThreads) kv_tables_kernel(const TableParams P) {
    __shared__ int64_t warp_sums[32];
    __shared__ int32_t cu_s[kMaxRequests + 1];      // tokens before request b
    __shared__ int32_t first_s[kMaxRequests];       // pages handed out before request b
    pdl_wait_trigger();
    const int tid = threadIdx.x;
    const int64_t head = P.ring_in[0], tail = P.ring_in[1];
    int64_t free_pages = tail - head;
    const bool bad_ring = head < 0 || free_pages < 0 || free_pages > P.n_pages;
    int64_t room = P.n_pages - free_pages;
    if (bad_ring) free_pages = room = 0;
    const int64_t page = P.page;
    int64_t c_wants = 0, c_need = 0, c_n = 0, c_given = 0, c_back_asked = 0, c_back = 0;
    bool refused = false;
    for (int base = 0; base < P.B; base += kTabThreads) {
        const int b = base + tid;
        const bool in = b < P.B;
        const int64_t cached = in ? P.cached[b] : 0, fresh = in ? P.fresh[b] : 0;
        const int64_t held = (cached + page - 1) >> P.lpage;
        bool ok = in && cached >= 0 && fresh >= -1 && cached + max(fresh, int64_t(0)) <= P.max_pages * page;
        const bool ends = ok && fresh == -1;
        const int64_t wants = ok && !ends ? fresh : 0;
        int64_t total;
        int64_t run = block_scan(wants, warp_sums, &total) + c_wants;
        c_wants += total;
        ok = ok && (wants == 0 || run <= P.T_cap);
        int64_t need = ok && !ends ? ((cached + wants + page - 1) >> P.lpage) - held : 0;
        run = block_scan(need, warp_sums, &total) + c_need;
        c_need += total;
        ok = ok && (need == 0 || run <= free_pages);
        if (!ok) need = 0;
        int64_t back = ends ? held : 0;
        run = block_scan(back, warp_sums, &total) + c_back_asked;
        c_back_asked += total;
        if (back && run > room) ok = false;
        if (!ok) back = 0;
        const int64_t n = ok ? wants : 0;
        const int64_t n_run = block_scan(n, warp_sums, &total) + c_n;
        c_n += total;
        const int64_t given = block_scan(need, warp_sums, &total) + c_given;
        c_given += total;
        const int64_t back_run = block_scan(back, warp_sums, &total) + c_back;
        c_back += total;
        if (in) {
            cu_s[b + 1] = static_cast<int32_t>(n_run);
            first_s[b] = static_cast<int32_t>(given - need);
            P.kv_len[b] = static_cast<int32_t>(ok && ends ? 0 : cached + n);
            P.cu[b + 1] = static_cast<int32_t>(n_run);
            refused |= !ok;
            int32_t* row = P.table + b * P.max_pages;
            for (int64_t k = 0; k < need; ++k) row[held + k] = P.ring[(head + given - need + k) % P.n_pages];
            for (int64_t k = 0; k < back; ++k) P.ring[(tail + back_run - back + k) % P.n_pages] = row[k];
        }
    }
    if (tid == 0) {
        cu_s[0] = 0;
        P.cu[0] = 0;
        P.ring_out[0] = head + c_given;
        P.ring_out[1] = tail + c_back;
        if (bad_ring) atomicOr(P.status, GEM_DEVFLAG_PAGE_RANGE);
    }
    if (refused) atomicOr(P.status, GEM_DEVFLAG_NO_ROOM);
    __syncthreads();
    for (int64_t t = tid; t < P.T_cap; t += kTabThreads) {
        int32_t slot = -1, pos = -1, seq = -1;
        if (t < c_n) {
            int lo = 0, hi = P.B - 1;   // the last request whose tokens begin at or before t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu_s[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            const int64_t cached = P.cached[lo], held = (cached + page - 1) >> P.lpage;
            const int64_t p = cached + (t - cu_s[lo]), pi = p >> P.lpage;
            const int32_t id = pi < held ? P.table[lo * P.max_pages + pi]
                                         : P.ring[(head + first_s[lo] + (pi - held)) % P.n_pages];
            slot = static_cast<int32_t>(id * page + (p & (page - 1)));
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
    const gem_status st = flag_word(&P.status);
    if (st != GEM_OK) return st;
    void* args[] = {&P};
    return launch_pdl(reinterpret_cast<const void*>(kv_tables_kernel), dim3(1), dim3(kTabThreads), 0,
                      static_cast<cudaStream_t>(stream), args);
}
