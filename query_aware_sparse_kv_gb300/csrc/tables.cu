// Page tables, slot map and touched-page list of one scheduler step, from
// the requests' lengths and a list of free pages.
//
// Request b holds old_b tokens and brings new_b more.  With the prefix sums
// over the requests of tokens (new), of pages to take (need = ceil((old +
// new) / P) - ceil(old / P)) and of pages touched (those that the new tokens
// fall into), every output entry is independent of every other: token i and
// touched page e find their request by binary search in a prefix and compute
// their place from it.  A page that is new takes free_pages[need prefix +
// its rank]; the token loop reads it there too, so nothing waits for the
// page-table entry another thread writes.
//
// Admission is in order: a request fits while the token and page prefixes,
// its own share included, stay within max_tokens and n_free.  The prefixes
// only grow, so once one request does not fit no later one that adds tokens
// does, and the prefixes of the requests that fit hold only such requests.
//
// Bound by latency: a step of 256 requests with a token each takes 4.3 us on
// one GB300 (launch, lengths, scan, page, store in turn), 1500 requests with
// 400000 token places 7.6 us (3.6 MB of outputs).  Up to kScanRequests requests
// every CTA scans all lengths itself into shared memory, one launch (3900
// requests: 8.7 us, 20.8 with two); beyond, a first launch writes the prefixes
// to the workspace, CTA c summing what lies before its requests by itself.  No
// CTA waits for another.
//
// Other kernels of this library may read page_table and seq_lens before
// their own wait for the kernel ahead.  This one therefore never lets its
// successor start early, and makes its writes visible before it exits.
#include "qskv_internal.h"
#include "qskv_kvq.cuh"

namespace qskv {
namespace {

constexpr int kThreads = 512;
constexpr int kScanRequests = kTablesScanRequests;

struct Need {
    int64_t tok, need, touch;
    __device__ __forceinline__ Need &operator+=(const Need &o) {
        tok += o.tok, need += o.need, touch += o.touch;
        return *this;
    }
};

// Exclusive prefixes with a last entry for the total, saturated at INT32_MAX
// (only entries below the capacities, which are smaller, are used further).
struct Prefix {
    int32_t *tok, *need, *touch;
    __device__ __forceinline__ void set(int i, const Need &n) const {
        const int64_t top = 0x7fffffff;
        tok[i] = int32_t(min(n.tok, top)), need[i] = int32_t(min(n.need, top)), touch[i] = int32_t(min(n.touch, top));
    }
};

// Pages hold 16 or 32 tokens.
__device__ __forceinline__ int page_shift(const TablesArgs &a) { return a.page_size == 16 ? 4 : 5; }

struct Request {
    int32_t old, add;
    bool valid;
    int32_t have, now;  // pages before and after (valid requests)
    __device__ __forceinline__ Request(const TablesArgs &a, int b) : Request(a, a.seq_lens[b], a.new_lens[b]) {}
    __device__ __forceinline__ Request(const TablesArgs &a, int32_t length, int32_t more) {
        old = length;
        add = more;
        const int64_t cap = int64_t(a.max_pages) * a.page_size;
        valid = old >= 0 && add >= 0 && int64_t(old) + add <= cap;
        const uint32_t P = a.page_size;  // unsigned: the sums may pass 2^31 - 1 by P - 1
        have = valid ? int32_t((uint32_t(old) + P - 1) >> page_shift(a)) : 0;
        now = valid ? int32_t((uint32_t(old) + uint32_t(add) + P - 1) >> page_shift(a)) : 0;
    }
    __device__ __forceinline__ Need need(const TablesArgs &a) const {
        Need n;
        n.tok = max(add, 0);
        n.need = now - have;
        n.touch = valid && add > 0 ? now - (old >> page_shift(a)) : 0;
        return n;
    }
};

__device__ __forceinline__ Need shfl_up_need(const Need &n, int o) {
    Need r;
    r.tok = __shfl_up_sync(0xffffffffu, n.tok, o);
    r.need = __shfl_up_sync(0xffffffffu, n.need, o);
    r.touch = __shfl_up_sync(0xffffffffu, n.touch, o);
    return r;
}

// Exclusive prefix of `mine` over the CTA's threads, plus `base`; *total is
// the sum over all threads plus `base`.
__device__ __forceinline__ Need block_scan(const Need &mine, const Need &base, Need *total) {
    __shared__ Need warp_sum[kThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Need incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Need up = shfl_up_need(incl, o);
        if (lane >= o) incl += up;
    }
    __syncthreads();
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    Need before = base, all = base;
#pragma unroll
    for (int w = 0; w < kThreads / 32; w++) {
        if (w < warp) before += warp_sum[w];
        all += warp_sum[w];
    }
    *total = all;
    before.tok += incl.tok - mine.tok, before.need += incl.need - mine.need, before.touch += incl.touch - mine.touch;
    return before;
}

// Prefixes of requests [r0, r1), r1 - r0 <= kScanRequests, into p[r0 ..]; a
// thread's lengths are all loaded before the first is used.
__device__ void scan_requests(const TablesArgs &a, int r0, int r1, const Need &base, const Prefix &p) {
    constexpr int kEach = (kScanRequests + kThreads - 1) / kThreads;
    const int per = (r1 - r0 + kThreads - 1) / kThreads;
    const int b0 = r0 + int(threadIdx.x) * per, n = max(0, min(per, r1 - b0));
    int32_t old[kEach], add[kEach];
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        old[i] = add[i] = 0;
        if (i < n) old[i] = a.seq_lens[b0 + i], add[i] = a.new_lens[b0 + i];
    }
    Need mine = {0, 0, 0};
#pragma unroll
    for (int i = 0; i < kEach; i++)
        if (i < n) mine += Request(a, old[i], add[i]).need(a);
    Need total, run = block_scan(mine, base, &total);
#pragma unroll
    for (int i = 0; i < kEach; i++) {
        if (i >= n) break;
        p.set(b0 + i, run);
        run += Request(a, old[i], add[i]).need(a);
    }
    if (threadIdx.x == 0 && r1 == a.batch) p.set(r1, total);
}

// Last index i of prefix[0..n] with prefix[i] <= x (prefix[0] = 0 <= x).
__device__ __forceinline__ int find(const int32_t *prefix, int n, int x) {
    int lo = 0, hi = n + 1;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ __forceinline__ bool admitted(const TablesArgs &a, const Prefix &p, const Request &r, int b) {
    return r.valid && r.add > 0 && p.tok[b + 1] <= a.max_tokens && p.need[b + 1] <= a.n_free;
}

// Physical page of request b's logical page j; -1 (flagged) if the free list
// or the table names a page outside the pool.
__device__ __forceinline__ int page_of(const TablesArgs &a, const Prefix &p, const Request &r, int b, int j) {
    const int id = j >= r.have ? a.free_pages[p.need[b] + (j - r.have)]
                               : a.page_table[int64_t(b) * a.max_pages + j];
    if (id >= 0 && id < a.num_pool_pages) return id;
    raise_error(a.flags, kErrPageId);
    return -1;
}

// n <= 4 values at dst[i], i a multiple of 4: one store where the buffer allows it.
__device__ __forceinline__ void store4(int32_t *dst, int64_t i, int n, const int (&v)[4]) {
    if (n == 4 && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
        *reinterpret_cast<int4 *>(dst + i) = make_int4(v[0], v[1], v[2], v[3]);
        return;
    }
#pragma unroll
    for (int k = 0; k < 4; k++)
        if (k < n) dst[i + k] = v[k];
}

// Slots and positions of the tokens from i on, SPAN (1 or 4) of them.
template <int SPAN>
__device__ __forceinline__ void write_tokens(const TablesArgs &a, const Prefix &p, int64_t i) {
    const int P = a.page_size, B = a.batch, n = int(min(int64_t(SPAN), a.max_tokens - i));
    int slot[4], pos[4], b = find(p.tok, B, int(i)), last = -1, page = -1, id = -1;
    bool fits = false;
    Request r(a, 0, 0);
#pragma unroll 1
    for (int k = 0; k < SPAN; k++) {
        slot[k] = pos[k] = -1;
        if (k >= n) continue;
        while (b < B && p.tok[b + 1] <= int(i) + k) b++;
        if (b >= B) continue;
        if (b != last) r = Request(a, b), fits = admitted(a, p, r, b), last = b, page = -1;
        if (!fits) continue;
        pos[k] = r.old + int(i) + k - p.tok[b];
        const int j = pos[k] >> page_shift(a);
        if (j != page) page = j, id = page_of(a, p, r, b, j);
        if (id >= 0) slot[k] = id * P + (pos[k] - j * P);
    }
    if (SPAN == 1) {
        a.slot_map[i] = slot[0];
        if (a.positions) a.positions[i] = pos[0];
        return;
    }
    store4(a.slot_map, i, n, slot);
    if (a.positions) store4(a.positions, i, n, pos);
}

// The CTAs below `token_ctas` write the tokens' outputs, the others those of
// the requests and of the touched pages; the last one also the counts.
template <int SPAN>
__device__ void write_tables(const TablesArgs &a, const Prefix &p, int token_ctas) {
    const int P = a.page_size, B = a.batch;
    const int cta = blockIdx.x, others = gridDim.x - token_ctas;
    if (cta < token_ctas) {
        const int64_t step = int64_t(token_ctas) * kThreads * SPAN;
        for (int64_t i = (int64_t(cta) * kThreads + threadIdx.x) * SPAN; i < a.max_tokens; i += step)
            write_tokens<SPAN>(a, p, i);
        return;
    }
    const int64_t first = int64_t(cta - token_ctas) * kThreads + threadIdx.x, step = int64_t(others) * kThreads;
    for (int64_t b = first; b < B; b += step) {
        const Request r(a, int(b));
        const bool ok = admitted(a, p, r, int(b));
        a.seq_lens_out[b] = ok ? r.old + r.add : r.old;
        a.cu_new[b] = min(p.tok[b], a.max_tokens);
        if (!r.valid) raise_error(a.flags, kErrSeqLen);
        if (r.valid && r.add > 0 && !ok) raise_error(a.flags, kErrCapacity);
    }
    if (first == 0) a.cu_new[B] = min(p.tok[B], a.max_tokens);
    for (int64_t e = first; e < a.max_touched; e += step) {
        int id = -1, valid = 0;
        const int b = find(p.touch, B, int(e));
        if (b < B) {
            const Request r(a, b);
            if (admitted(a, p, r, b)) {
                const int j = (r.old >> page_shift(a)) + int(e) - p.touch[b];
                id = page_of(a, p, r, b, j);
                if (j >= r.have) a.page_table[int64_t(b) * a.max_pages + j] = id;
                if (id >= 0) valid = min(P, r.old + r.add - j * P);
            }
        }
        if (a.touched_ids) a.touched_ids[e] = id, a.touched_valid[e] = valid;
    }
    if (a.counts && cta == gridDim.x - 1) {
        Need mine = {0, 0, 0};
        int64_t refused = 0;
        for (int b = threadIdx.x; b < B; b += kThreads) {
            const Request r(a, b);
            if (admitted(a, p, r, b)) {
                const Need n = r.need(a);
                mine.need += n.need, mine.touch += n.touch;
            } else if (r.add != 0) {
                refused++;
            }
        }
        mine.tok = refused;
        Need total;
        block_scan(mine, Need{0, 0, 0}, &total);
        if (threadIdx.x == 0) {
            a.counts[0] = min(p.tok[B], a.max_tokens);
            a.counts[1] = int32_t(total.need), a.counts[2] = int32_t(total.touch), a.counts[3] = int32_t(total.tok);
        }
    }
}

template <int SPAN>
__global__ void __launch_bounds__(kThreads) tables_kernel(TablesArgs a, int token_ctas) {
    __shared__ int32_t s[3][kScanRequests + 1];
    pdl_wait();
    const Prefix p{s[0], s[1], s[2]};
    scan_requests(a, 0, a.batch, Need{0, 0, 0}, p);
    __syncthreads();
    write_tables<SPAN>(a, p, token_ctas);
    __threadfence();
}

__global__ void __launch_bounds__(kThreads) tables_scan_kernel(TablesArgs a, Prefix p) {
    pdl_wait();
    const int r0 = blockIdx.x * kScanRequests, r1 = min(r0 + kScanRequests, a.batch);
    Need mine = {0, 0, 0}, base;
    for (int b = threadIdx.x; b < r0; b += kThreads) mine += Request(a, b).need(a);
    block_scan(mine, Need{0, 0, 0}, &base);
    scan_requests(a, r0, r1, base, p);
    __threadfence();
}

template <int SPAN>
__global__ void __launch_bounds__(kThreads) tables_write_kernel(TablesArgs a, Prefix p, int token_ctas) {
    pdl_wait();
    write_tables<SPAN>(a, p, token_ctas);
    __threadfence();
}

}  // namespace

cudaError_t launch_extend_tables(const TablesArgs &a, int32_t *scratch, int num_sms, cudaStream_t stream) {
    // One token a thread while that fits one CTA an SM (a step's latency is one chain of loads then), else four
    // neighbouring ones, which mostly share their request and page, up to two CTAs an SM.
    const bool few = (int64_t(a.max_tokens) + kThreads - 1) / kThreads <= num_sms;
    const int64_t per_cta = few ? kThreads : 4 * kThreads;
    int64_t tok = (int64_t(a.max_tokens) + per_cta - 1) / per_cta;
    if (tok > 2 * num_sms) tok = 2 * num_sms;
    int64_t rest = (int64_t(a.max_touched > a.batch ? a.max_touched : a.batch) + kThreads - 1) / kThreads;
    if (rest > num_sms) rest = num_sms;
    const dim3 grid(unsigned(tok + rest)), block(kThreads);
    if (a.batch <= kScanRequests)
        return few ? launch_pdl(tables_kernel<1>, grid, block, 0, stream, a, int(tok))
                   : launch_pdl(tables_kernel<4>, grid, block, 0, stream, a, int(tok));
    const Prefix p{scratch, scratch + (a.batch + 1), scratch + 2 * (a.batch + 1)};
    const cudaError_t e = launch_pdl(tables_scan_kernel, dim3(unsigned((a.batch + kScanRequests - 1) / kScanRequests)),
                                     block, 0, stream, a, p);
    if (e != cudaSuccess) return e;
    return few ? launch_pdl(tables_write_kernel<1>, grid, block, 0, stream, a, p, int(tok))
               : launch_pdl(tables_write_kernel<4>, grid, block, 0, stream, a, p, int(tok));
}

}  // namespace qskv
