// The work items of one prefill call (qskv_prefill.cuh), from the lengths on
// the device: one CTA, a few passes over the tiles.
//
// A tile of a long row has up to len / block_keys key blocks, one of a short
// row few.  Tiles longer than a share of all work (blocks over all SMs, over
// `waves`) are cut into equal parts, whose partial results are merged by the
// attention kernel, so that few long rows fill the GPU; and the list is sorted
// by length, longest first, so that the CTAs that take items from it end at
// about the same time.  The order (and the slots of partial results) may
// differ from run to run; no result depends on it.  It takes 6 to 7 us, cold:
// the latency of lengths, prefix and list.
#include "qskv_prefill.cuh"

namespace qskv {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32, kBuckets = 256;
constexpr int kSharedRows = 4096;

struct Shared {
    int warp_sum[kWarps];
    unsigned long long blocks;  // of all tiles
    int longest;                // blocks of the longest part
    int begin[kBuckets];        // items of a bucket, then its first place in the list
    int slots;
    int tile_begin[kSharedRows + 1];  // a row's first tile, of as many rows (more: in the workspace)
};

// Sum of x over the threads before this one, and over all of them.
__device__ int exclusive_sum(Shared &s, int x, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += up;
    }
    if (lane == 31) s.warp_sum[warp] = incl;
    __syncthreads();
    const int mine = s.warp_sum[lane];
    int before = lane < warp ? mine : 0, all = mine;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        before += __shfl_xor_sync(0xffffffffu, before, o);
        all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    __syncthreads();
    total = all;
    return before + incl - x;
}

struct Tile {
    int row, token, tokens, pos, blocks;
};

__device__ Tile tile_at(const PrefillArgs &a, const int *tile_begin, int tile) {
    int lo = 0, hi = a.batch;  // the last row whose first tile is at or before this one
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (tile_begin[mid] <= tile)
            lo = mid;
        else
            hi = mid;
    }
    int first, n, len;
    prefill_row(a, lo, first, n, len);
    const int per = a.tile_rows / a.group, at = (tile - tile_begin[lo]) * per;
    Tile t;
    t.row = lo, t.token = first + at, t.tokens = min(per, n - at), t.pos = len - n + at;
    t.blocks = (max(t.pos + t.tokens, 0) + a.block_keys - 1) / a.block_keys;
    return t;
}

__global__ void __launch_bounds__(kThreads) prefill_plan_kernel(PrefillArgs a) {
    __shared__ Shared s;
    const int tid = threadIdx.x, per = a.tile_rows / a.group;
    pdl_trigger();
    pdl_wait();
    if (tid == 0) s.blocks = 0, s.longest = 0, s.slots = 0;
    if (tid < kBuckets) s.begin[tid] = 0;
    for (int i = tid; i < a.max_slots * a.num_kv_heads; i += kThreads) a.tickets[i] = 0;
    // ---- tiles a row, and their prefix
    int *tile_begin = a.batch <= kSharedRows ? s.tile_begin : a.tile_begin;
    int tiles = 0;
    for (int base = 0; base < a.batch; base += kThreads) {
        const int b = base + tid;
        int count = 0;
        if (b < a.batch) {
            int first, n, len;
            prefill_row(a, b, first, n, len);
            count = (n + per - 1) / per;
        }
        int total;
        const int before = exclusive_sum(s, count, total);
        if (b < a.batch) tile_begin[b] = tiles + before;
        tiles += total;
    }
    tiles = min(tiles, a.max_items - a.max_slots);  // sequences that overlap in q may have more: those are cut off
    __syncthreads();
    // ---- all blocks
    Tile own = {};  // the thread's first tile, looked up once
    if (tid < tiles) own = tile_at(a, tile_begin, tid);
    auto tile_of = [&](int i) { return i == tid ? own : tile_at(a, tile_begin, i); };
    unsigned long long sum = 0;
    for (int i = tid; i < tiles; i += kThreads) sum += tile_of(i).blocks;
    if (sum) atomicAdd(&s.blocks, sum);
    __syncthreads();
    int cap = 0x7fffffff;  // blocks a part has at most
    if (a.waves > 0) {
        const unsigned long long share = s.blocks * a.num_kv_heads / (unsigned(a.num_sms) * unsigned(a.waves)) + 1;
        cap = int(min(max(share, (unsigned long long)kPrefillMinBlocks), 0x7fffffffull));
    }
    auto parts_of = [&](int blocks) { return blocks > cap ? (blocks + cap - 1) / cap : 1; };
    // ---- lengths
    for (int i = tid; i < tiles; i += kThreads) {
        const int blocks = tile_of(i).blocks, parts = parts_of(blocks);
        atomicMax(&s.longest, (blocks + parts - 1) / parts);
    }
    __syncthreads();
    const int longest = s.longest;
    auto bucket_of = [&](int blocks) { return kBuckets - 1 - int(int64_t(blocks) * (kBuckets - 1) / max(longest, 1)); };
    for (int i = tid; i < tiles; i += kThreads) {
        const int blocks = tile_of(i).blocks, parts = parts_of(blocks);
        atomicAdd(&s.begin[bucket_of((blocks + parts - 1) / parts)], parts);
    }
    __syncthreads();
    int items;
    const int mine = tid < kBuckets ? s.begin[tid] : 0;
    const int before = exclusive_sum(s, mine, items);
    if (tid < kBuckets) s.begin[tid] = before;
    __syncthreads();
    // ---- the list
    for (int i = tid; i < tiles; i += kThreads) {
        const Tile t = tile_of(i);
        const int parts = parts_of(t.blocks);
        const int at = atomicAdd(&s.begin[bucket_of((t.blocks + parts - 1) / parts)], parts);
        const int slot = parts > 1 ? atomicAdd(&s.slots, parts) : 0;
        for (int p = 0; p < parts; p++) {
            PrefillItem x = {};
            x.row = t.row, x.token = t.token, x.tokens = t.tokens, x.pos = t.pos;
            x.block0 = int(int64_t(t.blocks) * p / parts), x.block1 = int(int64_t(t.blocks) * (p + 1) / parts);
            x.part = p, x.parts = parts, x.slot = slot;
            a.items[at + p] = x;
        }
    }
    if (tid == 0) a.plan->next = 0, a.plan->items = items;
}

}  // namespace

cudaError_t launch_prefill_plan(const PrefillArgs &a, cudaStream_t stream) {
    return launch_pdl(prefill_plan_kernel, dim3(1), dim3(kThreads), 0, stream, a);
}

}  // namespace qskv
