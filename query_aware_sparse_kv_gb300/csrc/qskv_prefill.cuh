// Causal attention of the newest tokens of every row of a batch (a prompt, or
// a chunk of one behind what is cached) over the row's pages: argument block,
// work items and launchers (prefill_plan.cu, prefill_fp32.cu, prefill_tc.cu).
//
// Row b holds seq_lens[b] tokens; the last n_b = cu_new[b + 1] - cu_new[b] of
// them are the queries cu_new[b].. of q.  Query i stands at pos = seq_len -
// n_b + i, and for each of its heads h (KV head g = h / G)
//     l_t = scale q_h . k_t,  t <= pos;   out = sum_t softmax(l)_t v_t,
//     lse = log sum_t exp(l_t).
//
// The G heads of a token that share a KV head are G neighbouring rows of one
// product: a tile is `tile_rows` such rows, tile_rows / G tokens of one
// sequence, so short prompts and single tokens fill their tiles as far as
// their heads go.  A work item is one tile, one KV head and a range of
// key blocks.  The lengths are on the device, so a kernel of one CTA
// (prefill_plan_kernel) makes the list of items; the CTAs of the attention
// take them by a counter, the longest first.  Where every row's queries fit one
// tile for sure (few tokens of few rows), there is no list: a CTA finds its own
// share from the lengths.
#pragma once

#include "qskv_device.cuh"
#include "qskv_internal.h"

namespace qskv {

// One tile's range of key blocks, for every KV head.
struct __align__(16) PrefillItem {
    int32_t row;        // sequence
    int32_t token;      // first query (a row of q)
    int32_t tokens;     // queries, 1 .. tile_rows / G
    int32_t pos;        // position of the first one (below 0: attends to nothing)
    int32_t block0, block1;
    int32_t part, parts;  // of the tile's ranges
    int32_t slot;       // parts > 1: where the partial results of part 0 lie
    int32_t pad[3];
};

struct PrefillPlan {
    uint32_t next;      // the counter the CTAs take items from
    uint32_t items;     // PrefillItems (each for every KV head)
    uint32_t pad[62];
};

struct PrefillArgs {
    const void *q;             // [n_tokens][Hq][D], rows q_stride elements apart
    const void *k_pool, *v_pool;
    const uint8_t *pool;       // 8-bit cache (kvf), else nullptr
    const int32_t *page_table, *seq_lens, *cu_new;
    void *out;                 // [n_tokens][Hq][D], q's type
    float *lse;                // [n_tokens][Hq] or nullptr
    uint32_t *flags;
    PrefillPlan *plan;
    int32_t *tile_begin;       // [batch + 1]: a sequence's first tile
    PrefillItem *items;
    uint32_t *tickets;         // [Hkv][max_slots]: parts of a tile that are done (counted at the slot of part 0);
                               // direct: [batch][Hkv], zero between calls
    float *part_o;             // [Hkv][max_slots][tile_rows][D]: a part's outputs
    float *part_lse;           // [Hkv][max_slots][tile_rows], log2 domain
    int64_t q_stride;
    int32_t n_tokens, batch, num_q_heads, num_kv_heads, group, page_size, max_pages, num_pool_pages;
    int32_t tile_rows, block_keys;  // rows of a tile, keys of a block
    int32_t max_items, max_slots;   // room of the lists
    int32_t waves;             // parts are made so that an SM has about this many (0: no tile is cut)
    int32_t num_sms;
    int32_t direct;            // no list: every row has one tile at most
    float scale_log2;          // sm_scale * log2(e)
};

// Queries of row b: their number and the first one, and the row's length, each clamped to what there is.
__device__ __forceinline__ void prefill_row(const PrefillArgs &a, int b, int &first, int &n, int &len) {
    const int lo = __ldg(a.cu_new + b), hi = __ldg(a.cu_new + b + 1), s = __ldg(a.seq_lens + b);
    const int cap = a.max_pages * a.page_size;
    first = min(max(lo, 0), a.n_tokens);
    n = min(max(hi, first), a.n_tokens) - first;
    len = min(max(s, 0), cap);
    if (lo != first || hi != first + n || s != len || n > len) raise_error(a.flags, kErrSeqLen);
}

// Which kernel a call takes, and the sizes of its work: tiles of kPrefillTcRows rows on the tensor cores (bf16 queries
// over bf16 or 8-bit caches), of kPrefillFp32Rows where
// fp32 is kept.
constexpr int kPrefillTcRows = 256, kPrefillTcKeys = 128;
constexpr int kPrefillWaves = 2;
constexpr int kPrefillMinBlocks = 8;   // a part has at least as many key blocks
constexpr int kPrefillDirectRows = 32; // rows of a batch that needs no list
constexpr int kPrefillFp32Rows = 64;
constexpr int prefill_fp32_keys(int head_dim) { return head_dim == 64 ? 64 : 32; }
constexpr int prefill_fp32_ctas(int num_sms) { return 2 * num_sms; }

cudaError_t launch_prefill_plan(const PrefillArgs &a, cudaStream_t stream);
// q: the queries as [n_tokens][Hq][D], boxes of 64 dims x G heads x 128 / G tokens; k, v: the pools' 16 x 64 boxes.
cudaError_t launch_prefill_tc(const PrefillArgs &a, const CUtensorMap *q, const CUtensorMap *k, const CUtensorMap *v,
                              int head_dim, cudaStream_t stream);
cudaError_t launch_prefill_fp32(const PrefillArgs &a, int q_dtype, int kv_dtype, int head_dim, cudaStream_t stream);

}  // namespace qskv
