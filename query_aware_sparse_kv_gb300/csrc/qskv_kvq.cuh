// The 4-bit paged KV cache: block format, argument blocks and launchers of
// its kernels (kvq_cache.cu, kvq_decode.cu) and of the page-table builder
// (tables.cu).
//
// Numbers in 4 bits.  A group of gs neighbouring dims of one token and head,
// x_0..x_{gs-1}, is held as a scale s, a minimum m (both bf16) and codes u:
//     m = bf16(min x),  s = bf16((max x - m) / 15)  (0 below 2^-100),
//     u = clamp(rint((x - m) / s), 0, 15)           (0 where s = 0)
// every rounding to nearest even of the exact value, so two implementations
// agree bit for bit; the group stands for m + s u.
//
// One (page, KV head) block of P tokens, NG = d / gs groups, W = d / 8
// 32-bit code words a token, in words:
//     [P][W] key codes | [P][W] value codes | [NG][P] key params | [NG][P] value params
// A code word holds dims 8w..8w+7, dim 8w+k in bits 4k..4k+3; a param word is
// s in the low half, m in the high half.  The whole block is contiguous, so
// one bulk copy brings a page of one head.  Words are placed in their rows so
// that the decode's matrix fragments come out of shared memory without bank
// conflicts: a key's word w = 4i + t at t * (d / 32) + i (lane t of a quad
// reads its words as one vector, the four lanes of a quad together cover 32
// neighbouring dims, hence one group, per word index i); a value's 16-byte
// chunk c = w / 4 of token t at chunk c ^ ((t / 2) % 4) (d = 128) or
// c ^ ((t / 4) % 2) (d = 64), which spreads the eight rows an ldmatrix reads
// over all banks.
#pragma once

#include "qskv_device.cuh"

namespace qskv {

__host__ __device__ constexpr int kvq_block_words(int head_dim, int page_size, int groups) {
    return page_size * head_dim / 4 + 2 * page_size * groups;
}

template <int D>
__device__ __forceinline__ int kvq_key_place(int w) {
    return (w & 3) * (D / 32) + (w >> 2);
}
// Inverse of kvq_key_place.
template <int D>
__device__ __forceinline__ int kvq_key_word(int place) {
    return (place % (D / 32)) * 4 + place / (D / 32);
}
template <int D>
__device__ __forceinline__ int kvq_value_place(int w, int token) {
    const int x = D == 128 ? (token >> 1) & 3 : (token >> 2) & 1;
    return (((w >> 2) ^ x) << 2) | (w & 3);
}

// Untiled bulk copy global -> shared (16-byte aligned, whole 16 bytes) that completes on `bar`.
__device__ __forceinline__ void bulk_load(void *dst, const void *src, uint32_t bytes, uint64_t *bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void bulk_load_hint(void *dst, const void *src, uint32_t bytes, uint64_t *bar,
                                               uint64_t policy) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
            smem_u32(dst)),
        "l"(src), "r"(bytes), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

struct KvqStoreArgs {
    const void *k, *v;         // append: [n][Hkv][d], rows k_stride / v_stride elements apart
    void *k_out, *v_out;       // gather: [n][Hkv][d]
    uint32_t *pool;
    const int32_t *slots;      // page * page_size + place; < 0: skipped
    uint32_t *flags;
    int64_t k_stride, v_stride;
    int32_t n_tokens, num_kv_heads, page_size, num_pool_pages, group_size;
};

struct KvqMetaArgs {
    const uint32_t *pool;
    const int32_t *page_ids, *valid_tokens;
    void *meta;                // [Npool][Hkv][2][d]
    uint32_t *flags;
    int32_t n_list, num_kv_heads, page_size, num_pool_pages, group_size;
};

struct KvqDecodeArgs {
    const void *q;
    const uint32_t *pool;
    const int32_t *page_table, *seq_lens;
    const int32_t *selected, *n_selected;  // selected: [rows][top_k], or nullptr (all pages)
    float *out, *lse;                      // lse may be nullptr
    uint32_t *flags;
    int32_t batch, num_q_heads, num_kv_heads, group, page_size, max_pages, num_pool_pages, top_k, group_size;
    int32_t q_is_bf16;
    float scale_log2;                      // sm_scale * log2(e)
    uint32_t *tickets;                     // [rows], zero between calls
    float *part_ml;                        // [2 CTAs][2][8]: reference and weight sum of a CTA's open rows
    float *part_o;                         // [2 CTAs][G][d]: their unnormalised outputs
    float *first_o;                        // [CTAs][warps][G][d]: a warp's piece of a row that ends in its range
    int32_t stages;                        // ring stages a warp (set by the launcher)
    int32_t row_ctas;                      // CTAs a row; 0: even split of all rows' units (set by the launcher)
    int32_t warp_units;                    // places a row where rows go to warps whole, 0 elsewhere (set by the launcher)
    int32_t evict_first;                   // 1: the pages are read with L2's evict-first policy (set by the launcher)
};

struct TablesArgs {
    const int32_t *seq_lens, *new_lens, *free_pages;
    int32_t *page_table, *seq_lens_out, *cu_new, *slot_map, *positions, *touched_ids, *touched_valid, *counts;
    uint32_t *flags;
    int32_t batch, page_size, max_pages, num_pool_pages, n_free, max_tokens, max_touched;
};

cudaError_t launch_kvq_append(const KvqStoreArgs &a, int dtype, int head_dim, cudaStream_t stream);
cudaError_t launch_kvq_gather(const KvqStoreArgs &a, int dtype, int head_dim, cudaStream_t stream);
cudaError_t launch_kvq_meta(const KvqMetaArgs &a, int meta_dtype, int head_dim, int num_sms, cudaStream_t stream);
// Largest decode grid on a device with num_sms SMs, and its warps a CTA (for the workspace).
int kvq_decode_ctas(int num_sms);
int kvq_decode_warps();
cudaError_t launch_kvq_decode_page32(KvqDecodeArgs a, int head_dim, int num_sms, cudaStream_t stream);
cudaError_t launch_kvq_decode(KvqDecodeArgs a, int head_dim, int num_sms, cudaStream_t stream);
// Requests that one CTA of the page-table builder scans in shared memory (three prefixes, below 48 KB).
constexpr int kTablesScanRequests = 4032;
// scratch: 3 (batch + 1) int32, used beyond kTablesScanRequests requests.
cudaError_t launch_extend_tables(const TablesArgs &a, int32_t *scratch, int num_sms, cudaStream_t stream);

}  // namespace qskv
