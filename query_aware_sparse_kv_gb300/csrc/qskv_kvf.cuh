// The 8-bit paged KV cache: block format, argument blocks and launchers of its
// kernels (kvf_cache.cu, kvf_decode.cu).
//
// Numbers in 8 bits.  The d dims x of one token and head, of its key or its
// value, are held as codes u and one power of two:
//     e = the smallest whole number with max |x| <= 448 2^e, clamped to
//         [-100, 119] (-100 where all are zero),  u = e4m3(x 2^-e)
// (e4m3: 4 exponent bits, 3 of fraction, largest 448; to nearest, ties to
// even; x 2^-e is exact), and stand for u 2^e.  A power of two instead of
// max |x| / 448 costs nothing in a floating-point format, and u 2^e is exact
// in bf16 and fp32: the cache can be read back, summarised or attended to in
// either with no further rounding.
//
// One (page, KV head) block is page_size / 16 parts of 16 tokens, in bytes:
//     [16][d] key codes | [8][d][2] value codes | [16] key e + 127 | [16] value e + 127
// so a part is one bulk copy, 16 (2 d + 2) bytes.  Keys lie token by token,
// values as pairs of tokens, dim by dim: the two codes that a register of the
// product weights x values wants side by side are side by side.  A key's
// 16-byte chunk c (16 dims) of token t is at place c ^ 4 (t % 2) of its row (d = 128;
// at c for d = 64), a pair's chunk c (8 dims) of pair p at c ^ f, f = (p & 1) | (p & 2) << 1
// (d = 128) or 2 (p % 4) (d = 64): the eight lanes that a shared-memory access
// of 16 bytes a lane serves at once then meet all banks.
#pragma once

#include "qskv_device.cuh"
#include "qskv_kvq.cuh"

namespace qskv {

constexpr int kKvfPartTokens = 16;
constexpr int kKvfLowExp = -100, kKvfHighExp = 119;

__host__ __device__ constexpr int kvf_part_bytes(int head_dim) { return kKvfPartTokens * (2 * head_dim + 2); }

// Place of a key's 16-byte chunk c in the row of token t, and of a value pair's in row p.
template <int D>
__device__ __forceinline__ int kvf_key_chunk(int c, int t) {
    return D == 128 ? c ^ ((t & 1) << 2) : c;
}
template <int D>
__device__ __forceinline__ int kvf_value_chunk(int c, int p) {
    return c ^ (D == 128 ? (p & 1) | (p & 2) << 1 : (p & 3) << 1);
}

// 2^(b - 127) of a stored power.
__device__ __forceinline__ float kvf_power(uint32_t b) { return __uint_as_float(b << 23); }

// Two e4m3 codes (the low half of w) as a pair of fp16, exactly.
__device__ __forceinline__ uint32_t kvf_half2(uint32_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(uint16_t(w)));
    return r;
}

struct KvfStoreArgs {
    const void *k, *v;     // append: [n][Hkv][d], rows k_stride / v_stride elements apart
    void *k_out, *v_out;   // gather: [n][Hkv][d]
    uint8_t *pool;
    const int32_t *slots;  // page * page_size + place; < 0: skipped
    uint32_t *flags;
    int64_t k_stride, v_stride;
    int32_t n_tokens, num_kv_heads, page_size, num_pool_pages;
};

struct KvfMetaArgs {
    const uint8_t *pool;
    const int32_t *page_ids, *valid_tokens;
    void *meta;            // [Npool][Hkv][2][d]
    uint32_t *flags;
    int32_t n_list, num_kv_heads, page_size, num_pool_pages;
};

cudaError_t launch_kvf_append(const KvfStoreArgs &a, int dtype, int head_dim, int num_sms, cudaStream_t stream);
cudaError_t launch_kvf_gather(const KvfStoreArgs &a, int dtype, int head_dim, int num_sms, cudaStream_t stream);
cudaError_t launch_kvf_meta(const KvfMetaArgs &a, int meta_dtype, int head_dim, int num_sms, cudaStream_t stream);
// The decode takes the argument block, the workspace and the grid of the 4-bit one; group_size is not used.
cudaError_t launch_kvf_decode(KvqDecodeArgs a, int head_dim, int num_sms, cudaStream_t stream);

}  // namespace qskv
