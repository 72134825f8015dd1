// Writing to, reading from and summarising the 8-bit paged KV cache (format:
// qskv_kvf.cuh).
//
// All three move bytes: append reads 2 d elements a token and head and writes
// 2 d + 2 bytes, gather does the reverse, the metadata build reads the keys'
// d + 1 bytes a token and writes 2 d elements a page.  A thread of append and
// gather owns 8 dims, so a bf16 row is read (or written) 16 bytes a lane and a
// token's largest magnitude is found over d / 8 neighbouring lanes.  One GB300:
// 32768 tokens x 8 heads of 128 dims (bf16) stored and read back in 67.5 us
// (6.0 TB/s of 6.78 copied), 131072 read back in 119.8 us (6.7 TB/s), the
// metadata of 36864 pages x 8 heads made in 131.5 us (5.8 TB/s): HBM bounds them.
#include "qskv_internal.h"
#include "qskv_kvf.cuh"

#include <cuda_fp16.h>

namespace qskv {
namespace {

constexpr int kCacheThreads = 256;

// The 8 values of a thread as loaded, and as floats.
template <bool BF16>
struct Raw8 {
    uint4 a, b;
    __device__ __forceinline__ void load(const void *base, int64_t at) {
        if constexpr (BF16) {
            a = ldg_stream_v4(static_cast<const uint16_t *>(base) + at);
        } else {
            a = ldg_stream_v4(static_cast<const float *>(base) + at);
            b = ldg_stream_v4(static_cast<const float *>(base) + at + 4);
        }
    }
    // Largest magnitude, as the bits of a float.
    __device__ __forceinline__ uint32_t top() const {
        constexpr uint32_t abs2 = 0x7fff7fffu, abs1 = 0x7fffffffu;
        if constexpr (BF16) {  // magnitudes order as their bits do
            const uint32_t r = __vmaxu2(__vmaxu2(a.x & abs2, a.y & abs2), __vmaxu2(a.z & abs2, a.w & abs2));
            return max(r & 0xffff0000u, r << 16);
        } else {
            return max(max(max(a.x & abs1, a.y & abs1), max(a.z & abs1, a.w & abs1)),
                       max(max(b.x & abs1, b.y & abs1), max(b.z & abs1, b.w & abs1)));
        }
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const {
        if constexpr (BF16) {
            const uint32_t r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; i++) x[2 * i] = bf16_lo_to_float(r[i]), x[2 * i + 1] = bf16_hi_to_float(r[i]);
        } else {
            const uint32_t r[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 8; i++) x[i] = __uint_as_float(r[i]);
        }
    }
};

// e + 127 for the largest magnitude `top` (bits): 448 is 1.75 2^8.
__device__ __forceinline__ int kvf_exponent(uint32_t top) {
    const int e = int(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u);
    return min(max(e, 127 + kKvfLowExp), 127 + kKvfHighExp);
}

// Four codes of x times `up` (a power of two), byte i from x[i].
__device__ __forceinline__ uint32_t kvf_codes(const float *x, float up) {
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * up), "f"(x[0] * up));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * up), "f"(x[2] * up));
    return uint32_t(lo) | uint32_t(hi) << 16;
}

// First byte of the part that a slot lies in, for one head.
template <int D>
__device__ __forceinline__ int64_t part_at(int slot, int page_size, int num_kv_heads, int head) {
    const int shift = page_size == 16 ? 4 : 5, parts = page_size >> 4;  // (parts of a pool are fewer than 2^27)
    return int64_t(((slot >> shift) * num_kv_heads + head) * parts + ((slot & (page_size - 1)) >> 4)) * kvf_part_bytes(D);
}

// A thread takes 8 dims, of the key and of the value, of ITEMS tokens that
// follow one another.  A run of tokens goes to slots in order, so that two of
// them are a pair of the cache, whose value codes leave as one 16-byte store:
// a pair's second token is taken with its first, by whichever thread that is
// (so a thread may have one token more, or one less).  A token alone in its
// pair is stored byte by byte.
template <bool BF16, int D, int ITEMS>
__global__ void __launch_bounds__(kCacheThreads) kvf_append_kernel(KvfStoreArgs a) {
    constexpr int W = D / 8, TPB = kCacheThreads / W, N = ITEMS + 1;
    pdl_trigger();
    pdl_wait();
    const int chunk = blockIdx.x / a.num_kv_heads, head = blockIdx.x % a.num_kv_heads;
    const int w = threadIdx.x % W, token0 = (chunk * TPB + threadIdx.x / W) * ITEMS;
    const int64_t col = head * D + w * 8;
    const int slots = a.num_pool_pages * a.page_size;  // below 2^31
    Raw8<BF16> k[N], v[N];
    int slot[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int t = min(token0 + i, a.n_tokens - 1);
        slot[i] = token0 + i < a.n_tokens ? __ldg(a.slots + t) : -1;
        if (i < ITEMS) k[i].load(a.k, t * a.k_stride + col), v[i].load(a.v, t * a.v_stride + col);
    }
    const int before = token0 > 0 && token0 < a.n_tokens ? __ldg(a.slots + token0 - 1) : -1;
    const bool second = (slot[0] & 1) && before >= 0 && before + 1 == slot[0];  // taken with the token before
    const bool more = slot[ITEMS - 1] >= 0 && (slot[ITEMS] & 1) && slot[ITEMS - 1] + 1 == slot[ITEMS];
    if (more) {
        k[ITEMS].load(a.k, (token0 + ITEMS) * a.k_stride + col);
        v[ITEMS].load(a.v, (token0 + ITEMS) * a.v_stride + col);
    } else {
        slot[ITEMS] = -1;
        k[ITEMS] = k[0], v[ITEMS] = v[0];
    }
    if (second) slot[0] = -1;
    uint2 codes[N];
#pragma unroll
    for (int i = 0; i < N; i++) {
        uint32_t top_k = k[i].top(), top_v = v[i].top();
        if constexpr (BF16) {  // both in one word: magnitudes of 16 bits
            uint32_t r = (top_k & 0xffff0000u) | top_v >> 16;
#pragma unroll
            for (int o = 1; o < W; o <<= 1) r = __vmaxu2(r, __shfl_xor_sync(0xffffffffu, r, o));
            top_k = r & 0xffff0000u, top_v = r << 16;
        } else {
#pragma unroll
            for (int o = 1; o < W; o <<= 1) {
                top_k = max(top_k, __shfl_xor_sync(0xffffffffu, top_k, o));
                top_v = max(top_v, __shfl_xor_sync(0xffffffffu, top_v, o));
            }
        }
        const int ek = kvf_exponent(top_k), ev = kvf_exponent(top_v);
        float x[8];
        k[i].floats(x);
        const float up_k = kvf_power(254 - ek), up_v = kvf_power(254 - ev);
        const uint2 key = make_uint2(kvf_codes(x, up_k), kvf_codes(x + 4, up_k));
        v[i].floats(x);
        codes[i] = make_uint2(kvf_codes(x, up_v), kvf_codes(x + 4, up_v));
        if (slot[i] >= slots) {
            if (w == 0) raise_error(a.flags, kErrPageId);
            slot[i] = -1;
        }
        if (slot[i] < 0) continue;
        uint8_t *part = a.pool + part_at<D>(slot[i], a.page_size, a.num_kv_heads, head);
        const int t = slot[i] & 15;
        if (w == 0) part[32 * D + t] = uint8_t(ek), part[32 * D + 16 + t] = uint8_t(ev);
        *reinterpret_cast<uint2 *>(part + t * D + kvf_key_chunk<D>(w >> 1, t) * 16 + (w & 1) * 8) = key;
    }
    bool taken = false;  // the token before this one was stored together with it
#pragma unroll
    for (int i = 0; i < N; i++) {
        if (slot[i] < 0 || taken) {
            taken = false;
            continue;
        }
        const int t = slot[i] & 15, p = t >> 1;
        uint8_t *to = a.pool + part_at<D>(slot[i], a.page_size, a.num_kv_heads, head) + 16 * D + p * 2 * D +
                      kvf_value_chunk<D>(w, p) * 16;
        if (i + 1 < N && !(t & 1) && slot[i + 1 < N ? i + 1 : i] == slot[i] + 1) {
            const uint2 x = codes[i], y = codes[i + 1 < N ? i + 1 : i];
            *reinterpret_cast<uint4 *>(to) = make_uint4(__byte_perm(x.x, y.x, 0x5140), __byte_perm(x.x, y.x, 0x7362),
                                                        __byte_perm(x.y, y.y, 0x5140), __byte_perm(x.y, y.y, 0x7362));
            taken = true;
        } else {
#pragma unroll
            for (int b = 0; b < 4; b++) {
                to[2 * b + (t & 1)] = uint8_t(codes[i].x >> (8 * b));
                to[8 + 2 * b + (t & 1)] = uint8_t(codes[i].y >> (8 * b));
            }
        }
    }
}

// The values u 2^e of 8 codes.
__device__ __forceinline__ void kvf_values(uint2 codes, float power, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t h = kvf_half2((i & 2 ? codes.y : codes.x) >> (16 * (i & 1)));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        x[2 * i] = f.x * power, x[2 * i + 1] = f.y * power;
    }
}

template <bool BF16>
__device__ __forceinline__ void write_values(void *out, int64_t at, uint2 codes, float power) {
    float x[8];
    kvf_values(codes, power, x);
    if constexpr (BF16) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) =
            make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
    } else {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// A thread 8 dims of the key and of the value of ITEMS tokens that follow one another.
template <bool BF16, int D, int ITEMS>
__global__ void __launch_bounds__(kCacheThreads) kvf_gather_kernel(KvfStoreArgs a) {
    constexpr int W = D / 8, TPB = kCacheThreads / W;
    pdl_trigger();
    pdl_wait();
    const int chunk = blockIdx.x / a.num_kv_heads, head = blockIdx.x % a.num_kv_heads;
    const int w = threadIdx.x % W, token0 = (chunk * TPB + threadIdx.x / W) * ITEMS;
    const int slots = a.num_pool_pages * a.page_size;  // below 2^31
    int slot[ITEMS];
    uint2 keys[ITEMS];
    uint4 pairs[ITEMS];
    uint32_t ek[ITEMS], ev[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; i++) slot[i] = token0 + i < a.n_tokens ? __ldg(a.slots + token0 + i) : -1;
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        keys[i] = make_uint2(0, 0), pairs[i] = make_uint4(0, 0, 0, 0), ek[i] = ev[i] = 127;
        if (slot[i] >= slots) {
            if (w == 0) raise_error(a.flags, kErrPageId);
            continue;
        }
        if (slot[i] < 0) continue;
        const uint8_t *part = a.pool + part_at<D>(slot[i], a.page_size, a.num_kv_heads, head);
        const int t = slot[i] & 15, p = t >> 1;
        ek[i] = __ldg(part + 32 * D + t), ev[i] = __ldg(part + 32 * D + 16 + t);
        keys[i] = __ldg(reinterpret_cast<const uint2 *>(part + t * D + kvf_key_chunk<D>(w >> 1, t) * 16 + (w & 1) * 8));
        pairs[i] = __ldg(reinterpret_cast<const uint4 *>(part + 16 * D + p * 2 * D + kvf_value_chunk<D>(w, p) * 16));
    }
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        if (token0 + i >= a.n_tokens) break;
        const int64_t at = (int64_t(token0 + i) * a.num_kv_heads + head) * D + w * 8;
        const uint32_t pick = slot[i] & 1 ? 0x7531 : 0x6420;
        write_values<BF16>(a.k_out, at, keys[i], kvf_power(ek[i]));
        write_values<BF16>(a.v_out, at, make_uint2(__byte_perm(pairs[i].x, pairs[i].y, pick), __byte_perm(pairs[i].z, pairs[i].w, pick)),
                           kvf_power(ev[i]));
    }
}

__device__ __forceinline__ uint32_t half2_mul(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t half2_min(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("min.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t half2_max(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A lane group of D / 4 lanes takes (listed page, KV head) tiles, a lane four
// dims of all their tokens: nothing is combined across lanes, and the loads of
// 16 tokens are in flight together.  The values of a part are compared as
// pairs of fp16 less its largest power, which is exact unless its powers are
// more than 14 apart (then as floats).  The page of the next tile is looked up
// while one is summarised.
constexpr int kMetaThreads = 128, kMetaCtas = 8;  // CTAs an SM: 36864 pages 131 us, with 10 of them 153 (spills)

template <bool BF16, int D>
__global__ void __launch_bounds__(kMetaThreads, kMetaCtas) kvf_meta_kernel(KvfMetaArgs a) {
    constexpr int L = D / 4;
    pdl_trigger();
    pdl_wait();
    const int w = threadIdx.x % L, P = a.page_size;
    const uint32_t group = L == 32 ? 0xffffffffu : 0xffffu << (threadIdx.x & 16);  // lanes of this tile
    const int64_t tiles = int64_t(a.n_list) * a.num_kv_heads, stride = int64_t(gridDim.x) * (kMetaThreads / L);
    int64_t tile = (int64_t(blockIdx.x) * kMetaThreads + threadIdx.x) / L;
    int p = -1, valid = 0;
    auto look_up = [&] {
        if (tile >= tiles) return;
        const int e = int(tile / a.num_kv_heads);
        p = __ldg(a.page_ids + e), valid = __ldg(a.valid_tokens + e);
    };
    look_up();
    while (tile < tiles) {
        const int64_t row = int64_t(p) * a.num_kv_heads + tile % a.num_kv_heads;
        const int page = p, n = valid;
        tile += stride;
        look_up();
        if (page < 0) continue;
        if (page >= a.num_pool_pages || n < 1 || n > P) {
            if (w == 0) raise_error(a.flags, page >= a.num_pool_pages ? kErrPageId : kErrValid);
            continue;
        }
        const uint8_t *block = a.pool + row * (P >> 4) * kvf_part_bytes(D);
        float mn[4], mx[4];
#pragma unroll
        for (int k = 0; k < 4; k++) mn[k] = INFINITY, mx[k] = -INFINITY;
        for (int c = 0; c < n; c += 16) {
            const uint8_t *part = block + (c >> 4) * kvf_part_bytes(D);
            // lane t (of 16) holds the power of token t; a token past the end stands for the last one
            const int last = min(n - c, 16) - 1, own = min(int(threadIdx.x & 15), last);
            const uint32_t stored = __ldg(part + 32 * D + own);
            const uint8_t *even = part + kvf_key_chunk<D>(w >> 2, 0) * 16 + (w & 3) * 4;
            const uint8_t *odd = part + kvf_key_chunk<D>(w >> 2, 1) * 16 + (w & 3) * 4;
            uint32_t codes[16];
            if (last == 15) {
#pragma unroll
                for (int t = 0; t < 16; t++) codes[t] = __ldg(reinterpret_cast<const uint32_t *>((t & 1 ? odd : even) + t * D));
            } else {
#pragma unroll
                for (int t = 0; t < 16; t++) {
                    const int u = min(t, last);
                    codes[t] = __ldg(reinterpret_cast<const uint32_t *>((u & 1 ? odd : even) + u * D));
                }
            }
            const uint32_t top = __reduce_max_sync(group, stored);
            if (__reduce_min_sync(group, stored) + 14 >= top) {
                // 2^(e - largest e) of the part is 2^-14 or more, so a code (a multiple of 2^-9) times it is a fp16 number
                const uint32_t mine = (15 + stored - top) << 10, power = mine | mine << 16;
                uint32_t lo[2] = {0x7c007c00u, 0x7c007c00u}, hi[2] = {0xfc00fc00u, 0xfc00fc00u};
#pragma unroll
                for (int t = 0; t < 16; t++) {
                    const uint32_t f = __shfl_sync(group, power, t, 16);
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t x = half2_mul(kvf_half2(codes[t] >> (16 * h)), f);
                        lo[h] = half2_min(lo[h], x), hi[h] = half2_max(hi[h], x);
                    }
                }
                const float unit = kvf_power(top);
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&lo[h]));
                    const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&hi[h]));
                    mn[2 * h] = fminf(mn[2 * h], x.x * unit), mn[2 * h + 1] = fminf(mn[2 * h + 1], x.y * unit);
                    mx[2 * h] = fmaxf(mx[2 * h], y.x * unit), mx[2 * h + 1] = fmaxf(mx[2 * h + 1], y.y * unit);
                }
            } else {
#pragma unroll
                for (int t = 0; t < 16; t++) {
                    const float power = kvf_power(__shfl_sync(group, stored, t, 16));
#pragma unroll
                    for (int h = 0; h < 2; h++) {
                        const uint32_t x2 = kvf_half2(codes[t] >> (16 * h));
                        const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&x2));
                        mn[2 * h] = fminf(mn[2 * h], x.x * power), mn[2 * h + 1] = fminf(mn[2 * h + 1], x.y * power);
                        mx[2 * h] = fmaxf(mx[2 * h], x.x * power), mx[2 * h + 1] = fmaxf(mx[2 * h + 1], x.y * power);
                    }
                }
            }
        }
        const int64_t to = row * 2 * D + w * 4;
        if constexpr (BF16) {  // exact: a value has 4 significant bits
            uint16_t *o = static_cast<uint16_t *>(a.meta) + to;
            *reinterpret_cast<uint2 *>(o) = make_uint2(pack_bf16x2(mn[0], mn[1]), pack_bf16x2(mn[2], mn[3]));
            *reinterpret_cast<uint2 *>(o + D) = make_uint2(pack_bf16x2(mx[0], mx[1]), pack_bf16x2(mx[2], mx[3]));
        } else {
            float *o = static_cast<float *>(a.meta) + to;
            *reinterpret_cast<float4 *>(o) = make_float4(mn[0], mn[1], mn[2], mn[3]);
            *reinterpret_cast<float4 *>(o + D) = make_float4(mx[0], mx[1], mx[2], mx[3]);
        }
    }
}

// CTAs of `items` tokens a thread.
int64_t token_ctas(const KvfStoreArgs &a, int head_dim, int items) {
    const int per_cta = kCacheThreads / (head_dim / 8) * items;
    return (int64_t(a.n_tokens) + per_cta - 1) / per_cta * a.num_kv_heads;
}
// Tokens a thread: with 2, 4 and 8 32768 tokens stored and read back take 70.8, 70.7 and 82.7 us, 131072 read back 119.8,
// 132.4 and 142.1.  One a thread where several would leave SMs without a CTA: with one and with several, 32 tokens x 8 heads
// stored and read back take 4.4 and 6.1 us, 600 4.9 and 5.3, 1200 7.2 and 6.1.
constexpr int kAppendItems = 4, kGatherItems = 2;

}  // namespace

#define KVF_TOKENS(kernel, kItems)                                                                              \
    const bool bf16 = dtype == kDtypeBf16, many = token_ctas(a, head_dim, kItems) >= num_sms;                   \
    const dim3 grid(unsigned(token_ctas(a, head_dim, many ? kItems : 1))), block(kCacheThreads);                \
    if (head_dim == 128) {                                                                                      \
        if (many) return bf16 ? launch_pdl(kernel<true, 128, kItems>, grid, block, 0, stream, a)                \
                              : launch_pdl(kernel<false, 128, kItems>, grid, block, 0, stream, a);              \
        return bf16 ? launch_pdl(kernel<true, 128, 1>, grid, block, 0, stream, a)                               \
                    : launch_pdl(kernel<false, 128, 1>, grid, block, 0, stream, a);                             \
    }                                                                                                           \
    if (many) return bf16 ? launch_pdl(kernel<true, 64, kItems>, grid, block, 0, stream, a)                     \
                          : launch_pdl(kernel<false, 64, kItems>, grid, block, 0, stream, a);                   \
    return bf16 ? launch_pdl(kernel<true, 64, 1>, grid, block, 0, stream, a)                                    \
                : launch_pdl(kernel<false, 64, 1>, grid, block, 0, stream, a);

cudaError_t launch_kvf_append(const KvfStoreArgs &a, int dtype, int head_dim, int num_sms, cudaStream_t stream) {
    KVF_TOKENS(kvf_append_kernel, kAppendItems)
}

cudaError_t launch_kvf_gather(const KvfStoreArgs &a, int dtype, int head_dim, int num_sms, cudaStream_t stream) {
    KVF_TOKENS(kvf_gather_kernel, kGatherItems)
}

cudaError_t launch_kvf_meta(const KvfMetaArgs &a, int meta_dtype, int head_dim, int num_sms, cudaStream_t stream) {
    const bool bf16 = meta_dtype == kDtypeBf16;
    const int per_cta = kMetaThreads / (head_dim / 4);
    const int64_t tiles = int64_t(a.n_list) * a.num_kv_heads, ctas = (tiles + per_cta - 1) / per_cta;
    const dim3 grid(unsigned(ctas < kMetaCtas * num_sms ? ctas : kMetaCtas * num_sms)), block(kMetaThreads);
    if (head_dim == 128)
        return bf16 ? launch_pdl(kvf_meta_kernel<true, 128>, grid, block, 0, stream, a)
                    : launch_pdl(kvf_meta_kernel<false, 128>, grid, block, 0, stream, a);
    return bf16 ? launch_pdl(kvf_meta_kernel<true, 64>, grid, block, 0, stream, a)
                : launch_pdl(kvf_meta_kernel<false, 64>, grid, block, 0, stream, a);
}

}  // namespace qskv
