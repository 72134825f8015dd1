// Writing to, reading from and summarising the 4-bit paged KV cache (format:
// qskv_kvq.cuh).
//
// All three are bound by HBM: append reads 2 d elements a token and head and
// writes d + 8 NG bytes, gather does the reverse, the metadata build reads
// half a block and writes 2 d bf16.  A thread owns one 32-bit code word
// (8 dims), so a bf16 row is read (or written) 16 bytes a lane and the
// reductions over a group run over 4, 8 or 16 neighbouring lanes.
#include "qskv_internal.h"
#include "qskv_kvq.cuh"

namespace qskv {
namespace {

__device__ __forceinline__ float bits_f(uint32_t b) { return __uint_as_float(b); }

// x - m and the rounding error of that difference: their sum is exact.
__device__ __forceinline__ void exact_diff(float x, float m, float &d, float &err) {
    d = x - m;
    const float mm = d - x;
    err = (x - (d - mm)) + (-m - mm);
}

// bf16((mx - m) / 15) as a float, rounded once (to nearest even); 0 where the
// quotient is below 2^-100 or mx <= m.  The fp32 quotient only proposes the
// bf16 below; which neighbour is nearer is decided on the exact remainder
// against the midpoint (15 * midpoint has 13 bits, so the fma's product is exact).
__device__ __forceinline__ float kvq_scale(float mx, float m) {
    float d, err;
    exact_diff(mx, m, d, err);
    if (!(d >= 15.f * 7.888609052210118e-31f)) return 0.f;  // 2^-100
    const uint32_t lo = __float_as_uint(d * (1.f / 15.f)) & 0xffff0000u;
    const float rem = fmaf(-15.f, bits_f(lo | 0x8000u), d) + err;
    const bool up = rem > 0.f || (rem == 0.f && (lo & 0x10000u));
    return bits_f(up ? lo + 0x10000u : lo);
}

// rint((x - m) / s) clamped to [0, 15], ties to even, of the exact quotient.
// d * (1 / s) is within 3 ulp of it (15.5 * 3 * 2^-24 < 2^-18), so rounding
// it is right unless it lies within 2^-16 of a half; there the sign of the
// exact remainder against that half decides.
__device__ __forceinline__ uint32_t kvq_code(float x, float m, float s, float inv) {
    const float d = x - m;
    const float q = fminf(fmaxf(d * inv, -1.f), 17.f);
    float u = rintf(q);
    if (fabsf(q - u) > 0.5f - 1.52587890625e-5f) {
        const float k = floorf(q);
        float dd, err;
        exact_diff(x, m, dd, err);
        const float rem = fmaf(-(k + 0.5f), s, dd) + err;
        u = rem > 0.f ? k + 1.f : (rem < 0.f ? k : 2.f * rintf(0.5f * k + 0.25f));
    }
    u = fminf(fmaxf(u, 0.f), 15.f);
    return __float_as_uint(u + 8388608.f) & 15u;
}

template <bool BF16>
__device__ __forceinline__ void load8(const void *base, int64_t at, float (&x)[8]) {
    if constexpr (BF16) {
        const uint4 w = ldg_stream_v4(static_cast<const uint16_t *>(base) + at);
        const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; i++) {
            x[2 * i] = bf16_lo_to_float(r[i]);
            x[2 * i + 1] = bf16_hi_to_float(r[i]);
        }
    } else {
        const uint4 a = ldg_stream_v4(static_cast<const float *>(base) + at);
        const uint4 b = ldg_stream_v4(static_cast<const float *>(base) + at + 4);
        x[0] = bits_f(a.x), x[1] = bits_f(a.y), x[2] = bits_f(a.z), x[3] = bits_f(a.w);
        x[4] = bits_f(b.x), x[5] = bits_f(b.y), x[6] = bits_f(b.z), x[7] = bits_f(b.w);
    }
}

// Thread -> (token, key or value, head, code word), words fastest.
template <int D>
struct WordIndex {
    int token, which, head, word;
    __device__ __forceinline__ WordIndex(int64_t i, int heads) {
        constexpr int W = D / 8;
        word = int(i % W);
        int64_t r = i / W;
        head = int(r % heads);
        r /= heads;
        which = int(r & 1);
        token = int(r >> 1);
    }
};

template <bool BF16, int D>
__global__ void __launch_bounds__(256) kvq_append_kernel(KvqStoreArgs a) {
    constexpr int W = D / 8;
    pdl_trigger();
    pdl_wait();
    const int64_t total = int64_t(a.n_tokens) * 2 * a.num_kv_heads * W;
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    const bool in = i < total;
    const WordIndex<D> ix(in ? i : 0, a.num_kv_heads);
    const int slot = in ? a.slots[ix.token] : -1;
    const int page = slot / a.page_size;
    bool live = slot >= 0;
    if (live && page >= a.num_pool_pages) {
        live = false;
        if (ix.word == 0) raise_error(a.flags, kErrPageId);
    }
    float x[8];
    const int64_t row = int64_t(ix.token) * (ix.which ? a.v_stride : a.k_stride) + ix.head * D + ix.word * 8;
    load8<BF16>(ix.which ? a.v : a.k, row, x);
    float mn = x[0], mx = x[0];
#pragma unroll
    for (int k = 1; k < 8; k++) mn = fminf(mn, x[k]), mx = fmaxf(mx, x[k]);
    const int lanes = a.group_size / 8;  // lanes of one group: 4, 8 or 16
    for (int o = 1; o < lanes; o <<= 1) {
        mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    const uint32_t mbits = __bfloat16_as_ushort(__float2bfloat16_rn(mn));
    const float m = bits_f(mbits << 16);
    const float s = kvq_scale(mx, m);
    uint32_t word = 0;
    if (s > 0.f) {
        const float inv = 1.f / s;
#pragma unroll
        for (int k = 0; k < 8; k++) word |= kvq_code(x[k], m, s, inv) << (4 * k);
    }
    if (!live) return;
    const int P = a.page_size, t = slot % P, ng = D / a.group_size;
    uint32_t *block = a.pool + (int64_t(page) * a.num_kv_heads + ix.head) * kvq_block_words(D, P, ng);
    const int place = ix.which ? kvq_value_place<D>(ix.word, t) : kvq_key_place<D>(ix.word);
    block[ix.which * P * W + t * W + place] = word;
    if (ix.word % lanes == 0)
        block[2 * P * W + (ix.which * ng + ix.word / lanes) * P + t] = (__float_as_uint(s) >> 16) | (mbits << 16);
}

template <bool BF16, int D>
__global__ void __launch_bounds__(256) kvq_gather_kernel(KvqStoreArgs a) {
    constexpr int W = D / 8;
    pdl_trigger();
    pdl_wait();
    const int64_t total = int64_t(a.n_tokens) * 2 * a.num_kv_heads * W;
    const int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x;
    if (i >= total) return;
    const WordIndex<D> ix(i, a.num_kv_heads);
    const int slot = a.slots[ix.token];
    const int P = a.page_size, page = slot / P;
    uint32_t word = 0, par = 0;
    if (slot >= 0 && page >= a.num_pool_pages) {
        if (ix.word == 0) raise_error(a.flags, kErrPageId);
    } else if (slot >= 0) {
        const int t = slot % P, ng = D / a.group_size;
        const uint32_t *block = a.pool + (int64_t(page) * a.num_kv_heads + ix.head) * kvq_block_words(D, P, ng);
        const int place = ix.which ? kvq_value_place<D>(ix.word, t) : kvq_key_place<D>(ix.word);
        word = block[ix.which * P * W + t * W + place];
        par = block[2 * P * W + (ix.which * ng + ix.word * 8 / a.group_size) * P + t];
    }
    const float s = bf16_lo_to_float(par), m = bf16_hi_to_float(par);
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; k++) x[k] = fmaf(float((word >> (4 * k)) & 15u), s, m);
    const int64_t at = (int64_t(ix.token) * a.num_kv_heads + ix.head) * D + ix.word * 8;
    void *out = ix.which ? a.v_out : a.k_out;
    if constexpr (BF16) {
        uint4 w = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                             pack_bf16x2(x[6], x[7]));
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) = w;
    } else {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
        o[0] = make_float4(x[0], x[1], x[2], x[3]);
        o[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// fp32 -> bf16 bits, rounded towards -inf or +inf: the metadata stays a bound
// of every cached key after the rounding.
__device__ __forceinline__ uint32_t bf16_down(float x) {
    return __bfloat16_as_ushort(__float2bfloat16_rd(x));
}
__device__ __forceinline__ uint32_t bf16_up(float x) { return __bfloat16_as_ushort(__float2bfloat16_ru(x)); }

// One warp per (listed page, KV head): D / 8 lanes cover a token's code
// words, 32 / (D / 8) tokens at a time; lanes of the same word combine by
// shuffles.
template <bool BF16, int D>
__global__ void __launch_bounds__(256) kvq_meta_kernel(KvqMetaArgs a) {
    constexpr int W = D / 8, TP = 32 / W;
    pdl_trigger();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const int64_t tile = int64_t(blockIdx.x) * (blockDim.x >> 5) + (threadIdx.x >> 5);
    if (tile >= int64_t(a.n_list) * a.num_kv_heads) return;
    const int e = int(tile / a.num_kv_heads), g = int(tile % a.num_kv_heads);
    const int p = a.page_ids[e], valid = a.valid_tokens[e];
    if (p < 0) return;
    if (p >= a.num_pool_pages) {
        if (lane == 0) raise_error(a.flags, kErrPageId);
        return;
    }
    if (valid < 1 || valid > a.page_size) {
        if (lane == 0) raise_error(a.flags, kErrValid);
        return;
    }
    const int P = a.page_size, ng = D / a.group_size;
    const uint32_t *block = a.pool + (int64_t(p) * a.num_kv_heads + g) * kvq_block_words(D, P, ng);
    const int place = lane % W, t0 = lane / W, w = kvq_key_word<D>(place);
    const uint32_t *params = block + 2 * P * W + (w * 8 / a.group_size) * P;
    float mn[8], mx[8];
#pragma unroll
    for (int k = 0; k < 8; k++) mn[k] = INFINITY, mx[k] = -INFINITY;
    for (int t = t0; t < valid; t += TP) {
        const uint32_t word = block[t * W + place], par = params[t];
        const float s = bf16_lo_to_float(par), m = bf16_hi_to_float(par);
#pragma unroll
        for (int k = 0; k < 8; k++) {
            const float x = fmaf(float((word >> (4 * k)) & 15u), s, m);
            mn[k] = fminf(mn[k], x), mx[k] = fmaxf(mx[k], x);
        }
    }
#pragma unroll
    for (int o = W; o < 32; o <<= 1)
#pragma unroll
        for (int k = 0; k < 8; k++) {
            mn[k] = fminf(mn[k], __shfl_xor_sync(0xffffffffu, mn[k], o));
            mx[k] = fmaxf(mx[k], __shfl_xor_sync(0xffffffffu, mx[k], o));
        }
    if (t0 > 0) return;
    const int64_t at = (int64_t(p) * a.num_kv_heads + g) * 2 * D + w * 8;
    if constexpr (BF16) {
        uint32_t lo[4], hi[4];
#pragma unroll
        for (int k = 0; k < 4; k++) {
            lo[k] = bf16_down(mn[2 * k]) | (bf16_down(mn[2 * k + 1]) << 16);
            hi[k] = bf16_up(mx[2 * k]) | (bf16_up(mx[2 * k + 1]) << 16);
        }
        uint16_t *meta = static_cast<uint16_t *>(a.meta);
        *reinterpret_cast<uint4 *>(meta + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        *reinterpret_cast<uint4 *>(meta + at + D) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    } else {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.meta) + at);
        o[0] = make_float4(mn[0], mn[1], mn[2], mn[3]);
        o[1] = make_float4(mn[4], mn[5], mn[6], mn[7]);
        o = reinterpret_cast<float4 *>(static_cast<float *>(a.meta) + at + D);
        o[0] = make_float4(mx[0], mx[1], mx[2], mx[3]);
        o[1] = make_float4(mx[4], mx[5], mx[6], mx[7]);
    }
}

}  // namespace

#define KVQ_DISPATCH(kernel, bf16, d, grid, stream, args)                                            \
    ((d) == 128 ? ((bf16) ? launch_pdl(kernel<true, 128>, grid, dim3(256), 0, stream, args)          \
                          : launch_pdl(kernel<false, 128>, grid, dim3(256), 0, stream, args))        \
                : ((bf16) ? launch_pdl(kernel<true, 64>, grid, dim3(256), 0, stream, args)           \
                          : launch_pdl(kernel<false, 64>, grid, dim3(256), 0, stream, args)))

cudaError_t launch_kvq_append(const KvqStoreArgs &a, int dtype, int head_dim, cudaStream_t stream) {
    const int64_t n = int64_t(a.n_tokens) * 2 * a.num_kv_heads * (head_dim / 8);
    const dim3 grid(unsigned((n + 255) / 256));
    return KVQ_DISPATCH(kvq_append_kernel, dtype == kDtypeBf16, head_dim, grid, stream, a);
}

cudaError_t launch_kvq_gather(const KvqStoreArgs &a, int dtype, int head_dim, cudaStream_t stream) {
    const int64_t n = int64_t(a.n_tokens) * 2 * a.num_kv_heads * (head_dim / 8);
    const dim3 grid(unsigned((n + 255) / 256));
    return KVQ_DISPATCH(kvq_gather_kernel, dtype == kDtypeBf16, head_dim, grid, stream, a);
}

cudaError_t launch_kvq_meta(const KvqMetaArgs &a, int meta_dtype, int head_dim, cudaStream_t stream) {
    const int64_t n = int64_t(a.n_list) * a.num_kv_heads;
    const dim3 grid(unsigned((n + 7) / 8));
    return KVQ_DISPATCH(kvq_meta_kernel, meta_dtype == kDtypeBf16, head_dim, grid, stream, a);
}

}  // namespace qskv
