// Writing to, reading from and summarising the 4-bit paged KV cache (format:
// qskv_kvq.cuh).
//
// Append reads 2 d elements a token and head and writes d + 8 NG bytes, gather
// does the reverse, the metadata build reads half a block and writes 2 d bf16.
// A thread owns one 32-bit code word (8 dims), so a bf16 row is read (or
// written) 16 bytes a lane and the reductions over a group run over 4, 8 or 16
// neighbouring lanes.  One GB300: 131072 tokens x 8 heads of 128 dims read
// back to bf16 in 118 us (6.0 TB/s of 6.76 copied: HBM); 32768 tokens stored
// in 47 us (3.7 TB/s) and the metadata of 36864 pages x 8 heads made in 115 us
// (4.3 TB/s), at 74 and 80 % of the issue slots with the ALU pipe at 73 %:
// bound by the instructions a code costs, 20 in the append (about half of them
// a word's or a group's: scale, shuffles, smallest magnitude, addresses).
#include <cuda_fp16.h>

#include "qskv_internal.h"
#include "qskv_kvq.cuh"

namespace qskv {
namespace {

__device__ __forceinline__ float bits_f(uint32_t b) { return __uint_as_float(b); }

// Two floats in one 64-bit register, an instruction for both.
struct Float2 {
    uint64_t r;
    __device__ __forceinline__ Float2() {}
    __device__ __forceinline__ Float2(float a, float b) { asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b)); }
    __device__ __forceinline__ void get(float &a, float &b) const {
        asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
    }
};
__device__ __forceinline__ Float2 operator+(Float2 a, Float2 b) {
    Float2 c;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(c.r) : "l"(a.r), "l"(b.r));
    return c;
}
__device__ __forceinline__ Float2 operator*(Float2 a, Float2 b) {
    Float2 c;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(c.r) : "l"(a.r), "l"(b.r));
    return c;
}
__device__ __forceinline__ Float2 fma(Float2 a, Float2 b, Float2 c) {
    Float2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.r) : "l"(a.r), "l"(b.r), "l"(c.r));
    return d;
}

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

// Code word of 8 values: rint((x - m) / s) clamped to [0, 15], ties to even,
// of the exact quotients.  Adding d * (1 / s) to 1.5 2^23 rounds to a
// candidate u within one of the right one; d - u s is exact and says whether
// it is: below s / 2 in magnitude it is.  A word with a remainder at s / 2
// (a tie, or d itself rounded: 2^-19 s covers that) is looked at once more,
// value by value, with the rounding error of d.  The candidates' bits are the
// codes plus a constant; `acc * 16 + bits` packs them and the constants' sum
// is taken off at the end.  CLAMP: m may lie above the smallest value (fp32
// inputs, whose minimum is rounded); a bf16 minimum is exact, and then the
// quotients are 0 to 15.06 and round into range by themselves.
template <bool CLAMP>
__device__ __forceinline__ uint32_t kvq_word(const float (&x)[8], float m, float s) {
    constexpr float magic = 12582912.f;  // 1.5 * 2^23, bits 0x4b400000
    constexpr uint32_t sum16 = 0x11111111u * 0x4b400000u;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    uint32_t acc = 0;
    float off = 0.f;
    const Float2 inv2(inv, inv), s2(s, s), minus_m(-m, -m), magic2(magic, magic), minus1(-1.f, -1.f);
#pragma unroll
    for (int k = 6; k >= 0; k -= 2) {
        const Float2 d = Float2(x[k], x[k + 1]) + minus_m, t = fma(d, inv2, magic2);
        const Float2 r = fma(fma(t, minus1, magic2), s2, d);
        float a, b, ra, rb;
        t.get(a, b), r.get(ra, rb);
        off = fmaxf(fmaxf(fabsf(ra), fabsf(rb)), off);
        if (CLAMP) a = fminf(fmaxf(a, magic), magic + 15.f), b = fminf(fmaxf(b, magic), magic + 15.f);
        acc = (acc * 16 + __float_as_uint(b)) * 16 + __float_as_uint(a);
    }
    const float half = 0.5f * s;
    if (off > half - s * 1.9073486328125e-6f) {
        acc = 0;
#pragma unroll
        for (int k = 7; k >= 0; k--) {
            float d, err;
            exact_diff(x[k], m, d, err);
            float t = fmaf(d, inv, magic);
            const float r = fmaf(magic - t, s, d);
            const float over = (fabsf(r) - half) + (r > 0.f ? err : -err);
            if (over > 0.f || (over == 0.f && (__float_as_uint(t) & 1u))) t += r > 0.f ? 1.f : -1.f;
            if (CLAMP) t = fminf(fmaxf(t, magic), magic + 15.f);
            acc = acc * 16 + __float_as_uint(t);
        }
    }
    return acc - sum16;
}

// The same for bf16 values with an exact minimum: the quotients are 0 to 15.06,
// nothing to clamp, and unless a value is tiny against s they are rational
// numbers with few bits: rounded to fp32 correctly (one residual step does
// that), none but an exact tie lands on a tie, and adding 1.5 2^23 then rounds
// it to even.  A quotient is (whole multiple of the smallest unit of x and m)
// / s with an 8-bit s, so one that is no tie is at least that unit / 2^9 s
// away from one; with x and m zero or above s / 2^10 that is 2^-19 or more,
// beyond fp32's rounding at 15.
__device__ __forceinline__ uint32_t kvq_word_plain(const float (&x)[8], float m, float s) {
    constexpr float magic = 12582912.f;
    constexpr uint32_t sum16 = 0x11111111u * 0x4b400000u;
    float inv;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    const Float2 inv2(inv, inv), minus_s(-s, -s), minus_m(-m, -m), magic2(magic, magic);
    uint32_t acc = 0;
#pragma unroll
    for (int k = 6; k >= 0; k -= 2) {
        const Float2 d = Float2(x[k], x[k + 1]) + minus_m, q0 = d * inv2, q = fma(fma(q0, minus_s, d), inv2, q0);
        float a, b;
        (q + magic2).get(a, b);
        acc = (acc * 16 + __float_as_uint(b)) * 16 + __float_as_uint(a);
    }
    return acc - sum16;
}

// The 8 raw 16-bit pairs or the 8 floats of a word as loaded.
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
    // Smallest magnitude among the word's values and m (bf16).
    __device__ __forceinline__ float smallest(float m) const {
        constexpr uint32_t abs2 = 0x7fff7fffu;
        uint32_t r = Bf16Ops::vmin(Bf16Ops::vmin(a.x & abs2, a.y & abs2), Bf16Ops::vmin(a.z & abs2, a.w & abs2));
        return fminf(fminf(bf16_lo_to_float(r), bf16_hi_to_float(r)), fabsf(m));
    }
    __device__ __forceinline__ void floats(float (&x)[8]) const {
        if constexpr (BF16) {
            const uint32_t r[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
            for (int i = 0; i < 4; i++) x[2 * i] = bf16_lo_to_float(r[i]), x[2 * i + 1] = bf16_hi_to_float(r[i]);
        } else {
            x[0] = bits_f(a.x), x[1] = bits_f(a.y), x[2] = bits_f(a.z), x[3] = bits_f(a.w);
            x[4] = bits_f(b.x), x[5] = bits_f(b.y), x[6] = bits_f(b.z), x[7] = bits_f(b.w);
        }
    }
};

// Smallest and largest value of the group a lane's word belongs to; LANES
// neighbouring lanes hold the group.
template <bool BF16, int LANES>
__device__ __forceinline__ void group_range(const Raw8<BF16> &raw, const float (&x)[8], float &mn, float &mx) {
    if constexpr (BF16) {
        // as pairs of bf16, exactly: (min, -max) of the word, then one shuffle a round for both
        const uint32_t lo = Bf16Ops::vmin(Bf16Ops::vmin(raw.a.x, raw.a.y), Bf16Ops::vmin(raw.a.z, raw.a.w));
        const uint32_t hi = Bf16Ops::vmax(Bf16Ops::vmax(raw.a.x, raw.a.y), Bf16Ops::vmax(raw.a.z, raw.a.w)) ^ 0x80008000u;
        uint32_t r = Bf16Ops::vmin(__byte_perm(lo, hi, 0x5410), __byte_perm(lo, hi, 0x7632));
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) r = Bf16Ops::vmin(r, __shfl_xor_sync(0xffffffffu, r, o));
        mn = bf16_lo_to_float(r), mx = bf16_hi_to_float(r ^ 0x80000000u);
    } else {
        mn = x[0], mx = x[0];
#pragma unroll
        for (int k = 1; k < 8; k++) mn = fminf(mn, x[k]), mx = fmaxf(mx, x[k]);
#pragma unroll
        for (int o = 1; o < LANES; o <<= 1) {
            mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
    }
}

// A CTA takes neighbouring tokens of one head's keys or values (the heads of
// a token run in neighbouring CTAs, so whole rows are read at about the same
// time); a thread one code word of ITEMS tokens, all loaded before the first
// is used: 4 where that still fills the GPU, 1 below (a decode step's tokens).
constexpr int kCacheThreads = 256;

template <bool BF16, int D, int GS, int ITEMS>
__global__ void __launch_bounds__(kCacheThreads) kvq_append_kernel(KvqStoreArgs a) {
    constexpr int W = D / 8, LANES = GS / 8, NG = D / GS, TPB = kCacheThreads / W;
    pdl_trigger();
    pdl_wait();
    const int per_chunk = 2 * a.num_kv_heads;
    const int chunk = blockIdx.x / per_chunk, y = blockIdx.x % per_chunk;
    const int which = y >= a.num_kv_heads, head = which ? y - a.num_kv_heads : y;
    const int w = threadIdx.x % W, token0 = chunk * (TPB * ITEMS) + threadIdx.x / W;
    const void *src = which ? a.v : a.k;
    const int64_t stride = which ? a.v_stride : a.k_stride, col = head * D + w * 8;
    Raw8<BF16> raw[ITEMS];
    int slot[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        const int t = token0 + i * TPB, in = min(t, a.n_tokens - 1);
        slot[i] = t < a.n_tokens ? __ldg(a.slots + in) : -1;
        raw[i].load(src, in * stride + col);
    }
    const int P = a.page_size, shift = P == 16 ? 4 : 5;
    const int words = kvq_block_words(D, P, NG);
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        float x[8], mn, mx;
        raw[i].floats(x);
        group_range<BF16, LANES>(raw[i], x, mn, mx);
        const uint32_t mbits = BF16 ? __float_as_uint(mn) >> 16 : __bfloat16_as_ushort(__float2bfloat16_rn(mn));
        const float m = bits_f(mbits << 16), s = kvq_scale(mx, m);
        uint32_t word = 0;
        if (s > 0.f) {
            if (BF16 && raw[i].smallest(m) * 1024.f >= s)
                word = kvq_word_plain(x, m, s);
            else
                word = kvq_word<!BF16>(x, m, s);
        }
        const int page = slot[i] >> shift, t = slot[i] & (P - 1);
        if (slot[i] < 0) continue;
        if (page >= a.num_pool_pages) {
            if (w == 0) raise_error(a.flags, kErrPageId);
            continue;
        }
        uint32_t *block = a.pool + (int64_t(page) * a.num_kv_heads + head) * words;
        block[(which * P + t) * W + (which ? kvq_value_place<D>(w, t) : kvq_key_place<D>(w))] = word;
        if (w % LANES == 0)
            block[2 * P * W + (which * NG + w / LANES) * P + t] = (__float_as_uint(s) >> 16) | (mbits << 16);
    }
}

// m + s u of the 8 codes of a word, each with fp32's one rounding.  A pair of
// codes cut out in place is a pair of fp16 subnormals u 2^-24 (or 16 u 2^-24),
// which one conversion each makes floats; the scale carries the 2^24 back.
__device__ __forceinline__ void kvq_values(uint32_t word, uint32_t par, float (&x)[8]) {
    const float m = bf16_hi_to_float(par), s = bf16_lo_to_float(par) * 16777216.f, s16 = s * 0.0625f;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const uint32_t w = h ? word >> 8 : word;
        const uint32_t even = w & 0x000f000fu, odd = w & 0x00f000f0u;
        const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&even));
        const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&odd));
        fma(Float2(a.x, a.y), Float2(s, s), Float2(m, m)).get(x[2 * h], x[2 * h + 4]);
        fma(Float2(b.x, b.y), Float2(s16, s16), Float2(m, m)).get(x[2 * h + 1], x[2 * h + 5]);
    }
}

template <bool BF16, int D, int GS, int ITEMS>
__global__ void __launch_bounds__(kCacheThreads) kvq_gather_kernel(KvqStoreArgs a) {
    constexpr int W = D / 8, NG = D / GS, TPB = kCacheThreads / W;
    pdl_trigger();
    pdl_wait();
    const int per_chunk = 2 * a.num_kv_heads;
    const int chunk = blockIdx.x / per_chunk, y = blockIdx.x % per_chunk;
    const int which = y >= a.num_kv_heads, head = which ? y - a.num_kv_heads : y;
    const int w = threadIdx.x % W, token0 = chunk * (TPB * ITEMS) + threadIdx.x / W;
    const int P = a.page_size, shift = P == 16 ? 4 : 5;
    const int words = kvq_block_words(D, P, NG);
    int slot[ITEMS];
    uint32_t word[ITEMS], par[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        const int t = token0 + i * TPB;
        slot[i] = t < a.n_tokens ? __ldg(a.slots + t) : -1;
    }
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        const int page = slot[i] >> shift, t = slot[i] & (P - 1);
        word[i] = par[i] = 0;
        if (slot[i] < 0) continue;
        if (page >= a.num_pool_pages) {
            if (w == 0) raise_error(a.flags, kErrPageId);
            continue;
        }
        const uint32_t *block = a.pool + (int64_t(page) * a.num_kv_heads + head) * words;
        word[i] = __ldg(block + (which * P + t) * W + (which ? kvq_value_place<D>(w, t) : kvq_key_place<D>(w)));
        par[i] = __ldg(block + 2 * P * W + (which * NG + w / (GS / 8)) * P + t);
    }
    void *out = which ? a.v_out : a.k_out;
#pragma unroll
    for (int i = 0; i < ITEMS; i++) {
        const int t = token0 + i * TPB;
        if (t >= a.n_tokens) break;
        float x[8];
        kvq_values(word[i], par[i], x);
        const int64_t at = (int64_t(t) * a.num_kv_heads + head) * D + w * 8;
        if constexpr (BF16) {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + at) =
                make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                           pack_bf16x2(x[6], x[7]));
        } else {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(out) + at);
            o[0] = make_float4(x[0], x[1], x[2], x[3]);
            o[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
    }
}

// Two floats -> bf16x2, rounded down.
__device__ __forceinline__ uint32_t pack_bf16x2_down(float lo, float hi) {
    // truncation rounds towards zero: a negative value goes up by one if anything is cut off
    const uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
    return __byte_perm(a + (uint32_t(int32_t(a) >> 31) & 0xffffu), b + (uint32_t(int32_t(b) >> 31) & 0xffffu), 0x7632);
}

// A lane group of D / 8 lanes, one a code word of a token, takes whole (listed
// page, KV head) tiles: a warp 2 or 4 at a time, so that nothing is combined
// across lanes.  The tiles come through a ring of bulk copies, a warp's own (a
// tile's key codes and key params are 1.1 KB a page of 16 tokens; direct loads
// of one tile a warp left the kernel waiting: 262 us for 36864 pages x 8
// heads).  One tile a warp, its tokens on two lane groups joined by shuffles,
// took 157 us there, whole tiles 125 (64-dim heads 123 and 69), and with two
// values an fma 115 (4.3 TB/s; 63): the mask, conversion, min and max of each
// code bound it (ALU 73 %, issue 80 %), not HBM.
// CTAs of 4 warps: 300 and 600 pages take 3.6 and 4.3 us, with 8 warps 4.2 and
// 4.7 (36864 pages: 125 against 123, before the pairs); pages of 32 tokens leave room for 5 CTAs an SM.
constexpr int kMetaWarps = 4, kMetaStages = 2;

// Words of a tile in the ring: D / 8 more than a multiple of the banks, so that the lane groups meet different ones.
__host__ __device__ constexpr int kvq_meta_tile_words(int words, int page_size, int groups) {
    return page_size * (words + groups) + ((words - page_size * (words + groups)) & 31);
}

template <bool BF16, int D, int GS>
__global__ void __launch_bounds__(kMetaWarps * 32, 8) kvq_meta_kernel(KvqMetaArgs a) {
    constexpr int W = D / 8, T = 32 / W, NG = D / GS, S = kMetaStages, R = 32 / T;
    extern __shared__ __align__(128) uint32_t ring_mem[];
    __shared__ uint64_t bars[kMetaWarps][S];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int P = a.page_size, warps = blockDim.x >> 5;  // at most kMetaWarps
    const int code_words = P * W, tile_words = kvq_meta_tile_words(W, P, NG), stage_words = T * tile_words;
    uint32_t *ring = ring_mem + warp * (S * stage_words);
    if (lane < S) mbar_init(&bars[warp][lane], T);
    mbar_fence_init();
    __syncwarp();
    pdl_trigger();
    pdl_wait();
    const int64_t tiles = int64_t(a.n_list) * a.num_kv_heads, steps = (tiles + T - 1) / T;
    const int64_t first = int64_t(blockIdx.x) * warps + warp, stride = int64_t(gridDim.x) * warps;
    const int n = first < steps ? int((steps - first + stride - 1) / stride) : 0;
    // lane T i + k describes tile k of the warp's steps i, R + i, ..: (page, head) block and valid tokens
    int64_t at = 0;
    int valid = 0;
    auto describe = [&](int i) {
        valid = 0;
        const int64_t tile = (first + (i + lane / T) * stride) * T + lane % T;
        if (i + lane / T >= n || tile >= tiles) return;
        const int e = int(tile / a.num_kv_heads), g = int(tile - int64_t(e) * a.num_kv_heads);
        const int p = __ldg(a.page_ids + e), v = __ldg(a.valid_tokens + e);
        if (p < 0) return;
        if (p >= a.num_pool_pages) {
            raise_error(a.flags, kErrPageId);
            return;
        }
        if (v < 1 || v > P) {
            raise_error(a.flags, kErrValid);
            return;
        }
        at = int64_t(p) * a.num_kv_heads + g, valid = v;
    };
    int put = 0, got = 0, parity = 0;
    auto issue = [&](int i) {  // lane k copies tile k
        if (i >= n) return;
        const int from = i % R * T + lane % T;
        const int v = __shfl_sync(0xffffffffu, valid, from);
        const int64_t b = __shfl_sync(0xffffffffu, at, from);
        if (lane < T) {
            const uint32_t *block = a.pool + b * kvq_block_words(D, P, NG);
            uint64_t *bar = &bars[warp][put];
            uint32_t *dst = ring + put * stage_words + lane * tile_words;
            if (v > 0) {
                mbar_arrive_expect_tx(bar, (code_words + NG * P) * 4);
                bulk_load(dst, block, code_words * 4, bar);
                bulk_load(dst + code_words, block + 2 * code_words, NG * P * 4, bar);
            } else {
                mbar_arrive(bar);
            }
        }
        if (++put == S) put = 0;
    };
    const int place = lane % W, tile = lane / W, w = kvq_key_word<D>(place);
    describe(0);
    for (int i = 0; i < S - 1; i++) issue(i);
    // a description is replaced once its steps are under way, so what the loop needs of the older ones is kept
    int64_t kept_at = 0;
    int kept_valid = 0;
    for (int i = 0; i < n; i++) {
        if (i % R == 0) kept_at = at, kept_valid = valid;
        if ((i + S - 1) % R == 0) describe(i + S - 1);
        issue(i + S - 1);
        const int v = __shfl_sync(0xffffffffu, kept_valid, i % R * T + tile);
        const int64_t b = __shfl_sync(0xffffffffu, kept_at, i % R * T + tile);
        if (!mbar_wait_bounded(&bars[warp][got], parity, kWaitLimitNs)) {
            // a lost copy: flagged, the rest is given up once the copies in flight had their time
            if (lane == 0) raise_error(a.flags, kErrTimeout);
            for (int k = i + 1; k < min(i + S, n); k++) {
                if (++got == S) got = 0, parity ^= 1;
                mbar_wait_bounded(&bars[warp][got], parity, kWaitLimitNs);
            }
            return;
        }
        const uint32_t *codes = ring + got * stage_words + tile * tile_words + place;
        const uint32_t *params = codes - place + code_words + w / (GS / 8) * P;
        float mn[8], mx[8];
#pragma unroll
        for (int k = 0; k < 8; k++) mn[k] = INFINITY, mx[k] = -INFINITY;
        auto take = [&](int ta, int tb, uint32_t pa, uint32_t pb) {
            float x[8], y[8];
            kvq_values(codes[ta * W], pa, x);
            kvq_values(codes[tb * W], pb, y);
#pragma unroll
            for (int k = 0; k < 8; k++) {
                mn[k] = fminf(fminf(x[k], y[k]), mn[k]);
                mx[k] = fmaxf(fmaxf(x[k], y[k]), mx[k]);
            }
        };
        if (__all_sync(0xffffffffu, v == P)) {
            for (int c = 0; c < P; c += 16)
#pragma unroll
                for (int t = 0; t < 16; t += 4) {
                    const uint4 p = *reinterpret_cast<const uint4 *>(params + c + t);
                    take(c + t, c + t + 1, p.x, p.y);
                    take(c + t + 2, c + t + 3, p.z, p.w);
                }
        } else {  // a token past the end repeats the last one
            const int last = max(v - 1, 0), most = __reduce_max_sync(0xffffffffu, v);
#pragma unroll 1
            for (int t = 0; t < most; t += 2) {
                const int ta = min(t, last), tb = min(t + 1, last);
                take(ta, tb, params[ta], params[tb]);
            }
        }
        if (v > 0) {
            const int64_t to = b * 2 * D + w * 8;
            if constexpr (BF16) {  // the maximum up: the negated one down
                uint16_t *o = static_cast<uint16_t *>(a.meta) + to;
                constexpr uint32_t sign = 0x80008000u;
                *reinterpret_cast<uint4 *>(o) =
                    make_uint4(pack_bf16x2_down(mn[0], mn[1]), pack_bf16x2_down(mn[2], mn[3]),
                               pack_bf16x2_down(mn[4], mn[5]), pack_bf16x2_down(mn[6], mn[7]));
                *reinterpret_cast<uint4 *>(o + D) =
                    make_uint4(pack_bf16x2_down(-mx[0], -mx[1]) ^ sign, pack_bf16x2_down(-mx[2], -mx[3]) ^ sign,
                               pack_bf16x2_down(-mx[4], -mx[5]) ^ sign, pack_bf16x2_down(-mx[6], -mx[7]) ^ sign);
            } else {
                float *o = static_cast<float *>(a.meta) + to;
                reinterpret_cast<float4 *>(o)[0] = make_float4(mn[0], mn[1], mn[2], mn[3]);
                reinterpret_cast<float4 *>(o)[1] = make_float4(mn[4], mn[5], mn[6], mn[7]);
                reinterpret_cast<float4 *>(o + D)[0] = make_float4(mx[0], mx[1], mx[2], mx[3]);
                reinterpret_cast<float4 *>(o + D)[1] = make_float4(mx[4], mx[5], mx[6], mx[7]);
            }
        }
        if (++got == S) got = 0, parity ^= 1;
        __syncwarp();
    }
}

// Launches of kernel<bf16, head_dim, group_size, ..>.
#define KVQ_FORMATS(CASE) CASE(128, 128) CASE(128, 64) CASE(128, 32) CASE(64, 64) CASE(64, 32)

// Tokens a CTA takes with `items` a thread, and its CTAs.
int64_t token_ctas(const KvqStoreArgs &a, int head_dim, int items) {
    const int per_cta = kCacheThreads / (head_dim / 8) * items;
    return (int64_t(a.n_tokens) + per_cta - 1) / per_cta * 2 * a.num_kv_heads;
}
// 4 tokens a thread from four CTAs an SM on (one GB300 has 152): below, the loads of one token a thread already cover
// what few CTAs there are, and the other three would only follow one another.  Stored tokens of 8 heads of 128 dims, with
// 1 and 4 a thread: 600 in 2.2 and 4.2 us, 1200 in 3.3 and 4.9, 2400 (the border) in 5.5 and 5.5, 4800 in 10.0 and 8.2,
// 32768 in 62.7 and 46.9; read back, 600 in 1.9 and 2.4, 1200 in 2.6 and 2.3, 2400 in 3.9 and 3.0, 32768 in 49.1 and 30.9.
constexpr int64_t kManyCtas = 608;

}  // namespace

#define KVQ_TOKENS(kernel, d, gs)                                                                              \
    if (head_dim == d && a.group_size == gs) {                                                                 \
        if (many) return bf16 ? launch_pdl(kernel<true, d, gs, 4>, grid, dim3(kCacheThreads), 0, stream, a)    \
                              : launch_pdl(kernel<false, d, gs, 4>, grid, dim3(kCacheThreads), 0, stream, a);  \
        return bf16 ? launch_pdl(kernel<true, d, gs, 1>, grid, dim3(kCacheThreads), 0, stream, a)              \
                    : launch_pdl(kernel<false, d, gs, 1>, grid, dim3(kCacheThreads), 0, stream, a);            \
    }

cudaError_t launch_kvq_append(const KvqStoreArgs &a, int dtype, int head_dim, cudaStream_t stream) {
    const bool bf16 = dtype == kDtypeBf16, many = token_ctas(a, head_dim, 4) >= kManyCtas;
    const dim3 grid(unsigned(token_ctas(a, head_dim, many ? 4 : 1)));
#define KVQ_APPEND(d, gs) KVQ_TOKENS(kvq_append_kernel, d, gs)
    KVQ_FORMATS(KVQ_APPEND)
    return cudaErrorInvalidValue;
}

cudaError_t launch_kvq_gather(const KvqStoreArgs &a, int dtype, int head_dim, cudaStream_t stream) {
    const bool bf16 = dtype == kDtypeBf16, many = token_ctas(a, head_dim, 4) >= kManyCtas;
    const dim3 grid(unsigned(token_ctas(a, head_dim, many ? 4 : 1)));
#define KVQ_GATHER(d, gs) KVQ_TOKENS(kvq_gather_kernel, d, gs)
    KVQ_FORMATS(KVQ_GATHER)
    return cudaErrorInvalidValue;
}

cudaError_t launch_kvq_meta(const KvqMetaArgs &a, int meta_dtype, int head_dim, int num_sms, cudaStream_t stream) {
    const bool bf16 = meta_dtype == kDtypeBf16;
    const int words = head_dim / 8, groups = head_dim / a.group_size, per_warp = 32 / words;
    const int64_t tiles = int64_t(a.n_list) * a.num_kv_heads;
    int warps = kMetaWarps;
    while (warps > 1 && tiles <= int64_t(warps / 2) * per_warp * num_sms) warps /= 2;  // few tiles: all SMs take a share
    const int per_cta = warps * per_warp;
    const int64_t ctas = (tiles + per_cta - 1) / per_cta;
    const dim3 grid(unsigned(ctas < 8 * num_sms ? ctas : 8 * num_sms));
    const int bytes = per_cta * kMetaStages * kvq_meta_tile_words(words, a.page_size, groups) * 4;  // at most 41 KB
#define KVQ_META(d, gs)                                                                                                 \
    if (head_dim == d && a.group_size == gs)                                                                            \
        return bf16 ? launch_pdl(kvq_meta_kernel<true, d, gs>, grid, dim3(warps * 32), bytes, stream, a)                \
                    : launch_pdl(kvq_meta_kernel<false, d, gs>, grid, dim3(warps * 32), bytes, stream, a);
    KVQ_FORMATS(KVQ_META)
    return cudaErrorInvalidValue;
}

}  // namespace qskv
