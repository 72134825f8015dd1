// Attention of one query token a sequence over the 4-bit paged cache (format:
// qskv_kvq.cuh).
//
// With k = m + s u per group j of dims, the logit of token t is
//     l_t = scale * sum_j (s_tj (q_j . u_tj) + m_tj sum(q_j)),
// and the output sum_t p_t (m_tj + s_tj u_t) over softmax weights p, so the
// matrix products run on the codes u themselves and scales and minima are
// applied per token and group, outside them.
//
// Bound: the latency of dependent instructions.  128 registers a thread leave
// 16 warps an SM, of which 0.8 to 1.4 a scheduler can issue in a cycle: 40 to
// 63 % of the issue slots are used, ALU 31 to 51 %, tensor cores 15 to 26 %,
// DRAM 24 to 56 %, and waits of a fixed latency are the largest stall.  (With
// all pages in L2 the kernel takes as long as from HBM.)  A token and head is
// d + 8 NG bytes, 23 bytes a clock and SM at the copy rate; the arithmetic on
// it should fit that time, which shapes the inner loop:
//   * a code is a fp16 number almost as it stands.  Keys: one byte permutation
//     puts a byte, two codes c0 + 16 c1, under a zero byte, the subnormal
//     (c0 + 16 c1) 2^-24; masking the upper code off gives c0 2^-24.  The
//     query of c1 is taken a sixteenth, and that much off c0's.  Values: the
//     same under 0x64 (1024 + x, exact), less the middle of the codes, so that
//     sums of signed, normal numbers are made.
//   * S (16 tokens x 8 columns) = K_tile Q^T and O^T (dims x 8) += V_tile^T P^T
//     as mma.sync m16n8k16 with fp32 accumulators; at most 8 query heads share
//     a cache row, so there is no 128-row tile to feed tcgen05 with, and the
//     codes would have to be widened into shared memory for it.
//   * fp32 precision from fp16 operands: queries (scaled by a power of two
//     into fp16's range) and weights enter as two halves hi + lo.  With at
//     most 4 heads (HC = 4) the halves share the 8 columns: column 2h is head
//     h's hi, 2h + 1 its lo; with 8 heads they are two products.  bf16 queries
//     of 8 heads need no lo half as long as a code's query stays as it is, so
//     their keys' upper codes are masked out instead (one product; permuted
//     ones with the lo half take 119 instead of 110 us at 32 x 8 rows of 8192
//     tokens in groups of 32; fp32 queries gain: 87 instead of 92 us in groups
//     of 128).  Root mean square error of the outputs against fp64, as a share
//     of theirs, over all formats, 300 and 3000 tokens: 1.4e-7 to 2.8e-7, with
//     8 heads up to 3.4e-7 (fp32 queries) and 5.0e-7 (bf16).  What a half drops
//     is measured against the largest entry of its head: a query with one entry
//     4096 times the others has logits within 1.5e-6 of sum |q| (|m| + s u).
//   * a key's words lie so that a lane's operands are one vector load; values
//     come through ldmatrix.trans, whose 16-bit elements are four codes of one
//     token: the pair of a register is two tokens, as the product needs.
//
// Softmax.  Running references per head: M for the exponent and sg for the
// weights times value scales (p s sg is what becomes fp16).  Both are moved
// only when a weight would pass 2^12, or p s sg 2^14 (rare after the first
// tile), so the usual step has no rescaling and one vote.  Sums of weights
// and of p m stay per lane until the row ends.
//
// Work split.  A unit is one page of one (sequence, KV head) row.  A warp has
// its own ring of stages of about 4 KB (one bulk copy a page, one mbarrier a
// stage) and its own running state, and takes a range of units:
//   * many rows of few pages: rows to warps in turn, whole;
//   * rows that fit one wave of CTAs and are cut alike (selections, short
//     tables): a group of CTAs a row, whose warps share its units;
//   * else all units in row order in equal ranges, one a warp, for a grid of
//     two CTAs an SM; every CTA finds its ranges from a scan of the lengths
//     (or selection counts) in shared memory, so ragged batches balance.
// A row that lies within a warp is finished by it, pieces of a row within a
// CTA are folded there, and pieces of several CTAs by the CTA that draws the
// row's last ticket, always in unit order: results do not depend on timing.
//
// One GB300, GPU time: 32 sequences x 8 KV heads x 128 pages of 16 tokens, 4
// heads a group: 22.8 us (3.2 TB/s); 4 x 65536..131072 tokens, groups of 32
// dims: 106 us (4.8 TB/s, 70 % of the copy rate); 64 ragged sequences up to
// 4095 tokens with 8 heads a group, fp32 queries: 68.5 us (2.3 TB/s); 32 x 8
// rows of 8192 tokens, 8 heads a group, one group of 128 dims: 80.6 us with
// bf16 queries, 86.0 with fp32 ones (3.5 TB/s); two short rows: 5.8 us.
#pragma once

#include <cuda_fp16.h>

#include "qskv_internal.h"
#include "qskv_kvq.cuh"

namespace qskv {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kEntries = 512;      // entries of the unit prefix held in shared memory
constexpr int kFill = 16;          // units a warp describes at once (a multiple of the units a stage)
constexpr int kRowModePages = 64, kRowCtas = 16, kRowUnits = 32, kWarpUnits = 12, kWarpUnitsMany = 32;
constexpr int kMaxRing = 3;        // stages a warp: 2 or 3 fit, by the format
constexpr float kNoRef = -3e38f;   // M before the first token: below any finite logit, so that the first token moves it
// sg before the first token whose share p s is 2^-100 or more: tokens of one value have a scale of zero and say nothing of
// the scales to come, and on this reference any share above 2^-86 passes kTopW, so that it is fitted then.
constexpr float kNoScale = 1.2676506002282294e30f;  // 2^100
// Largest weight, and largest weight times value scale, in the references' units.
constexpr float kTopP = 4096.f, kTopW = 16383.f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The same with a zero accumulator in.
__device__ __forceinline__ void mma_f16_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t add_half2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
// Bytes 0 and 2 (BYTE 0) or 1 and 3 (BYTE 1) of a word as a pair of fp16
// numbers under the high byte `top`: two codes c0 + 16 c1 each, on 1024 and
// exact with top 0x64 (normal numbers), times 2^-24 with 0 (subnormals).
template <int BYTE>
__device__ __forceinline__ uint32_t byte_pair(uint32_t w, uint32_t top) {
    return __byte_perm(w, top, BYTE ? 0x4341 : 0x4240);
}
constexpr uint32_t kTop = 0x64646464u;
// The lower code alone of such a pair on 1024, less 8; and both less their
// middles, 8 + 16 * 8.
__device__ __forceinline__ uint32_t less8(uint32_t x) { return add_half2(x & 0xff0fff0fu, 0xe408e408u); }
__device__ __forceinline__ uint32_t less136(uint32_t x) { return add_half2(x, 0xe488e488u); }

// a0 += b0, a1 += b1 as one instruction.
__device__ __forceinline__ void add_pair(float &a0, float &a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b;\n\t"
        "mov.b64 a, {%0, %1};\n\tmov.b64 b, {%2, %3};\n\t"
        "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
        : "+f"(a0), "+f"(a1)
        : "f"(b0), "f"(b1));
}

// c0 += a0 * b0, c1 += a1 * b1 likewise.
__device__ __forceinline__ void fma_pair(float &c0, float &c1, float a0, float a1, float b0, float b1) {
    asm("{\n\t.reg .b64 a, b, c;\n\t"
        "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%0, %1};\n\t"
        "fma.rn.f32x2 c, a, b, c;\n\tmov.b64 {%0, %1}, c;\n\t}"
        : "+f"(c0), "+f"(c1)
        : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// x rounded to fp16, as a float.
__device__ __forceinline__ float to_half(float x) { return __half2float(__float2half_rn(x)); }

// x rounded to a multiple of `grid`, a power of two.  The hi halves of fp32
// queries are multiples of one grid with at most 11 bits.  Key codes are
// subnormal operands, which the tensor cores line up 7 bits lower than their
// value; on a grid a hi half times a code, and sums of them up to 2^24 grid
// units, lose nothing by that.  (Value codes are normal numbers, and the
// weights' hi halves simply rounded.)
__device__ __forceinline__ float on_grid(float x, float grid) {
    const float c = 12582912.f * grid;  // 1.5 * 2^23 units
    return (x + c) - c;
}

__device__ __forceinline__ float max_over_tokens(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum_over_tokens(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// ------------------------------------------------------------------ units --
__device__ __forceinline__ int seq_of(const KvqDecodeArgs &a, int b) {
    const int s = __ldg(a.seq_lens + b), cap = a.max_pages * a.page_size;
    if (s < 0 || s > cap) {
        raise_error(a.flags, kErrSeqLen);
        return s < 0 ? 0 : cap;
    }
    return s;
}
__device__ __forceinline__ int pages_of(const KvqDecodeArgs &a, int b) {
    return (seq_of(a, b) + a.page_size - 1) / a.page_size;
}
// Units of list item i: a row's selected pages, or all pages of a sequence
// (of one of its KV heads).
__device__ __forceinline__ int units_of(const KvqDecodeArgs &a, int i) {
    if (!a.selected) return pages_of(a, i);
    const int n = __ldg(a.n_selected + i), lim = min(a.top_k, pages_of(a, i / a.num_kv_heads));
    if (n < 0 || n > lim) {
        raise_error(a.flags, kErrSelected);
        return max(0, min(n, lim));
    }
    return n;
}

struct Unit {
    const uint8_t *src;  // its block; nullptr: skipped
    int row_valid;       // row << 6 | valid tokens
    int slot, count;     // its place among the row's units, and how many those are
};

struct Shared {
    int prefix[kEntries + 1];
    int warp_sum[kWarps];
    Unit desc[kWarps][2 * kFill];
    uint64_t bar[kWarps][kMaxRing];
    // pieces of rows that no warp owns whole: 2w ends in, 2w + 1 runs on from, warp w's range
    int piece_row[2 * kWarps], piece_begin[2 * kWarps], piece_end[2 * kWarps];
    float piece_m[2 * kWarps][8], piece_l[2 * kWarps][8], piece_f[2 * kWarps][8];
    // rows that other CTAs hold pieces of
    int open, open_row[2], open_slot0[2], open_slot1[2], open_n[2], open_last[2];
    float row_m[8], row_l[8];
};

// The unit of row `row` at place `slot` of `count`.
__device__ __forceinline__ Unit unit_of(const KvqDecodeArgs &a, int row, int slot, int count, uint32_t block_bytes) {
    const int b = row / a.num_kv_heads, seq = seq_of(a, b);
    const int j = a.selected ? __ldg(a.selected + int64_t(row) * a.top_k + slot) : slot;
    Unit r;
    r.src = nullptr, r.row_valid = row << 6, r.slot = slot, r.count = count;
    if (j < 0 || j * int64_t(a.page_size) >= seq) {
        raise_error(a.flags, kErrSelected);
        return r;
    }
    const int p = __ldg(a.page_table + int64_t(b) * a.max_pages + j);
    if (p < 0 || p >= a.num_pool_pages) {
        raise_error(a.flags, kErrPageId);
        return r;
    }
    r.src = reinterpret_cast<const uint8_t *>(a.pool) + (int64_t(p) * a.num_kv_heads + row % a.num_kv_heads) * block_bytes;
    r.row_valid |= min(a.page_size, seq - j * a.page_size);
    return r;
}

// The unit of row `row` at place `slot` of the `row_units` places a row has at
// most (rows to warps): empty past the row's end.
__device__ __forceinline__ Unit place_of(const KvqDecodeArgs &a, int row, int slot, int row_units, uint32_t block_bytes) {
    if (slot < units_of(a, a.selected ? row : row / a.num_kv_heads)) return unit_of(a, row, slot, row_units, block_bytes);
    Unit r;
    r.src = nullptr, r.row_valid = row << 6, r.slot = slot, r.count = row_units;
    return r;
}

// The unit with global index u (even split).
__device__ __forceinline__ Unit unit_at(const KvqDecodeArgs &a, const Shared &s, int entries, int per, int u,
                                        uint32_t block_bytes) {
    int lo = 0, hi = entries;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s.prefix[mid] <= u)
            lo = mid;
        else
            hi = mid;
    }
    const int heads = a.selected ? 1 : a.num_kv_heads;  // rows of a list item
    const int last = (a.selected ? a.batch * a.num_kv_heads : a.batch) - 1;
    int i = lo * per, off = u - s.prefix[lo], n = units_of(a, i);
    while (off >= n * heads && i < last) off -= n * heads, n = units_of(a, ++i);
    if (off >= n * heads) {  // the lengths (or counts) became shorter while the kernel ran
        raise_error(a.flags, a.selected ? kErrSelected : kErrSeqLen);
        Unit r;
        r.src = nullptr, r.row_valid = (i * heads) << 6, r.slot = 0, r.count = 1;
        return r;
    }
    const int g = off / n;
    return unit_of(a, i * heads + g, off - g * n, n, block_bytes);
}

// ----------------------------------------------------- one row in a warp --
// Lane 4g + t of a warp works, for every 16-token tile, on tokens g and g + 8
// and on head t (HC = 4) or heads 2t and 2t + 1 (HC = 8).
template <int D, int NG, int HC, int P>
struct RowState {
    static constexpr int NW = D / 32;     // 32-dim chunks of a row; code words a lane holds of a token's key
    static constexpr int GW = NW / NG;    // chunks a group
    static constexpr int NH = HC / 4;     // heads a lane
    uint32_t qh[NW][4];
    uint4 *ql;  // HC = 8: the lo halves' fragments, in the warp's shared memory ([NW][32 lanes]): registers are short
    float qa[NH], qb[NH][NG];
    float m[NH], l[NH], sg[NH], pm[NH][NG];
    bool q_lo;  // HC = 8: the queries have lo halves (fp32 ones; bf16 fits fp16 as it is, half the products)
    // of a lane, for each of its heads and each chunk: the sums of dim 4g's codes and of those plus 16 times dim 4g + 1's
    // (rows g and g + 8 of [0]), and the same of dims 4g + 2 and 4g + 3 ([1])
    float o[NW][2][2 * NH];

    __device__ __forceinline__ void load_query(const KvqDecodeArgs &a, int row) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int h = HC == 4 ? g >> 1 : g;
        q_lo = !a.q_is_bf16;
        const int b = row / a.num_kv_heads, kh = row % a.num_kv_heads;
        const int64_t at = (int64_t(b) * a.num_q_heads + kh * a.group + h) * D + 8 * t;
        float q[NW][8];
#pragma unroll
        for (int i = 0; i < NW; i++) {
            uint4 x = make_uint4(0, 0, 0, 0), y = x;
            if (h < a.group) {
                if (a.q_is_bf16) {
                    const uint4 w = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at + 32 * i);
                    x = make_uint4(w.x << 16, w.x & 0xffff0000u, w.y << 16, w.y & 0xffff0000u);
                    y = make_uint4(w.z << 16, w.z & 0xffff0000u, w.w << 16, w.w & 0xffff0000u);
                } else {
                    const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const float *>(a.q) + at + 32 * i);
                    x = p[0], y = p[1];
                }
            }
            q[i][0] = __uint_as_float(x.x), q[i][1] = __uint_as_float(x.y), q[i][2] = __uint_as_float(x.z);
            q[i][3] = __uint_as_float(x.w), q[i][4] = __uint_as_float(y.x), q[i][5] = __uint_as_float(y.y);
            q[i][6] = __uint_as_float(y.z), q[i][7] = __uint_as_float(y.w);
        }
        float top = 0.f, sum[NG];
#pragma unroll
        for (int j = 0; j < NG; j++) sum[j] = 0.f;
#pragma unroll
        for (int i = 0; i < NW; i++)
#pragma unroll
            for (int k = 0; k < 8; k++) top = fmaxf(top, fabsf(q[i][k])), sum[i / GW] += q[i][k];
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
#pragma unroll
        for (int j = 0; j < NG; j++) {
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 1);
            sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], 2);
            sum[j] *= a.scale_log2;
        }
        // q 2^(13 - e) has its largest entry, and a sixteenth more of it, below 2^14: hi in multiples of 2^3 (exact up
        // to there), lo (at most 2^2) held times 2^11
        const int e = min(max(int(__float_as_uint(top * 1.0625f) >> 23) - 127, -100), 100);
        const float up = __uint_as_float(uint32_t(140 - e) << 23);
        const float back = __uint_as_float(uint32_t(127 + e + 11) << 23) * a.scale_log2;  // 2^24 / up
#pragma unroll
        for (int i = 0; i < NW; i++)
#pragma unroll
            for (int r = 0; r < 4; r++) {  // codes r and r + 4
                // odd r meets 16 times its code, alone (HC = 8, bf16 queries) or with the code before added, whose query
                // then loses what that code has got there already
                const float f = r & 1 ? up * 0.0625f : up;
                float x = q[i][r] * f, y = q[i][r + 4] * f;
                if ((HC == 4 || q_lo) && !(r & 1)) {
                    x = fmaf(q[i][r + 1], -0.0625f * up, x);
                    y = fmaf(q[i][r + 5], -0.0625f * up, y);
                }
                float gx = on_grid(x, r & 1 ? 0.5f : 8.f), gy = on_grid(y, r & 1 ? 0.5f : 8.f);
                if (HC == 8 && !q_lo) gx = x, gy = y;
                const uint32_t hi = pack_half2(gx, gy), lo = pack_half2((x - gx) * 2048.f, (y - gy) * 2048.f);
                if constexpr (HC == 4) {
                    qh[i][r] = g & 1 ? lo : hi;
                } else {
                    qh[i][r] = hi;
                    if (q_lo) reinterpret_cast<uint32_t *>(ql + i * 32 + lane)[r] = lo;  // read by this lane alone
                }
            }
#pragma unroll
        for (int h2 = 0; h2 < NH; h2++) {
            const int from = HC == 4 ? 8 * t : 8 * t + 4 * h2;
            qa[h2] = __shfl_sync(0xffffffffu, back, from);
#pragma unroll
            for (int j = 0; j < NG; j++) qb[h2][j] = __shfl_sync(0xffffffffu, sum[j], from);
        }
    }

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int h = 0; h < NH; h++) {
            m[h] = kNoRef, l[h] = 0.f, sg[h] = kNoScale;
#pragma unroll
            for (int j = 0; j < NG; j++) pm[h][j] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < NW; c++)
#pragma unroll
            for (int r = 0; r < 2 * NH; r++) o[c][0][r] = o[c][1][r] = 0.f;
    }

    // Logits of one 16-token tile (`tile` of the block at `st`) in x, and its value params in va, vb.
    __device__ __forceinline__ void logits(const uint8_t *st, int tile, float (&x)[2][NH], uint32_t (&va)[NG],
                                           uint32_t (&vb)[NG]) const {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int ta = tile * 16 + g;
        // ---- keys: codes of tokens g and g + 8, logits
        uint32_t ka[NW], kb[NW];
        const uint8_t *kp = st + ta * (D / 2) + t * (D / 8);
        if constexpr (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4 *>(kp), y = *reinterpret_cast<const uint4 *>(kp + 4 * D);
            ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
            kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
        } else {
            const uint2 x = *reinterpret_cast<const uint2 *>(kp), y = *reinterpret_cast<const uint2 *>(kp + 4 * D);
            ka[0] = x.x, ka[1] = x.y, kb[0] = y.x, kb[1] = y.y;
        }
        const uint32_t *par = reinterpret_cast<const uint32_t *>(st + P * D) + ta;
        float xm[2][NH];
#pragma unroll
        for (int h = 0; h < NH; h++) x[0][h] = x[1][h] = xm[0][h] = xm[1][h] = 0.f;
#pragma unroll
        for (int j = 0; j < NG; j++) {
            const uint32_t pa = par[j * P], pb = par[j * P + 8];
            va[j] = par[(NG + j) * P], vb[j] = par[(NG + j) * P + 8];
            float c0[4], c1[4];
            constexpr uint32_t lo = 0x000f000fu, hi = 0x00f000f0u;
            constexpr float lo_unit = 1.f / 2048.f;
            float ua[NH], ub[NH];
            if constexpr (HC == 4) {  // two chains where a group has more than one chunk
#pragma unroll
                for (int i = 0; i < GW; i++) {
                    const uint32_t a = ka[j * GW + i], b = kb[j * GW + i];
                    const uint32_t x = byte_pair<0>(a, 0), y = byte_pair<0>(b, 0);
                    const uint32_t x2 = byte_pair<1>(a, 0), y2 = byte_pair<1>(b, 0);
                    const uint32_t(&q)[4] = qh[j * GW + i];
                    if (i == 0) {
                        mma_f16_first(c0, a & lo, b & lo, x, y, q[0], q[1]);
                        if (GW > 1)
                            mma_f16_first(c1, x2 & lo, y2 & lo, x2, y2, q[2], q[3]);
                        else
                            mma_f16(c0, x2 & lo, y2 & lo, x2, y2, q[2], q[3]);
                    } else {
                        mma_f16(c0, a & lo, b & lo, x, y, q[0], q[1]);
                        mma_f16(c1, x2 & lo, y2 & lo, x2, y2, q[2], q[3]);
                    }
                }
                if (GW > 1) c0[0] += c1[0], c0[1] += c1[1], c0[2] += c1[2], c0[3] += c1[3];
                ua[0] = fmaf(c0[1], lo_unit, c0[0]);
                ub[0] = fmaf(c0[3], lo_unit, c0[2]);
            } else {
                if (q_lo) {  // one product's operands for both halves: a permutation saves the masks of the upper codes
#pragma unroll
                    for (int i = 0; i < GW; i++) {
                        const uint32_t a = ka[j * GW + i], b = kb[j * GW + i];
                        const uint32_t x = byte_pair<0>(a, 0), y = byte_pair<0>(b, 0);
                        const uint32_t x2 = byte_pair<1>(a, 0), y2 = byte_pair<1>(b, 0);
                        const uint32_t(&q)[4] = qh[j * GW + i];
                        const uint4 ql4 = ql[(j * GW + i) * 32 + lane];
                        if (i == 0) {
                            mma_f16_first(c0, a & lo, b & lo, x, y, q[0], q[1]);
                            mma_f16_first(c1, a & lo, b & lo, x, y, ql4.x, ql4.y);
                        } else {
                            mma_f16(c0, a & lo, b & lo, x, y, q[0], q[1]);
                            mma_f16(c1, a & lo, b & lo, x, y, ql4.x, ql4.y);
                        }
                        mma_f16(c0, x2 & lo, y2 & lo, x2, y2, q[2], q[3]);
                        mma_f16(c1, x2 & lo, y2 & lo, x2, y2, ql4.z, ql4.w);
                    }
#pragma unroll
                    for (int k = 0; k < 4; k += 2) fma_pair(c0[k], c0[k + 1], c1[k], c1[k + 1], lo_unit, lo_unit);
                } else {  // masked: a code's query stays the bf16 value, which fp16 holds whole, and no lo half is needed
#pragma unroll
                    for (int i = 0; i < GW; i++) {
                        const uint32_t a = ka[j * GW + i], b = kb[j * GW + i], a8 = a >> 8, b8 = b >> 8;
                        const uint32_t(&q)[4] = qh[j * GW + i];
                        if (i == 0)
                            mma_f16_first(c0, a & lo, b & lo, a & hi, b & hi, q[0], q[1]);
                        else
                            mma_f16(c0, a & lo, b & lo, a & hi, b & hi, q[0], q[1]);
                        mma_f16(c0, a8 & lo, b8 & lo, a8 & hi, b8 & hi, q[2], q[3]);
                    }
                }
                ua[0] = c0[0], ua[NH - 1] = c0[1];
                ub[0] = c0[2], ub[NH - 1] = c0[3];
            }
            const float sa = bf16_lo_to_float(pa), ma = bf16_hi_to_float(pa);
            const float sb = bf16_lo_to_float(pb), mb = bf16_hi_to_float(pb);
            if constexpr (NH == 2) {  // in pairs: 32 x 8 rows of 8192 tokens, fp32, in 85.4 against 87.5 us
                fma_pair(x[0][0], x[0][1], sa, sa, ua[0], ua[1]), fma_pair(xm[0][0], xm[0][1], ma, ma, qb[0][j], qb[1][j]);
                fma_pair(x[1][0], x[1][1], sb, sb, ub[0], ub[1]), fma_pair(xm[1][0], xm[1][1], mb, mb, qb[0][j], qb[1][j]);
            } else {
                x[0][0] = fmaf(sa, ua[0], x[0][0]), xm[0][0] = fmaf(ma, qb[0][j], xm[0][0]);
                x[1][0] = fmaf(sb, ub[0], x[1][0]), xm[1][0] = fmaf(mb, qb[0][j], xm[1][0]);
            }
        }
#pragma unroll
        for (int h = 0; h < NH; h++) x[0][h] = fmaf(qa[h], x[0][h], xm[0][h]), x[1][h] = fmaf(qa[h], x[1][h], xm[1][h]);
    }

    // NT tiles, tile i of them number tile0 + i of the blocks from st on.  The first nv (1..16) tokens of the last one
    // count, all of the others.
    template <int NT>
    __device__ __forceinline__ void tiles(const uint8_t *st, int tile0, int nv) {
        constexpr int PT = P / 16;
        constexpr uint32_t block_bytes = kvq_block_words(D, P, NG) * 4;
        const int lane = threadIdx.x & 31, g = lane >> 2;
        uint32_t va[NT][NG], vb[NT][NG];
        float x[NT][2][NH];
#pragma unroll
        for (int i = 0; i < NT; i++) logits(st + (tile0 + i) / PT * block_bytes, (tile0 + i) % PT, x[i], va[i], vb[i]);
        if (NT == 1 && nv < 16) {  // places past the end: no weight, and nothing of their params
            const bool off_a = g >= nv, off_b = g + 8 >= nv;
#pragma unroll
            for (int h = 0; h < NH; h++) {
                if (off_a) x[0][0][h] = -INFINITY;
                if (off_b) x[0][1][h] = -INFINITY;
            }
#pragma unroll
            for (int j = 0; j < NG; j++) {
                if (off_a) va[0][j] = 0;
                if (off_b) vb[0][j] = 0;
            }
        }
        // ---- weights
        float p[NT][2][NH], w[NT][2][NH][NG];
        float most_p = 0.f, most_w = 0.f;
#pragma unroll
        for (int i = 0; i < NT; i++)
#pragma unroll
            for (int h = 0; h < NH; h++) {
                p[i][0][h] = ex2(x[i][0][h] - m[h]), p[i][1][h] = ex2(x[i][1][h] - m[h]);
                most_p = fmaxf(most_p, fmaxf(p[i][0][h], p[i][1][h]));
                const float ps0 = p[i][0][h] * sg[h], ps1 = p[i][1][h] * sg[h];
#pragma unroll
                for (int j = 0; j < NG; j++) {
                    w[i][0][h][j] = ps0 * bf16_lo_to_float(va[i][j]);
                    w[i][1][h][j] = ps1 * bf16_lo_to_float(vb[i][j]);
                    most_w = fmaxf(most_w, fmaxf(w[i][0][h][j], w[i][1][h][j]));
                }
            }
        if (!__all_sync(0xffffffffu, most_p <= kTopP && most_w <= kTopW)) {
#pragma unroll
            for (int h = 0; h < NH; h++) {
                float mn = m[h];
#pragma unroll
                for (int i = 0; i < NT; i++) mn = fmaxf(mn, fmaxf(x[i][0][h], x[i][1][h]));
                mn = max_over_tokens(mn);
                const float f = ex2(m[h] - mn);
                float top = 0.f;
#pragma unroll
                for (int i = 0; i < NT; i++) {
                    p[i][0][h] = ex2(x[i][0][h] - mn), p[i][1][h] = ex2(x[i][1][h] - mn);
#pragma unroll
                    for (int j = 0; j < NG; j++)
                        top = fmaxf(top, fmaxf(p[i][0][h] * bf16_lo_to_float(va[i][j]), p[i][1][h] * bf16_lo_to_float(vb[i][j])));
                }
                top = max_over_tokens(top);
                // sg such that the tiles' largest p s sg lies in [2^8, 2^9), but no higher than the references' move f lets
                // what is summed already stay where it is: sums never grow by being rescaled (a head whose reference
                // stands still, rescaled because another one's moves, would take its sums up to infinity step by step).
                // References are powers of two and handled by their exponents: two divisions a head here, at a row's start
                // most of all, took 74.4 instead of 68.6 us in the ragged batch.
                float s = sg[h];
                if (top >= 7.888609052210118e-31f)  // 2^-100; a move of 2^128 or more sets no limit (infinity)
                    s = fminf(__int_as_float((262 << 23) - (__float_as_int(top) & 0x7f800000)),
                              s * __int_as_float((127 + int(fminf(mn - m[h], 128.f))) << 23));
                const float r = f * s * __int_as_float((254 << 23) - __float_as_int(sg[h]));
                m[h] = mn, sg[h] = s, l[h] *= f;
#pragma unroll
                for (int j = 0; j < NG; j++) {
                    pm[h][j] *= f;
#pragma unroll
                    for (int i = 0; i < NT; i++) {
                        w[i][0][h][j] = p[i][0][h] * (bf16_lo_to_float(va[i][j]) * s);
                        w[i][1][h][j] = p[i][1][h] * (bf16_lo_to_float(vb[i][j]) * s);
                    }
                }
#pragma unroll
                for (int c = 0; c < NW; c++)
#pragma unroll
                    for (int k = h; k < 2 * NH; k += NH) o[c][0][k] *= r, o[c][1][k] *= r;
            }
        }
        // the value codes enter their product less 8 (sums of signed numbers: the tensor cores cut what they add
        // towards zero, which on 0..15 is a bias), so pm takes the middle m + 8 s of each group
#pragma unroll
        for (int i = 0; i < NT; i++) {
#pragma unroll
            for (int h = 0; h < NH; h++) l[h] += p[i][0][h] + p[i][1][h];
#pragma unroll
            for (int j = 0; j < NG; j++) {
                const float mida = fmaf(8.f, bf16_lo_to_float(va[i][j]), bf16_hi_to_float(va[i][j]));
                const float midb = fmaf(8.f, bf16_lo_to_float(vb[i][j]), bf16_hi_to_float(vb[i][j]));
#pragma unroll
                for (int h = 0; h < NH; h++) pm[h][j] = fmaf(p[i][1][h], midb, fmaf(p[i][0][h], mida, pm[h][j]));
            }
        }
        values<NT>(st, tile0, w);
    }

    // The outputs' sums take NT tiles' values with weights w.  A chunk of 32 dims at a time goes through accumulators
    // that start at zero and are added to the sums in fp32: the tensor cores cut what they add towards zero, which
    // along a whole row would shrink the sums (1.1e-6 of them over 82 tiles); and with hi and lo columns (HC = 4) one
    // sum of both is all that is kept.
    template <int NT>
    __device__ __forceinline__ void values(const uint8_t *st, int tile0, const float (&w)[NT][2][NH][NG]) {
        constexpr int PT = P / 16;
        constexpr uint32_t block_bytes = kvq_block_words(D, P, NG) * 4;
        const int lane = threadIdx.x & 31, mat = lane >> 3, r = lane & 7;
        const int sw = D == 128 ? (r >> 1) & 3 : (r >> 2) & 1;
        const uint32_t vrow = smem_u32(st) + P * (D / 2) + ((mat & 1) * 8 + r) * (D / 2);
        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
        for (int c2 = 0; c2 < NW / 2; c2++) {
            uint32_t v[NT][4];
#pragma unroll
            for (int i = 0; i < NT; i++)
                ldmatrix_x4_trans(v[i], vrow + (tile0 + i) / PT * block_bytes + (tile0 + i) % PT * 16 * (D / 2) +
                                            (((2 * c2 + (mat >> 1)) ^ sw) << 4));
#pragma unroll
            for (int cc = 0; cc < 2; cc++) {
                const int c = 2 * c2 + cc;
                float x0[4], x1[4];
#pragma unroll
                for (int i = 0; i < NT; i++) {
                    if (c % GW == 0) {
                        const int j = c / GW;
#pragma unroll
                        for (int k = 0; k < 2; k++) {
                            const float x = to_half(w[i][k][0][j]), y = to_half(w[i][k][NH - 1][j]);
                            if constexpr (HC == 4) {
                                bh[i][k] = movmatrix_trans(pack_half2(x, w[i][k][0][j] - x));
                            } else {
                                bh[i][k] = movmatrix_trans(pack_half2(x, y));
                                bl[i][k] = movmatrix_trans(pack_half2(w[i][k][0][j] - x, w[i][k][NH - 1][j] - y));
                            }
                        }
                    }
                    // rows g: the lower code of each byte; rows g + 8: both, lower + 16 * upper
                    const uint32_t v0 = v[i][2 * cc], v1 = v[i][2 * cc + 1];
                    const uint32_t e0 = byte_pair<0>(v0, kTop), e1 = byte_pair<0>(v1, kTop);
                    const uint32_t f0 = byte_pair<1>(v0, kTop), f1 = byte_pair<1>(v1, kTop);
                    const uint32_t a[4] = {less8(e0), less136(e0), less8(e1), less136(e1)};
                    const uint32_t b[4] = {less8(f0), less136(f0), less8(f1), less136(f1)};
                    if (i == 0) {
                        mma_f16_first(x0, a[0], a[1], a[2], a[3], bh[i][0], bh[i][1]);
                        mma_f16_first(x1, b[0], b[1], b[2], b[3], bh[i][0], bh[i][1]);
                    } else {
                        mma_f16(x0, a[0], a[1], a[2], a[3], bh[i][0], bh[i][1]);
                        mma_f16(x1, b[0], b[1], b[2], b[3], bh[i][0], bh[i][1]);
                    }
                    if constexpr (HC == 8) {
                        mma_f16(x0, a[0], a[1], a[2], a[3], bl[i][0], bl[i][1]);
                        mma_f16(x1, b[0], b[1], b[2], b[3], bl[i][0], bl[i][1]);
                    }
                }
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    if constexpr (HC == 4) {
                        o[c][0][k] += x0[2 * k] + x0[2 * k + 1], o[c][1][k] += x1[2 * k] + x1[2 * k + 1];
                    } else {
                        add_pair(o[c][0][2 * k], o[c][0][2 * k + 1], x0[2 * k], x0[2 * k + 1]);
                        add_pair(o[c][1][2 * k], o[c][1][2 * k + 1], x1[2 * k], x1[2 * k + 1]);
                    }
                }
            }
        }
    }

    // Sums over the lanes; the row's outputs (final) or its piece's reference,
    // weight sum and unnormalised output.
    __device__ __forceinline__ void finish(const KvqDecodeArgs &a, int row, bool final, float *piece_o, float *piece_m,
                                           float *piece_l) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int64_t head0 = int64_t(row / a.num_kv_heads) * a.num_q_heads + int64_t(row % a.num_kv_heads) * a.group;
#pragma unroll
        for (int h = 0; h < NH; h++) {
            l[h] = sum_over_tokens(l[h]);
#pragma unroll
            for (int j = 0; j < NG; j++) pm[h][j] = sum_over_tokens(pm[h][j]);
            const int head = NH * t + h;
            if (head >= a.group) continue;
            const float unit = 1.f / sg[h];
            const float inv = !final ? 1.f : l[h] > 0.f ? 1.f / l[h] : 0.f;
            float *dst = final ? a.out + (head0 + head) * D : piece_o + head * D;
#pragma unroll
            for (int c = 0; c < NW; c++) {
                const float base = pm[h][c / GW];
                float v[4];
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const float lower = o[c][k >> 1][h], both = o[c][k >> 1][NH + h];
                    v[k] = fmaf(lower, unit, base) * inv;
                    v[k + 1] = fmaf(both - lower, unit * 0.0625f, base) * inv;
                }
                *reinterpret_cast<float4 *>(dst + 32 * c + 4 * g) = make_float4(v[0], v[1], v[2], v[3]);
            }
            if (g == 0) {
                if (final) {
                    if (a.lse) a.lse[head0 + head] = l[h] > 0.f ? (m[h] + log2f(l[h])) * kLn2 : -INFINITY;
                } else {
                    piece_m[head] = m[h], piece_l[head] = l[h];
                }
            }
        }
    }
};

// --------------------------------------------------------- the kernel --
template <int D, int NG, int HC, int P>
__global__ void __launch_bounds__(kThreads, 2) kvq_decode_kernel(KvqDecodeArgs a) {
    extern __shared__ __align__(128) uint8_t ring_mem[];
    __shared__ Shared s;
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int U = 4096 / (P * D), kPageTiles = P / 16, kTiles = U * kPageTiles;
    constexpr uint32_t block_bytes = kvq_block_words(D, P, NG) * 4;
    static_assert(U >= 1 && kFill % U == 0, "a stage is a whole number of pages, a fill of stages");
    const int G = a.group, S = a.stages;
    uint8_t *ring = ring_mem + warp * (S * U * block_bytes);
    if (lane < S) mbar_init(&s.bar[warp][lane], 1);
    if (tid < 2 * kWarps) s.piece_row[tid] = -1;
    if (tid == 0) s.open = 0;
    mbar_fence_init();
    // Nothing is read before this, the lengths neither: whoever wrote them may have let this kernel start early.
    pdl_wait();

    // ---- this warp's units [u0, u1): of its CTA's row, or of all rows in order
    int u0, u1, cta_begin, cta_end;
    int entries = 0, per = 1, upc = 0;
    const int warp_index = blockIdx.x * kWarps + warp, all_warps = gridDim.x * kWarps;
    const int row0 = a.row_ctas ? blockIdx.x / a.row_ctas : 0;
    int count0 = 0;
    if (a.warp_units) {  // rows to warps in turn: this warp's rows, warp_units places each
        const int rows = a.batch * a.num_kv_heads;
        u0 = 0, u1 = warp_index < rows ? (rows - warp_index + all_warps - 1) / all_warps * a.warp_units : 0;
        cta_begin = cta_end = 0;
    } else if (a.row_ctas) {
        count0 = units_of(a, a.selected ? row0 : row0 / a.num_kv_heads);
        upc = (count0 + a.row_ctas - 1) / a.row_ctas;
        const int part = blockIdx.x - row0 * a.row_ctas;
        cta_begin = min(part * upc, count0), cta_end = min(cta_begin + upc, count0);
        const int n = cta_end - cta_begin;
        u0 = cta_begin + n * warp / kWarps, u1 = cta_begin + n * (warp + 1) / kWarps;
        if (count0 == 0 && part == 0) {
            const int64_t h0 = int64_t(row0 / a.num_kv_heads) * a.num_q_heads + int64_t(row0 % a.num_kv_heads) * G;
            for (int c = tid; c < G * D / 4; c += kThreads)
                reinterpret_cast<float4 *>(a.out + h0 * D)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (a.lse && tid < G) a.lse[h0 + tid] = -INFINITY;
        }
    } else {
        // prefix of the units over the list (rows, or sequences)
        const int heads = a.selected ? 1 : a.num_kv_heads;
        const int items = a.selected ? a.batch * a.num_kv_heads : a.batch;
        per = (items + kEntries - 1) / kEntries, entries = (items + per - 1) / per;
        const int ept = (entries + kThreads - 1) / kThreads;
        int mine = 0;
        for (int e = tid * ept; e < min((tid + 1) * ept, entries); e++) {
            int n = 0;
            for (int i = e * per; i < min((e + 1) * per, items); i++) n += units_of(a, i) * heads;
            s.prefix[e] = n;
            mine += n;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += up;
        }
        if (lane == 31) s.warp_sum[warp] = incl;
        __syncthreads();
        int before = incl - mine, total = 0;
#pragma unroll
        for (int w = 0; w < kWarps; w++) {
            if (w < warp) before += s.warp_sum[w];
            total += s.warp_sum[w];
        }
        for (int e = tid * ept; e < min((tid + 1) * ept, entries); e++) {
            const int n = s.prefix[e];
            s.prefix[e] = before;
            before += n;
        }
        __syncthreads();
        const int upw = max(int((uint32_t(total) + all_warps - 1) / all_warps), 1);
        upc = upw * kWarps;
        const int64_t c0 = int64_t(blockIdx.x) * upc;
        u0 = int(min(c0 + int64_t(warp) * upw, int64_t(total))), u1 = int(min(int64_t(u0) + upw, int64_t(total)));
        cta_begin = int(min(c0, int64_t(total))), cta_end = int(min(c0 + upc, int64_t(total)));
        // rows without a token or a selected page
        for (int base = blockIdx.x * kWarps + warp; base < items; base += 32 * all_warps) {
            const int64_t i = base + int64_t(lane) * all_warps;
            uint32_t none = __ballot_sync(0xffffffffu, i < items && units_of(a, int(i)) == 0);
            while (none) {
                const int k = __ffs(none) - 1;
                none &= none - 1;
                const int item_heads = a.selected ? G : a.num_q_heads;
                const int64_t h0 = int64_t(base + k * all_warps) * item_heads;  // a row's, or a sequence's, lie together
                for (int c = lane; c < item_heads * D / 4; c += 32)
                    reinterpret_cast<float4 *>(a.out + h0 * D)[c] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (a.lse)
                    for (int h = lane; h < item_heads; h += 32) a.lse[h0 + h] = -INFINITY;
            }
        }
    }
    __syncthreads();  // piece_row, open

    // ---- the warp's pipeline: stage k holds units kU .. kU + U - 1 of its range
    const int n = u1 - u0, stages = (n + U - 1) / U;
    int put = 0, got = 0, parity = 0;
    const uint64_t policy = l2_evict_first_policy();
    uint32_t plain = 0;  // bit per ring stage: all its units are whole pages of the row before them
    uint32_t live = 0, whole = 0;
    int fill_last = -64;  // the unit before the first has no row
    auto issue = [&](int k) {
        if (k >= stages) return;
        const int first = k * U;
        if (first % kFill == 0) {  // describe the next kFill units
            __syncwarp();
            const int u = u0 + first + lane;
            Unit d;
            d.src = nullptr, d.row_valid = -1;
            if (lane < kFill && u < u1) {
                d = a.warp_units ? place_of(a, warp_index + u / a.warp_units * all_warps, u % a.warp_units, a.warp_units, block_bytes)
                    : a.row_ctas ? unit_of(a, row0, u, count0, block_bytes)
                                 : unit_at(a, s, entries, per, u, block_bytes);
                s.desc[warp][(first + lane) % (2 * kFill)] = d;
            }
            // bit i: unit i is there; it is a whole page of the row before it
            int before = __shfl_up_sync(0xffffffffu, d.row_valid, 1);
            if (lane == 0) before = fill_last;
            live = __ballot_sync(0xffffffffu, d.src != nullptr);
            whole = __ballot_sync(0xffffffffu, d.src != nullptr && d.row_valid == ((before & ~63) | P));
            fill_last = __shfl_sync(0xffffffffu, d.row_valid, kFill - 1);
            __syncwarp();
        }
        constexpr uint32_t stage_mask = (1u << U) - 1;
        const uint32_t here = live >> (first % kFill) & stage_mask;
        const bool same = (whole >> (first % kFill) & stage_mask) == stage_mask;
        plain = (plain & ~(1u << put)) | (uint32_t(same) << put);
        const uint8_t *src = nullptr;
        if (lane < U && (here >> lane & 1)) src = s.desc[warp][(first + lane) % (2 * kFill)].src;
        uint64_t *bar = &s.bar[warp][put];
        if (lane == 0) mbar_arrive_expect_tx(bar, __popc(here) * block_bytes);
        __syncwarp();
        if (src) {
            if (a.evict_first)
                bulk_load_hint(ring + (put * U + lane) * block_bytes, src, block_bytes, bar, policy);
            else
                bulk_load(ring + (put * U + lane) * block_bytes, src, block_bytes, bar);
        }
        if (++put == S) put = 0;
    };
    RowState<D, NG, HC, P> st;
    st.ql = reinterpret_cast<uint4 *>(ring_mem + kWarps * (S * U * block_bytes)) + warp * (D / 32 * 32);
    int row = -1, row_begin = 0, row_end = 0;
    float *piece_first = a.first_o + (int64_t(blockIdx.x) * kWarps + warp) * (G * D);
    auto close = [&](bool at_end) {
        const bool final = row_begin >= u0 && row_end <= u1;
        const int k = 2 * warp + (at_end ? 1 : 0);
        st.finish(a, row, final, at_end ? reinterpret_cast<float *>(ring) : piece_first, s.piece_m[k], s.piece_l[k]);
        if (!final && lane == 0) s.piece_row[k] = row, s.piece_begin[k] = row_begin, s.piece_end[k] = row_end;
    };
    auto enter = [&](const Unit &u, int it) {  // the state moves to the row of the warp's unit `it`
        if ((u.row_valid >> 6) == row) return;
        if (row >= 0) close(false);
        row = u.row_valid >> 6, row_begin = u0 + it - u.slot, row_end = row_begin + u.count;
        st.load_query(a, row);
        st.clear();
    };
    for (int k = 0; k < S; k++) issue(k);
    for (int k = 0; k < stages; k++) {
        const bool same = (plain >> got) & 1;
        if (!same) enter(s.desc[warp][k * U % (2 * kFill)], k * U);  // its query loads while the pages are on their way
        if (!mbar_wait_bounded(&s.bar[warp][got], parity, kWaitLimitNs)) {
            // a lost copy: flagged, the rest is given up once the copies in flight had their time
            if (lane == 0) raise_error(a.flags, kErrTimeout);
            for (int i = k + 1; i < min(k + S, stages); i++) {
                if (++got == S) got = 0, parity ^= 1;
                mbar_wait_bounded(&s.bar[warp][got], parity, kWaitLimitNs);
            }
            break;
        }
        const uint8_t *stage = ring + got * (U * block_bytes);
        // Two tiles a step share the vote and hide each other's latencies, where the registers suffice: with 8 heads only
        // for one group a row (32 x 8 rows of 8192 tokens: 84 us, 89 tile by tile; a ragged batch with two groups 77 and 74).
        constexpr bool kPairs = HC == 4 || NG == 1;
        if (kPairs && same) {
#pragma unroll
            for (int t = 0; t < kTiles; t += 2) st.template tiles<2>(stage, t, 16);
        } else {
#pragma unroll 1
            for (int t = 0; t < kTiles; t++) {
                int nv = 16;
                if (kPairs || !same) {
                    const int it = k * U + t / kPageTiles;
                    if (it >= n) break;
                    const Unit u = s.desc[warp][it % (2 * kFill)];
                    enter(u, it);
                    nv = min((u.row_valid & 63) - t % kPageTiles * 16, 16);
                    if (!u.src || nv <= 0) continue;
                }
                st.template tiles<1>(stage, t, nv);
            }
        }
        if (++got == S) got = 0, parity ^= 1;
        __syncwarp();
        issue(k + S);
    }
    if (row >= 0) close(true);
    if (a.warp_units) return;  // every row was one warp's
    __syncthreads();

    // ---- pieces of one row within the CTA, in unit order
    const int elems = G * D / 4;
    if (tid < 16 * kWarps) {  // weight of each piece for each head
        const int k = tid >> 3, h = tid & 7, r = s.piece_row[k];
        if (r >= 0 && h < G) {
            float m = kNoRef;
#pragma unroll
            for (int i = 0; i < 2 * kWarps; i++)
                if (s.piece_row[i] == r) m = fmaxf(m, s.piece_m[i][h]);
            s.piece_f[k][h] = ex2(s.piece_m[k][h] - m);
        }
    }
    __syncthreads();
    const int piece_row = lane < 2 * kWarps ? s.piece_row[lane] : -1;
    const uint32_t pieces = __ballot_sync(0xffffffffu, piece_row >= 0);
    // a run starts at a piece whose row the piece before it (of those there are) does not have
    const uint32_t earlier = pieces & ((1u << lane) - 1);
    const int previous = __shfl_sync(0xffffffffu, piece_row, earlier ? 31 - __clz(earlier) : 0);
    const uint32_t runs = __ballot_sync(0xffffffffu, piece_row >= 0 && (!earlier || previous != piece_row));
    const int chunks = (elems + 31) / 32, items = __popc(runs) * chunks;  // an item: 32 float4 of a run
    for (int i = warp; i < items; i += kWarps) {
        uint32_t left = runs;
        for (int k = i / chunks; k > 0; k--) left &= left - 1;
        const int first = __ffs(left) - 1, e = i % chunks * 32 + lane;
        const int r = __shfl_sync(0xffffffffu, piece_row, first);
        const uint32_t members = __ballot_sync(0xffffffffu, piece_row == r);
        const int begin_u = s.piece_begin[first], end_u = s.piece_end[first];
        const bool whole = begin_u >= cta_begin && end_u <= cta_end;
        const int slot = a.row_ctas ? blockIdx.x : 2 * blockIdx.x + (begin_u < cta_begin ? 0 : 1);
        if (e < elems) {
            const int h = e * 4 / D;
            float m = kNoRef, l = 0.f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            auto add = [&](int k, const float *src) {
                const float f = s.piece_f[k][h];
                const float4 v = reinterpret_cast<const float4 *>(src)[e];
                l = fmaf(f, s.piece_l[k][h], l), m = fmaxf(m, s.piece_m[k][h]);
                o.x = fmaf(f, v.x, o.x), o.y = fmaf(f, v.y, o.y), o.z = fmaf(f, v.z, o.z), o.w = fmaf(f, v.w, o.w);
            };
#pragma unroll
            for (int w = 0; w < kWarps; w++) {
                if (members >> (2 * w) & 1) add(2 * w, a.first_o + (int64_t(blockIdx.x) * kWarps + w) * (G * D));
                if (members >> (2 * w + 1) & 1)
                    add(2 * w + 1, reinterpret_cast<const float *>(ring_mem + w * (S * U * block_bytes)));
            }
            const int64_t head0 = int64_t(r / a.num_kv_heads) * a.num_q_heads + int64_t(r % a.num_kv_heads) * G;
            if (whole) {
                const float inv = l > 0.f ? 1.f / l : 0.f;
                reinterpret_cast<float4 *>(a.out + head0 * D)[e] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
                if (a.lse && e * 4 % D == 0) a.lse[head0 + h] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
            } else {
                reinterpret_cast<float4 *>(a.part_o)[int64_t(slot) * elems + e] = o;
                if (e * 4 % D == 0) a.part_ml[slot * 16 + h] = m, a.part_ml[slot * 16 + 8 + h] = l;
            }
        }
        if (!whole) {
            __threadfence();
            if (lane == 0 && i % chunks == 0) {  // at most two: a row from before, a row beyond the CTA's range
                // pieces of the row: one for each CTA its units fall into
                int c = row0 * a.row_ctas, np = (count0 + upc - 1) / upc;
                if (!a.row_ctas) c = begin_u / upc, np = (end_u - 1) / upc - c + 1;
                const int x = atomicAdd(&s.open, 1);
                s.open_row[x] = r, s.open_n[x] = np;
                // the CTA where a row begins wrote its slot 1, the later ones their slot 0
                s.open_slot0[x] = a.row_ctas ? c : 2 * c + 1, s.open_slot1[x] = a.row_ctas ? c : 2 * c;
            }
        }
    }
    __syncthreads();
    if (s.open == 0) return;
    if (tid < s.open) {
        const bool last = atomicAdd(a.tickets + s.open_row[tid], 1u) == uint32_t(s.open_n[tid] - 1);
        if (last) a.tickets[s.open_row[tid]] = 0;
        s.open_last[tid] = last;
    }
    __syncthreads();

    // ---- rows whose last ticket this CTA drew: pieces of several CTAs, in unit order
    for (int f = 0; f < s.open; f++) {
        if (!s.open_last[f]) continue;
        const int r = s.open_row[f], np = s.open_n[f], slot0 = s.open_slot0[f], slot1 = s.open_slot1[f];
        const int step = a.row_ctas ? 1 : 2;
        float *pw = reinterpret_cast<float *>(ring_mem);  // [np][G] weights, then [kThreads] float4
        float4 *red = reinterpret_cast<float4 *>(ring_mem + (size_t(np) * G * 4 + 15) / 16 * 16);
        __threadfence();
        const int groups = kThreads / elems, grp = tid / elems, e = tid % elems, h = e * 4 / D;
        auto piece = [&](int k) {
            const int slot = k == 0 ? slot0 : slot1 + k * step;
            return __ldcg(reinterpret_cast<const float4 *>(a.part_o) + int64_t(slot) * elems + e);
        };
        float4 early[4];
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (grp + i * groups < np) early[i] = piece(grp + i * groups);
        if (warp < G) {
            float m = kNoRef, l = 0.f;
            for (int k = lane; k < np; k += 32) {
                const int slot = k == 0 ? slot0 : slot1 + k * step;
                const float x = __ldcg(a.part_ml + slot * 16 + warp), y = __ldcg(a.part_ml + slot * 16 + 8 + warp);
                const float mn = fmaxf(m, x);
                l = fmaf(l, ex2(m - mn), y * ex2(x - mn));
                pw[k * G + warp] = x;
                m = mn;
            }
            float top = m;
#pragma unroll
            for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            l *= ex2(m - top);
#pragma unroll
            for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            for (int k = lane; k < np; k += 32) pw[k * G + warp] = ex2(pw[k * G + warp] - top);
            if (lane == 0) s.row_m[warp] = top, s.row_l[warp] = l;
        }
        __syncthreads();
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        auto add = [&](const float4 &v, int k) {
            const float x = pw[k * G + h];
            o.x = fmaf(x, v.x, o.x), o.y = fmaf(x, v.y, o.y), o.z = fmaf(x, v.z, o.z), o.w = fmaf(x, v.w, o.w);
        };
#pragma unroll
        for (int i = 0; i < 4; i++)
            if (grp + i * groups < np) add(early[i], grp + i * groups);
#pragma unroll 4
        for (int k = grp + 4 * groups; k < np; k += groups) add(piece(k), k);
        red[tid] = o;
        __syncthreads();
        if (grp == 0) {
            for (int k = 1; k < groups; k++) {
                const float4 v = red[k * elems + e];
                o.x += v.x, o.y += v.y, o.z += v.z, o.w += v.w;
            }
            const float l = s.row_l[h], inv = l > 0.f ? 1.f / l : 0.f;
            const int64_t head0 = int64_t(r / a.num_kv_heads) * a.num_q_heads + int64_t(r % a.num_kv_heads) * G;
            reinterpret_cast<float4 *>(a.out + head0 * D)[e] = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
            if (a.lse && e * 4 % D == 0) a.lse[head0 + h] = l > 0.f ? (s.row_m[h] + log2f(l)) * kLn2 : -INFINITY;
        }
        __syncthreads();
    }
}

// Shared memory a CTA may take beside its static part with two CTAs an SM
// (228 KB an SM, 1 KB of each CTA's reserved).
constexpr int kRingBudget = 113 * 1024 - int(sizeof(Shared));
template <int D, int HC>
constexpr int kQueryBytes = HC == 8 ? kWarps * D * 16 : 0;  // the lo halves of 8 heads

template <int D, int NG, int HC, int P>
cudaError_t launch_one(KvqDecodeArgs &a, int num_sms, cudaStream_t stream) {
    // a stage is about 4 KB: with fewer pages its fixed cost shows, with more the ring has too few stages
    constexpr int stage = kWarps * (4096 / (P * D)) * kvq_block_words(D, P, NG) * 4;
    constexpr int stages = (kRingBudget - kQueryBytes<D, HC>) / stage;
    constexpr int bytes = stages * stage + kQueryBytes<D, HC>;
    static_assert(stages >= 2 && stages <= kMaxRing, "the ring needs two stages, and a barrier each");
    a.stages = stages;
    const int rows = a.batch * a.num_kv_heads, slots = kvq_decode_ctas(num_sms);
    const int row_units = a.selected && a.top_k < a.max_pages ? a.top_k : a.max_pages;
    // Rows of few pages, more of them than CTAs: whole rows to warps, nothing to join (2048 rows of 7 pages: 15.3 us,
    // 28.7 split evenly; 512 rows of 1 to 32 pages: 28.0 and 19.6, so longer rows only if every warp gets one).  Rows
    // that fit one wave of CTAs and are cut about alike (selections, short tables): a group of CTAs each, which need
    // no prefix over the lengths (256 rows of 128 selected pages 22.7 us, 29.0 split evenly; 8 rows of 32 pages 8.5 and
    // 10.6; longer tables are split evenly for their lengths' sake).  A CTA of the group for every 32 places: 8 rows of
    // 32, 64, 128 pages take 8.6, 11.7, 11.7 us so, 10.6, 10.5, 10.9 with 16 places and 8.6, 10.8, 13.8 with 64; at most
    // 16 CTAs: 8 rows of 1024 and 2048 pages take 17.0 and 24.5 us, 19.8 and 33.2 with 8, 15.0 and 21.4 with 64, which
    // shorter rows and more of them do not tell apart.  The split goes by the table's width, the lengths being on the
    // device: 32 rows of 7 pages take 13 us in a table of 2048 pages, 7 in one of 8.  Else the even split.
    const bool whole = rows > slots && (row_units <= kWarpUnits || (row_units <= kWarpUnitsMany && rows >= slots * kWarps));
    a.row_ctas = 0, a.warp_units = whole ? row_units : 0;
    if (rows <= slots && (a.selected || row_units <= kRowModePages)) {
        const int most = slots / rows, want = (row_units + kRowUnits - 1) / kRowUnits;
        a.row_ctas = want < most ? want : most;
        if (a.row_ctas > kRowCtas) a.row_ctas = kRowCtas;
    }
    // The pages are read once a call.  Above half of L2 they are marked to leave it first, which keeps queries, tables
    // and partial outputs in it: 24.8 -> 23.7 us at 71 MB; below, pages that stay serve the next call: 10.1 us at
    // 19 MB with the plain policy, 11.2 with the other.
    a.evict_first = int64_t(rows) * row_units * (stage / kWarps / (4096 / (P * D))) * 2 > l2_cache_bytes();
    const int64_t even = (int64_t(rows) * row_units + kWarps - 1) / kWarps;
    const unsigned grid = a.warp_units ? unsigned(slots < (rows + kWarps - 1) / kWarps ? slots : (rows + kWarps - 1) / kWarps)
                          : a.row_ctas ? unsigned(rows * a.row_ctas) : unsigned(even < slots ? even : slots);
    const cudaError_t e = cudaFuncSetAttribute(kvq_decode_kernel<D, NG, HC, P>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               bytes);
    if (e != cudaSuccess) return e;
    return launch_pdl(kvq_decode_kernel<D, NG, HC, P>, dim3(grid), dim3(kThreads), bytes, stream, a);
}

template <int P>
cudaError_t launch_page(KvqDecodeArgs &a, int head_dim, int num_sms, cudaStream_t stream) {
    const int ng = head_dim / a.group_size;
    const bool few = a.group <= 4;
    if (head_dim == 128) {
        if (ng == 1) return few ? launch_one<128, 1, 4, P>(a, num_sms, stream) : launch_one<128, 1, 8, P>(a, num_sms, stream);
        if (ng == 2) return few ? launch_one<128, 2, 4, P>(a, num_sms, stream) : launch_one<128, 2, 8, P>(a, num_sms, stream);
        return few ? launch_one<128, 4, 4, P>(a, num_sms, stream) : launch_one<128, 4, 8, P>(a, num_sms, stream);
    }
    if (ng == 1) return few ? launch_one<64, 1, 4, P>(a, num_sms, stream) : launch_one<64, 1, 8, P>(a, num_sms, stream);
    return few ? launch_one<64, 2, 4, P>(a, num_sms, stream) : launch_one<64, 2, 8, P>(a, num_sms, stream);
}

}  // namespace
}  // namespace qskv
