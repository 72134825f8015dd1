// Attention of one query token a sequence over the 8-bit paged cache (format:
// qskv_kvf.cuh).  Split of the work, pipeline and folds are those of the 4-bit
// decode (kvq_decode.cuh); here is what a warp does with 16 tokens.
//
// Bound: HBM.  A token and head is 2 d + 2 bytes, 24 bytes a clock and SM at
// the copy rate: 170 clocks a part of 16 tokens of 128 dims, in which the
// arithmetic on it has to fit.
//   * A code is a fp16 number after one conversion of two.  With the keys'
//     powers taken out, the logit of token t is scale 2^e_t (q . u_t), and
//     with w_t = p_t 2^f_t of the values' powers f, the output sum_t w_t u_t.
//   * S (16 x 8 tokens) = Q K^T and O (16 x 8 dims) += W V as mma.sync m16n8k16
//     with fp32 accumulators: at most 8 query heads share a cache row, so there
//     is no 128-row tile to feed tcgen05 with.
//   * fp32 precision from fp16 operands: queries (scaled by a power of two into
//     fp16's range) and weights enter as two halves hi + lo, head h's hi half
//     in row h, its lo half in row h + 8, so one product does both.  A lane's
//     logits are then head g's of its own tokens, exactly what the second
//     product takes from it: nothing is moved between lanes.
//   * The order of dims within a product is free: a lane's operands of a key
//     are 16-byte chunks of its row, those of a value pair's row likewise.
//
// Softmax.  Two running references a head, whole numbers: M of the logits,
// p = 2^(x - M), and R of the values' powers on top of it, w = 2^(x - M + f - R).
// They move only when a p or a w would pass 2^15 (fp16): M to the largest
// logit, R to where the largest w is above 2^8, but never so far down that
// outputs would grow.  A sum of both, as one number, would lose the powers
// beside large logits; and moves by powers of two are exact.  Sums of p stay
// per lane until the row ends.
//
// One GB300, GPU time: 32 sequences x 8 KV heads x 128 pages of 16 tokens, 4
// heads a group: 32.2 us (4.2 TB/s; the start and the fold are 6 us of it, and
// of 152 SMs 104 have two rows, which they read at 91 % of an SM's share of the
// copy rate, the others one); 4 x 65536..131072 tokens, 8 heads a group: 138 us
// (5.9 TB/s, 87 % of the copy rate); two short rows: 6.5 us.
#include "kvq_decode.cuh"
#include "qskv_kvf.cuh"

namespace qskv {
namespace {

// fp16 pair of two floats, and what is left of them.
__device__ __forceinline__ uint32_t split_half2(float &x, float &y) {
    const float a = to_half(x), b = to_half(y);
    x -= a, y -= b;
    return pack_half2(a, b);
}

// Lane 4g + t of a warp works on head g; of every 16 tokens on those of the
// pairs t and t + 4 (logits and weights), 2t, 2t + 1, 2t + 8 and 2t + 9.
template <int D>
struct KvfState {
    static constexpr int KS = D / 16;  // steps of 16 dims of the first product
    static constexpr int ND = D / 8;   // groups of 8 dims of the second; lane g's dims in them are g ND + i
    static constexpr int KC = D / 64;  // 16-byte chunks of a key's row a lane reads: t and t + 4
    static constexpr int VC = D / 64;  // and of a value pair's row: VC g + i
    uint32_t q[KS][4];
    float scale;      // logits, in units of log2, of the products
    float m, l;
    float r;          // R + 127, of stored powers
    float o[ND][2];   // head g, dims (2 t) ND + i and (2 t + 1) ND + i; times 2^(M + R)

    __device__ __forceinline__ void attach(uint8_t *, int) {}

    __device__ __forceinline__ void load_query(const KvqDecodeArgs &a, int row) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int b = row / a.num_kv_heads, kh = row % a.num_kv_heads;
        const int64_t at = (int64_t(b) * a.num_q_heads + kh * a.group + g) * D + 16 * t;
        float x[KC][16];
        float top = 0.f;
#pragma unroll
        for (int c = 0; c < KC; c++)
#pragma unroll
            for (int i = 0; i < 16; i += 8) {
                uint4 u = make_uint4(0, 0, 0, 0), v = u;
                if (g < a.group) {
                    if (a.q_is_bf16) {
                        const uint4 w =
                            *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at + 64 * c + i);
                        u = make_uint4(w.x << 16, w.x & 0xffff0000u, w.y << 16, w.y & 0xffff0000u);
                        v = make_uint4(w.z << 16, w.z & 0xffff0000u, w.w << 16, w.w & 0xffff0000u);
                    } else {
                        const uint4 *p =
                            reinterpret_cast<const uint4 *>(static_cast<const float *>(a.q) + at + 64 * c + i);
                        u = p[0], v = p[1];
                    }
                }
                x[c][i] = __uint_as_float(u.x), x[c][i + 1] = __uint_as_float(u.y);
                x[c][i + 2] = __uint_as_float(u.z), x[c][i + 3] = __uint_as_float(u.w);
                x[c][i + 4] = __uint_as_float(v.x), x[c][i + 5] = __uint_as_float(v.y);
                x[c][i + 6] = __uint_as_float(v.z), x[c][i + 7] = __uint_as_float(v.w);
            }
#pragma unroll
        for (int c = 0; c < KC; c++)
#pragma unroll
            for (int i = 0; i < 16; i++) top = fmaxf(top, fabsf(x[c][i]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // q 2^(13 - e) has its largest entry in [2^13, 2^14): the hi half drops 2^-11 of an entry, the lo half, normal
        // down to 2^-14, 2^-11 of that, or 2^-38 of the largest entry
        const int e = min(max(int(__float_as_uint(top) >> 23) - 127, -100), 100);
        const float up = __uint_as_float(uint32_t(140 - e) << 23);
        scale = __uint_as_float(uint32_t(114 + e) << 23) * a.scale_log2;
#pragma unroll
        for (int s = 0; s < KS; s++) {
            float *y = x[s / 4] + s % 4 * 4;
#pragma unroll
            for (int k = 0; k < 4; k++) y[k] *= up;
            q[s][0] = split_half2(y[0], y[1]), q[s][1] = pack_half2(y[0], y[1]);
            q[s][2] = split_half2(y[2], y[3]), q[s][3] = pack_half2(y[2], y[3]);
        }
    }

    __device__ __forceinline__ void clear() {
        m = kNoRef, l = 0.f, r = 127.f;
#pragma unroll
        for (int i = 0; i < ND; i++) o[i][0] = o[i][1] = 0.f;
    }

    // Part `tile` of those from st on; its first nv (1..16) tokens count.
    template <int NT>
    __device__ __forceinline__ void tiles(const uint8_t *st, int tile, int nv) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const uint8_t *part = st + tile * kvf_part_bytes(D);
        // ---- logits: c[j] of tokens 8 j + 2t (elements 0 and, of the lo halves, 2) and 8 j + 2t + 1
        float c[2][4], c2[2][4];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const uint8_t *row = part + (8 * j + g) * D;
#pragma unroll
            for (int k = 0; k < KC; k++) {
                const uint4 w = *reinterpret_cast<const uint4 *>(row + kvf_key_chunk<D>(t + 4 * k, g) * 16);
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t(&qa)[4] = q[4 * k + i];
                    const uint32_t b0 = kvf_half2(x[i]), b1 = kvf_half2(x[i] >> 16);
                    float(&to)[4] = i & 1 ? c2[j] : c[j];
                    if (k == 0 && i < 2)
                        mma_f16_first(to, qa[0], qa[1], qa[2], qa[3], b0, b1);
                    else
                        mma_f16(to, qa[0], qa[1], qa[2], qa[3], b0, b1);
                }
            }
        }
        // powers of tokens 8 j + 2t and the next: keys, values
        const uint8_t *pow = part + 32 * D + 2 * t;
        float x[2][2], f[2][2];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const uint32_t pk = *reinterpret_cast<const uint16_t *>(pow + 8 * j);
            const uint32_t pv = *reinterpret_cast<const uint16_t *>(pow + 16 + 8 * j);
#pragma unroll
            for (int k = 0; k < 2; k++) {
                const float s = (c[j][k] + c2[j][k]) + (c[j][2 + k] + c2[j][2 + k]);
                x[j][k] = s * (kvf_power(pk >> (8 * k) & 255) * scale);
                f[j][k] = float(pv >> (8 * k) & 255) - r;
                if (8 * j + 2 * t + k >= nv) x[j][k] = -INFINITY, f[j][k] = 0.f;
            }
        }
        // ---- weights
        float p[2][2], w[2][2], most = 0.f;
        auto weigh = [&] {
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int k = 0; k < 2; k++) {
                    const float y = x[j][k] - m;
                    p[j][k] = ex2(y), w[j][k] = ex2(y + f[j][k]);
                    most = fmaxf(most, fmaxf(p[j][k], w[j][k]));
                }
        };
        weigh();
        if (!__all_sync(0xffffffffu, most <= 32768.f)) {
            float mn = -INFINITY, top = -INFINITY;
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int k = 0; k < 2; k++) mn = fmaxf(mn, x[j][k]);
            mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 1));
            mn = fmaxf(m, ceilf(fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, 2))));
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int k = 0; k < 2; k++) top = fmaxf(top, x[j][k] - mn + f[j][k]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // sums go down by 2^down, outputs by 2^(down - more)
            const float down = fmaxf(m - mn, -1000.f), more = fmaxf(ceilf(top) - 9.f, down);
            const float power = kvf_power(max(int(down - more) + 127, 0));
            m = mn, r += more, l *= kvf_power(max(int(down) + 127, 0));
#pragma unroll
            for (int i = 0; i < ND; i++) o[i][0] *= power, o[i][1] *= power;
#pragma unroll
            for (int j = 0; j < 2; j++)
#pragma unroll
                for (int k = 0; k < 2; k++) f[j][k] -= more;
            weigh();
        }
        l += (p[0][0] + p[0][1]) + (p[1][0] + p[1][1]);
        uint32_t a[4];
#pragma unroll
        for (int j = 0; j < 2; j++) {
            a[2 * j] = split_half2(w[j][0], w[j][1]);
            a[2 * j + 1] = pack_half2(w[j][0], w[j][1]);
        }
        // ---- values: pairs t and t + 4.  Each product starts at zero and is added to the sums in fp32: the tensor
        // cores cut what they add towards zero, which along a row would add up.
#pragma unroll
        for (int v = 0; v < VC; v++) {
            uint32_t y[2][4];
#pragma unroll
            for (int j = 0; j < 2; j++) {
                const int pair = t + 4 * j;
                const uint4 u = *reinterpret_cast<const uint4 *>(part + 16 * D + pair * 2 * D +
                                                                 kvf_value_chunk<D>(VC * g + v, pair) * 16);
                y[j][0] = u.x, y[j][1] = u.y, y[j][2] = u.z, y[j][3] = u.w;
                if (nv < 16) {  // what lies past the end may be no number
                    const uint32_t keep = (2 * pair < nv ? 0x00ff00ffu : 0u) | (2 * pair + 1 < nv ? 0xff00ff00u : 0u);
#pragma unroll
                    for (int k = 0; k < 4; k++) y[j][k] &= keep;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; i++) {
                float z[4];
                mma_f16_first(z, a[0], a[1], a[2], a[3], kvf_half2(y[0][i >> 1] >> (16 * (i & 1))),
                              kvf_half2(y[1][i >> 1] >> (16 * (i & 1))));
                add_pair(o[8 * v + i][0], o[8 * v + i][1], z[0] + z[2], z[1] + z[3]);
            }
        }
    }

    // Sums over the lanes; the row's outputs (final) or its piece's reference,
    // weight sum and unnormalised output.
    __device__ __forceinline__ void finish(const KvqDecodeArgs &a, int row, bool final, float *piece_o, float *piece_m,
                                           float *piece_l) {
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (g >= a.group) return;
        const int64_t head0 = int64_t(row / a.num_kv_heads) * a.num_q_heads + int64_t(row % a.num_kv_heads) * a.group;
        const float inv = !final ? 1.f : l > 0.f ? 1.f / l : 0.f, power = kvf_power(uint32_t(r));
        float *dst = (final ? a.out + (head0 + g) * D : piece_o + g * D) + t * (D / 4);
#pragma unroll
        for (int k = 0; k < 2; k++)
#pragma unroll
            for (int i = 0; i < ND; i += 4)
                *reinterpret_cast<float4 *>(dst + k * ND + i) =
                    make_float4(o[i][k] * inv * power, o[i + 1][k] * inv * power, o[i + 2][k] * inv * power,
                                o[i + 3][k] * inv * power);
        if (t == 0) {
            if (final) {
                if (a.lse) a.lse[head0 + g] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
            } else {
                piece_m[g] = m, piece_l[g] = l;
            }
        }
    }
};

// Pages of P tokens, cut into parts of 16: a unit each.
template <int D_, int P>
struct KvfFormat {
    using State = KvfState<D_>;
    static constexpr int D = D_, TOKENS = kKvfPartTokens, SUB = P / kKvfPartTokens, BYTES = kvf_part_bytes(D_);
    static constexpr int U = 4096 / (2 * kKvfPartTokens * D_);  // a stage is about 4 KB
    static constexpr int STATE_BYTES = 0;
    static constexpr bool PAIRS = false;
};

}  // namespace

// The rules by which rows are split count units, here parts of 16 tokens, with the constants of the 4-bit decode.  What they
// take over this cache (pages of 16 tokens, 4 heads a group), and what other splits do: 256 rows of 128 selected pages, a CTA
// each, 32.2 us, evenly 37.0; 2048 rows of 7 pages, to warps, 17.2, evenly 29.0; 2560 rows of 1 to 32 pages, to warps, 78.6,
// evenly 61.5 (there the rule costs); 8 rows of 32, 64, 128 pages, a CTA for every 32 places, 10.3, 13.3, 13.6, for every 16
// 11.2, 11.5, 11.8, for every 64 10.3, 14.1, 17.3; 8 rows of 1024, 2048 selected pages, at most 16 CTAs each, 21.0, 30.2, at
// most 8 26.0, 42.3, at most 64 19.0, 24.0.
cudaError_t launch_kvf_decode(KvqDecodeArgs a, int head_dim, int num_sms, cudaStream_t stream) {
    if (head_dim == 128)
        return a.page_size == 16 ? launch_one<KvfFormat<128, 16>>(a, num_sms, stream)
                                 : launch_one<KvfFormat<128, 32>>(a, num_sms, stream);
    return a.page_size == 16 ? launch_one<KvfFormat<64, 16>>(a, num_sms, stream)
                             : launch_one<KvfFormat<64, 32>>(a, num_sms, stream);
}

}  // namespace qskv
