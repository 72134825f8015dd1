// Prefill that keeps fp32 (qskv_prefill.cuh), for fp32 queries over any cache
// and bf16 queries over an fp32 one: what one bf16 operand would cut.
//
// Products go through mma.sync as sums of products of bf16 parts: an fp32
// number is x0 + x1 + x2, each part the next 8 bits, over fp32's whole range,
// and x y = x0 y0 + (x0 y1 + x1 y0) + (x0 y2 + x1 y1 + x2 y0) within 2^-22 of
// itself (x1 y2 < 2^-23, x2 y1 < 2^-24); a cached value that is a bf16 number is one part, of three products.
// x0 y0 and the rest are summed apart and joined in fp32, a block's outputs
// likewise, so that the products' own summation runs over few terms.  Keys and
// values are cut (hi bits as they are, which is exact and cannot overflow),
// queries and weights rounded to nearest, so that what is left out has no sign.
//
// A CTA takes 64 rows of queries, 16 a warp, against kKeys keys at a time.  It
// splits keys and values once, on their way to shared memory, and reads
// operands by ldmatrix; a weight is split in the registers that it is made in,
// as the next product's operand.  What is needed next is read into registers
// before the products and stored after them.
//
// Bound: six products of 1022 FMAs a clock and SM (measured), 170 of fp32,
// where the fp32 pipes have 128 and a kernel of them reached 68.  Tensor pipes
// are busy 55 % of the time; what is left is the latency of a block's steps
// with two warps a scheduler.  One GB300: 6 prompts of up to 500 tokens, 16
// heads of 64 dims, in 52 us (82 with fp32 FMAs); 6 of 2048 tokens, the same
// heads, 0.96 ms (1.52), 32 heads of 128 dims over 8 3.5 ms (5.28; 59 TFLOP/s),
// over an 8-bit cache 2.6 ms.  Outputs of the first are off by 1.1e-7 from
// fp64, 2.4e-7 with fp32 FMAs.  A tile's keys are one CTA's, one block after the
// other, so few tokens over a long cache leave the GPU nearly idle: 4 rows of 1
// to 4 tokens over 65536, 32 heads of 128 dims over 8, 6.9 ms over fp32 pages
// (the bf16 kernel over bf16 pages, which cuts rows into parts: 0.17 ms).
#include <cuda_fp16.h>

#include "qskv_kvf.cuh"
#include "qskv_prefill.cuh"

namespace qskv {
namespace {

constexpr int kRows = kPrefillFp32Rows, kThreads = 128;
// Blocks of 64 keys of 64 dims, two CTAs an SM: 52 us and 0.96 ms for the prompts above.  Three CTAs spill (54.6, 0.99);
// three or four on blocks of 32 take 69 and 0.89, or 89 and 0.87: better full, but a tile's blocks are then done one by one
// among more warps, and short prompts are as long as their longest tile.  128 dims leave room for 32 keys.
template <int D>
constexpr int kKeys = prefill_fp32_keys(D);
constexpr int kCtas = prefill_fp32_ctas(1);  // an SM

enum Cache { kF32 = 0, kBf16 = 1, kKvf = 2 };
template <int CACHE>
constexpr int kCacheParts = CACHE == kF32 ? 3 : 1;

template <int D, int QPARTS, int PARTS>
struct Smem {
    uint16_t q[QPARTS][kRows][D + 8], k[PARTS][kKeys<D>][D + 8], v[PARTS][kKeys<D>][D + 8];  // (8 more: rows 4 banks apart)
    PrefillItem item;
    int next;
};

// Parts of two numbers, as pairs of bf16: the next 8 bits each, as they are.
template <int PARTS>
__device__ __forceinline__ void cut(float x, float y, uint32_t (&p)[PARTS]) {
#pragma unroll
    for (int i = 0; i < PARTS; i++) {
        const uint32_t a = __float_as_uint(x), b = __float_as_uint(y);
        p[i] = __byte_perm(a, b, 0x7632);
        x -= __uint_as_float(a & 0xffff0000u), y -= __uint_as_float(b & 0xffff0000u);
    }
}

// The same, each part to nearest; CLAMP: also of numbers above the largest bf16 one.
template <bool CLAMP>
__device__ __forceinline__ void split(float x, float y, uint32_t (&p)[3]) {
    const float most = __uint_as_float(0x7f7f0000u);
#pragma unroll
    for (int i = 0; i < 3; i++) {
        p[i] = CLAMP && i == 0 ? pack_bf16x2(fminf(fmaxf(x, -most), most), fminf(fmaxf(y, -most), most)) : pack_bf16x2(x, y);
        x -= bf16_lo_to_float(p[i]), y -= bf16_hi_to_float(p[i]);
    }
}

template <int D>
constexpr int kPages = kKeys<D> / 16;  // pages of a block at most

// The pages of a block of the item's row, 16 tokens each; -1 where there is none.
template <int D>
__device__ __forceinline__ void pages_of(const PrefillArgs &a, int row, int block, int end, int (&ids)[kPages<D>]) {
    const int shift = a.page_size == 16 ? 4 : 5;
#pragma unroll
    for (int i = 0; i < kPages<D>; i++) {
        const int t = block * kKeys<D> + 16 * i;
        ids[i] = t < end ? __ldg(a.page_table + int64_t(row) * a.max_pages + (t >> shift)) : -1;
        if (ids[i] >= a.num_pool_pages) ids[i] = -1;
    }
}

// A thread's 4 dims of every (kThreads / (D / 4))th token: keys (which 0) or values of a block, zeros where there are none;
// as they lie in the cache until they are stored, so that nothing waits for them before.
template <int D, int CACHE>
struct Chunk {
    static constexpr int ROWS = kThreads / (D / 4), N = kKeys<D> / ROWS, PARTS = kCacheParts<CACHE>;
    uint4 x[N];  // fp32: 4 numbers; bf16: 4 in x, y; 8 bits: 4 codes in x, their power in y

    __device__ __forceinline__ void load(const PrefillArgs &a, const int (&ids)[kPages<D>], int g, int which, int block,
                                         int end) {
        const int P = a.page_size, c = threadIdx.x % (D / 4), r = threadIdx.x / (D / 4);
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int t = block * kKeys<D> + i * ROWS + r, p = ids[i * ROWS / 16];
            x[i] = make_uint4(0, 0, 0, 0);
            if (t >= end || p < 0) continue;
            const int64_t tile = int64_t(p) * a.num_kv_heads + g;
            const int64_t at = (tile * P + (t & (P - 1))) * D + c * 4;
            if constexpr (CACHE == kF32) {
                x[i] = __ldg(reinterpret_cast<const uint4 *>(static_cast<const float *>(which ? a.v_pool : a.k_pool) + at));
            } else if constexpr (CACHE == kBf16) {
                const uint2 w =
                    __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(which ? a.v_pool : a.k_pool) + at));
                x[i].x = w.x, x[i].y = w.y;
            } else {
                const int u = t & 15;
                const uint8_t *part = a.pool + (tile * (P >> 4) + ((t & (P - 1)) >> 4)) * kvf_part_bytes(D);
                if (which) {  // a row holds two tokens
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(
                        part + 16 * D + (u >> 1) * 2 * D + kvf_value_chunk<D>(c >> 1, u >> 1) * 16 + (c & 1) * 8));
                    x[i].x = w.x, x[i].z = w.y;
                } else {
                    x[i].x = __ldg(reinterpret_cast<const uint32_t *>(part + u * D + kvf_key_chunk<D>(c >> 2, u) * 16 + (c & 3) * 4));
                }
                x[i].y = __ldg(part + 32 * D + 16 * which + u);
            }
        }
    }
    __device__ __forceinline__ void store(uint16_t (&to)[PARTS][kKeys<D>][D + 8], int which) const {
        const int c = threadIdx.x % (D / 4), r = threadIdx.x / (D / 4);
#pragma unroll
        for (int i = 0; i < N; i++) {
            uint32_t u[PARTS], v[PARTS];
            if constexpr (CACHE == kF32) {
                cut(__uint_as_float(x[i].x), __uint_as_float(x[i].y), u);
                cut(__uint_as_float(x[i].z), __uint_as_float(x[i].w), v);
            } else if constexpr (CACHE == kBf16) {
                u[0] = x[i].x, v[0] = x[i].y;
            } else {
                // (blocks begin at even tokens and r's parity is the thread's: a token's codes are bytes of one parity)
                const uint32_t codes = which ? __byte_perm(x[i].x, x[i].z, (i * ROWS + r) & 1 ? 0x7531 : 0x6420) : x[i].x;
                const float power = kvf_power(x[i].y);
                const uint32_t lo = kvf_half2(codes), hi = kvf_half2(codes >> 16);
                const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
                const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                cut(y.x * power, y.y * power, u);
                cut(z.x * power, z.y * power, v);
            }
#pragma unroll
            for (int p = 0; p < PARTS; p++) *reinterpret_cast<uint2 *>(&to[p][i * ROWS + r][c * 4]) = make_uint2(u[p], v[p]);
        }
    }
};

// Four 8-column tiles += a (parts of 16 x 16) times b (parts of 16 x 32, a tile's in b[.][tile / 2][2 (tile % 2)..]): the
// product of the first parts in top, the others that count in rest, the small ones first.
template <int APARTS, int BPARTS>
__device__ __forceinline__ void multiply(float (&top)[4][4], float (&rest)[4][4], const uint32_t (&a)[APARTS][4],
                                         const uint32_t (&b)[BPARTS][2][4]) {
#pragma unroll
    for (int sum = 2; sum >= 0; sum--)
#pragma unroll
        for (int i = 0; i < APARTS; i++) {
            const int j = sum - i;
            if (j < 0 || j >= BPARTS) continue;
#pragma unroll
            for (int t = 0; t < 4; t++)
                mma_bf16_16816(sum ? rest[t] : top[t], a[i], b[j][t / 2][t % 2 * 2], b[j][t / 2][t % 2 * 2 + 1]);
        }
}

template <int D, int CACHE, bool QBF16>
__global__ void __launch_bounds__(kThreads, kCtas) prefill_fp32_kernel(PrefillArgs a) {
    constexpr int QPARTS = QBF16 ? 1 : 3, PARTS = kCacheParts<CACHE>, KEYS = kKeys<D>;
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D, QPARTS, PARTS> &s = *reinterpret_cast<Smem<D, QPARTS, PARTS> *>(raw);
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, G = a.group, shift = 31 - __clz(G);
    // ldmatrix rows: of queries and values (16 rows, then the next 8 columns), and of keys (8 rows by 16 columns, the next 8)
    const uint32_t q_at = smem_u32(&s.q[0][16 * warp + lane % 16][lane / 16 * 8]);
    const uint32_t k_at = smem_u32(&s.k[0][lane % 8 + lane / 16 * 8][lane / 8 % 2 * 8]);
    const uint32_t v_at = smem_u32(&s.v[0][lane % 16][lane / 16 * 8]);
    constexpr uint32_t kRow = (D + 8) * 2, kQPart = kRows * kRow, kPart = KEYS * kRow;
    pdl_trigger();
    pdl_wait();
    const int total = (a.direct ? a.batch : int(__ldcg(&a.plan->items))) * a.num_kv_heads;
    for (int round = 0;; round++) {
        if (tid == 0) s.next = a.direct ? round ? total : int(blockIdx.x) : int(atomicAdd(&a.plan->next, 1u));
        __syncthreads();
        const int next = s.next;
        if (next >= total) return;
        if (tid == 0 && !a.direct) s.item = a.items[next / a.num_kv_heads];
        if (tid == 0 && a.direct) {  // a row's only tile
            int len;
            s.item.row = next / a.num_kv_heads;
            prefill_row(a, next / a.num_kv_heads, s.item.token, s.item.tokens, len);
            s.item.pos = len - s.item.tokens, s.item.block0 = 0;
            s.item.block1 = s.item.tokens ? (len + KEYS - 1) / KEYS : 0;
        }
        __syncthreads();
        const PrefillItem it = s.item;
        const int g = next % a.num_kv_heads, rows = it.tokens * G, last = it.pos + it.tokens;  // keys the tile sees
        int ids[kPages<D>];
        Chunk<D, CACHE> ahead;
        if (it.block0 < it.block1) {
            pages_of<D>(a, it.row, it.block0, last, ids);
            ahead.load(a, ids, g, 0, it.block0, last);
        }
#pragma unroll 4
        for (int i = tid; i < kRows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = i % (D / 4);
            uint2 parts[QPARTS];
#pragma unroll
            for (int p = 0; p < QPARTS; p++) parts[p] = make_uint2(0, 0);
            if (r < rows) {
                const int64_t at = int64_t(it.token + (r >> shift)) * a.q_stride + (g * G + (r & (G - 1))) * D + c * 4;
                if constexpr (QBF16) {
                    parts[0] = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) + at));
                } else {
                    const float4 x = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + at));
                    uint32_t u[3], v[3];
                    split<true>(x.x, x.y, u);
                    split<true>(x.z, x.w, v);
#pragma unroll
                    for (int p = 0; p < 3; p++) parts[p] = make_uint2(u[p], v[p]);
                }
            }
#pragma unroll
            for (int p = 0; p < QPARTS; p++) *reinterpret_cast<uint2 *>(&s.q[p][r][c * 4]) = parts[p];
        }
        // the lane's rows of its warp's 16: lane / 4 and that + 8; columns 2 (lane % 4).. of every 8
        const int row0 = 16 * warp + lane / 4;
        const int pos[2] = {it.pos + (row0 >> shift), it.pos + ((row0 + 8) >> shift)};
        const int furthest = 16 * warp < rows ? it.pos + min((16 * warp + 15) >> shift, it.tokens - 1) : -1;  // of the warp
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f}, o[D / 8][4];
#pragma unroll
        for (int t = 0; t < D / 8; t++)
#pragma unroll
            for (int e = 0; e < 4; e++) o[t][e] = 0.f;
        if (it.block0 < it.block1) ahead.store(s.k, 0);
        __syncthreads();
        for (int block = it.block0; block < it.block1; block++) {
            const int key0 = block * KEYS;
            ahead.load(a, ids, g, 1, block, last);  // its values, while the logits are made
            float x[KEYS / 8][4];
#pragma unroll
            for (int part = 0; part < KEYS / 32; part++) {
                float top[4][4] = {}, rest[4][4] = {};
                if (key0 + 32 * part <= furthest) {
#pragma unroll 2
                    for (int c = 0; c < D; c += 16) {
                        uint32_t qa[QPARTS][4], kb[PARTS][2][4];
#pragma unroll
                        for (int p = 0; p < QPARTS; p++) ldmatrix_x4(qa[p], q_at + p * kQPart + c * 2);
#pragma unroll
                        for (int p = 0; p < PARTS; p++)
#pragma unroll
                            for (int i = 0; i < 2; i++) ldmatrix_x4(kb[p][i], k_at + p * kPart + (32 * part + 16 * i) * kRow + c * 2);
                        multiply(top, rest, qa, kb);
                    }
                }
#pragma unroll
                for (int t = 0; t < 4; t++)
#pragma unroll
                    for (int e = 0; e < 4; e++) x[4 * part + t][e] = top[t][e] + rest[t][e];
            }
            // places without a key: past the row's position, or of a page that is not there
#pragma unroll
            for (int i = 0; i < kPages<D>; i++)
                if (ids[i] < 0 && tid == 0 && key0 + 16 * i < last) raise_error(a.flags, kErrPageId);
            float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int t = 0; t < KEYS / 8; t++)
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    const bool there = ids[t / 2] >= 0 && key0 + 8 * t + 2 * (lane % 4) + e % 2 <= pos[e / 2];
                    x[t][e] = there ? x[t][e] * a.scale_log2 : -INFINITY;
                    top[e / 2] = fmaxf(top[e / 2], x[t][e]);
                }
            float base[2], down[2];
#pragma unroll
            for (int h = 0; h < 2; h++) {
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
                top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
                const float mn = fmaxf(m[h], top[h]);
                base[h] = mn == -INFINITY ? 0.f : mn;
                down[h] = exp2f(m[h] - base[h]);
                m[h] = mn, l[h] *= down[h];
            }
            uint32_t weights[KEYS / 16][3][4];  // the lane's part of 16 x 16 of them
#pragma unroll
            for (int t = 0; t < KEYS / 8; t++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float u = exp2f(x[t][2 * h] - base[h]), v = exp2f(x[t][2 * h + 1] - base[h]);
                    l[h] += u + v;
                    uint32_t parts[3];
                    split<false>(u, v, parts);
#pragma unroll
                    for (int p = 0; p < 3; p++) weights[t / 2][p][t % 2 * 2 + h] = parts[p];
                }
            ahead.store(s.v, 1);
            __syncthreads();
            if (block + 1 < it.block1) {  // the next keys, while the outputs are made
                pages_of<D>(a, it.row, block + 1, last, ids);
                ahead.load(a, ids, g, 0, block + 1, last);
            }
#pragma unroll
            for (int part = 0; part < D / 32; part++) {
                float top[4][4] = {}, rest[4][4] = {};
#pragma unroll
                for (int c = 0; c < KEYS / 16; c++) {
                    if (key0 + 16 * c > furthest) break;
                    uint32_t vb[PARTS][2][4];
#pragma unroll
                    for (int p = 0; p < PARTS; p++)
#pragma unroll
                        for (int i = 0; i < 2; i++)
                            ldmatrix_x4_trans(vb[p][i], v_at + p * kPart + 16 * c * kRow + (32 * part + 16 * i) * 2);
                    multiply(top, rest, weights[c], vb);
                }
#pragma unroll
                for (int t = 0; t < 4; t++)
#pragma unroll
                    for (int e = 0; e < 4; e++)
                        o[4 * part + t][e] = fmaf(o[4 * part + t][e], down[e / 2], top[t][e] + rest[t][e]);
            }
            if (block + 1 < it.block1) ahead.store(s.k, 0);
            __syncthreads();
        }
#pragma unroll
        for (int h = 0; h < 2; h++) {
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
            l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
            const int r = row0 + 8 * h;
            if (r >= rows) continue;
            const float inv = l[h] > 0.f ? 1.f / l[h] : 0.f;
            const int64_t head = int64_t(it.token + (r >> shift)) * a.num_q_heads + g * G + (r & (G - 1));
#pragma unroll
            for (int t = 0; t < D / 8; t++) {
                const int64_t at = head * D + 8 * t + 2 * (lane % 4);
                const float u = o[t][2 * h] * inv, v = o[t][2 * h + 1] * inv;
                if constexpr (QBF16)
                    *reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(a.out) + at) = pack_bf16x2(u, v);
                else
                    *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at) = make_float2(u, v);
            }
            if (a.lse && lane % 4 == 0) a.lse[head] = l[h] > 0.f ? (m[h] + log2f(l[h])) * 0.6931471805599453f : -INFINITY;
        }
        __syncthreads();
    }
}

template <int D, int CACHE, bool QBF16>
cudaError_t launch_one(const PrefillArgs &a, cudaStream_t stream) {
    auto kernel = prefill_fp32_kernel<D, CACHE, QBF16>;
    constexpr size_t bytes = sizeof(Smem<D, QBF16 ? 1 : 3, kCacheParts<CACHE>>);
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
    if (e != cudaSuccess) return e;
    const int64_t most = int64_t(a.direct ? a.batch : a.max_items) * a.num_kv_heads, ctas = prefill_fp32_ctas(a.num_sms);
    return launch_pdl(kernel, dim3(unsigned(most < ctas ? most : ctas)), dim3(kThreads), bytes, stream, a);
}

template <int D>
cudaError_t launch_dim(const PrefillArgs &a, int q_dtype, int kv_dtype, cudaStream_t stream) {
    if (a.pool) return launch_one<D, kKvf, false>(a, stream);  // bf16 queries over these two: the tensor cores' kernel
    if (kv_dtype == kDtypeBf16) return launch_one<D, kBf16, false>(a, stream);
    return q_dtype == kDtypeBf16 ? launch_one<D, kF32, true>(a, stream) : launch_one<D, kF32, false>(a, stream);
}

}  // namespace

cudaError_t launch_prefill_fp32(const PrefillArgs &a, int q_dtype, int kv_dtype, int head_dim, cudaStream_t stream) {
    return head_dim == 128 ? launch_dim<128>(a, q_dtype, kv_dtype, stream) : launch_dim<64>(a, q_dtype, kv_dtype, stream);
}

}  // namespace qskv
