// Prefill in fp32 arithmetic (qskv_prefill.cuh), for fp32 queries over any
// cache and bf16 queries over an fp32 one: what the tensor cores' bf16 operands
// would cut.
//
// Bound: fp32 FMAs, 4 d a (query head, key) pair.  A CTA takes 64 rows of
// queries against 64 keys at a time.  A thread's 8 x 4 logits and 8 x (d / 16)
// outputs are in registers, so 128 FMAs need 12 vector loads from shared
// memory, 256 need 16.  Keys and values take turns in two buffers: what is
// needed next is read into registers before the products and stored after them.
// One GB300: 6 prompts of up to 500 tokens, 16 heads of 64 dims, in 82 us, where
// the few tiles of up to 9 blocks bound it.
#include <cuda_fp16.h>

#include "qskv_kvf.cuh"
#include "qskv_prefill.cuh"

namespace qskv {
namespace {

constexpr int kRows = kPrefillSimtRows, kKeys = kPrefillSimtKeys, kThreads = 128;

template <int D>
struct Smem {
    float q[kRows][D + 4], k[kKeys][D + 4], v[kKeys][D + 4];
    float p[D == 64 ? kRows : 1][kKeys + 4];  // d = 128: weights lie over the keys, so that two CTAs fit an SM
    PrefillItem item;
    int next;
};

enum Cache { kF32 = 0, kBf16 = 1, kKvf = 2 };

constexpr int kPages = kKeys / 16;  // pages of a block at most

// The pages of a block of the item's row, 16 tokens each; -1 where there is none.
__device__ __forceinline__ void pages_of(const PrefillArgs &a, int row, int block, int end, int (&ids)[kPages]) {
    const int shift = a.page_size == 16 ? 4 : 5;
#pragma unroll
    for (int i = 0; i < kPages; i++) {
        const int t = block * kKeys + 16 * i;
        ids[i] = t < end ? __ldg(a.page_table + int64_t(row) * a.max_pages + (t >> shift)) : -1;
        if (ids[i] >= a.num_pool_pages) ids[i] = -1;
    }
}

// A thread's 4 dims of every (kThreads / (D / 4))th token: keys (which 0) or values of a block, zeros where there are none.
template <int D>
struct Chunk {
    static constexpr int ROWS = kThreads / (D / 4), N = kKeys / ROWS;
    float4 x[N];

    template <int CACHE>
    __device__ __forceinline__ void load(const PrefillArgs &a, const int (&ids)[kPages], int g, int which, int block, int end) {
        const int P = a.page_size, c = threadIdx.x % (D / 4), r = threadIdx.x / (D / 4);
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int k = i * ROWS + r, t = block * kKeys + k, p = ids[i * ROWS / 16];
            x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (t >= end || p < 0) continue;
            const int64_t tile = int64_t(p) * a.num_kv_heads + g;
            const int64_t at = (tile * P + (t & (P - 1))) * D + c * 4;
            if constexpr (CACHE == kF32) {
                x[i] = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(which ? a.v_pool : a.k_pool) + at));
            } else if constexpr (CACHE == kBf16) {
                const uint2 w =
                    __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(which ? a.v_pool : a.k_pool) + at));
                x[i] = make_float4(bf16_lo_to_float(w.x), bf16_hi_to_float(w.x), bf16_lo_to_float(w.y), bf16_hi_to_float(w.y));
            } else {
                const int u = t & 15;
                const uint8_t *part = a.pool + (tile * (P >> 4) + ((t & (P - 1)) >> 4)) * kvf_part_bytes(D);
                uint32_t codes;
                if (which) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(
                        part + 16 * D + (u >> 1) * 2 * D + kvf_value_chunk<D>(c >> 1, u >> 1) * 16 + (c & 1) * 8));
                    codes = __byte_perm(w.x, w.y, u & 1 ? 0x7531 : 0x6420);
                } else {
                    codes = __ldg(reinterpret_cast<const uint32_t *>(part + u * D + kvf_key_chunk<D>(c >> 2, u) * 16 + (c & 3) * 4));
                }
                const float power = kvf_power(__ldg(part + 32 * D + 16 * which + u));
                const uint32_t lo = kvf_half2(codes), hi = kvf_half2(codes >> 16);
                const float2 y = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
                const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
                x[i] = make_float4(y.x * power, y.y * power, z.x * power, z.y * power);
            }
        }
    }
    __device__ __forceinline__ void store(float (&to)[kKeys][D + 4]) const {
        const int c = threadIdx.x % (D / 4), r = threadIdx.x / (D / 4);
#pragma unroll
        for (int i = 0; i < N; i++) *reinterpret_cast<float4 *>(&to[i * ROWS + r][c * 4]) = x[i];
    }
};

// Thread (ty, tx) of 8 x 16 owns rows 8 ty .. 8 ty + 7 of the tile, keys tx + 16 j and dims 4 tx + 64 j ..
template <int D, int CACHE, bool QBF16>
__global__ void __launch_bounds__(kThreads) prefill_simt_kernel(PrefillArgs a) {
    extern __shared__ __align__(16) uint8_t raw[];
    Smem<D> &s = *reinterpret_cast<Smem<D> *>(raw);
    const int tid = threadIdx.x, ty = tid / 16, tx = tid % 16, G = a.group;
    float(*const weights)[kKeys + 4] = D == 64 ? s.p : reinterpret_cast<float(*)[kKeys + 4]>(s.k);
    pdl_trigger();
    pdl_wait();
    const int total = int(__ldcg(&a.plan->items)) * a.num_kv_heads;
    while (true) {
        if (tid == 0) s.next = int(atomicAdd(&a.plan->next, 1u));
        __syncthreads();
        const int next = s.next;
        if (next >= total) return;
        if (tid == 0) s.item = a.items[next / a.num_kv_heads];
        __syncthreads();
        const PrefillItem it = s.item;
        const int g = next % a.num_kv_heads, rows = it.tokens * G, last = it.pos + it.tokens;  // keys the tile sees
        auto head_of = [&](int r) { return (int64_t(it.token + r / G) * a.num_q_heads) + g * G + r % G; };
        for (int i = tid; i < kRows * (D / 4); i += kThreads) {
            const int r = i / (D / 4), c = i % (D / 4);
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            if (r < rows) {
                const int64_t at = int64_t(it.token + r / G) * a.q_stride + (g * G + r % G) * D + c * 4;
                if constexpr (QBF16) {
                    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.q) + at));
                    x = make_float4(bf16_lo_to_float(w.x), bf16_hi_to_float(w.x), bf16_lo_to_float(w.y),
                                    bf16_hi_to_float(w.y));
                } else {
                    x = __ldg(reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + at));
                }
            }
            *reinterpret_cast<float4 *>(&s.q[r][c * 4]) = x;
        }
        float m[8], l[8], o[8][D / 16];
#pragma unroll
        for (int r = 0; r < 8; r++) {
            m[r] = -INFINITY, l[r] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; i++) o[r][i] = 0.f;
        }
        int ids[kPages];
        Chunk<D> ahead;
        if (it.block0 < it.block1) {
            pages_of(a, it.row, it.block0, last, ids);
            ahead.template load<CACHE>(a, ids, g, 0, it.block0, last);
            ahead.store(s.k);
        }
        __syncthreads();
        for (int block = it.block0; block < it.block1; block++) {
            ahead.template load<CACHE>(a, ids, g, 1, block, last);  // its values, while the logits are made
            float x[8][4];
#pragma unroll
            for (int r = 0; r < 8; r++)
#pragma unroll
                for (int j = 0; j < 4; j++) x[r][j] = 0.f;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
                float4 k[4];
#pragma unroll
                for (int j = 0; j < 4; j++) k[j] = *reinterpret_cast<const float4 *>(&s.k[tx + 16 * j][c]);
#pragma unroll
                for (int r = 0; r < 8; r++) {
                    const float4 q = *reinterpret_cast<const float4 *>(&s.q[8 * ty + r][c]);
#pragma unroll
                    for (int j = 0; j < 4; j++)
                        x[r][j] = fmaf(q.w, k[j].w, fmaf(q.z, k[j].z, fmaf(q.y, k[j].y, fmaf(q.x, k[j].x, x[r][j]))));
                }
            }
            if (D == 128) __syncthreads();
            // places without a key: past the row's position, or of a page that is not there
            bool there[4];
#pragma unroll
            for (int j = 0; j < 4; j++) {  // (keys tx + 16 j lie in the block's page j)
                there[j] = ids[j] >= 0;
                if (!there[j] && tx == 0 && block * kKeys + 16 * j < last) raise_error(a.flags, kErrPageId);
            }
#pragma unroll
            for (int r = 0; r < 8; r++) {
                const int pos = it.pos + (8 * ty + r) / G;
                float top = -INFINITY;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    x[r][j] = there[j] && block * kKeys + tx + 16 * j <= pos ? x[r][j] * a.scale_log2 : -INFINITY;
                    top = fmaxf(top, x[r][j]);
                }
#pragma unroll
                for (int i = 1; i < 16; i <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, i));
                const float mn = fmaxf(m[r], top), base = mn == -INFINITY ? 0.f : mn;
                const float down = exp2f(m[r] - base);
                m[r] = mn, l[r] *= down;
#pragma unroll
                for (int i = 0; i < D / 16; i++) o[r][i] *= down;
#pragma unroll
                for (int j = 0; j < 4; j++) {
                    const float p = exp2f(x[r][j] - base);
                    l[r] += p;
                    weights[8 * ty + r][tx + 16 * j] = p;
                }
            }
            ahead.store(s.v);
            __syncthreads();
            if (block + 1 < it.block1) {  // the next keys, while the outputs are made
                pages_of(a, it.row, block + 1, last, ids);
                ahead.template load<CACHE>(a, ids, g, 0, block + 1, last);
            }
#pragma unroll 2
            for (int k = 0; k < kKeys; k += 4) {
                float4 p[8];
#pragma unroll
                for (int r = 0; r < 8; r++) p[r] = *reinterpret_cast<const float4 *>(&weights[8 * ty + r][k]);
#pragma unroll
                for (int e = 0; e < 4; e++) {
#pragma unroll
                    for (int i = 0; i < D / 64; i++) {
                        const float4 v = *reinterpret_cast<const float4 *>(&s.v[k + e][64 * i + 4 * tx]);
#pragma unroll
                        for (int r = 0; r < 8; r++) {
                            const float w = e == 0 ? p[r].x : e == 1 ? p[r].y : e == 2 ? p[r].z : p[r].w;
                            o[r][4 * i] = fmaf(w, v.x, o[r][4 * i]), o[r][4 * i + 1] = fmaf(w, v.y, o[r][4 * i + 1]);
                            o[r][4 * i + 2] = fmaf(w, v.z, o[r][4 * i + 2]);
                            o[r][4 * i + 3] = fmaf(w, v.w, o[r][4 * i + 3]);
                        }
                    }
                }
            }
            if (D == 128) __syncthreads();
            if (block + 1 < it.block1) ahead.store(s.k);
            __syncthreads();
        }
#pragma unroll
        for (int r = 0; r < 8; r++) {
#pragma unroll
            for (int i = 1; i < 16; i <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], i);
            const int row = 8 * ty + r;
            if (row >= rows) continue;
            const float inv = l[r] > 0.f ? 1.f / l[r] : 0.f;
            const int64_t head = head_of(row);
#pragma unroll
            for (int i = 0; i < D / 64; i++) {
                const float4 v = make_float4(o[r][4 * i] * inv, o[r][4 * i + 1] * inv, o[r][4 * i + 2] * inv,
                                             o[r][4 * i + 3] * inv);
                const int64_t at = head * D + 64 * i + 4 * tx;
                if constexpr (QBF16)
                    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
                        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                else
                    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = v;
            }
            if (a.lse && tx == 0) a.lse[head] = l[r] > 0.f ? (m[r] + log2f(l[r])) * 0.6931471805599453f : -INFINITY;
        }
        __syncthreads();
    }
}

template <int D, int CACHE, bool QBF16>
cudaError_t launch_one(const PrefillArgs &a, cudaStream_t stream) {
    auto kernel = prefill_simt_kernel<D, CACHE, QBF16>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(sizeof(Smem<D>)));
    if (e != cudaSuccess) return e;
    const int64_t most = int64_t(a.max_items) * a.num_kv_heads, ctas = 2 * a.num_sms;
    return launch_pdl(kernel, dim3(unsigned(most < ctas ? most : ctas)), dim3(kThreads), sizeof(Smem<D>), stream, a);
}

template <int D>
cudaError_t launch_dim(const PrefillArgs &a, int q_dtype, int kv_dtype, cudaStream_t stream) {
    if (a.pool) return launch_one<D, kKvf, false>(a, stream);  // bf16 queries over these two: the tensor cores' kernel
    if (kv_dtype == kDtypeBf16) return launch_one<D, kBf16, false>(a, stream);
    return q_dtype == kDtypeBf16 ? launch_one<D, kF32, true>(a, stream) : launch_one<D, kF32, false>(a, stream);
}

}  // namespace

cudaError_t launch_prefill_simt(const PrefillArgs &a, int q_dtype, int kv_dtype, int head_dim, cudaStream_t stream) {
    return head_dim == 128 ? launch_dim<128>(a, q_dtype, kv_dtype, stream) : launch_dim<64>(a, q_dtype, kv_dtype, stream);
}

}  // namespace qskv
