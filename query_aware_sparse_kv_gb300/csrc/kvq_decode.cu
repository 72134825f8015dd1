// Attention of one query token a sequence over the 4-bit paged cache (format:
// qskv_kvq.cuh).
//
// With k = m + s u per group j of dims, the logit of token t is
//     l_t = scale * sum_j (s_tj (q_j . u_tj) + m_tj sum(q_j)),
// and the output sum_t p_t (m_tj + s_tj u_t) over softmax weights p.
#include "qskv_internal.h"
#include "qskv_kvq.cuh"

namespace qskv {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// One CTA per (sequence, KV head), one thread per dim, one head and token at
// a time with a running maximum and sum.
template <int D>
__global__ void __launch_bounds__(D) kvq_decode_kernel(KvqDecodeArgs a) {
    __shared__ float part[D / 32];
    pdl_trigger();
    pdl_wait();
    const int row = blockIdx.x, b = row / a.num_kv_heads, g = row % a.num_kv_heads, c = threadIdx.x;
    const int P = a.page_size, ng = D / a.group_size, w = c / 8, j = c / a.group_size;
    int seq = a.seq_lens[b];
    if (seq < 0 || seq > a.max_pages * P) {
        if (c == 0) raise_error(a.flags, kErrSeqLen);
        seq = seq < 0 ? 0 : a.max_pages * P;
    }
    const int n_b = (seq + P - 1) / P;
    int n = n_b;
    if (a.selected) {
        n = a.n_selected[row];
        const int lim = min(a.top_k, n_b);
        if (n < 0 || n > lim) {
            if (c == 0) raise_error(a.flags, kErrSelected);
            n = max(0, min(n, lim));
        }
    }
    for (int h = 0; h < a.group; h++) {
        const int64_t at = (int64_t(b) * a.num_q_heads + g * a.group + h) * D + c;
        const float q = a.q_is_bf16 ? __uint_as_float(uint32_t(static_cast<const uint16_t *>(a.q)[at]) << 16)
                                    : static_cast<const float *>(a.q)[at];
        float top = -1e30f, sum = 0.f, o = 0.f;
        for (int i = 0; i < n; i++) {
            const int page = a.selected ? a.selected[int64_t(row) * a.top_k + i] : i;
            if (page < 0 || page >= n_b) {
                if (c == 0) raise_error(a.flags, kErrSelected);
                continue;
            }
            const int id = a.page_table[int64_t(b) * a.max_pages + page];
            if (id < 0 || id >= a.num_pool_pages) {
                if (c == 0) raise_error(a.flags, kErrPageId);
                continue;
            }
            const uint32_t *block = a.pool + (int64_t(id) * a.num_kv_heads + g) * kvq_block_words(D, P, ng);
            for (int t = 0; t < min(P, seq - page * P); t++) {
                const uint32_t kw = block[t * (D / 8) + kvq_key_place<D>(w)];
                const uint32_t vw = block[(P + t) * (D / 8) + kvq_value_place<D>(w, t)];
                const uint32_t kp = block[2 * P * (D / 8) + j * P + t], vp = block[2 * P * (D / 8) + (ng + j) * P + t];
                const float k = fmaf(float((kw >> (c % 8 * 4)) & 15u), bf16_lo_to_float(kp), bf16_hi_to_float(kp));
                const float v = fmaf(float((vw >> (c % 8 * 4)) & 15u), bf16_lo_to_float(vp), bf16_hi_to_float(vp));
                float x = q * k;
                for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
                __syncthreads();
                if (c % 32 == 0) part[c / 32] = x;
                __syncthreads();
                x = 0.f;
                for (int d = 0; d < D / 32; d++) x += part[d];
                x *= a.scale_log2;
                const float m = fmaxf(top, x), f = exp2f(top - m), p = exp2f(x - m);
                sum = sum * f + p, o = o * f + p * v, top = m;
            }
        }
        a.out[at] = sum > 0.f ? o / sum : 0.f;
        if (c == 0 && a.lse) a.lse[at / D] = sum > 0.f ? (top + log2f(sum)) * kLn2 : -INFINITY;
    }
}

}  // namespace

cudaError_t launch_kvq_decode(const KvqDecodeArgs &a, int head_dim, cudaStream_t stream) {
    const dim3 grid(unsigned(a.batch * a.num_kv_heads));
    return head_dim == 128 ? launch_pdl(kvq_decode_kernel<128>, grid, dim3(128), 0, stream, a)
                           : launch_pdl(kvq_decode_kernel<64>, grid, dim3(64), 0, stream, a);
}

}  // namespace qskv
