// The 4-bit decode for pages of 16 tokens, and the choice between page sizes.
#include "kvq_decode.cuh"

namespace qskv {

int kvq_decode_ctas(int num_sms) { return 2 * num_sms; }
int kvq_decode_warps() { return kWarps; }

cudaError_t launch_kvq_decode(KvqDecodeArgs a, int head_dim, int num_sms, cudaStream_t stream) {
    return a.page_size == 16 ? launch_page<16>(a, head_dim, num_sms, stream)
                             : launch_kvq_decode_page32(a, head_dim, num_sms, stream);
}

}  // namespace qskv
