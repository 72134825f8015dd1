// The 4-bit decode for pages of 32 tokens (a file of its own, so that the two compile side by side).
#include "kvq_decode.cuh"

namespace qskv {

cudaError_t launch_kvq_decode_page32(KvqDecodeArgs a, int head_dim, int num_sms, cudaStream_t stream) {
    return launch_page<32>(a, head_dim, num_sms, stream);
}

}  // namespace qskv
