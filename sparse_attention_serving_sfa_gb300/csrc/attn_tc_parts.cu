// Attention of many query rows over parts of a sequence's keys: through a sliding
// window with sinks, or in the two phases behind a shared prefix (attn_tc.cuh).
#include "attn_tc.cuh"

namespace sfa {

cudaError_t launch_attn_tc_parts(const SeqAttn& a, sfa_dtype dtype, int num_sms, cudaStream_t stream) {
    return launch_tc<true>(a, dtype, num_sms, stream);
}

}  // namespace sfa
