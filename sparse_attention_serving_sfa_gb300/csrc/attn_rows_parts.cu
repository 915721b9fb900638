// Attention of a few query rows over parts of a sequence's keys: through a sliding
// window with sinks, or in the two phases behind a shared prefix (attn_rows.cuh).
#include "attn_rows.cuh"

namespace sfa {

cudaError_t launch_attn_rows_parts(const SeqAttn& p, sfa_dtype dtype, int num_sms, cudaStream_t stream) {
    return launch_rows<true>(p, dtype, num_sms, stream);
}

}  // namespace sfa
