// Attention of a few query rows over all of a sequence's keys (attn_rows.cuh).
#include "attn_rows.cuh"

namespace sfa {

size_t attn_rows_ws_bytes(int D) { return (size_t)2 * kMaxCtas * kRows * (D + 2) * 4; }

cudaError_t launch_attn_rows(const SeqAttn& p, sfa_dtype dtype, int num_sms, cudaStream_t stream) {
    return launch_rows<false>(p, dtype, num_sms, stream);
}

}  // namespace sfa
