// Attention of many query rows over all of a sequence's keys (attn_tc.cuh).
#include "attn_tc.cuh"

namespace sfa {

bool attn_tc_supported(const SeqKV& kv, int G) {
    // (a gathered row is named by a 32-bit number)
    return G <= kTileM &&
           (!kv.page_table || (int64_t)kv.num_pages * kv.page_size * kv.Hkv < 0xffffffffLL);
}

size_t attn_tc_ws_bytes(int G, int D) {
    return G <= kTileM ? (size_t)2 * kMaxCtas * kItemRows * (D + 2) * 4 + kMaxCtas * sizeof(CutItem) : 0;
}

cudaError_t launch_attn_tc(const SeqAttn& a, sfa_dtype dtype, int num_sms, cudaStream_t stream) {
    return launch_tc<false>(a, dtype, num_sms, stream);
}

}  // namespace sfa
