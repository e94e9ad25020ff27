// smr_ffn8.cu -- the experts' products on E4M3 operands with one fp32 scale per
// 128 values of a row and per 128 x 128 block of a weight (the kernel is
// smr_ffn.cuh's).
#include "smr_ffn.cuh"

namespace smr {

template <bool UP, bool F32>
static cudaError_t launch_rows(const FfnLaunch &a, int sms, cudaStream_t stream) {
    if (expert_pairs(a.numel, a.num_experts)) return launch_product<false, UP, true, 1, F32, true>(a, sms, stream);
    return a.A == 64 ? launch_product<false, UP, false, 2, F32, true>(a, sms, stream)
                     : launch_product<false, UP, false, 1, F32, true>(a, sms, stream);
}

cudaError_t launch_expert_product_fp8(const FfnLaunch &a, int sms, cudaStream_t stream) {
    if (a.gated) return launch_rows<true, false>(a, sms, stream);
    return a.out32 ? launch_rows<false, true>(a, sms, stream) : launch_rows<false, false>(a, sms, stream);
}

}  // namespace smr
