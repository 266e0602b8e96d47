// paged_prefill_bf16_f8.cu -- instantiations of paged_prefill.cuh.
#include "paged_prefill.cuh"

namespace attn {
cudaError_t launch_paged_prefill_bf16_f8(const PagedParams& p, int cache, const PrefillMaps& maps, cudaStream_t s) {
    return prefill::launch_hd<true, true>(p, cache, maps, s);
}
}  // namespace attn
