// paged_prefill_f16.cu -- instantiations of paged_prefill.cuh.
#include "paged_prefill.cuh"

namespace attn {
cudaError_t launch_paged_prefill_f16(const PagedParams& p, int cache, const PrefillMaps& maps, cudaStream_t s) {
    return prefill::launch_hd<false, false>(p, cache, maps, s);
}
}  // namespace attn
