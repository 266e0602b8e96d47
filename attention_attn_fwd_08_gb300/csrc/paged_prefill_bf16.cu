// paged_prefill_bf16.cu -- instantiations of paged_prefill.cuh, and its workspace's size.
#include "paged_prefill.cuh"

namespace attn {
cudaError_t launch_paged_prefill_bf16(const PagedParams& p, int cache, const PrefillMaps& maps, cudaStream_t s) {
    return prefill::launch_hd<true, false>(p, cache, maps, s);
}
size_t paged_prefill_workspace(int total, int B, int G, int hd) {
    const int tiles = hd == 256 ? 1 : 2;
    return prefill::plan_bytes(total, B, tiles * (prefill::kM / G)) + prefill::part_bytes(tiles * prefill::kM, hd);
}
}  // namespace attn
