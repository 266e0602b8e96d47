// paged_decode_e4m3.cu -- the paged decode's kernels for 8-bit pools, e4m3.
#include "paged_decode.cuh"

namespace attn {

cudaError_t launch_paged_decode_e4m3(const PagedParams& p, bool bf16, const PagedMaps& maps, cudaStream_t s) {
    return paged::decode_hd<CACHE_E4M3, false>(p, bf16, maps, s);
}

}  // namespace attn
