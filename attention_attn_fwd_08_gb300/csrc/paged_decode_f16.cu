// paged_decode_f16.cu -- the paged decode's kernels for 16-bit pools of fp16.
#include "paged_decode.cuh"

namespace attn {

cudaError_t launch_paged_decode_f16(const PagedParams& p, bool bf16, const PagedMaps& maps, cudaStream_t s) {
    return paged::decode_hd<CACHE_16, false>(p, bf16, maps, s);
}

}  // namespace attn
