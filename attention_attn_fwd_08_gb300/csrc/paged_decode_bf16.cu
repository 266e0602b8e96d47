// paged_decode_bf16.cu -- the paged decode's kernels for 16-bit pools of bfloat16, and the
// workspace they share with the other types'.
#include "paged_decode.cuh"

namespace attn {

size_t paged_decode_workspace(int rows, int hd) { return paged::ws_bytes(rows, hd); }

cudaError_t launch_paged_decode_bf16(const PagedParams& p, bool bf16, const PagedMaps& maps, cudaStream_t s) {
    return paged::decode_hd<CACHE_16, true>(p, bf16, maps, s);
}

}  // namespace attn
