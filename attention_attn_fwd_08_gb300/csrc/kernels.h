// kernels.h -- launchers the C ABI layer (api.cu) dispatches to.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace attn {

// dt: 0 = fp32, 1 = fp16, 2 = bf16 (the attn_dtype values).
cudaError_t launch_simt_fwd(const Params& p, int dt, cudaStream_t s);
// phases: bit 1 = D = rowsum(dO*O), bit 2 = dK/dV, bit 4 = dQ
cudaError_t launch_simt_bwd(const Params& p, int dt, int phases, cudaStream_t s);
cudaError_t launch_bwd_preprocess(const Params& p, int dt, cudaStream_t s);

// tcgen05 prefill forward / backward (fp16 / bf16; hd 64 or 128, and 32 / 96 through
// 4-D maps padded to 64 / 128).  The tensor maps are built by the caller.
struct FwdMaps {
    CUtensorMap q, k, v;
    CUtensorMap o;  // 32-row boxes, for the epilogue's stores
};
cudaError_t launch_tc_fwd_bf16(const Params& p, const FwdMaps& maps, cudaStream_t s);  // fwd_tc_bf16.cu
cudaError_t launch_tc_fwd_f16(const Params& p, const FwdMaps& maps, cudaStream_t s);   // fwd_tc_f16.cu
inline cudaError_t launch_tc_fwd(const Params& p, int dt, const FwdMaps& maps, cudaStream_t s) {
    return dt == 2 ? launch_tc_fwd_bf16(p, maps, s) : launch_tc_fwd_f16(p, maps, s);
}
struct BwdMaps {
    CUtensorMap q, dout, k, v;          // 128-row boxes
    CUtensorMap q64, dout64, k64, v64;  // 64-row boxes
    CUtensorMap o;                      // 128-row boxes (D = rowsum(dO*O) in the dQ pass)
    CUtensorMap dq32, dk32, dv32;       // 32-row boxes, for the epilogues' stores
};
cudaError_t launch_tc_bwd_bf16(const Params& p, const BwdMaps& maps, int phases, cudaStream_t s);  // bwd_tc_bf16.cu
cudaError_t launch_tc_bwd_f16(const Params& p, const BwdMaps& maps, int phases, cudaStream_t s);   // bwd_tc_f16.cu
inline cudaError_t launch_tc_bwd(const Params& p, int dt, const BwdMaps& maps, int phases, cudaStream_t s) {
    return dt == 2 ? launch_tc_bwd_bf16(p, maps, phases, s) : launch_tc_bwd_f16(p, maps, phases, s);
}

// split-KV decode (fp16 / bf16, hd 64 or 128).
struct DecMaps {
    CUtensorMap k, v;
};
cudaError_t launch_decode(const Params& p, int dt, const DecMaps& maps, cudaStream_t s);

// Fixed scratch for attn_decode_noalloc (split partials), defined in decode.cu.
constexpr size_t kDecodeScratchBytes = size_t(32) << 20;
// Device address of that scratch on the current device (looked up once per device).
cudaError_t decode_noalloc_scratch(float** out);

cudaError_t launch_selftest_wait(unsigned int* status, unsigned int timeout_us, cudaStream_t s);

// rotate-half rotary embedding of src [B][T][H*hd] into dst (src == dst: in place), hd 8 .. 256
// a multiple of 4; inverse turns every pair the other way
cudaError_t launch_rope(const void* src, void* dst, int dt, int B, int T, int H, int hd, int pos, double theta,
                        bool inverse, cudaStream_t s);
// cosine/sine table of rotary positions pos .. pos+npos-1 for the forward's fused rotation
cudaError_t launch_rope_table(float* tab, int npos, int hd, int pos, double theta, cudaStream_t s);

// rotary positions in every form (rope_ex.cu); fields as attn_rope_ex's arguments
struct RopeExCall {
    const void* x;
    void* y;
    long long x_stride, y_stride;
    const int* positions;
    const double* inv_freq;
    int pos, period, rows, H, hd, rotary_dim, rotary_start;
    bool interleaved, backward;
    float amplitude;
};
cudaError_t launch_rope_ex(const RopeExCall& c, int dt, cudaStream_t s);

// ---- paged key/value cache (paged.cu, paged_decode.cu): fp16 / bf16 rows, hd 64, 128 or 256
enum : int { CACHE_16 = 0, CACHE_E4M3 = 1, CACHE_E5M2 = 2 };  // element type of the pages (16: that of the rows)
// status bit, after those of common.cuh (which the dense kernels' captured figures are tied to, byte by byte)
enum : unsigned int { ST_PAGED_BOUNDS = 1u << 10 };  // a paged call's page, length or prefix sum outside its range
struct PagedParams {
    const void* q;  // append: rows to turn, or NULL; decode: [B][Lq][H*hd]
    const void* k;  // append: new rows
    const void* v;
    void* q_out;
    long long q_stride, k_stride, v_stride;  // elements from row to row
    void* k_cache;                           // [num_pages][Hkv][page_size][hd]
    void* v_cache;
    float* k_scale;  // [num_pages][Hkv], 8-bit pages only
    float* v_scale;
    void* k_out;  // gather
    void* v_out;
    void* o;  // decode
    float* lse;
    float* ws;
    const int* cu;       // append, gather: packed rows of the sequences
    const int* lengths;  // append, decode: valid tokens of each sequence
    const int* table;    // [B][max_pages]
    int B, Lq, total, num_pages, page_size, page_shift, max_pages, H, Hkv, G, hd;
    float scale, softcap;
    int wl, wr;
    unsigned int* status;
};
// bf16: type of the 16-bit rows; theta = 0: nothing is turned
cudaError_t launch_paged_append(const PagedParams& p, bool bf16, int cache, double theta, cudaStream_t s);
cudaError_t launch_paged_gather(const PagedParams& p, bool bf16, int cache, cudaStream_t s);
// 2-D maps over the pools' rows, boxes of up to 128 bytes by min(page_size, 64) rows
struct PagedMaps {
    CUtensorMap k, v;
};
size_t paged_decode_workspace(int rows, int hd);
cudaError_t launch_paged_decode_bf16(const PagedParams& p, bool bf16, const PagedMaps& maps, cudaStream_t s);
cudaError_t launch_paged_decode_f16(const PagedParams& p, bool bf16, const PagedMaps& maps, cudaStream_t s);
cudaError_t launch_paged_decode_e4m3(const PagedParams& p, bool bf16, const PagedMaps& maps, cudaStream_t s);
cudaError_t launch_paged_decode_e5m2(const PagedParams& p, bool bf16, const PagedMaps& maps, cudaStream_t s);
inline cudaError_t launch_paged_decode(const PagedParams& p, bool bf16, int cache, const PagedMaps& maps, cudaStream_t s) {
    if (cache == CACHE_E4M3) return launch_paged_decode_e4m3(p, bf16, maps, s);
    if (cache == CACHE_E5M2) return launch_paged_decode_e5m2(p, bf16, maps, s);
    return bf16 ? launch_paged_decode_bf16(p, bf16, maps, s) : launch_paged_decode_f16(p, bf16, maps, s);
}

// attention of a chunk of new tokens over the pages (paged_prefill.cuh): q rows packed by cu, q_stride apart
constexpr int kPrefillCtas = 152;
struct PrefillMaps {
    CUtensorMap q;     // [rows][H][hd], boxes of 64 columns by G heads by 128 / G rows
    CUtensorMap k, v;  // as PagedMaps
};
cudaError_t launch_paged_prefill_bf16(const PagedParams& p, int cache, const PrefillMaps& maps, cudaStream_t s);
cudaError_t launch_paged_prefill_f16(const PagedParams& p, int cache, const PrefillMaps& maps, cudaStream_t s);
cudaError_t launch_paged_prefill_bf16_f8(const PagedParams& p, int cache, const PrefillMaps& maps, cudaStream_t s);
cudaError_t launch_paged_prefill_f16_f8(const PagedParams& p, int cache, const PrefillMaps& maps, cudaStream_t s);
inline cudaError_t launch_paged_prefill(const PagedParams& p, bool bf16, int cache, const PrefillMaps& maps, cudaStream_t s) {
    if (cache == CACHE_16) return bf16 ? launch_paged_prefill_bf16(p, cache, maps, s) : launch_paged_prefill_f16(p, cache, maps, s);
    return bf16 ? launch_paged_prefill_bf16_f8(p, cache, maps, s) : launch_paged_prefill_f16_f8(p, cache, maps, s);
}
// The layout of PagedParams::ws, whose partial rows are stored 32 bytes at a time, begins on a multiple of kPrefillAlign.
constexpr size_t kPrefillAlign = 256;
size_t paged_prefill_workspace(int total, int B, int G, int hd);

}  // namespace attn
