// Paged key/value cache: derived sizes and launchers.
#pragma once

#include "common.cuh"

namespace nsa {

struct PagedShape {
    int B, Tq, Hq, Hkv, G, dqk, dv;
    int P, logP;        // tokens per page, its log2
    int n_pages, cols;  // pages of the pool, columns of the table
    int win;            // 0: no window
    int ns;             // sink tokens
    float scale;
};

// Attention of the newest tokens (paged_attn.cu); ws: paged_attn_ws_bytes().
size_t paged_attn_ws_bytes(const PagedShape& s);
cudaError_t launch_paged_attn(const PagedShape& s, const __nv_bfloat16* q, const __nv_bfloat16* kp,
                              const __nv_bfloat16* vp, const int32_t* table, const int32_t* lens,
                              __nv_bfloat16* out, float* lse, uint8_t* ws, cudaStream_t st);

// The cache's pages (pages.cu).
constexpr int APPEND_MAX_B = 8192;
size_t paged_append_ws_bytes(const PagedShape& s);
cudaError_t launch_paged_append(const PagedShape& s, const __nv_bfloat16* k_new, const __nv_bfloat16* v_new,
                                const int32_t* n_new, __nv_bfloat16* kp, __nv_bfloat16* vp, int32_t* table,
                                int32_t* lens, int32_t* ref, int32_t* short_pages, uint8_t* ws, cudaStream_t st);
cudaError_t launch_pages_fork(const PagedShape& s, int n, const int32_t* src, const int32_t* dst, int32_t* table,
                              int32_t* lens, int32_t* ref, int32_t* done, cudaStream_t st);
cudaError_t launch_pages_free(const PagedShape& s, int n, const int32_t* rows, const int32_t* keep, int32_t* table,
                              int32_t* lens, int32_t* ref, int32_t* done, cudaStream_t st);
size_t pages_compact_ws_bytes(const PagedShape& s);
cudaError_t launch_pages_compact(const PagedShape& s, __nv_bfloat16* kp, __nv_bfloat16* vp, int32_t* table,
                                 const int32_t* lens, int32_t* ref, int32_t* remap, int32_t* n_live, uint8_t* ws,
                                 cudaStream_t st);

// Length of row b, inside the table's columns whatever lens holds.
__device__ __forceinline__ int paged_len(const PagedShape& s, const int32_t* lens, int b) {
    return max(0, min(lens[b], s.cols << s.logP));
}

}  // namespace nsa
