// Sliding-window attention with sink tokens: derived sizes and launchers.
#pragma once

#include "common.cuh"

namespace nsa {

// Sizes of one problem, window and sink clamped to the cache.
struct WinShape {
    int B, Tq, Tk, q0, Hq, Hkv, G, dqk, dv;
    int win;      // 1 .. Tk
    int ns;       // 0 .. Tk
    float scale;
};

// The backward's weights are p = exp(s - lse) <= 1, but lse has 24 bits: at |lse| = 2^20 its last
// place moves p by a tenth, from 2^31 on by more than fp32's range.  So where |lse| > LARGE_LSE the
// exponent is clamped to 0, and lse enters lowered by 2^-20 of its size, more than the roundings
// of lse and of the scores add up to (16 of 2^-24): a key that has all the weight gets p = 1.
constexpr float LARGE_LSE = 4096.f;
__device__ __forceinline__ float bwd_lse(float lse) {
    return lse > LARGE_LSE ? lse * (1.f - 0x1p-20f) : lse < -LARGE_LSE ? lse * (1.f + 0x1p-20f) : lse;
}
__device__ __forceinline__ float at_most_0(float x) { return x > 0.f ? 0.f : x; }       // (NaN stays NaN)

// delta = do.o reads the rounded out.  A row of few keys has an out as large as its values, and ds = p (do.v
// - delta) carries that rounding whole.  As the exact ds of a row add up to 0, rows of up to FEW_KEYS keys
// first walk their keys for the sum of the ds under that delta, in fp32, and add it to delta.  (2000
// tokens, 8 heads on 2, d 128: dq is off by 3.8e-3 without that walk at a window of 2, 2.7e-3 at 8, 2.4e-3 at
// 64, and with it by 2.35e-3, what ds and dq lose in bf16.)
constexpr int FEW_KEYS = 64;
// Keys that the query at position t sees.
__device__ __forceinline__ int visible_keys(const WinShape& s, int t) {
    const int lo = max(0, t - s.win + 1);
    return t - lo + 1 + min(s.ns, lo);
}

// Any shape: FFMA, one warp per row (window_rowwise.cu).  delta [B, Tq, Hq].
cudaError_t launch_window_rowwise_fwd(const WinShape& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                      const __nv_bfloat16* v, __nv_bfloat16* out, float* lse, cudaStream_t st);
cudaError_t launch_window_rowwise_bwd(const WinShape& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                      const __nv_bfloat16* v, const __nv_bfloat16* out, const float* lse,
                                      const __nv_bfloat16* d_out, __nv_bfloat16* dq, __nv_bfloat16* dk,
                                      __nv_bfloat16* dv, float* delta, cudaStream_t st);

// Tensor cores (window_fwd_tc.cu): d_qk <= 192, d_v <= 128, at most 64 heads per group.
bool window_tc_supported(const WinShape& s);
cudaError_t launch_window_fwd_tc(const WinShape& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                 const __nv_bfloat16* v, __nv_bfloat16* out, float* lse, cudaStream_t st);
int read_and_clear_win_fwd_status();
cudaError_t set_win_fwd_wait_limit(uint64_t limit_ns);      // 0: one second
// Backward for the same shapes (window_bwd_tc.cu); part: window_bwd_tc_part_bytes().
size_t window_bwd_tc_part_bytes(const WinShape& s);
cudaError_t launch_window_bwd_tc(const WinShape& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                 const __nv_bfloat16* v, const __nv_bfloat16* out, const float* lse,
                                 const __nv_bfloat16* d_out, __nv_bfloat16* dq, __nv_bfloat16* dk,
                                 __nv_bfloat16* dv, float* delta, float* part, cudaStream_t st);
int read_and_clear_win_bwd_status();
cudaError_t set_win_bwd_wait_limit(uint64_t limit_ns);
}  // namespace nsa
