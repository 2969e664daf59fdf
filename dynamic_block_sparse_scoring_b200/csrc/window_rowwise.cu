// Sliding-window attention with sink tokens for any shape, on FFMA: one warp
// per (query, head) row, or per key for dk / dv.
//
// Transcript #94 (bidclub.ai) §4: the window and the attention sink.  With
// s_u = scale q.k_u over the visible keys, the forward keeps the running
// maximum m and the sum l of exp(s_u - m) and the values' sum under the same
// weights; the backward rebuilds p_u = exp(s_u - lse) and uses
//   ds_u = p_u (do.v_u - delta), delta = do.o
//   dq = scale sum_u ds_u k_u;  dk_u = scale sum_t ds_u q;  dv_u = sum_t p_u do.
// A lane holds columns 64 i + 2 lane + {0, 1}.  The dot products' shuffles
// bound these kernels; the tensor-core kernels serve the shapes that fit them
// and these the rest (head dimensions of 256, more than 64 heads per group).
// 2 x 8192 tokens, 16 heads, d 128, window 1000 + 16: 29.1 ms, 4.4 TFLOP/s.
#include <math.h>

#include "window.cuh"

namespace nsa {
namespace {

constexpr int MAXP = 4;          // column pairs per lane: d <= 256
constexpr int KU = 4;            // keys (or rows) per step

__device__ __forceinline__ void load_row(const __nv_bfloat16* p, int np, int lane, float2* f) {
#pragma unroll
    for (int i = 0; i < MAXP; ++i)
        f[i] = i < np ? __bfloat1622float2(reinterpret_cast<const __nv_bfloat162*>(p)[32 * i + lane])
                      : make_float2(0.f, 0.f);
}

__device__ __forceinline__ void store_row(__nv_bfloat16* p, int np, int lane, const float2* f, float w) {
#pragma unroll
    for (int i = 0; i < MAXP; ++i)
        if (i < np)
            reinterpret_cast<__nv_bfloat162*>(p)[32 * i + lane] = __floats2bfloat162_rn(f[i].x * w, f[i].y * w);
}

__device__ __forceinline__ float dot(const float2* a, const float2* b) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < MAXP; ++i) s = fmaf(a[i].x, b[i].x, fmaf(a[i].y, b[i].y, s));
    return s;
}

struct Row {
    int b, t, h, kvh;
    size_t plane;
};

__device__ __forceinline__ bool row_of(const WinShape& s, long long w, Row* r) {
    if (w >= (long long)s.B * s.Tq * s.Hq) return false;
    r->h = (int)(w % s.Hq);
    const long long bt = w / s.Hq;
    r->t = s.q0 + (int)(bt % s.Tq);
    r->b = (int)(bt / s.Tq);
    r->kvh = r->h / s.G;
    r->plane = (size_t)r->b * s.Hkv + r->kvh;
    return true;
}

// f(u0, n): keys u0 .. u0 + n - 1 (n <= KU) of everything the query at t sees.
template <class F>
__device__ __forceinline__ void for_keys(const WinShape& s, int t, F f) {
    const int lo = max(0, t - s.win + 1);
    const int sinks = min(s.ns, lo);
    for (int u = 0; u < sinks; u += KU) f(u, min(KU, sinks - u));
    for (int u = lo; u <= t; u += KU) f(u, min(KU, t + 1 - u));
}

__global__ void __launch_bounds__(128) window_fwd_kernel(WinShape s, const __nv_bfloat16* __restrict__ q,
                                                         const __nv_bfloat16* __restrict__ k,
                                                         const __nv_bfloat16* __restrict__ v,
                                                         __nv_bfloat16* __restrict__ out,
                                                         float* __restrict__ lse) {
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    Row r;
    if (!row_of(s, w, &r)) return;
    const int nq = s.dqk / 64, nv = s.dv / 64;
    float2 qf[MAXP], o[MAXP];
    load_row(q + (size_t)w * s.dqk, nq, lane, qf);
#pragma unroll
    for (int i = 0; i < MAXP; ++i) o[i] = make_float2(0.f, 0.f);
    float m = -INFINITY, l = 0.f;
    for_keys(s, r.t, [&](int u0, int n) {
        float sc[KU];
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            float2 kf[MAXP];
            load_row(k + (r.plane * s.Tk + u0 + min(j, n - 1)) * s.dqk, nq, lane, kf);
            sc[j] = dot(qf, kf);
        }
        float mx = m;
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            sc[j] = j < n ? __fmul_rn(warp_sum(sc[j]), s.scale) : -INFINITY;   // (the maximum's weight is 1)
            mx = fmaxf(mx, sc[j]);
        }
        const float alpha = expf(m - mx);
        m = mx;
        l *= alpha;
#pragma unroll
        for (int i = 0; i < MAXP; ++i) o[i] = make_float2(o[i].x * alpha, o[i].y * alpha);
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            if (j >= n) break;
            const float p = expf(sc[j] - m);
            l += p;
            float2 vf[MAXP];
            load_row(v + (r.plane * s.Tk + u0 + j) * s.dv, nv, lane, vf);
#pragma unroll
            for (int i = 0; i < MAXP; ++i) o[i] = make_float2(fmaf(p, vf[i].x, o[i].x), fmaf(p, vf[i].y, o[i].y));
        }
    });
    store_row(out + (size_t)w * s.dv, nv, lane, o, 1.f / l);
    if (lse && lane == 0) lse[w] = m + logf(l);
}

__global__ void __launch_bounds__(128) window_dq_kernel(WinShape s, const __nv_bfloat16* __restrict__ q,
                                                        const __nv_bfloat16* __restrict__ k,
                                                        const __nv_bfloat16* __restrict__ v,
                                                        const __nv_bfloat16* __restrict__ out,
                                                        const float* __restrict__ lse,
                                                        const __nv_bfloat16* __restrict__ d_out,
                                                        __nv_bfloat16* __restrict__ dq,
                                                        float* __restrict__ delta) {
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
    Row r;
    if (!row_of(s, w, &r)) return;
    const int nq = s.dqk / 64, nv = s.dv / 64;
    float2 qf[MAXP], df[MAXP], acc[MAXP];
    load_row(out + (size_t)w * s.dv, nv, lane, acc);
    load_row(d_out + (size_t)w * s.dv, nv, lane, df);
    load_row(q + (size_t)w * s.dqk, nq, lane, qf);
    float dl = warp_sum(dot(acc, df));
    const float ls = bwd_lse(lse[w]);
    if (visible_keys(s, r.t) <= FEW_KEYS) {
        float ds = 0.f;
        for_keys(s, r.t, [&](int u0, int n) {
            for (int j = 0; j < n; ++j) {
                float2 kf[MAXP], vf[MAXP];
                load_row(k + (r.plane * s.Tk + u0 + j) * s.dqk, nq, lane, kf);
                load_row(v + (r.plane * s.Tk + u0 + j) * s.dv, nv, lane, vf);
                const float p = expf(at_most_0(warp_sum(dot(qf, kf)) * s.scale - ls));
                ds = fmaf(p, warp_sum(dot(df, vf)) - dl, ds);
            }
        });
        dl += ds;
    }
    if (lane == 0) delta[w] = dl;
#pragma unroll
    for (int i = 0; i < MAXP; ++i) acc[i] = make_float2(0.f, 0.f);
    for_keys(s, r.t, [&](int u0, int n) {
#pragma unroll
        for (int j = 0; j < KU; ++j) {
            if (j >= n) break;
            float2 kf[MAXP], vf[MAXP];
            load_row(k + (r.plane * s.Tk + u0 + j) * s.dqk, nq, lane, kf);
            load_row(v + (r.plane * s.Tk + u0 + j) * s.dv, nv, lane, vf);
            const float p = expf(at_most_0(warp_sum(dot(qf, kf)) * s.scale - ls));
            const float ds = p * (warp_sum(dot(df, vf)) - dl);
#pragma unroll
            for (int i = 0; i < MAXP; ++i)
                acc[i] = make_float2(fmaf(ds, kf[i].x, acc[i].x), fmaf(ds, kf[i].y, acc[i].y));
        }
    });
    store_row(dq + (size_t)w * s.dqk, nq, lane, acc, s.scale);
}

__global__ void __launch_bounds__(128) window_dkv_kernel(WinShape s, const __nv_bfloat16* __restrict__ q,
                                                         const __nv_bfloat16* __restrict__ k,
                                                         const __nv_bfloat16* __restrict__ v,
                                                         const float* __restrict__ lse,
                                                         const __nv_bfloat16* __restrict__ d_out,
                                                         const float* __restrict__ delta,
                                                         __nv_bfloat16* __restrict__ dk,
                                                         __nv_bfloat16* __restrict__ dv) {
    const int lane = threadIdx.x & 31;
    const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);     // (plane, key)
    if (w >= (long long)s.B * s.Hkv * s.Tk) return;
    const int u = (int)(w % s.Tk);
    const int plane = (int)(w / s.Tk), b = plane / s.Hkv, kvh = plane % s.Hkv;
    const int nq = s.dqk / 64, nv = s.dv / 64;
    float2 kf[MAXP], vf[MAXP], ak[MAXP], av[MAXP];
    load_row(k + (size_t)w * s.dqk, nq, lane, kf);
    load_row(v + (size_t)w * s.dv, nv, lane, vf);
#pragma unroll
    for (int i = 0; i < MAXP; ++i) ak[i] = av[i] = make_float2(0.f, 0.f);
    const int t0 = max(u, s.q0);
    const int t1 = u < s.ns ? s.q0 + s.Tq : (int)min((long long)s.q0 + s.Tq, (long long)u + s.win);
    for (int t = t0; t < t1; ++t)
        for (int g = 0; g < s.G; ++g) {
            const size_t row = ((size_t)b * s.Tq + (t - s.q0)) * s.Hq + kvh * s.G + g;
            float2 qf[MAXP], df[MAXP];
            load_row(q + row * s.dqk, nq, lane, qf);
            load_row(d_out + row * s.dv, nv, lane, df);
            const float p = expf(at_most_0(warp_sum(dot(qf, kf)) * s.scale - bwd_lse(lse[row])));
            const float ds = p * (warp_sum(dot(df, vf)) - delta[row]);
#pragma unroll
            for (int i = 0; i < MAXP; ++i) {
                ak[i] = make_float2(fmaf(ds, qf[i].x, ak[i].x), fmaf(ds, qf[i].y, ak[i].y));
                av[i] = make_float2(fmaf(p, df[i].x, av[i].x), fmaf(p, df[i].y, av[i].y));
            }
        }
    store_row(dk + (size_t)w * s.dqk, nq, lane, ak, s.scale);
    store_row(dv + (size_t)w * s.dv, nv, lane, av, 1.f);
}

unsigned warps_grid(long long warps) { return (unsigned)((warps + 3) / 4); }

}  // namespace

cudaError_t launch_window_rowwise_fwd(const WinShape& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                      const __nv_bfloat16* v, __nv_bfloat16* out, float* lse, cudaStream_t st) {
    window_fwd_kernel<<<warps_grid((long long)s.B * s.Tq * s.Hq), 128, 0, st>>>(s, q, k, v, out, lse);
    return cudaGetLastError();
}

cudaError_t launch_window_rowwise_bwd(const WinShape& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                      const __nv_bfloat16* v, const __nv_bfloat16* out, const float* lse,
                                      const __nv_bfloat16* d_out, __nv_bfloat16* dq, __nv_bfloat16* dk,
                                      __nv_bfloat16* dv, float* delta, cudaStream_t st) {
    window_dq_kernel<<<warps_grid((long long)s.B * s.Tq * s.Hq), 128, 0, st>>>(s, q, k, v, out, lse, d_out, dq,
                                                                              delta);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    window_dkv_kernel<<<warps_grid((long long)s.B * s.Hkv * s.Tk), 128, 0, st>>>(s, q, k, v, lse, d_out, delta,
                                                                                dk, dv);
    return cudaGetLastError();
}

}  // namespace nsa
