// Sliding-window attention with sink tokens on the 5th-generation tensor cores
// (tcgen05 + TMEM + TMA), backward.
//
// With x = log2 e (scale q.k - lse), p = 2^x (rebuilt from the forward's lse),
// delta = do.o and ds = p (do.v - delta):
//   dq = scale sum_u ds k_u,   dk_u = scale sum_t ds q_t,   dv_u = sum_t p do_t
// (Transcript #94, bidclub.ai, §2 and §4: each output is a softmax-weighted sum
// over the window and the sinks.)
//
// Two kernels of one shape.  128 rows stay resident, 64 rows at a time stream
// past them, and every sum over the streamed side accumulates in TMEM:
//             resident (M = 128)      streamed (N = 64)       accumulates
//   DQ        Q, dO of a query tile   K, V of 64 keys         dQ += dS K
//   DKV       K, V of a key tile      Q, dO of 64 query rows  dV += P dO, dK += dS Q
// S = R1 T1^T and D = R2 T2^T are products of shared-memory operands, P and dS
// (bf16, written over S in TMEM) are the A operand of the gradient products,
// whose B is the streamed tile again, read MN-major.  So the scores are built
// twice (seven products instead of five), but no gradient is added to memory:
// no atomics, no fp32 dq in HBM, the same bits on every run.
//
// Queries are (token, head) rows of one KV head's group, so dk / dv sum over
// the group in TMEM.  A key tile that many queries see (the sinks', or any on
// a small problem) is cut into items over its queries, whose fp32 partial
// sums window_bwd_join_kernel adds in order.
//
// A query tile whose first row sees few keys (FEW_KEYS) is walked twice in DQ: the first walk sums ds,
// which corrects delta, the second builds dQ with that.
//
// Warps (384 threads): 0 TMA, 1 MMA issue (one lane), 2-3 the rows' (lse,
// delta), 4-7 and 8-11 two warpgroups taking the steps in turn, one thread per
// resident row.  The issue order S(i+1) D(i+1) | gradients(i) gives the softmax
// of a step the tensor cores' time of a whole step.
// Bound by the tensor cores and shared memory: a step (64 streamed rows) is
// 128 x 64 x (2 d_qk + d_v) MACs in DQ, (2 d_qk + 2 d_v) in DKV, at 4096 a
// clock; S and D (N = 64, both operands in shared memory) take 48 clocks for 32
// of MMA, for the 6 KB that they read, and the copies write 40 KB a step.
// Measured in bursts, forward included: 8192 tokens, 64 heads on 4, 192/128,
// window 512 + 64: 980 us, 684 TFLOP/s; 4096 tokens, 16 heads, d 128, fully
// causal: 363 us, 662 TFLOP/s (counting five products of the backward, not the
// seven done); 1119-1148 and 371-380 us back to back under the power cap.  Of these
// the clamp of large scores and the sums of ds are 0.5 % each.
#include <math.h>

#include <algorithm>

#include "launch.cuh"
#include "rows_out.cuh"
#include "tc.cuh"
#include "tmap.cuh"
#include "window.cuh"

namespace nsa {

__device__ int g_win_bwd_status = 0;
// Limit of the roles' waits (WAIT_NS unless nsa_set_wait_limit_ns shortened it); the drains keep WAIT_NS.
__constant__ uint64_t c_win_bwd_wait_ns = 1000000000ull;

namespace {

constexpr int BM = 128, BN = 64;
constexpr int RCHUNK = 16384, TCHUNK = 8192;    // 128 / 64 rows x 64 columns of bf16
constexpr int THREADS = 384;
constexpr uint64_t WAIT_NS = 1000000000ull;
constexpr int SMS = 148;                        // the split of key tiles is planned for this many SMs
constexpr int MAX_FLAGS = 256;                  // most CTAs of the dq kernel
// Least steps of an item of a split key tile: 1000 tokens, 4 heads on 1, d 64, window 128 + 4
// took 35.3 us at 8, 32.5 at 4, 32.4 at 2; fewer steps only mean more partial sums.
constexpr int MIN_CHUNK = 4;
constexpr float LOG2E = 1.4426950408889634f;

enum { DQ = 0, DKV = 1 };

template <int DQK, int DV, int MODE>
struct Smem {
    static constexpr int QC = DQK / 64, VC = DV / 64;
    static constexpr int R_BYTES = (QC + VC) * RCHUNK, T_BYTES = (QC + VC) * TCHUNK;
    static constexpr int NST = (216 * 1024 - R_BYTES) / T_BYTES >= 4 ? 4 : 3;
    static constexpr int T_OFF = R_BYTES;
    // DQ: float2 (lse log2 e, delta) of the rows of two query tiles.  DKV: 16 more columns for
    // the products, 32 bytes a row: a constant [BM] of the residents, then per stage [BN] for S, [BN] for D
    static constexpr int AUX_OFF = T_OFF + NST * T_BYTES;
    static constexpr int EXT_A = BM * 32, EXT_B = BN * 32;
    // DQ: behind them, per (work, warpgroup) of two works each row's sum of ds of the first walk
    static constexpr int SUM_OFF = AUX_OFF + 2 * BM * 8;
    static constexpr int AUX_BYTES = MODE == DQ ? 2 * BM * 8 + 4 * BM * 4 : EXT_A + NST * 2 * EXT_B;
    static constexpr int BAR_OFF = AUX_OFF + AUX_BYTES;
    static_assert(AUX_OFF % 1024 == 0, "swizzled rows");
    static constexpr int ALLOC = BAR_OFF + 512 + 1024;
    static constexpr int ACC = MODE == DQ ? DQK : DQK + DV;     // accumulator columns
    static constexpr int ND = 128 + 128 + ACC <= 512 ? 2 : 1;   // D buffers in TMEM
    static constexpr int D_COL = 128, ACC_COL = 128 + 64 * ND;  // columns: S0 S1 | D .. | dQ  or  dV dK
};

struct Bars {
    uint64_t r_full, r_empty, t_full[4], t_empty[4], s_full[2], d_full[2], d_read[2], p_full[2];
    uint64_t acc_full, acc_free, aux_full[2], aux_empty[2], sum_full, drain;
    uint32_t tmem;
    int abort;
    int large;          // DQ: a row with |lse| > LARGE_LSE has been among the CTA's
};

// How the key tiles are cut into items (DKV): key tiles below nsk hold sinks
// and are seen by every later query, the others by the window's.
struct Split {
    int nk, nsk;        // key tiles, those with sinks
    int chunk_s, chunk_o;   // steps per item
    int sp_s, sp_o;     // most items of a key tile
    int slots_s;        // partial-sum slots of the key tiles with sinks (0 if they are whole)
};

struct Args {
    WinShape s;
    Split p;
    const __nv_bfloat16* out;
    const __nv_bfloat16* d_out;
    const float* lse;
    float* delta;
    __nv_bfloat16* dq;
    __nv_bfloat16* dk;
    __nv_bfloat16* dv;
    float* part;        // partial sums [slot][BM][DV + DQK]
    int* flags;         // [n_flags] Bars::large of the dq kernel's CTAs
    int n_flags;
    int tok;            // tokens per query tile (DQ) or per step (DKV)
    int n_tt;           // query tiles per (sequence, KV head) (DQ)
    int n_work;
    bool turned;        // DKV: see Work::token
    float scale_log2;
};

__host__ __device__ __forceinline__ int ceil_div(int a, int b) { return (a + b - 1) / b; }

// Tokens [i0, i1) of the queries that see a key of the tile at u0.
__host__ __device__ __forceinline__ void tile_queries(const WinShape& s, int u0, int* i0, int* i1) {
    const long long last = u0 < s.ns ? (long long)s.q0 + s.Tq - 1
                                     : min((long long)s.q0 + s.Tq - 1, (long long)u0 + BM - 1 + s.win - 1);
    *i0 = max(u0, s.q0) - s.q0;
    *i1 = max((int)(last + 1 - s.q0), *i0);
}

// One work item: the steps of a query tile (DQ) or of a share of a key tile's queries (DKV).
struct Work {
    int b, kvh, n;      // n: steps
    int m;              // DQ: steps of a walk over the keys, n or, where the tile is walked twice, n / 2
    int first;          // DQ: first token of the query tile.  DKV: first key of the tile
    int base, rot;      // DKV: first token, and which step's place the first step takes
    int nst, sl, lo;    // DQ: sink steps, sinks before the window, first key of the window's steps
    int slot;           // DKV: partial-sum slot, -1: the only item of its key tile

    // DQ: first key of step i; does the step hold sinks before the window?
    __device__ __forceinline__ int key(int i) const {
        const int j = i < m ? i : i - m;
        return j < nst ? j * BN : lo + (j - nst) * BN;
    }
    __device__ __forceinline__ bool sink_step(int i) const { return (i < m ? i : i - m) < nst; }
    // DKV: first token of step i.  Turned (rot >= 0), the steps run backwards from rot on and
    // around, so that CTAs whose key tiles share queries come to them at the same time: block
    // b of tok tokens is taken at step (last block - b) mod n.
    __device__ __forceinline__ int token(int i, int tok) const {
        return base + (rot < 0 ? i : rot >= i ? rot - i : rot - i + n) * tok;
    }
};

template <int MODE>
__device__ __forceinline__ bool decode_work(const Args& a, int w, Work* k) {
    const WinShape& s = a.s;
    const int planes = s.B * s.Hkv;
    if (MODE == DQ) {
        const int r = w % planes, tt = a.n_tt - 1 - w / planes;     // the latest first
        k->b = r / s.Hkv;
        k->kvh = r % s.Hkv;
        k->first = tt * a.tok;
        const int pf = s.q0 + k->first, pl = min(pf + a.tok, s.q0 + s.Tq) - 1;
        k->lo = max(0, pf - s.win + 1);
        k->sl = min(s.ns, k->lo);
        k->nst = ceil_div(k->sl, BN);
        if (k->lo < k->nst * BN) k->lo = k->sl = k->nst = 0;        // they meet: one range from 0
        k->m = k->nst + (pl - k->lo) / BN + 1;
        k->n = visible_keys(s, pf) <= FEW_KEYS ? 2 * k->m : k->m;
        return true;
    }
    const int n_s = planes * a.p.nsk * a.p.sp_s;
    const bool sinks = w < n_s;
    const int x = sinks ? w : w - n_s;
    const int plane = x % planes, y = x / planes;
    const int tiles = sinks ? a.p.nsk : a.p.nk - a.p.nsk;
    const int kt = (sinks ? 0 : a.p.nsk) + y % tiles, c = y / tiles;
    const int chunk = sinks ? a.p.chunk_s : a.p.chunk_o, sp = sinks ? a.p.sp_s : a.p.sp_o;
    k->b = plane / s.Hkv;
    k->kvh = plane % s.Hkv;
    k->first = kt * BM;
    int i0, i1;
    tile_queries(s, k->first, &i0, &i1);
    const int steps = ceil_div(i1 - i0, a.tok);
    const int items = max(1, ceil_div(steps, chunk));
    if (c >= items) return false;
    k->base = i0 + c * chunk * a.tok;
    k->n = min(chunk, steps - c * chunk);
    k->rot = a.turned && k->n > 0 ? (ceil_div(s.Tq, a.tok) - 1 - k->base / a.tok) % k->n : -1;
    k->slot = items == 1 ? -1
                         : (sinks ? 0 : a.p.slots_s) + (plane * tiles + kt - (sinks ? 0 : a.p.nsk)) * sp + c;
    return true;
}

// The w-th item of CTA c: items are dealt back and forth, heaviest first.
__device__ __forceinline__ int dealt(int round) {
    return round * (int)gridDim.x + ((round & 1) ? (int)(gridDim.x - 1 - blockIdx.x) : (int)blockIdx.x);
}

__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int w) {
    const int a = max(lo - 32 * w, 0), b = min(hi - 32 * w, 31);
    if (b < a) return 0u;
    return (0xFFFFFFFFu >> (31 - b)) & (0xFFFFFFFFu << a);
}

// DQ: (lse log2 e, delta) of N rows of a query tile, from row r0 on, by one warp: into dst and,
// delta, into global memory.  LPR lanes hold a row's d_v values, 16 bytes each, U x RPI rows
// are in flight at a time.  Their sums over the lanes are taken together: each round halves
// the rows that a lane carries.
template <int DV, int N, int U>
__device__ __forceinline__ void rows_delta(const Args& a, const Work& k, int r0, int lane, float2* dst) {
    constexpr int LPR = DV / 8, RPI = 32 / LPR, E = (N + 31) / 32;
    static_assert(N % (RPI * U) == 0 && U <= LPR, "rows per step");
    const WinShape& s = a.s;
    const int sub = lane / LPR, col = (lane % LPR) * 8;
    const int toks = min(a.tok, s.Tq - k.first);
    const long long row0 = ((long long)k.b * s.Tq + k.first) * s.Hq + k.kvh * s.G;
    float ls[E];                                    // lse of rows r0 + 32 e + lane
    long long at[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int r = r0 + 32 * e + lane, tt = r / s.G;
        at[e] = tt < toks && 32 * e + lane < N ? row0 + (long long)tt * s.Hq + (r - tt * s.G) : -1;
        ls[e] = at[e] >= 0 ? a.lse[at[e]] : INFINITY;
    }
    int tt = (r0 + sub) / s.G, h = r0 + sub - tt * s.G;
#pragma unroll 1
    for (int i = 0; i < N; i += RPI * U) {
        uint4 x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = y[u] = make_uint4(0, 0, 0, 0);
            if (tt < toks) {
                const size_t o = (size_t)(row0 + (long long)tt * s.Hq + h) * DV + col;
                x[u] = *reinterpret_cast<const uint4*>(a.out + o);
                y[u] = *reinterpret_cast<const uint4*>(a.d_out + o);
            }
            for (h += RPI; h >= s.G; h -= s.G) ++tt;
        }
        float d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float f[8], g[8];
            unpack8(x[u], f);
            unpack8(y[u], g);
            d[u] = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) d[u] = fmaf(f[e], g[e], d[u]);
        }
        // after the rounds the high bits of the lane within its row name the row u
        int u0 = 0;
#pragma unroll
        for (int c = U / 2, o = LPR / 2; c > 0; c >>= 1, o >>= 1) {
            const bool up = lane & o;
            u0 += up ? c : 0;
#pragma unroll
            for (int u = 0; u < c; ++u) {
                const float send = up ? d[u] : d[u + c];
                d[u] = (up ? d[u + c] : d[u]) + __shfl_xor_sync(0xffffffffu, send, o);
            }
        }
#pragma unroll
        for (int o = LPR / 2 / U; o > 0; o >>= 1) d[0] += __shfl_xor_sync(0xffffffffu, d[0], o);
        if ((lane & (LPR / U - 1)) == 0) dst[i + u0 * RPI + sub].y = d[0];
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < E; ++e) {
        if (32 * e + lane >= N) continue;
        float2* v = dst + 32 * e + lane;
        v->x = bwd_lse(ls[e]) * LOG2E;
        if (at[e] >= 0) a.delta[at[e]] = v->y;
    }
}

template <int DQK, int DV, int MODE>
__global__ void __launch_bounds__(THREADS, 1)
    window_bwd_tc_kernel(const __grid_constant__ CUtensorMap map_r1, const __grid_constant__ CUtensorMap map_r2,
                         const __grid_constant__ CUtensorMap map_t1, const __grid_constant__ CUtensorMap map_t2,
                         const Args a) {
    using L = Smem<DQK, DV, MODE>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars& bar = *reinterpret_cast<Bars*>(sm + L::BAR_OFF);
    float2* aux = reinterpret_cast<float2*>(sm + L::AUX_OFF);
    volatile int* abort_flag = &bar.abort;
    volatile int* large = &bar.large;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WinShape& s = a.s;
    // What follows in the stream may start on the SMs that this grid leaves idle: of its results
    // the DKV kernel reads delta and the flags, and waits for them.  There every role waits for this
    // grid's end before its first wait that needs them, so that the bounded waits count the
    // time of their own grid only; the copies of the first stages go before.
    pdl_launch();

    if (threadIdx.x == 0) {
        tc::mbar_init(&bar.r_full, 1);
        tc::mbar_init(&bar.r_empty, 1);
        for (int i = 0; i < 4; ++i) {
            tc::mbar_init(&bar.t_full[i], MODE == DKV ? 2 : 1);     // the copies, and the (lse, delta) columns
            tc::mbar_init(&bar.t_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.d_full[i], 1);
            tc::mbar_init(&bar.d_read[i], 4);
            tc::mbar_init(&bar.p_full[i], 4);
            tc::mbar_init(&bar.aux_full[i], 2);
            tc::mbar_init(&bar.aux_empty[i], 8);
        }
        tc::mbar_init(&bar.acc_full, 1);
        tc::mbar_init(&bar.acc_free, 8);
        tc::mbar_init(&bar.sum_full, 8);
        tc::mbar_init(&bar.drain, 1);
        bar.abort = 0;
        bar.large = 0;
        tc::fence_mbar_init();
        tc::prefetch_map(&map_r1);
        tc::prefetch_map(&map_r2);
        tc::prefetch_map(&map_t1);
        tc::prefetch_map(&map_t2);
    }
    if (MODE == DKV && a.tok * s.G < BN) {
        // rows of a step that no query fills stay zero: they enter the sums over rows
        for (int i = threadIdx.x; i < L::NST * L::T_BYTES / 16; i += THREADS)
            reinterpret_cast<uint4*>(sm + L::T_OFF)[i] = make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async_smem();
    }
    if (MODE == DKV && threadIdx.x < BM) {          // (1, 1, 1, 0, ..) in every row of the constant
        const int half = (threadIdx.x >> 2) & 1;
        uint4* row = reinterpret_cast<uint4*>(sm + L::AUX_OFF + threadIdx.x * 32);
        row[half] = make_uint4(0x3F803F80u, 0x00003F80u, 0, 0);
        row[half ^ 1] = make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async_smem();
    }
    if (warp == 1) {
        tc::tmem_alloc(&bar.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = bar.tmem;
    auto wait = [&](uint64_t* b, uint32_t parity) { return tc::mbar_wait(b, parity, abort_flag, c_win_bwd_wait_ns); };
    auto warp_wait = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)); };
    auto give_up = [&]() {
        *abort_flag = 1;
        atomicExch(&g_win_bwd_status, (int)NSA_ERR_TIMEOUT);
    };

    if (warp < 4) {
        // 4 x 32 x 88 + 8 x 32 x 208 = 64512, the 384 x 168 registers of the launch
        asm volatile("setmaxnreg.dec.sync.aligned.u32 88;" ::: "memory");
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ copies
            uint32_t nr = 0, g = 0;
            bool ok = true;
            const int rows = a.tok * s.G;
            const uint32_t r_bytes = (L::QC + L::VC) * (MODE == DQ ? rows * 128 : RCHUNK);
            const uint32_t t_bytes = (L::QC + L::VC) * (MODE == DQ ? TCHUNK : rows * 128);
            for (int round = 0, w; ok && (w = dealt(round)) < a.n_work; ++round) {
                Work k;
                if (!decode_work<MODE>(a, w, &k) || k.n == 0) continue;
                const int plane = k.b * s.Hkv + k.kvh, h0 = k.kvh * s.G;
                if (MODE == DKV && nr == 1) pdl_wait();
                if (!wait(&bar.r_empty, (nr & 1) ^ 1)) { ok = false; break; }
                tc::mbar_arrive_expect_tx(&bar.r_full, r_bytes);
#pragma unroll
                for (int c = 0; c < L::QC + L::VC; ++c) {
                    const CUtensorMap* m = c < L::QC ? &map_r1 : &map_r2;
                    const int x = 64 * (c < L::QC ? c : c - L::QC);
                    if (MODE == DQ) tc::tma_load_4d(sm + c * RCHUNK, m, &bar.r_full, x, h0, k.first, k.b);
                    else tc::tma_load_3d(sm + c * RCHUNK, m, &bar.r_full, x, k.first, plane);
                }
                ++nr;
                for (int i = 0; i < k.n; ++i, ++g) {
                    const int st = g % L::NST;
                    if (MODE == DKV && g == L::NST) pdl_wait();
                    if (!wait(&bar.t_empty[st], ((g / L::NST) & 1) ^ 1)) { ok = false; break; }
                    tc::mbar_arrive_expect_tx(&bar.t_full[st], t_bytes);
                    uint8_t* dst = sm + L::T_OFF + st * L::T_BYTES;
#pragma unroll
                    for (int c = 0; c < L::QC + L::VC; ++c) {
                        const CUtensorMap* m = c < L::QC ? &map_t1 : &map_t2;
                        const int x = 64 * (c < L::QC ? c : c - L::QC);
                        if (MODE == DQ)
                            tc::tma_load_3d(dst + c * TCHUNK, m, &bar.t_full[st], x, k.key(i), plane);
                        else
                            tc::tma_load_4d(dst + c * TCHUNK, m, &bar.t_full[st], x, h0, k.token(i, a.tok), k.b);
                    }
                    // the rows after the stages' into L2 (rows outside the tensor are not fetched)
                    if (MODE == DKV && i + 2 < k.n) {
#pragma unroll
                        for (int c = 0; c < L::QC + L::VC; ++c)
                            tc::tma_prefetch_l2_4d(c < L::QC ? &map_t1 : &map_t2, 64 * (c < L::QC ? c : c - L::QC), h0,
                                                   k.token(i + 2, a.tok), k.b);
                    }
                }
            }
            if (!ok) give_up();
            if (MODE == DKV) pdl_wait();
            // every copy issued here has landed before the CTA ends (one limit for all: t_full never
            // completes where the warps that fill its other half have given up)
            const uint64_t t0 = tc::globaltimer_ns();
            auto drain = [&](uint64_t* b, uint32_t parity) {
                const uint64_t used = tc::globaltimer_ns() - t0;
                tc::mbar_wait_bounded(b, parity, used < WAIT_NS ? WAIT_NS - used : 0);
            };
            if (nr > 0) drain(&bar.r_full, (nr - 1) & 1);
            for (uint32_t i = 0; i < L::NST && i < g; ++i) {
                const uint32_t last = i + ((g - 1 - i) / L::NST) * L::NST;
                drain(&bar.t_full[i], (last / L::NST) & 1);
            }
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issue
            // The whole warp walks the schedule, one lane issues: the operands stay in
            // uniform registers.
            const uint32_t idesc_sd = tc::idesc_bf16_f32(BM, BN, false, false);
            const uint32_t idesc_q = tc::idesc_bf16_f32(BM, DQK, false, true);
            const uint32_t idesc_v = tc::idesc_bf16_f32(BM, DV, false, true);
            const uint64_t r_desc = tc::sdesc_sw128(tc::smem_u32(sm), 16, 1024),
                           t_desc = tc::sdesc_sw128(tc::smem_u32(sm + L::T_OFF), 16, 1024),      // K-major
                           g_desc = tc::sdesc_sw128(tc::smem_u32(sm + L::T_OFF), TCHUNK, 1024);  // MN-major
            const uint64_t x_desc = tc::sdesc_sw32(tc::smem_u32(sm + L::AUX_OFF));
            const uint32_t tG = tmem + L::ACC_COL, tGq = MODE == DKV ? tG + DV : tG;
            uint32_t g = 0, works = 0;          // steps whose scores are issued, works before this one
            uint32_t sst = 0, sph = 0, gst = 0; // stage (and phase) of the next scores, of the next gradients
            bool ok = true;
            // The tensor pipe queues only a few MMAs, so a gap of 100 clocks between them is a
            // stall: each barrier is tested (soon) in the middle of the issue before it is
            // needed, and waited for only if it was not there yet.
            auto soon = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, tc::mbar_test(b, parity)); };
            bool t_soon = false;
            if (MODE == DKV) pdl_wait();
            // S and D of step g; p_bar: the barrier that is needed next (null: none), *p_soon: it is there
            auto scores = [&](uint64_t* p_bar, uint32_t p_parity, bool* p_soon) {
                const uint32_t e = g, b = e & 1;
                const uint64_t td = tc::desc_at(t_desc, sst * L::T_BYTES);
                const uint64_t xd = tc::desc_at(x_desc, L::EXT_A + sst * 2 * L::EXT_B);
                const uint32_t tD = tmem + L::D_COL + (L::ND == 2 ? b * 64 : 0);
                if (!t_soon && !warp_wait(&bar.t_full[sst], sph)) return false;
                tc::fence_after_sync();
                bool d_soon = true;
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if (tc::elect_one()) {
#pragma unroll
                        for (int kk = part * (DQK / 32); kk < (part + 1) * (DQK / 32); ++kk)
                            tc::mma_ss(tmem + b * 64, tc::desc_at(r_desc, (kk >> 2) * RCHUNK + (kk & 3) * 32),
                                       tc::desc_at(td, (kk >> 2) * TCHUNK + (kk & 3) * 32), idesc_sd, kk > 0);
                        if (MODE == DKV && part == 1) tc::mma_ss(tmem + b * 64, x_desc, xd, idesc_sd, 1);
                        if (part == 1) tc::mma_commit(&bar.s_full[b]);
                    }
                    __syncwarp();
                    // one D buffer: the step before this one must have read it
                    if (L::ND == 1 && part == 0 && e > 0) d_soon = soon(&bar.d_read[b ^ 1], ((e - 1) >> 1) & 1);
                }
                if (L::ND == 1) {
                    if (!d_soon && !warp_wait(&bar.d_read[b ^ 1], ((e - 1) >> 1) & 1)) return false;
                    tc::fence_after_sync();
                }
#pragma unroll
                for (int part = 0; part < 2; ++part) {
                    if (tc::elect_one()) {
#pragma unroll
                        for (int kk = part * (DV / 32); kk < (part + 1) * (DV / 32); ++kk)
                            tc::mma_ss(tD, tc::desc_at(r_desc, (L::QC + (kk >> 2)) * RCHUNK + (kk & 3) * 32),
                                       tc::desc_at(td, (L::QC + (kk >> 2)) * TCHUNK + (kk & 3) * 32), idesc_sd, kk > 0);
                        if (MODE == DKV && part == 1) tc::mma_ss(tD, x_desc, tc::desc_at(xd, L::EXT_B), idesc_sd, 1);
                        if (part == 1) tc::mma_commit(&bar.d_full[b]);
                    }
                    __syncwarp();
                    if (part == 0 && p_bar) *p_soon = soon(p_bar, p_parity);
                }
                if (++sst == L::NST) sst = 0, sph ^= 1;
                t_soon = false;
                ++g;
                return true;
            };
            for (int round = 0, w; ok && (w = dealt(round)) < a.n_work; ++round) {
                Work k;
                if (!decode_work<MODE>(a, w, &k) || k.n == 0) continue;
                if (!warp_wait(&bar.r_full, works & 1) || !scores(nullptr, 0, nullptr)) { ok = false; break; }
                for (int i = 0; i < k.n; ++i) {
                    const uint32_t e = g - 1, b = e & 1;        // the step of these gradients
                    bool p_soon = false;
                    if (i + 1 < k.n && !scores(&bar.p_full[b], (e >> 1) & 1, &p_soon)) { ok = false; break; }
                    if (i + 2 == k.n || k.n == 1) {             // the residents' last use is issued
                        if (tc::elect_one()) tc::mma_commit(&bar.r_empty);
                        __syncwarp();
                    }
                    const uint64_t gd = tc::desc_at(g_desc, gst * L::T_BYTES);
                    const uint32_t tA = tmem + b * 64, tAq = MODE == DKV ? tA + 32 : tA;
                    const uint32_t acc = i > 0 && (MODE == DKV || i != k.m) ? 1u : 0u;      // (the second walk starts anew)
                    if (i == 0 && !warp_wait(&bar.acc_free, (works & 1) ^ 1)) { ok = false; break; }
                    if (!p_soon && !warp_wait(&bar.p_full[b], (e >> 1) & 1)) { ok = false; break; }
                    tc::fence_after_sync();
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        if (tc::elect_one()) {
                            if (MODE == DKV && part == 0) {
#pragma unroll
                                for (int kk = 0; kk < BN / 16; ++kk)
                                    tc::mma_ts(tG, tA + kk * 8, tc::desc_at(gd, L::QC * TCHUNK + kk * 2048), idesc_v,
                                               kk > 0 ? 1u : acc);
                            }
                            if (MODE == DQ || part == 1) {
#pragma unroll
                                for (int kk = MODE == DQ ? part * 2 : 0; kk < (MODE == DQ ? part * 2 + 2 : 4); ++kk)
                                    tc::mma_ts(tGq, tAq + kk * 8, tc::desc_at(gd, kk * 2048), idesc_q,
                                               kk > 0 ? 1u : acc);
                            }
                            if (part == 1) {
                                tc::mma_commit(&bar.t_empty[gst]);
                                if (i + 1 == k.n) tc::mma_commit(&bar.acc_full);
                            }
                        }
                        __syncwarp();
                        if (part == 0) t_soon = soon(&bar.t_full[sst], sph);    // the next step's rows
                    }
                    if (++gst == L::NST) gst = 0;
                }
                ++works;
            }
            if (!ok && lane == 0) give_up();
            if (tc::elect_one()) tc::mma_commit(&bar.drain);    // every MMA has completed before TMEM is freed
            tc::mbar_wait_bounded(&bar.drain, 0, WAIT_NS);
        } else if (MODE == DQ && warp >= 2) {
            // ------------------------------------------------ (lse, delta) of a query tile's rows
            // warps 2 and 3 take half of the rows, a tile ahead; the first tile's are the softmax warps'
            uint32_t n = 0;
            bool ok = true;
            for (int round = 0, w; ok && (w = dealt(round)) < a.n_work; ++round, ++n) {
                const int buf = n & 1, half = (warp - 2) * (BM / 2);
                if (!warp_wait(&bar.aux_empty[buf], ((n >> 1) & 1) ^ 1)) { ok = false; break; }
                if (n > 0) {
                    Work k;
                    decode_work<MODE>(a, w, &k);
                    rows_delta<DV, BM / 2, 4>(a, k, half, lane, aux + buf * BM + half);
                }
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.aux_full[buf]);
            }
            if (!ok) give_up();
        } else if (MODE == DKV && warp >= 2) {
            // ------------------------------------------------ (lse, delta) of a step's rows
            // As 16 more columns of the products: -lse / scale and -delta, each the sum of
            // three bf16 (24 bits), against the residents' (1, 1, 1, 0, ..).  S and D then come
            // as q.k - lse / scale and do.v - delta, and the threads, whose columns the
            // queries are, need no other value of theirs.  Warps 2 and 3 take the steps in
            // turn; the values of a warp's next step are on their way while it writes this one's.
            pdl_wait();                             // delta
            const float inv_scale = 1.f / s.scale;
            auto three = [](float v) {
                const __nv_bfloat16 h = __float2bfloat16_rn(v);
                const float r1 = v - bf2f(h);
                const __nv_bfloat16 m = __float2bfloat16_rn(r1);
                return make_uint4(tc::pack_bf16x2(bf2f(h), bf2f(m)), tc::pack_bf16x2(r1 - bf2f(m), 0.f), 0, 0);
            };
            int tt[2], head[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                tt[e] = (lane + 32 * e) / s.G;
                head[e] = lane + 32 * e - tt[e] * s.G;
            }
            Work k;
            int round = -1, i = 0;
            uint32_t g = 0;                         // step i of work k, of all steps
            // the next step of an odd (warp 3) or even number; false: there is none
            auto advance = [&](int by) {
                i += by;
                g += by;
                while (round < 0 || i >= k.n) {
                    if (round >= 0) i -= k.n;
                    const int w = dealt(++round);
                    if (w >= a.n_work) return false;
                    if (!decode_work<MODE>(a, w, &k)) k.n = 0;
                }
                return true;
            };
            auto load = [&](float2* v) {
                const int first = k.token(i, a.tok);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    v[e] = make_float2(3e38f, 0.f);             // p = 0: no query
                    if (tt[e] < a.tok && first + tt[e] < s.Tq) {
                        const size_t row = ((size_t)k.b * s.Tq + first + tt[e]) * s.Hq + k.kvh * s.G + head[e];
                        v[e] = make_float2(bwd_lse(a.lse[row]), a.delta[row]);
                    }
                }
            };
            bool ok = true;
            float2 v[2], next[2];
            bool more = advance(warp - 2);
            if (more) load(next);
            while (more) {
                const uint32_t e0 = g;
                v[0] = next[0];
                v[1] = next[1];
                more = advance(2);
                if (more) load(next);
                const int st = e0 % L::NST;
                if (!warp_wait(&bar.t_empty[st], ((e0 / L::NST) & 1) ^ 1)) { ok = false; break; }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int r = lane + 32 * e, half = (r >> 2) & 1;
                    uint4* x = reinterpret_cast<uint4*>(sm + L::AUX_OFF + L::EXT_A + st * 2 * L::EXT_B + r * 32);
                    // (of a row without a query: -3e38, not times 1 / scale, which could pass fp32)
                    x[half] = three(v[e].x == 3e38f ? -3e38f : -v[e].x * inv_scale);
                    x[half ^ 1] = make_uint4(0, 0, 0, 0);
                    x[L::EXT_B / 16 + half] = three(-v[e].y);
                    x[L::EXT_B / 16 + (half ^ 1)] = make_uint4(0, 0, 0, 0);
                }
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.t_full[st]);
            }
            if (!ok) give_up();
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 208;" ::: "memory");
        // ---------------------------------------------------- P and dS of every second step, gradients out
        const int wg = (warp - 4) >> 2;
        const int r = (warp & 3) * 32 + lane;
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + wg * 64 + lane_off;
        const uint32_t tD = tmem + L::D_COL + (L::ND == 2 ? wg * 64 : 0) + lane_off;
        const uint32_t tG = tmem + L::ACC_COL + lane_off;
        const int tt = r / s.G;
        TileRows tile_rows;
        if (MODE == DQ) tile_rows.init(r, s.G);
        uint32_t g = 0, works = 0, n = 0, walks = 0;
        bool ok = true;
        bool clamp = false;                         // a large lse could lift exponents above 0 (bwd_lse)
        if (MODE == DKV) {
            pdl_wait();
            for (int i = lane; i < a.n_flags; i += 32) clamp |= a.flags[i] != 0;
            clamp = __any_sync(0xffffffffu, clamp);
        }
        for (int round = 0, w; ok && (w = dealt(round)) < a.n_work; ++round) {
            Work k;
            if (!decode_work<MODE>(a, w, &k)) continue;
            float2 mine = make_float2(0.f, 0.f);
            const int pos = MODE == DQ ? s.q0 + k.first + tt : k.first + r;     // query position or key
            if (MODE == DQ) {
                const int buf = n & 1;
                if (n == 0) {                       // with eight warps: 16 rows each, in one step
                    constexpr int SHARE = BM / 8;
                    rows_delta<DV, SHARE, SHARE * DV / 256>(a, k, (warp - 4) * SHARE, lane, aux + (warp - 4) * SHARE);
                    asm volatile("bar.sync 1, 256;" ::: "memory");
                }
                if (!warp_wait(&bar.aux_full[buf], (n >> 1) & 1)) { ok = false; break; }
                mine = aux[buf * BM + r];
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.aux_empty[buf]);
                ++n;
            }
            if (MODE == DQ) {                       // (infinity: not a row)
                clamp = __any_sync(0xffffffffu, fabsf(mine.x) > LARGE_LSE && mine.x != INFINITY);
                if (clamp) *large = 1;
            }
            // exponents are scores times sc2 + lse2, or, to be clamped, taken beforehand
            const uint64_t sc2 = clamp ? tc::f2_pack(1.f, 1.f) : tc::f2_pack(a.scale_log2, a.scale_log2);
            const float neg = clamp ? 0.f : -mine.x;
            const uint64_t lse2 = tc::f2_pack(neg, neg);
            uint64_t del2 = tc::f2_pack(-mine.y, -mine.y), ds_sum[2] = {0, 0};
            for (int i = 0; i < k.n; ++i, ++g) {
                if (MODE == DQ && i == k.m) {       // the first walk is done
                    float* sum = reinterpret_cast<float*>(sm + L::SUM_OFF) + (walks & 1) * 2 * BM;
                    float s0, s1;
                    tc::f2_unpack(tc::f2_add(ds_sum[0], ds_sum[1]), s0, s1);
                    sum[wg * BM + r] = s0 + s1;
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.sum_full);
                    if (!warp_wait(&bar.sum_full, walks & 1)) { ok = false; break; }
                    ++walks;
                    const float delta = mine.y + (sum[r] + sum[BM + r]);
                    del2 = tc::f2_pack(-delta, -delta);
                    if (wg == 0 && tt < min(a.tok, s.Tq - k.first))        // for DKV, over the one of the rounded out
                        a.delta[((long long)k.b * s.Tq + k.first + tt) * s.Hq + k.kvh * s.G + (r - tt * s.G)] = delta;
                }
                if ((int)(g & 1) != wg) continue;
                if (!warp_wait(&bar.s_full[wg], (g >> 1) & 1)) { ok = false; break; }
                tc::fence_after_sync();
                uint32_t x[64], y[64];
                tc::tmem_ld32(tS, x);
                tc::tmem_ld32(tS + 32, x + 32);
                // visible columns [lo, hi] and [0, sk)
                int lo, hi, sk = 0;
                if (MODE == DQ) {
                    const int u0 = k.key(i);
                    if (k.sink_step(i)) {
                        lo = 0;
                        hi = k.sl - 1 - u0;
                    } else {
                        lo = pos - s.win + 1 - u0;
                        hi = pos - u0;
                        sk = min(s.ns - u0, hi + 1);
                    }
                } else {
                    // tokens from pos on, up to pos + win - 1 unless the key is a sink
                    const int tb = s.q0 + k.token(i, a.tok);
                    lo = max(min(pos - tb, BN), -BN) * s.G;
                    hi = pos < s.ns ? BN - 1 : max(min(pos - tb + s.win, BN), -BN) * s.G - 1;
                }
                tc::tmem_wait_ld32(x);
                tc::tmem_wait_ld32(x + 32);
                const bool full = hi >= BN - 1 && (lo <= 0 || sk >= BN);
                if (!__all_sync(0xffffffffu, full && !clamp)) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t bits = range_bits(lo, hi, c) | range_bits(0, sk - 1, c);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((bits >> e) & 1u)) x[32 * c + e] = 0xFF800000u;
                    }
                    if (clamp) {                    // (bwd_lse)
#pragma unroll
                        for (int c = 0; c < 64; ++c)
                            x[c] = __float_as_uint(at_most_0(fmaf(__uint_as_float(x[c]), a.scale_log2, -mine.x)));
                    }
                }
                // (DKV: mine = 0, S and D carry the queries' lse and delta)
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    float y0, y1;
                    tc::f2_unpack(tc::f2_fma(tc::f2_pack(__uint_as_float(x[c]), __uint_as_float(x[c + 1])), sc2, lse2),
                                  y0, y1);
                    x[c] = __float_as_uint(tc::ex2(y0));
                    x[c + 1] = __float_as_uint(tc::ex2(y1));
                }
                if (!warp_wait(&bar.d_full[wg], (g >> 1) & 1)) { ok = false; break; }
                tc::fence_after_sync();
                tc::tmem_ld32(tD, y);
                tc::tmem_ld32(tD + 32, y + 32);
                tc::tmem_wait_ld32(y);
                tc::tmem_wait_ld32(y + 32);
                if (L::ND == 1) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&bar.d_read[wg]);
                }
                // bf16 weights and ds: half a step, 2^-8 relative of each term at most
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    const uint64_t p2 = tc::f2_pack(__uint_as_float(x[c]), __uint_as_float(x[c + 1]));
                    const uint64_t d2 = tc::f2_pack(__uint_as_float(y[c]), __uint_as_float(y[c + 1]));
                    float e0, e1;
                    const uint64_t ds2 = tc::f2_mul(p2, MODE == DQ ? tc::f2_add(d2, del2) : d2);
                    if (MODE == DQ) ds_sum[(c >> 1) & 1] = tc::f2_add(ds_sum[(c >> 1) & 1], ds2);
                    tc::f2_unpack(ds2, e0, e1);
                    y[c / 2] = tc::pack_bf16x2(e0, e1);
                    x[c / 2] = tc::pack_bf16x2(__uint_as_float(x[c]), __uint_as_float(x[c + 1]));
                }
                if (MODE == DKV) {
                    tc::tmem_st32(tS, x);
                    tc::tmem_st32(tS + 32, y);
                } else {
                    tc::tmem_st32(tS, y);
                }
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.p_full[wg]);
            }
            if (!ok) break;
            if (k.n > 0) {
                if (!warp_wait(&bar.acc_full, works & 1)) { ok = false; break; }
                tc::fence_after_sync();
            }
            // this warpgroup's 32-column pieces of the accumulator rows
            auto acc_read = [&]() {                 // the next work may overwrite the accumulators
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.acc_free);
            };
            if (MODE == DQ) {
                // all pieces into registers first: the next query tile's products start while
                // they are stored
                constexpr int PIECES = DQK / 64;
                uint4 u[PIECES][4];
#pragma unroll
                for (int p = 0; p < PIECES; ++p) {
                    uint32_t o[32];
                    tc::tmem_ld32(tG + wg * 32 + 64 * p, o);
                    tc::tmem_wait_ld32(o);
                    pack32(o, s.scale, u[p]);
                }
                acc_read();
                const OutRows rows = tile_rows.at(((long long)k.b * s.Tq + k.first) * s.Hq + k.kvh * s.G,
                                                  min(a.tok, s.Tq - k.first), s.Hq);
#pragma unroll
                for (int p = 0; p < PIECES; ++p) store_bf16x32(u[p], a.dq, rows, DQK, wg * 32 + 64 * p, lane);
                ++works;
            } else {
                OutRows rows;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int rj = (r & ~3) + j, u = k.first + rj;
                    rows.off[j] = u >= s.Tk       ? -1
                                  : k.slot >= 0 ? (long long)k.slot * BM + rj
                                                : ((long long)k.b * s.Hkv + k.kvh) * s.Tk + u;
                }
#pragma unroll 1
                for (int c = wg * 32; c < L::ACC; c += 64) {
                    uint32_t o[32];
                    uint4 u[4];
                    if (k.n > 0) {
                        tc::tmem_ld32(tG + c, o);
                        tc::tmem_wait_ld32(o);
                    } else {                        // keys that no query sees
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = 0u;
                    }
                    if (k.slot >= 0) {
                        store_f32x32(o, a.part, rows, L::ACC, c, lane);
                    } else {
                        pack32(o, c < DV ? 1.f : s.scale, u);
                        if (c < DV) store_bf16x32(u, a.dv, rows, DV, c, lane);
                        else store_bf16x32(u, a.dk, rows, DQK, c - DV, lane);
                    }
                }
                if (k.n > 0) {
                    acc_read();
                    ++works;
                }
            }
        }
        if (!ok) give_up();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_dealloc(tmem, 512);
    if (MODE == DQ && threadIdx.x == 0) a.flags[blockIdx.x] = *large;
}

// Adds the items' partial sums of a split key tile, in order: one thread per
// (row, four columns), JROWS rows per CTA.
constexpr int JROWS = 4;

template <int DQK, int DV>
__global__ void __launch_bounds__(JROWS*(DQK + DV) / 4) window_bwd_join_kernel(const Args a) {
    constexpr int C4 = (DQK + DV) / 4;
    const WinShape& s = a.s;
    const int planes = s.B * s.Hkv;
    const int plane = blockIdx.x % planes, kt = blockIdx.x / planes;
    const bool sinks = kt < a.p.nsk;
    int i0, i1;
    tile_queries(s, kt * BM, &i0, &i1);
    const int items = ceil_div(ceil_div(i1 - i0, a.tok), sinks ? a.p.chunk_s : a.p.chunk_o);
    pdl_wait();
    if (items <= 1) return;
    const int tiles = sinks ? a.p.nsk : a.p.nk - a.p.nsk, sp = sinks ? a.p.sp_s : a.p.sp_o;
    const size_t slot = (sinks ? 0 : a.p.slots_s) + (size_t)(plane * tiles + kt - (sinks ? 0 : a.p.nsk)) * sp;
    const int r = blockIdx.y * JROWS + threadIdx.x / C4, c = (threadIdx.x % C4) * 4;
    const int u = kt * BM + r;
    if (u >= s.Tk) return;
    const float4* src = reinterpret_cast<const float4*>(a.part + (slot * BM + r) * (DQK + DV) + c);
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
    for (int i = 0; i < items; ++i) {
        const float4 x = src[(size_t)i * BM * C4];
        t = make_float4(t.x + x.x, t.y + x.y, t.z + x.z, t.w + x.w);
    }
    const size_t row = (size_t)plane * s.Tk + u;
    const float f = c < DV ? 1.f : s.scale;
    __nv_bfloat16* dst = c < DV ? a.dv + row * DV + c : a.dk + row * DQK + (c - DV);
    *reinterpret_cast<uint2*>(dst) = make_uint2(tc::pack_bf16x2(t.x * f, t.y * f), tc::pack_bf16x2(t.z * f, t.w * f));
}

Split make_split(const WinShape& s) {
    Split p;
    const int tok = BN / s.G;
    const long long planes = (long long)s.B * s.Hkv;
    p.nk = ceil_div(s.Tk, BM);
    p.nsk = ceil_div(s.ns, BM);
    const int n_s = ceil_div(s.Tq, tok);                        // steps of a key tile that every query sees
    const int n_o = std::min(n_s, (int)(((long long)BM + s.win + tok - 2) / tok));     // of one the window sees
    const int others = p.nk - p.nsk;
    const long long total = planes * ((long long)p.nsk * n_s + (long long)others * n_o);
    // items of about half an SM's share; whole key tiles where there are enough of them
    const int half = (int)std::min<long long>(std::max<long long>((total / SMS + 1) / 2, MIN_CHUNK), INT32_MAX);
    p.chunk_s = std::max(1, std::min(half, n_s));
    p.chunk_o = std::max(1, planes * others >= 2 * SMS ? n_o : std::min(half, n_o));
    p.sp_s = p.nsk > 0 ? ceil_div(n_s, p.chunk_s) : 1;
    p.sp_o = others > 0 ? ceil_div(n_o, p.chunk_o) : 1;
    p.slots_s = p.sp_s > 1 ? (int)(planes * p.nsk * p.sp_s) : 0;
    return p;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

size_t part_slots(const WinShape& s, const Split& p) {
    return (size_t)p.slots_s + (p.sp_o > 1 ? (size_t)s.B * s.Hkv * (p.nk - p.nsk) * p.sp_o : 0);
}

template <int DQK, int DV>
cudaError_t launch_impl(Args a, const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                        cudaStream_t st) {
    const WinShape& s = a.s;
    const int planes = s.B * s.Hkv;
    int dev, nsm;
    cudaError_t e = sm_count(&nsm, &dev);
    if (e != cudaSuccess) return e;
    static std::atomic<bool> dq_allowed[MAX_DEVICES], dkv_allowed[MAX_DEVICES];
    const int tok_q = BM / s.G, tok_s = BN / s.G;
    CUtensorMap q128, do128, k64, v64, k128, v128, q64, do64;
    if (!tmap::heads_map(&q128, q, DQK, s.Hq, s.Tq, s.B, s.G, tok_q) ||
        !tmap::heads_map(&do128, a.d_out, DV, s.Hq, s.Tq, s.B, s.G, tok_q) ||
        !tmap::heads_map(&q64, q, DQK, s.Hq, s.Tq, s.B, s.G, tok_s) ||
        !tmap::heads_map(&do64, a.d_out, DV, s.Hq, s.Tq, s.B, s.G, tok_s) ||
        !tmap::rows_map(&k64, k, DQK, s.Tk, planes, BN) || !tmap::rows_map(&v64, v, DV, s.Tk, planes, BN) ||
        !tmap::rows_map(&k128, k, DQK, s.Tk, planes, BM) || !tmap::rows_map(&v128, v, DV, s.Tk, planes, BM))
        return cudaErrorInvalidValue;
    {
        using L = Smem<DQK, DV, DQ>;
        auto kernel = window_bwd_tc_kernel<DQK, DV, DQ>;
        e = allow_smem(reinterpret_cast<const void*>(kernel), L::ALLOC, dev, dq_allowed);
        if (e != cudaSuccess) return e;
        a.tok = tok_q;
        a.n_tt = ceil_div(s.Tq, tok_q);
        a.n_work = a.n_tt * planes;
        a.n_flags = std::min(std::min(a.n_work, nsm), MAX_FLAGS);
        kernel<<<a.n_flags, THREADS, L::ALLOC, st>>>(q128, do128, k64, v64, a);
        e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    using L = Smem<DQK, DV, DKV>;
    auto kernel = window_bwd_tc_kernel<DQK, DV, DKV>;
    e = allow_smem(reinterpret_cast<const void*>(kernel), L::ALLOC, dev, dkv_allowed);
    if (e != cudaSuccess) return e;
    a.tok = tok_s;
    a.n_work = planes * (a.p.nsk * a.p.sp_s + (a.p.nk - a.p.nsk) * a.p.sp_o);
    e = launch_dependent(kernel, dim3(std::min(a.n_work, nsm)), THREADS, L::ALLOC, st, k128, v128, q64, do64, a);
    if (e != cudaSuccess || (a.p.sp_s <= 1 && a.p.sp_o <= 1)) return e;
    const int tiles = a.p.sp_o > 1 ? a.p.nk : a.p.nsk;
    return launch_dependent(window_bwd_join_kernel<DQK, DV>, dim3(tiles * planes, BM / JROWS), JROWS * (DQK + DV) / 4, 0,
                            st, a);
}

}  // namespace

size_t window_bwd_tc_part_bytes(const WinShape& s) {
    const Split p = make_split(s);
    return MAX_FLAGS * 4 + up256(part_slots(s, p) * BM * (s.dqk + s.dv) * 4);
}

cudaError_t launch_window_bwd_tc(const WinShape& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                 const __nv_bfloat16* v, const __nv_bfloat16* out, const float* lse,
                                 const __nv_bfloat16* d_out, __nv_bfloat16* dq, __nv_bfloat16* dk,
                                 __nv_bfloat16* dv, float* delta, float* part, cudaStream_t st) {
    Args a;
    a.s = s;
    a.p = make_split(s);
    a.out = out;
    a.d_out = d_out;
    a.lse = lse;
    a.delta = delta;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.flags = reinterpret_cast<int*>(part);
    a.part = part + MAX_FLAGS;
    a.tok = a.n_tt = a.n_work = a.n_flags = 0;
    // Neighbouring key tiles read the same rows of q and d_out.  While these fit the L2 (126 MB)
    // beside everything else, each tile takes them in its own order (4096 tokens, 16 heads, d 128,
    // 34 MB: 358 us a training step, 368 turned: every CTA asks for the same lines at once); larger
    // ones would come from HBM once per key tile (8192 tokens, 64 heads, 336 MB: 1127 us, 1071 turned).
    a.turned = (size_t)s.B * s.Tq * s.Hq * (s.dqk + s.dv) * 2 > ((size_t)64 << 20);
    a.scale_log2 = s.scale * LOG2E;
#define NSA_WIN_CASE(A, B) \
    if (s.dqk == A && s.dv == B) return launch_impl<A, B>(a, q, k, v, st);
    NSA_WIN_CASE(64, 64)
    NSA_WIN_CASE(64, 128)
    NSA_WIN_CASE(128, 64)
    NSA_WIN_CASE(128, 128)
    NSA_WIN_CASE(192, 64)
    NSA_WIN_CASE(192, 128)
#undef NSA_WIN_CASE
    return cudaErrorInvalidValue;
}

cudaError_t set_win_bwd_wait_limit(uint64_t limit_ns) {
    const uint64_t v = limit_ns ? limit_ns : WAIT_NS;
    return cudaMemcpyToSymbol(c_win_bwd_wait_ns, &v, sizeof(v));
}

int read_and_clear_win_bwd_status() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_win_bwd_status, sizeof(int)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_win_bwd_status, &zero, sizeof(int));
    return v;
}

}  // namespace nsa
