// Sliding-window attention with sink tokens on the 5th-generation tensor cores
// (tcgen05 + TMEM + TMA), forward.
//
// Transcript #94 (bidclub.ai) §4 (window and attention sink), §5 (the heads of
// a group stacked as rows of one product with their shared keys).  With
// s_u = scale q.k_u over the visible keys, x_u = s_u log2 e:
//   S = Q K^T;  p_u = 2^(x_u - m), m a running reference of the row;
//   O += P V;  l += sum p;  out = O / l;  lse = ln 2 (m + log2 l).
// The reference moves only when the row's maximum passes it by more than 2^8
// (any reference gives the same quotient; 2^8 keeps p far from overflow), so O
// is rarely rescaled.  p enters P V rounded to bf16, l sums it unrounded.
//
// A query tile is 128 rows: 128 / G tokens (rounded down) x the G heads of a
// KV head.  A CTA takes two neighbouring query tiles with the same keys and
// walks their key tiles of 128: first the sinks' (when they lie before the
// window), then the window's.  While one tile's softmax runs, the tensor
// cores work for the other; the single issuing lane's order is
//   S0(0) S1(0) | O0(0) S0(1) O1(0) S1(1) | O0(1) S0(2) O1(1) S1(2) | ...
// As tcgen05 operations of one lane complete in order, S_t(j + 1) being there
// means that O_t(j) is: the softmax may then rescale O and overwrite P without
// another wait.
//
// Warps (384 threads): 0 loads Q and K, 1 issues the MMAs, 2 loads V, 3 idle;
// 4-7 softmax and epilogue of tile 0, 8-11 of tile 1, one thread per row.
// TMEM: S0, S1 (128 columns each, P over them as bf16), O0, O1 (d_v each).
// Shared memory at d 192/128: Q 2 x 48 KB, K 2 x 48 KB, V 32 KB.
// Bound by the tensor cores: a pair of tiles needs 2 x 128 x 128 x (d_qk + d_v)
// MACs per key tile at 4096 a clock, its exponentials 2 x 16384 at 16 a clock;
// in fact by the round trip softmax -> P V, Q K^T -> softmax of each tile, in
// which both pipes are about half busy (without any softmax 136 us of 175).
// Measured in bursts, on two cards: 2 x 8192 tokens, 16 heads, d 128, window
// 1000 + 16: 177 and 186 us, 722 and 687 TFLOP/s; 16384 tokens, 64 heads on 4,
// 192/128, window 512 + 64: 417 and 430 us, 911 and 884 TFLOP/s (196-202 and
// 485-496 us back to back under the power cap).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "launch.cuh"
#include "rows_out.cuh"
#include "tc.cuh"
#include "tmap.cuh"
#include "window.cuh"

namespace nsa {

__device__ int g_win_fwd_status = 0;
// Limit of the roles' waits (WAIT_NS unless nsa_set_wait_limit_ns shortened it); the drains keep WAIT_NS.
__constant__ uint64_t c_win_fwd_wait_ns = 1000000000ull;

namespace {

constexpr int BM = 128, BN = 128;
constexpr int CHUNK = 16384;                    // 128 rows x 64 columns of bf16
constexpr int THREADS = 384;
constexpr uint64_t WAIT_NS = 1000000000ull;
// From this |m| on a row takes the largest power of two below scale log2 e for its scale.  The weights
// 2^(fma(s, c2, -m)) carry the rounding of m, up to here 2^5 at most: a power that O and l share.
// From here on it would pass fp32's range, so m = maximum 2^i is exact; and as different scores are 2^5
// or more apart, a smaller scale moves no weight by more than 2^-32.
constexpr float LARGE_REF = 1073741824.f;

template <int DQK, int DV>
struct Smem {
    static constexpr int QC = DQK / 64, VC = DV / 64;
    static constexpr int KS = 2;
    static constexpr int ROOM = 227 * 1024 - 1024 - 512 - (2 + KS) * QC * CHUNK;
    static constexpr int VS = ROOM / (VC * CHUNK) >= 2 ? 2 : 1;
    static constexpr int Q_OFF = 0;
    static constexpr int K_OFF = 2 * QC * CHUNK;
    static constexpr int V_OFF = K_OFF + KS * QC * CHUNK;
    static constexpr int BAR_OFF = V_OFF + VS * VC * CHUNK;
    static constexpr int ALLOC = BAR_OFF + 512 + 1024;      // slack to align the base to 1024 B
};

struct Bars {
    uint64_t q_full[2], q_empty[2], k_full[2], k_empty[2], v_full[2], v_empty[2];
    uint64_t s_full[2], p_full[2], o_full[2], drain;
    uint32_t tmem;
    int abort;
};

struct Args {
    WinShape s;
    __nv_bfloat16* out;
    float* lse;
    int tok;        // tokens per query tile
    int n_tt;       // query tiles per (sequence, KV head)
    int nt;         // query tiles per work item (1 or 2)
    int n_work;
    float scale_log2;
};

// One work item: query tiles tt0 .. tt0 + nt - 1 of one (sequence, KV head) and
// the key tiles that any of them needs.  Query tile t needs the key tiles
// [0, c[t]) (sinks) and [f[t], e[t]) (window); e[t] = 0 if it does not exist.
struct Work {
    int b, kvh, tt0, nt;
    int pf[2];          // first position of each query tile
    int c[2], f[2], e[2];
    int nst;            // key tiles of the sinks before the window
    int sl;             // those sinks: keys [0, sl)
    int lo;             // first key of the window's tiles
    int n;              // key tiles in all
    int last;           // last key that is needed

    __device__ __forceinline__ int key(int j) const { return j < nst ? j * BN : lo + (j - nst) * BN; }
    // keys of tile j, rounded up to 32
    __device__ __forceinline__ int width(int j) const {
        const int left = (j < nst ? sl : last + 1) - key(j);
        return left >= BN ? BN : (left + 31) & ~31;
    }
    __device__ __forceinline__ bool needs(int t, int j) const { return j < e[t] && (j >= f[t] || j < c[t]); }
};

__device__ __forceinline__ Work decode_work(const Args& a, int w) {
    const WinShape& s = a.s;
    const int planes = s.B * s.Hkv;
    const int items = (a.n_tt + a.nt - 1) / a.nt;
    Work k;
    k.tt0 = (items - 1 - w / planes) * a.nt;    // the latest (with most keys) first
    const int r = w % planes;
    k.b = r / s.Hkv;
    k.kvh = r % s.Hkv;
    k.nt = min(a.nt, a.n_tt - k.tt0);
    k.pf[0] = s.q0 + k.tt0 * a.tok;
    k.pf[1] = k.pf[0] + a.tok;
    const int end = s.q0 + s.Tq;
    k.last = min(k.pf[0] + k.nt * a.tok, end) - 1;
    k.lo = max(0, k.pf[0] - s.win + 1);
    k.sl = min(s.ns, k.lo);
    k.nst = (k.sl + BN - 1) / BN;
    // They meet, or sinks lie in the window's tiles (which the second query tile may need for
    // these alone): one range from 0.
    if (k.lo < k.nst * BN || s.ns > k.lo) k.lo = k.sl = k.nst = 0;
    k.n = k.nst + (k.last - k.lo) / BN + 1;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const int first = max(0, k.pf[t] - s.win + 1), pl = min(k.pf[t] + a.tok, end) - 1;
        // tiles that start below ns hold sinks (k.nst of them, or some of the one range)
        k.c[t] = k.nst > 0 ? k.nst : (max(0, s.ns - k.lo) + BN - 1) / BN;
        k.f[t] = k.nst + (first - k.lo) / BN;
        k.e[t] = t < k.nt ? k.nst + (pl - k.lo) / BN + 1 : 0;
        k.c[t] = min(k.c[t], k.e[t]);
    }
    return k;
}

// Bits k of [0, 32 w + 32) in [lo, hi] for word w.
__device__ __forceinline__ uint32_t range_bits(int lo, int hi, int w) {
    const int a = max(lo - 32 * w, 0), b = min(hi - 32 * w, 31);
    if (b < a) return 0u;
    return (0xFFFFFFFFu >> (31 - b)) & (0xFFFFFFFFu << a);
}

template <int DQK, int DV>
__global__ void __launch_bounds__(THREADS, 1)
    window_fwd_tc_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                         const __grid_constant__ CUtensorMap map_v, const Args a) {
    using L = Smem<DQK, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    Bars& bar = *reinterpret_cast<Bars*>(sm + L::BAR_OFF);
    volatile int* abort_flag = &bar.abort;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const WinShape& s = a.s;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            tc::mbar_init(&bar.q_full[i], 1);
            tc::mbar_init(&bar.q_empty[i], 1);
            tc::mbar_init(&bar.k_full[i], 1);
            tc::mbar_init(&bar.k_empty[i], 1);
            tc::mbar_init(&bar.v_full[i], 1);
            tc::mbar_init(&bar.v_empty[i], 1);
            tc::mbar_init(&bar.s_full[i], 1);
            tc::mbar_init(&bar.p_full[i], 4);
            tc::mbar_init(&bar.o_full[i], 1);
        }
        tc::mbar_init(&bar.drain, 1);
        bar.abort = 0;
        tc::fence_mbar_init();
        tc::prefetch_map(&map_q);
        tc::prefetch_map(&map_k);
        tc::prefetch_map(&map_v);
    }
    if (warp == 1) {
        tc::tmem_alloc(&bar.tmem, 512);
        tc::tmem_relinquish();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    const uint32_t tmem = bar.tmem;
    auto wait = [&](uint64_t* b, uint32_t parity) { return tc::mbar_wait(b, parity, abort_flag, c_win_fwd_wait_ns); };
    auto give_up = [&]() {
        *abort_flag = 1;
        atomicExch(&g_win_fwd_status, (int)NSA_ERR_TIMEOUT);
    };

    if (warp < 4) {
        // 4 x 32 x 104 + 8 x 32 x 200 = 64512, the 384 x 168 registers of the launch
        asm volatile("setmaxnreg.dec.sync.aligned.u32 104;" ::: "memory");
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------ Q and K
            uint32_t nq[2] = {0, 0}, nk = 0;
            bool ok = true;
            const uint32_t q_bytes = (uint32_t)(L::QC * a.tok * s.G * 128);
            for (int w = blockIdx.x; ok && w < a.n_work; w += gridDim.x) {
                const Work k = decode_work(a, w);
                const int plane = k.b * s.Hkv + k.kvh;
                for (int j = 0; ok && j < k.n; ++j) {
                    const int st = nk % L::KS;
                    if (j == 0) {
                        // the first query tile goes before the first keys, the second behind them
                        if (!wait(&bar.q_empty[0], (nq[0] & 1) ^ 1)) { ok = false; break; }
                        tc::mbar_arrive_expect_tx(&bar.q_full[0], q_bytes);
                        for (int c = 0; c < L::QC; ++c)
                            tc::tma_load_4d(sm + L::Q_OFF + c * CHUNK, &map_q, &bar.q_full[0], 64 * c, k.kvh * s.G,
                                            k.tt0 * a.tok, k.b);
                        ++nq[0];
                    }
                    if (!wait(&bar.k_empty[st], ((nk / L::KS) & 1) ^ 1)) { ok = false; break; }
                    tc::mbar_arrive_expect_tx(&bar.k_full[st], L::QC * CHUNK);
                    for (int c = 0; c < L::QC; ++c)
                        tc::tma_load_3d(sm + L::K_OFF + (st * L::QC + c) * CHUNK, &map_k, &bar.k_full[st], 64 * c,
                                        k.key(j), plane);
                    ++nk;
                    if (j == 0 && k.nt == 2) {
                        if (!wait(&bar.q_empty[1], (nq[1] & 1) ^ 1)) { ok = false; break; }
                        tc::mbar_arrive_expect_tx(&bar.q_full[1], q_bytes);
                        for (int c = 0; c < L::QC; ++c)
                            tc::tma_load_4d(sm + L::Q_OFF + (L::QC + c) * CHUNK, &map_q, &bar.q_full[1], 64 * c,
                                            k.kvh * s.G, (k.tt0 + 1) * a.tok, k.b);
                        ++nq[1];
                    }
                }
            }
            if (!ok) give_up();
            // every copy issued here has landed before the CTA ends
            for (uint32_t i = 0; i < L::KS && i < nk; ++i) {
                const uint32_t last = i + ((nk - 1 - i) / L::KS) * L::KS;
                tc::mbar_wait_bounded(&bar.k_full[i], (last / L::KS) & 1, WAIT_NS);
            }
            for (int t = 0; t < 2; ++t)
                if (nq[t] > 0) tc::mbar_wait_bounded(&bar.q_full[t], (nq[t] - 1) & 1, WAIT_NS);
        } else if (warp == 2 && lane == 0) {
            // ------------------------------------------------ V
            uint32_t nv = 0;
            bool ok = true;
            for (int w = blockIdx.x; ok && w < a.n_work; w += gridDim.x) {
                const Work k = decode_work(a, w);
                const int plane = k.b * s.Hkv + k.kvh;
                for (int j = 0; j < k.n; ++j) {
                    const int st = nv % L::VS;
                    if (!wait(&bar.v_empty[st], ((nv / L::VS) & 1) ^ 1)) { ok = false; break; }
                    tc::mbar_arrive_expect_tx(&bar.v_full[st], L::VC * CHUNK);
                    for (int c = 0; c < L::VC; ++c)
                        tc::tma_load_3d(sm + L::V_OFF + (st * L::VC + c) * CHUNK, &map_v, &bar.v_full[st], 64 * c,
                                        k.key(j), plane);
                    ++nv;
                }
            }
            if (!ok) give_up();
            for (uint32_t i = 0; i < L::VS && i < nv; ++i) {
                const uint32_t last = i + ((nv - 1 - i) / L::VS) * L::VS;
                tc::mbar_wait_bounded(&bar.v_full[i], (last / L::VS) & 1, WAIT_NS);
            }
        } else if (warp == 1) {
            // ------------------------------------------------ MMA issue
            // The whole warp walks the schedule, one lane issues: with the operands in
            // uniform registers an MMA costs a few issue slots beside the softmax warps.
            const uint32_t idesc_pv = tc::idesc_bf16_f32(BM, DV, false, true);
            const uint64_t q_desc = tc::sdesc_sw128(tc::smem_u32(sm + L::Q_OFF), 16, 1024),
                           k_desc = tc::sdesc_sw128(tc::smem_u32(sm + L::K_OFF), 16, 1024),
                           v_desc = tc::sdesc_sw128(tc::smem_u32(sm + L::V_OFF), CHUNK, 1024);
            auto uwait = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)); };
            // The loops stay rolled: the short code is a little faster than the unrolled one (at the
            // two sizes of the head comment 175.6 us against 177.0 and 424.9 against 433.9).
            uint32_t ks = 0, kph = 0, vs = 0, vph = 0;      // stage and phase of the next key / value tile
            uint32_t nq = 0, np = 0;                        // bit t: parity of tile t's next Q, next P
            bool ok = true;
            for (int w = blockIdx.x; ok && w < a.n_work; w += gridDim.x) {
                const Work k = decode_work(a, w);
                int wp = 0;                     // width of key tile j - 1
                uint32_t pv = 0;                // bit t: P V of key tile j - 1 is still to be issued
                // Per key tile j and query tile t: one look at the barriers (a wait for those
                // that are not there yet) and one run of MMAs, P V of j - 1 and Q K^T of j.
#pragma unroll 1
                for (int j = 0; ok && j <= k.n; ++j) {
                    const int wj = j < k.n ? k.width(j) : 0;
                    const uint32_t idesc_w = tc::idesc_bf16_f32(BM, 0, false, false) | ((uint32_t)(wj >> 3) << 17);
                    const uint64_t kd = tc::desc_at(k_desc, ks * L::QC * CHUNK), vd = tc::desc_at(v_desc, vs * L::VC * CHUNK);
                    const uint32_t qk = (k.needs(0, j) ? 1u : 0u) | (k.needs(1, j) ? 2u : 0u);
#pragma unroll 1
                    for (int t = 0; t < 2; ++t) {
                        const bool p = (pv >> t) & 1, q = (qk >> t) & 1;
                        if (!p && !q) continue;
                        const int e = t ? k.e[1] : k.e[0], jf = (t ? k.c[1] : k.c[0]) > 0 ? 0 : (t ? k.f[1] : k.f[0]);
                        const uint32_t want = (p ? 3u : 0u) | (q ? 4u : 0u);
                        const uint32_t got = tc::mbar_test3(&bar.p_full[t], (np >> t) & 1, &bar.v_full[vs], vph,
                                                            &bar.k_full[ks], kph);
                        if (!__all_sync(0xffffffffu, (got & want) == want)) {
                            if (p && (!uwait(&bar.v_full[vs], vph) || !uwait(&bar.p_full[t], (np >> t) & 1))) {
                                ok = false;
                                break;
                            }
                            if (q && !uwait(&bar.k_full[ks], kph)) { ok = false; break; }
                        }
                        if (q && j == jf && !uwait(&bar.q_full[t], (nq >> t) & 1)) { ok = false; break; }
                        tc::fence_after_sync();
                        const uint32_t tS = tmem + t * 128, tO = tmem + 256 + t * DV;
                        const uint64_t qd = tc::desc_at(q_desc, t * L::QC * CHUNK);
                        if (tc::elect_one()) {
                            if (p) {
                                uint32_t acc = j - 1 != jf;
#pragma unroll 1
                                for (int kk = 0; kk * 16 < wp; kk += 2) {       // (widths are multiples of 32)
                                    tc::mma_ts(tO, tS + kk * 8, tc::desc_at(vd, kk * 2048), idesc_pv, acc);
                                    tc::mma_ts(tO, tS + kk * 8 + 8, tc::desc_at(vd, kk * 2048 + 2048), idesc_pv, 1);
                                    acc = 1;
                                }
                                if (t == 1 || !(pv & 2)) tc::mma_commit(&bar.v_empty[vs]);
                                if (j == e) tc::mma_commit(&bar.o_full[t]);
                            }
                            if (q) {
#pragma unroll 1
                                for (int c = 0; c < L::QC; ++c)
#pragma unroll
                                    for (int kk = 0; kk < 4; ++kk)
                                        tc::mma_ss(tS, tc::desc_at(qd, c * CHUNK + kk * 32), tc::desc_at(kd, c * CHUNK + kk * 32),
                                                   idesc_w, kk > 0 || c > 0);
                                tc::mma_commit(&bar.s_full[t]);
                                if (t == 1 || !(qk & 2)) tc::mma_commit(&bar.k_empty[ks]);
                                if (j == e - 1) tc::mma_commit(&bar.q_empty[t]);
                            }
                        }
                        __syncwarp();
                        if (p) np ^= 1u << t;
                        if (j == e - 1) nq ^= 1u << t;
                    }
                    if (j > 0 && ++vs == L::VS) vs = 0, vph ^= 1;
                    if (j < k.n && ++ks == L::KS) ks = 0, kph ^= 1;
                    pv = qk;
                    wp = wj;
                }
            }
            if (!ok && lane == 0) give_up();
            if (tc::elect_one()) tc::mma_commit(&bar.drain);    // every MMA has completed before TMEM is freed
            tc::mbar_wait_bounded(&bar.drain, 0, WAIT_NS);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 200;" ::: "memory");
        // ---------------------------------------------------- softmax and epilogue of one query tile
        const int t = (warp - 4) >> 2;
        const int r = (warp & 3) * 32 + lane;                   // row of the tile
        const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + t * 128 + lane_off, tO = tmem + 256 + t * DV + lane_off;
        const int tt = r / s.G, g = r - tt * s.G;
        TileRows tile_rows;
        tile_rows.init(r, s.G);
        uint32_t ns = 0, no = 0;
        bool ok = true;
        auto warp_wait = [&](uint64_t* b, uint32_t parity) { return __all_sync(0xffffffffu, wait(b, parity)); };
        const float pow2_log2 = __uint_as_float(__float_as_uint(a.scale_log2) & 0x7F800000u);
        for (int w = blockIdx.x; ok && w < a.n_work; w += gridDim.x) {
            const Work k = decode_work(a, w);
            if (t >= k.nt) continue;
            const int pos = (t ? k.pf[1] : k.pf[0]) + tt;
            const bool row_ok = tt < a.tok && pos < s.q0 + s.Tq;
            const int kc = t ? k.c[1] : k.c[0], kf = t ? k.f[1] : k.f[0], ke = t ? k.e[1] : k.e[0];
            float m = -INFINITY, l = 0.f, c2 = a.scale_log2;        // m = maximum c2 (LARGE_REF)
            for (int j = kc > 0 ? 0 : kf, first = 1; j < ke; first = 0, j = j + 1 < kc ? j + 1 : max(j + 1, kf)) {
                const int u0 = k.key(j), nc = k.width(j) >> 5;
                // visible offsets: [lo, hi] and, behind the window, [0, sk)
                int lo, hi, sk;
                if (j < k.nst) {
                    lo = 0;
                    hi = k.sl - 1 - u0;
                    sk = 0;
                } else {
                    lo = pos - s.win + 1 - u0;
                    hi = pos - u0;
                    sk = min(s.ns - u0, hi + 1);
                }
                const bool full = __all_sync(0xffffffffu, (hi >= BN - 1 && (lo <= 0 || sk >= BN)) || !row_ok);
                if (!warp_wait(&bar.s_full[t], ns & 1)) { ok = false; break; }
                ++ns;
                tc::fence_after_sync();
                // all scores of the row in registers; the maximum of the first half is taken
                // while the second half is on its way
                uint32_t x[128];
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
                auto load = [&](auto masked_tag) {
                    constexpr bool MASKED = decltype(masked_tag)::value;
                    tc::tmem_ld32(tS, x);
                    if (!MASKED || nc > 1) tc::tmem_ld32(tS + 32, x + 32);
                    tc::tmem_wait_ld32(x);
                    tc::tmem_wait_ld32(x + 32);
                    if (!MASKED || nc > 2) tc::tmem_ld32(tS + 64, x + 64);
                    if (!MASKED || nc > 3) tc::tmem_ld32(tS + 96, x + 96);
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (MASKED && c >= nc) break;
                        if (c == 2) {
                            tc::tmem_wait_ld32(x + 64);
                            tc::tmem_wait_ld32(x + 96);
                        }
                        if (MASKED) {
                            const uint32_t bits = range_bits(lo, hi, c) | range_bits(0, sk - 1, c);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((bits >> i) & 1u)) x[32 * c + i] = 0xFF800000u;
                        }
#pragma unroll
                        for (int i = 0; i < 32; i += 2)
                            mx[(i >> 1) & 3] = tc::max3(mx[(i >> 1) & 3], __uint_as_float(x[32 * c + i]),
                                                        __uint_as_float(x[32 * c + i + 1]));
                    }
                };
                if (full) load(std::false_type{});
                else load(std::true_type{});
                // scale > 0, so the scaled maximum is the maximum of the scaled scores
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                float mt = __fmul_rn(top, c2);                  // (not fused with a difference: the weights' reference)
                float alpha = 1.f;                              // for what was summed under the reference before
                if (mt > m + 8.f || m == -INFINITY) {           // (-inf > -inf is false: m stays)
                    c2 = fabsf(top * a.scale_log2) < LARGE_REF ? a.scale_log2 : pow2_log2;
                    mt = __fmul_rn(top, c2);
                    if (m != -INFINITY) alpha = tc::ex2(m - mt);
                    m = mt;
                }
                const uint64_t sc2 = tc::f2_pack(c2, c2);
                const float neg = m == -INFINITY ? 0.f : -m;
                const uint64_t neg2 = tc::f2_pack(neg, neg);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (c >= nc) break;         // (also keeps the chunks' code apart: fewer values live at once)
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float y0, y1;
                        tc::f2_unpack(tc::f2_fma(tc::f2_pack(__uint_as_float(x[32 * c + i]),
                                                             __uint_as_float(x[32 * c + i + 1])), sc2, neg2), y0, y1);
                        const float p0 = tc::ex2(y0), p1 = tc::ex2(y1);
                        sum[(i >> 1) & 1] = tc::f2_add(sum[(i >> 1) & 1], tc::f2_pack(p0, p1));
                        x[16 * c + (i >> 1)] = tc::pack_bf16x2(p0, p1);     // in place: 16 c + i / 2 <= 32 c + i
                    }
                    tc::tmem_st16(tS + 16 * c, x + 16 * c);
                }
                float s0, s1;
                tc::f2_unpack(tc::f2_add(sum[0], sum[1]), s0, s1);
                const float psum = s0 + s1;
                if (__any_sync(0xffffffffu, alpha != 1.f)) {    // O holds the tiles before this one
#pragma unroll 1
                    for (int c = 0; c < DV; c += 32) {
                        uint32_t o[32];
                        tc::tmem_ld32(tO + c, o);
                        tc::tmem_wait_ld32(o);
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tc::tmem_st32(tO + c, o);
                    }
                    l *= alpha;
                }
                l += psum;
                tc::tmem_wait_st();
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&bar.p_full[t]);
            }
            if (!ok) break;
            if (!warp_wait(&bar.o_full[t], no & 1)) { ok = false; break; }
            ++no;
            tc::fence_after_sync();
            const int i0 = (k.tt0 + t) * a.tok;
            const OutRows rows = tile_rows.at(((long long)k.b * s.Tq + i0) * s.Hq + k.kvh * s.G, min(a.tok, s.Tq - i0), s.Hq);
            const float inv = 1.f / l;
#pragma unroll 1
            for (int c = 0; c < DV; c += 32) {
                uint32_t o[32];
                uint4 u[4];
                tc::tmem_ld32(tO + c, o);
                tc::tmem_wait_ld32(o);
                pack32(o, inv, u);
                store_bf16x32(u, a.out, rows, DV, c, lane);
            }
            if (row_ok && a.lse)
                a.lse[((size_t)k.b * s.Tq + (pos - s.q0)) * s.Hq + k.kvh * s.G + g] =
                    c2 == a.scale_log2 ? (m + log2f(l)) * 0.6931471805599453f : fmaf(m, s.scale / c2, logf(l));
            tc::fence_before_sync();
        }
        if (!ok) give_up();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

template <int DQK, int DV>
cudaError_t launch_impl(const WinShape& s, const __nv_bfloat16* q, const __nv_bfloat16* k, const __nv_bfloat16* v,
                        __nv_bfloat16* out, float* lse, cudaStream_t st) {
    Args a;
    a.s = s;
    a.out = out;
    a.lse = lse;
    a.tok = BM / s.G;
    a.n_tt = (s.Tq + a.tok - 1) / a.tok;
    a.scale_log2 = s.scale * 1.4426950408889634f;
    int dev, nsm;
    cudaError_t e = sm_count(&nsm, &dev);
    if (e != cudaSuccess) return e;
    const long long planes = (long long)s.B * s.Hkv;
    // pairs of query tiles unless that would leave SMs without work: a pair's chains overlap
    // (singles 280 us against 175, 710 against 420), 32 query tiles finish earlier on 32 SMs
    // (1000 tokens, 4 heads on 1, d 64: 8.1 us against 9.6)
    a.nt = (a.n_tt + 1) / 2 * planes >= nsm ? 2 : 1;
    a.n_work = (int)((a.n_tt + a.nt - 1) / a.nt * planes);
    CUtensorMap mq, mk, mv;
    if (!tmap::heads_map(&mq, q, DQK, s.Hq, s.Tq, s.B, s.G, a.tok) ||
        !tmap::rows_map(&mk, k, DQK, s.Tk, s.B * s.Hkv, BN) || !tmap::rows_map(&mv, v, DV, s.Tk, s.B * s.Hkv, BN))
        return cudaErrorInvalidValue;
    const int smem = Smem<DQK, DV>::ALLOC;
    static std::atomic<bool> allowed[MAX_DEVICES];
    e = allow_smem(reinterpret_cast<const void*>(window_fwd_tc_kernel<DQK, DV>), smem, dev, allowed);
    if (e != cudaSuccess) return e;
    window_fwd_tc_kernel<DQK, DV><<<std::min(a.n_work, nsm), THREADS, smem, st>>>(mq, mk, mv, a);
    return cudaGetLastError();
}

}  // namespace

// What fits TMEM (512 columns) and shared memory, and a token's heads in half a query tile.
// Everything else runs on FFMA, 160 times slower where both serve (16384 tokens, 64 heads
// on 4, 192/128, window 512 + 64: 68.4 ms against 0.42).
bool window_tc_supported(const WinShape& s) {
    return s.dqk <= 192 && s.dv <= 128 && s.G <= 64;
}

cudaError_t launch_window_fwd_tc(const WinShape& s, const __nv_bfloat16* q, const __nv_bfloat16* k,
                                 const __nv_bfloat16* v, __nv_bfloat16* out, float* lse, cudaStream_t st) {
#define NSA_WIN_CASE(A, B) \
    if (s.dqk == A && s.dv == B) return launch_impl<A, B>(s, q, k, v, out, lse, st);
    NSA_WIN_CASE(64, 64)
    NSA_WIN_CASE(64, 128)
    NSA_WIN_CASE(128, 64)
    NSA_WIN_CASE(128, 128)
    NSA_WIN_CASE(192, 64)
    NSA_WIN_CASE(192, 128)
#undef NSA_WIN_CASE
    return cudaErrorInvalidValue;
}

cudaError_t set_win_fwd_wait_limit(uint64_t limit_ns) {
    const uint64_t v = limit_ns ? limit_ns : WAIT_NS;
    return cudaMemcpyToSymbol(c_win_fwd_wait_ns, &v, sizeof(v));
}

int read_and_clear_win_fwd_status() {
    int v = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&v, g_win_fwd_status, sizeof(int)) != cudaSuccess) return -1;
    cudaMemcpyToSymbol(g_win_fwd_status, &zero, sizeof(int));
    return v;
}

}  // namespace nsa
