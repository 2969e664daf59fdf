// Attention of the newest tokens over a paged key/value cache, split over the
// cache's length and joined.
//
// Transcript #94 (bidclub.ai) §6: decoding is memory-bound and costs the KV
// bytes it reads.  Every visible key and value row is read once for all the
// heads of its group: a (sequence, KV head) has rows = seqlen_q * G query rows,
// cut into tiles of 16 (the M of one mma.sync; a unit is one such tile), and
// its visible keys into tiles of 16 (a tile lies inside one page, pages being
// multiples of 16).  The tiles of all units, in order, are dealt in equal
// contiguous shares to the workers, one worker per warp of a grid that fills
// the GPU once; the shares follow the lengths found on the device.  A worker
// walks its share with its own cp.async rings (3 key and 2 value tiles), never
// waiting for another warp:
//   S = Q K^T (16 x 16), p = exp2(S - m) under the running row maximum m,
//   O = O exp2(m_old - m) + P V, l += sum p.
// A unit inside one share is finished there; a unit cut by shares leaves one
// (O / l, m, l) per share, joined by paged_join_kernel under the largest m, M:
//   w_i = 2^(m_i - M) l_i,  o = sum_i w_i o_i / sum_i w_i,  lse = M + log2 sum_i w_i.
// (m and l apart: in m + log2 l a large m would swallow the sum.)
// mma.sync rather than tcgen05: with the group's 1-16 heads as M the products
// need a few percent of the tensor cores at full HBM rate, and a warp keeps
// its whole state in registers, without a CTA-wide hand-over per tile.
// Bound by HBM: 64 sequences of up to 32768 keys, 64 heads on 4, 192/128:
// 394-431 us, 6.1-6.6 TB/s; 48 x 4 tokens, 32 heads on 8, d 128, window
// 4096 + 16, pages of 16: 136 us, 5.6 TB/s, the join 6 of them.  One sequence of
// 1000 keys is two launches of dependent loads: 10.8 us (7.8 without the join).
#include <math.h>

#include <algorithm>

#include "launch.cuh"
#include "paged.cuh"
#include "tc.cuh"

namespace nsa {
namespace {

constexpr int TILE = 16;                // keys per tile
constexpr int ROWS = 16;                // query rows per unit
// Ring stages of a worker: at 192/128 they fill shared memory with 8 workers, 208 KB in flight
// per SM, four times what HBM's latency needs.
constexpr int KST = 3, VST = 2;
// Least share of a worker: 1000 keys, 16 heads, d 128 take 11.1 us at 1, 10.8 at 2, 12.9 at 4
// (more to join against a longer walk).
constexpr int MIN_TILES = 2;

template <int DQK, int DV>
struct Dim {
    static constexpr int K_STAGE = TILE * DQK * 2, V_STAGE = TILE * DV * 2;
    static constexpr int RING = KST * K_STAGE + VST * V_STAGE;
    static constexpr int WARPS = 8 * RING <= 220 * 1024 ? 8 : 4;
    static constexpr int SMEM = WARPS * RING;
};

// Tiles of one sequence: i < nA are the sinks' (keys 16 i ..), the others run
// from b0 on to the newest key.
struct SeqTiles {
    int nA, b0, n, len, wlo;
};

__device__ __forceinline__ SeqTiles seq_tiles(const PagedShape& s, int len) {
    SeqTiles t;
    t.len = len;
    const int t_first = max(len - s.Tq, 0);
    t.wlo = s.win ? max(0, t_first - s.win + 1) : 0;      // lowest key in any query's window
    t.b0 = t.wlo / TILE * TILE;
    t.nA = min((min(s.ns, t.wlo) + TILE - 1) / TILE, t.b0 / TILE);
    t.n = len > 0 ? t.nA + (len - t.b0 + TILE - 1) / TILE : 0;
    return t;
}

__device__ __forceinline__ int tile_key(const SeqTiles& t, int i) {
    return i < t.nA ? i * TILE : t.b0 + (i - t.nA) * TILE;
}

struct PagedArgs {
    PagedShape s;
    const __nv_bfloat16* q;
    const __nv_bfloat16* kp;
    const __nv_bfloat16* vp;
    const int32_t* table;
    const int32_t* lens;
    __nv_bfloat16* out;
    float* lse;
    float* part_o;          // [2 * workers][ROWS][dv]
    float2* part_ml;        // [2 * workers][ROWS] running maximum and sum
    int RT;                 // row tiles per (sequence, KV head)
    float scale_log2;
};

// a / b for a >= 0, b > 0, by the short 32-bit division where both fit.
__device__ __forceinline__ long long quotient(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// Tiles per worker when `total` tiles are dealt to `workers`.
__device__ __forceinline__ long long share_of(long long total, int workers) {
    const long long x = quotient(total + workers - 1, workers);
    return x < MIN_TILES ? MIN_TILES : x;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0)
                 : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk c of row r in a tile of rows of D bf16: chunks
// are swizzled by the row, so that eight rows' chunks at one column lie in
// eight different bank groups (ldmatrix without conflicts).
template <int D>
__device__ __forceinline__ uint32_t tile_off(int r, int c) {
    return (uint32_t)(r * (D * 2) + ((c ^ (r & 7)) << 4));
}

// The 16 rows of a tile, contiguous at src, into a ring stage; rows outside
// `rows` (a bit mask) become zeros.
template <int D>
__device__ __forceinline__ void load_tile(uint32_t dst, const __nv_bfloat16* src, uint32_t rows, int lane) {
    constexpr int C = D / 8;
#pragma unroll
    for (int j = 0; j < TILE * C / 32; ++j) {
        const int e = lane + 32 * j, r = e / C, c = e % C;
        const bool ok = (rows >> r) & 1u;
        cp_async16(dst + tile_off<D>(r, c), ok ? src + (size_t)e * 8 : src, ok);
    }
}

template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int DQK, int DV>
__global__ void __launch_bounds__(Dim<DQK, DV>::WARPS * 32, 1) paged_attn_kernel(const PagedArgs a) {
    using L = Dim<DQK, DV>;
    constexpr int THREADS = L::WARPS * 32;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long pre[THREADS + 1];
    __shared__ long long wsum[L::WARPS];
    const PagedShape& s = a.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_launch();

    // first tile of every sequence: thread i sums the chunk of sequences
    // [i C, (i + 1) C), the block scans the sums
    const int per_seq = s.Hkv * a.RT;
    const int C = (s.B + THREADS - 1) / THREADS;
    const int c0 = threadIdx.x * C, c1 = min(s.B, c0 + C);
    long long mine = 0;
    for (int b = c0; b < c1; ++b) mine += (long long)seq_tiles(s, paged_len(s, a.lens, b)).n * per_seq;
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    for (int w = 0; w < warp; ++w) inc += wsum[w];
    pre[threadIdx.x] = inc - mine;
    if (threadIdx.x == THREADS - 1) pre[THREADS] = inc;
    __syncthreads();
    const long long total = pre[THREADS];
    const int workers = gridDim.x * L::WARPS;
    const int me = warp * gridDim.x + blockIdx.x;  // neighbours on different SMs
    const long long per = share_of(total, workers);
    long long g = me * per;
    const long long g1 = min(total, g + per);
    if (g >= g1) return;
    int lo = 0, hi = THREADS;                      // chunk that holds tile g
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (pre[mid] <= g) lo = mid;
        else hi = mid;
    }
    int b = lo * C;
    long long base = pre[lo];                      // first tile of sequence b
    SeqTiles sq = seq_tiles(s, paged_len(s, a.lens, b));
    while (g >= base + (long long)sq.n * per_seq) {
        base += (long long)sq.n * per_seq;
        ++b;
        sq = seq_tiles(s, paged_len(s, a.lens, b));
    }

    const uint32_t ring = tc::smem_u32(smem) + warp * L::RING;
    const int qr = lane >> 2, qc = (lane & 3) * 2;  // fragment row and column
    const int nrows = s.Tq * s.G;

    while (g < g1) {
        if (g >= base + (long long)sq.n * per_seq) {    // next sequence with keys
            base += (long long)sq.n * per_seq;
            ++b;
            sq = seq_tiles(s, paged_len(s, a.lens, b));
            continue;
        }
        const int unit = (int)quotient(g - base, sq.n);
        const int i0 = (int)(g - base - (long long)unit * sq.n);
        const int i1 = (int)min((long long)sq.n, i0 + (g1 - g));
        const int h = unit / a.RT, rt = unit % a.RT;
        const int t_first = sq.len - s.Tq;              // position of query 0 (may be below 0)

        // this thread's two rows
        int trow[2];
        size_t orow[2];
        bool rok[2];
        uint32_t qf[DQK / 16][4];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = rt * ROWS + qr + 8 * e;
            rok[e] = r < nrows;
            const int qi = min(r, nrows - 1) / s.G, gh = min(r, nrows - 1) % s.G;
            trow[e] = t_first + qi;
            orow[e] = ((size_t)b * s.Tq + qi) * s.Hq + h * s.G + gh;
            const uint32_t* src = reinterpret_cast<const uint32_t*>(a.q + orow[e] * DQK + qc);
#pragma unroll
            for (int kk = 0; kk < DQK / 16; ++kk) {
                qf[kk][e] = rok[e] ? src[kk * 8] : 0u;
                qf[kk][2 + e] = rok[e] ? src[kk * 8 + 4] : 0u;
            }
        }

        // page ids, 32 tiles at a time: lane l holds that of tile batch + l
        const int32_t* trow_pages = a.table + (size_t)b * s.cols;
        auto page_batch = [&](int first) {
            const int i = first + lane;
            return i < i1 ? trow_pages[tile_key(sq, i) >> s.logP] : -1;
        };
        int pg = page_batch(i0), pg_next = page_batch(i0 + 32);
        int k_page = -1;                                // page of the newest key tile
        auto rows_of = [&](int u0, int page) -> uint32_t {
            if ((unsigned)page >= (unsigned)s.n_pages) return 0u;
            if (u0 + TILE <= sq.len && (u0 >= sq.wlo || u0 + TILE <= s.ns)) return 0xFFFFu;
            uint32_t m = 0;
#pragma unroll
            for (int r = 0; r < TILE; ++r) {
                const int u = u0 + r;
                if (u < sq.len && (u >= sq.wlo || u < s.ns)) m |= 1u << r;
            }
            return m;
        };
        auto issue_k = [&](int i) {
            if (i < i1) {
                const int o = i - i0;
                if (o > 0 && (o & 31) == 0) {
                    pg = pg_next;
                    pg_next = page_batch(i + 32);
                }
                k_page = __shfl_sync(0xffffffffu, pg, o & 31);
                const int u0 = tile_key(sq, i);
                const uint32_t rows = rows_of(u0, k_page);
                const int page = rows ? k_page : 0;
                load_tile<DQK>(ring + (o % KST) * L::K_STAGE,
                               a.kp + (((size_t)page * s.Hkv + h) * s.P + (u0 & (s.P - 1))) * DQK, rows, lane);
            }
            tc::cp_async_commit();
        };
        auto issue_v = [&](int i, int pid) {
            if (i < i1) {
                const int o = i - i0;
                const int u0 = tile_key(sq, i);
                const uint32_t rows = rows_of(u0, pid);
                const int page = rows ? pid : 0;
                load_tile<DV>(ring + KST * L::K_STAGE + (o % VST) * L::V_STAGE,
                              a.vp + (((size_t)page * s.Hkv + h) * s.P + (u0 & (s.P - 1))) * DV, rows, lane);
            }
            tc::cp_async_commit();
        };
        issue_k(i0);
        issue_v(i0, k_page);
        issue_k(i0 + 1);
        issue_v(i0 + 1, k_page);
        issue_k(i0 + 2);

        float o[DV / 8][4];
#pragma unroll
        for (int n = 0; n < DV / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        for (int i = i0; i < i1; ++i) {
            cp_wait<4>();                               // key tile i has landed
            __syncwarp();
            const uint32_t ks = ring + ((i - i0) % KST) * L::K_STAGE;
            float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int kk = 0; kk < DQK / 16; ++kk) {
                uint32_t f[4];
                ldsm4(ks + tile_off<DQK>((lane & 7) + ((lane >> 4) << 3), 2 * kk + ((lane >> 3) & 1)), f);
                mma_bf16(sc[0], qf[kk], f[0], f[1]);
                mma_bf16(sc[1], qf[kk], f[2], f[3]);
            }
            const int u0 = tile_key(sq, i);
            const bool all = u0 + TILE - 1 <= t_first &&
                             (s.win == 0 || u0 > t_first + s.Tq - 1 - s.win || u0 + TILE <= s.ns);
            uint32_t pf[4];
            float alpha[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[j] = __fmul_rn(sc[j >> 1][2 * e + (j & 1)], a.scale_log2);    // (the maximum's weight is 1)
                    if (!all) {
                        const int u = u0 + (j >> 1) * 8 + qc + (j & 1);
                        const bool vis = u <= trow[e] && (s.win == 0 || u > trow[e] - s.win || u < s.ns);
                        if (!vis) x[j] = -INFINITY;
                    }
                }
                float mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                mx = fmaxf(mx, m[e]);
                const float ref = mx == -INFINITY ? 0.f : mx;
                alpha[e] = tc::ex2(m[e] - ref);
                m[e] = mx;
                float p[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) p[j] = tc::ex2(x[j] - ref);
                l[e] = l[e] * alpha[e] + ((p[0] + p[1]) + (p[2] + p[3]));
                pf[e] = tc::pack_bf16x2(p[0], p[1]);        // bf16 weights: half a step, 2^-8 relative
                pf[2 + e] = tc::pack_bf16x2(p[2], p[3]);    // at most, independent per key
            }
            if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                for (int n = 0; n < DV / 8; ++n) {
                    o[n][0] *= alpha[0];
                    o[n][1] *= alpha[0];
                    o[n][2] *= alpha[1];
                    o[n][3] *= alpha[1];
                }
            }
            __syncwarp();                               // every lane has read key tile i
            const int vp_next = k_page;                 // page of tile i + 2
            issue_k(i + KST);
            cp_wait<3>();                               // value tile i has landed
            __syncwarp();
            const uint32_t vs = ring + KST * L::K_STAGE + ((i - i0) % VST) * L::V_STAGE;
#pragma unroll
            for (int n = 0; n < DV / 16; ++n) {
                uint32_t f[4];
                ldsm4_t(vs + tile_off<DV>((lane & 7) + (((lane >> 3) & 1) << 3), 2 * n + (lane >> 4)), f);
                mma_bf16(o[2 * n], pf, f[0], f[1]);
                mma_bf16(o[2 * n + 1], pf, f[2], f[3]);
            }
            __syncwarp();                               // every lane has read value tile i
            issue_v(i + VST, vp_next);
        }
        cp_wait<0>();
        __syncwarp();

#pragma unroll
        for (int e = 0; e < 2; ++e) {
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
            l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
        }
        const bool whole = i0 == 0 && i1 == sq.n;
        const int slot = 2 * me + (i0 == 0 ? 1 : 0);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (!rok[e]) continue;
            const float inv = l[e] == 0.f ? 0.f : 1.f / l[e];
            if (whole) {
                uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow[e] * DV + qc);
#pragma unroll
                for (int n = 0; n < DV / 8; ++n)
                    dst[n * 4] = tc::pack_bf16x2(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
                if (a.lse && (lane & 3) == 0)
                    a.lse[orow[e]] = l[e] == 0.f ? -INFINITY : (m[e] + log2f(l[e])) * 0.6931471805599453f;
            } else {
                const size_t pr = (size_t)slot * ROWS + qr + 8 * e;
                float2* dst = reinterpret_cast<float2*>(a.part_o + pr * DV + qc);
#pragma unroll
                for (int n = 0; n < DV / 8; ++n) dst[n * 4] = make_float2(o[n][2 * e] * inv, o[n][2 * e + 1] * inv);
                if ((lane & 3) == 0) a.part_ml[pr] = make_float2(m[e], l[e]);
            }
        }
        g += i1 - i0;
    }
}

// Joins the shares of a unit's rows; units without keys get 0 and -inf.  A warp
// has a row (blockIdx.y: four rows), or, with fewer than four rows (one query
// head per KV head), the four warps have one row's shares w, w + 4, ...: such
// units are few and their shares many (both kernels, one sequence of 1000 keys,
// 16 heads: 10.8 us, with a warp per row 12.2; 48 x 4 tokens with 4 heads a KV
// head: 148 us, with a warp per row 135).
constexpr int JOIN_WARPS = 4;

template <int DV, bool SPLIT>
__global__ void __launch_bounds__(JOIN_WARPS * 32) paged_join_kernel(const PagedArgs a, int workers) {
    constexpr int NC = DV / 64;                     // column pairs per lane
    __shared__ float2 acc_s[SPLIT ? JOIN_WARPS : 1][SPLIT ? DV / 2 : 1], ml_s[JOIN_WARPS];
    __shared__ long long pre_s[JOIN_WARPS], tot_s[JOIN_WARPS];
    const PagedShape& s = a.s;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per_seq = s.Hkv * a.RT;
    const int b = blockIdx.x / per_seq, unit = blockIdx.x % per_seq;
    const int h = unit / a.RT, rt = unit % a.RT;
    const int ru = SPLIT ? blockIdx.y : blockIdx.y * JOIN_WARPS + warp;     // row of the unit
    const int r = rt * ROWS + ru;
    // which shares the unit was cut into: from the lengths, while the shares are still computed
    long long p0 = 0, total = 0;
    for (int i = threadIdx.x; i < s.B; i += JOIN_WARPS * 32) {
        const long long t = (long long)seq_tiles(s, paged_len(s, a.lens, i)).n * per_seq;
        total += t;
        if (i < b) p0 += t;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        p0 += __shfl_xor_sync(0xffffffffu, p0, o);
        total += __shfl_xor_sync(0xffffffffu, total, o);
    }
    if (lane == 0) {
        pre_s[warp] = p0;
        tot_s[warp] = total;
    }
    __syncthreads();
    p0 = total = 0;
#pragma unroll
    for (int w = 0; w < JOIN_WARPS; ++w) {
        p0 += pre_s[w];
        total += tot_s[w];
    }
    const int n = seq_tiles(s, paged_len(s, a.lens, b)).n;
    const long long per = share_of(total, workers);
    const long long first = p0 + (long long)unit * n, last = first + n - 1;
    const int w0 = (int)quotient(first, per), w1 = n > 0 ? (int)quotient(last, per) : w0 - 1;
    pdl_wait();
    if (r >= s.Tq * s.G) return;                    // (whole CTAs when SPLIT)
    if (n > 0 && w0 == w1) return;                  // finished by its worker
    const size_t orow = ((size_t)b * s.Tq + r / s.G) * s.Hq + h * s.G + r % s.G;
    auto part_row = [&](int w) {                    // only w0 starts the unit
        return (size_t)(2 * w + (w == w0 ? 1 : 0)) * ROWS + ru;
    };
    // lane's columns of the shares so far: acc and sum under the running maximum mx
    float mx = -INFINITY, sum = 0.f;
    float2 acc[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c) acc[c] = make_float2(0.f, 0.f);
    constexpr int U = 8, STEP = SPLIT ? JOIN_WARPS : 1;
    for (int w = w0 + (SPLIT ? warp : 0); w <= w1; w += U * STEP) {
        float2 ml[U], x[U][NC];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const bool ok = w + u * STEP <= w1;
            const size_t pr = part_row(ok ? w + u * STEP : w);
            ml[u] = ok ? a.part_ml[pr] : make_float2(-INFINITY, 0.f);
#pragma unroll
            for (int c = 0; c < NC; ++c)
                x[u][c] = ok ? reinterpret_cast<const float2*>(a.part_o + pr * DV)[c * 32 + lane] : make_float2(0.f, 0.f);
        }
        float top = mx;
#pragma unroll
        for (int u = 0; u < U; ++u) top = fmaxf(top, ml[u].x);
        const float ref = top == -INFINITY ? 0.f : top, old = tc::ex2(mx - ref);
        mx = top;
        sum *= old;
#pragma unroll
        for (int c = 0; c < NC; ++c) acc[c] = make_float2(acc[c].x * old, acc[c].y * old);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const float wt = tc::ex2(ml[u].x - ref) * ml[u].y;
            sum += wt;
#pragma unroll
            for (int c = 0; c < NC; ++c)
                acc[c] = make_float2(fmaf(wt, x[u][c].x, acc[c].x), fmaf(wt, x[u][c].y, acc[c].y));
        }
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(a.out + orow * DV);
    if (SPLIT) {
        if (lane == 0) ml_s[warp] = make_float2(mx, sum);
#pragma unroll
        for (int c = 0; c < NC; ++c) acc_s[warp][c * 32 + lane] = acc[c];
        __syncthreads();
        float wt[JOIN_WARPS];
        mx = -INFINITY;
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < JOIN_WARPS; ++w) mx = fmaxf(mx, ml_s[w].x);
#pragma unroll
        for (int w = 0; w < JOIN_WARPS; ++w) {
            wt[w] = mx == -INFINITY ? 0.f : tc::ex2(ml_s[w].x - mx);
            sum = fmaf(wt[w], ml_s[w].y, sum);
        }
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        for (int c = threadIdx.x; c < DV / 2; c += JOIN_WARPS * 32) {
            float x = 0.f, y = 0.f;
#pragma unroll
            for (int w = 0; w < JOIN_WARPS; ++w) {
                x = fmaf(wt[w], acc_s[w][c].x, x);
                y = fmaf(wt[w], acc_s[w][c].y, y);
            }
            dst[c] = tc::pack_bf16x2(x * inv, y * inv);
        }
    } else {
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
        for (int c = 0; c < NC; ++c) dst[c * 32 + lane] = tc::pack_bf16x2(acc[c].x * inv, acc[c].y * inv);
    }
    if (a.lse && lane == 0 && (!SPLIT || warp == 0))
        a.lse[orow] = sum == 0.f ? -INFINITY : (mx + log2f(sum)) * 0.6931471805599453f;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

constexpr int MAX_SMS = 160;                        // workers the workspace holds partials for
constexpr int MAX_WORKERS = MAX_SMS * 8;

template <int DQK, int DV>
cudaError_t launch_impl(PagedArgs a, int n_units, int rows, cudaStream_t st) {
    using L = Dim<DQK, DV>;
    int dev, nsm;
    cudaError_t e = sm_count(&nsm, &dev);
    if (e != cudaSuccess) return e;
    static std::atomic<bool> allowed[MAX_DEVICES];
    e = allow_smem(reinterpret_cast<const void*>(paged_attn_kernel<DQK, DV>), L::SMEM, dev, allowed);
    if (e != cudaSuccess) return e;
    const int grid = std::min(nsm, MAX_SMS);
    paged_attn_kernel<DQK, DV><<<grid, L::WARPS * 32, L::SMEM, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const bool split = rows < JOIN_WARPS;
    const dim3 join_grid(n_units, split ? rows : (std::min(rows, ROWS) + JOIN_WARPS - 1) / JOIN_WARPS);
    return launch_dependent(split ? paged_join_kernel<DV, true> : paged_join_kernel<DV, false>, join_grid,
                            JOIN_WARPS * 32, 0, st, a, grid * L::WARPS);
}

}  // namespace

size_t paged_attn_ws_bytes(const PagedShape& s) {
    return up256((size_t)2 * MAX_WORKERS * ROWS * s.dv * 4) + (size_t)2 * MAX_WORKERS * ROWS * sizeof(float2);
}

cudaError_t launch_paged_attn(const PagedShape& s, const __nv_bfloat16* q, const __nv_bfloat16* kp,
                              const __nv_bfloat16* vp, const int32_t* table, const int32_t* lens,
                              __nv_bfloat16* out, float* lse, uint8_t* ws, cudaStream_t st) {
    PagedArgs a;
    a.s = s;
    a.q = q;
    a.kp = kp;
    a.vp = vp;
    a.table = table;
    a.lens = lens;
    a.out = out;
    a.lse = lse;
    a.part_o = reinterpret_cast<float*>(ws);
    ws += up256((size_t)2 * MAX_WORKERS * ROWS * s.dv * 4);
    a.part_ml = reinterpret_cast<float2*>(ws);
    const int rows = s.Tq * s.G;
    a.RT = (rows + ROWS - 1) / ROWS;
    a.scale_log2 = s.scale * 1.4426950408889634f;
    const int n_units = s.B * s.Hkv * a.RT;
#define NSA_PAGED_CASE(A, B) \
    if (s.dqk == A && s.dv == B) return launch_impl<A, B>(a, n_units, rows, st);
    NSA_PAGED_CASE(64, 64)
    NSA_PAGED_CASE(64, 128)
    NSA_PAGED_CASE(64, 256)
    NSA_PAGED_CASE(128, 64)
    NSA_PAGED_CASE(128, 128)
    NSA_PAGED_CASE(128, 256)
    NSA_PAGED_CASE(192, 64)
    NSA_PAGED_CASE(192, 128)
    NSA_PAGED_CASE(192, 256)
    NSA_PAGED_CASE(256, 64)
    NSA_PAGED_CASE(256, 128)
    NSA_PAGED_CASE(256, 256)
#undef NSA_PAGED_CASE
    return cudaErrorInvalidValue;
}

}  // namespace nsa
