// The pages of a paged key/value cache: appending (allocation, copy-on-write,
// the rows), forking, shortening and compacting.
//
// Bookkeeping (which pages) runs in one CTA, because every choice depends on
// the ones before it: the lowest free ids in row order.  It is a handful of
// dependent global reads and two block-wide scans, so it costs latency, not
// bandwidth.  The bytes move in a second kernel over the whole GPU, started
// early (programmatic dependent launch) and waiting for the first kernel's
// result; it is bound by HBM for prompts and compaction and by latency for a
// decode step.
// Measured: 16 prompts, 182 MB read and written: 25.5 us (7.1 TB/s) behind a plan
// of 6; compaction of 456 MB: 78 us (5.9 TB/s) behind a plan of 8.
#include <algorithm>

#include "launch.cuh"
#include "paged.cuh"

namespace nsa {
namespace {

constexpr int PLAN_THREADS = 1024;

// Exclusive scan of x over the CTA's 1024 threads; *total receives the sum.
__device__ __forceinline__ int block_scan(int x, int* total, int* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int inc = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    __syncthreads();                               // warp_sums is free again
    if (lane == 31) warp_sums[warp] = inc;
    __syncthreads();
    if (warp == 0) {
        int w = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += up;
        }
        warp_sums[lane] = w;
    }
    __syncthreads();
    *total = warp_sums[31];
    return inc - x + (warp ? warp_sums[warp - 1] : 0);
}

// ------------------------------------------------------------------ append

struct AppendArgs {
    PagedShape s;
    const __nv_bfloat16* k_new;
    const __nv_bfloat16* v_new;
    const int32_t* n_new;
    __nv_bfloat16* kp;
    __nv_bfloat16* vp;
    int32_t* table;
    int32_t* lens;
    int32_t* ref;
    int32_t* short_pages;
    int32_t* free_list;   // [n_pages]
    // [B] {length before, tokens (0: nothing to do), page to copy from or -1, flag}.  A row that keeps
    // a page writes behind its own tokens there.  Where a row that copies the page has more tokens
    // of it, the copy has to come first: then both rows' flag is 1, and the keeper's CTAs do both.
    int4* plan;
};

__device__ __forceinline__ int append_count(const AppendArgs& a, int b) {
    return a.n_new ? max(0, min(a.n_new[b], a.s.Tq)) : a.s.Tq;
}

// Shared memory: tail[B] (the row's shared last page, or -1), begin[B] (rank of
// its first new page; bit 31: it keeps its shared page), used[B] (rows of its last page).
constexpr int APPEND_SMEM_ROW = 9;

__global__ void __launch_bounds__(PLAN_THREADS) append_plan_kernel(const AppendArgs a) {
    extern __shared__ int32_t sh[];
    __shared__ int warp_sums[32];
    __shared__ int over;
    const PagedShape& s = a.s;
    int32_t* tail = sh;
    int32_t* begin = sh + s.B;
    uint8_t* used = reinterpret_cast<uint8_t*>(sh + 2 * s.B);       // below P <= 256
    pdl_launch();
    if (threadIdx.x == 0) over = 0;
    for (int b = threadIdx.x; b < s.B; b += PLAN_THREADS) {
        const int L = paged_len(s, a.lens, b), n = append_count(a, b);
        int page = -1;
        if (n > 0 && (L & (s.P - 1)) != 0) {
            page = a.table[(size_t)b * s.cols + (L >> s.logP)];
            if ((unsigned)page >= (unsigned)s.n_pages || a.ref[page] < 2) page = -1;
        }
        tail[b] = page;
        used[b] = (uint8_t)(L & (s.P - 1));
    }
    __syncthreads();
    // pages that each row takes; rows in order, PLAN_THREADS at a time
    int need = 0;
    for (int b0 = 0; b0 < s.B; b0 += PLAN_THREADS) {
        const int b = b0 + threadIdx.x;
        int want = 0;
        if (b < s.B) {
            const int L = paged_len(s, a.lens, b), n = append_count(a, b);
            const int have = (L + s.P - 1) >> s.logP;
            const long long then = ((long long)L + n + s.P - 1) >> s.logP;
            if (then > s.cols) over = 1;
            want = (int)(then - have);
            if (tail[b] >= 0) {
                // as if row by row: the rows before this one that append to the same
                // page have each taken a copy
                int earlier = 0;
                for (int e = 0; e < b; ++e) earlier += tail[e] == tail[b];
                if (a.ref[tail[b]] - earlier > 1) want += 1;
                else want |= 1 << 30;                  // keeps the page
            }
        }
        const bool keeps = (want >> 30) & 1;
        want &= ~(1 << 30);
        int sum;
        const int at = block_scan(want, &sum, warp_sums);
        if (b < s.B) {
            begin[b] = need + at;
            if (keeps) begin[b] |= 1 << 31;
        }
        need += sum;
    }
    __syncthreads();
    // the `need` lowest free ids
    int found = 0;
    for (int p0 = 0; p0 < s.n_pages && found < need; p0 += 4 * PLAN_THREADS) {
        const int p = p0 + 4 * threadIdx.x;
        int r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = p + i < s.n_pages ? a.ref[p + i] : 1;
        int sum;
        int at = found + block_scan((r[0] <= 0) + (r[1] <= 0) + (r[2] <= 0) + (r[3] <= 0), &sum, warp_sums);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (r[i] <= 0) a.free_list[at++] = p + i;
        found += sum;
    }
    __syncthreads();
    const bool ok = !over && found >= need;
    if (threadIdx.x == 0) *a.short_pages = over ? -1 : found >= need ? 0 : need - found;
    // a warp per row: its new entries, its plan
    const int lane = threadIdx.x & 31;
    for (int b = threadIdx.x >> 5; b < s.B; b += PLAN_THREADS / 32) {
        const int L = paged_len(s, a.lens, b), n = ok ? append_count(a, b) : 0;
        const bool copy = n > 0 && tail[b] >= 0 && begin[b] >= 0;
        const int have = (L + s.P - 1) >> s.logP, then = n > 0 ? (L + n + s.P - 1) >> s.logP : 0;
        const int col0 = copy ? have - 1 : have;
        const int32_t* mine = a.free_list + (begin[b] & 0x7FFFFFFF);
        bool first = false;                         // copies have to come before the keeper's tokens
        if (n > 0 && tail[b] >= 0)
            for (int e = lane; e < s.B; e += 32)
                first |= tail[e] == tail[b] && (copy ? begin[e] < 0 && used[e] < used[b]
                                                     : begin[e] >= 0 && used[e] > used[b]);
        first = __any_sync(0xffffffffu, first);
        for (int c = col0 + lane; c < then; c += 32) {
            const int page = mine[c - col0];
            a.table[(size_t)b * s.cols + c] = page;
            a.ref[page] = 1;
        }
        if (lane == 0) {
            if (copy) atomicSub(&a.ref[tail[b]], 1);
            a.plan[b] = make_int4(L, n, copy ? tail[b] : -1, first);
        }
        __syncwarp();
        if (lane == 0 && n > 0) a.lens[b] = L + n;
    }
}

// Rows [r0, r0 + n) of a page's K or V plane: n * d bf16 from src to dst, both 16-byte aligned.
__device__ __forceinline__ void copy_rows(uint4* dst, const uint4* src, int nvec) {
    constexpr int U = 4;
    int e = threadIdx.x;
    for (; e + (U - 1) * (int)blockDim.x < nvec; e += U * blockDim.x) {
        uint4 x[U];
#pragma unroll
        for (int i = 0; i < U; ++i) x[i] = __ldcs(src + e + i * blockDim.x);
#pragma unroll
        for (int i = 0; i < U; ++i) dst[e + i * blockDim.x] = x[i];
    }
    for (; e < nvec; e += blockDim.x) dst[e] = __ldcs(src + e);
}

// One CTA per (page column among those the row touches, KV head, sequence).
__global__ void __launch_bounds__(256) append_write_kernel(const AppendArgs a) {
    const PagedShape& s = a.s;
    const int j = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
    pdl_wait();
    const int4 plan = a.plan[b];
    const int L = plan.x, n = plan.y;
    const int col = (L >> s.logP) + j;
    const int lo = max(L, col << s.logP), hi = min(L + n, (col + 1) << s.logP);     // tokens of this page
    if (hi <= lo) return;
    const int page = a.table[(size_t)b * s.cols + col];
    if ((unsigned)page >= (unsigned)s.n_pages) return;
    const size_t at = ((size_t)page * s.Hkv + h) * s.P;
    // the r rows of page `from` that a row has, into its own page `to`
    auto copy_page = [&](int from, int to, int r) {
        const size_t f = ((size_t)from * s.Hkv + h) * s.P, t = ((size_t)to * s.Hkv + h) * s.P;
        copy_rows(reinterpret_cast<uint4*>(a.kp + t * s.dqk), reinterpret_cast<const uint4*>(a.kp + f * s.dqk),
                  r * (s.dqk / 8));
        copy_rows(reinterpret_cast<uint4*>(a.vp + t * s.dv), reinterpret_cast<const uint4*>(a.vp + f * s.dv),
                  r * (s.dv / 8));
    };
    if (j == 0 && plan.z >= 0 && !plan.w) copy_page(plan.z, page, L & (s.P - 1));
    if (j == 0 && plan.z < 0 && plan.w) {           // the copies of this page that reach behind this row's end
        __shared__ int rows[256], n_rows;
        for (int e0 = 0; e0 < s.B; e0 += 256) {
            __syncthreads();
            if (threadIdx.x == 0) n_rows = 0;
            __syncthreads();
            const int e = e0 + threadIdx.x;
            if (e < s.B && a.plan[e].w && a.plan[e].z == page) rows[atomicAdd(&n_rows, 1)] = e;
            __syncthreads();
            for (int i = 0; i < n_rows; ++i) {
                const int Le = a.plan[rows[i]].x;
                const int to = a.table[(size_t)rows[i] * s.cols + (Le >> s.logP)];
                if ((unsigned)to < (unsigned)s.n_pages) copy_page(page, to, Le & (s.P - 1));
            }
        }
        __syncthreads();                            // read, before the tokens below are written
    }
    const size_t src = ((size_t)b * s.Hkv + h) * s.Tq + (lo - L);
    const size_t dst = at + (lo & (s.P - 1));
    copy_rows(reinterpret_cast<uint4*>(a.kp + dst * s.dqk), reinterpret_cast<const uint4*>(a.k_new + src * s.dqk),
              (hi - lo) * (s.dqk / 8));
    copy_rows(reinterpret_cast<uint4*>(a.vp + dst * s.dv), reinterpret_cast<const uint4*>(a.v_new + src * s.dv),
              (hi - lo) * (s.dv / 8));
}

// ------------------------------------------------------------------ fork, free

// One CTA per entry.  Only the list decides which entries are refused, and the
// lengths read here belong to rows that no other entry writes.
__global__ void __launch_bounds__(128) pages_fork_kernel(PagedShape s, int n, const int32_t* __restrict__ src,
                                                         const int32_t* __restrict__ dst, int32_t* table,
                                                         int32_t* lens, int32_t* ref, int32_t* done) {
    const int i = blockIdx.x;
    const int from = src[i], to = dst[i];
    bool bad = (unsigned)from >= (unsigned)s.B || (unsigned)to >= (unsigned)s.B;
    for (int e = threadIdx.x; e < n; e += blockDim.x) bad |= dst[e] == from || (e < i && dst[e] == to);
    if (!bad) bad = lens[to] != 0;
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) done[i] = !bad;
    if (bad) return;
    const int len = paged_len(s, lens, from), used = (len + s.P - 1) >> s.logP;
    for (int c = threadIdx.x; c < s.cols; c += blockDim.x) {
        const int page = c < used ? table[(size_t)from * s.cols + c] : -1;
        table[(size_t)to * s.cols + c] = page;
        if ((unsigned)page < (unsigned)s.n_pages) atomicAdd(&ref[page], 1);
    }
    if (threadIdx.x == 0) lens[to] = len;
}

__global__ void __launch_bounds__(128) pages_free_kernel(PagedShape s, int n, const int32_t* __restrict__ rows,
                                                         const int32_t* __restrict__ keep, int32_t* table,
                                                         int32_t* lens, int32_t* ref, int32_t* done) {
    const int i = blockIdx.x, b = rows[i];
    bool bad = (unsigned)b >= (unsigned)s.B;
    for (int e = threadIdx.x; e < i; e += blockDim.x) bad |= rows[e] == b;
    int len = 0;
    if (!bad) len = paged_len(s, lens, b);
    bad = __syncthreads_or(bad);                   // every thread has read the length
    if (threadIdx.x == 0) done[i] = !bad;
    if (bad) return;
    const int want = keep ? keep[i] : 0;
    const int now = want < 0 || want > len ? len : want;
    const int c0 = (now + s.P - 1) >> s.logP, c1 = (len + s.P - 1) >> s.logP;
    for (int c = c0 + threadIdx.x; c < c1; c += blockDim.x) {
        int32_t* e = table + (size_t)b * s.cols + c;
        const int page = *e;
        *e = -1;
        if ((unsigned)page < (unsigned)s.n_pages) atomicSub(&ref[page], 1);
    }
    if (threadIdx.x == 0) lens[b] = now;
}

// ------------------------------------------------------------------ compact

struct CompactArgs {
    PagedShape s;
    __nv_bfloat16* kp;
    __nv_bfloat16* vp;
    int32_t* table;
    const int32_t* lens;
    int32_t* ref;
    int32_t* remap;
    int32_t* n_live;
    int32_t* moves;       // [1] how many
    int32_t* from;        // [n_pages] i-th used page behind the live count
    int32_t* to;          // [n_pages] i-th free page below it
};

__global__ void __launch_bounds__(PLAN_THREADS) compact_plan_kernel(const CompactArgs a) {
    __shared__ int warp_sums[32];
    const int n = a.s.n_pages;
    pdl_launch();
    int mine = 0, live;
    for (int p = threadIdx.x; p < n; p += PLAN_THREADS) mine += a.ref[p] > 0;
    block_scan(mine, &live, warp_sums);
    int holes = 0, movers = 0;
    for (int p0 = 0; p0 < n; p0 += 4 * PLAN_THREADS) {
        const int p = p0 + 4 * threadIdx.x;
        bool hole[4], mover[4];
        int h = 0, m = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool in = p + i < n, used = in && a.ref[p + i] > 0;
            hole[i] = in && !used && p + i < live;
            mover[i] = used && p + i >= live;
            h += hole[i];
            m += mover[i];
            if (in && !mover[i]) a.remap[p + i] = used ? p + i : -1;
        }
        // one scan for both: at most 4096 of each per step
        int sum;
        const int at = block_scan((h << 16) | m, &sum, warp_sums);
        int ah = holes + (at >> 16), am = movers + (at & 0xFFFF);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (hole[i]) a.to[ah++] = p + i;
            if (mover[i]) a.from[am++] = p + i;
        }
        holes += sum >> 16;
        movers += sum & 0xFFFF;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < movers; i += PLAN_THREADS) {
        const int f = a.from[i], t = a.to[i];
        a.remap[f] = t;
        a.ref[t] = a.ref[f];
        a.ref[f] = 0;
    }
    if (threadIdx.x == 0) {
        *a.n_live = live;
        *a.moves = movers;
    }
}

// Pages move from ids >= n_live into ids below it, so no copy reads what another writes.
constexpr int PIECE = 4096;              // bytes of a page per CTA step: 256 threads x 16

__global__ void __launch_bounds__(256) compact_move_kernel(const CompactArgs a) {
    const PagedShape& s = a.s;
    pdl_wait();
    const int moves = *a.moves;
    if (moves == 0) return;                        // then no entry changes either
    const size_t kb = (size_t)s.Hkv * s.P * s.dqk * 2, vb = (size_t)s.Hkv * s.P * s.dv * 2;
    constexpr int U = 4;
    const int kn = (int)((kb + PIECE * U - 1) / (PIECE * U)), vn = (int)((vb + PIECE * U - 1) / (PIECE * U));
    const long long items = (long long)moves * (kn + vn);
    for (long long it = blockIdx.x; it < items; it += gridDim.x) {
        const int i = (int)(it / (kn + vn)), c = (int)(it % (kn + vn));
        const size_t f = a.from[i], t = a.to[i];
        const bool key = c < kn;
        const size_t bytes = key ? kb : vb, off = (size_t)(key ? c : c - kn) * PIECE * U;
        uint8_t* pool = reinterpret_cast<uint8_t*>(key ? a.kp : a.vp);
        const uint8_t* src = pool + f * bytes;
        uint8_t* dst = pool + t * bytes;
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const size_t o = off + u * PIECE + threadIdx.x * 16;
            if (o < bytes) x[u] = __ldcs(reinterpret_cast<const uint4*>(src + o));
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const size_t o = off + u * PIECE + threadIdx.x * 16;
            if (o < bytes) __stcs(reinterpret_cast<uint4*>(dst + o), x[u]);
        }
    }
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < (long long)s.B * s.cols;
         e += (long long)gridDim.x * 256) {
        const int b = (int)(e / s.cols), c = (int)(e % s.cols);
        if (c >= (paged_len(s, a.lens, b) + s.P - 1) >> s.logP) continue;
        const int page = a.table[e];
        if ((unsigned)page < (unsigned)s.n_pages && a.remap[page] >= 0) a.table[e] = a.remap[page];
    }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t paged_append_ws_bytes(const PagedShape& s) {
    return up256((size_t)s.B * sizeof(int4)) + up256((size_t)s.n_pages * 4);
}

cudaError_t launch_paged_append(const PagedShape& s, const __nv_bfloat16* k_new, const __nv_bfloat16* v_new,
                                const int32_t* n_new, __nv_bfloat16* kp, __nv_bfloat16* vp, int32_t* table,
                                int32_t* lens, int32_t* ref, int32_t* short_pages, uint8_t* ws, cudaStream_t st) {
    AppendArgs a{s, k_new, v_new, n_new, kp, vp, table, lens, ref, short_pages, nullptr, nullptr};
    a.plan = reinterpret_cast<int4*>(ws);
    a.free_list = reinterpret_cast<int32_t*>(ws + up256((size_t)s.B * sizeof(int4)));
    const int smem = s.B * APPEND_SMEM_ROW;
    static std::atomic<bool> allowed[MAX_DEVICES];
    int dev;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = allow_smem(reinterpret_cast<const void*>(append_plan_kernel), APPEND_MAX_B * APPEND_SMEM_ROW, dev, allowed);
    if (e != cudaSuccess) return e;
    append_plan_kernel<<<1, PLAN_THREADS, smem, st>>>(a);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const int touched = (s.Tq + 2 * s.P - 2) / s.P;      // pages that Tq tokens can lie in
    return launch_dependent(append_write_kernel, dim3(touched, s.Hkv, s.B), 256, 0, st, a);
}

cudaError_t launch_pages_fork(const PagedShape& s, int n, const int32_t* src, const int32_t* dst, int32_t* table,
                              int32_t* lens, int32_t* ref, int32_t* done, cudaStream_t st) {
    pages_fork_kernel<<<n, 128, 0, st>>>(s, n, src, dst, table, lens, ref, done);
    return cudaGetLastError();
}

cudaError_t launch_pages_free(const PagedShape& s, int n, const int32_t* rows, const int32_t* keep, int32_t* table,
                              int32_t* lens, int32_t* ref, int32_t* done, cudaStream_t st) {
    pages_free_kernel<<<n, 128, 0, st>>>(s, n, rows, keep, table, lens, ref, done);
    return cudaGetLastError();
}

size_t pages_compact_ws_bytes(const PagedShape& s) { return 256 + 2 * up256((size_t)s.n_pages * 4); }

cudaError_t launch_pages_compact(const PagedShape& s, __nv_bfloat16* kp, __nv_bfloat16* vp, int32_t* table,
                                 const int32_t* lens, int32_t* ref, int32_t* remap, int32_t* n_live, uint8_t* ws,
                                 cudaStream_t st) {
    CompactArgs a{s, kp, vp, table, lens, ref, remap, n_live, nullptr, nullptr, nullptr};
    a.moves = reinterpret_cast<int32_t*>(ws);
    a.from = reinterpret_cast<int32_t*>(ws + 256);
    a.to = reinterpret_cast<int32_t*>(ws + 256 + up256((size_t)s.n_pages * 4));
    compact_plan_kernel<<<1, PLAN_THREADS, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_dependent(compact_move_kernel, dim3(148 * 8), 256, 0, st, a);
}

}  // namespace nsa
