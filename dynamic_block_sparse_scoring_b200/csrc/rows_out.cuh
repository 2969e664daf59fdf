// Rows of a TMEM accumulator to global memory.  A thread holds a piece of its
// own row, so storing it directly touches 32 lines per instruction; four lanes
// first trade 16-byte units (a 4 x 4 transpose by shuffles), after which each
// store covers 64 contiguous bytes of eight rows.
#pragma once

#include "common.cuh"

namespace nsa {

// Lane i of a group of four: u[j] becomes lane j's u[i].
__device__ __forceinline__ void transpose4(uint4* u, int lane) {
#pragma unroll
    for (int k = 1; k < 4; k <<= 1) {
        const bool hi = lane & k;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            if (a & k) continue;
            uint4 v = hi ? u[a] : u[a | k];
            v.x = __shfl_xor_sync(0xffffffffu, v.x, k);
            v.y = __shfl_xor_sync(0xffffffffu, v.y, k);
            v.z = __shfl_xor_sync(0xffffffffu, v.z, k);
            v.w = __shfl_xor_sync(0xffffffffu, v.w, k);
            if (hi) u[a] = v;
            else u[a | k] = v;
        }
    }
}

// The four rows that a lane stores for its group: 4-row group base of its quarter + j.
struct OutRows {
    long long off[4];       // in rows of the output, -1: not a row of the output
};

// 32 fp32 columns of a lane's row times f, as bf16.
__device__ __forceinline__ void pack32(const uint32_t* o, float f, uint4* u) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        float z[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) z[e] = __uint_as_float(o[8 * q + e]) * f;
        u[q] = pack8(z);
    }
}

// 32 bf16 columns of every lane's row to column col of a row-major output of d
// columns.  All lanes of the warp call it.
__device__ __forceinline__ void store_bf16x32(uint4* u, __nv_bfloat16* out, const OutRows& r, int d, int col, int lane) {
    transpose4(u, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (r.off[j] >= 0) *reinterpret_cast<uint4*>(out + r.off[j] * d + col + (lane & 3) * 8) = u[j];
}

// The four rows (token, head) of a query tile: token << 16 | head, the same for every tile.
struct TileRows {
    int id[4];

    __device__ __forceinline__ void init(int r, int G) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int rj = (r & ~3) + j, t = rj / G;
            id[j] = (t << 16) | (rj - t * G);
        }
    }
    // Rows of the tile of `tokens` tokens whose first is row `base` of an output with H rows a token.
    __device__ __forceinline__ OutRows at(long long base, int tokens, int H) const {
        OutRows o;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = id[j] >> 16;
            o.off[j] = t < tokens ? base + (long long)t * H + (id[j] & 0xFFFF) : -1;
        }
        return o;
    }
};

// The same 32 columns unscaled, as fp32.
__device__ __forceinline__ void store_f32x32(const uint32_t* o, float* out, const OutRows& r, int d, int col, int lane) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint4 u[4];
#pragma unroll
        for (int q = 0; q < 4; ++q)
            u[q] = make_uint4(o[16 * h + 4 * q], o[16 * h + 4 * q + 1], o[16 * h + 4 * q + 2], o[16 * h + 4 * q + 3]);
        transpose4(u, lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (r.off[j] >= 0) *reinterpret_cast<uint4*>(out + r.off[j] * d + col + 16 * h + (lane & 3) * 4) = u[j];
    }
}

}  // namespace nsa
