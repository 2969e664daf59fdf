// What the entry points' host-side checks share.
#pragma once

#include "common.cuh"

namespace nsa {

inline bool aligned16(const void* p) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// a b c <= INT32_MAX for counts a, b, c < 2^31, whose product may pass 64 bits.
inline bool fits32(int64_t a, int64_t b, int64_t c) { return a * b <= INT32_MAX && a * b * c <= INT32_MAX; }
inline bool supported_dqk(int d) { return d == 64 || d == 128 || d == 192 || d == 256; }
inline bool supported_dv(int d) { return d == 64 || d == 128 || d == 256; }

// NSA_OK or NSA_ERR_CUDA, remembering the error for nsa_last_cuda_error (nsa_abi.cu).
nsa_status cuda_status(cudaError_t e);

}  // namespace nsa
