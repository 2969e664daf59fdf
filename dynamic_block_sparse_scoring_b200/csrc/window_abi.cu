// C ABI of the sliding-window attention with sink tokens: host-side validation
// and the choice of kernel (include/nsa.h).
#include <stdint.h>

#include <algorithm>

#include "abi_checks.cuh"
#include "window.cuh"

namespace {

using nsa::WinShape;
using nsa::aligned16;
using nsa::cuda_status;

nsa_status make_win_shape(const nsa_window_config* cfg, WinShape* s) {
    if (!cfg) return NSA_ERR_INVALID_ARG;
    const nsa_window_config& c = *cfg;
    if (c.flags != 0) return NSA_ERR_INVALID_ARG;
    if (c.batch < 1 || c.seqlen_q < 0 || c.seqlen_kv < 1 || c.q_pos0 < 0) return NSA_ERR_INVALID_ARG;
    if ((int64_t)c.q_pos0 + c.seqlen_q > c.seqlen_kv) return NSA_ERR_INVALID_ARG;
    if (c.h_q < 1 || c.h_kv < 1 || c.h_q % c.h_kv != 0) return NSA_ERR_INVALID_ARG;
    if (c.d_qk < 1 || c.d_v < 1 || c.window < 1 || c.sink < 0) return NSA_ERR_INVALID_ARG;
    if (!(c.scale >= 1e-30f && c.scale <= 1e30f)) return NSA_ERR_INVALID_ARG;       // (NaN too)
    if (!nsa::supported_dqk(c.d_qk) || !nsa::supported_dv(c.d_v)) return NSA_ERR_UNSUPPORTED;
    // rows and planes are counted in 32 bits, and positions a tile behind the last one exist
    if (!nsa::fits32(c.batch, c.seqlen_q, c.h_q) || !nsa::fits32(c.batch, c.h_kv, c.seqlen_kv) ||
        c.seqlen_kv > INT32_MAX - 1024)
        return NSA_ERR_UNSUPPORTED;
    s->B = c.batch;
    s->Tq = c.seqlen_q;
    s->Tk = c.seqlen_kv;
    s->q0 = c.q_pos0;
    s->Hq = c.h_q;
    s->Hkv = c.h_kv;
    s->G = c.h_q / c.h_kv;
    s->dqk = c.d_qk;
    s->dv = c.d_v;
    s->win = std::min(c.window, c.seqlen_kv);
    s->ns = std::min(c.sink, c.seqlen_kv);
    s->scale = c.scale;
    return NSA_OK;
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Workspace of the backward: delta [B, Tq, Hq], then the tensor-core kernel's partial sums.
size_t delta_bytes(const WinShape& s) { return up256((size_t)s.B * s.Tq * s.Hq * 4); }

size_t bwd_bytes(const WinShape& s) {
    return delta_bytes(s) + (nsa::window_tc_supported(s) && s.Tq > 0 ? nsa::window_bwd_tc_part_bytes(s) : 0);
}

}  // namespace

extern "C" {

nsa_status nsa_window_attn_fwd(const nsa_window_config* cfg, const void* q, const void* k, const void* v,
                               void* out, float* lse, void* stream) {
    WinShape s;
    nsa_status st = make_win_shape(cfg, &s);
    if (st != NSA_OK) return st;
    if (s.Tq > 0 && (!q || !out)) return NSA_ERR_INVALID_ARG;     // (buffers of zero elements may be NULL)
    if (!k || !v) return NSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(lse))
        return NSA_ERR_INVALID_ARG;
    if (s.Tq == 0) return NSA_OK;
    const __nv_bfloat16* qb = static_cast<const __nv_bfloat16*>(q);
    const __nv_bfloat16* kb = static_cast<const __nv_bfloat16*>(k);
    const __nv_bfloat16* vb = static_cast<const __nv_bfloat16*>(v);
    __nv_bfloat16* ob = static_cast<__nv_bfloat16*>(out);
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (nsa::window_tc_supported(s)) return cuda_status(nsa::launch_window_fwd_tc(s, qb, kb, vb, ob, lse, cs));
    return cuda_status(nsa::launch_window_rowwise_fwd(s, qb, kb, vb, ob, lse, cs));
}

nsa_status nsa_window_bwd_workspace_size(const nsa_window_config* cfg, size_t* bytes) {
    if (!bytes) return NSA_ERR_INVALID_ARG;
    WinShape s;
    nsa_status st = make_win_shape(cfg, &s);
    if (st != NSA_OK) return st;
    *bytes = bwd_bytes(s);
    return NSA_OK;
}

nsa_status nsa_window_attn_bwd(const nsa_window_config* cfg, const void* q, const void* k, const void* v,
                               const void* out, const float* lse, const void* d_out, void* dq, void* dk,
                               void* dv, void* workspace, size_t ws_bytes, void* stream) {
    WinShape s;
    nsa_status st = make_win_shape(cfg, &s);
    if (st != NSA_OK) return st;
    if (s.Tq > 0 && (!q || !out || !lse || !d_out || !dq)) return NSA_ERR_INVALID_ARG;
    if (!k || !v || !dk || !dv) return NSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out) || !aligned16(lse) ||
        !aligned16(d_out) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv) || !aligned16(workspace))
        return NSA_ERR_INVALID_ARG;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    if (s.Tq == 0) {                               // no query: the keys' gradients are zero
        st = cuda_status(cudaMemsetAsync(dk, 0, (size_t)s.B * s.Hkv * s.Tk * s.dqk * 2, cs));
        return st != NSA_OK ? st : cuda_status(cudaMemsetAsync(dv, 0, (size_t)s.B * s.Hkv * s.Tk * s.dv * 2, cs));
    }
    if (!workspace || ws_bytes < bwd_bytes(s)) return NSA_ERR_WORKSPACE;
    if (nsa::window_tc_supported(s))
        return cuda_status(nsa::launch_window_bwd_tc(
            s, static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
            static_cast<const __nv_bfloat16*>(v), static_cast<const __nv_bfloat16*>(out), lse,
            static_cast<const __nv_bfloat16*>(d_out), static_cast<__nv_bfloat16*>(dq),
            static_cast<__nv_bfloat16*>(dk), static_cast<__nv_bfloat16*>(dv), static_cast<float*>(workspace),
            reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + delta_bytes(s)), cs));
    return cuda_status(nsa::launch_window_rowwise_bwd(
        s, static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k),
        static_cast<const __nv_bfloat16*>(v), static_cast<const __nv_bfloat16*>(out), lse,
        static_cast<const __nv_bfloat16*>(d_out), static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dk),
        static_cast<__nv_bfloat16*>(dv), static_cast<float*>(workspace), cs));
}

}  // extern "C"
