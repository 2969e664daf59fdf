// C ABI of the paged key/value cache: host-side validation (include/nsa.h).
#include <stdint.h>

#include "abi_checks.cuh"
#include "paged.cuh"

namespace {

using nsa::PagedShape;
using nsa::aligned16;
using nsa::aligned4;
using nsa::cuda_status;

nsa_status make_paged_shape(const nsa_paged_config* cfg, PagedShape* s) {
    if (!cfg) return NSA_ERR_INVALID_ARG;
    const nsa_paged_config& c = *cfg;
    if (c.flags != 0) return NSA_ERR_INVALID_ARG;
    if (c.batch < 1 || c.seqlen_q < 1 || c.n_pages < 1 || c.max_pages < 1) return NSA_ERR_INVALID_ARG;
    if (c.h_q < 1 || c.h_kv < 1 || c.h_q % c.h_kv != 0) return NSA_ERR_INVALID_ARG;
    if (c.d_qk < 1 || c.d_v < 1 || c.page_size < 1 || c.window < 0 || c.sink < 0) return NSA_ERR_INVALID_ARG;
    if (!(c.scale >= 1e-30f && c.scale <= 1e30f)) return NSA_ERR_INVALID_ARG;       // (NaN too)
    if (!nsa::supported_dqk(c.d_qk) || !nsa::supported_dv(c.d_v)) return NSA_ERR_UNSUPPORTED;
    int log_p = 4;
    while (log_p < 8 && (1 << log_p) != c.page_size) ++log_p;
    if ((1 << log_p) != c.page_size) return NSA_ERR_UNSUPPORTED;
    // positions and table entries are counted in 32 bits
    const int64_t cap = (int64_t)c.max_pages * c.page_size;
    if (cap > INT32_MAX - 1024 || c.seqlen_q > INT32_MAX / 2 || (int64_t)c.batch * c.max_pages > INT32_MAX)
        return NSA_ERR_UNSUPPORTED;
    if (c.h_kv > 65535) return NSA_ERR_UNSUPPORTED;
    s->B = c.batch;
    s->Tq = c.seqlen_q;
    s->Hq = c.h_q;
    s->Hkv = c.h_kv;
    s->G = c.h_q / c.h_kv;
    s->dqk = c.d_qk;
    s->dv = c.d_v;
    s->P = c.page_size;
    s->logP = log_p;
    s->n_pages = c.n_pages;
    s->cols = c.max_pages;
    s->win = c.window >= cap ? 0 : c.window;       // such a window hides nothing
    s->ns = c.sink;
    s->scale = c.scale;
    return NSA_OK;
}

}  // namespace

extern "C" {

nsa_status nsa_paged_workspace_size(const nsa_paged_config* cfg, size_t* bytes) {
    if (!bytes) return NSA_ERR_INVALID_ARG;
    PagedShape s;
    nsa_status st = make_paged_shape(cfg, &s);
    if (st != NSA_OK) return st;
    *bytes = nsa::paged_attn_ws_bytes(s);
    return NSA_OK;
}

nsa_status nsa_paged_attn_fwd(const nsa_paged_config* cfg, const void* q, const void* k_pages,
                              const void* v_pages, const int32_t* table, const int32_t* lens, void* out,
                              float* lse, void* workspace, size_t ws_bytes, void* stream) {
    PagedShape s;
    nsa_status st = make_paged_shape(cfg, &s);
    if (st != NSA_OK) return st;
    if (!q || !k_pages || !v_pages || !table || !lens || !out) return NSA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k_pages) || !aligned16(v_pages) || !aligned16(table) || !aligned16(lens) ||
        !aligned16(out) || !aligned16(lse) || !aligned16(workspace))
        return NSA_ERR_INVALID_ARG;
    // units (16 query rows of a sequence and KV head) are counted in 32 bits
    if ((int64_t)s.Tq * s.G > INT32_MAX / 2 || !nsa::fits32(s.B, s.Hkv, ((int64_t)s.Tq * s.G + 15) / 16))
        return NSA_ERR_UNSUPPORTED;
    if (!workspace || ws_bytes < nsa::paged_attn_ws_bytes(s)) return NSA_ERR_WORKSPACE;
    return cuda_status(nsa::launch_paged_attn(
        s, static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(k_pages),
        static_cast<const __nv_bfloat16*>(v_pages), table, lens, static_cast<__nv_bfloat16*>(out), lse,
        static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

nsa_status nsa_paged_append_workspace_size(const nsa_paged_config* cfg, size_t* bytes) {
    if (!bytes) return NSA_ERR_INVALID_ARG;
    PagedShape s;
    nsa_status st = make_paged_shape(cfg, &s);
    if (st != NSA_OK) return st;
    *bytes = nsa::paged_append_ws_bytes(s);
    return NSA_OK;
}

nsa_status nsa_paged_append(const nsa_paged_config* cfg, const void* k_new, const void* v_new,
                            const int32_t* n_new, void* k_pages, void* v_pages, int32_t* table, int32_t* lens,
                            int32_t* ref, int32_t* short_pages, void* workspace, size_t ws_bytes, void* stream) {
    PagedShape s;
    nsa_status st = make_paged_shape(cfg, &s);
    if (st != NSA_OK) return st;
    if (!k_new || !v_new || !k_pages || !v_pages || !table || !lens || !ref || !short_pages)
        return NSA_ERR_INVALID_ARG;
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(n_new) || !aligned16(k_pages) ||
        !aligned16(v_pages) || !aligned16(table) || !aligned16(lens) || !aligned16(ref) ||
        !aligned4(short_pages) || !aligned16(workspace))
        return NSA_ERR_INVALID_ARG;
    if (s.B > nsa::APPEND_MAX_B) return NSA_ERR_UNSUPPORTED;
    if (!workspace || ws_bytes < nsa::paged_append_ws_bytes(s)) return NSA_ERR_WORKSPACE;
    return cuda_status(nsa::launch_paged_append(
        s, static_cast<const __nv_bfloat16*>(k_new), static_cast<const __nv_bfloat16*>(v_new), n_new,
        static_cast<__nv_bfloat16*>(k_pages), static_cast<__nv_bfloat16*>(v_pages), table, lens, ref, short_pages,
        static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

nsa_status nsa_pages_fork(const nsa_paged_config* cfg, int32_t n, const int32_t* src, const int32_t* dst,
                          int32_t* table, int32_t* lens, int32_t* ref, int32_t* done, void* stream) {
    PagedShape s;
    nsa_status st = make_paged_shape(cfg, &s);
    if (st != NSA_OK) return st;
    if (n < 0 || !table || !lens || !ref) return NSA_ERR_INVALID_ARG;
    if (!aligned16(table) || !aligned16(lens) || !aligned16(ref)) return NSA_ERR_INVALID_ARG;
    if (n == 0) return NSA_OK;
    if (!src || !dst || !done || !aligned4(src) || !aligned4(dst) || !aligned4(done)) return NSA_ERR_INVALID_ARG;
    return cuda_status(
        nsa::launch_pages_fork(s, n, src, dst, table, lens, ref, done, static_cast<cudaStream_t>(stream)));
}

nsa_status nsa_pages_free(const nsa_paged_config* cfg, int32_t n, const int32_t* rows, const int32_t* keep,
                          int32_t* table, int32_t* lens, int32_t* ref, int32_t* done, void* stream) {
    PagedShape s;
    nsa_status st = make_paged_shape(cfg, &s);
    if (st != NSA_OK) return st;
    if (n < 0 || !table || !lens || !ref) return NSA_ERR_INVALID_ARG;
    if (!aligned16(table) || !aligned16(lens) || !aligned16(ref)) return NSA_ERR_INVALID_ARG;
    if (n == 0) return NSA_OK;
    if (!rows || !done || !aligned4(rows) || !aligned4(keep) || !aligned4(done)) return NSA_ERR_INVALID_ARG;
    return cuda_status(
        nsa::launch_pages_free(s, n, rows, keep, table, lens, ref, done, static_cast<cudaStream_t>(stream)));
}

nsa_status nsa_pages_compact_workspace_size(const nsa_paged_config* cfg, size_t* bytes) {
    if (!bytes) return NSA_ERR_INVALID_ARG;
    PagedShape s;
    nsa_status st = make_paged_shape(cfg, &s);
    if (st != NSA_OK) return st;
    *bytes = nsa::pages_compact_ws_bytes(s);
    return NSA_OK;
}

nsa_status nsa_pages_compact(const nsa_paged_config* cfg, void* k_pages, void* v_pages, int32_t* table,
                             const int32_t* lens, int32_t* ref, int32_t* remap, int32_t* n_live,
                             void* workspace, size_t ws_bytes, void* stream) {
    PagedShape s;
    nsa_status st = make_paged_shape(cfg, &s);
    if (st != NSA_OK) return st;
    if (!k_pages || !v_pages || !table || !lens || !ref || !remap || !n_live) return NSA_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(v_pages) || !aligned16(table) || !aligned16(lens) || !aligned16(ref) ||
        !aligned16(remap) || !aligned4(n_live) || !aligned16(workspace))
        return NSA_ERR_INVALID_ARG;
    if (!workspace || ws_bytes < nsa::pages_compact_ws_bytes(s)) return NSA_ERR_WORKSPACE;
    return cuda_status(nsa::launch_pages_compact(
        s, static_cast<__nv_bfloat16*>(k_pages), static_cast<__nv_bfloat16*>(v_pages), table, lens, ref, remap,
        n_live, static_cast<uint8_t*>(workspace), static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
