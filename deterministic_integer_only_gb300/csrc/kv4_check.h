// Host checks that the entry points of the 4-bit paged K/V cache share
// (internal to the library).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>
#include <stdio.h>

#include "../../include/detint.h"
#include "kernels.h"

namespace detint {

constexpr int KV4_MAX_LEN = 1 << 19;       // keys: the limb sums stay in int32

inline int failed(int code, const char* where, const char* what) {
    char msg[160];
    snprintf(msg, sizeof msg, "%s: %s", where, what);
    return set_last_error(code, msg);
}
// (the error is reported here and not left for the check of the next launch)
inline int cuda_fail(const char* where, cudaError_t e) {
    cudaGetLastError();
    return failed(DETINT_E_CUDA, where, cudaGetErrorString(e));
}
inline bool mis(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) != 0; }
// an array of a call; null ones overlap nothing
struct Span {
    const void* p;
    size_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x && y && x < y + b.bytes && y < x + a.bytes;
}
// whether an array that is written overlaps another one, written or read
template <int NO, int NI>
inline bool clash(const Span (&out)[NO], const Span (&in)[NI]) {
    for (int i = 0; i < NO; ++i) {
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return true;
        for (int j = 0; j < NI; ++j)
            if (overlap(out[i], in[j])) return true;
    }
    return false;
}

// the checks every entry point shares; fills the kernels' view of the cache
inline int check_cache(const char* where, const detint_kv4_t* c, Kv4Args* a) {
    auto err = [&](int code, const char* what) { return failed(code, where, what); };
    if (!c) return err(DETINT_E_ARG, "null cache");
    if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->block_table || !c->params) return err(DETINT_E_ARG, "null pointer in the cache");
    if (c->head_dim != 64 && c->head_dim != 128) return err(DETINT_E_SHAPE, "head_dim must be 64 or 128");
    if (c->n_kv < 1 || c->n_q < 1 || c->n_q > 1024 || c->n_q % c->n_kv || c->n_q / c->n_kv > 64)
        return err(DETINT_E_SHAPE, "n_q must be n_kv times 1..64, at most 1024");
    if (c->n_blocks < 1 || c->n_seq < 1 || c->max_blocks < 1) return err(DETINT_E_ARG, "n_blocks, n_seq and max_blocks must be positive");
    if (mis(c->k, 16) || mis(c->v, 16) || mis(c->k_scale, 16) || mis(c->v_scale, 16) || mis(c->params, 16))
        return err(DETINT_E_ARG, "pages, scale codes and parameters must be 16-byte aligned");
    if (mis(c->block_table, 4) || mis(c->status, 4)) return err(DETINT_E_ARG, "block_table and status must be 4-byte aligned");
    a->nq = c->n_q; a->n_kv = c->n_kv; a->n_blocks = c->n_blocks; a->n_seq = c->n_seq; a->max_blocks = c->max_blocks;
    a->gmul = (65536 + c->n_q / c->n_kv - 1) / (c->n_q / c->n_kv);
    a->k = c->k; a->v = c->v; a->ks = c->k_scale; a->vs = c->v_scale;
    a->block_table = c->block_table; a->params = c->params; a->status = c->status;
    return DETINT_OK;
}

inline int check_attn(const char* where, const detint_kv4_t* c, const int8_t* q8, const int32_t* mq, const int32_t* kq,
               const int32_t* tok_seq, const int32_t* tok_pos, int n_tok, int max_len, int window, int32_t* o,
               long long o_stride, Kv4Args* a, Kv4Attn* p) {
    auto err = [&](int code, const char* what) { return failed(code, where, what); };
    const int rc = check_cache(where, c, a);
    if (rc) return rc;
    if (!q8 || !mq || !kq || !tok_seq || !tok_pos || !o) return err(DETINT_E_ARG, "null pointer");
    if (n_tok < 1) return err(DETINT_E_ARG, "n_tok must be positive");
    if (max_len < 1 || max_len > KV4_MAX_LEN) return err(DETINT_E_ARG, "max_len must be in 1..524288");
    if (window < 0) return err(DETINT_E_ARG, "window must not be negative");
    if (mis(tok_seq, 4) || mis(tok_pos, 4) || mis(mq, 4) || mis(kq, 4)) return err(DETINT_E_ARG, "tokens and scales must be 4-byte aligned");
    if (mis(q8, 16) || mis(o, 8)) return err(DETINT_E_ARG, "q8 must be 16-byte and o 8-byte aligned");
    if (o_stride < (long long)c->n_q * c->head_dim || (o_stride & 1)) return err(DETINT_E_ARG, "o_stride must be even and hold a row");
    *p = Kv4Attn{};
    p->q8 = q8; p->mq = mq; p->kq = kq; p->tok_seq = tok_seq; p->tok_pos = tok_pos; p->o = o; p->o_stride = (size_t)o_stride;
    p->T = n_tok; p->G = c->n_q / c->n_kv; p->max_len = max_len;
    p->window = window < max_len ? window : 0;      // a window that every key is in: none (any int, so no sum with it may overflow)
    return DETINT_OK;
}

}  // namespace detint
