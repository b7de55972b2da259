// Checks that the cache's entry points share (host code).
#pragma once

#include "qmv.h"
#include "qmv_internal.h"
#include "qmv_kv.h"

namespace qmv {

inline bool aligned(const void *p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline qmv_status from_hip(hipError_t e) {
    if (e == hipSuccess) return QMV_OK;
    set_last_hip_error(e);
    return QMV_EHIP;
}

// The sizes of a cache (the pointers apart).
inline qmv_status check_cache_shape(const qmv_kv_cache *c) {
    if (!c || !kv_type_ok(c->type)) return QMV_EINVAL;
    if (!qmv_kv_page_bytes(c->type, c->n_kv_heads, c->head_dim, c->page_size)) return QMV_ESHAPE;
    if (c->n_pages < 1 || c->n_pages > 0x7FFFFFFFll) return QMV_ESHAPE;
    if (c->n_seq < 1 || c->n_seq > 65535) return QMV_ESHAPE;
    if (c->table_ld < 1 || c->table_ld > (1ll << 30) / c->page_size) return QMV_ESHAPE;
    return QMV_OK;
}

inline qmv_status check_cache(const qmv_kv_cache *c, KvArgs &k) {
    qmv_status st = check_cache_shape(c);
    if (st != QMV_OK) return st;
    if (!c->pages || !c->table || !c->seq_len) return QMV_EINVAL;
    if (!aligned(c->pages, 16) || !aligned(c->table, 4) || !aligned(c->seq_len, 4)) return QMV_EALIGN;
    k = KvArgs{};
    k.pages = (uint8_t *)c->pages;
    k.table = c->table;
    k.seq_len = c->seq_len;
    k.table_ld = c->table_ld;
    k.head_bytes = kv_head_bytes(c->type, c->head_dim, c->page_size);
    k.n_pages = (int32_t)c->n_pages;
    k.n_seq = (int32_t)c->n_seq;
    k.n_kv = c->n_kv_heads;
    k.hd = c->head_dim;
    k.page_shift = __builtin_ctz((unsigned)c->page_size);
    k.cap = (int32_t)(c->table_ld * c->page_size);
    return QMV_OK;
}

// n rows, divided by a start array or evenly.
inline qmv_status check_rows(const qmv_kv_cache *c, int64_t n, const int32_t *start) {
    if (n < 1 || n > QMV_MAX_KV_ROWS) return QMV_ESHAPE;
    if (!start && n % c->n_seq != 0) return QMV_ESHAPE;
    if (!aligned(start, 4)) return QMV_EALIGN;
    return QMV_OK;
}

}  // namespace qmv
