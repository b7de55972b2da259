// C ABI of what stands around a cache's attention: rows read back, norms and
// rotation of queries and keys, pages taken and given back.  Argument checks on
// the host, then kernel launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <math.h>

#include "qmv.h"
#include "qmv_cache_api.h"
#include "qmv_pages.h"
#include "qmv_rope.h"

using namespace qmv;

extern "C" {

qmv_status qmv_kv_read(const qmv_kv_cache *cache, int64_t n, const int32_t *start, float *k, int64_t ldk,
                       float *v, int64_t ldv, hipStream_t stream) {
    KvArgs c;
    qmv_status st = check_cache(cache, c);
    if (st != QMV_OK) return st;
    st = check_rows(cache, n, start);
    if (st != QMV_OK) return st;
    const int64_t w = (int64_t)c.n_kv * c.hd;
    if (ldk < w || ldv < w || ldk > (1ll << 40) || ldv > (1ll << 40)) return QMV_ESHAPE;
    if (!k || !v) return QMV_EINVAL;
    if (!aligned(k, 4) || !aligned(v, 4)) return QMV_EALIGN;
    return from_hip(launch_kv_read(cache->type, c, n, start, k, ldk, v, ldv, stream));
}

static qmv_status check_rope(const qmv_qk_rope *r, int32_t head_dim, RopeArgs &a) {
    if (!r || (r->pairs != QMV_ROPE_HALVES && r->pairs != QMV_ROPE_ADJACENT)) return QMV_EINVAL;
    if (!kv_head_dim_ok(head_dim) || r->rot_dim < 0 || r->rot_dim > head_dim || r->rot_dim % 8 != 0) return QMV_ESHAPE;
    if (!(r->eps >= 0.f) || isinf(r->eps)) return QMV_EINVAL;
    if (r->rot_dim > 0 && !r->freq) return QMV_EINVAL;
    if (!aligned(r->freq, 8) || !aligned(r->q_norm, 4) || !aligned(r->k_norm, 4)) return QMV_EALIGN;
    a = RopeArgs{r->q_norm, r->k_norm, r->freq, r->eps, r->rot_dim, r->pairs == QMV_ROPE_ADJACENT};
    return QMV_OK;
}

// Rows of heads that are turned: out may be in itself.
static qmv_status check_heads(int32_t head_dim, int32_t heads, const float *in, int64_t ld_in, float *out,
                              int64_t ld_out, HeadRows &h) {
    if (heads < 0 || heads > 32767) return QMV_ESHAPE;
    h = HeadRows{in, ld_in, out, ld_out, heads};
    if (heads == 0) return QMV_OK;
    const int64_t w = (int64_t)heads * head_dim;
    if (ld_in < w || ld_out < w || ld_in > (1ll << 40) || ld_out > (1ll << 40)) return QMV_ESHAPE;
    if (!in || !out) return QMV_EINVAL;
    if (!aligned(in, 4) || !aligned(out, 4)) return QMV_EALIGN;
    if (in == out && ld_in != ld_out) return QMV_EINVAL;
    return QMV_OK;
}

qmv_status qmv_qk_norm_rope(const qmv_qk_rope *rope, int32_t head_dim, int64_t n, const int32_t *pos,
                            int32_t n_heads, const float *q, int64_t ldq, float *q_out, int64_t ldqo,
                            int32_t n_kv_heads, const float *k, int64_t ldk, float *k_out, int64_t ldko,
                            hipStream_t stream) {
    RopeArgs r;
    HeadRows qr, kr;
    qmv_status st = check_rope(rope, head_dim, r);
    if (st != QMV_OK) return st;
    if (n < 1 || n > QMV_MAX_KV_ROWS) return QMV_ESHAPE;
    st = check_heads(head_dim, n_heads, q, ldq, q_out, ldqo, qr);
    if (st != QMV_OK) return st;
    st = check_heads(head_dim, n_kv_heads, k, ldk, k_out, ldko, kr);
    if (st != QMV_OK) return st;
    if (n_heads + n_kv_heads < 1) return QMV_ESHAPE;
    if (!pos) return QMV_EINVAL;
    if (!aligned(pos, 4)) return QMV_EALIGN;
    return from_hip(launch_qk_norm_rope(r, head_dim, n, pos, qr, kr, stream));
}

qmv_status qmv_kv_append_rope(const qmv_kv_cache *cache, const qmv_qk_rope *rope, int64_t n,
                              const int32_t *start, int32_t n_heads, const float *q, int64_t ldq,
                              float *q_out, int64_t ldqo, const float *k, int64_t ldk, const float *v,
                              int64_t ldv, hipStream_t stream) {
    KvArgs c;
    RopeArgs r;
    HeadRows qr;
    qmv_status st = check_cache(cache, c);
    if (st != QMV_OK) return st;
    st = check_rope(rope, cache->head_dim, r);
    if (st != QMV_OK) return st;
    st = check_rows(cache, n, start);
    if (st != QMV_OK) return st;
    if (n_heads < 1 || n_heads + c.n_kv > 65535) return QMV_ESHAPE;
    st = check_heads(c.hd, n_heads, q, ldq, q_out, ldqo, qr);
    if (st != QMV_OK) return st;
    const int64_t w = (int64_t)c.n_kv * c.hd;
    if (ldk < w || ldv < w || ldk > (1ll << 40) || ldv > (1ll << 40)) return QMV_ESHAPE;
    if (!k || !v) return QMV_EINVAL;
    if (!aligned(k, 4) || !aligned(v, 4)) return QMV_EALIGN;
    return from_hip(launch_kv_append_rope(cache->type, c, r, n, start, qr, k, ldk, v, ldv, stream));
}

// The table and the lengths are the caller's to change; the struct, which other
// calls only read, has them as constant.
qmv_status qmv_kv_reserve(const qmv_kv_cache *cache, const int32_t *add, const int32_t *free_pages,
                          int32_t *free_count, int64_t n, int32_t *granted, int32_t *start, int32_t *pos,
                          int64_t *slot, hipStream_t stream) {
    KvArgs c;
    qmv_status st = check_cache(cache, c);
    if (st != QMV_OK) return st;
    if (n < 1 || n > QMV_MAX_KV_ROWS) return QMV_ESHAPE;
    if (!add || !free_pages || !free_count || !granted || !start) return QMV_EINVAL;
    if (!aligned(add, 4) || !aligned(free_pages, 4) || !aligned(free_count, 4) || !aligned(granted, 4) ||
        !aligned(start, 4) || !aligned(pos, 4) || !aligned(slot, 8))
        return QMV_EALIGN;
    const ReserveArgs a{add, free_pages, free_count, (int32_t)n, granted, start};
    return from_hip(launch_kv_reserve(c, const_cast<int32_t *>(c.table), const_cast<int32_t *>(c.seq_len), a, pos, slot, stream));
}

qmv_status qmv_kv_release(const qmv_kv_cache *cache, const int32_t *new_len, int32_t *free_pages,
                          int32_t *free_count, hipStream_t stream) {
    KvArgs c;
    qmv_status st = check_cache(cache, c);
    if (st != QMV_OK) return st;
    if (c.n_seq * c.table_ld > 1ll << 30) return QMV_ESHAPE;  // the sums of pages end there
    if (!new_len || !free_pages || !free_count) return QMV_EINVAL;
    if (!aligned(new_len, 4) || !aligned(free_pages, 4) || !aligned(free_count, 4)) return QMV_EALIGN;
    return from_hip(launch_kv_release(c, const_cast<int32_t *>(c.table), const_cast<int32_t *>(c.seq_len), new_len,
                                      free_pages, free_count, stream));
}

}  // extern "C"
