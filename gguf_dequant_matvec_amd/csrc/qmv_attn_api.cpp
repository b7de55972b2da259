// C ABI of the paged key-value cache and its attention: argument checks on the
// host, then kernel launches on the caller's stream.  Nothing here allocates,
// copies or synchronises.
#include <hip/hip_runtime.h>

#include <math.h>

#include "qmv.h"
#include "qmv_attn_plan.h"
#include "qmv_cache_api.h"
#include "qmv_internal.h"
#include "qmv_kv.h"

using namespace qmv;

extern "C" {

size_t qmv_kv_page_bytes(int32_t type, int32_t n_kv_heads, int32_t head_dim, int32_t page_size) {
    if (!kv_type_ok(type) || !kv_head_dim_ok(head_dim) || !kv_page_size_ok(page_size)) return 0;
    if (n_kv_heads < 1 || n_kv_heads > 65535) return 0;
    return (size_t)n_kv_heads * (size_t)kv_head_bytes(type, head_dim, page_size);
}

qmv_status qmv_kv_append(const qmv_kv_cache *cache, int64_t n, const int32_t *start,
                         const float *k, int64_t ldk, const float *v, int64_t ldv,
                         hipStream_t stream) {
    KvArgs c;
    qmv_status st = check_cache(cache, c);
    if (st != QMV_OK) return st;
    st = check_rows(cache, n, start);
    if (st != QMV_OK) return st;
    const int64_t w = (int64_t)c.n_kv * c.hd;
    if (ldk < w || ldv < w || ldk > (1ll << 40) || ldv > (1ll << 40)) return QMV_ESHAPE;
    if (!k || !v) return QMV_EINVAL;
    if (!aligned(k, 4) || !aligned(v, 4)) return QMV_EALIGN;
    return from_hip(launch_kv_append(cache->type, c, n, start, k, ldk, v, ldv, stream));
}

// Heads, window and length of an attention call; the window is dropped where
// it covers every length.
static qmv_status check_attn(const qmv_kv_cache *c, int32_t n_heads, int64_t max_len,
                             int32_t &window, int32_t &sinks, int32_t *limit) {
    if (n_heads < 1 || n_heads > 65535 || n_heads % c->n_kv_heads != 0) return QMV_ESHAPE;
    if (max_len < 1 || max_len > c->table_ld * c->page_size) return QMV_ESHAPE;
    if (window < 0 || sinks < 0) return QMV_ESHAPE;
    if (window >= max_len) window = 0;
    if (sinks > max_len) sinks = (int32_t)max_len;
    *limit = (int32_t)max_len;
    return QMV_OK;
}

static void fill_attn(AttnArgs &a, const AttnPlan &p, float scale, void *ws) {
    // the kernels want a positive factor; the sign goes to the queries
    const float f = (scale < 0.f ? -scale : scale) * kLog2e;
    a.scale_log2 = scale == 0.f ? 1.f : f;
    a.q_sign = scale == 0.f ? 0.f : scale < 0.f ? -1.f : 1.f;
    // `limit` probabilities of at most 2^(bias + kSlack): less than 1 in all
    a.bias = -1.f - kSlack - (32 - __builtin_clz((unsigned)a.limit));
    a.unit = ldexpf(1.f, (int)(a.bias - kBias));
    a.group = a.n_heads / a.c.n_kv;
    a.tiles = p.tiles;
    a.splits = p.splits;
    a.parts = p.parts;
    a.part_rows = p.part_rows;
    a.part_ml = (float2 *)((uint8_t *)ws + p.ml_off);
    a.part_o = (float *)((uint8_t *)ws + p.o_off);
}

static qmv_status decode_plan(const qmv_kv_cache *c, int32_t n, int32_t n_heads, int64_t max_len,
                              int32_t &window, int32_t &sinks, bool with_acc, int32_t *limit,
                              AttnPlan &p) {
    qmv_status st = check_attn(c, n_heads, max_len, window, sinks, limit);
    if (st != QMV_OK) return st;
    if (n < 1 || n > QMV_MAX_ATTN_N) return QMV_ESHAPE;
    if (c->n_seq * n * n_heads > 0x7FFFFFFFll) return QMV_ESHAPE;
    p = attn_decode_plan(c->type, c->head_dim, c->n_seq, c->n_kv_heads, n_heads / c->n_kv_heads, n,
                         max_len, window, sinks, with_acc);
    if ((int64_t)p.tiles * c->n_kv_heads > 65535) return QMV_ESHAPE;
    // the joining launch takes a workgroup of 256 threads a row, and for the
    // weights one for every 256 positions of a key-value head
    int64_t blocks = p.slots > c->n_seq || with_acc ? p.part_rows : 0;
    if (with_acc) blocks += c->n_seq * c->n_kv_heads * ((max_len + 255) / 256);
    if (blocks >= (1ll << 24)) return QMV_ESHAPE;
    return QMV_OK;
}

size_t qmv_attn_decode_workspace(const qmv_kv_cache *cache, int32_t n, int32_t n_heads,
                                 int64_t max_len, int32_t window, int32_t sinks, int32_t with_acc) {
    AttnPlan p;
    int32_t limit;
    if (check_cache_shape(cache) != QMV_OK) return 0;
    if (decode_plan(cache, n, n_heads, max_len, window, sinks, with_acc != 0, &limit, p) != QMV_OK) return 0;
    return p.bytes;
}

qmv_status qmv_attn_decode(const qmv_kv_cache *cache, int32_t n, int32_t n_heads, const float *q,
                           int64_t ldq, float scale, int32_t window, int32_t sinks, float *out,
                           int64_t max_len, float *acc, int64_t ld_acc, void *workspace,
                           size_t ws_bytes, hipStream_t stream) {
    AttnArgs a{};
    AttnPlan p;
    qmv_status st = check_cache(cache, a.c);
    if (st != QMV_OK) return st;
    st = decode_plan(cache, n, n_heads, max_len, window, sinks, acc != nullptr, &a.limit, p);
    if (st != QMV_OK) return st;
    if (ldq < (int64_t)n_heads * a.c.hd || ldq > (1ll << 40)) return QMV_ESHAPE;
    if (acc && ld_acc < max_len) return QMV_ESHAPE;
    if (!q || !out) return QMV_EINVAL;
    if (!aligned(q, 4) || !aligned(out, 4) || !aligned(acc, 4)) return QMV_EALIGN;
    if (p.bytes > 0 && (!workspace || ws_bytes < p.bytes)) return QMV_EWORKSPACE;
    if (p.bytes > 0 && !aligned(workspace, 16)) return QMV_EALIGN;
    a.n = n;
    a.rows = cache->n_seq * n;
    a.q = q;
    a.ldq = ldq;
    a.out = out;
    a.n_heads = n_heads;
    a.window = window;
    a.sinks = sinks;
    fill_attn(a, p, scale, workspace);
    a.share = (int2 *)((uint8_t *)workspace + p.share_off);
    a.logits = (float *)((uint8_t *)workspace + p.logits_off);
    a.ld_logits = p.ld_logits;
    a.acc = acc;
    a.ld_acc = ld_acc;
    return from_hip(launch_attn_decode(cache->type, a, p, stream));
}

static qmv_status prefill_plan(const qmv_kv_cache *c, int64_t n, int32_t n_heads, int64_t max_len,
                               int32_t &window, int32_t &sinks, int32_t *limit, AttnPlan &p) {
    qmv_status st = check_attn(c, n_heads, max_len, window, sinks, limit);
    if (st != QMV_OK) return st;
    if (n < 1 || n > QMV_MAX_KV_ROWS || n > 0x7FFFFFFFll / n_heads) return QMV_ESHAPE;
    p = attn_prefill_plan(c->type, c->head_dim, c->n_seq, c->n_kv_heads, n_heads / c->n_kv_heads, n,
                          max_len, window, sinks);
    if (p.tiles > 65535) return QMV_ESHAPE;
    return QMV_OK;
}

size_t qmv_attn_prefill_workspace(const qmv_kv_cache *cache, int64_t n, int32_t n_heads,
                                  int64_t max_len, int32_t window, int32_t sinks) {
    AttnPlan p;
    int32_t limit;
    if (check_cache_shape(cache) != QMV_OK) return 0;
    if (prefill_plan(cache, n, n_heads, max_len, window, sinks, &limit, p) != QMV_OK) return 0;
    return p.bytes;
}

qmv_status qmv_attn_prefill(const qmv_kv_cache *cache, int64_t n, const int32_t *start,
                            int32_t n_heads, const float *q, int64_t ldq, float scale,
                            int32_t window, int32_t sinks, float *out, int64_t max_len,
                            void *workspace, size_t ws_bytes, hipStream_t stream) {
    AttnArgs a{};
    AttnPlan p;
    qmv_status st = check_cache(cache, a.c);
    if (st != QMV_OK) return st;
    st = check_rows(cache, n, start);
    if (st != QMV_OK) return st;
    st = prefill_plan(cache, n, n_heads, max_len, window, sinks, &a.limit, p);
    if (st != QMV_OK) return st;
    if (ldq < (int64_t)n_heads * a.c.hd || ldq > (1ll << 40)) return QMV_ESHAPE;
    if (!q || !out) return QMV_EINVAL;
    if (!aligned(q, 4) || !aligned(out, 4)) return QMV_EALIGN;
    if (p.bytes > 0 && (!workspace || ws_bytes < p.bytes)) return QMV_EWORKSPACE;
    if (p.bytes > 0 && !aligned(workspace, 16)) return QMV_EALIGN;
    a.start = start;
    a.n = start ? 0 : n / cache->n_seq;
    a.rows = n;
    a.q = q;
    a.ldq = ldq;
    a.out = out;
    a.n_heads = n_heads;
    a.window = window;
    a.sinks = sinks;
    fill_attn(a, p, scale, workspace);
    return from_hip(launch_attn_prefill(cache->type, a, p, stream));
}

qmv_status qmv_kv_evict(const qmv_kv_cache *cache, const int32_t *dst_table, int64_t dst_ld,
                        int32_t keep, int32_t first, int32_t recent, const float *acc,
                        int64_t ld_acc, int32_t *kept, float *acc_out, int64_t ld_out,
                        int32_t *len_out, hipStream_t stream) {
    KvArgs c;
    qmv_status st = check_cache(cache, c);
    if (st != QMV_OK) return st;
    if (!dst_table || !acc || !kept || !acc_out || !len_out) return QMV_EINVAL;
    if (dst_ld < 1 || dst_ld > (1ll << 30) / cache->page_size) return QMV_ESHAPE;
    if (keep < 1 || keep > dst_ld * cache->page_size) return QMV_ESHAPE;
    if (keep > (1 << 30) - 64) return QMV_ESHAPE;  // 2^24 workgroups of 256 threads are one too many
    if (first < 0 || recent < 0 || (int64_t)first + recent > keep) return QMV_ESHAPE;
    if (ld_acc < 1 || ld_acc > (1ll << 40) || ld_out < keep || ld_out > (1ll << 40)) return QMV_ESHAPE;
    if (!aligned(dst_table, 4) || !aligned(acc, 4) || !aligned(kept, 4) || !aligned(acc_out, 4) || !aligned(len_out, 4))
        return QMV_EALIGN;
    EvictArgs e{};
    e.dst = dst_table;
    e.dst_ld = dst_ld;
    e.keep = keep;
    e.first = first;
    e.recent = recent;
    e.limit = ld_acc < c.cap ? (int32_t)ld_acc : c.cap;
    e.acc = acc;
    e.ld_acc = ld_acc;
    e.kept = kept;
    e.acc_out = acc_out;
    e.ld_out = ld_out;
    e.len_out = len_out;
    return from_hip(launch_kv_evict(cache->type, c, e, stream));
}

}  // extern "C"
