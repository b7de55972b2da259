// Host-side driver for a sanitizer build of the calls around a cache's
// attention (qmv_serve_api.cpp) and of the plans and checks of calls over
// 4-bit caches, which attn_sanitize_driver.cpp's stubs and sweep serve as well.
// The stubs here check what reaches the launches: grids and sums that they
// take.  tests/test_serve_sanitizers.py builds and runs it; device pointers are
// fake addresses that nothing dereferences.
#define main attention_main
#include "attn_sanitize_driver.cpp"
#undef main

#include <math.h>

#include "qmv_pages.h"
#include "qmv_rope.h"

static long g_rope = 0, g_pages = 0;

namespace qmv {
static void rows_fit(int64_t n, int64_t per, int64_t y) {  // workgroups of 256 threads take `per` rows
    EXPECT(n >= 1 && (n + per - 1) / per * 256 < (1ll << 32) && y >= 1 && y <= 65535);
}
static void rope_fits(const RopeArgs &r, int hd) {
    EXPECT(r.rot >= 0 && r.rot <= hd && r.rot % 8 == 0 && (r.rot == 0 || r.freq) && r.eps >= 0.f);
    g_rope++;
}

hipError_t launch_kv_read(int, const KvArgs &c, int64_t n, const int32_t *, float *, int64_t ldk, float *, int64_t ldv,
                          hipStream_t) {
    rows_fit(n, 32, c.n_kv);
    EXPECT(ldk >= (int64_t)c.n_kv * c.hd && ldv >= (int64_t)c.n_kv * c.hd);
    return hipSuccess;
}

hipError_t launch_qk_norm_rope(const RopeArgs &r, int hd, int64_t n, const int32_t *, const HeadRows &q,
                               const HeadRows &k, hipStream_t) {
    rope_fits(r, hd);
    rows_fit(n, 16, (int64_t)q.heads + k.heads);
    EXPECT(q.heads >= 0 && k.heads >= 0 && (q.heads == 0 || q.ld_in >= (int64_t)q.heads * hd));
    return hipSuccess;
}

hipError_t launch_kv_append_rope(int, const KvArgs &c, const RopeArgs &r, int64_t n, const int32_t *, const HeadRows &q,
                                 const float *, int64_t, const float *, int64_t, hipStream_t) {
    rope_fits(r, c.hd);
    rows_fit(n, 16, (int64_t)c.n_kv + q.heads);
    return hipSuccess;
}

hipError_t launch_kv_reserve(const KvArgs &c, int32_t *, int32_t *, const ReserveArgs &a, int32_t *, int64_t *,
                             hipStream_t) {
    // what a sequence can be given, and all rows, stay below the sums' end (2^30)
    EXPECT(a.n >= 1 && a.n <= QMV_MAX_KV_ROWS && c.cap >= 16 && c.cap <= 1 << 30 && c.n_seq >= 1 && c.n_seq <= 65535);
    g_pages++;
    return hipSuccess;
}

hipError_t launch_kv_release(const KvArgs &c, int32_t *, int32_t *, const int32_t *, int32_t *, int32_t *, hipStream_t) {
    EXPECT(c.n_seq * c.table_ld <= 1ll << 30);
    g_pages++;
    return hipSuccess;
}
}  // namespace qmv

static void serve(const qmv_kv_cache &c, int64_t n, int32_t heads) {
    float *x = (float *)(uintptr_t)(1 << 20), *y = (float *)(uintptr_t)(2 << 20);
    int32_t *i = (int32_t *)(uintptr_t)(1 << 20);
    const int64_t w = (int64_t)c.n_kv_heads * c.head_dim, wq = (int64_t)heads * c.head_dim;
    const qmv_qk_rope r = {(const double *)x, (int32_t)(rnd() % (c.head_dim / 8 + 1) * 8), (int32_t)(rnd() % 2),
                           rnd() % 2 ? x : nullptr, rnd() % 2 ? x : nullptr, 1e-5f};
    for (int use = 0; use < 2; use++) {
        const int64_t rows = use ? n : (n + c.n_seq - 1) / c.n_seq * c.n_seq;
        qmv_status st = qmv_kv_read(&c, rows, use ? i : nullptr, x, w, y, w, nullptr);
        EXPECT(st == QMV_OK || st == QMV_ESHAPE);
        st = qmv_kv_append_rope(&c, &r, rows, use ? i : nullptr, heads, x, wq, use ? x : y, wq, x, w, x, w, nullptr);
        EXPECT(st == QMV_OK || st == QMV_ESHAPE);
    }
    qmv_status st = qmv_qk_norm_rope(&r, c.head_dim, n, i, heads, x, wq, y, wq, rnd() % 2 ? c.n_kv_heads : 0, x, w, y, w, nullptr);
    EXPECT(st == QMV_OK || st == QMV_ESHAPE);
    st = qmv_kv_reserve(&c, i, i, i, n, i, i, rnd() % 2 ? i : nullptr, rnd() % 2 ? (int64_t *)x : nullptr, nullptr);
    EXPECT(st == QMV_OK || st == QMV_ESHAPE);
    st = qmv_kv_release(&c, i, i, i, nullptr);
    EXPECT(st == QMV_OK || st == QMV_ESHAPE);
}

int main() {
    const int hds[] = {64, 96, 128, 256};
    qmv_kv_cache c{};
    c.type = QMV_KV_Q4;
    c.pages = (void *)(uintptr_t)(1 << 20);
    c.table = (const int32_t *)(uintptr_t)(1 << 20);
    c.seq_len = (const int32_t *)(uintptr_t)(1 << 20);
    c.n_pages = 1;
    for (int i = 0; i < 300000; i++) {
        c.head_dim = hds[rnd() % 4];
        c.page_size = 16 << (rnd() % 9);
        c.n_seq = spread(1, 65535);
        c.n_kv_heads = (int)spread(1, rnd() % 4 ? 32 : 65535);
        c.table_ld = spread(1, (1ll << 30) / c.page_size);
        const int64_t len = spread(1, c.table_ld * c.page_size), n = spread(1, rnd() % 2 ? 16 : QMV_MAX_KV_ROWS);
        const int group = (int)spread(1, rnd() % 4 ? 16 : 65535);
        if ((int64_t)c.n_kv_heads * group > 65535) continue;
        calls(c, n, c.n_kv_heads * group, len, rnd() % 2 ? 0 : (int32_t)spread(1, 0x7FFFFFFF),
              rnd() % 2 ? 0 : (int32_t)spread(1, 0x7FFFFFFF));
        serve(c, n, c.n_kv_heads * group);
    }
    EXPECT(g_split > 5000 && g_ranges > 5000 && g_acc > 5000 && g_rope > 50000 && g_pages > 50000);
    // refusals at the ends of the numbers
    c.head_dim = 64, c.n_seq = 2, c.n_kv_heads = 2, c.page_size = 16, c.table_ld = 4;
    float *x = (float *)(uintptr_t)(1 << 20), *y = (float *)(uintptr_t)(2 << 20);
    int32_t *i = (int32_t *)x;
    qmv_qk_rope r = {(const double *)x, 64, QMV_ROPE_HALVES, nullptr, nullptr, 0.f};
    EXPECT(qmv_kv_read(nullptr, 2, nullptr, x, 128, y, 128, nullptr) == QMV_EINVAL);
    EXPECT(qmv_kv_read(&c, INT64_MAX, nullptr, x, 128, y, 128, nullptr) == QMV_ESHAPE);
    EXPECT(qmv_kv_read(&c, 2, nullptr, x, INT64_MAX, y, 128, nullptr) == QMV_ESHAPE);
    EXPECT(qmv_qk_norm_rope(&r, 64, 2, i, INT32_MAX, x, INT64_MAX, y, INT64_MAX, 0, x, 0, y, 0, nullptr) == QMV_ESHAPE);
    EXPECT(qmv_qk_norm_rope(&r, 64, 2, i, INT32_MIN, x, 64, y, 64, 0, x, 0, y, 0, nullptr) == QMV_ESHAPE);
    EXPECT(qmv_qk_norm_rope(&r, 64, INT64_MIN, i, 1, x, 64, y, 64, 0, x, 0, y, 0, nullptr) == QMV_ESHAPE);
    EXPECT(qmv_qk_norm_rope(&r, 64, 2, i, 0, nullptr, 0, nullptr, 0, 0, nullptr, 0, nullptr, 0, nullptr) == QMV_ESHAPE);
    r.rot_dim = INT32_MIN;
    EXPECT(qmv_qk_norm_rope(&r, 64, 2, i, 1, x, 64, y, 64, 0, x, 0, y, 0, nullptr) == QMV_ESHAPE);
    r.rot_dim = 64, r.eps = NAN;
    EXPECT(qmv_kv_append_rope(&c, &r, 2, nullptr, 1, x, 64, y, 64, x, 128, x, 128, nullptr) == QMV_EINVAL);
    r.eps = -1.f;
    EXPECT(qmv_kv_append_rope(&c, &r, 2, nullptr, 1, x, 64, y, 64, x, 128, x, 128, nullptr) == QMV_EINVAL);
    EXPECT(qmv_kv_append_rope(&c, nullptr, 2, nullptr, 1, x, 64, y, 64, x, 128, x, 128, nullptr) == QMV_EINVAL);
    EXPECT(qmv_kv_reserve(&c, i, i, i, INT64_MAX, i, i, nullptr, nullptr, nullptr) == QMV_ESHAPE);
    c.table_ld = INT64_MAX;
    EXPECT(qmv_kv_release(&c, i, i, i, nullptr) == QMV_ESHAPE);
    if (g_fail) {
        fprintf(stderr, "%d expectations failed\n", g_fail);
        return 1;
    }
    printf("sanitized host layer around the attention: ok (%ld attention launches, %ld rotations, %ld of pages)\n", g_calls,
           g_rope, g_pages);
    return 0;
}
