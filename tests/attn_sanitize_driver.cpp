// Host-side driver for a sanitizer build of the cache and attention calls'
// host layer (qmv_attn_api.cpp: argument checks; qmv_attn_plan.cpp: how calls
// are cut, what their workspaces hold).  The launch functions are stubs that
// check what reaches them, over the corners of every argument and a sweep of
// random ones: pieces that the join takes, grids that a launch takes, every
// part of the workspace inside the bytes that the caller was told, none
// overlapping another.  tests/test_oracle_sanitizers.py builds and runs it;
// device pointers here are fake addresses that nothing dereferences.
#include <stdio.h>

#include "qmv.h"
#include "qmv_attn_plan.h"
#include "qmv_internal.h"

static int g_fail = 0;
static long g_calls = 0, g_split = 0, g_ranges = 0, g_acc = 0;
static size_t g_need = 0;  // bytes the caller was told
#define EXPECT(cond)                                                        \
    do {                                                                    \
        if (!(cond)) {                                                      \
            if (g_fail++ < 20)                                              \
                fprintf(stderr, "%s:%d: expectation failed: %s\n", __FILE__, \
                        __LINE__, #cond);                                   \
        }                                                                   \
    } while (0)

static uint8_t *const kWs = (uint8_t *)(uintptr_t)(1ull << 40);

namespace qmv {
void set_last_hip_error(hipError_t) {}

hipError_t launch_kv_append(int, const KvArgs &c, int64_t n, const int32_t *, const float *, int64_t, const float *,
                            int64_t, hipStream_t) {
    g_calls++;
    EXPECT(c.cap > 0 && (1 << c.page_shift) >= 16 && (n + 15) / 16 < (1ll << 24));
    return hipSuccess;
}

hipError_t launch_kv_evict(int, const KvArgs &c, const EvictArgs &e, hipStream_t) {
    g_calls++;
    EXPECT(((int64_t)e.keep + 63) / 64 * 256 < (1ll << 32) && e.limit >= 1 && e.limit <= c.cap);
    return hipSuccess;
}

// [off, off + bytes) of the workspace, behind `at`; returns its end.
static size_t region(size_t at, size_t off, size_t bytes) {
    EXPECT(off >= at && off % 16 == 0 && off + bytes >= off && off + bytes <= g_need);
    return off + bytes;
}

hipError_t launch_attn_decode(int type, const AttnArgs &a, const AttnPlan &p, hipStream_t) {
    g_calls++;
    const KvArgs &c = a.c;
    const int64_t rows = a.n * a.group, pieces = (int64_t)p.slots * a.n * a.n_heads;
    EXPECT(p.bytes == g_need && (p.rt == 1 || (p.rt == 2 && c.hd <= 128)) && (p.waves == 4 || p.waves == 8));
    EXPECT((int64_t)p.tiles * 16 * p.rt >= rows && ((int64_t)p.tiles - 1) * 16 * p.rt < rows);
    EXPECT((int64_t)p.tiles * c.n_kv <= 65535 && c.n_seq <= 65535);
    EXPECT(p.part_rows == c.n_seq * rows * c.n_kv && a.part_rows == p.part_rows);
    // every sequence's pieces are at most what the join takes, and have slots of their own
    EXPECT(p.splits >= 1 && p.splits <= kMaxPieces && p.parts >= 0 && p.parts <= kMaxPieces);
    EXPECT(p.parts ? p.slots >= p.parts + c.n_seq - 1 : p.slots == c.n_seq * p.splits);
    const int ck = decode_chunk(type);
    if (p.parts) {  // units are counted in 32 bits; 16-row tiles of eight waves do not take ranges
        // a sequence's: 4 for entering, and the chunks that hold its visible
        // positions, of which two runs (sinks, window) begin and end inside one
        const int64_t seen = a.window > 0 ? (int64_t)a.window + a.n + a.sinks : a.limit;
        const int64_t most = seen < a.limit ? seen : a.limit;
        EXPECT((most / ck + 4 + 4) * c.n_seq < 0x7FFFFFFFll && (p.rt == 2 || p.waves == 4));
        g_ranges++;
    }
    if (p.waves == 8) EXPECT(eight_fit(type, c.hd, p.rt));
    const bool joins = a.acc || p.slots > c.n_seq;
    EXPECT(joins || p.bytes == 0);
    if (joins) {
        EXPECT((uint8_t *)a.part_ml == kWs + p.ml_off && (uint8_t *)a.part_o == kWs + p.o_off);
        EXPECT((uint8_t *)a.share == kWs + p.share_off && (uint8_t *)a.logits == kWs + p.logits_off);
        size_t at = region(0, p.ml_off, sizeof(float2) * (size_t)pieces);
        at = region(at, p.o_off, sizeof(float) * (size_t)pieces * c.hd);
        at = region(at, p.share_off, sizeof(int2) * (size_t)c.n_seq);
        if (a.acc) {
            // whole chunks of logits are written
            EXPECT(p.ld_logits >= (int64_t)(a.limit + ck - 1) / ck * ck && p.ld_logits % 4 == 0);
            region(at, p.logits_off, sizeof(float) * (size_t)p.part_rows * (size_t)p.ld_logits);
            const int64_t blocks = p.part_rows + (int64_t)c.n_seq * c.n_kv * (((int64_t)a.limit + 255) / 256);
            EXPECT(blocks * 256 < (1ll << 32));
            g_acc++;
        } else {
            EXPECT(a.n * a.n_heads * 256 < (1ll << 32));
        }
        g_split++;
    }
    EXPECT(a.window >= 0 && a.window < a.limit && a.sinks >= 0 && a.sinks <= a.limit);
    EXPECT(a.bias <= -6.f && a.bias >= -36.f && a.unit > 0.f && a.scale_log2 >= 0.f);
    return hipSuccess;
}

hipError_t launch_attn_prefill(int, const AttnArgs &a, const AttnPlan &p, hipStream_t) {
    g_calls++;
    const KvArgs &c = a.c;
    EXPECT(p.bytes == g_need && p.splits >= 1 && p.splits <= kMaxPieces && p.tiles <= 65535);
    // a row tile for every 128 rows of a sequence
    const int64_t each = a.start ? 0 : (a.n * a.group + kBM - 1) / kBM;
    EXPECT(a.start || c.n_seq * each <= p.tiles);
    EXPECT((a.rows * a.group + kBM - 1) / kBM + (a.start ? c.n_seq : 0) <= p.tiles);
    EXPECT(p.part_rows == a.rows * a.n_heads && p.part_rows <= 0x7FFFFFFFll);
    if (p.splits > 1) {
        const size_t pieces = (size_t)p.splits * p.part_rows;
        size_t at = region(0, p.ml_off, sizeof(float2) * pieces);
        region(at, p.o_off, sizeof(float) * pieces * c.hd);
        EXPECT((uint8_t *)a.part_ml == kWs + p.ml_off && (uint8_t *)a.part_o == kWs + p.o_off);
        EXPECT(p.part_rows * 256 < (1ll << 32));
        g_split++;
    } else {
        EXPECT(p.bytes == 0);
    }
    return hipSuccess;
}
}  // namespace qmv

static uint64_t g_state = 12345;
static uint32_t rnd() {
    g_state = g_state * 6364136223846793005ull + 1442695040888963407ull;
    return (uint32_t)(g_state >> 33);
}
// spread over the magnitudes of lo .. hi
static int64_t spread(int64_t lo, int64_t hi) {
    int bits = 0;
    while ((hi >> bits) > 1) bits++;
    const int b = rnd() % (bits + 1);
    const int64_t v = (1ll << b) + (int64_t)(((uint64_t)rnd() << 16 | (rnd() & 0xFFFF)) & ((1ull << b) - 1));
    return v < lo ? lo : v > hi ? hi : v;
}

static void calls(const qmv_kv_cache &c, int64_t n, int32_t heads, int64_t max_len, int32_t window, int32_t sinks) {
    float *x = (float *)(uintptr_t)(1 << 20);
    int32_t *start = (int32_t *)(uintptr_t)(1 << 20);
    const int64_t ld = (int64_t)heads * c.head_dim;
    const int nd = (int)(n < QMV_MAX_ATTN_N ? n : QMV_MAX_ATTN_N);
    for (int acc = 0; acc < 2; acc++) {
        g_need = qmv_attn_decode_workspace(&c, nd, heads, max_len, window, sinks, acc);
        qmv_status st = qmv_attn_decode(&c, nd, heads, x, ld, 0.125f, window, sinks, x, max_len, acc ? x : nullptr, max_len,
                                        g_need ? kWs : nullptr, g_need, nullptr);
        EXPECT(st == QMV_OK || (st == QMV_ESHAPE && g_need == 0));
        if (st == QMV_OK && g_need) {
            EXPECT(qmv_attn_decode(&c, nd, heads, x, ld, 0.125f, window, sinks, x, max_len, acc ? x : nullptr, max_len, kWs,
                                   g_need - 1, nullptr) == QMV_EWORKSPACE);
        }
    }
    for (int use = 0; use < 2; use++) {
        const int64_t rows = use ? n : (n + c.n_seq - 1) / c.n_seq * c.n_seq;
        g_need = qmv_attn_prefill_workspace(&c, rows, heads, max_len, window, sinks);
        qmv_status st = qmv_attn_prefill(&c, rows, use ? start : nullptr, heads, x, ld, -0.125f, window, sinks, x, max_len,
                                         g_need ? kWs : nullptr, g_need, nullptr);
        EXPECT(st == QMV_OK || st == QMV_ESHAPE);
        const int64_t w = (int64_t)c.n_kv_heads * c.head_dim;
        st = qmv_kv_append(&c, rows, use ? start : nullptr, x, w, x, w, nullptr);
        EXPECT(st == QMV_OK || st == QMV_ESHAPE);
    }
    const int64_t ldp = c.table_ld;
    const int32_t keep = (int32_t)spread(1, ldp * c.page_size);
    qmv_status st = qmv_kv_evict(&c, start, ldp, keep, keep / 3, keep / 3, x, max_len, start, x, keep, start, nullptr);
    EXPECT(st == QMV_OK || st == QMV_ESHAPE);
}

int main() {
    const int types[] = {QMV_KV_F16, QMV_KV_I8, QMV_KV_BF16}, hds[] = {64, 96, 128, 256};
    qmv_kv_cache c{};
    c.pages = (void *)(uintptr_t)(1 << 20);
    c.table = (const int32_t *)(uintptr_t)(1 << 20);
    c.seq_len = (const int32_t *)(uintptr_t)(1 << 20);
    c.n_pages = 1;
    const int64_t seqs[] = {1, 2, 3, 7, 64, 1024, 1025, 65535}, ns[] = {1, 2, 16, 17, 4096, QMV_MAX_KV_ROWS};
    const int64_t lens[] = {1, 33, 4352, 131072, 1ll << 30};
    const int kvs[] = {1, 3, 8, 65535}, groups[] = {1, 4, 17};
    for (int t : types)
        for (int hd : hds)
            for (int64_t s : seqs)
                for (int kv : kvs)
                    for (int g : groups)
                        for (int64_t n : ns)
                            for (int64_t len : lens) {
                                c.type = t, c.head_dim = hd, c.n_seq = s, c.n_kv_heads = kv;
                                c.page_size = len > 4096 ? 4096 : 16;
                                c.table_ld = (len + c.page_size - 1) / c.page_size;
                                if ((int64_t)kv * g > 65535) continue;
                                calls(c, n, kv * g, len, 0, 0);
                            }
    for (int i = 0; i < 300000; i++) {
        c.type = types[rnd() % 3];
        c.head_dim = hds[rnd() % 4];
        c.page_size = 16 << (rnd() % 9);
        c.n_seq = spread(1, 65535);
        c.n_kv_heads = (int)spread(1, rnd() % 4 ? 32 : 65535);
        c.table_ld = spread(1, (1ll << 30) / c.page_size);
        const int64_t len = spread(1, c.table_ld * c.page_size);
        const int group = (int)spread(1, rnd() % 4 ? 16 : 65535);
        if ((int64_t)c.n_kv_heads * group > 65535) continue;
        calls(c, spread(1, rnd() % 2 ? 16 : QMV_MAX_KV_ROWS), c.n_kv_heads * group, len,
              rnd() % 2 ? 0 : (int32_t)spread(1, 0x7FFFFFFF), rnd() % 2 ? 0 : (int32_t)spread(1, 0x7FFFFFFF));
    }
    EXPECT(g_split > 10000 && g_ranges > 10000 && g_acc > 10000);
    // refusals
    c.type = QMV_KV_F16, c.head_dim = 64, c.n_seq = 2, c.n_kv_heads = 2, c.page_size = 16, c.table_ld = 4;
    float *x = (float *)(uintptr_t)(1 << 20);
    EXPECT(qmv_kv_append(nullptr, 2, nullptr, x, 128, x, 128, nullptr) == QMV_EINVAL);
    EXPECT(qmv_kv_append(&c, 2, nullptr, x, 127, x, 128, nullptr) == QMV_ESHAPE);
    EXPECT(qmv_kv_append(&c, 2, nullptr, x, INT64_MAX, x, 128, nullptr) == QMV_ESHAPE);
    EXPECT(qmv_attn_decode(&c, 1, 4, x, 256, 0.1f, INT32_MAX, INT32_MAX, x, 64, nullptr, 0, nullptr, 0, nullptr) == QMV_OK);
    EXPECT(qmv_attn_decode(&c, INT32_MIN, 4, x, 256, 0.1f, 0, 0, x, 64, nullptr, 0, nullptr, 0, nullptr) == QMV_ESHAPE);
    EXPECT(qmv_attn_decode(&c, 1, 4, x, 256, 0.1f, 0, 0, x, INT64_MAX, nullptr, 0, nullptr, 0, nullptr) == QMV_ESHAPE);
    EXPECT(qmv_attn_prefill(&c, INT64_MAX - 1, nullptr, 4, x, 256, 0.1f, 0, 0, x, 64, nullptr, 0, nullptr) == QMV_ESHAPE);
    EXPECT(qmv_attn_prefill_workspace(&c, INT64_MIN, 4, 64, 0, 0) == 0);
    EXPECT(qmv_kv_evict(&c, (int32_t *)x, 4, 64, INT32_MAX, INT32_MAX, x, 64, (int32_t *)x, x, 64, (int32_t *)x, nullptr) ==
           QMV_ESHAPE);
    c.table_ld = INT64_MAX;
    EXPECT(qmv_attn_decode_workspace(&c, 1, 4, 64, 0, 0, 1) == 0);
    c.table_ld = 4, c.n_pages = INT64_MAX;
    EXPECT(qmv_attn_decode_workspace(&c, 1, 4, 64, 0, 0, 1) == 0);
    EXPECT(qmv_kv_page_bytes(QMV_KV_F16, INT32_MAX, 256, 4096) == 0);
    if (g_fail) {
        fprintf(stderr, "%d expectations failed\n", g_fail);
        return 1;
    }
    printf("sanitized attention host layer: ok (%ld launches, %ld joined, %ld of even ranges, %ld with weights)\n", g_calls,
           g_split, g_ranges, g_acc);
    return 0;
}
