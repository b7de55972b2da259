// The paged key-value cache: its layout, shared by the append, attention and
// eviction kernels (the layout is described in include/qmv.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace qmv {

enum { kKvF16 = 1, kKvI8 = 24, kKvBF16 = 30 };

inline bool kv_type_ok(int t) { return t == kKvF16 || t == kKvBF16 || t == kKvI8; }
inline bool kv_head_dim_ok(int hd) { return hd == 64 || hd == 96 || hd == 128 || hd == 256; }

inline bool kv_page_size_ok(int p) { return p >= 16 && p <= 4096 && (p & (p - 1)) == 0; }

constexpr int kVBlock = 16;  // positions of one V block

// Bytes of one head's part of a page: K rows, V blocks, 8-bit row scales.
__host__ __device__ inline int64_t kv_head_bytes(int type, int hd, int page_size) {
    return type == kKvI8 ? 2ll * page_size * hd + 8ll * page_size : 4ll * page_size * hd;
}

// A cache as the kernels take it.
struct KvArgs {
    uint8_t *pages;
    const int32_t *table;
    const int32_t *seq_len;
    int64_t table_ld;    // table entries per sequence
    int64_t head_bytes;  // bytes of one head's part of a page
    int32_t n_pages;
    int32_t n_seq;
    int32_t n_kv;
    int32_t hd;
    int32_t page_shift;  // log2(page_size)
    int32_t cap;         // positions a table row can address
};

// Length of sequence s, whatever the array holds: 0 .. limit.
__device__ __forceinline__ int kv_len(const KvArgs &c, int s, int limit) {
    const int len = c.seq_len[s];
    return len < 0 ? 0 : len > limit ? limit : len;
}

// Page of position pos (0 <= pos < cap) of sequence s; -1 if the entry is a hole.
__device__ __forceinline__ int kv_page(const KvArgs &c, int s, int pos) {
    const int pg = c.table[(int64_t)s * c.table_ld + (pos >> c.page_shift)];
    return (uint32_t)pg < (uint32_t)c.n_pages ? pg : -1;
}

__device__ __forceinline__ uint8_t *kv_head(const KvArgs &c, int page, int h) {
    return c.pages + ((int64_t)page * c.n_kv + h) * c.head_bytes;
}

hipError_t launch_kv_append(int type, const KvArgs &c, int64_t n, const int32_t *start,
                            const float *k, int64_t ldk, const float *v, int64_t ldv,
                            hipStream_t s);

struct EvictArgs {
    const int32_t *dst;
    int64_t dst_ld;
    int32_t keep, first, recent;
    int32_t limit;       // longest sequence the scores cover
    const float *acc;
    int64_t ld_acc;
    int32_t *kept;
    float *acc_out;
    int64_t ld_out;
    int32_t *len_out;
};
hipError_t launch_kv_evict(int type, const KvArgs &c, const EvictArgs &e, hipStream_t s);

// One attention call over a cache.
struct AttnArgs {
    KvArgs c;
    const int32_t *start;  // first row of each sequence (prompts of different lengths), or null
    int64_t n;             // rows per sequence (start == null)
    int64_t rows;          // rows in all
    const float *q;
    int64_t ldq;
    float *out;
    int32_t n_heads, group;  // query heads, query heads per key-value head
    int32_t window, sinks;   // window 0: none
    int32_t limit;           // longest sequence (max_len, and what the table addresses)
    int32_t tiles, splits;   // splits: pieces of each sequence's length
    int32_t parts;           // decode, not 0: instead, workgroups of a head over all sequences
    float scale_log2;        // |scale| * log2(e), not zero
    float q_sign;            // what queries are multiplied by: the scale's sign (0 for scale 0)
    float bias;              // -(5 + bits of limit).  bf16: log2 of what probabilities are multiplied by;
                             // 8-bit: of what the sums that leave a wave are
    float unit;              // 8-bit: 2^(bias - kBias), from the probabilities' factor to that of the sums
    float2 *part_ml;         // running maximum and sum of each piece of an output row
    float *part_o;           // [hd] of each
    int64_t part_rows;       // rows * n_heads; prompts: piece i of output row r is at i * part_rows + r
    int2 *share;             // parts: first and last slot of each sequence; decode: the piece of a sequence's
                             // row r in a slot is at slot * n * n_heads + r
    float *logits;           // [n_seq][n_kv][n * group][ld_logits], base-2 logits (weights wanted)
    int64_t ld_logits;
    float *acc;              // [n_seq][n_kv][ld_acc]
    int64_t ld_acc;
};

struct AttnPlan;
hipError_t launch_attn_decode(int type, const AttnArgs &a, const AttnPlan &p, hipStream_t s);
hipError_t launch_attn_prefill(int type, const AttnArgs &a, const AttnPlan &p, hipStream_t s);

}  // namespace qmv
