// The pages of a cache kept on the GPU: a stack of free ones, from which
// sequences take what their next tokens need and to which they give back what
// lies behind a shorter length, so that a serving loop's steps follow each
// other without the host.
//
// Whole numbers and little of them: both calls are chains of latencies.  One
// workgroup does all of it (nothing waits for another one's sums), 1024
// sequences at a time: prefix sums say who gets what, then pages, and the rows
// of a call of few, are dealt out evenly, each thread finding the sequence of
// its first one by bisection of the sums in LDS.
#include "qmv_device.h"
#include "qmv_internal.h"
#include "qmv_pages.h"

namespace qmv {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kItems = 4;  // pages a thread takes at a time: their loads fly together
// Sums stop here, above any row or page count that a call can be given.
constexpr uint32_t kSat = 1u << 30;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return a + b < kSat ? a + b : kSat; }

struct Sums {
    uint32_t before, all;
};
// Prefix sum over the workgroup; `tmp` is the call's own.
__device__ __forceinline__ Sums block_sum(uint32_t x, uint32_t *tmp) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    uint32_t upto = x;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const uint32_t y = __shfl_up(upto, off);
        if (lane >= off) upto = sat_add(upto, y);
    }
    if (lane == 63) tmp[wave] = upto;
    uint32_t before = __shfl_up(upto, 1);
    if (lane == 0) before = 0;
    __syncthreads();
    uint32_t all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        if (w == wave) before = sat_add(all, before);
        all = sat_add(all, tmp[w]);
    }
    return Sums{before, all};
}

// The last of `n` entries whose sum before it is at most i: the one that i is in.
__device__ __forceinline__ int entry_of(const uint32_t *before, int n, uint32_t i) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (before[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ int clamped(int x, int most) { return x < 0 ? 0 : x > most ? most : x; }

__device__ __forceinline__ int64_t slot_of(const KvArgs &c, int page, int pos) {
    if ((uint32_t)page >= (uint32_t)c.n_pages) return -1;
    return ((int64_t)page << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

__global__ __launch_bounds__(kThreads) void kv_reserve(KvArgs c, int32_t *table, int32_t *seq_len, ReserveArgs a,
                                                       int32_t *pos, int64_t *slot) {
    __shared__ uint32_t s_tmp[4][kWaves], s_pages[kThreads], s_rows[kThreads];
    __shared__ int s_len[kThreads];
    const int tid = threadIdx.x, mask = (1 << c.page_shift) - 1;
    const int count = clamped(*a.free_count, c.n_pages);
    uint32_t need_all = 0, rows_all = 0;  // what was asked for so far
    int popped = 0, row0 = 0;             // what was given
    for (int base = 0; base < c.n_seq; base += kThreads) {
        const int s = base + tid, here = c.n_seq - base < kThreads ? c.n_seq - base : kThreads;
        const int len = tid < here ? seq_len[s] : 0, add = tid < here ? a.add[s] : 0;
        const bool fits = add > 0 && len >= 0 && (int64_t)len + add <= c.cap;
        // (for a length that does not fit the sums below may overflow, and are not used)
        const int first = (int)(((uint32_t)len + mask) >> c.page_shift);
        const int need = fits ? ((len + add + mask) >> c.page_shift) - first : 0, rows = fits ? add : 0;
        const Sums p = block_sum(need, s_tmp[0]), r = block_sum(rows, s_tmp[1]);
        const uint32_t p_upto = sat_add(sat_add(need_all, p.before), need), r_upto = sat_add(sat_add(rows_all, r.before), rows);
        const bool given = fits && r_upto <= (uint32_t)a.n && (need == 0 || (p_upto <= (uint32_t)count && p_upto < kSat));
        const Sums pg = block_sum(given ? need : 0, s_tmp[2]), rg = block_sum(given ? rows : 0, s_tmp[3]);
        s_pages[tid] = pg.before;
        s_rows[tid] = rg.before;
        s_len[tid] = len;
        if (tid < here) {
            a.granted[s] = given ? add : 0;
            a.start[s] = row0 + (int)rg.before;
            if (given) seq_len[s] = len + add;
        }
        __syncthreads();
        // the i-th page of these goes to its sequence
        for (uint32_t i = tid * kItems; i < pg.all; i += kThreads * kItems) {
            int32_t page[kItems];
#pragma unroll
            for (int j = 0; j < kItems; j++) page[j] = i + j < pg.all ? a.free_pages[count - 1 - popped - (int)i - j] : -1;
            int t = entry_of(s_pages, here, i);
#pragma unroll
            for (int j = 0; j < kItems; j++) {
                if (i + j >= pg.all) break;
                while (t + 1 < here && s_pages[t + 1] <= i + j) t++;
                const int at = ((s_len[t] + mask) >> c.page_shift) + (int)(i + j - s_pages[t]);
                table[(int64_t)(base + t) * c.table_ld + at] = page[j];
            }
        }
        if (pos || slot) {
            for (uint32_t i = tid; i < rg.all; i += kThreads) {
                const int t = entry_of(s_rows, here, i), at = s_len[t] + (int)(i - s_rows[t]);
                const int own = (s_len[t] + mask) >> c.page_shift, k = at >> c.page_shift;
                if (pos) pos[row0 + (int)i] = at;
                if (slot) {
                    const int page = k >= own ? a.free_pages[count - 1 - popped - (int)s_pages[t] - (k - own)]
                                              : table[(int64_t)(base + t) * c.table_ld + k];
                    slot[row0 + (int)i] = slot_of(c, page, at);
                }
            }
        }
        need_all = sat_add(need_all, p.all);
        rows_all = sat_add(rows_all, r.all);
        popped += (int)pg.all;
        row0 += (int)rg.all;
        __syncthreads();
    }
    if (pos || slot) {
        for (int i = row0 + tid; i < a.n; i += kThreads) {
            if (pos) pos[i] = -1;
            if (slot) slot[i] = -1;
        }
    }
    if (tid == 0) {
        a.start[c.n_seq] = row0;
        *a.free_count = count - popped;
    }
}

// Positions and slots of many rows, by the start, lengths and table that
// kv_reserve left.
__global__ __launch_bounds__(256) void kv_row_slots(KvArgs c, int n, const int32_t *start, int32_t *pos, int64_t *slot) {
    const int r = blockIdx.x * 256 + threadIdx.x;
    if (r >= n) return;
    int at = -1;
    int64_t to = -1;
    if (r < start[c.n_seq]) {
        int lo = 0, hi = c.n_seq;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (start[mid] <= r) lo = mid; else hi = mid;
        }
        at = c.seq_len[lo] - (start[lo + 1] - r);
        if (slot) to = slot_of(c, c.table[(int64_t)lo * c.table_ld + (at >> c.page_shift)], at);
    }
    if (pos) pos[r] = at;
    if (slot) slot[r] = to;
}

// From the last sequence to the first and from a sequence's last page to the
// first of those it gives back: taken again in the same order they would go to
// the same places.
__global__ __launch_bounds__(kThreads) void kv_release(KvArgs c, int32_t *table, int32_t *seq_len, const int32_t *new_len,
                                                       int32_t *free_pages, int32_t *free_count) {
    __shared__ uint32_t s_tmp[3][kWaves], s_before[kThreads];
    __shared__ int s_last[kThreads];
    const int tid = threadIdx.x, mask = (1 << c.page_shift) - 1;
    const int count = clamped(*free_count, c.n_pages);
    uint32_t pushed = 0;
    for (int base = (c.n_seq - 1) / kThreads * kThreads; base >= 0; base -= kThreads) {
        const int here = c.n_seq - base < kThreads ? c.n_seq - base : kThreads, s = base + here - 1 - tid;
        const int len = tid < here ? clamped(seq_len[s], c.cap) : 0, to = tid < here ? new_len[s] : -1;
        const bool cut = to >= 0 && to < len;
        const int first = (to + mask) >> c.page_shift, last = (len + mask) >> c.page_shift;
        const Sums p = block_sum(cut ? last - first : 0, s_tmp[0]);
        s_before[tid] = p.before;
        s_last[tid] = last;
        if (cut) seq_len[s] = to;
        __syncthreads();
        int turn = 1;
        for (uint32_t i0 = 0; i0 < p.all; i0 += kThreads * kItems) {
            const uint32_t i = i0 + tid * kItems;
            int32_t page[kItems];
            uint32_t valid = 0;
            int t = i < p.all ? entry_of(s_before, here, i) : 0;
            int32_t *at[kItems];
#pragma unroll
            for (int j = 0; j < kItems; j++) page[j] = -1, at[j] = nullptr;
#pragma unroll
            for (int j = 0; j < kItems; j++) {
                if (i + j >= p.all) break;
                while (t + 1 < here && s_before[t + 1] <= i + j) t++;
                at[j] = table + (int64_t)(base + here - 1 - t) * c.table_ld + (s_last[t] - 1 - (int)(i + j - s_before[t]));
                page[j] = *at[j];
            }
#pragma unroll
            for (int j = 0; j < kItems; j++) {
                if (at[j]) *at[j] = -1;
                valid += (uint32_t)page[j] < (uint32_t)c.n_pages;
            }
            const Sums v = block_sum(valid, s_tmp[turn]);
            int64_t to_at = (int64_t)count + pushed + v.before;
#pragma unroll
            for (int j = 0; j < kItems; j++)
                if ((uint32_t)page[j] < (uint32_t)c.n_pages) {
                    if (to_at < c.n_pages) free_pages[to_at] = page[j];
                    to_at++;
                }
            pushed = sat_add(pushed, v.all);
            turn = 3 - turn;  // the sums' memory is used again two turns later, behind the barrier between
        }
        __syncthreads();
    }
    if (tid == 0) {
        const int64_t now = (int64_t)count + pushed;
        *free_count = (int)(now < c.n_pages ? now : c.n_pages);
    }
}

// Rows that the one workgroup writes beside the pages; more get a launch of
// their own.
constexpr int64_t kFewRows = 4096;

}  // namespace

hipError_t launch_kv_reserve(const KvArgs &c, int32_t *table, int32_t *seq_len, const ReserveArgs &a, int32_t *pos,
                             int64_t *slot, hipStream_t s) {
    const bool few = a.n <= kFewRows;
    const hipError_t e = launch_main(kv_reserve, dim3(1), dim3(kThreads), 0, s, c, table, seq_len, a, few ? pos : nullptr,
                                     few ? slot : nullptr);
    if (e != hipSuccess || few || (!pos && !slot)) return e;
    return launch_aux(kv_row_slots, dim3((a.n + 255) / 256), dim3(256), 0, s, c, a.n, (const int32_t *)a.start, pos, slot);
}

hipError_t launch_kv_release(const KvArgs &c, int32_t *table, int32_t *seq_len, const int32_t *new_len,
                             int32_t *free_pages, int32_t *free_count, hipStream_t s) {
    return launch_main(kv_release, dim3(1), dim3(kThreads), 0, s, c, table, seq_len, new_len, free_pages, free_count);
}

}  // namespace qmv
