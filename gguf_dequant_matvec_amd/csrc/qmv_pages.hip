// The pages of a cache kept on the GPU: a stack of free ones, from which
// sequences take what their next tokens need and to which they give back what
// lies behind a shorter length, so that a serving loop's steps follow each
// other without the host.
//
// Whole numbers and little of them: both calls are chains of latencies.  One
// workgroup does all of it (nothing waits for another one's sums), as many
// sequences at a time as it has threads: prefix sums say who gets what, then
// pages, and the rows of a call of few, are dealt out evenly, the threads finding
// their sequences by bisection of the sums in LDS.  Small batches take four waves
// (barriers and the sums across waves are shorter), others sixteen.
#include "qmv_device.h"
#include "qmv_internal.h"
#include "qmv_pages.h"

#include <type_traits>

namespace qmv {

namespace {

// Pages a thread takes at a time, so that their loads fly together: 4096 in all.
template <int T>
constexpr int kItems = 4096 / T;
// Threads.  Few pages to move: 256 (64 sequences, a token each: 2.7 us to release,
// 3.7 to reserve, with 1024 threads 3.2 and 4.9), many: 1024 (10500 pages of 96
// sequences: 8.9 and 9.3 us, with 256 threads 20 and 19).
constexpr int kSmall = 256, kLarge = 1024;
// Sums stop here: no call can be given more rows, or give back more pages.
constexpr uint32_t kSat = 1u << 30;

__device__ __forceinline__ uint32_t sat_add(uint32_t a, uint32_t b) { return a + b < kSat ? a + b : kSat; }

// Inclusive sum over the wave's 64 lanes: within rows of 16, then across them.
__device__ __forceinline__ uint32_t wave_upto(uint32_t x) {
    x = sat_add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x111, 0xF, 0xF, false));  // row_shr 1, 2, 4, 8
    x = sat_add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x112, 0xF, 0xF, false));
    x = sat_add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x114, 0xF, 0xF, false));
    x = sat_add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x118, 0xF, 0xF, false));
    x = sat_add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x142, 0xA, 0xF, false));  // row_bcast 15, 31
    x = sat_add(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x143, 0xC, 0xF, false));
    return x;
}

struct Sums {
    uint32_t before, all;
};
// Prefix sums of two values over the workgroup; `tmp` is the call's own.
template <int W>
__device__ __forceinline__ void block_sums(uint32_t x, uint32_t y, uint32_t (*tmp)[W], Sums &sx, Sums &sy) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t ux = wave_upto(x), uy = wave_upto(y);
    if (lane == 63) tmp[0][wave] = ux, tmp[1][wave] = uy;
    lds_barrier();  // (nothing that a launch writes to memory is read again in it)
    sx = sy = Sums{0, 0};
#pragma unroll
    for (int w = 0; w < W; w++) {
        if (w == wave) sx.before = sx.all, sy.before = sy.all;
        sx.all = sat_add(sx.all, tmp[0][w]), sy.all = sat_add(sy.all, tmp[1][w]);
    }
    // (a sum that stopped at its largest gives no smaller one for the lane: what is
    // before it is then too much as well, and not used)
    sx.before = sat_add(sx.before, ux - x), sy.before = sat_add(sy.before, uy - y);
}

// The last of `n` entries whose sum before it is at most i: the one that i is in.
// As many steps for every i, so that several searches run beside each other.
template <int N>
__device__ __forceinline__ void entries_of(const uint32_t *before, int n, const uint32_t (&i)[N], int (&t)[N]) {
#pragma unroll
    for (int j = 0; j < N; j++) t[j] = 0;
    for (int step = n > 1 ? 1 << (31 - __builtin_clz(n - 1)) : 0; step; step >>= 1) {
#pragma unroll
        for (int j = 0; j < N; j++) {
            const int to = t[j] + step;
            if (to < n && before[to < n ? to : 0] <= i[j]) t[j] = to;
        }
    }
}

__device__ __forceinline__ int clamped(int x, int most) { return x < 0 ? 0 : x > most ? most : x; }

__device__ __forceinline__ int64_t slot_of(const KvArgs &c, int page, int pos) {
    if ((uint32_t)page >= (uint32_t)c.n_pages) return -1;
    return ((int64_t)page << c.page_shift) + (pos & ((1 << c.page_shift) - 1));
}

// What a row needs is in LDS when its turn comes: the page that its sequence ends
// in (loaded beside the sums) and the first kKept pages that are handed out.
constexpr int kKept = 2048;

template <int T>
__global__ __launch_bounds__(T) void kv_reserve(KvArgs c, int32_t *table, int32_t *seq_len, ReserveArgs a,
                                                       int32_t *pos, int64_t *slot) {
    __shared__ uint32_t s_tmp[4][T / 64], s_pages[T], s_rows[T];
    __shared__ int s_len[T], s_end[T], s_kept[kKept];
    const int tid = threadIdx.x, mask = (1 << c.page_shift) - 1;
    const int count = clamped(*a.free_count, c.n_pages);
    uint32_t need_all = 0, rows_all = 0;  // what was asked for so far
    int popped = 0, row0 = 0;             // what was given
    for (int base = 0; base < c.n_seq; base += T) {
        const int s = base + tid, here = c.n_seq - base < T ? c.n_seq - base : T;
        const int len = tid < here ? seq_len[s] : 0, add = tid < here ? a.add[s] : 0;
        // the page of this thread's turn, if there will be so many
        int32_t page[kItems<T>];
        page[0] = count - 1 - popped - tid >= 0 ? a.free_pages[count - 1 - popped - tid] : -1;
        const bool fits = add > 0 && len >= 0 && (int64_t)len + add <= c.cap;
        if (slot) s_end[tid] = fits && (len & mask) ? table[(int64_t)s * c.table_ld + (len >> c.page_shift)] : -1;
        // (for a length that does not fit the sums below may overflow, and are not used)
        const int first = (int)(((uint32_t)len + mask) >> c.page_shift);
        const uint32_t need = fits ? ((len + add + mask) >> c.page_shift) - first : 0, rows = fits ? add : 0;
        Sums p, r, pg, rg;
        block_sums(need, rows, s_tmp, p, r);
        const uint32_t p_upto = sat_add(sat_add(need_all, p.before), need), r_upto = sat_add(sat_add(rows_all, r.before), rows);
        const bool given = fits && r_upto <= (uint32_t)a.n && (need == 0 || (p_upto <= (uint32_t)count && p_upto < kSat));
        block_sums(given ? need : 0, given ? rows : 0, s_tmp + 2, pg, rg);
        s_pages[tid] = pg.before;
        s_rows[tid] = rg.before;
        s_len[tid] = len;
        if (tid < here) {
            a.granted[s] = given ? add : 0;
            a.start[s] = row0 + (int)rg.before;
            if (given) seq_len[s] = len + add;
        }
        lds_barrier();
        // the i-th page of these goes to its sequence: N for each thread, T apart
        auto take = [&](auto n_items, uint32_t i0) {
            constexpr int N = decltype(n_items)::value;
            uint32_t i[N];
            int t[N];
#pragma unroll
            for (int j = 0; j < N; j++) {
                i[j] = i0 + tid + j * T;
                if (i0 > 0 || j > 0) page[j] = i[j] < pg.all ? a.free_pages[count - 1 - popped - (int)i[j]] : -1;
            }
            entries_of(s_pages, here, i, t);
#pragma unroll
            for (int j = 0; j < N; j++) {
                if (i[j] >= pg.all) continue;
                const int at = ((s_len[t[j]] + mask) >> c.page_shift) + (int)(i[j] - s_pages[t[j]]);
                table[(int64_t)(base + t[j]) * c.table_ld + at] = page[j];
                if (i[j] < kKept) s_kept[i[j]] = page[j];
            }
        };
        if (pg.all <= T) {
            if (pg.all > 0) take(std::integral_constant<int, 1>(), 0);
        } else {
            for (uint32_t i0 = 0; i0 < pg.all; i0 += 4096) take(std::integral_constant<int, kItems<T>>(), i0);
        }
        if (pos || slot) {
            lds_barrier();
            for (uint32_t i = tid; i < rg.all; i += T) {
                const uint32_t i1[1] = {i};
                int t1[1];
                entries_of(s_rows, here, i1, t1);
                const int t = t1[0], at = s_len[t] + (int)(i - s_rows[t]);
                const int own = (s_len[t] + mask) >> c.page_shift, k = at >> c.page_shift;
                if (pos) pos[row0 + (int)i] = at;
                if (slot) {
                    const int rank = (int)s_pages[t] + k - own;  // of the row's page among those handed out
                    const int pg_of = k < own ? s_end[t] : rank < kKept ? s_kept[rank] : a.free_pages[count - 1 - popped - rank];
                    slot[row0 + (int)i] = slot_of(c, pg_of, at);
                }
            }
        }
        need_all = sat_add(need_all, p.all);
        rows_all = sat_add(rows_all, r.all);
        popped += (int)pg.all;
        row0 += (int)rg.all;
        lds_barrier();
    }
    if (pos || slot) {
        for (int i = row0 + tid; i < a.n; i += T) {
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
template <int T>
__global__ __launch_bounds__(T) void kv_release(KvArgs c, int32_t *table, int32_t *seq_len, const int32_t *new_len,
                                                       int32_t *free_pages, int32_t *free_count) {
    constexpr int W = T / 64;
    __shared__ uint32_t s_tmp[2][W], s_before[T], s_count[64], s_all;
    __shared__ int s_last[T];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tid = threadIdx.x, mask = (1 << c.page_shift) - 1;
    const int count = clamped(*free_count, c.n_pages);
    uint32_t pushed = 0;
    for (int base = (c.n_seq - 1) / T * T; base >= 0; base -= T) {
        const int here = c.n_seq - base < T ? c.n_seq - base : T, s = base + here - 1 - tid;
        const int len = tid < here ? clamped(seq_len[s], c.cap) : 0, to = tid < here ? new_len[s] : -1;
        const bool cut = to >= 0 && to < len;
        const int first = (to + mask) >> c.page_shift, last = (len + mask) >> c.page_shift;
        Sums p, none;
        block_sums(cut ? last - first : 0, 0, s_tmp, p, none);
        s_before[tid] = p.before;
        s_last[tid] = last;
        if (cut) seq_len[s] = to;
        lds_barrier();
        // N pages a thread, T apart, from the i0-th on
        auto give = [&](auto n_items, uint32_t i0) {
            constexpr int N = decltype(n_items)::value;
            uint32_t i[N];
            int32_t page[N], *at[N];
            int t[N];
#pragma unroll
            for (int j = 0; j < N; j++) i[j] = i0 + tid + j * T;
            entries_of(s_before, here, i, t);
#pragma unroll
            for (int j = 0; j < N; j++) {
                at[j] = table + (int64_t)(base + here - 1 - t[j]) * c.table_ld + (s_last[t[j]] - 1 - (int)(i[j] - s_before[t[j]]));
                page[j] = i[j] < p.all ? *at[j] : -1;
            }
            uint64_t valid[N];
#pragma unroll
            for (int j = 0; j < N; j++) {
                if (i[j] < p.all) *at[j] = -1;
                valid[j] = __ballot((uint32_t)page[j] < (uint32_t)c.n_pages);
                if (lane == 0) s_count[j * W + wave] = __popcll(valid[j]);
            }
            lds_barrier();
            if (wave == 0) {  // 64 counts at most: sums up to each
                const uint32_t own = lane < N * W ? s_count[lane] : 0, upto = wave_upto(own);
                if (lane < N * W) s_count[lane] = upto - own;
                if (lane == 63) s_all = upto;
            }
            lds_barrier();
            const uint64_t below = (1ull << lane) - 1;
#pragma unroll
            for (int j = 0; j < N; j++) {
                const int64_t to_at = (int64_t)count + pushed + s_count[j * W + wave] + __popcll(valid[j] & below);
                if ((uint32_t)page[j] < (uint32_t)c.n_pages && to_at < c.n_pages) free_pages[to_at] = page[j];
            }
            pushed = sat_add(pushed, s_all);
            lds_barrier();  // the counts' memory is used again
        };
        if (p.all <= T) {
            if (p.all > 0) give(std::integral_constant<int, 1>(), 0);
        } else {
            for (uint32_t i0 = 0; i0 < p.all; i0 += 4096) give(std::integral_constant<int, kItems<T>>(), i0);
        }
        lds_barrier();
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
    auto launch = [&](auto kernel, int threads) {
        return launch_main(kernel, dim3(1), dim3(threads), 0, s, c, table, seq_len, a, few ? pos : nullptr, few ? slot : nullptr);
    };
    const bool small = c.n_seq <= kSmall && a.n <= kSmall;  // a row needs a page at most
    const hipError_t e = small ? launch(kv_reserve<kSmall>, kSmall) : launch(kv_reserve<kLarge>, kLarge);
    if (e != hipSuccess || few || (!pos && !slot)) return e;
    return launch_aux(kv_row_slots, dim3((a.n + 255) / 256), dim3(256), 0, s, c, a.n, (const int32_t *)a.start, pos, slot);
}

hipError_t launch_kv_release(const KvArgs &c, int32_t *table, int32_t *seq_len, const int32_t *new_len,
                             int32_t *free_pages, int32_t *free_count, hipStream_t s) {
    auto launch = [&](auto kernel, int threads) {
        return launch_main(kernel, dim3(1), dim3(threads), 0, s, c, table, seq_len, new_len, free_pages, free_count);
    };
    const bool small = c.n_seq <= kSmall && c.n_seq * c.table_ld <= 8192;  // the most pages there can be
    return small ? launch(kv_release<kSmall>, kSmall) : launch(kv_release<kLarge>, kLarge);
}

}  // namespace qmv
