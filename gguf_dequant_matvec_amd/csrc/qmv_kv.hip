// Writing the paged key-value cache: appending new tokens' rows, and cutting
// a cache down to the positions with the largest accumulated weight.
#include "qmv_device.h"
#include "qmv_internal.h"
#include "qmv_kv.h"

#include <type_traits>

namespace qmv {

namespace {

// ---- append -----------------------------------------------------------------
// A workgroup takes ROWS consecutive rows of one key-value head.  All f32
// values are on their way before the positions are looked up (two dependent
// loads).  K rows are rounded and stored as they come, 16 bytes a thread.  V
// goes through LDS, already rounded, because a V block keeps the 16 positions
// of one column next to each other: a thread gathers 8 positions of a column
// and stores them at once where the workgroup's rows cover all 8, else one by
// one.  Bound by memory, or for few rows by latency: 16 rows keep more
// workgroups in flight, 32 leave fewer partly covered runs.  Measured: 6808
// rows of 8 heads of 128, bf16, 83.7 MB: 20.2 us (4.1 TB/s); 16 rows: 4.3 us.
template <int TYPE>
__device__ __forceinline__ uint32_t kv_round(float x) {
    if constexpr (TYPE == kKvF16) {
        return __builtin_bit_cast(uint16_t, (_Float16)x);  // nearest even
    } else {
        return __builtin_bit_cast(uint16_t, (__bf16)x);  // nearest even
    }
}

// 8-bit rows: d = max |x| / 127, code = x / d to the nearest integer.
__device__ __forceinline__ int kv_code(float x, float d) {
    const float r = d > 0.f ? rintf(x / d) : 0.f;
    return (int)fminf(fmaxf(r, -127.f), 127.f);
}

template <int TYPE, int HD, int ROWS>
__global__ __launch_bounds__(256) void kv_append(KvArgs c, int64_t n, const int32_t *start,
                                                 const float *__restrict__ k, int64_t ldk,
                                                 const float *__restrict__ v, int64_t ldv) {
    constexpr int SZ = TYPE == kKvI8 ? 1 : 2;
    constexpr int PIECES = HD / 8;                         // 8 columns a thread
    constexpr int N = (ROWS * PIECES + 255) / 256;         // pieces a thread
    constexpr int VROW = HD + (TYPE == kKvI8 ? 4 : 2);     // padded row in LDS, values
    typedef typename std::conditional<TYPE == kKvI8, int8_t, uint16_t>::type Val;
    __shared__ int s_page[ROWS], s_slot[ROWS];
    __shared__ bool s_run[ROWS];  // the row's aligned group of 8 positions is here, row by row
    __shared__ __align__(16) Val s_v[ROWS * VROW];
    __shared__ float s_d[2][ROWS];
    __shared__ float s_part[TYPE == kKvI8 ? 2 : 1][TYPE == kKvI8 ? ROWS * PIECES : 1];
    const int tid = threadIdx.x, h = blockIdx.y;
    const int64_t row0 = (int64_t)blockIdx.x * ROWS;
    const int rows = n - row0 < ROWS ? (int)(n - row0) : ROWS;

    float kf[N][8], vf[N][8];
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int e = tid + 256 * i, r = e / PIECES, p = e % PIECES;
        if (r < rows) {
            const uint8_t *ks = reinterpret_cast<const uint8_t *>(k + (row0 + r) * ldk + (int64_t)h * HD + p * 8);
            const uint8_t *vs = reinterpret_cast<const uint8_t *>(v + (row0 + r) * ldv + (int64_t)h * HD + p * 8);
            const float4 a = __builtin_bit_cast(float4, load16(ks)), b = __builtin_bit_cast(float4, load16(ks + 16));
            const float4 x = __builtin_bit_cast(float4, load16(vs)), y = __builtin_bit_cast(float4, load16(vs + 16));
            kf[i][0] = a.x, kf[i][1] = a.y, kf[i][2] = a.z, kf[i][3] = a.w;
            kf[i][4] = b.x, kf[i][5] = b.y, kf[i][6] = b.z, kf[i][7] = b.w;
            vf[i][0] = x.x, vf[i][1] = x.y, vf[i][2] = x.z, vf[i][3] = x.w;
            vf[i][4] = y.x, vf[i][5] = y.y, vf[i][6] = y.z, vf[i][7] = y.w;
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) kf[i][j] = vf[i][j] = 0.f;
        }
    }
    if (tid < ROWS) {
        const int64_t r = row0 + tid;
        int page = -1, slot = 0;
        if (r < n) {
            int seq = 0;
            int64_t first = 0, next = 0;
            if (start) {  // the last sequence that starts at or before r
                int lo = 0, hi = c.n_seq;
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (start[mid] <= r) lo = mid; else hi = mid;
                }
                seq = lo;
                first = start[seq];
                next = start[seq + 1];
            } else {
                const int64_t each = n / c.n_seq;
                seq = (int)(r / each);
                first = (int64_t)seq * each;
                next = first + each;
            }
            const int64_t pos = (int64_t)c.seq_len[seq] - (next - r);
            if (r >= first && r < next && pos >= 0 && pos < c.cap) {
                page = kv_page(c, seq, (int)pos);
                slot = (int)pos & ((1 << c.page_shift) - 1);
            }
        }
        s_page[tid] = page;
        s_slot[tid] = slot;
    }
    if constexpr (TYPE == kKvI8) {
        // row maxima; a NaN anywhere makes the maximum NaN
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int e = tid + 256 * i;
            float mk = 0.f, mv = 0.f;
#pragma unroll
            for (int j = 0; j < 8; j++) {
                mk = fmaxf(mk, fabsf(kf[i][j]));
                mv = fmaxf(mv, fabsf(vf[i][j]));
            }
#pragma unroll
            for (int j = 0; j < 8; j++) {  // (fmaxf drops a NaN)
                mk = kf[i][j] != kf[i][j] ? kf[i][j] : mk;
                mv = vf[i][j] != vf[i][j] ? vf[i][j] : mv;
            }
            if (e < ROWS * PIECES) {
                s_part[0][e] = mk;
                s_part[1][e] = mv;
            }
        }
        __syncthreads();
        for (int e = tid; e < 2 * ROWS; e += 256) {
            const int which = e / ROWS, r = e % ROWS;
            float m = 0.f;
            bool nan = false;
            for (int p = 0; p < PIECES; p++) {
                const float x = s_part[which][r * PIECES + p];
                nan = nan || x != x;
                m = fmaxf(m, x);
            }
            s_d[which][r] = nan ? __builtin_nanf("") : m / 127.f;
        }
    }
    __syncthreads();

    const int64_t page_size = 1ll << c.page_shift;
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int e = tid + 256 * i, r = e / PIECES, p = e % PIECES;
        if (r >= ROWS) continue;
        const int page = s_page[r];
        uint32_t w[4] = {0, 0, 0, 0}, x[4] = {0, 0, 0, 0};
#pragma unroll
        for (int j = 0; j < 8; j++) {
            if constexpr (TYPE == kKvI8) {
                w[j >> 2] |= (uint32_t)(kv_code(kf[i][j], s_d[0][r]) & 0xFF) << (8 * (j & 3));
                x[j >> 2] |= (uint32_t)(kv_code(vf[i][j], s_d[1][r]) & 0xFF) << (8 * (j & 3));
            } else {
                w[j >> 1] |= kv_round<TYPE>(kf[i][j]) << (16 * (j & 1));
                x[j >> 1] |= kv_round<TYPE>(vf[i][j]) << (16 * (j & 1));
            }
        }
        uint32_t *sv = reinterpret_cast<uint32_t *>(s_v + r * VROW + p * 8);
#pragma unroll
        for (int j = 0; j < 2 * SZ; j++) sv[j] = x[j];
        if (page < 0) continue;
        uint8_t *dst = kv_head(c, page, h) + ((int64_t)s_slot[r] * HD + p * 8) * SZ;
        if constexpr (TYPE == kKvI8)
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        else
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    if (tid < ROWS) {
        const int r8 = tid - (s_slot[tid] & 7);
        bool run = r8 >= 0 && r8 + 8 <= ROWS;
        for (int j = 0; run && j < 8; j++)
            run = s_page[r8 + j] == s_page[tid] && s_slot[r8 + j] == (s_slot[tid] & ~7) + j;
        s_run[tid] = run;
    }
    if (TYPE == kKvI8 && tid < 2 * ROWS) {
        const int r = tid % ROWS, which = tid / ROWS;
        if (s_page[r] >= 0) {
            float *sc = reinterpret_cast<float *>(kv_head(c, s_page[r], h) + 2 * page_size * HD);
            sc[which * page_size + s_slot[r]] = s_d[which][r];
        }
    }
    __syncthreads();
    // V: lanes run over columns; a whole group leaves with its first row
    for (int e = tid; e < ROWS * HD; e += 256) {
        const int r = e / HD, d = e % HD;
        const int page = s_page[r], slot = s_slot[r];
        if (page < 0) continue;
        uint8_t *dst = kv_head(c, page, h) + page_size * HD * SZ +
                       ((int64_t)(slot / kVBlock) * (HD * kVBlock) + d * kVBlock + slot % kVBlock) * SZ;
        if (!s_run[r]) {
            *reinterpret_cast<Val *>(dst) = s_v[r * VROW + d];
        } else if ((slot & 7) == 0) {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t b = TYPE == kKvI8 ? (uint8_t)s_v[(r + j) * VROW + d] : (uint16_t)s_v[(r + j) * VROW + d];
                w[j / (4 / SZ)] |= b << (8 * SZ * (j % (4 / SZ)));
            }
            if constexpr (TYPE == kKvI8)
                *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---- eviction: choosing -------------------------------------------------------
// One workgroup per sequence and key-value head, 1024 PER positions at a time,
// PER a thread (thread t has t, t + 1024, ...: neighbouring lanes read
// neighbouring scores; with no more positions than that they stay in registers).  The
// m-th largest score of the middle positions is found by four 8-bit radix
// passes over an order-preserving integer key (counts in LDS), then counts per
// wave and step, one prefix sum over them and the lanes' ballots place the
// kept positions in order; among equal scores at the border the lowest
// positions are kept.  Bound by latency, three barriers a pass:
// 64 heads of 4352 positions 11.1 us, 3 of 1001 5.6 us.
constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;

// 16 bytes that are read once and not again (the old pages are given back).
__device__ __forceinline__ uint4 load_once(const uint8_t *p) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const u32x4 v = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
    return make_uint4(v.x, v.y, v.z, v.w);
}

__device__ __forceinline__ uint32_t score_key(float v) {
    if (v != v) return 0xFFFFFFFFu;   // NaN ranks above everything
    return float_key(v + 0.f);        // -0 counts as +0
}

template <int PER>
__global__ __launch_bounds__(kSelThreads) void kv_evict_select(KvArgs c, EvictArgs e) {
    constexpr int STEP = kSelThreads * PER;
    constexpr int COUNTS = PER * kSelWaves, EACH = (COUNTS + 63) / 64;  // counts, and a lane's share
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    const int lane = tid & 63, wave = tid >> 6;
    const int len = kv_len(c, s, e.limit);
    const int64_t head = (int64_t)s * c.n_kv + h;
    int32_t *kept = e.kept + head * e.keep;
    float *acc_out = e.acc_out + head * e.ld_out;
    const float *acc = e.acc + head * e.ld_acc;
    const int out_len = len < e.keep ? len : e.keep;
    for (int i = out_len + tid; i < e.keep; i += kSelThreads) {
        kept[i] = -1;
        acc_out[i] = 0.f;
    }
    if (len <= e.keep) {
        for (int i = tid; i < len; i += kSelThreads) {
            kept[i] = i;
            acc_out[i] = acc[i];
        }
        return;
    }
    const int lo = e.first, hi = len - e.recent;   // candidates: lo <= position < hi
    const int m = e.keep - e.first - e.recent;     // of which m stay, 0 <= m < hi - lo

    float f[PER];  // the thread's scores, and their keys
    uint32_t key[PER];
    auto load_keys = [&](int base) {
#pragma unroll
        for (int j = 0; j < PER; j++) {
            const int i = base + j * kSelThreads + tid;
            f[j] = i < len ? acc[i] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < PER; j++) key[j] = score_key(f[j]);
    };
    load_keys(0);

    __shared__ int hist[256];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    uint32_t prefix = 0, mask = 0;
    int left = m;  // rank still to go inside the current prefix
    if (m > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int base = 0; base < len; base += STEP) {
                if (len > STEP) load_keys(base);
#pragma unroll
                for (int j = 0; j < PER; j++) {
                    const int i = base + j * kSelThreads + tid;
                    if (i >= lo && i < hi && (key[j] & mask) == prefix) atomicAdd(&hist[(key[j] >> shift) & 255], 1);
                }
            }
            __syncthreads();
            if (wave == 0) {
                // lane l has the four bins 255 - 4 l downwards; the one in
                // which the count from the top reaches `left` says the digit
                int cnt[4], all = 0;
                for (int j = 0; j < 4; j++) all += cnt[j] = hist[255 - 4 * lane - j];
                int upto = all;
                for (int off = 1; off < 64; off <<= 1) {
                    const int x = __shfl_up(upto, off);
                    if (lane >= off) upto += x;
                }
                int above = upto - all;
                if (above < left && left <= upto) {
                    int j = 0;
                    while (j < 3 && above + cnt[j] < left) above += cnt[j++];
                    s_prefix = prefix | ((uint32_t)(255 - 4 * lane - j) << shift);
                    s_left = left - above;
                }
            }
            __syncthreads();
            prefix = s_prefix;
            left = s_left;
            mask |= 255u << shift;
        }
    }
    // kept: everything protected, every key above `prefix`, and the first
    // `left` candidates equal to it
    __shared__ int s_cnt[2][EACH * 64], s_all[2];
    // exclusive prefix sum of the counts, by wave 0
    auto scan = [&](int which) {
        if (wave == 0) {
            int own[EACH], all = 0;
#pragma unroll
            for (int j = 0; j < EACH; j++) all += own[j] = lane * EACH + j < COUNTS ? s_cnt[which][lane * EACH + j] : 0;
            int upto = all;
            for (int off = 1; off < 64; off <<= 1) {
                const int x = __shfl_up(upto, off);
                if (lane >= off) upto += x;
            }
            int at = upto - all;
#pragma unroll
            for (int j = 0; j < EACH; j++) {
                s_cnt[which][lane * EACH + j] = at;
                at += own[j];
            }
            if (lane == 63) s_all[which] = upto;
        }
    };
    const uint64_t below = (1ull << lane) - 1;
    int ties_before = 0, kept_before = 0;
    for (int base = 0; base < len; base += STEP) {
        if (len > STEP) load_keys(base);
        uint32_t sure = 0, tie = 0;
#pragma unroll
        for (int j = 0; j < PER; j++) {
            const int i = base + j * kSelThreads + tid;
            const bool mid = i >= lo && i < hi;
            if (i < len && (!mid || (m > 0 && key[j] > prefix))) sure |= 1u << j;
            if (mid && m > 0 && key[j] == prefix) tie |= 1u << j;
            const uint64_t b = __ballot((tie >> j) & 1);
            if (lane == 0) s_cnt[0][j * kSelWaves + wave] = (int)__popcll(b);
        }
        __syncthreads();
        scan(0);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < PER; j++) {
            const uint64_t b = __ballot((tie >> j) & 1);
            const int rank = ties_before + s_cnt[0][j * kSelWaves + wave] + (int)__popcll(b & below);
            if (((tie >> j) & 1) && rank < left) sure |= 1u << j;
            const uint64_t k = __ballot((sure >> j) & 1);
            if (lane == 0) s_cnt[1][j * kSelWaves + wave] = (int)__popcll(k);
        }
        __syncthreads();
        scan(1);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < PER; j++) {
            const uint64_t k = __ballot((sure >> j) & 1);
            const int at = kept_before + s_cnt[1][j * kSelWaves + wave] + (int)__popcll(k & below);
            if (((sure >> j) & 1) && at < e.keep) {
                kept[at] = base + j * kSelThreads + tid;
                acc_out[at] = f[j];
            }
        }
        ties_before += s_all[0];
        kept_before += s_all[1];
        __syncthreads();
    }
}

// ---- eviction: moving -----------------------------------------------------------
// A workgroup fills 64 positions (four V blocks) of the destination.  K rows
// are copied as they are.  The sources are in order, so they lie in few
// source V blocks (five where one position in sixteen is dropped): those are
// read whole, up to GROUP at a time, into LDS rows padded so that columns
// fall into different banks, and each thread picks the kept positions of its
// columns, 16 bytes of the new block at a time.  Bound by memory, both caches
// once: 64 heads of 4352 -> 4096 rows of 128 f16 columns, 269 MB, 63 us (4.3
// TB/s; a plain copy runs at 4.98).
constexpr int kMove = 64;

template <int SZ, int HD>
__global__ __launch_bounds__(256) void kv_evict_move(KvArgs c, EvictArgs e) {
    constexpr int ROW = HD * SZ;                         // bytes of a K row
    constexpr int KP = kMove * ROW / 16;                 // 16-byte pieces of the K rows
    constexpr int KN = (KP + 255) / 256;
    constexpr int VB = HD * kVBlock * SZ;                // bytes of a V block
    constexpr int VP = VB / 16, VN = (VP + 255) / 256;   // its pieces
    constexpr int PAD = SZ == 2 ? 40 : 20;               // LDS bytes of a column of a block
    constexpr int GROUP = HD == 256 ? 4 : 6;             // source blocks in LDS
    constexpr int PER = 16 / SZ;                         // positions in a piece
    constexpr int OUT = kMove / PER * HD;                // pieces of the new blocks
    constexpr int ON = (OUT + 255) / 256;
    typedef typename std::conditional<SZ == 2, uint16_t, uint8_t>::type Val;

    const int h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x;
    const int len = kv_len(c, s, e.limit);
    const int out_len = len < e.keep ? len : e.keep;
    // (seq_len itself may be len_out: cutting a cut length changes nothing)
    if (blockIdx.x == 0 && h == 0 && tid == 0) e.len_out[s] = out_len;
    const int i0 = blockIdx.x * kMove;
    if (i0 >= out_len) return;
    const int cnt = out_len - i0 < kMove ? out_len - i0 : kMove;
    const int64_t page_size = 1ll << c.page_shift;
    const int pmask = (int)page_size - 1;

    __shared__ int s_src[kMove], s_page[kMove], s_ord[kMove];
    __shared__ int s_first[kMove + 1];   // first source of each source block
    __shared__ int s_dst[kMove / kVBlock];
    __shared__ int s_blocks;
    __shared__ __align__(16) uint8_t s_v[GROUP * HD * PAD];
    if (tid < kMove) {
        int src = -1, page = -1;
        if (tid < cnt) {
            src = e.kept[((int64_t)s * c.n_kv + h) * e.keep + i0 + tid];
            page = kv_page(c, s, src);
        }
        s_src[tid] = src;
        s_page[tid] = page;
        const int prev = __shfl_up(src, 1);
        const bool first = tid < cnt && (tid == 0 || src / kVBlock != prev / kVBlock);
        const uint64_t all = __ballot(first);
        const int ord = __popcll(all & ((2ull << tid) - 1)) - 1;
        s_ord[tid] = ord;
        if (first) s_first[ord] = tid;
        if (tid == 0) s_blocks = __popcll(all);
    } else if (tid < kMove + kMove / kVBlock) {
        const int at = i0 + (tid - kMove) * kVBlock;
        int pg = -1;
        if (at < out_len) {
            pg = e.dst[(int64_t)s * e.dst_ld + (at >> c.page_shift)];
            if ((uint32_t)pg >= (uint32_t)c.n_pages) pg = -1;
        }
        s_dst[tid - kMove] = pg;
    }
    __syncthreads();

    // K: all loads, then all stores
    uint4 kw[KN];
#pragma unroll
    for (int j = 0; j < KN; j++) {
        const int o = (tid + 256 * j) * 16, i = o / ROW, b = o % ROW;
        kw[j] = make_uint4(0, 0, 0, 0);
        if (i < cnt && s_page[i] >= 0)
            kw[j] = load_once(kv_head(c, s_page[i], h) + (int64_t)(s_src[i] & pmask) * ROW + b);
    }
    const int blocks = s_blocks;
    uint4 vw[GROUP][VN];
    auto load_group = [&](int g0) {
#pragma unroll
        for (int k = 0; k < GROUP; k++) {
            const int b = g0 + k;
            const int a = b < blocks ? s_first[b] : 0;
            const int page = b < blocks ? s_page[a] : -1;
            const uint8_t *src = kv_head(c, page < 0 ? 0 : page, h) + page_size * ROW + (int64_t)((s_src[a] & pmask) / kVBlock) * VB;
#pragma unroll
            for (int j = 0; j < VN; j++) {
                const int p = tid + 256 * j;
                vw[k][j] = make_uint4(0, 0, 0, 0);
                if (page >= 0 && p < VP) vw[k][j] = load_once(src + p * 16);
            }
        }
    };
    load_group(0);
#pragma unroll
    for (int j = 0; j < KN; j++) {
        const int o = (tid + 256 * j) * 16, i = o / ROW, b = o % ROW;
        if (i >= cnt || s_dst[i / kVBlock] < 0) continue;
        *reinterpret_cast<uint4 *>(kv_head(c, s_dst[i / kVBlock], h) + (int64_t)((i0 + i) & pmask) * ROW + b) = kw[j];
    }
    uint32_t out[ON][4];
#pragma unroll
    for (int j = 0; j < ON; j++) out[j][0] = out[j][1] = out[j][2] = out[j][3] = 0;
    for (int g0 = 0; g0 < blocks; g0 += GROUP) {
        if (g0 > 0) load_group(g0);
#pragma unroll
        for (int k = 0; k < GROUP; k++) {
#pragma unroll
            for (int j = 0; j < VN; j++) {
                const int p = tid + 256 * j;  // SZ 2: half of a column; SZ 1: a column
                if (p >= VP) continue;
                const uint4 w = vw[k][j];
                if constexpr (SZ == 2) {
                    uint2 *at = reinterpret_cast<uint2 *>(s_v + (k * HD + p / 2) * PAD + 16 * (p % 2));
                    at[0] = make_uint2(w.x, w.y);
                    at[1] = make_uint2(w.z, w.w);
                } else {
                    uint32_t *at = reinterpret_cast<uint32_t *>(s_v + (k * HD + p) * PAD);
                    at[0] = w.x, at[1] = w.y, at[2] = w.z, at[3] = w.w;
                }
            }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < ON; j++) {
            const int u = tid + 256 * j, d = u % HD, i = u / HD * PER;  // column, first position
            if (u >= OUT) continue;
#pragma unroll
            for (int x = 0; x < PER; x++) {
                const int k = s_ord[i + x] - g0;
                if (i + x < cnt && k >= 0 && k < GROUP) {
                    const Val *col = reinterpret_cast<const Val *>(s_v + (k * HD + d) * PAD);
                    out[j][x * SZ / 4] |= (uint32_t)col[s_src[i + x] % kVBlock] << (8 * SZ * (x % (4 / SZ)));
                }
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < ON; j++) {
        const int u = tid + 256 * j, d = u % HD, i = u / HD * PER;
        if (u >= OUT || i >= cnt || s_dst[i / kVBlock] < 0) continue;
        const int slot = (i0 + i) & pmask;
        uint8_t *dst = kv_head(c, s_dst[i / kVBlock], h) + page_size * ROW + (int64_t)(slot / kVBlock) * VB + (d * kVBlock + slot % kVBlock) * SZ;
        if (i + PER <= cnt) {
            *reinterpret_cast<uint4 *>(dst) = make_uint4(out[j][0], out[j][1], out[j][2], out[j][3]);
        } else {  // positions past the new length stay as they were
#pragma unroll
            for (int x = 0; x < PER; x++)
                if (i + x < cnt) reinterpret_cast<Val *>(dst)[x] = (Val)(out[j][x * SZ / 4] >> (8 * SZ * (x % (4 / SZ))));
        }
    }
    if (SZ == 1 && tid < 2 * kMove) {
        const int i = tid % kMove, which = tid / kMove;
        if (i < cnt && s_dst[i / kVBlock] >= 0) {
            float f = 0.f;
            if (s_page[i] >= 0)
                f = reinterpret_cast<const float *>(kv_head(c, s_page[i], h) + 2 * page_size * HD)[which * page_size + (s_src[i] & pmask)];
            reinterpret_cast<float *>(kv_head(c, s_dst[i / kVBlock], h) + 2 * page_size * HD)[which * page_size + ((i0 + i) & pmask)] = f;
        }
    }
}

template <int HD, int ROWS>
hipError_t append_rows(int type, const KvArgs &c, int64_t n, const int32_t *start, const float *k,
                       int64_t ldk, const float *v, int64_t ldv, hipStream_t s) {
    const dim3 grid((uint32_t)((n + ROWS - 1) / ROWS), c.n_kv);
    if (type == kKvF16)
        return launch_main(kv_append<kKvF16, HD, ROWS>, grid, dim3(256), 0, s, c, n, start, k, ldk, v, ldv);
    if (type == kKvBF16)
        return launch_main(kv_append<kKvBF16, HD, ROWS>, grid, dim3(256), 0, s, c, n, start, k, ldk, v, ldv);
    return launch_main(kv_append<kKvI8, HD, ROWS>, grid, dim3(256), 0, s, c, n, start, k, ldk, v, ldv);
}

template <int HD>
hipError_t append_hd(int type, const KvArgs &c, int64_t n, const int32_t *start, const float *k,
                     int64_t ldk, const float *v, int64_t ldv, hipStream_t s) {
    // 32 rows once that still gives two workgroups per compute unit (6808 rows
    // of 8 heads of 128: 20.8 us, with 16 rows 23.5, with 64 rows 23.6)
    if (n * c.n_kv >= 32 * 512) return append_rows<HD, 32>(type, c, n, start, k, ldk, v, ldv, s);
    return append_rows<HD, 16>(type, c, n, start, k, ldk, v, ldv, s);
}

template <int HD>
hipError_t move_hd(int type, const KvArgs &c, const EvictArgs &e, hipStream_t s) {
    const dim3 grid((e.keep + kMove - 1) / kMove, c.n_kv, c.n_seq);
    if (type == kKvI8) return launch_main(kv_evict_move<1, HD>, grid, dim3(256), 0, s, c, e);
    return launch_main(kv_evict_move<2, HD>, grid, dim3(256), 0, s, c, e);
}

}  // namespace

hipError_t launch_kv_append(int type, const KvArgs &c, int64_t n, const int32_t *start,
                            const float *k, int64_t ldk, const float *v, int64_t ldv,
                            hipStream_t s) {
    switch (c.hd) {
    case 64: return append_hd<64>(type, c, n, start, k, ldk, v, ldv, s);
    case 96: return append_hd<96>(type, c, n, start, k, ldk, v, ldv, s);
    case 128: return append_hd<128>(type, c, n, start, k, ldk, v, ldv, s);
    case 256: return append_hd<256>(type, c, n, start, k, ldk, v, ldv, s);
    default: return hipErrorInvalidValue;
    }
}

hipError_t launch_kv_evict(int type, const KvArgs &c, const EvictArgs &e, hipStream_t s) {
    const dim3 grid(c.n_kv, c.n_seq);
    // short sequences take the short code (1001 positions: 8.9 -> 6.3 us)
    hipError_t r = e.limit <= kSelThreads
                       ? launch_aux(kv_evict_select<1>, grid, dim3(kSelThreads), 0, s, c, e)
                       : launch_aux(kv_evict_select<8>, grid, dim3(kSelThreads), 0, s, c, e);
    if (r != hipSuccess) return r;
    switch (c.hd) {
    case 64: return move_hd<64>(type, c, e, s);
    case 96: return move_hd<96>(type, c, e, s);
    case 128: return move_hd<128>(type, c, e, s);
    case 256: return move_hd<256>(type, c, e, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmv
