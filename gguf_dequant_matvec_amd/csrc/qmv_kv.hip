// Writing the paged key-value cache: appending new tokens' rows, and cutting
// a cache down to the positions with the largest accumulated weight.
#include "qmv_device.h"
#include "qmv_internal.h"
#include "qmv_kv.h"

namespace qmv {

namespace {

// ---- append -----------------------------------------------------------------
// A workgroup takes 16 consecutive rows of one key-value head.  K rows are
// rounded and stored as they come (16 bytes a thread); V goes through LDS,
// because a V block keeps the 16 positions of one column next to each other:
// lanes run over the rows first, so the 16 two-byte stores of a column land in
// one 32-byte run.  Bound by the f32 reads.
constexpr int kAppendRows = 16;

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

template <int TYPE, int HD>
__global__ __launch_bounds__(256) void kv_append(KvArgs c, int64_t n, const int32_t *start,
                                                 const float *__restrict__ k, int64_t ldk,
                                                 const float *__restrict__ v, int64_t ldv) {
    constexpr int SZ = TYPE == kKvI8 ? 1 : 2;
    constexpr int PIECES = HD / 8;  // 8 columns a thread
    __shared__ int s_page[kAppendRows], s_slot[kAppendRows];
    __shared__ float s_v[kAppendRows][HD + 1];
    __shared__ float s_d[2][kAppendRows];
    const int tid = threadIdx.x, h = blockIdx.y;
    const int64_t row0 = (int64_t)blockIdx.x * kAppendRows;

    if (tid < kAppendRows) {
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
    if (TYPE == kKvI8) {
        // row maxima: 16 lanes a row
        const int i = tid >> 4, l = tid & 15;
        float mk = 0.f, mv = 0.f;
        if (row0 + i < n) {
            const float *kr = k + (row0 + i) * ldk + (int64_t)h * HD;
            const float *vr = v + (row0 + i) * ldv + (int64_t)h * HD;
            for (int d = l; d < HD; d += 16) {
                // (x > m keeps m for a NaN: the sum of the row's NaN with 0 * x stays NaN below)
                mk = fabsf(kr[d]) > mk || kr[d] != kr[d] ? fabsf(kr[d]) : mk;
                mv = fabsf(vr[d]) > mv || vr[d] != vr[d] ? fabsf(vr[d]) : mv;
            }
        }
        for (int o = 8; o; o >>= 1) {
            const float a = __shfl_xor(mk, o, 16), b = __shfl_xor(mv, o, 16);
            mk = a > mk || a != a ? a : mk;
            mv = b > mv || b != b ? b : mv;
        }
        if (l == 0) {
            s_d[0][i] = mk / 127.f;
            s_d[1][i] = mv / 127.f;
        }
    }
    for (int e = tid; e < kAppendRows * HD; e += 256) {
        const int i = e / HD, d = e % HD;
        if (row0 + i < n) s_v[i][d] = v[(row0 + i) * ldv + (int64_t)h * HD + d];
    }
    __syncthreads();

    const int64_t page_size = 1ll << c.page_shift;
    for (int e = tid; e < kAppendRows * PIECES; e += 256) {
        const int i = e / PIECES, p = e % PIECES;
        if (s_page[i] < 0) continue;
        const uint8_t *src = reinterpret_cast<const uint8_t *>(k + (row0 + i) * ldk + (int64_t)h * HD + p * 8);
        const float4 x = __builtin_bit_cast(float4, load16(src));
        const float4 y = __builtin_bit_cast(float4, load16(src + 16));
        const float f[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        uint8_t *dst = kv_head(c, s_page[i], h) + ((int64_t)s_slot[i] * HD + p * 8) * SZ;
        uint32_t w[4] = {0, 0, 0, 0};
        if constexpr (TYPE == kKvI8) {
            for (int j = 0; j < 8; j++) w[j >> 2] |= (uint32_t)(kv_code(f[j], s_d[0][i]) & 0xFF) << (8 * (j & 3));
            *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        } else {
            for (int j = 0; j < 8; j++) w[j >> 1] |= kv_round<TYPE>(f[j]) << (16 * (j & 1));
            *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
    for (int e = tid; e < kAppendRows * HD; e += 256) {
        const int i = e % kAppendRows, d = e / kAppendRows;
        if (s_page[i] < 0) continue;
        const int slot = s_slot[i];
        uint8_t *dst = kv_head(c, s_page[i], h) + page_size * HD * SZ +
                       ((int64_t)(slot / kVBlock) * (HD * kVBlock) + d * kVBlock + slot % kVBlock) * SZ;
        if constexpr (TYPE == kKvI8)
            *reinterpret_cast<int8_t *>(dst) = (int8_t)kv_code(s_v[i][d], s_d[1][i]);
        else
            *reinterpret_cast<uint16_t *>(dst) = (uint16_t)kv_round<TYPE>(s_v[i][d]);
    }
    if (TYPE == kKvI8 && tid < 2 * kAppendRows) {
        const int i = tid & 15, which = tid >> 4;
        if (s_page[i] >= 0) {
            float *sc = reinterpret_cast<float *>(kv_head(c, s_page[i], h) + 2 * page_size * HD);
            sc[which * page_size + s_slot[i]] = s_d[which][i];
        }
    }
}

// ---- eviction: choosing -------------------------------------------------------
// One workgroup per sequence and key-value head.  The m-th largest score of
// the middle positions is found by four 8-bit radix passes over an
// order-preserving integer key (counts in LDS), then one ordered pass writes
// the kept positions by prefix sums; among equal scores at the border the
// lowest positions are kept.
constexpr int kSelThreads = 1024;
constexpr int kSelWaves = kSelThreads / 64;

__device__ __forceinline__ uint32_t score_key(float v) {
    if (v != v) return 0xFFFFFFFFu;   // NaN ranks above everything
    return float_key(v + 0.f);        // -0 counts as +0
}

__global__ __launch_bounds__(kSelThreads) void kv_evict_select(KvArgs c, EvictArgs e) {
    const int h = blockIdx.x, s = blockIdx.y, tid = threadIdx.x;
    const int lane = tid & 63, wave = tid >> 6;
    const int len = kv_len(c, s, e.limit);
    const int64_t head = (int64_t)s * c.n_kv + h;
    int32_t *kept = e.kept + head * e.keep;
    float *acc_out = e.acc_out + head * e.ld_out;
    const float *acc = e.acc + head * e.ld_acc;
    const int out_len = len < e.keep ? len : e.keep;
    if (h == 0 && tid == 0) e.len_out[s] = out_len;
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

    __shared__ int hist[256];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    uint32_t prefix = 0, mask = 0;
    int left = m;  // rank still to go inside the current prefix
    if (m > 0) {
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            for (int i = lo + tid; i < hi; i += kSelThreads) {
                const uint32_t key = score_key(acc[i]);
                if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
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
    __shared__ int w_ties[kSelWaves], w_kept[kSelWaves];
    int ties_before = 0, kept_before = 0;
    for (int base = 0; base < len; base += kSelThreads) {
        const int i = base + tid;
        bool sure = false, tie = false;
        float v = 0.f;
        if (i < len) {
            v = acc[i];
            if (i < lo || i >= hi) {
                sure = true;
            } else if (m > 0) {
                const uint32_t key = score_key(v);
                sure = key > prefix;
                tie = key == prefix;
            }
        }
        const uint64_t below = (1ull << lane) - 1;
        const uint64_t tb = __ballot(tie);
        if (lane == 0) w_ties[wave] = __popcll(tb);
        __syncthreads();
        int rank = ties_before + __popcll(tb & below), all_ties = 0;
        for (int w = 0; w < kSelWaves; w++) {
            if (w < wave) rank += w_ties[w];
            all_ties += w_ties[w];
        }
        const bool keep = sure || (tie && rank < left);
        const uint64_t kb = __ballot(keep);
        if (lane == 0) w_kept[wave] = __popcll(kb);
        __syncthreads();
        int at = kept_before + __popcll(kb & below), all_kept = 0;
        for (int w = 0; w < kSelWaves; w++) {
            if (w < wave) at += w_kept[w];
            all_kept += w_kept[w];
        }
        if (keep && at < e.keep) {
            kept[at] = i;
            acc_out[at] = v;
        }
        ties_before += all_ties;
        kept_before += all_kept;
        __syncthreads();
    }
}

// ---- eviction: moving -----------------------------------------------------------
// A workgroup fills one V block (16 positions) of the destination.  K rows are
// copied as they are; for V it reads each source block once (kept positions
// are in order, so the 16 sources lie in few blocks) and picks the kept
// columns into LDS, from where the new block leaves in one run.
template <int SZ, int HD>
__global__ __launch_bounds__(256) void kv_evict_move(KvArgs c, EvictArgs e) {
    const int h = blockIdx.y, s = blockIdx.z, tid = threadIdx.x;
    const int len = kv_len(c, s, e.limit);
    const int out_len = len < e.keep ? len : e.keep;
    const int i0 = blockIdx.x * kVBlock;
    if (i0 >= out_len) return;
    const int cnt = out_len - i0 < kVBlock ? out_len - i0 : kVBlock;
    const int64_t page_size = 1ll << c.page_shift;
    const int dpg = e.dst[(int64_t)s * e.dst_ld + (i0 >> c.page_shift)];
    if ((uint32_t)dpg >= (uint32_t)c.n_pages) return;
    uint8_t *dst = kv_head(c, dpg, h);
    const int slot0 = i0 & (int)(page_size - 1);

    __shared__ int s_src[kVBlock], s_page[kVBlock];
    __shared__ __align__(16) uint8_t s_v[HD * kVBlock * SZ];
    if (tid < kVBlock) {
        int src = -1, page = -1;
        if (tid < cnt) {
            src = e.kept[((int64_t)s * c.n_kv + h) * e.keep + i0 + tid];
            page = kv_page(c, s, src);
        }
        s_src[tid] = src;
        s_page[tid] = page;
    }
    // a block that is not filled keeps its other positions
    constexpr int VB = HD * kVBlock * SZ;  // bytes of a V block
    uint8_t *vdst = dst + page_size * HD * SZ + (int64_t)(slot0 / kVBlock) * VB;
    if (cnt < kVBlock)
        for (int o = tid * 16; o < VB; o += 256 * 16) *reinterpret_cast<uint4 *>(s_v + o) = *reinterpret_cast<const uint4 *>(vdst + o);
    __syncthreads();

    constexpr int ROW = HD * SZ;
    for (int o = tid * 16; o < cnt * ROW; o += 256 * 16) {
        const int i = o / ROW, b = o % ROW;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (s_page[i] >= 0)
            w = *reinterpret_cast<const uint4 *>(kv_head(c, s_page[i], h) + (s_src[i] & (page_size - 1)) * ROW + b);
        *reinterpret_cast<uint4 *>(dst + (int64_t)(slot0 + i) * ROW + b) = w;
    }
    for (int a = 0; a < cnt;) {
        // sources a .. z-1 share one source block
        int z = a + 1;
        while (z < cnt && s_src[z] / kVBlock == s_src[a] / kVBlock) z++;
        const uint8_t *vsrc = nullptr;
        if (s_page[a] >= 0)
            vsrc = kv_head(c, s_page[a], h) + page_size * HD * SZ +
                   (int64_t)((s_src[a] & (int)(page_size - 1)) / kVBlock) * VB;
        for (int o = tid * 16; o < VB; o += 256 * 16) {
            uint4 w = make_uint4(0, 0, 0, 0);
            if (vsrc) w = *reinterpret_cast<const uint4 *>(vsrc + o);
            constexpr int PER = 16 / SZ;  // positions in 16 bytes
            const int d = o / (kVBlock * SZ), p0 = (o / SZ) % kVBlock;
            const uint32_t wd[4] = {w.x, w.y, w.z, w.w};
            for (int i = a; i < z; i++) {
                const int p = s_src[i] % kVBlock - p0;
                if (p < 0 || p >= PER) continue;
                if constexpr (SZ == 2) {
                    const uint32_t x = p < 4 ? (p < 2 ? wd[0] : wd[1]) : (p < 6 ? wd[2] : wd[3]);
                    reinterpret_cast<uint16_t *>(s_v)[d * kVBlock + i] = (uint16_t)(x >> (16 * (p & 1)));
                } else {
                    const uint32_t x = p < 8 ? (p < 4 ? wd[0] : wd[1]) : (p < 12 ? wd[2] : wd[3]);
                    s_v[d * kVBlock + i] = (uint8_t)(x >> (8 * (p & 3)));
                }
            }
        }
        a = z;
    }
    __syncthreads();
    for (int o = tid * 16; o < VB; o += 256 * 16) *reinterpret_cast<uint4 *>(vdst + o) = *reinterpret_cast<const uint4 *>(s_v + o);
    if (SZ == 1 && tid < 2 * cnt) {
        const int i = tid % cnt, which = tid / cnt;
        float f = 0.f;
        if (s_page[i] >= 0)
            f = reinterpret_cast<const float *>(kv_head(c, s_page[i], h) + 2 * page_size * HD)[which * page_size + (s_src[i] & (page_size - 1))];
        reinterpret_cast<float *>(dst + 2 * page_size * HD)[which * page_size + slot0 + i] = f;
    }
}

template <int HD>
hipError_t append_hd(int type, const KvArgs &c, int64_t n, const int32_t *start, const float *k,
                     int64_t ldk, const float *v, int64_t ldv, hipStream_t s) {
    const dim3 grid((uint32_t)((n + kAppendRows - 1) / kAppendRows), c.n_kv);
    if (type == kKvF16)
        return launch_main(kv_append<kKvF16, HD>, grid, dim3(256), 0, s, c, n, start, k, ldk, v, ldv);
    if (type == kKvBF16)
        return launch_main(kv_append<kKvBF16, HD>, grid, dim3(256), 0, s, c, n, start, k, ldk, v, ldv);
    return launch_main(kv_append<kKvI8, HD>, grid, dim3(256), 0, s, c, n, start, k, ldk, v, ldv);
}

template <int HD>
hipError_t move_hd(int type, const KvArgs &c, const EvictArgs &e, hipStream_t s) {
    const dim3 grid((e.keep + kVBlock - 1) / kVBlock, c.n_kv, c.n_seq);
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
    hipError_t r = launch_aux(kv_evict_select, dim3(c.n_kv, c.n_seq), dim3(kSelThreads), 0, s, c, e);
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
