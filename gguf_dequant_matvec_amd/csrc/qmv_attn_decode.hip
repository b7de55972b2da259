// Attention of the last n tokens of each sequence over its paged cache, split
// over the cache's length and joined.
//
// The operation streams K and V once per key-value head; everything else is
// arranged so that this stream never waits:
//  - The rows (tokens x query heads of one key-value head) are the columns of
//    the matrix operands, 16 at a time.  S^T = K Q^T puts one query in each
//    lane column and keys in the accumulator rows; with the K rows handed to
//    the operand in the order key = 8 g + 4 b + i (lane group g, tile b, row
//    i), each lane ends up holding 8 consecutive keys of its query, which is
//    the layout the second product O^T = V^T P^T wants its P operand in.  No
//    value moves between lanes from K to O.
//  - K rows are stored as they are read; V is stored in blocks of 16
//    positions, column-major, so its operand is a 16-byte load as well.  Both
//    go from memory to registers with no LDS in the loop.
//  - The softmax maximum is lazy: O and the sum are rescaled only when some
//    logit exceeds the running maximum by 2^kSlack; the probabilities then
//    are at most 2^(kBias + kSlack), which f16 pieces hold.
// A wave takes every NW-th chunk of its workgroup's piece of the length, the NW
// waves are joined through LDS, and the pieces by a second launch.
// Measured (mean of 60 profiled launches): 32 sequences up to 8150 positions, 32
// / 8 heads of 128, f16, 805 MB of cache: 129 - 130 us (6.2 TB/s; a streaming
// read of the same size reaches 7.1) and 5.0 us for the join; one of 131071 int8
// positions, 277 MB: 54 - 57 and 4.8 us; 301 positions, 9 / 3 heads of 64: 6.3
// us, a chain of latencies.  The same with 4 bits: 227 MB, 56 - 60 us (the least
// of 60 launches 51); 151 MB, 38 us (the least 35; 4.0 TB/s), bound by the
// instructions that make operands of codes, three a pair (with codes taken as they
// are, wrongly, 43 and 29 us at the least); 6.9 us.
#include "qmv_attn.h"
#include "qmv_internal.h"

namespace qmv {

namespace {

template <int TYPE>
constexpr int kChunk = decode_chunk(TYPE);  // positions a wave takes at a time

// Column of element j of the operand of step t in lane group g: 8-bit rows are
// read in 16-byte pieces of two steps where 64 divides the row.  (4-bit rows: the
// order of q4_cols, dword HD / 32 g + t.)
template <int TYPE, int HD>
__device__ __forceinline__ constexpr int col_of(int t, int g) {
    return TYPE == kKvI8 && HD % 64 == 0 ? 64 * (t / 2) + 16 * g + 8 * (t % 2) : 32 * t + 8 * g;
}

// K rows of a chunk in registers: rows + 4 r of a lane's positions, r = 2 u + b
// for tile b of sub-chunk u.
template <int TYPE, int HD>
struct KTile {
    static constexpr int SZ = TYPE == kKvI8 ? 1 : 2;
    static constexpr int R = kChunk<TYPE> / 16;
    static constexpr int W = HD * SZ / 16;  // dwords of a lane's quarter row
    uint32_t k[R][W];

    template <bool NT>
    __device__ __forceinline__ void load(const KvArgs &c, int h, int chunk, int page, int g, int m) {
        const int pos = chunk * kChunk<TYPE> + kChunk<TYPE> / 4 * (m >> 2);
        const int slot = (pos & ((1 << c.page_shift) - 1)) + (m & 3);
        const uint8_t *kp = kv_head(c, page < 0 ? 0 : page, h) + (int64_t)slot * (HD * SZ);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const uint8_t *row = kp + r * 4 * HD * SZ;
            if constexpr (TYPE == kKvI8 && HD % 64 != 0) {
#pragma unroll
                for (int t = 0; t < HD / 32; t++) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(row + 32 * t + 8 * g);
                    k[r][2 * t] = w.x, k[r][2 * t + 1] = w.y;
                }
            } else {
#pragma unroll
                for (int t = 0; t < HD * SZ / 64; t++) {
                    const u32x4 w = load_stream<NT>(row + 64 * t + 16 * g);
                    k[r][4 * t] = w.x, k[r][4 * t + 1] = w.y, k[r][4 * t + 2] = w.z, k[r][4 * t + 3] = w.w;
                }
            }
        }
    }
    template <class Vec>
    __device__ __forceinline__ Vec op(int u, int b, int t) const {
        const uint32_t *r = k[2 * u + b];
        if constexpr (TYPE == kKvI8) {
            const uint2 x = codes_to_f16(r[2 * t]), y = codes_to_f16(r[2 * t + 1]);
            return as_vec<Vec>(U128{{x.x, x.y, y.x, y.y}});
        } else {
            return as_vec<Vec>(U128{{r[4 * t], r[4 * t + 1], r[4 * t + 2], r[4 * t + 3]}});
        }
    }
};

// V columns of a chunk in registers (8 or 16 positions of a lane group in 16
// bytes), and the row scales of an 8-bit cache at those positions.
template <int TYPE, int HD>
struct VTile {
    static constexpr int SZ = TYPE == kKvI8 ? 1 : 2;
    static constexpr int DT = HD / 16;
    uint32_t v[DT][4];
    float ks[TYPE == kKvI8 ? 16 : 1], vs[TYPE == kKvI8 ? 16 : 1];

    template <bool NT>
    __device__ __forceinline__ void load(const KvArgs &c, int h, int chunk, int page, int g, int m) {
        const int pmask = (1 << c.page_shift) - 1;
        const int slot = (chunk * kChunk<TYPE> + kChunk<TYPE> / 4 * g) & pmask;
        const uint8_t *head = kv_head(c, page < 0 ? 0 : page, h) + ((int64_t)(HD * SZ) << c.page_shift);
        const uint8_t *vp = head + (int64_t)(slot / kVBlock) * (HD * kVBlock * SZ) + (m * kVBlock + slot % kVBlock) * SZ;
#pragma unroll
        for (int t = 0; t < DT; t++) {
            const u32x4 w = load_stream<NT>(vp + t * 16 * kVBlock * SZ);
            v[t][0] = w.x, v[t][1] = w.y, v[t][2] = w.z, v[t][3] = w.w;
        }
        if constexpr (TYPE == kKvI8) {
            const float *sc = reinterpret_cast<const float *>(head + ((int64_t)HD << c.page_shift)) + slot;
#pragma unroll
            for (int j = 0; j < 16; j++) ks[j] = sc[j];
            sc += pmask + 1;
#pragma unroll
            for (int j = 0; j < 16; j++) vs[j] = sc[j];
        }
    }
    template <class Vec>
    __device__ __forceinline__ Vec op(int u, int t) const {
        if constexpr (TYPE == kKvI8) {
            const uint2 x = codes_to_f16(v[t][2 * u]), y = codes_to_f16(v[t][2 * u + 1]);
            return as_vec<Vec>(U128{{x.x, x.y, y.x, y.y}});
        } else {
            return as_vec<Vec>(U128{{v[t][0], v[t][1], v[t][2], v[t][3]}});
        }
    }
};

// 4-bit rows: a lane's quarter of a row is HD / 32 dwords, and their scales; at
// 128 columns the quarter is one block.
template <int HD>
struct KTile<kKvQ4, HD> {
    static constexpr int R = kChunk<kKvQ4> / 16, W = HD / 32;
    static constexpr int NB = HD == 96 ? 3 : HD == 256 ? 2 : 1;  // scales (96: one a dword, its blocks change inside)
    uint32_t k[R][W];
    uint16_t d[R][NB];

    template <bool NT>
    __device__ __forceinline__ void load(const KvArgs &c, int h, int chunk, int page, int g, int m) {
        // the chunk's first slot is the wave's, the rest the lane's for all chunks
        const int mask = (1 << c.page_shift) - 1, s0 = chunk * kChunk<kKvQ4> & mask;
        const int mine = (kChunk<kKvQ4> / 4 * (m >> 2) & mask) + (m & 3);
        const uint8_t *head = kv_head(c, page < 0 ? 0 : page, h);
        const uint8_t *kp = head + (int64_t)(s0 + mine) * (HD / 2) + 4 * W * g;
        const uint16_t *dp = reinterpret_cast<const uint16_t *>(head + ((int64_t)HD << c.page_shift)) + (int64_t)(s0 + mine) * (HD / 32);
#pragma unroll
        for (int r = 0; r < R; r++) {
            const uint8_t *row = kp + r * 4 * (HD / 2);
            if constexpr (HD == 96) {
                __builtin_memcpy(k[r], row, 12);
            } else if constexpr (HD == 64) {
                const uint2 w = *reinterpret_cast<const uint2 *>(row);
                k[r][0] = w.x, k[r][1] = w.y;
            } else {
#pragma unroll
                for (int t = 0; t < W / 4; t++) {
                    const u32x4 w = load_stream<NT>(row + 16 * t);
                    k[r][4 * t] = w.x, k[r][4 * t + 1] = w.y, k[r][4 * t + 2] = w.z, k[r][4 * t + 3] = w.w;
                }
            }
#pragma unroll
            for (int j = 0; j < NB; j++) d[r][j] = dp[r * 4 * (HD / 32) + (HD == 96 ? (3 * g + j) / 4 : W * g / 4 + j)];
        }
    }
    template <class Vec>
    __device__ __forceinline__ Vec op(int u, int b, int t) const {
        const uint32_t s = d[2 * u + b][HD == 96 ? t : t / 4];
        return as_vec<Vec>(q4_row8(k[2 * u + b][t], s | s << 16));
    }
};

// ... V: a lane's piece is 16 positions of two columns, 16 apart.  All 16 lanes of
// a group want the same scales, eight dwords of pairs of positions a block: each
// lane loads its share of them (two dwords at 128 columns instead of 32), and they
// are handed round through LDS when they are wanted.
template <int HD>
struct VTile<kKvQ4, HD> {
    static constexpr int DT = HD / 16, NB = HD / 32;
    static constexpr int W = (NB + 1) / 2;  // dwords of scales a lane has: W m .. W m + W - 1 of the 8 NB
    uint32_t v[NB][4], d[W];

    template <bool NT>
    __device__ __forceinline__ void load(const KvArgs &c, int h, int chunk, int page, int g, int m) {
        const int mask = (1 << c.page_shift) - 1, s0 = chunk * kChunk<kKvQ4> & mask;
        const int mine = kChunk<kKvQ4> / 4 * g & mask;
        const uint8_t *head = kv_head(c, page < 0 ? 0 : page, h);
        const uint8_t *vp = head + ((int64_t)(HD / 2) << c.page_shift) + (int64_t)(s0 + mine) * (HD / 2) + 16 * m;
        const int at = W * m < 8 * NB ? W * m : 0;  // (96 columns: 12 lanes have all)
        const uint8_t *dp = head + ((int64_t)(HD + HD / 16 + 2 * (at / 8)) << c.page_shift) + 2 * (s0 + mine) + 4 * (at % 8);
#pragma unroll
        for (int b = 0; b < NB; b++) {
            const u32x4 w = load_stream<NT>(vp + 256 * b);
            v[b][0] = w.x, v[b][1] = w.y, v[b][2] = w.z, v[b][3] = w.w;
        }
        __builtin_memcpy(d, __builtin_assume_aligned(dp, 4 * W), 4 * W);
    }
    // the lane's share to the group's [8 NB] dwords
    __device__ __forceinline__ void share(uint32_t *group, int m) const {
        if (HD != 96 || W * m < 8 * NB) __builtin_memcpy(__builtin_assume_aligned(group + W * m, 4 * W), d, 4 * W);
    }
    // operands of tiles 2 b and 2 b + 1
    template <class Vec>
    __device__ __forceinline__ void op2(const uint32_t *group, int u, int b, Vec &x, Vec &y) const {
        const U128 s = *reinterpret_cast<const U128 *>(group + 8 * b + 4 * u);
        U128 p, q;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t w = v[b][2 * u + j / 2], c = q4_addend(s.w[j]);
            p.w[j] = j % 2 == 0 ? q4_pair<0>(w, s.w[j], c) : q4_pair<2>(w, s.w[j], c);
            q.w[j] = j % 2 == 0 ? q4_pair<1>(w, s.w[j], c) : q4_pair<3>(w, s.w[j], c);
        }
        x = as_vec<Vec>(p), y = as_vec<Vec>(q);
    }
};

// The sequences' chunks, one sequence behind the other, are divided evenly
// among the workgroups of a head that fit the chip at once: a workgroup takes
// the end of one sequence, whole ones, the start of another, as they come.
// Equal numbers of pieces for all sequences would end with the longest one's,
// and a workgroup that starts while others read costs about 5 us of waiting
// for lengths, table and first rows.  A sequence counts kEnter chunks more for
// that.  Workgroup p's piece of sequence s goes to slot p + s: the pairs are a
// staircase, so slots are distinct, and a sequence's are neighbours.
// Measured (32 / 8 heads of 128, f16), against equal numbers of pieces: 32
// sequences of 354 to 8192 positions, evenly spaced, 561 MB, 98 us against 123;
// 63 of 300 and one of 65536 among them, 68 us against 1161; 32 of 6144, 140 us
// against 138.
constexpr int kEnter = 4, kMinPiece = 8;  // chunks

struct Range {
    int s, at, len;  // first sequence, the unit it starts at, its length
    int lo, hi;      // the workgroup's units
};

__device__ __forceinline__ int clamp_len(int len, int limit) { return len < 0 ? 0 : len > limit ? limit : len; }

template <int CK>
__device__ __forceinline__ int units_of(const AttnArgs &a, int len) {
    const int c = visible_chunks(len - (int)a.n, len - 1, a.window, a.sinks, CK).n;
    return (c < 1 ? 1 : c) + kEnter;
}

// Inclusive prefix sum over the 64 lanes: within rows of 16, then across them.
__device__ __forceinline__ int scan64(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);  // row_shr 1, 2, 4, 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // row_bcast 15, 31
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);
    return x;
}

template <int CK>
__device__ __forceinline__ Range find_range(const AttnArgs &a, int p, int lane) {
    const int n_seq = a.c.n_seq;
    int len[4], upto[4];  // of 256 sequences: lengths, and sums of units up to each among its 64
    auto load = [&](int base) {
#pragma unroll
        for (int k = 0; k < 4; k++) len[k] = base + 64 * k + lane < n_seq ? a.c.seq_len[base + 64 * k + lane] : 0;
#pragma unroll
        for (int k = 0; k < 4; k++) {
            if (base + 64 * k >= n_seq) break;
            len[k] = clamp_len(len[k], a.limit);
            upto[k] = scan64(base + 64 * k + lane < n_seq ? units_of<CK>(a, len[k]) : 0);
        }
    };
    int all = 0;
    for (int base = 0; base < n_seq; base += 256) {
        load(base);
#pragma unroll
        for (int k = 0; k < 4; k++)
            if (base + 64 * k < n_seq) all += __builtin_amdgcn_readlane(upto[k], 63);
    }
    int parts = all / kMinPiece;  // (a range is never empty)
    parts = parts < 1 ? 1 : parts > a.parts ? a.parts : parts;
    Range r{-1, 0, 0, 0, 0};
    if (p >= parts) return r;
    const int each = all / parts, more = all - each * parts;  // `more` of them take one unit more
    r.lo = each * p + (p < more ? p : more);
    r.hi = r.lo + each + (p < more ? 1 : 0);
    int first = 0;
    for (int base = 0; base < n_seq; base += 256) {
        if (n_seq > 256) load(base);
#pragma unroll
        for (int k = 0; k < 4; k++) {
            if (base + 64 * k >= n_seq) break;
            const uint64_t past = __ballot(first + upto[k] > r.lo);
            if (past) {
                const int who = __builtin_ctzll(past);
                r.s = base + 64 * k + who;
                r.len = __builtin_amdgcn_readlane(len[k], who);
                r.at = first + (who > 0 ? __builtin_amdgcn_readlane(upto[k], who - 1) : 0);
                return r;
            }
            first += __builtin_amdgcn_readlane(upto[k], 63);
        }
    }
    return r;
}

// 4-bit rows take more instructions a byte than others, so that more waves are
// wanted; the operands of their queries lie in LDS and not in registers, and each
// wave makes one step's of them for all four.
constexpr bool queries_in_lds(int type, int hd, int rt, int nw) {
    return type == kKvQ4 && hd <= 128 && rt == 1 && nw == 4;
}

// PACK, 4-bit caches with few rows: the operand's 16 columns hold more than the
// rows.  2 (at most 8 rows): both f16 pieces of a row's queries, and of its
// probabilities, in columns of their own, so that each product is one matrix
// instruction and not two, and a column's sum is completed by its neighbour's.
// 4 (at most 4 rows): besides, each column's lanes take half of their 16
// positions' probabilities (the other half's are zeros in it).  The outputs'
// columns are added at the end.  Column m: row pack_row, piece pack_piece, half
// m / 8 (PACK 4); the neighbour of the other piece is m + 8, or 7 - m within
// eight, the DPP patterns that cost nothing beside the addition.
template <int PACK>
__device__ __forceinline__ int pack_row(int m) {
    return PACK == 4 ? (m & 4 ? 3 - (m & 3) : m & 3) : PACK == 2 ? m & 7 : m;
}
template <int PACK>
__device__ __forceinline__ int pack_piece(int m) { return PACK == 4 ? (m >> 2) & 1 : m >> 3; }
// a where the mask's bits are set, else b.  (Said with a condition, it becomes a
// choice of an address, and the array goes to memory.)
__device__ __forceinline__ float pick(uint32_t mask, float a, float b) {
    return __builtin_bit_cast(float, (__builtin_bit_cast(uint32_t, a) & mask) | (__builtin_bit_cast(uint32_t, b) & ~mask));
}
template <int PACK>
__device__ __forceinline__ float pack_add(float x) {
    return x + dpp_f32<PACK == 4 ? kDppHalfMirror : kDppRowRor8>(x);
}

template <int TYPE, int HD, int RT, int NW, int PACK, bool ACC, bool RANGES>
__global__ __launch_bounds__(NW * 64, (RANGES && RT == 1) || queries_in_lds(TYPE, HD, RT, NW) ? resident(TYPE, HD) : 1) void attn_decode(AttnArgs a) {
    typedef typename KvOp<TYPE>::Op Op;
    typedef typename Op::Vec Vec;
    constexpr int CK = kChunk<TYPE>, SUB = CK / 32, PER = CK / 4, NP = PACK ? 1 : Op::kPieces;
    static_assert(!PACK || (TYPE == kKvQ4 && RT == 1), "pieces in columns");
    constexpr int KS = HD / 32, DT = HD / 16;
    // With at most 16 rows a head's cache is read by one workgroup, once:
    // nontemporal loads (32 sequences up to 8150 positions of 128 columns: 148
    // -> 136 us).  More rows come with drafted tokens, whose tiles may read
    // the same chunks: ordinary loads (8 x 8 tokens, window 4096: 34 against 37
    // us).  256 columns always take 16-row tiles, one or several of them:
    // ordinary (16 x 8192 positions, 4 tiles: 259 against 334 us, one tile, both
    // with two workgroups a unit: 116 against 113).
    constexpr bool NT = RT == 1 && HD <= 128;
    constexpr bool QL = queries_in_lds(TYPE, HD, RT, NW);
    __shared__ U128 s_q[QL ? KS * NP : 1][QL ? 64 : 1];
    __shared__ float s_big[QL ? NW : 1][16];
    static_assert(!QL || KS <= NW, "a wave for every step");
    __shared__ __align__(16) uint32_t s_d4[TYPE == kKvQ4 ? NW : 1][4][TYPE == kKvQ4 ? HD / 4 : 1];  // scales of a chunk's V
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int h = blockIdx.y / a.tiles, tile = blockIdx.y % a.tiles;
    const KvArgs &c = a.c;
    const int n = (int)a.n;
    const int nrows = n * a.group;
    const int r0 = tile * 16 * RT;
    const int last = r0 + 16 * RT < nrows ? r0 + 16 * RT - 1 : nrows - 1;

    int s = blockIdx.z, at = 0, lo = 0, hi = 0, len = 0;
    if constexpr (RANGES) {
        const Range r = find_range<CK>(a, blockIdx.x, tid & 63);
        // (uniform, which the compiler does not see)
        s = __builtin_amdgcn_readfirstlane(r.s);
        at = __builtin_amdgcn_readfirstlane(r.at);
        lo = __builtin_amdgcn_readfirstlane(r.lo);
        hi = __builtin_amdgcn_readfirstlane(r.hi);
        len = __builtin_amdgcn_readfirstlane(r.len);
        if (s < 0) return;
    } else {
        len = kv_len(c, s, a.limit);
    }
    for (;;) {  // the workgroup's sequences
        // Taken as new each time: lane offsets kept from one sequence to the
        // next would take 20 to 80 registers, and some variants would spill.
        int lane = tid & 63;
        if constexpr (RANGES) asm volatile("" : "+v"(lane));
        const int m = lane & 15, g = lane >> 4;
        // what the rows of this tile see, and the first chunk on its way
        const int pmin = len - n + r0 / a.group, pmax = len - n + last / a.group;
        const Chunks ch = visible_chunks(pmin, pmax, a.window, a.sinks, CK);
        int begin, end, slot, units = 0, next = 0;
        bool opens, closes;  // this piece is the sequence's first, its last
        if constexpr (RANGES) {
            units = units_of<CK>(a, len);
            const int from = at + kEnter, all = units - kEnter;
            opens = lo <= from;
            closes = hi >= at + units;
            begin = opens ? 0 : lo - from;
            end = closes ? all : hi - from;
            if (all != ch.n) {  // a tile whose rows see less than all rows do
                begin = (int)((int64_t)begin * ch.n / all);
                end = (int)((int64_t)end * ch.n / all);
            }
            slot = blockIdx.x + s;
            if (s + 1 < c.n_seq) next = c.seq_len[s + 1];
        } else {
            const int piece = blockIdx.x;
            opens = piece == 0;
            closes = piece == a.splits - 1;
            begin = (int)((int64_t)ch.n * piece / a.splits);
            end = (int)((int64_t)ch.n * (piece + 1) / a.splits);
            slot = s * a.splits + piece;
        }
        const int last_page = len > 0 ? (len - 1) >> c.page_shift : 0;
        const int32_t *table = c.table + (int64_t)s * c.table_ld;
        // Page of a lane group's positions in chunk number i, by the table's entry.
        // The entry is loaded two chunks ahead and looked at only where the page is
        // wanted: a branch or a comparison behind the load would wait for it, and with
        // it for all that was asked for before.
        auto entry_of = [&](int i, int grp) {
            const int pi = (ch.at(i) * CK + PER * grp) >> c.page_shift;
            return table[pi < last_page ? pi : last_page];
        };
        auto page_of = [&](int i, int grp, int pg) {
            const int pi = (ch.at(i) * CK + PER * grp) >> c.page_shift;
            return i < end && pi <= last_page && (uint32_t)pg < (uint32_t)c.n_pages ? pg : -1;
        };
        // (the maximum is that of the unscaled x: x - m then is exact where it
        // matters, however large the logits, and the difference takes the factor)
        float mrun[RT], lrun[RT], qscale[RT];
        f32x4 o[RT][DT];
        // 8-bit: power of two that brings the row scales of V to at most 1, its
        // logarithm (it enters with the exponent) and its inverse
        float vmul = kVmulNone, vlog = TYPE == kKvI8 ? kVlogNone : 0.f, vback = 1.f / kVmulNone;
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
            mrun[rt] = kNoMax;
            qscale[rt] = 1.f;
            lrun[rt] = 0.f;
#pragma unroll
            for (int t = 0; t < DT; t++) o[rt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
        }

        // (with queries in LDS the waves without a chunk make some of them, and read page 0)
        if (QL || begin + wave < end) {
            int i = begin + wave;
            int kentry = entry_of(i, m >> 2), ventry = entry_of(i, g);
            const int kpage = page_of(i, m >> 2, kentry), vpage = page_of(i, g, ventry);
            KTile<TYPE, HD> kt;
            VTile<TYPE, HD> vt;
            bool ok = vpage >= 0;  // the lane group's positions are in a page (not a hole)
            kt.template load<NT>(c, h, ch.at(i), kpage, g, m);
            vt.template load<NT>(c, h, ch.at(i), vpage, g, m);
            kentry = entry_of(i + NW, m >> 2);
            ventry = entry_of(i + NW, g);

            // the rows
            int pos[RT];
            U128 qf[RT][QL ? 1 : KS][NP];
#pragma unroll
            for (int rt = 0; rt < RT; rt++) {
                const int rr = r0 + rt * 16 + pack_row<PACK>(m);
                const bool live = rr < nrows;
                const int j = live ? rr / a.group : 0, hg = live ? rr % a.group : 0;
                pos[rt] = live ? len - n + j : -1;
                const float *qp = a.q + ((int64_t)s * n + j) * a.ldq + (int64_t)(h * a.group + hg) * HD;
                constexpr int KP = QL ? 1 : KS;  // steps that the wave makes
                float f[KP][8];
                float big = 0.f;
#pragma unroll
                for (int tp = 0; tp < KP; tp++) {
                    const int t = QL ? (wave < KS ? wave : 0) : tp;
                    float w[8];
                    if constexpr (TYPE == kKvQ4) {
                        q4_cols(qp, KS * g + t, w);
                    } else {
                        const uint8_t *src = reinterpret_cast<const uint8_t *>(qp + col_of<TYPE, HD>(t, g));
                        const float4 x = __builtin_bit_cast(float4, load16(src)), y = __builtin_bit_cast(float4, load16(src + 16));
                        w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
                    }
#pragma unroll
                    for (int e = 0; e < 8; e++) {
                        f[tp][e] = live ? w[e] * a.q_sign : 0.f;
                        big = fmaxf(big, fabsf(f[tp][e]));
                    }
                }
                // f16 pieces: scale the row by a power of two so that its largest
                // value is in [2^14, 2^15)
                int sh = 0;
                if constexpr (TYPE != kKvBF16) {
                    big = fmaxf(big, __shfl_xor(big, 16));
                    big = fmaxf(big, __shfl_xor(big, 32));
                    if constexpr (QL) {
                        if (g == 0) s_big[wave][m] = big;
                        lds_barrier();
#pragma unroll
                        for (int w = 0; w < NW; w++) big = fmaxf(big, s_big[w][m]);
                    }
                    if (big > 0.f && big < __builtin_inff()) {
                        sh = 15 - __builtin_amdgcn_frexp_expf(big);
                        sh = sh > 100 ? 100 : sh;
                    }
                }
                qscale[rt] = logit_factor(a.scale_log2, sh);
#pragma unroll
                for (int t = 0; t < KP; t++) {
#pragma unroll
                    for (int e = 0; e < 8; e++) f[t][e] = ldexpf(f[t][e], sh);
                    if constexpr (PACK > 0) {
                        U128 both[Op::kPieces];
                        split8<Op>(f[t], both);
#pragma unroll
                        for (int j = 0; j < 4; j++) qf[0][t][0].w[j] = pack_piece<PACK>(m) ? both[1].w[j] : both[0].w[j];
                    } else {
                        split8<Op>(f[t], qf[rt][t]);
                    }
                }
                if constexpr (QL) {
                    if (wave < KS) {
#pragma unroll
                        for (int p = 0; p < NP; p++) s_q[wave * NP + p][lane] = qf[0][0][p];
                    }
                    lds_barrier();
                }
            }

            if (!QL || i < end) for (;;) {
                const bool more = i + NW < end;
                const int kentry2 = entry_of(i + 2 * NW, m >> 2), ventry2 = entry_of(i + 2 * NW, g);
                f32x4 sacc[RT][2 * SUB];
#pragma unroll
                for (int rt = 0; rt < RT; rt++)
#pragma unroll
                    for (int ub = 0; ub < 2 * SUB; ub++) sacc[rt][ub] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int t = 0; t < KS; t++) {
                    if constexpr (QL) {
#pragma unroll
                        for (int p = 0; p < NP; p++) qf[0][0][p] = s_q[t * NP + p][lane];
                    }
#pragma unroll
                    for (int ub = 0; ub < 2 * SUB; ub++) {
                        const Vec kx = kt.template op<Vec>(ub >> 1, ub & 1, t);
#pragma unroll
                        for (int rt = 0; rt < RT; rt++)
#pragma unroll
                            for (int p = 0; p < NP; p++) sacc[rt][ub] = Op::mfma16(kx, as_vec<Vec>(qf[rt][QL ? 0 : t][p]), sacc[rt][ub]);
                    }
                }
                // the K registers are free: the next chunk's K flies during the
                // softmax and the second product, its V during the next first one
                if (more) kt.template load<NT>(c, h, ch.at(i + NW), page_of(i + NW, m >> 2, kentry), g, m);

                const int key0 = ch.at(i) * CK + PER * g;  // the lane group's first position
                // a chunk that every row sees whole needs no masks
                const int c0 = ch.at(i) * CK, c1 = c0 + CK - 1;
                const bool whole = c1 <= pmin && (a.window <= 0 || c0 > pmax - a.window || c1 < a.sinks) && __all(ok);
                if constexpr (TYPE == kKvI8) {
                    float big = 0.f;
#pragma unroll
                    for (int e = 0; e < 16; e++) {
                        if (!whole) {
                            const bool any = ok && key0 + e <= pmax && (a.window <= 0 || key0 + e > pmin - a.window || key0 + e < a.sinks);
                            vt.vs[e] = any ? vt.vs[e] : 0.f;
                        }
                        big = fmaxf(big, fabsf(vt.vs[e]));
                    }
                    if (__any(big * vmul > 1.f)) {
                        big = 0.f;  // again, without infinities
#pragma unroll
                        for (int e = 0; e < 16; e++) big = fmaxf(big, fabsf(vt.vs[e]) < __builtin_inff() ? fabsf(vt.vs[e]) : 0.f);
                        for (int off = 32; off; off >>= 1) big = fmaxf(big, __shfl_xor(big, off));
                        if (big * vmul > 1.f) {
                            int ex = __builtin_amdgcn_frexp_expf(big);
                            ex = ex > 120 ? 120 : ex;
                            const float nm = ldexpf(1.f, -ex);
                            const float r = nm / vmul;
                            vmul = nm;
                            vlog = (float)-ex;
                            vback = ldexpf(1.f, ex);
#pragma unroll
                            for (int rt = 0; rt < RT; rt++)
#pragma unroll
                                for (int t = 0; t < DT; t++) o[rt][t] *= r;
                        }
                    }
                }
                U128 pf[RT][SUB][NP];
#pragma unroll
                for (int rt = 0; rt < RT; rt++) {
                    float x[PER];
#pragma unroll
                    for (int e = 0; e < PER; e++) {
                        x[e] = sacc[rt][e >> 2][e & 3];
                        if constexpr (PACK > 0) x[e] = pack_add<PACK>(x[e]);
                        if constexpr (TYPE == kKvI8) {
                            x[e] *= vt.ks[e];
                            if (!whole) x[e] = ok && sees(pos[rt], key0 + e, a.window, a.sinks) ? x[e] : -__builtin_inff();
                        }
                    }
                    // (one branch: inside the loop above it is one for every position.  The
                    // 8-bit kernel keeps those: 131071 positions 54 us, with one 64)
                    if (TYPE != kKvI8 && !whole) {
                        const int top = ok ? pos[rt] : -1, low = a.window > 0 ? pos[rt] - a.window : -1;
#pragma unroll
                        for (int e = 0; e < PER; e++)
                            x[e] = (key0 + e <= top) & ((key0 + e > low) | (key0 + e < a.sinks)) ? x[e] : -__builtin_inff();
                    }
                    if constexpr (ACC) {
                        const int rr = r0 + rt * 16 + m;
                        if (rr < nrows) {
                            float *lp = a.logits + (((int64_t)s * c.n_kv + h) * nrows + rr) * a.ld_logits + key0;
#pragma unroll
                            for (int e = 0; e < PER; e += 4)
                                *reinterpret_cast<float4 *>(lp + e) = make_float4(x[e] * qscale[rt], x[e + 1] * qscale[rt], x[e + 2] * qscale[rt], x[e + 3] * qscale[rt]);
                        }
                    }
                    float mx = x[0];
#pragma unroll
                    for (int e = 1; e < PER; e++) mx = fmaxf(mx, x[e]);
                    if (__any(minus(mx, mrun[rt]) * qscale[rt] > kSlack || (mrun[rt] == kNoMax && mx > kNoMax))) {
                        mx = fmaxf(mx, __shfl_xor(mx, 16));
                        mx = fmaxf(mx, __shfl_xor(mx, 32));
                        const float mnew = fmaxf(mrun[rt], mx);
                        const float r = exp2_fast((mrun[rt] - mnew) * qscale[rt]);
                        mrun[rt] = mnew;
                        lrun[rt] *= r;
#pragma unroll
                        for (int t = 0; t < DT; t++) o[rt][t] *= r;
                    }
                    const float off = bias_of<TYPE>(a) + vlog;
                    float sum = 0.f;
                    constexpr int MINE = PACK == 4 ? PER / 2 : PER;  // of them the lane takes
                    const uint32_t upper = m & 8 ? ~0u : 0u;
                    if constexpr (PACK == 4) {
#pragma unroll
                        for (int e = 0; e < MINE; e++) x[e] = pick(upper, x[MINE + e], x[e]);
                    }
#pragma unroll
                    for (int e = 0; e < MINE; e++) {
                        const bool hidden = TYPE == kKvI8 && !whole && x[e] == -__builtin_inff();
                        x[e] = exp2_fast(fmaf(minus(x[e], mrun[rt]), qscale[rt], off));
                        sum += x[e];
                        if constexpr (TYPE == kKvI8) x[e] = hidden ? 0.f : x[e] * vt.vs[e];  // (which may be NaN)
                    }
                    lrun[rt] += TYPE == kKvI8 ? sum * vback : sum;
                    if constexpr (PACK > 0) {
#pragma unroll
                        for (int u = 0; u < MINE / 8; u++) {
                            U128 both[Op::kPieces];
                            split8<Op>(x + 8 * u, both);
#pragma unroll
                            for (int j = 0; j < 4; j++) {
                                const uint32_t w = pack_piece<PACK>(m) ? both[1].w[j] : both[0].w[j];
                                if constexpr (PACK == 4) {
                                    pf[0][0][0].w[j] = w & ~upper;
                                    pf[0][1][0].w[j] = w & upper;
                                } else {
                                    pf[0][u][0].w[j] = w;
                                }
                            }
                        }
                    } else {
#pragma unroll
                        for (int u = 0; u < SUB; u++) split8<Op>(x + 8 * u, pf[rt][u]);
                    }
                }
                if constexpr (TYPE == kKvQ4) {  // a 4-bit value is not finite where its block's scale is too large
                    if (!whole) {
                        uint32_t bad = 0;
#pragma unroll
                        for (int j = 0; j < VTile<TYPE, HD>::W; j++) bad |= q4_not_finite(vt.d[j]);
                        if (__any(bad != 0)) {
                            vt.share(s_d4[wave][g], m);
                            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                            for (int u = 0; u < SUB; u++) {
                                U128 seen[RT];
#pragma unroll
                                for (int rt = 0; rt < RT; rt++) seen[rt] = seen8(ok, pos[rt], key0 + 8 * u, a.window, a.sinks);
#pragma unroll
                                for (int b = 0; b < HD / 32; b++) {
                                    U128 marks = *reinterpret_cast<const U128 *>(&s_d4[wave][g][8 * b + 4 * u]);
#pragma unroll
                                    for (int j = 0; j < 4; j++) marks.w[j] = q4_not_finite(marks.w[j]) * kHuge;
#pragma unroll
                                    for (int rt = 0; rt < RT; rt++) {
                                        o[rt][2 * b] = OpBF16::mfma16(as_vec<bf16x8>(marks), as_vec<bf16x8>(seen[rt]), o[rt][2 * b]);
                                        o[rt][2 * b + 1] = OpBF16::mfma16(as_vec<bf16x8>(marks), as_vec<bf16x8>(seen[rt]), o[rt][2 * b + 1]);
                                    }
                                }
                            }
                            __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
                            for (int j = 0; j < VTile<TYPE, HD>::W; j++) vt.d[j] &= ~(q4_not_finite(vt.d[j]) * 0xFFFFu);
                        }
                    }
                    vt.share(s_d4[wave][g], m);
                    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
                } else if constexpr (TYPE != kKvI8) {
                    if (!whole) {
                        uint32_t bad = 0;
#pragma unroll
                        for (int t = 0; t < DT; t++)
#pragma unroll
                            for (int j = 0; j < 4; j++) bad |= not_finite<Op>(vt.v[t][j]);
                        if (__any(bad != 0)) {
                            U128 seen[RT];
#pragma unroll
                            for (int rt = 0; rt < RT; rt++) seen[rt] = seen8(ok, pos[rt], key0, a.window, a.sinks);
#pragma unroll
                            for (int t = 0; t < DT; t++) {
                                U128 marks;
#pragma unroll
                                for (int j = 0; j < 4; j++) {
                                    const uint32_t b = not_finite<Op>(vt.v[t][j]);
                                    vt.v[t][j] &= ~(b * 0xFFFFu);
                                    marks.w[j] = b * kHuge;
                                }
#pragma unroll
                                for (int rt = 0; rt < RT; rt++)
                                    o[rt][t] = OpBF16::mfma16(as_vec<bf16x8>(marks), as_vec<bf16x8>(seen[rt]), o[rt][t]);
                            }
                        }
                    }
                }
#pragma unroll
                for (int u = 0; u < SUB; u++) {
                    if constexpr (TYPE == kKvQ4) {
#pragma unroll
                        for (int b = 0; b < HD / 32; b++) {
                            Vec x, y;
                            vt.template op2<Vec>(s_d4[wave][g], u, b, x, y);
#pragma unroll
                            for (int rt = 0; rt < RT; rt++)
#pragma unroll
                                for (int p = 0; p < NP; p++) {
                                    o[rt][2 * b] = Op::mfma16(x, as_vec<Vec>(pf[rt][u][p]), o[rt][2 * b]);
                                    o[rt][2 * b + 1] = Op::mfma16(y, as_vec<Vec>(pf[rt][u][p]), o[rt][2 * b + 1]);
                                }
                        }
                    } else {
#pragma unroll
                        for (int t = 0; t < DT; t++) {
                            const Vec vx = vt.template op<Vec>(u, t);
#pragma unroll
                            for (int rt = 0; rt < RT; rt++)
#pragma unroll
                                for (int p = 0; p < NP; p++) o[rt][t] = Op::mfma16(vx, as_vec<Vec>(pf[rt][u][p]), o[rt][t]);
                        }
                    }
                }
                const int next_vpage = page_of(i + NW, g, ventry);
                if (more) vt.template load<NT>(c, h, ch.at(i + NW), next_vpage, g, m);
                if (!more) break;
                i += NW;
                ok = next_vpage >= 0;
                kentry = kentry2;
                ventry = ventry2;
            }
        }

        // where row rr's sums go: to the outputs, divided, or, where the sequence has
        // other pieces, as a piece, with its maximum and sum (written by `first`)
        const bool direct = opens && closes && !ACC;
        auto row_of = [&](int rr, bool first, float mx, float l, float &mul) {
            mul = direct ? (l == 0.f ? 0.f : 1.f / l) : 1.f;  // a row that sees nothing: zeros
            const int64_t row = (int64_t)(direct ? s : slot) * n + rr / a.group;
            const int64_t at = row * a.n_heads + h * a.group + rr % a.group;
            if (!direct && first) a.part_ml[at] = make_float2(mx, l);
            return (direct ? a.out : a.part_o) + at * HD;
        };
        if (RANGES && blockIdx.y == 0 && tid == 0) {
            if (opens) a.share[s].x = slot;
            if (closes) a.share[s].y = slot;
        }
        if constexpr (PACK > 0) {
            // join the waves: their few rows' sums side by side in LDS, four columns a
            // thread after one barrier
            constexpr int ROWS = PACK == 4 ? 4 : 8, RS = HD / 4 + 1;
            __shared__ float s_m[NW][ROWS], s_l[NW][ROWS];
            __shared__ f32x4 s_o[NW][ROWS][RS];
            if constexpr (PACK == 4) lrun[0] += dpp_f32<kDppRowRor8>(lrun[0]);
            lrun[0] += __shfl_xor(lrun[0], 16);
            lrun[0] += __shfl_xor(lrun[0], 32);
            if (mrun[0] != kNoMax) mrun[0] *= qscale[0];
#pragma unroll
            for (int t = 0; t < DT; t++) {
#pragma unroll
                for (int e = 0; e < 4; e++) {
                    o[0][t][e] = pack_add<PACK>(o[0][t][e]);
                    if constexpr (PACK == 4) o[0][t][e] += dpp_f32<kDppRowRor8>(o[0][t][e]);
                }
                if (m < ROWS) s_o[wave][m][4 * t + g] = o[0][t];
            }
            if (m < ROWS && g == 0) s_m[wave][m] = mrun[0], s_l[wave][m] = lrun[0];
            lds_barrier();
            for (int e = tid; e < nrows * (HD / 4); e += NW * 64) {
                const int rr = e / (HD / 4), d = e % (HD / 4);
                float mm = kNoMax, l = 0.f, mul;
#pragma unroll
                for (int w = 0; w < NW; w++) mm = fmaxf(mm, s_m[w][rr]);
                f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int w = 0; w < NW; w++) {
                    const float r = exp2_fast(s_m[w][rr] - mm);
                    l += s_l[w][rr] * r;
                    v += s_o[w][rr][d] * r;
                }
                float *dst = row_of(rr, d == 0, mm, l, mul);
                v *= mul;
                __builtin_memcpy(dst + 4 * d, &v, 16);
            }
        } else {
            // join the waves: a common maximum, then the partial sums two by two
            __shared__ float s_m[NW][RT * 16], s_l[NW][RT * 16];
            __shared__ f32x4 s_o[2][RT * DT * 64];
#pragma unroll
            for (int rt = 0; rt < RT; rt++) {
                lrun[rt] += __shfl_xor(lrun[rt], 16);
                lrun[rt] += __shfl_xor(lrun[rt], 32);
                if (mrun[rt] != kNoMax) mrun[rt] *= qscale[rt];
                if (g == 0) s_m[wave][rt * 16 + m] = mrun[rt];
            }
            __syncthreads();
#pragma unroll
            for (int rt = 0; rt < RT; rt++) {
                float mm = kNoMax;
                for (int w = 0; w < NW; w++) mm = fmaxf(mm, s_m[w][rt * 16 + m]);
                // (a NaN maximum cannot be: fmaxf drops NaN; a NaN sum stays)
                const float r = exp2_fast(mrun[rt] - mm);
                mrun[rt] = mm;
                lrun[rt] *= r;
                if constexpr (TYPE == kKvI8) {
                    lrun[rt] *= a.unit;
                    const float back = vback * a.unit;  // a power of two (with r it might be subnormal and lose bits)
#pragma unroll
                    for (int t = 0; t < DT; t++) o[rt][t] *= back;
                }
                if (g == 0) s_l[wave][rt * 16 + m] = lrun[rt];
#pragma unroll
                for (int t = 0; t < DT; t++) o[rt][t] *= r;
            }
            for (int from = NW - 2; from >= 0; from -= 2) {
                // waves from, from + 1 add to the two before them; last 1 to 0
                const int w0 = from > 0 ? from : 1, n_from = from > 0 ? 2 : 1, to = from > 0 ? from - 2 : 0;
                if (wave >= w0 && wave < w0 + n_from) {
#pragma unroll
                    for (int rt = 0; rt < RT; rt++)
#pragma unroll
                        for (int t = 0; t < DT; t++) s_o[wave - w0][(rt * DT + t) * 64 + lane] = o[rt][t];
                }
                __syncthreads();
                if (wave >= to && wave < to + n_from) {
#pragma unroll
                    for (int rt = 0; rt < RT; rt++)
#pragma unroll
                        for (int t = 0; t < DT; t++) o[rt][t] += s_o[wave - to][(rt * DT + t) * 64 + lane];
                }
                __syncthreads();
            }
            if (wave == 0) {
#pragma unroll
                for (int rt = 0; rt < RT; rt++) {
                    const int rr = r0 + rt * 16 + m;
                    if (rr >= nrows) continue;
                    float l = 0.f;
                    for (int w = 0; w < NW; w++) l += s_l[w][rt * 16 + m];
                    float mul;
                    float *dst = row_of(rr, g == 0, mrun[rt], l, mul);
#pragma unroll
                    for (int t = 0; t < DT; t++) {
                        const f32x4 v = o[rt][t] * mul;
                        __builtin_memcpy(dst + 16 * t + 4 * g, &v, 16);
                    }
                }
            }
        }
        if constexpr (!RANGES) return;
        at += units;
        s++;
        if (s >= c.n_seq || at + kEnter >= hi) return;
        len = clamp_len(__builtin_amdgcn_readfirstlane(next), a.limit);
        __syncthreads();  // the joined waves' memory is used again
    }
}

// First and last slot of sequence s.
__device__ __forceinline__ int2 slots_of(const AttnArgs &a, int s) {
    return a.parts ? a.share[s] : make_int2(s * a.splits, (s + 1) * a.splits - 1);
}

// Joins the pieces of row r of sequence s.
template <int HD>
__device__ __forceinline__ void join_pieces(const AttnArgs &a, int s, int r, int2 sh) {
    const int64_t per = a.n * a.n_heads;
    join_row<HD>(a, s * per + r, sh.x * per + r, per, sh.y - sh.x + 1);
}

template <int HD>
__global__ __launch_bounds__(256) void attn_join_pieces(AttnArgs a) {
    const int2 sh = slots_of(a, blockIdx.y);
    if (sh.x != sh.y) join_pieces<HD>(a, blockIdx.y, blockIdx.x, sh);  // else the one workgroup wrote the row
}

// acc[s][h][key] += sum over the rows of 2^(x - m) / l, rows in order.
// The first part_rows workgroups join the pieces of a row each, the others take
// 256 positions of a key-value head each: one launch for both (4 sequences of
// 4352 positions: 4.8 us, latency; it reads the logits once).
template <int TYPE, int HD>
__global__ __launch_bounds__(256) void attn_join_weights(AttnArgs a, int rt16) {
    constexpr int CK = kChunk<TYPE>;
    if (blockIdx.x < a.part_rows) {
        const uint32_t per = (uint32_t)(a.n * a.n_heads), s = blockIdx.x / per;
        join_pieces<HD>(a, s, blockIdx.x % per, slots_of(a, s));
        return;
    }
    const int per = (a.limit + 255) / 256;  // workgroups a head
    const int64_t unit = (int64_t)blockIdx.x - a.part_rows;
    const int block = (int)(unit % per), h = (int)(unit / per % a.c.n_kv), s = (int)(unit / per / a.c.n_kv);
    const int len = kv_len(a.c, s, a.limit);
    const int n = (int)a.n, nrows = n * a.group;
    if ((int64_t)block * 256 >= len) return;
    const int key = block * 256 + threadIdx.x;
    const int64_t head = (int64_t)s * a.c.n_kv + h;
    const int2 sh = slots_of(a, s);
    const int count = sh.y - sh.x + 1;
    const int64_t per_seq = (int64_t)n * a.n_heads;
    __shared__ float s_m[16], s_r[16];
    float sum = 0.f;
    for (int r0 = 0; r0 < nrows; r0 += 16) {
        __syncthreads();
        const int row = threadIdx.x >> 4, l16 = threadIdx.x & 15;
        if (r0 + row < nrows) {
            const int rr = r0 + row;
            const float2 *ml = a.part_ml + sh.x * per_seq + (int64_t)(rr / a.group) * a.n_heads + h * a.group + rr % a.group;
            float mm = kNoMax, l = 0.f;
            for (int i = l16; i < count; i += 16) mm = fmaxf(mm, ml[i * per_seq].x);
            for (int off = 8; off; off >>= 1) mm = fmaxf(mm, __shfl_xor(mm, off, 16));
            for (int i = l16; i < count; i += 16) {
                const float2 x = ml[i * per_seq];
                l += exp2_fast(x.x - mm) * x.y;
            }
            for (int off = 8; off; off >>= 1) l += __shfl_xor(l, off, 16);
            if (l16 == 0) {
                s_m[row] = mm;
                s_r[row] = l == 0.f ? 0.f : exp2_fast(sum_bias_of<TYPE>(a)) / l;
            }
        }
        __syncthreads();
        if (key < len) {
            for (int i = 0; i < 16 && r0 + i < nrows; i++) {
                // what this row's tile read: other logits were not written
                const int t0 = (r0 + i) / rt16 * rt16;
                const int t1 = t0 + rt16 < nrows ? t0 + rt16 - 1 : nrows - 1;
                const int pmin = len - n + t0 / a.group, pmax = len - n + t1 / a.group;
                const Chunks ch = visible_chunks(pmin, pmax, a.window, a.sinks, CK);
                const int k = key / CK;
                const bool read = k < ch.sink || (k >= ch.win0 && k < ch.win0 + (ch.n - ch.sink));
                if (read && s_r[i] != 0.f) {
                    const float x = a.logits[(head * nrows + r0 + i) * a.ld_logits + key];
                    if (x != -__builtin_inff()) sum += exp2_fast(x - s_m[i]) * s_r[i];  // (0 times a NaN row's factor)
                }
            }
        }
    }
    if (key < len) a.acc[head * a.ld_acc + key] += sum;
}

template <int TYPE, int HD, int RT, int NW, int PACK, bool RANGES>
hipError_t launch_packed(const AttnArgs &a, const AttnPlan &p, hipStream_t s) {
    const dim3 grid(RANGES ? p.parts : p.splits, a.c.n_kv * p.tiles, RANGES ? 1 : a.c.n_seq);
    if (a.acc) return launch_main(attn_decode<TYPE, HD, RT, NW, PACK, true, RANGES>, grid, dim3(NW * 64), 0, s, a);
    return launch_main(attn_decode<TYPE, HD, RT, NW, PACK, false, RANGES>, grid, dim3(NW * 64), 0, s, a);
}

template <int TYPE, int HD, int RT, int NW, bool RANGES>
hipError_t launch_main_of(const AttnArgs &a, const AttnPlan &p, hipStream_t s) {
    if constexpr (TYPE == kKvQ4 && RT == 1) {
        const int64_t rows = a.n * a.group;
        if (rows <= 4) return launch_packed<TYPE, HD, RT, NW, 4, RANGES>(a, p, s);
        if (rows <= 8) return launch_packed<TYPE, HD, RT, NW, 2, RANGES>(a, p, s);
    }
    return launch_packed<TYPE, HD, RT, NW, 0, RANGES>(a, p, s);
}

template <int TYPE, int HD, int RT, int NW>
hipError_t launch_typed(const AttnArgs &a, const AttnPlan &p, hipStream_t s) {
    hipError_t e = hipErrorInvalidValue;
    if (!p.parts)
        e = launch_main_of<TYPE, HD, RT, NW, false>(a, p, s);
    else if constexpr (RT == 2 || NW == 4)  // 16-row tiles of eight waves are for short calls
        e = launch_main_of<TYPE, HD, RT, NW, true>(a, p, s);
    if (e != hipSuccess) return e;
    if (a.acc) {
        const int64_t blocks = p.part_rows + (int64_t)a.c.n_seq * a.c.n_kv * ((a.limit + 255) / 256);
        return launch_aux(attn_join_weights<TYPE, HD>, dim3((uint32_t)blocks), dim3(256), 0, s, a, 16 * RT);
    }
    if (p.slots == a.c.n_seq) return hipSuccess;
    return launch_aux(attn_join_pieces<HD>, dim3((uint32_t)(a.n * a.n_heads), a.c.n_seq), dim3(256), 0, s, a);
}

template <int TYPE, int HD, int RT>
hipError_t launch_rt(const AttnArgs &a, const AttnPlan &p, hipStream_t s) {
    // 32-row tiles take eight waves wherever they fit, 16-row tiles either
    if constexpr (eight_fit(TYPE, HD, RT)) {
        if (RT == 2 || p.waves == 8) return launch_typed<TYPE, HD, RT, 8>(a, p, s);
    }
    if constexpr (RT == 1 || !eight_fit(TYPE, HD, RT)) return launch_typed<TYPE, HD, RT, 4>(a, p, s);
    return hipErrorInvalidValue;
}

template <int TYPE, int HD>
hipError_t launch_hd(const AttnArgs &a, const AttnPlan &p, hipStream_t s) {
    if constexpr (HD <= 128) {
        if (p.rt == 2) return launch_rt<TYPE, HD, 2>(a, p, s);
    }
    return launch_rt<TYPE, HD, 1>(a, p, s);
}

template <int TYPE>
hipError_t launch_type(const AttnArgs &a, const AttnPlan &p, hipStream_t s) {
    switch (a.c.hd) {
    case 64: return launch_hd<TYPE, 64>(a, p, s);
    case 96: return launch_hd<TYPE, 96>(a, p, s);
    case 128: return launch_hd<TYPE, 128>(a, p, s);
    case 256: return launch_hd<TYPE, 256>(a, p, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_attn_decode(int type, const AttnArgs &a, const AttnPlan &p, hipStream_t s) {
    switch (type) {
    case kKvF16: return launch_type<kKvF16>(a, p, s);
    case kKvBF16: return launch_type<kKvBF16>(a, p, s);
    case kKvI8: return launch_type<kKvI8>(a, p, s);
    case kKvQ4: return launch_type<kKvQ4>(a, p, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmv
