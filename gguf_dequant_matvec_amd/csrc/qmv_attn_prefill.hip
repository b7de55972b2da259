// Causal attention of prompts over a paged cache, with an optional sliding
// window and first tokens that stay visible.
//
// Compute-bound: 4 * visible * head_dim operations a row, each product taking
// two f16 (three bf16) matrix instructions because queries and probabilities
// are f32.  A workgroup takes 128 rows (tokens x query heads of one key-value
// head, so the heads of a group share every K and V tile), 32 per wave, and
// walks over the visible chunks of 64 positions.  A chunk is staged through
// two LDS buffers by all four waves, wave w taking positions 16 w .. 16 w + 15
// (one page, one V block: 1 KB runs), while the previous chunk is computed.
// The products are S^T = K Q^T and O^T = V^T P^T: K rows lie in LDS in the
// order in which the 32x32 operand takes them so that each lane's
// accumulators are 8 consecutive positions of its query, the operand layout
// of P, and no value moves between lanes.  K rows are swizzled by 16-byte
// pieces and V keeps the cache's block layout; both are read without bank
// conflicts.  Measured: 4096 tokens, 32 / 8 heads of 128, f16: 250 - 274 us,
// 1.0 - 1.1 PFLOP/s of operand work where library products reach 1.15; int8
// prompts in a window of 1024, heads of 64: 258 - 273 us, bound by the softmax's
// vector instructions.
#include "qmv_attn.h"
#include "qmv_internal.h"

namespace qmv {

namespace {

template <int HD>
struct Lds {  // one buffer, bytes
    static constexpr int kRow = HD * 2;                 // K row
    static constexpr int kV = kBK * kRow;               // V blocks
    static constexpr int kScale = kV + kBK * HD * 2;    // 8-bit: row scales of K, then of V
    static constexpr int kVmax = kScale + 2 * kBK * 4;  // largest row scale of V, one a block
    static constexpr int kMarks = kScale;               // 16-bit: a bit for every value of V, [block][column][16]
    static constexpr int kBytes(int type) { return type == kKvI8 ? kVmax + 16 : kMarks + 4 * HD * 2; }
    static constexpr int kOk(int type) { return 2 * kBytes(type); }  // per buffer: 4 flags, one a block:
                                                                     // 1: no hole, 2: marks set
    static constexpr int kTotal(int type) { return kOk(type) + 32; }
};

// K rows lie in LDS in the order of the 32x32 operand, row 8 b + 4 h + i of a
// half chunk being position 16 (b / 2) + 8 h + 4 (b % 2) + i: bits 2 and 3
// change places, both ways.
__device__ __forceinline__ int krow(int j) { return (j & ~12) | ((j & 4) << 1) | ((j & 8) >> 1); }
// LDS delivers 256 bytes a cycle, 16 bytes to each of 16 lanes, so the lanes
// of 16 neighbouring rows (columns of V) that read the same piece must find it
// in 16 different places modulo 256 bytes.  Place of piece p in K row r:
template <int HD>
__device__ __forceinline__ int kslot(int r, int p) {
    return HD == 64 ? p ^ ((r >> 1) & 7) : HD == 96 ? p ^ ((r >> 2) & 3) : p ^ (r & 15);
}
// ... and of half p of column d of a V block:
__device__ __forceinline__ int vslot(int d, int p) { return 2 * d + (p ^ ((d >> 3) & 1)); }

// A wave's 16 positions of a chunk on their way to LDS.  f16 and bf16 values
// go straight from memory to LDS (each lane names the piece whose place its
// slot of the wave's run of 1 KB is), 8-bit codes are widened on the way.
template <int TYPE, int HD>
struct Stage {
    static constexpr int SZ = TYPE == kKvI8 ? 1 : 2;
    static constexpr int PIECES = HD * SZ;  // 16-byte pieces of 16 K rows, and of a V block
    static constexpr int N = (PIECES + 63) / 64;
    u32x4 k[TYPE == kKvI8 ? N : 1], v[TYPE == kKvI8 ? N : 1];
    float sc;
    bool ok;

    __device__ __forceinline__ void load(const KvArgs &c, int h, int page, int pos, uint8_t *buf, int w, int lane) {
        ok = page >= 0;
        const uint8_t *base = kv_head(c, page < 0 ? 0 : page, h);
        const int slot = pos & ((1 << c.page_shift) - 1);
        const uint8_t *kp = base + (int64_t)slot * (HD * SZ);
        const uint8_t *vp = base + ((int64_t)(HD * SZ) << c.page_shift) + (int64_t)slot * (HD * SZ);
        if constexpr (TYPE == kKvI8) {
#pragma unroll
            for (int i = 0; i < N; i++) {
                if (PIECES % 64 == 0 || lane + 64 * i < PIECES) {
                    k[i] = *reinterpret_cast<const u32x4 *>(kp + (lane + 64 * i) * 16);
                    v[i] = *reinterpret_cast<const u32x4 *>(vp + (lane + 64 * i) * 16);
                }
            }
            const float *s = reinterpret_cast<const float *>(base + ((int64_t)(2 * HD) << c.page_shift));
            sc = lane < 32 ? s[((lane >> 4) << c.page_shift) + slot + (lane & 15)] : 0.f;
        } else {
            constexpr int PPR = HD / 8;  // pieces of a row
            uint8_t *kd = buf + 16 * w * Lds<HD>::kRow, *vd = buf + Lds<HD>::kV + w * HD * 32;
#pragma unroll
            for (int i = 0; i < N; i++) {
                const int q = lane + 64 * i, row = q / PPR;
                const int from = krow(row) * (HD * 2) + kslot<HD>(row, q % PPR) * 16;
                to_lds(kp + from, kd + i * 1024);
                to_lds(vp + vslot(q / 2, q % 2) * 16, vd + i * 1024);
            }
        }
    }
    // live: positions of the 16 that some row may see, but for those from h0 to
    // before h1; 8-bit: scales of the others, which may be anything, are left
    // out.  whole: every row sees every position; where not, V values that are
    // not finite leave marks and zeros.
    __device__ __forceinline__ void store(uint8_t *buf, uint8_t *flag, int w, int lane, int live, int h0, int h1, bool whole) const {
        if (!ok) live = 0;
        bool marked = false;
        if constexpr (TYPE == kKvI8) {
#pragma unroll
            for (int i = 0; i < N; i++) {
                const int p = lane + 64 * i;
                if (PIECES % 64 != 0 && p >= PIECES) continue;
                const int pos = (p * 16) / HD, at = (p * 16) % HD / 8;  // K: position, piece in LDS
                const int row = 16 * w + krow(pos);
                uint8_t *kd = buf + row * Lds<HD>::kRow;
                const uint2 a = codes_to_f16(k[i].x), b = codes_to_f16(k[i].y), c2 = codes_to_f16(k[i].z), d = codes_to_f16(k[i].w);
                *reinterpret_cast<u32x4 *>(kd + kslot<HD>(row, at) * 16) = u32x4{a.x, a.y, b.x, b.y};
                *reinterpret_cast<u32x4 *>(kd + kslot<HD>(row, at + 1) * 16) = u32x4{c2.x, c2.y, d.x, d.y};
                const uint2 e = codes_to_f16(v[i].x), f = codes_to_f16(v[i].y), g = codes_to_f16(v[i].z), o = codes_to_f16(v[i].w);
                uint8_t *vd = buf + Lds<HD>::kV + w * HD * 32;  // a piece is one column
                *reinterpret_cast<u32x4 *>(vd + vslot(p, 0) * 16) = u32x4{e.x, e.y, f.x, f.y};
                *reinterpret_cast<u32x4 *>(vd + vslot(p, 1) * 16) = u32x4{g.x, g.y, o.x, o.y};
            }
            const int at = lane & 15;
            const float mine = at < live && (at < h0 || at >= h1) ? sc : 0.f;
            if (lane < 32) reinterpret_cast<float *>(buf + Lds<HD>::kScale)[(lane >> 4) * kBK + 16 * w + (lane & 15)] = mine;
            float big = fabsf(mine) < __builtin_inff() ? fabsf(mine) : 0.f;
            for (int off = 8; off; off >>= 1) big = fmaxf(big, __shfl_xor(big, off));
            if (lane == 16) reinterpret_cast<float *>(buf + Lds<HD>::kVmax)[w] = big;
        } else {
            __builtin_amdgcn_s_waitcnt(kWaitVm0);  // the wave's own pieces are in LDS
            if (!whole || !ok) {
                typedef typename KvOp<TYPE>::Op Op;
                uint8_t *vd = buf + Lds<HD>::kV + w * HD * 32;
                uint32_t any = 0;
#pragma unroll
                for (int i = 0; i < N; i++) {
                    const int q = lane + 64 * i, d = q / 2, half = vslot(d, q & 1) & 1;
                    U128 v = *reinterpret_cast<const U128 *>(vd + q * 16);
                    uint32_t bits = 0;
#pragma unroll
                    for (int j = 0; j < 4; j++) {
                        const uint32_t bad = not_finite<Op>(v.w[j]);
                        v.w[j] &= ~(bad * 0xFFFFu);
                        bits |= ((bad & 1) | (bad >> 15)) << (2 * j);
                    }
                    buf[Lds<HD>::kMarks + (w * HD + d) * 2 + half] = (uint8_t)bits;
                    if (bits) *reinterpret_cast<U128 *>(vd + q * 16) = v;
                    any |= bits;
                }
                marked = __any(any != 0);
            }
        }
        if (lane == 0) flag[w] = (ok ? 1 : 0) | (marked ? 2 : 0);
    }
    // s_waitcnt vmcnt(0), the other counters at their largest
    static constexpr int kWaitVm0 = 0x0F70;
    static __device__ __forceinline__ void to_lds(const uint8_t *from, uint8_t *to) {
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void *)from,
                                         (__attribute__((address_space(3))) void *)to, 16, 0, 0);
    }
};

template <int TYPE, int HD>
__global__ __launch_bounds__(256, HD == 256 ? 1 : HD == 64 ? 3 : 2) void attn_prefill(AttnArgs a) {
    typedef typename KvOp<TYPE>::Op Op;
    typedef typename Op::Vec Vec;
    constexpr int KS = HD / 16, DT = HD / 32, NP = Op::kPieces;
    extern __shared__ __align__(16) uint8_t lds[];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
    const int col = lane & 31, hh = lane >> 5;
    const int h = blockIdx.x, split = blockIdx.z;
    const KvArgs &c = a.c;

    // which sequence and tile: the last tiles, which see the most, first
    int slot = gridDim.y - 1 - blockIdx.y;
    int s, tile;
    int64_t row0, n;
    if (!a.start) {
        n = a.n;
        const int per = (int)((n * a.group + kBM - 1) / kBM);
        s = slot / per;
        tile = slot % per;
        row0 = (int64_t)s * n;
    } else {
        s = -1;
        for (int base = 0; base < c.n_seq; base += 64) {
            int64_t cnt = 0;
            if (base + lane < c.n_seq) {
                const int64_t len = (int64_t)a.start[base + lane + 1] - a.start[base + lane];
                cnt = len > 0 ? (len * a.group + kBM - 1) / kBM : 0;
            }
            int64_t upto = cnt;
            for (int off = 1; off < 64; off <<= 1) {
                const int64_t x = __shfl_up(upto, off);
                if (lane >= off) upto += x;
            }
            const int64_t all = __shfl(upto, 63);
            if (slot < all) {
                const int who = __builtin_ctzll(__ballot(upto > slot));
                s = base + who;
                tile = slot - (int)__shfl(upto - cnt, who);
                break;
            }
            slot -= (int)all;
        }
        if (s < 0) return;
        s = __builtin_amdgcn_readfirstlane(s);
        tile = __builtin_amdgcn_readfirstlane(tile);
        row0 = a.start[s];
        n = (int64_t)a.start[s + 1] - row0;
    }
    const int64_t nrows = n * a.group;
    const int64_t r0 = (int64_t)tile * kBM;

    // This wave's rows.  The queries do not wait for lengths and pages, and
    // loads return in order: issued first, they are split while the first
    // chunk is on its way (97 tokens 8.1 -> 7.3 us).
    const int64_t rr = r0 + 32 * wave + col;
    const int64_t tok = rr / a.group;
    const int hg = (int)(rr % a.group);
    const int64_t row = row0 + tok;
    const bool live = rr < nrows && row >= 0 && row < a.rows;
    float f[KS][8];
    {
        const float *qp = a.q + (live ? row : 0) * a.ldq + (int64_t)(h * a.group + (live ? hg : 0)) * HD + 8 * hh;
#pragma unroll
        for (int t = 0; t < KS; t++) {
            const uint8_t *src = reinterpret_cast<const uint8_t *>(qp + 16 * t);
            const float4 x = __builtin_bit_cast(float4, load16(src)), y = __builtin_bit_cast(float4, load16(src + 16));
            f[t][0] = x.x, f[t][1] = x.y, f[t][2] = x.z, f[t][3] = x.w;
            f[t][4] = y.x, f[t][5] = y.y, f[t][6] = y.z, f[t][7] = y.w;
        }
    }
    const int len = kv_len(c, s, a.limit);

    // what the tile's and this wave's rows see
    auto pos_of = [&](int64_t r) {
        const int64_t p = (int64_t)len - n + (r < nrows ? r : nrows - 1) / a.group;
        return p < -1 ? -1 : (int)p;
    };
    const int pmin = pos_of(r0), pmax = pos_of(r0 + kBM - 1);
    const bool wave_live = r0 + 32 * wave < nrows;
    const int wmin = pos_of(r0 + 32 * wave), wmax = wave_live ? pos_of(r0 + 32 * wave + 31) : -1;
    const Chunks ch = visible_chunks(pmin, pmax, a.window, a.sinks, kBK);
    const int begin = (int)((int64_t)ch.n * split / a.splits), end = (int)((int64_t)ch.n * (split + 1) / a.splits);

    const int last_page = len > 0 ? (len - 1) >> c.page_shift : 0;
    auto page_of = [&](int i) {  // page of this wave's 16 positions of chunk number i
        if (i >= end) return -1;
        const int pi = (ch.at(i) * kBK + 16 * wave) >> c.page_shift;
        if (pi > last_page) return -1;
        const int pg = c.table[(int64_t)s * c.table_ld + pi];
        return (uint32_t)pg < (uint32_t)c.n_pages ? pg : -1;
    };
    auto live_of = [&](int i) {  // how many of its 16 positions are not behind what any row sees
        const int left = pmax + 1 - (ch.at(i) * kBK + 16 * wave);
        return left > 16 ? 16 : left < 0 ? 0 : left;
    };
    // of these, behind the sinks and before every row's window: from .. to before
    const int hid0 = a.sinks, hid1 = a.window > 0 ? pmin - a.window + 1 : 0;
    auto whole_of = [&](int i) {  // whether every row of the tile sees all of it
        const int c0 = ch.at(i) * kBK, c1 = c0 + kBK - 1;
        return c1 <= pmin && (a.window <= 0 || c0 > pmax - a.window || c1 < a.sinks);
    };
    // the first chunk is on its way while the queries are split
    Stage<TYPE, HD> st;
    int page = __builtin_amdgcn_readfirstlane(page_of(begin));
    auto buf_of = [&](int i) { return lds + (i & 1) * Lds<HD>::kBytes(TYPE); };
    auto ok_of = [&](int i) { return lds + Lds<HD>::kOk(TYPE) + (i & 1) * 4; };
    st.load(c, h, page, begin < end ? ch.at(begin) * kBK + 16 * wave : 0, buf_of(begin), wave, lane);

    const int64_t pos64 = (int64_t)len - n + tok;
    const int pos = live && pos64 >= 0 ? (int)pos64 : -1;
    // first position in the row's window; the sinks before it stay visible
    const int wlo = a.window > 0 ? pos - a.window + 1 : -1;
    U128 qf[KS][NP];
    float qscale;
    {
        float big = 0.f;
        int sh = 0;
        if constexpr (TYPE != kKvBF16) {
#pragma unroll
            for (int t = 0; t < KS; t++)
#pragma unroll
                for (int e = 0; e < 8; e++) big = fmaxf(big, fabsf(f[t][e]));
            big = fmaxf(big, __shfl_xor(big, 32));
            if (big > 0.f && big < __builtin_inff()) {
                sh = 15 - __builtin_amdgcn_frexp_expf(big);
                sh = sh > 100 ? 100 : sh;
            }
        }
        qscale = logit_factor(a.scale_log2, sh);
#pragma unroll
        for (int t = 0; t < KS; t++) {
#pragma unroll
            for (int e = 0; e < 8; e++) f[t][e] = live ? ldexpf(f[t][e] * a.q_sign, sh) : 0.f;
            split8<Op>(f[t], qf[t]);
        }
    }
    float mrun = kNoMax, lrun = 0.f;
    bool far = false;  // some row's maximum is
    float vmul = kVmulNone, vlog = TYPE == kKvI8 ? kVlogNone : 0.f, vback = 1.f / kVmulNone;  // as in the decode kernel
    f32x16 o[DT];
#pragma unroll
    for (int t = 0; t < DT; t++)
#pragma unroll
        for (int e = 0; e < 16; e++) o[t][e] = 0.f;

    page = __builtin_amdgcn_readfirstlane(page_of(begin + 1));
    if (begin < end) st.store(buf_of(begin), ok_of(begin), wave, lane, live_of(begin), hid0 - ch.at(begin) * kBK - 16 * wave,
                               hid1 - ch.at(begin) * kBK - 16 * wave, whole_of(begin));
    for (int i = begin; i < end; i++) {
        const uint8_t *buf = buf_of(i);
        const bool more = i + 1 < end;
        __syncthreads();  // buffer i is written; everyone is done with buffer i - 1
        if (more) st.load(c, h, page, ch.at(i + 1) * kBK + 16 * wave, buf_of(i + 1), wave, lane);
        const int next_page = page_of(i + 2);
        const uint32_t okf = *reinterpret_cast<const uint32_t *>(ok_of(i));
        const float *ksc = reinterpret_cast<const float *>(buf + Lds<HD>::kScale);
        const float *vsc = ksc + kBK;
#pragma unroll
        for (int half = 0; half < 2; half++) {
            const int c0 = ch.at(i) * kBK + 32 * half, c1 = c0 + 31;
            // nothing for this wave's rows here?
            if (c0 > wmax || (a.window > 0 && c1 <= wmin - a.window && c0 >= a.sinks)) continue;
            const uint32_t ok2 = __builtin_amdgcn_readfirstlane((okf >> (16 * half)) & 0x0101u);
            const bool whole = c1 <= wmin && (a.window <= 0 || c0 > wmax - a.window || c1 < a.sinks) && ok2 == 0x0101u;
            if constexpr (TYPE != kKvI8) {
                const uint32_t marked = __builtin_amdgcn_readfirstlane((okf >> (16 * half)) & 0x0202u);
                if (marked) {
                    U128 seen[2];
#pragma unroll
                    for (int u = 0; u < 2; u++)
                        seen[u] = seen8((ok2 >> (8 * u)) & 1, pos, c0 + 16 * u + 8 * hh, a.window, a.sinks);
#pragma unroll
                    for (int t = 0; t < DT; t++) {
#pragma unroll
                        for (int u = 0; u < 2; u++) {
                            if (!((marked >> (8 * u)) & 2)) continue;
                            const uint32_t bits = buf[Lds<HD>::kMarks + ((2 * half + u) * HD + 32 * t + col) * 2 + hh];
                            U128 marks;
#pragma unroll
                            for (int j = 0; j < 4; j++)
                                marks.w[j] = ((bits >> (2 * j)) & 1) * kHuge | ((bits >> (2 * j + 1)) & 1) * (kHuge << 16);
                            o[t] = OpBF16::mfma32(as_vec<bf16x8>(marks), as_vec<bf16x8>(seen[u]), o[t]);
                        }
                    }
                }
            }
            f32x16 sa;
#pragma unroll
            for (int e = 0; e < 16; e++) sa[e] = 0.f;
            const uint8_t *kp = buf + (32 * half + col) * Lds<HD>::kRow;
            Vec kx[KS];
#pragma unroll
            for (int t = 0; t < KS; t++) kx[t] = *reinterpret_cast<const Vec *>(kp + kslot<HD>(col, 2 * t + hh) * 16);
#pragma unroll
            for (int t = 0; t < KS; t++)
#pragma unroll
                for (int p = 0; p < NP; p++) sa = Op::mfma32(kx[t], as_vec<Vec>(qf[t][p]), sa);
            // four K reads ahead of the products
            __builtin_amdgcn_sched_group_barrier(0x100, 4, 0);
#pragma unroll
            for (int t = 0; t < KS - 4; t++) {
                __builtin_amdgcn_sched_group_barrier(0x8, NP, 0);
                __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
            }
            __builtin_amdgcn_sched_group_barrier(0x8, 4 * NP, 0);
            // With two waves a SIMD and long products, the wave past its first
            // product goes first, so that the two fall out of step and one's
            // softmax runs beside the other's products (128 columns: 295 -> 282
            // us for 4096 tokens; 64 columns lose 1%).
            if constexpr (HD >= 128) __builtin_amdgcn_s_setprio(1);
            // V's operands fly during the softmax where there are registers for them
            constexpr int EARLY = HD == 256 ? 0 : TYPE == kKvF16 ? 2 : HD == 64 && TYPE == kKvBF16 ? 1 : 0;
            Vec vx[2][DT];
            const uint8_t *vp = buf + Lds<HD>::kV + 2 * half * HD * 32 + vslot(col, hh) * 16;
            auto read_v = [&](int u) {
#pragma unroll
                for (int t = 0; t < DT; t++) vx[u][t] = *reinterpret_cast<const Vec *>(vp + u * HD * 32 + t * 32 * 32);
            };
            if constexpr (EARLY > 0) read_v(0);
            if constexpr (EARLY > 1) read_v(1);
            float x[16];
            float mx = -__builtin_inff();
            f32x4 vs[4];
#pragma unroll
            for (int e = 0; e < 16; e++) x[e] = sa[e];
            if constexpr (TYPE == kKvI8) {
#pragma unroll
                for (int u = 0; u < 4; u++) {
                    const int at = 32 * half + 16 * (u >> 1) + 8 * hh + 4 * (u & 1);
                    const f32x4 ks = *reinterpret_cast<const f32x4 *>(ksc + at);
                    vs[u] = *reinterpret_cast<const f32x4 *>(vsc + at);
#pragma unroll
                    for (int e = 0; e < 4; e++) {
                        x[4 * u + e] *= ks[e];
                    }
                }
            }
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 16; e++) {
                    const int key = c0 + 16 * (e >> 3) + 8 * hh + (e & 7);
                    const int top = (ok2 >> (8 * (e >> 3))) & 1 ? pos : -1;  // a hole: nothing
                    const bool in = (key <= top) & ((key >= wlo) | (key < a.sinks));
                    x[e] = in ? x[e] : -__builtin_inff();
                    if constexpr (TYPE == kKvI8) vs[e >> 2][e & 3] = in ? vs[e >> 2][e & 3] : 0.f;  // it may be NaN
                }
            }
#pragma unroll
            for (int e = 0; e < 16; e++) mx = fmaxf(mx, x[e]);
            mx *= qscale;
            if (__any(above_max(mx, mrun))) {
                mx = fmaxf(mx, __shfl_xor(mx, 32));
                const float mnew = fmaxf(mrun, mx);
                const float r = exp2_fast(mrun - mnew);
                mrun = mnew;
                far = far || __any(is_far(mnew));
                lrun *= r;
#pragma unroll
                for (int t = 0; t < DT; t++) o[t] *= r;
            }
            float mbase = mrun;
            // (bf16 of 128 columns gains from the branch laid out of the way, 4096
            // tokens 329 -> 321 us; others would keep a register in scratch for it)
            if (TYPE == kKvBF16 && HD == 128 ? __builtin_expect(far, 0) : far) {
                mbase = 0.f;
                const float back = 1.f / qscale;
#pragma unroll
                for (int e = 0; e < 16; e++) x[e] = past_max(x[e], qscale, mrun) * back;
            }
            if constexpr (TYPE == kKvI8) {
                const f32x4 vm = *reinterpret_cast<const f32x4 *>(buf + Lds<HD>::kVmax);
                const float vbig = fmaxf(fmaxf(vm[0], vm[1]), fmaxf(vm[2], vm[3]));  // the chunk's
                if (vbig * vmul > 1.f) {
                    int ex = __builtin_amdgcn_frexp_expf(vbig);
                    ex = ex > 120 ? 120 : ex;
                    const float nm = ldexpf(1.f, -ex);
                    const float r = nm / vmul;
                    vmul = nm;
                    vlog = (float)-ex;
                    vback = ldexpf(1.f, ex);
#pragma unroll
                    for (int t = 0; t < DT; t++) o[t] *= r;
                }
            }
            const float off = bias_of<TYPE>(a) - mbase + vlog;
            float sum = 0.f;
#pragma unroll
            for (int e = 0; e < 16; e++) {
                x[e] = exp2_fast(fmaf(x[e], qscale, off));
                sum += x[e];
                if constexpr (TYPE == kKvI8) x[e] *= vs[e >> 2][e & 3];
            }
            lrun += TYPE == kKvI8 ? sum * vback : sum;
            U128 pf[2][NP];
            split8<Op>(x, pf[0]);
            split8<Op>(x + 8, pf[1]);
            if constexpr (EARLY < 1) read_v(0);
            if constexpr (EARLY < 2) read_v(1);
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int t = 0; t < DT; t++)
#pragma unroll
                    for (int p = 0; p < NP; p++) o[t] = Op::mfma32(vx[u][t], as_vec<Vec>(pf[u][p]), o[t]);
            if constexpr (HD >= 128) __builtin_amdgcn_s_setprio(0);
        }
        page = __builtin_amdgcn_readfirstlane(next_page);
        if (more) st.store(buf_of(i + 1), ok_of(i + 1), wave, lane, live_of(i + 1), hid0 - ch.at(i + 1) * kBK - 16 * wave,
                          hid1 - ch.at(i + 1) * kBK - 16 * wave, whole_of(i + 1));
    }

    lrun += __shfl_xor(lrun, 32);
    if (!live) return;
    const int64_t orow = row * a.n_heads + h * a.group + hg;
    float mul = 1.f;
    if constexpr (TYPE == kKvI8) {
        lrun *= a.unit;
        const float back = vback * a.unit;
#pragma unroll
        for (int t = 0; t < DT; t++) o[t] *= back;
    }
    float *dst;
    if (a.splits == 1) {
        mul = lrun == 0.f ? 0.f : 1.f / lrun;  // a row that sees nothing: zeros
        dst = a.out + orow * HD;
    } else {
        const int64_t at = (int64_t)split * a.part_rows + orow;
        if (hh == 0) a.part_ml[at] = make_float2(mrun, lrun);
        dst = a.part_o + at * HD;
    }
#pragma unroll
    for (int t = 0; t < DT; t++) {
#pragma unroll
        for (int b = 0; b < 4; b++) {
            const f32x4 v = f32x4{o[t][4 * b], o[t][4 * b + 1], o[t][4 * b + 2], o[t][4 * b + 3]} * mul;
            __builtin_memcpy(dst + 32 * t + 8 * b + 4 * hh, &v, 16);
        }
    }
}

template <int HD>
__global__ __launch_bounds__(256) void attn_join(AttnArgs a) {
    const int64_t prow = blockIdx.x;
    if (a.start) {  // rows of no sequence stay as they were
        const int64_t row = prow / a.n_heads;
        if (row < a.start[0] || row >= a.start[a.c.n_seq]) return;
    }
    join_row<HD>(a, prow, prow, a.part_rows, a.splits);
}

template <int TYPE, int HD>
hipError_t launch_typed(const AttnArgs &a, int64_t slots, hipStream_t s) {
    const void *fn = (const void *)attn_prefill<TYPE, HD>;
    hipError_t e = ensure_lds(fn, Lds<HD>::kTotal(TYPE));
    if (e != hipSuccess) return e;
    const dim3 grid(a.c.n_kv, (uint32_t)slots, a.splits);
    e = launch_main(attn_prefill<TYPE, HD>, grid, dim3(256), Lds<HD>::kTotal(TYPE), s, a);
    if (e != hipSuccess || a.splits == 1) return e;
    return launch_aux(attn_join<HD>, dim3((uint32_t)a.part_rows), dim3(256), 0, s, a);
}

template <int TYPE>
hipError_t launch_type(const AttnArgs &a, int64_t slots, hipStream_t s) {
    switch (a.c.hd) {
    case 64: return launch_typed<TYPE, 64>(a, slots, s);
    case 96: return launch_typed<TYPE, 96>(a, slots, s);
    case 128: return launch_typed<TYPE, 128>(a, slots, s);
    case 256: return launch_typed<TYPE, 256>(a, slots, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace

hipError_t launch_attn_prefill(int type, const AttnArgs &a, const AttnPlan &p, hipStream_t s) {
    const int64_t slots = a.start ? p.tiles : a.c.n_seq * ((a.n * a.group + kBM - 1) / kBM);
    switch (type) {
    case kKvF16: return launch_type<kKvF16>(a, slots, s);
    case kKvBF16: return launch_type<kKvBF16>(a, slots, s);
    case kKvI8: return launch_type<kKvI8>(a, slots, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmv
