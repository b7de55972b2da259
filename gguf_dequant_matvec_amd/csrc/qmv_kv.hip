// Writing the paged key-value cache: appending new tokens' rows, and cutting
// a cache down to the positions with the largest accumulated weight.
#include "qmv_device.h"
#include "qmv_internal.h"
#include "qmv_kv.h"
#include "qmv_rope.h"

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
// rows of 8 heads of 128, bf16, 83.7 MB: 20.2 - 20.9 us (4.1 TB/s); 16 rows: 4.3 -
// 4.7 us; the 6808 with 4 bits, 63.6 MB: 21.7 us.
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

// 4-bit blocks of 32 values: d is an eighth of the value of largest size (the
// positive one of two), of the other sign, so that this value has the code -8.
// It is rounded to eight bits of significand, then to f16: products of such a
// scale and a code are f16 values, and so is 24 d for d of at most 2720, which
// the readers use.
__device__ __forceinline__ uint32_t kv_scale4(float hi, float lo, bool nan) {
    if (nan) return 0x7E00;
    const float v = (float)(__bf16)((hi >= -lo ? hi : lo) * -0.125f);
    return __builtin_bit_cast(uint16_t, (_Float16)fminf(fmaxf(v, -2720.f), 2720.f));
}
__device__ __forceinline__ uint32_t kv_clamp4(float r) { return (uint32_t)(int)(fminf(fmaxf(r, -8.f), 7.f) + 8.f); }
// Codes 0 .. 15 of eight values, four bytes a dword.  x times 1 / d is off from the
// quotient by less than 2^-19 where the code is not clamped; only where it is that
// near to a border between two codes does the division itself decide, for all
// eight (a division is ten instructions: 6808 rows of 8 heads of 128 26.6 us).
__device__ __forceinline__ void kv_codes4(const float *x, float d, uint32_t *code) {
    const float inv = d != 0.f ? 1.f / d : 0.f;
    float r[8];
    bool near = false;
#pragma unroll
    for (int j = 0; j < 8; j++) {
        const float y = x[j] * inv;
        r[j] = rintf(y);
        near |= fabsf(y - r[j]) > 0.5f - 0x1p-18f;
    }
    if (near && d != 0.f) {
#pragma unroll
        for (int j = 0; j < 8; j++) r[j] = rintf(x[j] / d);
    }
#pragma unroll
    for (int j = 0; j < 8; j++) code[j >> 2] |= kv_clamp4(r[j]) << (8 * (j & 3));
}

// Where row r goes: its sequence's position (-1: none), page (-1: nowhere) and slot.
struct Place {
    int pos, page, slot;
};
__device__ __forceinline__ Place kv_place(const KvArgs &c, int64_t r, int64_t n, const int32_t *start) {
    Place at{-1, -1, 0};
    if (r >= n) return at;
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
        const uint32_t each = (uint32_t)n / (uint32_t)c.n_seq;  // (n is at most 2^27)
        seq = (int)((uint32_t)r / each);
        first = (int64_t)seq * each;
        next = first + each;
    }
    const int64_t pos = (int64_t)c.seq_len[seq] - (next - r);
    if (r >= first && r < next && pos >= 0 && pos < c.cap) {
        at.pos = (int)pos;
        at.page = kv_page(c, seq, (int)pos);
        at.slot = (int)pos & ((1 << c.page_shift) - 1);
    }
    return at;
}

__device__ __forceinline__ void load_cols8(const float *p, float *f) {
    const float4 a = __builtin_bit_cast(float4, load16(reinterpret_cast<const uint8_t *>(p)));
    const float4 b = __builtin_bit_cast(float4, load16(reinterpret_cast<const uint8_t *>(p + 4)));
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w;
    f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
}

// With ROPE the K rows are normed and turned on the way, and workgroups past
// the key-value heads do the same to HB heads of the rows' queries.  A K row
// then goes through LDS, because its pairs are half a row apart and the cache
// wants eight neighbours.  6808 rows of 32 / 8 heads of 128, bf16, 307 MB: 65 - 67
// us (4.6 TB/s, a large copy's rate); 16 rows: 5.9 us.  With the same rows each
// time, of which a part stays in the last cache: bf16 60 us, int8 60, 4 bits 58;
// 16 rows f16 6.4, int8 7.3, 4 bits 6.4.
template <int TYPE, int HD, int ROWS, int ROPE>
__global__ __launch_bounds__(256) void kv_append(KvArgs c, RopeArgs rope, HeadRows q, int64_t n, const int32_t *start,
                                                 const float *__restrict__ k, int64_t ldk,
                                                 const float *__restrict__ v, int64_t ldv) {
    constexpr int SZ = TYPE == kKvF16 || TYPE == kKvBF16 ? 2 : 1;
    constexpr int VC = TYPE == kKvQ4 ? HD / 2 : HD;        // columns of a V block: a byte has two 4-bit codes
    constexpr int PIECES = HD / 8;                         // 8 columns a thread
    constexpr int N = (ROWS * PIECES + 255) / 256;         // pieces a thread
    constexpr int VROW = VC + (SZ == 1 ? 4 : 2);           // padded row in LDS, values
    constexpr int L = kRopeLanes<HD>, RN = (ROWS * L + 255) / 256;
    constexpr int KROW = HD + 4;
    constexpr int NB = HD / 32;                            // 4-bit blocks of a row
    typedef typename std::conditional<SZ == 1, uint8_t, uint16_t>::type Val;
    __shared__ int s_page[ROWS], s_slot[ROWS];
    __shared__ bool s_run[ROWS];  // the row's aligned group of 8 positions is here, row by row
    __shared__ __align__(16) Val s_v[ROWS * VROW];
    __shared__ float s_d[2][ROWS];
    __shared__ float s_part[TYPE == kKvI8 ? 2 : 1][TYPE == kKvI8 ? ROWS * PIECES : 1];
    __shared__ uint16_t s_d4[2][TYPE == kKvQ4 ? NB * ROWS : 1];
    __shared__ int s_pos[ROPE ? ROWS : 1];
    __shared__ __align__(16) float s_k[ROPE ? ROWS * KROW : 1];
    const int tid = threadIdx.x;
    int h = blockIdx.y;
    int64_t row0 = (int64_t)blockIdx.x * ROWS;
    if constexpr (ROPE > 1) {
        // many rows of many heads: neighbouring workgroups, which start together,
        // take neighbouring heads of the same rows (6808 rows of 32 / 8 heads of 128,
        // 307 MB: 79 -> 70 us)
        const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
        h = (int)(id % gridDim.y);
        row0 = id / gridDim.y * ROWS;
    }
    const int rows = n - row0 < ROWS ? (int)(n - row0) : ROWS;

    const RopeLane rl = rope_lane<HD>(rope, tid % L);  // (L divides 256: the same for all of a thread's rows)
    if constexpr (ROPE > 0) {
        if (h >= c.n_kv) {
            const int h0 = (h - c.n_kv) * ROPE;
            const RopeWith with = rope_with(rope, rl, tid % L, rope.q_norm);
            // (few rows: everything is asked for at once; with many, rows held while
            // positions are looked up cost more registers than that gains)
            constexpr bool EARLY = ROPE == 1;
            RopeHeads<HD, ROPE> early[EARLY ? RN : 1];
            if constexpr (EARLY) {
#pragma unroll
                for (int i = 0; i < RN; i++) {
                    const int r = (tid + 256 * i) / L;
                    early[i].load(q, rl, row0 + (r < rows ? r : 0), h0);
                }
            }
            if (tid < ROWS) s_pos[tid] = kv_place(c, row0 + tid, n, start).pos;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < RN; i++) {
                const int r = (tid + 256 * i) / L;
                if (r >= ROWS || s_pos[r] < 0) continue;
                if constexpr (!EARLY) early[0].load(q, rl, row0 + r, h0);
                early[EARLY ? i : 0].finish(rope, q, rl, with, row0 + r, s_pos[r], h0);
            }
            return;
        }
    }
    float kf[N][8], vf[N][8];
    Cols8 kx[ROPE ? RN : 1];
    RopeWith with;
    if constexpr (ROPE > 0) {
        with = rope_with(rope, rl, tid % L, rope.k_norm);
#pragma unroll
        for (int i = 0; i < RN; i++) {
            const int r = (tid + 256 * i) / L;
            kx[i] = rope_load(k + (row0 + (r < rows ? r : 0)) * ldk + (int64_t)h * HD, rl);
        }
    }
#pragma unroll
    for (int i = 0; i < N; i++) {
        const int e = tid + 256 * i, r = e / PIECES, p = e % PIECES;
        if (r < rows) {
            if constexpr (ROPE == 0) load_cols8(k + (row0 + r) * ldk + (int64_t)h * HD + p * 8, kf[i]);
            load_cols8(v + (row0 + r) * ldv + (int64_t)h * HD + p * 8, vf[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; j++) kf[i][j] = vf[i][j] = 0.f;
        }
    }
    if (tid < ROWS) {
        const Place at = kv_place(c, row0 + tid, n, start);
        s_page[tid] = at.page;
        s_slot[tid] = at.slot;
        if constexpr (ROPE > 0) s_pos[tid] = at.pos;
    }
    if constexpr (ROPE > 0) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < RN; i++) {
            const int r = (tid + 256 * i) / L;
            if (r >= ROWS) continue;
            const Cols8 y = rope_apply<HD>(rope, rl, with, rope_turn(rl, with, s_pos[r]), kx[i]);
            if (rl.live) rope_store(s_k + r * KROW, rl, y);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int e = tid + 256 * i, r = e / PIECES, p = e % PIECES;
            if (r < ROWS) load_cols8(s_k + r * KROW + p * 8, kf[i]);
        }
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
        if constexpr (TYPE == kKvQ4) {
            // a block is four neighbouring lanes' (PIECES is a multiple of 4), the
            // upper two's codes the high halves of the lower two's bytes
            auto block = [&](const float *f, uint32_t *code, int which) {
                float hi = f[0], lo = f[0];
                int nan = f[0] != f[0];
#pragma unroll
                for (int j = 1; j < 8; j++) hi = fmaxf(hi, f[j]), lo = fminf(lo, f[j]), nan |= f[j] != f[j];
#pragma unroll
                for (int off = 1; off < 4; off <<= 1) {
                    hi = fmaxf(hi, __shfl_xor(hi, off)), lo = fminf(lo, __shfl_xor(lo, off));
                    nan |= __shfl_xor(nan, off);
                }
                const uint32_t d = kv_scale4(hi, lo, nan != 0);
                const float df = half_bits_to_float(d);
                kv_codes4(f, df, code);
#pragma unroll
                for (int j = 0; j < 2; j++) code[j] |= (uint32_t)__shfl_xor((int)code[j], 2) << 4;
                if (p % 4 == 0) s_d4[which][(p / 4) * ROWS + r] = (uint16_t)d;
            };
            block(kf[i], w, 0);
            block(vf[i], x, 1);
            if (p % 4 >= 2) continue;
            const int byte = p / 4 * 16 + p % 4 * 8;
            uint32_t *sv = reinterpret_cast<uint32_t *>(s_v + r * VROW + byte);
            sv[0] = x[0], sv[1] = x[1];
            if (page < 0) continue;
            *reinterpret_cast<uint2 *>(kv_head(c, page, h) + (int64_t)s_slot[r] * VC + byte) = make_uint2(w[0], w[1]);
        } else {
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
    if constexpr (TYPE == kKvQ4) {
        for (int e = tid; e < 2 * NB * ROWS; e += 256) {
            const int r = e % ROWS, b = e / ROWS % NB, which = e / (ROWS * NB);
            if (s_page[r] < 0) continue;
            uint16_t *sc = reinterpret_cast<uint16_t *>(kv_head(c, s_page[r], h) + page_size * HD);
            const int64_t at = which ? (page_size * NB + b * page_size + s_slot[r]) : ((int64_t)s_slot[r] * NB + b);
            sc[at] = s_d4[which][b * ROWS + r];
        }
    }
    // V: lanes run over columns; a whole group leaves with its first row
    for (int e = tid; e < ROWS * VC; e += 256) {
        const int r = e / VC, d = e % VC;
        const int page = s_page[r], slot = s_slot[r];
        if (page < 0) continue;
        const int in16 = TYPE == kKvQ4 ? kv_place4(slot % kVBlock) : slot % kVBlock;
        uint8_t *dst = kv_head(c, page, h) + page_size * VC * SZ +
                       ((int64_t)(slot / kVBlock) * (VC * kVBlock) + d * kVBlock + in16) * SZ;
        if (!s_run[r]) {
            *reinterpret_cast<Val *>(dst) = s_v[r * VROW + d];
        } else if ((slot & 7) == 0) {
            uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 8; j++) {
                const uint32_t b = s_v[(r + (TYPE == kKvQ4 ? kv_place4(j) : j)) * VROW + d];
                w[j / (4 / SZ)] |= b << (8 * SZ * (j % (4 / SZ)));
            }
            if constexpr (SZ == 1)
                *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
            else
                *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}

// ---- reading back ---------------------------------------------------------------
// A workgroup takes 32 consecutive rows of one key-value head, four columns a
// thread at a time.  K goes out as it comes.  V's lanes run over the rows first
// (16 positions of a column are neighbours in a block) and go through LDS.  6808
// rows of 8 heads of 128, 4 bits, 63.6 MB: 13.0 us (4.9 TB/s); f16 and bf16, 83.7
// MB, 15 us, int8 13.6 (the same rows each time); 16 rows 4.6 - 4.8 us.
constexpr int kReadRows = 32;

template <int TYPE>
__device__ __forceinline__ float kv_value(const uint8_t *p, int64_t i) {
    if constexpr (TYPE == kKvF16) return (float)reinterpret_cast<const _Float16 *>(p)[i];
    if constexpr (TYPE == kKvBF16) return (float)reinterpret_cast<const __bf16 *>(p)[i];
    return (float)reinterpret_cast<const int8_t *>(p)[i];
}

template <int TYPE, int HD>
__global__ __launch_bounds__(256) void kv_read(KvArgs c, int64_t n, const int32_t *start, float *__restrict__ k,
                                               int64_t ldk, float *__restrict__ v, int64_t ldv) {
    constexpr int SZ = TYPE == kKvF16 || TYPE == kKvBF16 ? 2 : 1;
    constexpr int VC = TYPE == kKvQ4 ? HD / 2 : HD, NB = HD / 32;
    constexpr int VN = kReadRows * VC / 256, N4 = kReadRows * HD / 4 / 256;  // V values (bytes) and pieces a thread
    constexpr int VROW = HD + 4;
    __shared__ int s_pos[kReadRows], s_page[kReadRows], s_slot[kReadRows];
    __shared__ __align__(16) float s_v[kReadRows * VROW];
    const int tid = threadIdx.x, h = blockIdx.y;
    const int64_t row0 = (int64_t)blockIdx.x * kReadRows, page_size = 1ll << c.page_shift;
    if (tid < kReadRows) {
        const Place at = kv_place(c, row0 + tid, n, start);
        s_pos[tid] = at.pos, s_page[tid] = at.page, s_slot[tid] = at.slot;
    }
    __syncthreads();
    // (slots of rows without a page are read from page 0, and not used)
    const int rv = tid % kReadRows, v_page = s_page[rv], v_slot = s_slot[rv];
    const uint8_t *v_head = kv_head(c, v_page < 0 ? 0 : v_page, h);
    const int in16 = TYPE == kKvQ4 ? kv_place4(v_slot % kVBlock) : v_slot % kVBlock;
    const uint8_t *v_codes = v_head + page_size * VC * SZ + ((int64_t)(v_slot / kVBlock) * (VC * kVBlock) + in16) * SZ;
    float vx[VN];
    uint32_t vb[TYPE == kKvQ4 ? VN : 1];
    uint16_t vd[TYPE == kKvQ4 ? VN : 1];
#pragma unroll
    for (int i = 0; i < VN; i++) {
        const int d = tid / kReadRows + 256 / kReadRows * i;
        if constexpr (TYPE == kKvQ4) {
            vb[i] = v_codes[d * kVBlock];
            vd[i] = reinterpret_cast<const uint16_t *>(v_head + page_size * HD)[page_size * NB + d / 16 * page_size + v_slot];
        } else {
            vx[i] = kv_value<TYPE>(v_codes, d * kVBlock);
        }
    }
    float v_scale = 1.f;
    if constexpr (TYPE == kKvI8) v_scale = reinterpret_cast<const float *>(v_head + 2 * page_size * HD)[page_size + v_slot];
#pragma unroll
    for (int i = 0; i < N4; i++) {
        const int e = tid + 256 * i, r = e / (HD / 4), d = e % (HD / 4) * 4, page = s_page[r], slot = s_slot[r];
        if (s_pos[r] < 0) continue;
        const uint8_t *head = kv_head(c, page < 0 ? 0 : page, h);
        float x[4];
        if constexpr (TYPE == kKvQ4) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(head + (int64_t)slot * VC + 16 * (d / 32) + d % 16) >> (d % 32 / 16 * 4);
            const float f = half_bits_to_float(reinterpret_cast<const uint16_t *>(head + page_size * HD)[(int64_t)slot * NB + d / 32]);
#pragma unroll
            for (int j = 0; j < 4; j++) x[j] = f * (float)((int)(w >> (8 * j) & 15) - 8);
        } else {
            float f = 1.f;
            if constexpr (TYPE == kKvI8) f = reinterpret_cast<const float *>(head + 2 * page_size * HD)[slot];
#pragma unroll
            for (int j = 0; j < 4; j++) {
                x[j] = kv_value<TYPE>(head, (int64_t)slot * HD + d + j);
                if constexpr (TYPE == kKvI8) x[j] *= f;
            }
        }
        const float4 y = page < 0 ? make_float4(0.f, 0.f, 0.f, 0.f) : make_float4(x[0], x[1], x[2], x[3]);
        __builtin_memcpy(k + (row0 + r) * ldk + (int64_t)h * HD + d, &y, 16);
    }
#pragma unroll
    for (int i = 0; i < VN; i++) {
        const int d = tid / kReadRows + 256 / kReadRows * i;
        if constexpr (TYPE == kKvQ4) {
            const int col = 32 * (d / 16) + d % 16;
            const float f = half_bits_to_float(vd[i]);
            s_v[rv * VROW + col] = v_page < 0 ? 0.f : f * (float)((int)(vb[i] & 15) - 8);
            s_v[rv * VROW + col + 16] = v_page < 0 ? 0.f : f * (float)((int)(vb[i] >> 4) - 8);
        } else {
            s_v[rv * VROW + d] = v_page < 0 ? 0.f : TYPE == kKvI8 ? vx[i] * v_scale : vx[i];
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N4; i++) {
        const int e = tid + 256 * i, r = e / (HD / 4), d = e % (HD / 4) * 4;
        if (s_pos[r] < 0) continue;
        const float4 y = *reinterpret_cast<const float4 *>(s_v + r * VROW + d);
        __builtin_memcpy(v + (row0 + r) * ldv + (int64_t)h * HD + d, &y, 16);
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

// KIND: 2 for 16-bit values, 1 for 8-bit codes, 0 for 4-bit ones, two columns a
// byte and the positions of a block in kv_place4's order.
template <int KIND, int HEAD_DIM>
__global__ __launch_bounds__(256) void kv_evict_move(KvArgs c, EvictArgs e) {
    constexpr int SZ = KIND == 2 ? 2 : 1;
    constexpr int HD = KIND == 0 ? HEAD_DIM / 2 : HEAD_DIM;  // values (bytes) of a row
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
    auto place = [](int i) { return KIND == 0 ? kv_place4(i) : i; };
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
                const int to = i + place(x), k = s_ord[to] - g0;
                if (to < cnt && k >= 0 && k < GROUP) {
                    const Val *col = reinterpret_cast<const Val *>(s_v + (k * HD + d) * PAD);
                    out[j][x * SZ / 4] |= (uint32_t)col[place(s_src[to] % kVBlock)] << (8 * SZ * (x % (4 / SZ)));
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
                if (i + place(x) < cnt) reinterpret_cast<Val *>(dst)[x] = (Val)(out[j][x * SZ / 4] >> (8 * SZ * (x % (4 / SZ))));
        }
    }
    if constexpr (KIND == 0) {
        constexpr int NB = HEAD_DIM / 32;
        for (int j = tid; j < 2 * NB * kMove; j += 256) {
            const int i = j % kMove, b = j / kMove % NB, which = j / (kMove * NB);
            if (i >= cnt || s_dst[i / kVBlock] < 0) continue;
            auto at = [&](int page, int slot) {
                uint16_t *sc = reinterpret_cast<uint16_t *>(kv_head(c, page, h) + page_size * HEAD_DIM);
                return sc + (which ? page_size * NB + b * page_size + slot : (int64_t)slot * NB + b);
            };
            uint16_t d = 0;
            if (s_page[i] >= 0) d = *at(s_page[i], s_src[i] & pmask);
            *at(s_dst[i / kVBlock], (i0 + i) & pmask) = d;
        }
    }
    if (KIND == 1 && tid < 2 * kMove) {
        const int i = tid % kMove, which = tid / kMove;
        if (i < cnt && s_dst[i / kVBlock] >= 0) {
            float f = 0.f;
            if (s_page[i] >= 0)
                f = reinterpret_cast<const float *>(kv_head(c, s_page[i], h) + 2 * page_size * HD)[which * page_size + (s_src[i] & pmask)];
            reinterpret_cast<float *>(kv_head(c, s_dst[i / kVBlock], h) + 2 * page_size * HD)[which * page_size + ((i0 + i) & pmask)] = f;
        }
    }
}

struct AppendCall {
    int type;
    const KvArgs &c;
    const RopeArgs &rope;
    const HeadRows &q;
    int64_t n;
    const int32_t *start;
    const float *k;
    int64_t ldk;
    const float *v;
    int64_t ldv;
    hipStream_t s;
};

template <int HD, int ROWS, int ROPE>
hipError_t append_rows(const AppendCall &a) {
    const dim3 grid((uint32_t)((a.n + ROWS - 1) / ROWS), a.c.n_kv + (ROPE ? (a.q.heads + ROPE - 1) / (ROPE ? ROPE : 1) : 0));
    auto launch = [&](auto kernel) {
        return launch_main(kernel, grid, dim3(256), 0, a.s, a.c, a.rope, a.q, a.n, a.start, a.k, a.ldk, a.v, a.ldv);
    };
    switch (a.type) {
    case kKvF16: return launch(kv_append<kKvF16, HD, ROWS, ROPE>);
    case kKvBF16: return launch(kv_append<kKvBF16, HD, ROWS, ROPE>);
    case kKvQ4: return launch(kv_append<kKvQ4, HD, ROWS, ROPE>);
    default: return launch(kv_append<kKvI8, HD, ROWS, ROPE>);
    }
}

template <int HD>
hipError_t append_hd(const AppendCall &a, bool rope) {
    // 32 rows once that still gives two workgroups per compute unit (6808 rows
    // of 8 heads of 128: 20.8 us, with 16 rows 23.5, with 64 rows 23.6; 4 bits, which
    // compute longer between reading and writing, 24.2 us and with 16 rows 21.5).
    // Turned rows take 32, of two heads a lane group, by the same count.  Measured
    // beside it, 6808 rows of 32 / 8 heads: bf16 60 us and with 16 rows 56, 4 bits 57
    // and 53, int8 59 and 58.  The count leaves queries out: 6808 rows of 16 / 2 heads
    // take 16 rows of one head, 28 us, where 32 rows of two heads would take 30 (16 of
    // two, 24).
    const bool many = a.n * a.c.n_kv >= 32 * 512;
    if (rope) return many ? append_rows<HD, 32, 2>(a) : append_rows<HD, 16, 1>(a);
    return many && a.type != kKvQ4 ? append_rows<HD, 32, 0>(a) : append_rows<HD, 16, 0>(a);
}

hipError_t append_call(const AppendCall &a, bool rope) {
    switch (a.c.hd) {
    case 64: return append_hd<64>(a, rope);
    case 96: return append_hd<96>(a, rope);
    case 128: return append_hd<128>(a, rope);
    case 256: return append_hd<256>(a, rope);
    default: return hipErrorInvalidValue;
    }
}

template <int HD>
hipError_t read_hd(int type, const KvArgs &c, int64_t n, const int32_t *start, float *k, int64_t ldk, float *v,
                   int64_t ldv, hipStream_t s) {
    const dim3 grid((uint32_t)((n + kReadRows - 1) / kReadRows), c.n_kv);
    auto launch = [&](auto kernel) { return launch_main(kernel, grid, dim3(256), 0, s, c, n, start, k, ldk, v, ldv); };
    switch (type) {
    case kKvF16: return launch(kv_read<kKvF16, HD>);
    case kKvBF16: return launch(kv_read<kKvBF16, HD>);
    case kKvQ4: return launch(kv_read<kKvQ4, HD>);
    default: return launch(kv_read<kKvI8, HD>);
    }
}

template <int HD>
hipError_t move_hd(int type, const KvArgs &c, const EvictArgs &e, hipStream_t s) {
    const dim3 grid((e.keep + kMove - 1) / kMove, c.n_kv, c.n_seq);
    if (type == kKvQ4) return launch_main(kv_evict_move<0, HD>, grid, dim3(256), 0, s, c, e);
    if (type == kKvI8) return launch_main(kv_evict_move<1, HD>, grid, dim3(256), 0, s, c, e);
    return launch_main(kv_evict_move<2, HD>, grid, dim3(256), 0, s, c, e);
}

}  // namespace

hipError_t launch_kv_append(int type, const KvArgs &c, int64_t n, const int32_t *start,
                            const float *k, int64_t ldk, const float *v, int64_t ldv,
                            hipStream_t s) {
    return append_call({type, c, RopeArgs{}, HeadRows{}, n, start, k, ldk, v, ldv, s}, false);
}

hipError_t launch_kv_append_rope(int type, const KvArgs &c, const RopeArgs &r, int64_t n, const int32_t *start,
                                 const HeadRows &q, const float *k, int64_t ldk, const float *v, int64_t ldv,
                                 hipStream_t s) {
    return append_call({type, c, r, q, n, start, k, ldk, v, ldv, s}, true);
}

hipError_t launch_kv_read(int type, const KvArgs &c, int64_t n, const int32_t *start, float *k, int64_t ldk, float *v,
                          int64_t ldv, hipStream_t s) {
    switch (c.hd) {
    case 64: return read_hd<64>(type, c, n, start, k, ldk, v, ldv, s);
    case 96: return read_hd<96>(type, c, n, start, k, ldk, v, ldv, s);
    case 128: return read_hd<128>(type, c, n, start, k, ldk, v, ldv, s);
    case 256: return read_hd<256>(type, c, n, start, k, ldk, v, ldv, s);
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
