// Norms of queries and keys for each head and the rotation of the position:
// device pieces shared by the call on plain rows and the one that appends.
#pragma once

#include "qmv_device.h"
#include "qmv_kv.h"

namespace qmv {

// A rotation as the kernels take it.
struct RopeArgs {
    const float *q_norm, *k_norm;  // [hd] or null: no norm
    const double *freq;            // [rot / 2], radians a position
    float eps;
    int32_t rot;                   // columns that turn
    int32_t adjacent;              // pairs (2 i, 2 i + 1); else (i, i + rot / 2)
};

// Rows of heads, in and out.
struct HeadRows {
    const float *in;
    int64_t ld_in;
    float *out;
    int64_t ld_out;
    int32_t heads;
};

hipError_t launch_qk_norm_rope(const RopeArgs &r, int hd, int64_t n, const int32_t *pos,
                               const HeadRows &q, const HeadRows &k, hipStream_t s);
hipError_t launch_kv_append_rope(int type, const KvArgs &c, const RopeArgs &r, int64_t n,
                                 const int32_t *start, const HeadRows &q, const float *k,
                                 int64_t ldk, const float *v, int64_t ldv, hipStream_t s);

// A head's row is HD / 8 lanes' work (of kRopeLanes neighbours), eight columns
// each: four at first and four at second.  With pairs half a rotation apart
// that is both ends of four pairs, so that nothing but the norm's sum crosses
// lanes.
template <int HD>
constexpr int kRopeLanes = HD == 96 ? 16 : HD / 8;

struct RopeLane {
    int first, second;
    bool live;   // the lane has columns (96 of 128)
    bool turns;  // they turn
};
template <int HD>
__device__ __forceinline__ RopeLane rope_lane(const RopeArgs &a, int p) {
    RopeLane l;
    l.live = p < HD / 8;
    l.turns = l.live && 8 * p < a.rot;
    const bool apart = l.turns && !a.adjacent;
    l.first = !l.live ? 0 : apart ? 4 * p : 8 * p;
    l.second = apart ? l.first + a.rot / 2 : l.first + 4;
    return l;
}

// Cosine and sine of pos * freq.  The product and its whole turns are taken in
// 64 bits (at position 2^30 f32 would not know the angle at all); what is left,
// at most an eighth of a turn, goes through the two series, whose next terms
// are below 2e-9 and 1e-10.
__device__ __forceinline__ void cos_sin(int pos, double freq, float &c, float &s) {
    const double turns = (double)pos * freq * 0.15915494309189533577;  // 1 / (2 pi)
    const double part = 4. * (turns - __builtin_rint(turns));         // quarters: -2 .. 2
    const float quarter = __builtin_rintf((float)part);
    const float x = (float)(part - (double)quarter) * 1.57079632679489662f, y = x * x;
    float sn = fmaf(y, 2.7557319e-6f, -1.9841270e-4f);
    sn = fmaf(y, sn, 8.3333333e-3f);
    sn = fmaf(y, sn, -1.6666667e-1f);
    sn = fmaf(y * x, sn, x);
    float cs = fmaf(y, -2.7557319e-7f, 2.4801587e-5f);
    cs = fmaf(y, cs, -1.3888889e-3f);
    cs = fmaf(y, cs, 4.1666667e-2f);
    cs = fmaf(y, cs, -0.5f);
    cs = fmaf(y, cs, 1.f);
    const int k = (int)quarter & 3;
    c = k & 1 ? sn : cs;
    s = k & 1 ? cs : sn;
    c = k == 1 || k == 2 ? -c : c;
    s = k & 2 ? -s : s;
}

struct Cols8 {
    float4 a, b;  // columns first .. first + 3 and second .. second + 3
};
__device__ __forceinline__ Cols8 rope_load(const float *row, const RopeLane &l) {
    Cols8 x;
    x.a = __builtin_bit_cast(float4, load16(reinterpret_cast<const uint8_t *>(row + l.first)));
    x.b = __builtin_bit_cast(float4, load16(reinterpret_cast<const uint8_t *>(row + l.second)));
    return x;
}
__device__ __forceinline__ void rope_store(float *row, const RopeLane &l, const Cols8 &x) {
    __builtin_memcpy(row + l.first, &x.a, 16);
    __builtin_memcpy(row + l.second, &x.b, 16);
}

// What a lane needs besides its row: loaded before anything is waited for.
struct RopeWith {
    double freq[4];  // of its four pairs
    Cols8 norm;
    bool normed;
};
__device__ __forceinline__ RopeWith rope_with(const RopeArgs &a, const RopeLane &l, int p, const float *w) {
    RopeWith r;
#pragma unroll
    for (int j = 0; j < 4; j++) r.freq[j] = l.turns ? a.freq[4 * p + j] : 0.;
    r.normed = w != nullptr;
    if (w) r.norm = rope_load(w, l);
    return r;
}

// The four rotations of a lane at one position.
struct Turn {
    float c[4], s[4];
};
__device__ __forceinline__ Turn rope_turn(const RopeLane &l, const RopeWith &with, int pos) {
    Turn t;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        t.c[j] = 1.f, t.s[j] = 0.f;
        if (l.turns) cos_sin(pos, with.freq[j], t.c[j], t.s[j]);
    }
    return t;
}

// x normed (if it is to be) and turned.  All lanes of a row take part.
template <int HD>
__device__ __forceinline__ Cols8 rope_apply(const RopeArgs &a, const RopeLane &l, const RopeWith &with, const Turn &t, Cols8 x) {
    if (with.normed) {
        float ss = x.a.x * x.a.x;
        ss = fmaf(x.a.y, x.a.y, ss), ss = fmaf(x.a.z, x.a.z, ss), ss = fmaf(x.a.w, x.a.w, ss);
        ss = fmaf(x.b.x, x.b.x, ss), ss = fmaf(x.b.y, x.b.y, ss), ss = fmaf(x.b.z, x.b.z, ss), ss = fmaf(x.b.w, x.b.w, ss);
        if (!l.live) ss = 0.f;
#pragma unroll
        for (int off = kRopeLanes<HD> / 2; off; off >>= 1) ss += __shfl_xor(ss, off);
        const float inv = 1.f / sqrtf(ss * (1.f / HD) + a.eps);
        const Cols8 &n = with.norm;
        x.a.x *= inv * n.a.x, x.a.y *= inv * n.a.y, x.a.z *= inv * n.a.z, x.a.w *= inv * n.a.w;
        x.b.x *= inv * n.b.x, x.b.y *= inv * n.b.y, x.b.z *= inv * n.b.z, x.b.w *= inv * n.b.w;
    }
    if (!l.turns) return x;
    Cols8 y;
    if (a.adjacent) {
        y.a.x = x.a.x * t.c[0] - x.a.y * t.s[0], y.a.y = x.a.x * t.s[0] + x.a.y * t.c[0];
        y.a.z = x.a.z * t.c[1] - x.a.w * t.s[1], y.a.w = x.a.z * t.s[1] + x.a.w * t.c[1];
        y.b.x = x.b.x * t.c[2] - x.b.y * t.s[2], y.b.y = x.b.x * t.s[2] + x.b.y * t.c[2];
        y.b.z = x.b.z * t.c[3] - x.b.w * t.s[3], y.b.w = x.b.z * t.s[3] + x.b.w * t.c[3];
    } else {
        y.a.x = x.a.x * t.c[0] - x.b.x * t.s[0], y.b.x = x.a.x * t.s[0] + x.b.x * t.c[0];
        y.a.y = x.a.y * t.c[1] - x.b.y * t.s[1], y.b.y = x.a.y * t.s[1] + x.b.y * t.c[1];
        y.a.z = x.a.z * t.c[2] - x.b.z * t.s[2], y.b.z = x.a.z * t.s[2] + x.b.z * t.c[2];
        y.a.w = x.a.w * t.c[3] - x.b.w * t.s[3], y.b.w = x.a.w * t.s[3] + x.b.w * t.c[3];
    }
    return y;
}

// Heads h0 .. h0 + HB - 1 of one row, by the row's lanes: all of them are read
// first.  A lane writes only what it has read, and a norm's sum comes before the
// row is written, so rows may be turned in place.
template <int HD, int HB>
struct RopeHeads {
    Cols8 v[HB];

    __device__ __forceinline__ void load(const HeadRows &x, const RopeLane &l, int64_t row, int h0) {
        const float *in = x.in + row * x.ld_in;
#pragma unroll
        for (int i = 0; i < HB; i++) v[i] = rope_load(in + (int64_t)(h0 + i < x.heads ? h0 + i : h0) * HD, l);
    }
    __device__ __forceinline__ void finish(const RopeArgs &a, const HeadRows &x, const RopeLane &l, const RopeWith &with,
                                           int64_t row, int pos, int h0) const {
        float *out = x.out + row * x.ld_out;
        const Turn t = rope_turn(l, with, pos);
#pragma unroll
        for (int i = 0; i < HB; i++) {
            const Cols8 y = rope_apply<HD>(a, l, with, t, v[i]);
            if (h0 + i < x.heads && l.live) rope_store(out + (int64_t)(h0 + i) * HD, l, y);
        }
    }
};

}  // namespace qmv
