// Device pieces shared by the decode and prefill attention kernels: operand
// types, the exact splits of f32 values into 16-bit pieces, the list of
// visible chunks of a cache.
#pragma once

#include "qmv_attn_plan.h"
#include "qmv_device.h"
#include "qmv_kv.h"

namespace qmv {

typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// Probabilities are held as 2^bias 2^(x - m), at most 2^(bias + kSlack)
// because m is moved as soon as a logit exceeds it by kSlack.  f16 pieces
// (largest 65504, smallest step 2^-24): bias kBias, so at most 2^15, resolves
// weights down to 2^-36 of the row's largest.  bf16 pieces have the exponents
// of f32 and cached values up to its largest: there the bias keeps the sum of
// all of a row's probabilities below 1, so that no sum of weighted values
// leaves f32 (AttnArgs::bias; a cache of 2^13 positions: -19).
constexpr float kNoMax = -3.4028235e38f;  // running maximum before any visible position: finite, so x - m never is inf - inf

// Prompts, which vector instructions bound: x factor - m is one fused operation
// while the logits are small.  Past kFar the roundings of m and of bias - m,
// 2^-24 of it each, would come into the exponent (beyond 2^24 they would be the
// exponent): there x is rounded as the maximum was, and the difference taken
// first.  (Decode holds the maximum of the unscaled x and takes (x - m) factor,
// an instruction more, which memory hides.)
constexpr float kFar = 1024.f;
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) > kFar && m > kNoMax; }
__device__ __forceinline__ float past_max(float x, float factor, float m) {
#pragma clang fp contract(off)
    const float t = x * factor;
    return t - m;
}
// The difference of two rounded values: never one operation with the product
// that x may come from, of which m knows the rounded value.
__device__ __forceinline__ float minus(float x, float m) {
#pragma clang fp contract(off)
    return x - m;
}
// Whether a logit is so far above the running maximum that this has to move.
__device__ __forceinline__ bool above_max(float x, float m) { return minus(x, m) > kSlack; }

// 8-bit V rows carry their scale into the probabilities; `vmul`, a power of
// two, keeps the largest scale so far at most 1.  Before the first row:
constexpr float kVmulNone = 0x1p100f, kVlogNone = 100.f;

// Matrix-core operands of a cache type.  f32 queries and probabilities are
// split into 16-bit pieces whose sum is the f32 value to 2^-22 or better (two
// f16 pieces of 11 bits, three bf16 pieces of 8), and each piece takes one
// matrix instruction; cached values are exact in the operand type (8-bit
// codes are integers up to 127).  So products are f32-exact and only the f32
// accumulation rounds.
struct OpF16 {
    typedef f16x8 Vec;
    static constexpr int kPieces = 2;
    static constexpr uint32_t kExp = 0x7C00, kExpStep = 0x0400;  // exponent bits, the lowest of them
    // to nearest even, one instruction for both: two pieces are off by at
    // most 2^-22 (truncation would leave 2^-20, all to one side)
    static __device__ __forceinline__ uint32_t pack(float a, float b) {
        const f32x2 v = {a, b};
        return __builtin_bit_cast(uint32_t, __builtin_convertvector(v, f16x2_t));
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return half_bits_to_float(w); }
    static __device__ __forceinline__ float hi(uint32_t w) { return half_bits_to_float(w >> 16); }
    static __device__ __forceinline__ f32x4 mfma16(Vec a, Vec b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(Vec a, Vec b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
    }
};
struct OpBF16 {
    typedef bf16x8 Vec;
    static constexpr int kPieces = 3;
    static constexpr uint32_t kExp = 0x7F80, kExpStep = 0x0080;
    static __device__ __forceinline__ uint32_t pack(float a, float b) {  // truncation
        return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, a), 0x07060302u);
    }
    static __device__ __forceinline__ float lo(uint32_t w) { return __builtin_bit_cast(float, w << 16); }
    static __device__ __forceinline__ float hi(uint32_t w) { return __builtin_bit_cast(float, w & 0xFFFF0000u); }
    static __device__ __forceinline__ f32x4 mfma16(Vec a, Vec b, f32x4 c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ f32x16 mfma32(Vec a, Vec b, f32x16 c) {
        return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};
template <int TYPE>
struct KvOp { typedef OpF16 Op; };
template <>
struct KvOp<kKvBF16> { typedef OpBF16 Op; };

// The factor of a row's logits, given the power of two its query was scaled
// by: positive, so that the maximum can be taken before it (and never 0, as a
// masked -inf has to stay one).
__device__ __forceinline__ float logit_factor(float scale_log2, int sh) {
    const float f = ldexpf(scale_log2, -sh);
    return f == 0.f ? 1.17549435e-38f : f;
}

// A 16-byte load; NT for data that one workgroup reads once.
template <bool NT>
__device__ __forceinline__ u32x4 load_stream(const uint8_t *p) {
    const u32x4 *q = reinterpret_cast<const u32x4 *>(p);
    if constexpr (NT) return __builtin_nontemporal_load(q);
    return *q;
}

template <int TYPE>
__device__ __forceinline__ float bias_of(const AttnArgs &a) {
    return TYPE == kKvBF16 ? a.bias : kBias;
}
// ... and of the sums that leave a wave.  8-bit ones take their factor back
// first (weighted values of row scales up to 2^100 would not stay finite
// with it).
template <int TYPE>
__device__ __forceinline__ float sum_bias_of(const AttnArgs &a) {
    return TYPE == kKvF16 ? kBias : a.bias;
}

struct U128 { uint32_t w[4]; };
template <class V>
__device__ __forceinline__ V as_vec(U128 u) { return __builtin_bit_cast(V, u); }

// f[8] as Op::kPieces operand vectors.  f is used up.
template <class Op>
__device__ __forceinline__ void split8(float *f, U128 *piece) {
#pragma unroll
    for (int p = 0; p < Op::kPieces; p++) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const uint32_t w = Op::pack(f[2 * j], f[2 * j + 1]);
            piece[p].w[j] = w;
            if (p + 1 < Op::kPieces) {
                f[2 * j] -= Op::lo(w);
                f[2 * j + 1] -= Op::hi(w);
            }
        }
    }
}

__device__ __forceinline__ bool sees(int p, int key, int window, int sinks) {
    return key <= p && (window <= 0 || key > p - window || key < sinks);
}

// A masked weight is 0, but 0 times a NaN or an infinity is NaN: where rows of
// a tile see different positions, V values that are not finite are taken out
// before the product, and the rows that do see one get an infinity in its
// column by a product of their own: kHuge, the largest bf16 value, in both
// operands overflows f32, and 0 in the other operand gives 0.
constexpr uint32_t kHuge = 0x7F7F;

// Bits 0 and 16: which of a dword's two values are not finite (all exponent
// bits set: adding the lowest of them carries into the sign bit).
template <class Op>
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
    return (((w & (Op::kExp * 0x10001u)) + Op::kExpStep * 0x10001u) & 0x80008000u) >> 15;
}
// The operand of "the row sees position key + e" for e = 0 .. 7.
__device__ __forceinline__ U128 seen8(bool there, int pos, int key, int window, int sinks) {
    U128 v;
#pragma unroll
    for (int j = 0; j < 4; j++)
        v.w[j] = (there && sees(pos, key + 2 * j, window, sinks) ? kHuge : 0u) |
                 (there && sees(pos, key + 2 * j + 1, window, sinks) ? kHuge << 16 : 0u);
    return v;
}

// Four int8 codes of a dword as two dwords of f16 pairs, exactly: 1024 + 128 +
// code is the f16 whose low byte is the code with its sign bit flipped.
__device__ __forceinline__ uint2 codes_to_f16(uint32_t v) {
    const uint32_t u = v ^ 0x80808080u;
    const f16x2_t bias = {(_Float16)1152.0f, (_Float16)1152.0f};
    const uint32_t a = __builtin_amdgcn_perm(0x64646464u, u, 0x07010700u);
    const uint32_t b = __builtin_amdgcn_perm(0x64646464u, u, 0x07030702u);
    return make_uint2(__builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, a) - bias),
                      __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, b) - bias));
}

// The chunks of `ck` positions that hold every position some query with
// pmin <= p <= pmax sees: first those of the sinks, then those of the window.
struct Chunks {
    int sink, win0, n;
    __device__ __forceinline__ int at(int i) const { return i < sink ? i : win0 + (i - sink); }
};
__device__ __forceinline__ Chunks visible_chunks(int pmin, int pmax, int window, int sinks, int ck) {
    Chunks v;
    const int end = pmax < 0 ? 0 : pmax / ck + 1;
    v.sink = 0;
    v.win0 = 0;
    if (window > 0) {
        const int lo = pmin - window + 1;  // first position in some query's window
        v.win0 = lo > 0 ? lo / ck : 0;
        const int sc = sinks > pmax ? end : (sinks + ck - 1) / ck;
        v.sink = sc < v.win0 ? sc : v.win0;
        if (v.sink > end) v.sink = end;
    }
    v.n = v.sink + (end > v.win0 ? end - v.win0 : 0);
    return v;
}

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Joins the `count` pieces of output row prow, which are at `first`, first +
// stride, ...: o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
// One workgroup of 256 threads a row.  The pieces' factors go to LDS first; then HD / 4 lanes
// read a piece (16 bytes each), 256 / (HD / 4) pieces at a time and four such
// rounds in flight.  Bound by latency: 64 pieces of 128 columns, eight loads a
// thread, 4.5 us.
template <int HD>
__device__ __forceinline__ void join_row(const AttnArgs &a, int64_t prow, int64_t first, int64_t stride, int count) {
    constexpr int L = HD / 4, G = 256 / L;
    const int tid = threadIdx.x, lane = tid & 63;
    __shared__ float s_r[kMaxPieces];
    __shared__ f32x4 s_o[G][L];
    // every wave finds the maximum and the sum for itself
    float2 ml[kMaxPieces / 64];
    float mm = kNoMax;
#pragma unroll
    for (int k = 0; k < kMaxPieces / 64; k++) {
        ml[k] = make_float2(kNoMax, 0.f);
        if (64 * k < count && lane + 64 * k < count) ml[k] = a.part_ml[first + (lane + 64 * k) * stride];
        mm = fmaxf(mm, ml[k].x);
    }
    for (int off = 32; off; off >>= 1) mm = fmaxf(mm, __shfl_xor(mm, off));
    float l = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxPieces / 64; k++) {
        const float r = exp2_fast(ml[k].x - mm);
        l += r * ml[k].y;
        if (tid < 64 && lane + 64 * k < count) s_r[lane + 64 * k] = r;
    }
    for (int off = 32; off; off >>= 1) l += __shfl_xor(l, off);
    __syncthreads();
    const int g = tid / L, d = tid % L;
    if (g < G) {
        const f32x4 *src = reinterpret_cast<const f32x4 *>(a.part_o) + first * L + d;
        f32x4 o = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
        for (int i = g; i < count; i += G) o += src[i * stride * L] * s_r[i];
        s_o[g][d] = o;
    }
    __syncthreads();
    if (tid >= L) return;
    f32x4 o = s_o[0][tid];
    for (int k = 1; k < G; k++) o += s_o[k][tid];
    const f32x4 v = o * (l == 0.f ? 0.f : 1.f / l);
    __builtin_memcpy(a.out + prow * HD + 4 * tid, &v, 16);
}

}  // namespace qmv
