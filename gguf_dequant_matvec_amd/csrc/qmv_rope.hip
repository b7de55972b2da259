// Norms of queries and keys for each head and the rotation of the position, on
// plain rows.
#include "qmv_internal.h"
#include "qmv_rope.h"

namespace qmv {

namespace {

// A lane group takes HB heads of one row: their angles are the same, so cosines
// and sines are found once for HB.  The first chunks of heads are Q's, the
// others K's.  Bound by memory, every value read and written once, or for few
// rows by latency.  Means of profiled launches: 6808 rows of 32 / 8 heads of 128,
// 279 MB, 46 us, four heads a group (the same rows each time, so that a part stays
// in the last cache; a large copy, 4.7 TB/s, would take 59); 3001 rows of 32 / 8
// heads of 64, 61 MB, 13.3 us (one head, below the bound of launch_hd); 16 rows
// of 32 / 8 heads of 128, 3.6 us.
// (16 rows at least: the most rows a call may have, in workgroups of eight, would
// be more threads than a launch takes.)
template <int HD>
constexpr int kRopeRows = HD == 64 ? 32 : 16;

template <int HD, int HB>
__global__ __launch_bounds__(256) void qk_norm_rope(RopeArgs a, int64_t n, const int32_t *pos, HeadRows q, HeadRows k) {
    constexpr int L = kRopeLanes<HD>, R = 256 / L;
    const int p = threadIdx.x % L, q_chunks = (q.heads + HB - 1) / HB;
    int chunk = blockIdx.y;
    int64_t tile = blockIdx.x;
    if constexpr (HB > 1) {  // neighbouring workgroups: neighbouring heads of the same rows
        const int64_t id = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
        chunk = (int)(id % gridDim.y);
        tile = id / gridDim.y;
    }
    const bool is_q = chunk < q_chunks;
    const HeadRows &x = is_q ? q : k;
    const int h0 = (is_q ? chunk : chunk - q_chunks) * HB;
    const RopeLane l = rope_lane<HD>(a, p);
    const RopeWith with = rope_with(a, l, p, is_q ? a.q_norm : a.k_norm);
#pragma unroll
    for (int i = 0; i < kRopeRows<HD>; i += R) {
        const int64_t row = tile * kRopeRows<HD> + i + threadIdx.x / L;
        if (row >= n) continue;
        RopeHeads<HD, HB> heads;
        heads.load(x, l, row, h0);
        const int at = pos[row];
        if (at >= 0) heads.finish(a, x, l, with, row, at, h0);
    }
}

template <int HD, int HB>
hipError_t launch_heads(const RopeArgs &r, int64_t n, const int32_t *pos, const HeadRows &q, const HeadRows &k,
                        hipStream_t s) {
    constexpr int R = kRopeRows<HD>;
    const dim3 grid((uint32_t)((n + R - 1) / R), (q.heads + HB - 1) / HB + (k.heads + HB - 1) / HB);
    return launch_main(qk_norm_rope<HD, HB>, grid, dim3(256), 0, s, r, n, pos, q, k);
}

template <int HD>
hipError_t launch_hd(const RopeArgs &r, int64_t n, const int32_t *pos, const HeadRows &q, const HeadRows &k,
                     hipStream_t s) {
    if (n * (q.heads + k.heads) * kRopeLanes<HD> >= 4 * 256 * 1024) return launch_heads<HD, 4>(r, n, pos, q, k, s);
    return launch_heads<HD, 1>(r, n, pos, q, k, s);
}

}  // namespace

hipError_t launch_qk_norm_rope(const RopeArgs &r, int hd, int64_t n, const int32_t *pos, const HeadRows &q,
                               const HeadRows &k, hipStream_t s) {
    switch (hd) {
    case 64: return launch_hd<64>(r, n, pos, q, k, s);
    case 96: return launch_hd<96>(r, n, pos, q, k, s);
    case 128: return launch_hd<128>(r, n, pos, q, k, s);
    case 256: return launch_hd<256>(r, n, pos, q, k, s);
    default: return hipErrorInvalidValue;
    }
}

}  // namespace qmv
