// Plans of the attention calls: pieces, tiles and workspaces.
#include "qmv_attn_plan.h"

namespace qmv {

namespace {

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

}  // namespace

AttnPlan attn_decode_plan(int type, int hd, int64_t n_seq, int n_kv, int group, int n,
                          int64_t max_len, int window, int sinks, bool with_acc) {
    AttnPlan p{};
    const int64_t rows = (int64_t)n * group;
    p.rt = rows > 16 && hd <= 128 ? 2 : 1;
    p.tiles = (int)((rows + 16 * p.rt - 1) / (16 * p.rt));
    p.part_rows = n_seq * n_kv * rows;
    // the most positions a tile reads, in chunks
    const int ck = decode_chunk(type);
    int64_t most = max_len;
    if (window > 0) {
        const int64_t w = (int64_t)window + n + sinks + 2 * ck;
        if (w < most) most = w;
    }
    const int64_t chunks = (most + ck - 1) / ck;
    // Workgroups for 256 compute units: about as many as fit at once, because a
    // second round of them waits for its lengths, table and first rows again (16
    // sequences of 8192 positions of 256 columns: one workgroup a unit 104 us,
    // two 110; 32 of 6144 of 64 columns: three 76 us, two 79, four 90).  Every
    // sequence is cut into the same whole number of pieces, the next above, which
    // for three or five to seven sequences is up to a tenth more than fit.  Tiles
    // of 32 rows take one workgroup, of eight waves (the drafted tokens: 24 us
    // against 26 with 512 of four and 34 with 1024) or, where registers say so,
    // of four.
    const int64_t heads = (int64_t)n_kv * p.tiles, base = n_seq * heads;
    const int64_t fit = 256 * (p.rt == 2 ? 1 : resident(type, hd));
    int64_t splits = (fit + base - 1) / base;
    if (splits > chunks / 8) splits = chunks / 8;    // at least a chunk, with four waves two, per wave
    if (splits > 128) splits = 128;
    p.splits = splits < 1 ? 1 : (int)splits;
    p.slots = (int)(n_seq * p.splits);
    // Where such a piece may be long, lengths decide: evenly cut ranges.  With
    // sequences enough for all workgroups the grid's own order balances them
    // better (512 of 768 to 1536 positions: 421 against 430 us; but 128 of 1 to
    // 2048: 122 against 108), so the more there are, the longer the longest
    // has to be.
    const int waves = p.rt == 2 && eight_fit(type, hd, 2) ? 8 : 4;
    const int64_t long_chunks = base < fit ? 5 * waves * p.splits : 8 * waves * base / fit;
    if (n_seq > 1 && n_seq <= 1024 && chunks >= long_chunks && chunks * n_seq < (1ll << 30) &&
        p.part_rows < (1ll << 24)) {
        p.parts = (int)((fit + heads - 1) / heads);
        if (p.parts > kMaxPieces) p.parts = kMaxPieces;  // one sequence may take all of them
        p.slots = (int)(p.parts + n_seq);
    }
    // a launch of few, unsplit workgroups is a chain of latencies: eight waves
    // halve the chunks in it (301 positions, 3 heads: 7.3 -> 6.6 us)
    p.waves = eight_fit(type, hd, p.rt) && (p.rt == 2 || (p.slots == n_seq && base <= 256)) ? 8 : 4;
    size_t at = 0;
    if (p.slots > n_seq || with_acc) {
        const size_t pieces = (size_t)p.slots * n * n_kv * group;
        p.ml_off = at;
        at = up256(at + sizeof(float2) * pieces);
        p.o_off = at;
        at = up256(at + sizeof(float) * pieces * hd);
        p.share_off = at;
        at = up256(at + sizeof(int2) * n_seq);
    }
    if (with_acc) {
        p.ld_logits = (max_len + ck - 1) / ck * ck;
        p.logits_off = at;
        at = up256(at + sizeof(float) * (size_t)p.part_rows * p.ld_logits);
    }
    p.bytes = at;
    return p;
}

AttnPlan attn_prefill_plan(int type, int hd, int64_t n_seq, int n_kv, int group, int64_t rows,
                           int64_t max_len, int window, int sinks) {
    AttnPlan p{};
    (void)type;
    // row tiles: at least these; with prompts of different lengths each
    // sequence may add a partly filled one
    const int64_t tiles = (rows * group + kBM - 1) / kBM;
    p.tiles = (int)(tiles + n_seq);
    p.part_rows = rows * n_kv * group;
    int64_t most = max_len;
    if (window > 0) {
        const int64_t w = (int64_t)window + kBM / group + sinks + 2 * kBK;
        if (w < most) most = w;
    }
    const int64_t chunks = (most + kBK - 1) / kBK;
    // two workgroups per compute unit (counted as if tiles ran on from sequence
    // to sequence: few rows of many sequences are cut further than that)
    const int64_t base = tiles * n_kv;
    int64_t splits = 512 / base;
    if (splits > chunks / 4) splits = chunks / 4;     // at least four chunks each
    if (splits > 64) splits = 64;
    p.splits = splits < 1 ? 1 : (int)splits;
    size_t at = 0;
    if (p.splits > 1) {
        p.ml_off = at;
        at = up256(at + sizeof(float2) * (size_t)p.splits * p.part_rows);
        p.o_off = at;
        at = up256(at + sizeof(float) * (size_t)p.splits * p.part_rows * hd);
    }
    p.bytes = at;
    return p;
}

}  // namespace qmv
